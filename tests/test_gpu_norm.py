"""Block norms against their definitions in 64 bits: types, row strides, odd and unaligned rows, gates, both
directions."""
import itertools

import pytest
import torch

import block_ref as br

import vector_quantized_moe_b200 as vq

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
EPS = 1e-6


def rows(T, H, dtype, seed, pad=0, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    t = (torch.randn((T, H + pad), generator=g) * scale).to(dtype).cuda()
    return t[:, pad // 2:pad // 2 + H]


def weight(H, dtype, seed, offset):
    g = torch.Generator().manual_seed(seed)
    return (1.0 - offset + 0.3 * torch.randn(H, generator=g)).to(dtype).cuda()


SHAPES = [(1, 1), (3, 7), (5, 64), (1, 257), (4, 256), (9, 264), (2, 1000), (1, 4096), (3, 4097), (2, 6144), (2, 8200),
          (1, 16384), (2, 16383), (700, 96), (601, 40)]


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("ht,wt,offset,pad", [(BF16, BF16, 0.0, 0), (F32, F32, 1.0, 8), (BF16, F32, 1.0, 3)])
def test_pre_and_backward(T, H, ht, wt, offset, pad):
    h, dx, dres = rows(T, H, ht, 1, pad, 3.0), rows(T, H, BF16, 2, pad), rows(T, H, ht, 3, pad)
    n = vq.Norm(weight(H, wt, 4, offset), EPS, offset)
    w = br.d64(n.weight)
    br.check("x", vq.norm_pre(n, h), *br.norm(br.d64(h), w, offset, EPS))
    (dv, dw), (mv, mw) = br.norm_backward(br.d64(h), w, offset, EPS, br.d64(dx))
    dh, dweight = vq.norm_pre_backward(n, h, dx, dres)
    br.check("dh", dh, dv + br.d64(dres), mv + br.d64(dres).abs())
    br.check("dweight", dweight, dw, mw)
    dh2, none = vq.norm_pre_backward(n, h, dx, weight_grad=False)
    assert none is None
    br.check("dh without dres", dh2, dv, mv)


POST = [
    # y, h, gate columns (0: none, 1, -1: hidden), gate type, post, next, res_scale, out_scale, offset, pad
    (F32, BF16, 1, BF16, True, True, 1.0, 1.0, 0.0, 0),
    (BF16, BF16, 0, None, True, False, 0.75, 1.5, 1.0, 5),
    (F32, F32, -1, F32, False, True, 1.0, 0.5, 1.0, 8),
    (BF16, F32, -1, BF16, True, True, -1.25, 1.0, 0.0, 16),
    (F32, BF16, 1, F32, False, False, 1.0, 1.0, 0.0, 0),
]


@pytest.mark.parametrize("T,H", [(1, 1), (3, 7), (5, 64), (1, 255), (4, 256), (6, 1032), (3, 4096), (2, 4099), (2, 6144),
                                 (1, 16384), (650, 48)])
@pytest.mark.parametrize("case", range(len(POST)))
def test_post_and_backward(T, H, case):
    yt, ht, gc, gt, post, nxt, a, b, offset, pad = POST[case]
    y, h = rows(T, H, yt, 10, pad, 0.5), rows(T, H, ht, 11, pad, 2.0)
    gate = None if gc == 0 else rows(T, 1 if gc == 1 else H, gt, 12, 0, 2.0)
    n1 = vq.Norm(weight(H, BF16, 13, offset), EPS, offset) if post else None
    n2 = vq.Norm(weight(H, F32, 14, offset), EPS, offset) if nxt else None
    w1, w2 = (None if n is None else br.d64(n.weight) for n in (n1, n2))
    ho, x = vq.norm_post(y, h, n1, gate, a, b, n2)
    v, mv = br.branch(br.d64(y), w1, offset, EPS, br.d64(gate), b)
    br.check("h_out", ho, a * br.d64(h) + v, abs(a) * br.d64(h).abs() + mv)
    if nxt:
        br.check("x_out", x, *br.norm(br.d64(ho), w2, offset, EPS))
    else:
        assert x is None
    for dho in (rows(T, H, ht, 15, pad), None):
        dx = rows(T, H, BF16, 16, pad) if nxt else None
        got = vq.norm_post_backward(y, ho, dho, dx, n1, gate, a, b, n2)
        ref, mag = br.post_backward(br.d64(y), br.d64(ho), br.d64(dho), br.d64(dx), w1, w2, offset, EPS, br.d64(gate), a,
                                    b)
        for name, g, r, m in zip(("dy", "dgate", "dh", "dpost", "dnext"), got, ref, mag):
            if r is None:
                assert g is None, name
            else:
                br.check(name, g, r, m)


def test_fused_next_norm_equals_a_norm_of_the_stored_row():
    T, H = 5, 4096
    y, h = rows(T, H, F32, 20), rows(T, H, BF16, 21)
    n1, n2 = vq.Norm(weight(H, BF16, 22, 0.0)), vq.Norm(weight(H, BF16, 23, 0.0))
    ho, x = vq.norm_post(y, h, n1, next=n2)
    assert torch.equal(x, vq.norm_pre(n2, ho))


def test_in_place_residual_and_given_outputs():
    T, H = 4, 640
    y, h = rows(T, H, F32, 30, 8), rows(T, H, BF16, 31, 8)
    n1, n2 = vq.Norm(weight(H, BF16, 32, 0.0)), vq.Norm(weight(H, BF16, 33, 0.0))
    want_h, want_x = vq.norm_post(y, h, n1, next=n2)
    wide = torch.full((T, H + 16), 7.0, dtype=BF16, device="cuda")
    x = wide[:, 8:8 + H]
    got_h, got_x = vq.norm_post(y, h, n1, next=n2, h_out=h, x_out=x)
    assert got_h is h and torch.equal(h, want_h) and torch.equal(x, want_x)
    assert bool((wide[:, :8] == 7).all()) and bool((wide[:, 8 + H:] == 7).all())


def test_nothing_behind_the_last_row_is_written():
    T, H = 3, 512
    buf = torch.full((T + 2, H), 5.0, dtype=BF16, device="cuda")
    vq.norm_pre(vq.Norm(weight(H, BF16, 40, 0.0)), rows(T, H, BF16, 41), out=buf[:T])
    assert bool((buf[T:] == 5).all())


def test_empty_batch():
    H = 64
    n = vq.Norm(weight(H, BF16, 50, 0.0))
    e = torch.empty((0, H), dtype=BF16, device="cuda")
    assert vq.norm_pre(n, e).shape == (0, H)
    dh, dw = vq.norm_pre_backward(n, e, e)
    assert dh.shape == (0, H) and bool((dw == 0).all())
    ho, x = vq.norm_post(e, e, n, next=n)
    assert ho.shape == x.shape == (0, H)
    got = vq.norm_post_backward(e, e, e, e, n, None, 1.0, 1.0, n)
    assert bool((got[3] == 0).all()) and bool((got[4] == 0).all())


def test_zero_rows_and_nan_stay_in_their_row():
    T, H = 4, 320
    h = rows(T, H, F32, 60)
    h[1] = 0
    h[2, 17] = float("nan")
    n = vq.Norm(weight(H, F32, 61, 0.0))
    x = vq.norm_pre(n, h)
    assert bool((x[1] == 0).all()) and bool(torch.isnan(x[2]).all())
    assert bool(torch.isfinite(x[[0, 3]]).all())
    dh, _ = vq.norm_pre_backward(n, h, rows(T, H, BF16, 62))
    assert bool(torch.isnan(dh[2]).all()) and bool(torch.isfinite(dh[[0, 1, 3]]).all())


def test_saturated_gates():
    # sigmoid(z) is exactly 0 or 1 far out; the gate's gradient vanishes there and the branch's does not turn NaN
    T, H = 4, 128
    y, h, dh = rows(T, H, F32, 70), rows(T, H, F32, 71), rows(T, H, F32, 72)
    gate = torch.tensor([[-200.0], [200.0], [-float("inf")], [float("inf")]], device="cuda")
    ho, _ = vq.norm_post(y, h, gate=gate)
    assert torch.equal(ho[[0, 2]], h[[0, 2]]) and torch.equal(ho[[1, 3]], (h + y)[[1, 3]])
    dy, dgate, _, _, _ = vq.norm_post_backward(y, ho, dh, gate=gate)
    assert bool((dgate == 0).all())
    assert bool((dy[[0, 2]] == 0).all()) and torch.equal(dy[[1, 3]], dh[[1, 3]])


def test_gradients_against_differences():
    # central differences of the fp32 call in a few directions. With step 2^-6 the quotient's own error is the
    # outputs' fp32 rounding (2^-24 * |h_out| <= 2^-21) over the step, summed over H = 96 elements, and the
    # third-order term (step^2): both below 2^-9 of the directional derivative's scale
    T, H = 2, 96
    y, h, gate = rows(T, H, F32, 80), rows(T, H, F32, 81), rows(T, 1, F32, 82)
    n1 = vq.Norm(weight(H, F32, 83, 0.0))
    G = rows(T, H, F32, 84)
    ho, _ = vq.norm_post(y, h, n1, gate, 0.5, 1.5)
    dy, dgate, dh, dpost, _ = vq.norm_post_backward(y, ho, G, None, n1, gate, 0.5, 1.5)
    step = 2.0 ** -6

    def value(dy_=0.0, dg_=0.0, dh_=0.0, dw_=0.0):
        o, _ = vq.norm_post(y + dy_, h + dh_, vq.Norm(n1.weight + dw_), gate + dg_, 0.5, 1.5)
        return (o.double() * G.double()).sum()

    for name, grad, arg in (("y", dy, "dy_"), ("gate", dgate, "dg_"), ("h", dh, "dh_"), ("weight", dpost, "dw_")):
        d = torch.randn(grad.shape, generator=torch.Generator().manual_seed(85)).cuda()
        slope = (value(**{arg: step * d}) - value(**{arg: -step * d})) / (2 * step)
        want = (grad.double() * d.double()).sum()
        scale = (grad.double().abs() * d.double().abs()).sum()
        assert abs(float(slope - want)) <= 2.0 ** -9 * float(scale), name


def test_repeatable_and_on_other_streams():
    T, H = 900, 1024
    h, dx = rows(T, H, BF16, 90), rows(T, H, BF16, 91)
    n = vq.Norm(weight(H, BF16, 92, 0.0))
    first = vq.norm_pre_backward(n, h, dx)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        again = vq.norm_pre_backward(n, h, dx, stream=s)
        s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_captured_and_replayed_on_new_inputs():
    T, H = 6, 2048
    y, h, gate = rows(T, H, F32, 100), rows(T, H, BF16, 101), rows(T, 1, BF16, 102)
    dho, dx = rows(T, H, BF16, 103), rows(T, H, BF16, 104)
    n1, n2 = vq.Norm(weight(H, BF16, 105, 0.0)), vq.Norm(weight(H, BF16, 106, 0.0))
    ws = torch.empty(vq._norm_ws(H, T) + 256, dtype=torch.uint8, device="cuda")

    def step():
        ho, x = vq.norm_post(y, h, n1, gate, 1.0, 1.0, n2)
        return (ho, x, *vq.norm_post_backward(y, ho, dho, dx, n1, gate, 1.0, 1.0, n2, workspace=ws))

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for k in range(2):
        y.copy_(rows(T, H, F32, 110 + k))
        h.copy_(rows(T, H, BF16, 120 + k))
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in out]
        assert all(torch.equal(a, b) for a, b in zip(got, step()))


# rows that stream (more than two per SM): every number of chunks a thread and of rows side by side, ragged last CTAs
STREAM = [(301, 8), (333, 256), (299, 264), (450, 520), (310, 1032), (601, 2056), (300, 4104), (297, 6144), (305, 8200),
          (298, 16384), (1000, 64), (777, 1024)]


@pytest.mark.parametrize("T,H", STREAM)
@pytest.mark.parametrize("ht,yt,gc,pad", [(BF16, F32, 1, 0), (F32, BF16, -1, 8), (BF16, BF16, 0, 3)])
def test_streaming_rows(T, H, ht, yt, gc, pad):
    y, h, dh, dx = (rows(T, H, t, 200 + i, pad) for i, t in enumerate((yt, ht, ht, BF16)))
    gate = None if gc == 0 else rows(T, 1 if gc == 1 else H, ht, 205, 0, 2.0)
    n1, n2 = vq.Norm(weight(H, BF16, 206, 0.0), EPS), vq.Norm(weight(H, F32, 207, 1.0), EPS, 1.0)
    w1, w2 = br.d64(n1.weight), br.d64(n2.weight)
    br.check("x", vq.norm_pre(n1, h), *br.norm(br.d64(h), w1, 0.0, EPS))
    (dv, dw), (mv, mw) = br.norm_backward(br.d64(h), w1, 0.0, EPS, br.d64(dx))
    got, dweight = vq.norm_pre_backward(n1, h, dx, dh)
    br.check("dh", got, dv + br.d64(dh), mv + br.d64(dh).abs())
    br.check("dweight", dweight, dw, mw)
    ho, x = vq.norm_post(y, h, n1, gate, 0.5, 2.0, n2)
    v, m = br.branch(br.d64(y), w1, 0.0, EPS, br.d64(gate), 2.0)
    br.check("h_out", ho, 0.5 * br.d64(h) + v, 0.5 * br.d64(h).abs() + m)
    br.check("x_out", x, *br.norm(br.d64(ho), w2, 1.0, EPS))
    # the definition takes one offset for both norms: the next norm's is folded into its weight
    got = vq.norm_post_backward(y, ho, dh, dx, n1, gate, 0.5, 2.0, n2)
    ref, mag = br.post_backward(br.d64(y), br.d64(ho), br.d64(dh), br.d64(dx), w1, w2 + 1.0, 0.0, EPS, br.d64(gate), 0.5,
                                2.0)
    for name, g, r, m in zip(("dy", "dgate", "dh", "dpost", "dnext"), got, ref, mag):
        if r is not None:
            br.check(name, g, r, m)


def _stream():
    return torch.cuda.current_stream().cuda_stream


@pytest.mark.parametrize("T,H", [(5, 512), (700, 512), (40, 257)])
def test_gradients_in_place(T, H):
    # the C calls allow dh on top of the residual gradient it adds
    n1, n2 = vq.Norm(weight(H, BF16, 220, 0.0)), vq.Norm(weight(H, BF16, 221, 0.0))
    h, dx, y = rows(T, H, BF16, 222), rows(T, H, BF16, 223), rows(T, H, F32, 224)
    grad = rows(T, H, BF16, 225)
    want, _ = vq.norm_pre_backward(n1, h, dx, grad, weight_grad=False)
    buf = grad.clone()
    st = vq._L().vq_norm_pre_backward(n1._ref, h.data_ptr(), vq.VQ_BF16, H, dx.data_ptr(), H, buf.data_ptr(), H, T,
                                      buf.data_ptr(), H, None, None, 0, _stream())
    assert st == 0 and torch.equal(buf, want)
    dy, _, dh, _, _ = vq.norm_post_backward(y, h, grad, dx, n1, None, 0.5, 1.0, n2)
    buf, dy2 = grad.clone(), torch.empty_like(y)
    st = vq._L().vq_norm_post_backward(n1._ref, n2._ref, H, y.data_ptr(), vq.VQ_F32, H, None, 0, 0, 0, h.data_ptr(),
                                       vq.VQ_BF16, H, 0.5, 1.0, T, buf.data_ptr(), H, dx.data_ptr(), H, dy2.data_ptr(), H,
                                       None, 0, buf.data_ptr(), H, None, None, None, 0, _stream())
    assert st == 0 and torch.equal(buf, dh) and torch.equal(dy2, dy)


def test_two_streams_at_once():
    T, H = 600, 1024
    n = vq.Norm(weight(H, BF16, 230, 0.0))
    ins = [(rows(T, H, BF16, 231 + i), rows(T, H, BF16, 235 + i)) for i in range(2)]
    want = [vq.norm_pre_backward(n, h, dx) for h, dx in ins]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ins]
    got = [[vq.norm_pre_backward(n, h, dx, stream=s) for (h, dx), s in zip(ins, streams)] for _ in range(10)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for one in got for p, q in zip(one, want) for a, b in zip(p, q))


def test_rows_far_apart():
    # rows 2^30 elements apart: offsets beyond 32 bits
    H = 512
    far = lambda: torch.zeros(2 * 2 ** 30 + H, dtype=BF16, device="cuda").as_strided((3, H), (2 ** 30, 1))  # noqa: E731
    h, x = far(), far()
    h.copy_(rows(3, H, BF16, 240))
    n = vq.Norm(weight(H, BF16, 241, 0.0))
    vq.norm_pre(n, h, out=x)
    br.check("x", x, *br.norm(br.d64(h), br.d64(n.weight), 0.0, EPS))
    dh, _ = vq.norm_pre_backward(n, h, x, h)
    (dv, _), (mv, _) = br.norm_backward(br.d64(h), br.d64(n.weight), 0.0, EPS, br.d64(x))
    br.check("dh", dh, dv + br.d64(h), mv + br.d64(h).abs())


def test_first_call_may_be_captured():
    # a width and types that nothing here has launched before: the launch's own set-up happens inside the capture
    T, H = 320, 12288
    y, h = rows(T, H, BF16, 250), rows(T, H, F32, 251)
    n1, n2 = vq.Norm(weight(H, F32, 252, 0.0)), vq.Norm(weight(H, F32, 253, 0.0))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out = vq.norm_post(y, h, n1, next=n2)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, vq.norm_post(y, h, n1, next=n2)))


@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 17, 300])
@pytest.mark.parametrize("H", [40, 640, 6144])
@pytest.mark.parametrize("offset", [0, 1])
def test_weight_gradients_of_few_rows_and_off_16_bytes(T, H, offset):
    n1, n2 = vq.Norm(weight(H, BF16, 260, 0.0), EPS), vq.Norm(weight(H, F32, 261, 0.0), EPS)
    h, dx, y = rows(T, H, BF16, 262), rows(T, H, BF16, 263), rows(T, H, F32, 264)
    ws = torch.empty(vq._norm_ws(H, T) + 256, dtype=torch.uint8, device="cuda")
    wp = (ws.data_ptr() + 255) // 256 * 256
    buf = torch.full((2, H + 8), float("nan"), device="cuda")
    d1, d2 = (b[offset:offset + H] for b in buf)
    dh, dy = torch.empty_like(h), torch.empty_like(y)
    st = vq._L().vq_norm_pre_backward(n1._ref, h.data_ptr(), vq.VQ_BF16, H, dx.data_ptr(), H, None, 0, T, dh.data_ptr(), H,
                                      d1.data_ptr(), wp, ws.numel() - 256, _stream())
    assert st == 0
    (dv, dw), (mv, mw) = br.norm_backward(br.d64(h), br.d64(n1.weight), 0.0, EPS, br.d64(dx))
    br.check("dh", dh, dv, mv)
    br.check("dweight", d1, dw, mw)
    st = vq._L().vq_norm_post_backward(n1._ref, n2._ref, H, y.data_ptr(), vq.VQ_F32, H, None, 0, 0, 0, h.data_ptr(),
                                       vq.VQ_BF16, H, 1.0, 1.0, T, None, 0, dx.data_ptr(), H, dy.data_ptr(), H, None, 0,
                                       None, 0, d1.data_ptr(), d2.data_ptr(), wp, ws.numel() - 256, _stream())
    assert st == 0
    ref, mag = br.post_backward(br.d64(y), br.d64(h), None, br.d64(dx), br.d64(n1.weight), br.d64(n2.weight), 0.0, EPS,
                                None, 1.0, 1.0)
    br.check("dy", dy, ref[0], mag[0])
    br.check("dpost", d1, ref[3], mag[3])
    br.check("dnext", d2, ref[4], mag[4])
    assert bool(torch.isnan(buf[:, offset + H:]).all()) and bool(torch.isnan(buf[:, :offset]).all())
