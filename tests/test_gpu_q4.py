"""Dense 4-bit matrix-vector products against their definition in 64 bits: groups, offsets, ragged sizes, token counts,
row strides, pairs."""
import numpy as np
import pytest
import torch

import block_ref as br

import vector_quantized_moe_b200 as vq

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def module(rows, cols, group, biased, seed):
    """(device arrays in row order, packed module); codes packed by the library's host packing."""
    g = np.random.default_rng(seed)
    codes = g.integers(0, 16, (1, rows, cols), dtype=np.uint16)
    words = torch.from_numpy(vq.pack(codes, 4).view(np.int32)).cuda()
    sc = torch.from_numpy(g.uniform(0.5, 2.0, (rows, cols // group)) / (5 * cols ** 0.5)).half()
    if rows > 2:
        sc[1] *= -1
    bi = None
    if biased:
        bi = (-sc.float() * torch.from_numpy(g.normal(7.5, 1.0, sc.shape)).float()).half().cuda()
    sc = sc.cuda()
    return (words, sc, bi), vq.Q4Module.from_rows(words, sc, bi, group=group)


def tokens(T, cols, seed, pad=0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn((T, cols + pad), generator=g).to(BF16).cuda()[:, :cols]


SIZES = [(1, 32, 32), (7, 64, 64), (16, 128, 128), (17, 96, 32), (40, 320, 64), (33, 4096, 128), (512, 1024, 64),
         (1000, 2048, 32), (2500, 256, 64), (9600, 128, 128), (5000, 160, 32)]


@pytest.mark.parametrize("rows,cols,group", SIZES)
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("T", [1, 5, 8, 13, 29, 40])
def test_gemv(rows, cols, group, biased, T):
    raw, m = module(rows, cols, group, biased, rows + cols)
    x = tokens(T, cols, T, 8 if T > 8 else 0)
    ref, mag = br.q4(*raw, group, br.d64(x))
    br.check("fp32", vq.q4_gemv(m, x, out_dtype=F32), ref, mag)
    br.check("bf16", vq.q4_gemv(m, x), ref, mag)


@pytest.mark.parametrize("rows,cols,group,biased,T", [(1, 32, 32, False, 1), (40, 256, 64, True, 3), (2040, 512, 32, False, 16),
                                                      (700, 1024, 128, True, 30), (5000, 128, 64, False, 9)])
def test_pair(rows, cols, group, biased, T):
    r0, m0 = module(rows, cols, group, biased, 1)
    r1, m1 = module(rows, cols, group, biased, 2)
    x = tokens(T, cols, 3)
    ref, mag = br.q4_pair(*br.q4(*r0, group, br.d64(x)), *br.q4(*r1, group, br.d64(x)))
    br.check("fp32", vq.q4_gemv(m0, x, m1, F32), ref, mag)
    br.check("bf16", vq.q4_gemv(m0, x, m1), ref, mag)


def test_one_hot_tokens_read_back_the_exact_weights():
    # y[c, r] = W[r, c] with one product per sum: the codes' exact value times the fp32 scale, bit for bit
    rows, cols, group = 50, 192, 64
    (words, sc, _), m = module(rows, cols, group, False, 4)
    y = vq.q4_gemv(m, torch.eye(cols, dtype=BF16, device="cuda"), out_dtype=F32)
    w = words.cpu().long() & 0xFFFFFFFF
    q = torch.stack([(w >> (4 * i)) & 15 for i in range(8)], 2).reshape(rows, cols)
    W = sc.cpu().float().repeat_interleave(group, 1) * (q - 8).float()
    assert torch.equal(y.cpu().T, W)


def test_agrees_with_the_codebook_module_of_the_same_weights():
    # the same codes as a d = 1, 4-bit codebook module (C[q] = q - 8, groups of 64): its tokens are rounded to fp16
    # at the scale of the group's largest (2^-11 of each product), this call's are not
    rows, cols, T = 300, 1024, 6
    g = np.random.default_rng(5)
    codes = g.integers(0, 16, (1, rows, cols), dtype=np.uint16)
    sc = (g.uniform(0.5, 2.0, (rows, cols // 64)) / 160).astype(np.float16).view(np.uint16)
    cb = (np.arange(16, dtype=np.float32) - 8).astype(np.float16).view(np.uint16).reshape(16, 1)
    words = vq.pack(codes, 4)
    cm = vq.Module.from_host(1, rows, cols, 1, 4, words, sc, cb)
    qm = vq.Q4Module.from_rows(torch.from_numpy(words.view(np.int32)).cuda(),
                               torch.from_numpy(sc.view(np.int16)).cuda(), group=64)
    x = tokens(T, cols, 6)
    a, b = vq.gemv(cm, 0, x), vq.q4_gemv(qm, x, out_dtype=F32)
    q = torch.from_numpy(codes[0].astype(np.float64)) - 8
    s = torch.from_numpy(sc.view(np.float16).astype(np.float64)).repeat_interleave(64, 1)
    mag = br.d64(x).abs() @ (s * q).abs().T
    assert bool(((a - b).cpu().double().abs() <= (2.0 ** -11 + 2 * br.SLACK) * mag).all())


def test_layout_follows_its_documentation():
    rows, cols, group = 21, 160, 32
    (words, sc, _), m = module(rows, cols, group, False, 7)
    w = words.cpu().numpy().view(np.uint32)
    code = lambda r, c: int(w[r, c // 8] >> (4 * (c % 8))) & 15 if r < rows and c < cols else 0  # noqa: E731
    nsb, ng = 2, 128 // group
    out = m.words.cpu().numpy().view(np.uint32)
    ps = m.scales.cpu().numpy()
    s = sc.cpu().view(torch.int16).numpy()
    assert out.size == 2 * nsb * 256 == vq._L().vq_q4_packed_words(rows, cols)
    assert ps.size == 2 * nsb * 16 * ng == vq._L().vq_q4_packed_scales(rows, cols, group)
    for i in range(2):
        for j in range(nsb):
            for b in range(2):
                for lane in range(32):
                    for p in range(4):
                        g, c = lane // 4, lane % 4
                        k = 128 * j + 64 * b + 32 * (p // 2) + 8 * c + 4 * (p % 2)
                        want = 0
                        for e in range(4):
                            r = 16 * i + g + 8 * (e % 2)
                            both = code(r, k + 2 * (e // 2)) | code(r, k + 2 * (e // 2) + 1) << 16
                            n = 3 + 4 * e   # rotated left
                            want |= (both << n | both >> (32 - n)) & 0xFFFFFFFF
                        assert out[(i * nsb + j) * 256 + (b * 32 + lane) * 4 + p] == want
            for g in range(8):
                for grp in range(ng):
                    for hi in range(2):
                        r, n = 16 * i + g + 8 * hi, j * ng + grp
                        want = s[r, n] if r < rows and n < cols // group else 0
                        assert ps[((i * nsb + j) * 8 + g) * ng * 2 + grp * 2 + hi] == want


def test_strided_rows_and_nothing_else_written():
    rows, cols, T = 100, 256, 11
    raw, m = module(rows, cols, 64, True, 8)
    x = tokens(T, cols, 9, 24)
    wide = torch.full((T + 1, rows + 9), 3.0, dtype=F32, device="cuda")
    y = wide[:T, 4:4 + rows]
    vq.q4_gemv(m, x, out=y)
    br.check("y", y, *br.q4(*raw, 64, br.d64(x)))
    assert bool((wide[T] == 3).all()) and bool((wide[:, :4] == 3).all()) and bool((wide[:, 4 + rows:] == 3).all())


def test_wide_range_of_activations():
    # bf16's whole exponent range is taken as it is: no fp16 in between
    rows, cols = 64, 256
    raw, m = module(rows, cols, 128, False, 10)
    x = tokens(2, cols, 11)
    x[0] *= 2.0 ** 100
    x[1] *= 2.0 ** -100
    ref, mag = br.q4(*raw, 128, br.d64(x))
    br.check("y", vq.q4_gemv(m, x, out_dtype=F32), ref, mag)


def test_non_finite_tokens_stay_in_their_row():
    rows, cols = 48, 128
    raw, m = module(rows, cols, 32, False, 12)
    x = tokens(3, cols, 13)
    x[1, 5] = float("nan")
    y = vq.q4_gemv(m, x, out_dtype=F32)
    assert bool(torch.isnan(y[1]).all()) and bool(torch.isfinite(y[[0, 2]]).all())


def test_empty_batch_streams_and_replay():
    rows, cols = 130, 512
    raw, m = module(rows, cols, 64, False, 14)
    assert vq.q4_gemv(m, torch.empty((0, cols), dtype=BF16, device="cuda")).shape == (0, rows)
    x = tokens(4, cols, 15)
    want = vq.q4_gemv(m, x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = vq.q4_gemv(m, x, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = vq.q4_gemv(m, x)
    x.copy_(tokens(4, cols, 16))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, vq.q4_gemv(m, x))


# shapes whose estimate picks each split: row tiles per warp x warps per row group, for one and for two token tiles
SPLITS = [(70000, 128, 64, False), (70016, 320, 32, True), (40000, 160, 32, False), (20000, 512, 128, True),
          (9600, 512, 64, False), (5000, 1024, 128, True), (40, 4096, 32, True)]


@pytest.mark.parametrize("rows,cols,group,biased", SPLITS)
@pytest.mark.parametrize("T", [3, 13])
def test_every_split(rows, cols, group, biased, T):
    raw, m = module(rows, cols, group, biased, rows)
    x = tokens(T, cols, 20)
    ref, mag = br.q4(*raw, group, br.d64(x))
    br.check("y", vq.q4_gemv(m, x, out_dtype=F32), ref, mag)


@pytest.mark.parametrize("rows,cols,T", [(40000, 128, 2), (20000, 160, 8), (9600, 512, 5), (9600, 512, 11), (100, 2048, 2)])
def test_every_split_of_a_pair(rows, cols, T):
    r0, m0 = module(rows, cols, 32, True, 21)
    r1, m1 = module(rows, cols, 32, True, 22)
    x = tokens(T, cols, 23)
    ref, mag = br.q4_pair(*br.q4(*r0, 32, br.d64(x)), *br.q4(*r1, 32, br.d64(x)))
    br.check("y", vq.q4_gemv(m0, x, m1, F32), ref, mag)


def test_two_streams_at_once():
    raw, m = module(3000, 1024, 64, True, 24)
    xs = [tokens(4, 1024, 25 + i) for i in range(2)]
    want = [vq.q4_gemv(m, x) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = [[vq.q4_gemv(m, x, stream=s) for x, s in zip(xs, streams)] for _ in range(20)]
    torch.cuda.synchronize()
    assert all(torch.equal(g, w) for pair in got for g, w in zip(pair, want))


def test_rows_of_q4_far_apart():
    # token and output rows 2^30 elements apart: offsets beyond 32 bits
    raw, m = module(64, 256, 64, False, 27)
    x = torch.zeros(2 * 2 ** 30 + 256, dtype=BF16, device="cuda").as_strided((3, 256), (2 ** 30, 1))
    y = torch.zeros(2 * 2 ** 30 + 64, dtype=BF16, device="cuda").as_strided((3, 64), (2 ** 30, 1))
    x.copy_(tokens(3, 256, 28))
    vq.q4_gemv(m, x, out=y)
    br.check("y", y, *br.q4(*raw, 64, br.d64(x)))


def test_most_tokens():
    T = 16 * 65535
    raw, m = module(3, 32, 32, True, 30)
    x = tokens(T, 32, 31)
    ref, mag = br.q4(*raw, 32, br.d64(x))
    br.check("y", vq.q4_gemv(m, x, out_dtype=F32), ref, mag)


@pytest.mark.parametrize("rows", [70000, 40000, 512])
def test_x_rewritten_by_the_call_before(rows):
    # each product reads the x that the launch before it wrote over the one that the product before that read
    raw, m = module(rows, 128, 64, False, 32)
    n = vq.Norm(torch.ones(128, device="cuda"))
    hs = [torch.randn((8, 128), generator=torch.Generator().manual_seed(33 + i)).cuda() for i in range(20)]
    xs = [vq.norm_pre(n, h) for h in hs]
    want = [vq.q4_gemv(m, x) for x in xs]
    x, got = torch.empty_like(xs[0]), []
    torch.cuda.synchronize()
    for h in hs:
        vq.norm_pre(n, h, out=x)
        got.append(vq.q4_gemv(m, x))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
