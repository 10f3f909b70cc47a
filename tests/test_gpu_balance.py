"""Per-expert counts and the router's balance loss, with its gradient, against the definition in 64 bits."""
import pytest
import torch

import block_ref as br

import vector_quantized_moe_b200 as vq

pytestmark = pytest.mark.gpu


def inputs(T, E, k, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    logits = torch.randn((T, E), generator=g) * spread + torch.randn(E, generator=g)
    return logits.cuda()


def run_and_check(logits, ids, mask, coef, dl=1.5):
    T, E = logits.shape
    k = ids.shape[1]
    loss, counts, probs = vq.balance_loss(logits, ids, mask, coef)
    rl, rc, rp = br.balance(br.d64(logits), ids.cpu(), mask, coef)
    assert torch.equal(counts.cpu().long(), rc)
    br.check("probs", probs, rp, rp)
    br.check("loss", loss, rl, rl.abs())
    dloss = torch.tensor(dl, device="cuda")
    d = vq.balance_loss_backward(logits, counts, k, dloss, mask, coef)
    br.check("dlogits", d, *br.balance_backward(br.d64(logits), rc, k, dl, mask, coef))
    return loss, counts, probs, d


SIZES = [(1, 1, 1), (1, 8, 2), (3, 5, 5), (17, 128, 8), (64, 512, 10), (65, 512, 10), (100, 33, 3), (257, 130, 4),
         (300, 256, 8), (70, 515, 7), (1000, 1024, 10), (40, 1025, 6), (130, 4096, 32), (5000, 64, 2)]


@pytest.mark.parametrize("T,E,k", SIZES)
@pytest.mark.parametrize("masked", [False, True])
def test_loss_counts_and_gradient(T, E, k, masked):
    logits = inputs(T, E, k, T + E)
    ids = vq.route(logits, k)[0]
    mask = None
    if masked:
        mask = (torch.rand(T, generator=torch.Generator().manual_seed(1)) < 0.7).cuda()
    run_and_check(logits, ids, mask, 0.01 * E)


def test_counts_match_the_routers_buckets():
    T, E, k = 200, 64, 6
    logits = inputs(T, E, k, 5)
    ids, _, offsets, _ = vq.route(logits, k)
    _, counts, _ = vq.balance_loss(logits, ids)
    assert torch.equal(counts[:E], offsets[1:] - offsets[:-1]) and int(counts[E]) == T


@pytest.mark.parametrize("T", [7, 300])
def test_all_masked_is_zero(T):
    E, k = 40, 3
    logits = inputs(T, E, k, 6)
    logits[0] = float("nan")   # a masked row is not read into anything
    ids = vq.route(logits, k)[0]
    mask = torch.zeros(T, dtype=torch.uint8, device="cuda")
    loss, counts, probs = vq.balance_loss(logits, ids, mask)
    d = vq.balance_loss_backward(logits, counts, k, None, mask)
    assert float(loss) == 0 and not counts.any() and not probs.any() and not d.any()


@pytest.mark.parametrize("T", [9, 200])
def test_masked_nan_rows_dropped_pairs_and_repeats(T):
    E, k = 48, 4
    logits = inputs(T, E, k, 7)
    ids = vq.route(logits, k)[0].clone()
    ids[1] = torch.tensor([3, 3, -1, E], device="cuda")   # one expert twice, two pairs dropped
    mask = torch.ones(T, dtype=torch.bool, device="cuda")
    mask[2] = False
    logits[2] = float("nan")
    clean = logits.clone()
    clean[2] = 0
    a = run_and_check(clean, ids, mask, 1.0)
    loss, counts, probs = vq.balance_loss(logits, ids, mask, 1.0)
    d = vq.balance_loss_backward(logits, counts, k, torch.tensor(1.5, device="cuda"), mask, 1.0)
    for x, y in zip(a, (loss, counts, probs, d)):
        assert torch.equal(x, y)


@pytest.mark.parametrize("E", [64, 65, 2000])
def test_masked_experts_and_empty_rows(E):
    T, k = 66, 2
    logits = inputs(T, E, k, 8)
    logits[:, E // 2:] = float("-inf")          # experts switched off
    logits[5] = float("-inf")                   # nothing left: probability 0 everywhere
    logits[6] = torch.finfo(torch.float32).min  # the type's lowest value: an even row
    ids = vq.route(logits, k)[0]
    _, _, _, d = run_and_check(logits, ids, None, 1.0)
    assert not d[5].any() and not d[:5, E // 2:].any() and bool(torch.isfinite(d).all())


@pytest.mark.parametrize("E", [64, 1500])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_nan_and_inf_rows_follow_ieee(E, value):
    T, k = 20, 2
    logits = inputs(T, E, k, 9)
    ids = vq.route(logits, k)[0]
    logits[3, 1] = value
    loss, counts, probs = vq.balance_loss(logits, ids)
    d = vq.balance_loss_backward(logits, counts, k)
    assert bool(torch.isnan(loss)) and bool(torch.isnan(probs[1])) and bool(torch.isnan(d[3]).any())
    assert bool(torch.isfinite(torch.cat([d[:3], d[4:]])).all())


def test_all_nan_row_is_nan():
    logits = inputs(4, 32, 2, 10)
    ids = vq.route(logits, 2)[0]
    logits[1] = float("nan")
    loss, _, probs = vq.balance_loss(logits, ids)
    assert bool(torch.isnan(loss)) and bool(torch.isnan(probs).all())


def test_empty_batch_and_in_place_gradient():
    E = 16
    e = torch.empty((0, E), device="cuda")
    loss, counts, probs = vq.balance_loss(e, torch.empty((0, 2), dtype=torch.int32, device="cuda"))
    assert float(loss) == 0 and not counts.any() and not probs.any()
    assert vq.balance_loss_backward(e, counts, 2).shape == (0, E)
    for E in (100, 1100):
        logits = inputs(50, E, 2, 11)
        ids = vq.route(logits, 2)[0]
        _, counts, _ = vq.balance_loss(logits, ids)
        want = vq.balance_loss_backward(logits, counts, 2)
        st = vq._L().vq_balance_loss_backward(logits.data_ptr(), counts.data_ptr(), None, 50, E, 2, 1.0, None,
                                              logits.data_ptr(), torch.cuda.current_stream().cuda_stream)
        assert st == 0
        assert torch.equal(logits, want)


def test_gradient_against_differences():
    # loss along a direction, counts held: central differences in fp32 with step 2^-7. The quotient's error is the
    # loss's rounding (2^-24 * 8 over the step) and the third-order term; the derivative itself is of order 1
    T, E, k = 6, 16, 3
    logits = inputs(T, E, k, 12)
    ids = vq.route(logits, k)[0]
    _, counts, _ = vq.balance_loss(logits, ids, None, 8.0)
    d = vq.balance_loss_backward(logits, counts, k, None, None, 8.0)
    v = torch.randn(logits.shape, generator=torch.Generator().manual_seed(13)).cuda()
    step = 2.0 ** -7
    up, dn = (vq.balance_loss(logits + s * step * v, ids, None, 8.0)[0].double() for s in (1, -1))
    slope, want = float((up - dn) / (2 * step)), float((d.double() * v.double()).sum())
    scale = float((d.double().abs() * v.double().abs()).sum())
    assert abs(slope - want) <= 2.0 ** -8 * scale


def test_repeatable_captured_and_replayed():
    T, E, k = 3000, 256, 8
    logits = inputs(T, E, k, 14)
    ids = vq.route(logits, k)[0]
    ws = torch.empty(vq._balance_ws(T, E) + 256, dtype=torch.uint8, device="cuda")

    def step():
        loss, counts, probs = vq.balance_loss(logits, ids, None, 0.1, workspace=ws)
        return loss, counts, probs, vq.balance_loss_backward(logits, counts, k, loss, None, 0.1)

    first = [o.clone() for o in step()]
    assert all(torch.equal(a, b) for a, b in zip(first, step()))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    logits.copy_(inputs(T, E, k, 15))
    ids.copy_(vq.route(logits, k)[0])
    graph.replay()
    torch.cuda.synchronize()
    got = [o.clone() for o in out]
    assert all(torch.equal(a, b) for a, b in zip(got, step()))


def test_two_streams_at_once():
    T, E, k = 900, 128, 4
    ins = []
    for i in range(2):
        logits = inputs(T, E, k, 20 + i)
        ins.append((logits, vq.route(logits, k)[0]))
    want = [vq.balance_loss(*a) for a in ins]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ins]
    got = [[vq.balance_loss(*a, stream=s) for a, s in zip(ins, streams)] for _ in range(10)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for one in got for p, q in zip(one, want) for a, b in zip(p, q))


def test_extreme_logits():
    # far from zero (the difference to the largest is what counts), and spreads beyond fp32's exponent range
    T, E, k = 70, 40, 3
    logits = inputs(T, E, k, 24)
    logits[:20] += 3.0e4
    logits[20:40] *= 1.0e4
    logits[40] = torch.finfo(torch.float32).max
    logits[41, ::2] = torch.finfo(torch.float32).max
    logits[41, 1::2] = torch.finfo(torch.float32).min
    ids = vq.route(logits, k)[0]
    run_and_check(logits, ids, None, 1.0)
