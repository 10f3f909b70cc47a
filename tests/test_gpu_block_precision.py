"""How exact the block operators' fp32 results are, beside the looser bounds of their other tests.

u = 2^-24, half a step of fp32, is the most that one rounding adds, relative to its result. Relative errors here are in
the L2 norm over an output, against the L2 norm of the magnitudes (the sums of the absolute values of its terms).

Norms. An element has about 10 roundings of its own, independent of each other: sqrt(10) u / sqrt(3) < 2 u. A row's
factor r is shared: its sum of squares has fewer than 24 roundings in a row (4 to 16 in a thread, 1, and 9 shuffles),
sqrt(24) u / sqrt(3) < 3 u, and r takes half of that; rsqrtf is within 2 ulp, 4 u. Gradients use r twice and another
sum. Together below 2 + 2 (1.5 + 4) = 13 u, taken as 16 u; a sigmoid adds the 2^-22 = 4 u of its exponential, 1 ulp
(2 u) of its reciprocal and |z| u / sqrt(3) of its argument's rounding, |z| < 8: 12 u more, taken as 32 u together.

Balance loss. A probability has the exponential's 4 u, its argument's rounding (|l - max| u / sqrt(3), up to 20 here:
12 u), the row sum's 3 u and three roundings of its own; column sums add up to 100 in a row, sqrt(100 / 3) = 6 u. Taken
as 32 u.

4-bit products. Of one product's fp32 arithmetic nothing is assumed but that an mma instruction, 16 products and an
accumulator, is off by at most one step (2 u, whichever way it rounds) of the absolute values that it has added so far.
A group has G / 16 instructions for sum (16 + q) x and for sum x each, so with P = |s| sum (16 + q) |x| and
X = 24 |s| sum |x| (with biases |b - 16 s| sum |x|) their errors are at most (G / 8) u (P + X); the two fused
multiply-adds that follow are off by at most u (|acc| + P) and u (|acc| + |s (q - 8)| |x|), |acc| at most the sum M of
all |w x|; splits and the store add 8 more. Bound, element by element:
u ((G / 8 + 2) sum (P + X) + (2 groups + 8) M).
"""
import pytest
import torch

import block_ref as br

import vector_quantized_moe_b200 as vq
from test_gpu_norm import rows, weight
from test_gpu_q4 import module, tokens

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24
EPS = 1e-6


def close(what, got, ref, mag, units):
    err = float((br.d64(got) - ref).norm() / mag.norm())
    assert err <= units * U, f"{what}: {err / U:.2f} u"


SHAPES = [(3, 512), (2, 4096), (300, 1000), (300, 2048), (17, 6144), (5, 4099)]


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("gate", [0, 1, -1])
def test_post_and_backward(T, H, gate):
    y, h, dho = rows(T, H, F32, 1), rows(T, H, F32, 2), rows(T, H, F32, 3)
    dx = rows(T, H, BF16, 4)
    z = None if gate == 0 else rows(T, 1 if gate == 1 else H, F32, 5, 0, 2.0).clamp(-8, 8)
    n1, n2 = vq.Norm(weight(H, F32, 6, 0.0), EPS), vq.Norm(weight(H, F32, 7, 0.0), EPS)
    w1, w2 = br.d64(n1.weight), br.d64(n2.weight)
    units = 16 if gate == 0 else 32
    ho, _ = vq.norm_post(y, h, n1, z, 0.75, 1.5, n2)
    v, mv = br.branch(br.d64(y), w1, 0.0, EPS, br.d64(z), 1.5)
    close("h_out", ho, 0.75 * br.d64(h) + v, 0.75 * br.d64(h).abs() + mv, units)
    got = vq.norm_post_backward(y, ho, dho, dx, n1, z, 0.75, 1.5, n2)
    ref, mag = br.post_backward(br.d64(y), br.d64(ho), br.d64(dho), br.d64(dx), w1, w2, 0.0, EPS, br.d64(z), 0.75, 1.5)
    for name, g, r, m in zip(("dy", "dgate", "dh", "dpost", "dnext"), got, ref, mag):
        if r is not None:
            close(name, g, r, m, units)


@pytest.mark.parametrize("T,H", SHAPES)
def test_pre_backward(T, H):
    h, dx = rows(T, H, F32, 10, 0, 3.0), rows(T, H, BF16, 11)
    n = vq.Norm(weight(H, F32, 12, 0.0), EPS)
    (dv, dw), (mv, mw) = br.norm_backward(br.d64(h), br.d64(n.weight), 0.0, EPS, br.d64(dx))
    dh, dweight = vq.norm_pre_backward(n, h, dx)
    close("dh", dh, dv, mv, 16)
    close("dweight", dweight, dw, mw, 16)


@pytest.mark.parametrize("T,E,k", [(16, 512, 10), (64, 7, 2), (1000, 256, 8), (5000, 100, 4), (700, 1500, 8)])
def test_balance(T, E, k):
    g = torch.Generator().manual_seed(T)
    logits = (2 * torch.randn((T, E), generator=g)).cuda()
    ids = vq.route(logits, k)[0]
    loss, counts, probs = vq.balance_loss(logits, ids)
    rl, rc, rp = br.balance(br.d64(logits), ids.cpu(), None, 1.0)
    close("loss", loss, rl, rl, 32)
    close("probs", probs, rp, rp, 32)
    d = vq.balance_loss_backward(logits, counts, k)
    close("dlogits", d, *br.balance_backward(br.d64(logits), rc, k, 1.0, None, 1.0), 32)


def bound(words, sc, bi, group, x):
    q = torch.stack([((words.cpu().long() & 0xFFFFFFFF) >> (4 * i)) & 15 for i in range(8)], 2).reshape(words.shape[0], -1).double()
    s = sc.cpu().double().repeat_interleave(group, 1)
    W = s * (q - 8)
    M24 = 24 * s.abs()
    if bi is not None:
        b = bi.cpu().double().repeat_interleave(group, 1)
        W, M24 = s * q + b, (b - 16 * s).abs()
    ax = x.abs()
    M = ax @ W.abs().T
    return x @ W.T, U * ((group / 8 + 2) * (ax @ (s.abs() * (16 + q) + M24).T) + (2 * sc.shape[1] + 8) * M), W


@pytest.mark.parametrize("rows_,cols,group", [(48, 4096, 128), (600, 1024, 64), (20000, 512, 32), (70000, 256, 128)])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("T", [1, 8, 13])
@pytest.mark.parametrize("offset", [0.0, 100.0])
def test_products_of_tokens_with_a_common_offset(rows_, cols, group, biased, T, offset):
    raw, m = module(rows_, cols, group, biased, 20)
    x = (tokens(T, cols, 21).float() + offset).to(BF16)
    ref, tol, _ = bound(*raw, group, br.d64(x))
    err = (br.d64(vq.q4_gemv(m, x, out_dtype=F32)) - ref).abs()
    assert bool((err <= tol).all()), f"{float((err / tol).max()):.2f} of the bound"


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("T", [1, 9])
def test_rows_of_zero_weights(group, T):
    # every code 8: the weights are 0, and what is left of 24 sum x against (16 + 8) x is within the bound
    rows_, cols = 40, 1024
    words = torch.full((rows_, cols // 8), -0x77777778, dtype=torch.int32, device="cuda")   # 0x88888888
    sc = torch.full((rows_, cols // group), 0.01, dtype=torch.float16, device="cuda")
    m = vq.Q4Module.from_rows(words, sc, group=group)
    x = (tokens(T, cols, 22).float() + 10).to(BF16)
    ref, tol, W = bound(words, sc, None, group, br.d64(x))
    assert bool((W == 0).all())
    assert bool((br.d64(vq.q4_gemv(m, x, out_dtype=F32)).abs() <= tol).all())
