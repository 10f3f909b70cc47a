"""Definitions of the block operators in 64 bits (torch on the CPU), with the magnitudes that bound their errors.

Each function returns (values, magnitudes): a computed fp32 value may be off by SLACK times its magnitude, the sum of
the absolute values of the terms that make it; a stored bf16 value by half a step (2^-8 of the value) more.

SLACK: a row sum adds at most 64 terms in a thread, then over 5 + 5 shuffle steps, with at most 3 roundings a term; a
weight gradient adds at most T / CTAs rows in a thread, then at most 74 partial rows and 8 strands. For the sizes
tested here no chain is longer than 200 roundings of 2^-24, and no formula multiplies more than two such sums:
2 * 200 * 2^-24 < 2^-15.
"""
import torch

SLACK = 2.0 ** -15
BF16_STEP = torch.finfo(torch.bfloat16).eps / 2   # half a step, relative


def d64(t):
    if t is None:
        return None
    if t.dtype == torch.int16:
        t = t.view(torch.bfloat16)
    return t.detach().cpu().double()


def check(what, got, ref, mag):
    """got (fp32 or bf16 tensor) against the 64-bit ref with error magnitudes mag."""
    assert got is not None, what
    assert tuple(got.shape) == tuple(ref.shape), (what, got.shape, ref.shape)
    g = got.detach().cpu().double()
    tol = SLACK * mag
    if got.dtype == torch.bfloat16:
        tol = tol + BF16_STEP * (ref.abs() + tol)
    bad = ~((g - ref).abs() <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {((g - ref).abs() - tol)[bad].max():.3e}"


def norm(v, w, offset, eps):
    n = v / torch.sqrt((v * v).mean(1, keepdim=True) + eps) * (w + offset)
    return n, n.abs()


def norm_backward(v, w, offset, eps, dn):
    """((dv, dw), magnitudes) of norm at v for the gradient dn >= its magnitude."""
    r = 1.0 / torch.sqrt((v * v).mean(1, keepdim=True) + eps)
    n = v * r
    g = (w + offset) * dn
    dv = r * (g - n * (g * n).mean(1, keepdim=True))
    mv = r * (g.abs() + n.abs() * (g * n).abs().mean(1, keepdim=True))
    return (dv, (dn * n).sum(0)), (mv, (dn * n).abs().sum(0))


def branch(y, w, offset, eps, gate, out_scale):
    u = y if w is None else norm(y, w, offset, eps)[0]
    v = out_scale * u * (1.0 if gate is None else torch.sigmoid(gate))
    return v, v.abs()


def post_backward(y, h_out, dh, dx, w1, w2, offset, eps, gate, res_scale, out_scale):
    """Values and magnitudes of dy, dgate, dh, dpost, dnext (None where there is none)."""
    T, H = y.shape
    dH = torch.zeros_like(y) if dh is None else dh
    mH = dH.abs()
    dnext = mnext = dpost = mpost = dgate = mgate = None
    if w2 is not None:
        (dv, dnext), (mv, mnext) = norm_backward(h_out, w2, offset, eps, dx)
        dH, mH = dH + dv, mH + mv
    u = y if w1 is None else norm(y, w1, offset, eps)[0]
    du, mu = out_scale * dH, abs(out_scale) * mH
    if gate is not None:
        on, off = torch.sigmoid(gate), torch.sigmoid(-gate)
        dgate, mgate = du * u, mu * u.abs()
        if gate.shape[1] == 1 and H > 1:
            dgate, mgate = dgate.sum(1, keepdim=True), mgate.sum(1, keepdim=True)
        dgate, mgate = dgate * on * off, mgate * on * off
        du, mu = du * on, mu * on
    dy, my = du, mu
    if w1 is not None:
        (dy, dpost), _ = norm_backward(y, w1, offset, eps, du)
        r = 1.0 / torch.sqrt((y * y).mean(1, keepdim=True) + eps)
        mg = (w1 + offset).abs() * mu
        my = r * (mg + (y * r).abs() * (mg * (y * r).abs()).mean(1, keepdim=True))
        mpost = (mu * (y * r).abs()).sum(0)
    return ((dy, dgate, res_scale * dH, dpost, dnext), (my, mgate, abs(res_scale) * mH, mpost, mnext))


def balance(logits, ids, mask, coef):
    """(loss, counts, probs), and magnitudes of loss and probs."""
    T, E = logits.shape
    live = torch.ones(T, dtype=torch.bool) if mask is None else mask.cpu().bool()
    V, k = int(live.sum()), ids.shape[1]
    used = ids[live].reshape(-1).long()
    used = used[(used >= 0) & (used < E)]
    counts = torch.cat([torch.bincount(used, minlength=E), torch.tensor([V])])
    p = softmax(logits)[live].sum(0) / max(V, 1)
    loss = coef * (E * counts[:E].double() / max(V * k, 1) * p).sum()
    return loss, counts, p


def softmax(logits):
    """Rows of -Inf give 0."""
    top = logits.max(1, keepdim=True).values
    e = torch.where(top == -torch.inf, torch.zeros_like(logits), torch.exp(logits - top))
    s = e.sum(1, keepdim=True)
    return torch.where(s == 0, torch.zeros_like(e), e / s)


def balance_backward(logits, counts, k, dloss, mask, coef):
    T, E = logits.shape
    V = int(counts[E])
    if V == 0:
        return torch.zeros_like(logits), torch.zeros_like(logits)
    live = torch.ones(T, 1, dtype=torch.float64) if mask is None else mask.cpu().double()[:, None]
    p = softmax(logits)
    d = counts[:E].double() * E / (V * k)
    f = dloss * coef / V * live * p
    # d may be shifted by a constant; the kernel works with d - 1
    mag = abs(dloss * coef) / V * live * p * ((d - 1).abs() + (p * (d - 1).abs()).sum(1, keepdim=True))
    # The formula below subtracts numbers of size d, so in 64 bits it is itself off by up to (E + 4) 2^-53 of
    # |f| (d + sum p d) < 2^-40 of it for E <= 4096 (at an even load, d = 1, the true gradient is 0 and the formula gives
    # 1e-18). 2^-25 of that size times SLACK is 2^-40 of it.
    mag = mag + 2.0 ** -25 * f.abs() * (d + (p * d).sum(1, keepdim=True))
    return f * (d - (p * d).sum(1, keepdim=True)), mag


def q4(words, scales, biases, group, x):
    """(y, magnitude) of the 4-bit product."""
    rows = words.shape[0]
    w = words.cpu().long() & 0xFFFFFFFF
    q = torch.stack([(w >> (4 * i)) & 15 for i in range(8)], 2).reshape(rows, -1).double()
    s = scales.cpu().double().repeat_interleave(group, 1)
    if biases is None:
        W, M = s * (q - 8), (s * (q - 8)).abs()
    else:
        b = biases.cpu().double().repeat_interleave(group, 1)
        W, M = s * q + b, (s * (q - 8)).abs() + b.abs() + 8 * s.abs()
    return x @ W.T, x.abs() @ M.T


def q4_pair(g, mg, u, mu):
    """silu(g) u, and its magnitude from the products' (|silu'| <= 1.1)."""
    return g * torch.sigmoid(g) * u, 1.1 * mg * u.abs() + (g * torch.sigmoid(g)).abs() * mu
