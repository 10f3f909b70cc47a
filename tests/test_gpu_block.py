"""The block operators together: norm -> router -> experts and 4-bit shared expert -> gate -> norm, residual, next norm,
then the router's balance loss, as a decode step and as a prompt, against the oracle's experts and the definitions."""
import numpy as np
import pytest
import torch

import block_ref as br
import oracle
import vector_quantized_moe_b200 as vq
from helpers import lib_module, oracle_module, small_module
from test_gpu_q4 import module as q4_module

pytestmark = pytest.mark.gpu

E, K, H, I, S = 8, 3, 1024, 512, 384
EPS = 1e-6


def make(post, gate, next_, res_scale=1.0, out_scale=1.0):
    mds = [small_module(E, I, H, 4, 9, seed=1), small_module(E, I, H, 4, 9, seed=2), small_module(E, H, I, 2, 8, seed=3)]
    g = torch.Generator().manual_seed(4)
    w = lambda: vq.Norm((1 + 0.2 * torch.randn(H, generator=g)).to(torch.bfloat16).cuda(), EPS)  # noqa: E731
    wr = (torch.randn((E, H), generator=g) / H ** 0.5).cuda()
    wg = (torch.randn((1, H), generator=g) / H ** 0.5).cuda()
    raw = [q4_module(S, H, 64, True, 5), q4_module(S, H, 64, True, 6), q4_module(H, S, 32, False, 7)]
    block = vq.MoEBlock(vq.MoELayer(*[lib_module(m) for m in mds]), w(), lambda x: x.float() @ wr.T, K,
                        post=w() if post else None, next=w() if next_ else None, shared=[m for _, m in raw],
                        shared_gate=(lambda x: x.float() @ wg.T) if gate else None, res_scale=res_scale,
                        out_scale=out_scale)
    return block, [oracle_module(m) for m in mds], [r for r, _ in raw]


def stream(T, seed, dtype=torch.float32):
    return torch.randn((T, H), generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


@pytest.mark.parametrize("T,prefill", [(1, False), (6, False), (40, True)])
@pytest.mark.parametrize("post,gate,next_,scales", [(False, True, True, (1.0, 1.0)), (True, False, True, (0.75, 0.5)),
                                                    (True, True, False, (1.0, 1.0))])
def test_block(T, prefill, post, gate, next_, scales):
    block, experts, raw = make(post, gate, next_, *scales)
    h = stream(T, 10 + T)
    ho, xo, logits = (block.prefill if prefill else block.decode)(h)
    # the block's x, and everything after it from that x
    x = vq.norm_pre(block.pre, h)
    br.check("x", x, *br.norm(br.d64(h), br.d64(block.pre.weight), 0.0, EPS))
    y = torch.from_numpy(oracle.moe(*experts, x.view(torch.int16).cpu().numpy().view(np.uint16), logits.cpu().numpy(), K))
    act, mact = br.q4_pair(*br.q4(*raw[0], 64, br.d64(x)), *br.q4(*raw[1], 64, br.d64(x)))
    s, _ = br.q4(*raw[2], 32, act)
    _, ms = br.q4(*raw[2], 32, br.BF16_STEP * act.abs() + br.SLACK * mact)   # the activation's own error through W
    z = 1.0 if block.shared_gate is None else torch.sigmoid(br.d64(block.shared_gate(x)))
    total = y + z * s
    # y is within the layer's bar (relative L2 2e-3), s within its activation's rounding and its own (bf16)
    err = 2e-3 * float(y.norm()) + float((ms + br.BF16_STEP * s.abs()).norm())
    v = total
    if post:   # a norm's relative L2 error: that of its argument, once in the row and once in its scale
        v, _ = br.norm(total, br.d64(block.post.weight), 0.0, EPS)
        err = 2 * err / float(total.norm(dim=1).min()) * float(v.norm())
    want = scales[0] * br.d64(h) + scales[1] * v
    got = br.d64(ho)
    assert float((got - want).norm()) <= scales[1] * err + br.SLACK * float(want.norm())
    if next_:
        br.check("next x", xo, *br.norm(got, br.d64(block.next.weight), 0.0, EPS))
    else:
        assert xo is None
    # the router's loss over the same logits and choices
    ids = vq.route(logits, K)[0]
    loss, counts, probs = vq.balance_loss(logits, ids, None, 0.01)
    rl, rc, rp = br.balance(br.d64(logits), ids.cpu(), None, 0.01)
    br.check("loss", loss, rl, rl.abs())
    assert torch.equal(counts.cpu().long(), rc)
    d = vq.balance_loss_backward(logits, counts, K, None, None, 0.01)
    br.check("dlogits", d, *br.balance_backward(br.d64(logits), rc, K, 1.0, None, 0.01))


def test_blocks_chain_through_the_next_norm():
    a, _, _ = make(True, True, True)
    b, _, _ = make(True, True, True)
    b.pre = a.next
    h = stream(4, 30, torch.bfloat16)
    h1, x1, _ = a.decode(h)
    fused = b.decode(h1, x1)
    plain = b.decode(h1)
    assert all(torch.equal(p, q) for p, q in zip(fused, plain))


def test_decode_step_captured_and_replayed():
    block, _, _ = make(True, True, True)
    h = stream(3, 31, torch.bfloat16)
    block.decode(h)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = block.decode(h)
    for seed in (32, 33):
        h.copy_(stream(3, seed, torch.bfloat16))
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in out]
        assert all(torch.equal(p, q) for p, q in zip(got, block.decode(h)))


def test_hidden_sizes_are_checked():
    block, _, _ = make(False, False, False)
    with pytest.raises(vq.VQError):
        vq.MoEBlock(block.layer, vq.Norm(torch.ones(H + 8, device="cuda")), block.router, K)
