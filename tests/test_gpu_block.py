"""The block operators together: norm -> router -> experts and 4-bit shared expert -> gate -> norm, residual, next norm,
then the router's balance loss, as a decode step and as a prompt, against the oracle's experts and the definitions."""
import types

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


def test_small_workspace_is_refused():
    n = vq.Norm(torch.ones(H, device="cuda"))
    h = stream(8, 40, torch.bfloat16)
    room = torch.empty(4096, dtype=torch.uint8, device="cuda")
    for ws in (room[128:130], room[:0], room[:1].expand(1 << 20)):
        with pytest.raises(vq.VQError):
            vq.norm_pre_backward(n, h, h, workspace=ws)


def test_stream_of_another_device_is_refused():
    h = stream(2, 41)
    with pytest.raises(vq.VQError):
        vq.norm_pre(vq.Norm(torch.ones(H, device="cuda")), h, stream=types.SimpleNamespace(device_index=1))


def test_weights_outlive_a_call_on_another_stream():
    # a weight given up right after the call may not be handed out again before the call has run
    h, s, last = stream(4096, 42), torch.cuda.Stream(), torch.cuda.Event()
    want = vq.norm_pre(vq.Norm(torch.full((H,), 2.0, device="cuda")), h)
    torch.cuda.synchronize()
    w = torch.full((H,), 2.0, device="cuda")
    n = vq.Norm(w)
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(20):
            torch.mm(h, h.T)   # work ahead of the call on its stream
    got = vq.norm_pre(n, h, stream=s)
    last.record(s)
    del n, w
    others = [torch.full((H,), 3.0, device="cuda") for _ in range(64)]
    last.synchronize()
    assert torch.equal(got, want) and len(others) == 64


def test_router_and_x_are_checked():
    block, _, _ = make(False, False, False)
    h = stream(3, 43)
    x = vq.norm_pre(block.pre, h)
    router = block.router
    for wrong in (lambda v: router(v).to(torch.bfloat16), lambda v: router(v)[:, :4], lambda v: router(v)[:2],
                  lambda v: router(v).T.contiguous().T, lambda v: router(v).cpu()):
        block.router = wrong
        with pytest.raises(vq.VQError):
            block.decode(h)
    block.router = router
    for wrong in (x[:2], x.float(), torch.zeros(3, 2 * H, dtype=torch.bfloat16, device="cuda")[:, :H]):
        with pytest.raises(vq.VQError):
            block.decode(h, wrong)
    assert torch.equal(block.decode(h)[0], block.decode(h, x)[0])


def test_two_graphs_and_a_larger_batch_share_nothing():
    # two captured steps replayed at once on two streams, after eager calls of other sizes have grown and gone
    block, _, _ = make(True, True, True)
    hs = [stream(2, 50, torch.bfloat16), stream(5, 51, torch.bfloat16)]
    want = [block.decode(h) for h in hs]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for h in hs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(block.decode(h))
        graphs.append(g)
    block.decode(stream(16, 52, torch.bfloat16))
    junk = [torch.full((1 << 20,), 255, dtype=torch.uint8, device="cuda") for _ in range(8)]
    streams = [torch.cuda.Stream() for _ in hs]
    torch.cuda.synchronize()
    for _ in range(10):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert len(junk) == 8
    for got, w in zip(outs, want):
        assert all(torch.equal(p, q) for p, q in zip(got, w))


def test_given_workspace_holds_the_error_word():
    block, _, _ = make(True, True, True)
    h = stream(4, 60, torch.bfloat16)
    ws = torch.empty(block.layer.workspace_size(4, K, vq.VQ_MODE_DECODE) + 256, dtype=torch.uint8, device="cuda")
    assert all(torch.equal(p, q) for p, q in zip(block.decode(h, workspace=ws), block.decode(h)))
    assert vq.fit_check(ws) == 0
