"""The block operators with weights and arrays that change between calls."""
import os
import subprocess
import sys

import pytest
import torch

import vector_quantized_moe_b200 as vq
from helpers import lib_module, small_module
from test_gpu_block import make
from test_gpu_q4 import module, tokens

pytestmark = pytest.mark.gpu


def test_a_norm_with_other_weights():
    T, H = 3, 512
    g = torch.Generator().manual_seed(1)
    h = torch.randn((T, H), generator=g).cuda()
    ws = [(1 + 0.3 * torch.randn(H, generator=g)).cuda() for _ in range(3)]
    want = [vq.norm_pre(vq.Norm(w.clone()), h) for w in ws]
    p = torch.nn.Parameter(ws[0].clone())
    n = vq.Norm(p)
    got = [vq.norm_pre(n, h)]
    p.data = ws[1]
    got.append(vq.norm_pre(n, h))
    n.weight = ws[2]
    got.append(vq.norm_pre(n, h))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert torch.equal(vq.norm_post(h, torch.zeros_like(h), n)[0].bfloat16(), want[2])


def test_a_4_bit_module_with_other_arrays():
    (_, m), (_, other) = module(100, 256, 64, True, 2), module(100, 256, 64, True, 3)
    x = tokens(3, 256, 4)
    want = vq.q4_gemv(other, x)
    assert not torch.equal(vq.q4_gemv(m, x), want)
    m.words, m.scales, m.biases = other.words.clone(), other.scales.clone(), other.biases.clone()
    assert torch.equal(vq.q4_gemv(m, x), want)


def layer_of(E, H, I, seed):
    return vq.MoELayer(*[lib_module(small_module(E, r, c, 2, 8, seed=seed + i))
                         for i, (r, c) in enumerate(((I, H), (I, H), (H, I)))])


@pytest.mark.parametrize("T", [1, 8, 200, 700])
@pytest.mark.parametrize("path", ["decode", "prefill"])
@pytest.mark.parametrize("writer", ["pre", "post"])
def test_x_rewritten_by_the_call_before_the_experts(T, path, writer):
    # the experts read the x that the launch before them wrote over the one that the calls before that have read
    E, H, I, K = 8, 512, 256, 2
    layer, n = layer_of(E, H, I, 40), vq.Norm(torch.ones(H, device="cuda"))
    _, m = module(64, H, 64, False, 43)
    g = torch.Generator().manual_seed(44)
    hs = [torch.randn((T, H), generator=g).cuda() for _ in range(12)]
    logits = torch.randn((T, E), generator=g).cuda()
    zero = torch.zeros_like(hs[0])
    experts = getattr(layer, path)
    xs = [vq.norm_pre(n, h) for h in hs]
    want = []
    for x in xs:
        torch.cuda.synchronize()
        want.append((experts(x, logits, K), vq.q4_gemv(m, x)))
    x, got = torch.empty_like(xs[0]), []
    torch.cuda.synchronize()
    for h in hs:
        if writer == "pre":
            vq.norm_pre(n, h, out=x)
        else:
            vq.norm_post(zero, h, next=n, x_out=x)
        y = experts(x, logits, K)
        got.append((y, vq.q4_gemv(m, x)))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for p, q in zip(got, want) for a, b in zip(p, q))


FIRST_CALLS = """
import torch
import vector_quantized_moe_b200 as vq
T, H = 700, 256
g = torch.Generator().manual_seed(1)
h, y = torch.randn((T, H), generator=g).cuda(), torch.randn((T, H), generator=g).cuda()
d = torch.randn((T, H), generator=g).bfloat16().cuda()
n = vq.Norm(torch.ones(H, device="cuda"))
def run():
    ho, x = vq.norm_post(y, h, n, next=n)
    return (vq.norm_pre(n, h), ho, x, *vq.norm_pre_backward(n, h, d), *vq.norm_post_backward(y, ho, h, d, n, next=n))
torch.zeros(1, device="cuda")
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = run()
graph.replay()
torch.cuda.synchronize()
assert all(a is b or torch.equal(a, b) for a, b in zip(got, run()))
print("equal")
"""


def test_the_first_calls_of_a_process_can_be_captured():
    # what the launches ask the runtime once (registers, shared memory) is allowed during a capture
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "equal", r.stderr[-2000:]


@pytest.mark.parametrize("path", ["decode", "prefill"])
def test_blocks_of_unusual_rows(path):
    # no rows, windows of wider rows, bit patterns of bf16, another stream: the same bits as plain rows give
    block, _, _ = make(True, True, True)
    run = getattr(block, path)
    H = block.layer.hidden
    for T in (0, 1, 7):
        h = torch.randn((T, H), generator=torch.Generator().manual_seed(50 + T)).bfloat16().cuda()
        want = run(h)
        assert want[0].shape == want[1].shape == (T, H) and want[2].shape == (T, block.layer.E)
        wide = torch.full((T + 1, H + 24), 9.0, dtype=torch.bfloat16, device="cuda")
        wide[:T, 8:8 + H] = h
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            other = run(h)
        s.synchronize()
        for got in (run(wide[:T, 8:8 + H]), run(h.view(torch.int16)), run(h, vq.norm_pre(block.pre, h)), other):
            assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_gates_of_any_stride():
    T, H = 5, 256
    g = torch.Generator().manual_seed(60)
    y, h = torch.randn((T, H), generator=g).cuda(), torch.randn((T, H), generator=g).cuda()
    z = torch.randn((T, 9), generator=g).cuda()
    want = vq.norm_post(y, h, gate=z[:, 3].contiguous())[0]
    back = vq.norm_post_backward(y, want, h, gate=z[:, 3].contiguous())
    assert back[1].shape == (T,)
    for gate in (z[:, 3], z[:, 3:4], z.T.contiguous().T[:, 3], z[:, 3].contiguous()[:, None]):
        assert torch.equal(vq.norm_post(y, h, gate=gate)[0], want)
        got = vq.norm_post_backward(y, want, h, gate=gate)
        assert got[1].shape == gate.shape and got[1].is_contiguous()
        assert torch.equal(got[1].reshape(T), back[1]) and torch.equal(got[0], back[0])
    flipped = z.flip(0)[:, 3]
    assert torch.equal(vq.norm_post(y, h, gate=flipped)[0], vq.norm_post(y, h, gate=flipped.contiguous())[0])
