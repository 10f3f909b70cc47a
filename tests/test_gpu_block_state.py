"""The block operators with weights and arrays that change between calls."""
import pytest
import torch

import vector_quantized_moe_b200 as vq
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
