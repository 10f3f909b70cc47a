"""Refusals of the block operators, through the C ABI and the binding. Nothing here reaches a GPU: every call fails its
checks, or is an empty batch that launches nothing."""
import ctypes

import pytest
import torch

import vector_quantized_moe_b200 as vq

ARG, ALIGN, UNSUPPORTED, WORKSPACE = 1, 2, 3, 4
NAN = float("nan")


def norm(hidden=64, dtype=1, weight=4096, eps=1e-6, offset=0.0):
    return vq.vq_norm(hidden, dtype, weight, eps, offset)


def pre(n=None, h=8192, hd=1, hl=64, T=4, x=16384, xl=64):
    n = norm() if n is None else n
    return vq._L().vq_norm_pre(ctypes.byref(n), h, hd, hl, T, x, xl, None)


@pytest.mark.parametrize("kw,status", [
    (dict(n=norm(hidden=0)), ARG), (dict(n=norm(hidden=16385), hl=16385, xl=16385), UNSUPPORTED),
    (dict(n=norm(weight=None)), ARG), (dict(n=norm(dtype=2)), ARG), (dict(n=norm(eps=-1.0)), ARG),
    (dict(n=norm(eps=NAN)), ARG), (dict(n=norm(offset=NAN)), ARG), (dict(n=norm(weight=4097)), ALIGN),
    (dict(h=None), ARG), (dict(x=None), ARG), (dict(T=-1), ARG), (dict(hd=5), ARG), (dict(hl=63), ARG),
    (dict(xl=0), ARG), (dict(h=8193), ALIGN), (dict(hd=0, h=8194), ALIGN), (dict(T=0, h=None, x=None), 0),
])
def test_norm_pre(kw, status):
    assert pre(**kw) == status
    assert vq._L().vq_norm_pre(None, 8192, 1, 64, 4, 16384, 64, None) == ARG


def test_norm_workspace_size():
    f = vq._L().vq_norm_workspace_size
    assert f(0, 4) == 0 and f(16385, 4) == 0 and f(64, -1) == 0
    assert f(64, 1) == 0 < f(64, 2) < f(64, 100) <= f(64, 1 << 30)


def pre_bwd(n=None, h=8192, hl=64, dx=16384, dxl=64, dres=None, dresl=0, T=8, dh=32768, dhl=64, dw=65536, ws=1 << 20,
            nws=1 << 30):
    n = norm() if n is None else n
    return vq._L().vq_norm_pre_backward(ctypes.byref(n), h, 1, hl, dx, dxl, dres, dresl, T, dh, dhl, dw, ws, nws, None)


@pytest.mark.parametrize("kw,status", [
    (dict(h=None), ARG), (dict(dx=None), ARG), (dict(dh=None), ARG), (dict(dres=8192, dresl=10), ARG),
    (dict(dxl=10), ARG), (dict(dhl=1), ARG), (dict(dw=65537), ALIGN), (dict(dx=16385), ALIGN),
    (dict(ws=None), WORKSPACE), (dict(ws=(1 << 20) + 16), WORKSPACE), (dict(nws=10), WORKSPACE),
    (dict(T=0, h=None, dx=None, dh=None, dw=None, ws=None), 0),
])
def test_norm_pre_backward(kw, status):
    assert pre_bwd(**kw) == status


def post(p=None, n=None, hidden=64, y=8192, yd=0, yl=64, gate=None, gd=1, gc=1, gl=1, h=16384, hd=1, hl=64, a=1.0, b=1.0,
         T=4, ho=32768, hol=64, x=None, xl=64):
    r = lambda v: None if v is None else ctypes.byref(v)  # noqa: E731
    return vq._L().vq_norm_post(r(p), r(n), hidden, y, yd, yl, gate, gd, gc, gl, h, hd, hl, a, b, T, ho, hol, x, xl, None)


@pytest.mark.parametrize("kw,status", [
    (dict(p=norm(hidden=32)), ARG), (dict(n=norm(hidden=128), x=65536), ARG), (dict(n=norm()), ARG),
    (dict(x=65536), ARG), (dict(hidden=0), ARG), (dict(hidden=20000, yl=20000, hl=20000, hol=20000), UNSUPPORTED),
    (dict(y=None), ARG), (dict(h=None), ARG), (dict(ho=None), ARG), (dict(yd=3), ARG), (dict(hd=-1), ARG),
    (dict(gate=4096, gc=2), ARG), (dict(gate=4096, gc=64, gl=8), ARG), (dict(gate=4096, gd=9), ARG),
    (dict(gate=4097), ALIGN), (dict(a=NAN), ARG), (dict(b=float("inf")), ARG), (dict(yl=4), ARG), (dict(hol=4), ARG),
    (dict(T=-2), ARG), (dict(y=8194), ALIGN), (dict(T=0, y=None, h=None, ho=None), 0),
])
def test_norm_post(kw, status):
    assert post(**kw) == status


def post_bwd(p=None, n=None, y=8192, gate=None, gc=1, ho=16384, T=8, dho=32768, dholl=64, dx=None, dy=65536, dyl=64,
             dgate=None, dh=131072, dp=None, dn=None, ws=1 << 20, nws=1 << 30, hd=1):
    r = lambda v: None if v is None else ctypes.byref(v)  # noqa: E731
    return vq._L().vq_norm_post_backward(r(p), r(n), 64, y, 0, 64, gate, 1, gc, gc, ho, hd, 64, 1.0, 1.0, T, dho, dholl,
                                         dx, 64, dy, dyl, dgate, gc, dh, 64, dp, dn, ws, nws, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dgate=4096), ARG), (dict(dp=4096), ARG), (dict(dn=4096), ARG), (dict(dx=4096), ARG), (dict(n=norm()), ARG),
    (dict(n=norm(), dx=4096, ho=None), ARG), (dict(y=None), ARG), (dict(dy=None), ARG), (dict(dyl=3), ARG),
    (dict(dholl=3), ARG), (dict(hd=7), ARG), (dict(p=norm(), dp=4098), ALIGN), (dict(p=norm(), dp=4096, ws=None), WORKSPACE),
    (dict(p=norm(), dp=4096, nws=8), WORKSPACE), (dict(gate=4096, gc=3), ARG),
    (dict(T=0, y=None, dy=None, dh=None, dho=None), 0),
])
def test_norm_post_backward(kw, status):
    assert post_bwd(**kw) == status


def loss(logits=4096, ids=8192, mask=None, T=100, E=16, k=2, coef=1.0, loss=16384, counts=20480, probs=24576, ws=1 << 20,
         nws=1 << 30):
    return vq._L().vq_balance_loss(logits, ids, mask, T, E, k, coef, loss, counts, probs, ws, nws, None)


@pytest.mark.parametrize("kw,status", [
    (dict(E=0), ARG), (dict(E=4097), ARG), (dict(k=0), ARG), (dict(k=17), ARG), (dict(E=64, k=33), ARG), (dict(T=-1), ARG),
    (dict(T=1 << 30, k=2), ARG), (dict(logits=None), ARG), (dict(ids=None), ARG), (dict(loss=None), ARG),
    (dict(counts=None), ARG), (dict(probs=None), ARG), (dict(coef=NAN), ARG), (dict(logits=4098), ALIGN),
    (dict(ids=8193), ALIGN), (dict(probs=24578), ALIGN), (dict(ws=None), WORKSPACE), (dict(ws=100), WORKSPACE),
    (dict(nws=64), WORKSPACE),
])
def test_balance_loss(kw, status):
    assert loss(**kw) == status


def test_balance_workspace_size():
    f = vq._L().vq_balance_workspace_size
    assert f(64, 512) == 0 and 0 < f(65, 512) == f(1 << 20, 512) and f(65, 4097) == 0 and f(-1, 8) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(E=0), ARG), (dict(k=17), ARG), (dict(logits=None), ARG), (dict(counts=None), ARG), (dict(out=None), ARG),
    (dict(coef=float("inf")), ARG), (dict(dloss=4097), ALIGN), (dict(out=16386), ALIGN),
    (dict(T=0, logits=None, counts=None, out=None), 0),
])
def test_balance_backward(kw, status):
    a = dict(dict(logits=4096, counts=8192, T=4, E=16, k=2, coef=1.0, dloss=None, out=16384), **kw)
    assert vq._L().vq_balance_loss_backward(a["logits"], a["counts"], None, a["T"], a["E"], a["k"], a["coef"], a["dloss"],
                                            a["out"], None) == status


def q4m(rows=64, cols=128, group=64, words=4096, scales=8192, biases=None):
    return vq.vq_q4_module(rows, cols, group, words, scales, biases)


@pytest.mark.parametrize("kw,status", [
    (dict(m=q4m(rows=0)), ARG), (dict(m=q4m(cols=96)), ARG), (dict(m=q4m(group=16)), ARG), (dict(m=q4m(words=None)), ARG),
    (dict(m=q4m(scales=None)), ARG), (dict(m=q4m(words=4100)), ALIGN), (dict(m=q4m(biases=8200)), ALIGN),
    (dict(up=q4m(rows=32)), ARG), (dict(up=q4m(group=128)), ARG), (dict(up=q4m(biases=8192)), ARG),
    (dict(x=None), ARG), (dict(y=None), ARG), (dict(T=-1), ARG), (dict(T=(1 << 20) + 1), UNSUPPORTED), (dict(yd=4), ARG),
    (dict(T=16 * 65535 + 1), UNSUPPORTED),
    (dict(xl=64), ARG), (dict(yl=8), ARG), (dict(x=16392), ALIGN), (dict(xl=132), ALIGN), (dict(y=32770, yd=0), ALIGN),
    (dict(y=32769), ALIGN), (dict(T=0, x=None, y=None), 0),
])
def test_q4_gemv(kw, status):
    a = dict(dict(m=q4m(), up=None, x=16384, xl=128, T=4, y=32768, yd=1, yl=64), **kw)
    up = None if a["up"] is None else ctypes.byref(a["up"])
    assert vq._L().vq_q4_gemv(ctypes.byref(a["m"]), up, a["x"], a["xl"], a["T"], a["y"], a["yd"], a["yl"], None) == status


def test_q4_pack_and_sizes():
    L = vq._L()
    assert L.vq_q4_packed_words(17, 160) == 2 * 2 * 256 and L.vq_q4_packed_scales(17, 160, 32) == 2 * 2 * 16 * 4
    assert L.vq_q4_packed_words(0, 64) == 0 and L.vq_q4_packed_words(4, 48) == 0
    assert L.vq_q4_packed_scales(4, 64, 128) == 0 and L.vq_q4_packed_scales(4, 64, 48) == 0
    ok = dict(codes=4096, scales=8192, biases=None, rows=4, cols=64, group=64, w=16384, s=32768, b=None)

    def call(**kw):
        a = dict(ok, **kw)
        return L.vq_q4_pack(a["codes"], a["scales"], a["biases"], a["rows"], a["cols"], a["group"], a["w"], a["s"], a["b"],
                            None)
    assert call(codes=None) == ARG and call(biases=4096) == ARG and call(b=4096) == ARG and call(group=8) == ARG
    assert call(cols=40) == ARG and call(w=16388) == ALIGN and call(codes=4097) == ALIGN


# ---------------------------------------------------------------- the binding's own checks (CPU tensors)

def t(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def refused(f, *a, **k):
    with pytest.raises(vq.VQError) as e:
        f(*a, **k)
    assert e.value.status == ARG


def test_binding_refuses_wrong_tensors():
    n = vq.Norm(t(64))
    refused(vq.Norm, t(64, dtype=torch.float16))
    refused(vq.Norm, t(8, 8))
    refused(vq.norm_pre, n, t(4, 64))                                   # not on a GPU
    refused(vq.norm_pre, n, t(4, 32))
    refused(vq.norm_pre, n, t(4, 64, dtype=torch.float16))
    refused(vq.norm_pre, n, t(64, 4).T)                                 # columns not consecutive
    refused(vq.norm_pre, n, t(1, 64).expand(4, 64))                     # one row for all
    refused(vq.norm_pre, n, t(4, 64), out=t(4, 64, dtype=torch.float32))
    refused(vq.norm_pre_backward, n, t(4, 64), t(3, 64))
    refused(vq.norm_pre_backward, n, t(4, 64), t(4, 64), dres=t(4, 64, dtype=torch.float32))
    refused(vq.norm_post, t(4, 64), t(4, 64), vq.Norm(t(32)))
    refused(vq.norm_post, t(4, 64), t(4, 64), gate=t(4, 3))
    refused(vq.norm_post, t(4, 64), t(4, 64), gate=t(5))
    refused(vq.norm_post, t(4, 64), t(4, 64), x_out=t(4, 64))
    refused(vq.norm_post_backward, t(4, 64), t(4, 64), t(4, 64), t(4, 64))
    refused(vq.norm_post_backward, t(4, 64), t(4, 64), t(4, 64), next=n)
    refused(vq.balance_loss, t(4, 8), t(4, 2, dtype=torch.int32))
    refused(vq.balance_loss, t(4, 8, dtype=torch.float32), t(4, 2, dtype=torch.int64))
    refused(vq.balance_loss, t(4, 8, dtype=torch.float32), t(3, 2, dtype=torch.int32))
    refused(vq.balance_loss, t(4, 8, dtype=torch.float32), t(4, 2, dtype=torch.int32), t(4, dtype=torch.float32))
    refused(vq.balance_loss, t(4, 8, dtype=torch.float32), t(4, 2, dtype=torch.int32))
    refused(vq.balance_loss_backward, t(4, 8, dtype=torch.float32), t(8, dtype=torch.int32), 2)
    refused(vq.balance_loss_backward, t(4, 8, dtype=torch.float32), t(9, dtype=torch.int32), 2, t(2, dtype=torch.float32))
    refused(vq.Q4Module.from_rows, t(4, 8), t(4, 1, dtype=torch.float16))
    refused(vq.Q4Module.from_rows, t(4, 8, dtype=torch.int32), t(4, 2, dtype=torch.float16))
    refused(vq.Q4Module.from_rows, t(4, 8, dtype=torch.int32), t(4, 1, dtype=torch.float16), group=48)
    refused(vq.Q4Module.from_rows, t(4, 8, dtype=torch.int32), t(4, 1, dtype=torch.float16))
    m = vq.Q4Module(64, 64, 64, t(256, dtype=torch.int32), t(16, dtype=torch.int16))
    refused(vq.q4_gemv, m, t(2, 32))
    refused(vq.q4_gemv, m, t(2, 64))
    refused(vq.q4_gemv, m, t(2, 64), out_dtype=torch.float32, out=t(2, 64))
    refused(vq.q4_gemv, m, t(2, 64), out=t(2, 60))


def test_workspaces_too_small_or_scattered():
    like = t(1)
    room = t(1024, dtype=torch.uint8)
    for first in range(0, 257, 16):   # fewer bytes than to the next 256-byte boundary: none are usable, never less
        _, at, n = vq._workspace(64, room[first:first + 8], like)
        assert at % 256 == 0 and 0 <= n <= 8
    refused(vq._workspace, 64, room[:1].expand(1 << 20), like)
    refused(vq._workspace, 64, room[::2], like)
