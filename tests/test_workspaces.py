"""Workspaces that the caller gives: none is taken for larger than it is. CPU tensors; the calls that would launch are
recorded instead, except those that the library refuses."""
import types

import pytest
import torch

import vector_quantized_moe_b200 as vq
from helpers import lib_module, small_module

ARG, WORKSPACE = 1, 4
E, K, H, I, T = 8, 2, 512, 256, 3
STREAM = types.SimpleNamespace(cuda_stream=0)

room = torch.zeros(4096, dtype=torch.uint8)
START = -room.data_ptr() % 256   # of the first 256-byte boundary in room


def short_views():
    """Views with less than 512 bytes behind their first 256-byte boundary, and views that are no buffer at all."""
    yield "ends before its first boundary", room[START + 1:START + 33]
    yield "one byte", room[START + 8:START + 9]
    yield "empty", room[:0]
    yield "a boundary and 16 bytes", room[START:START + 16]
    yield "one byte for many", room[:1].expand(1 << 30)
    yield "every second byte", torch.zeros(1 << 22, dtype=torch.uint8)[::2]


VIEWS = dict(short_views())


class Recorder:
    """The library, except that the calls that would launch record their arguments and succeed."""

    def __init__(self, lib, names):
        self.lib, self.names, self.made = lib, names, []

    def __getattr__(self, name):
        if name not in self.names:
            return getattr(self.lib, name)
        return lambda *a: self.made.append((name, a)) or 0


# where a call's workspace pointer and its bytes are among the library's arguments
PLACES = {"vq_moe_decode": 8, "vq_moe_prefill": 8, "vq_moe_prefill_chunked": 9, "vq_gemm": 7, "vq_fit": 12,
          "vq_norm_pre_backward": 12, "vq_norm_post_backward": 28, "vq_balance_loss": 10}


@pytest.fixture
def lib(monkeypatch):
    vq.Norm(torch.ones(8))
    rec = Recorder(vq._L(), (*PLACES, "vq_moe_check"))
    monkeypatch.setattr(vq, "_lib_handle", rec)
    monkeypatch.setattr(vq, "_one_device", lambda *a: 0)
    monkeypatch.setattr(vq, "_device", lambda: 0)
    monkeypatch.setattr(vq, "_raw_stream", lambda dev: 0)
    return rec


@pytest.fixture(scope="module")
def layer():
    return vq.MoELayer(*[lib_module(small_module(E, r, c, 2, 8, seed=i), device="cpu")
                         for i, (r, c) in enumerate(((I, H), (I, H), (H, I)))])


def calls(layer):
    x, logits = torch.zeros((T, H), dtype=torch.bfloat16), torch.zeros((T, E))
    i32 = lambda *n: torch.zeros(n, dtype=torch.int32)  # noqa: E731
    n = vq.Norm(torch.ones(H))
    return {
        "decode": lambda ws: layer.decode(x, logits, K, workspace=ws, stream=STREAM),
        "prefill": lambda ws: layer.prefill(x, logits, K, workspace=ws, stream=STREAM),
        "prefill_chunked": lambda ws: layer.prefill_chunked(x, logits, K, workspace=ws, stream=STREAM),
        "gemm": lambda ws: vq.gemm(layer.gate, 0, x, workspace=ws, stream=STREAM),
        "fit": lambda ws: vq.fit(torch.zeros((16, 256), dtype=torch.int16), 4, 16, i32(64), i32(16), 2, workspace=ws,
                                 stream=STREAM),
        "norm_pre_backward": lambda ws: vq.norm_pre_backward(n, x, x, workspace=ws),
        "norm_post_backward": lambda ws: vq.norm_post_backward(x, x, x, post=n, workspace=ws),
        "balance_loss": lambda ws: vq.balance_loss(torch.zeros((100, 64)), i32(100, 2), workspace=ws),
    }


CALLS = ("decode", "prefill", "prefill_chunked", "gemm", "fit", "norm_pre_backward", "norm_post_backward", "balance_loss")


@pytest.mark.parametrize("view", VIEWS)
@pytest.mark.parametrize("call", CALLS)
def test_no_more_bytes_than_the_tensor_has(layer, lib, call, view):
    ws = VIEWS[view]
    try:
        calls(layer)[call](ws)
    except vq.VQError as e:
        assert e.status in (ARG, WORKSPACE) and not lib.made
        return
    (name, a), = lib.made
    at, n = a[PLACES[name]:PLACES[name] + 2]
    assert ws.is_contiguous() and at % 256 == 0
    assert 0 <= n <= ws.numel() * ws.element_size()
    assert n == 0 or ws.data_ptr() <= at and at + n <= ws.data_ptr() + ws.numel() * ws.element_size()


@pytest.mark.parametrize("call", CALLS)
def test_bytes_not_elements_and_one_device(layer, lib, call):
    run = calls(layer)[call]
    ws = torch.zeros(1 << 16, dtype=torch.int64)
    run(ws)
    (name, a), = lib.made
    at, n = a[PLACES[name]:PLACES[name] + 2]
    assert at == (ws.data_ptr() + 255) // 256 * 256 and at + n == ws.data_ptr() + (8 << 16)
    with pytest.raises(vq.VQError):   # on another device than the call's tensors
        run(types.SimpleNamespace(is_contiguous=lambda: True, get_device=lambda: 5, data_ptr=lambda: 4096,
                                  numel=lambda: 1 << 30, element_size=lambda: 1))
    assert len(lib.made) == 1


@pytest.mark.parametrize("view", VIEWS)
def test_error_word(lib, view):
    ws = VIEWS[view]
    try:
        vq.fit_check(ws, stream=STREAM)
    except vq.VQError as e:
        assert e.status in (ARG, WORKSPACE) and not lib.made
        return
    (_, (at, _)), = lib.made
    assert ws.is_contiguous() and at % 256 == 0
    assert ws.data_ptr() <= at and at + 4 <= ws.data_ptr() + ws.numel()


def test_small_workspaces_are_refused_by_the_library(layer):
    x, logits = torch.zeros((T, H), dtype=torch.bfloat16), torch.zeros((T, E))
    for ws in (VIEWS["ends before its first boundary"], VIEWS["a boundary and 16 bytes"]):
        with pytest.raises(vq.VQError) as e:
            layer.decode(x, logits, K, workspace=ws, stream=STREAM)
        assert e.value.status == WORKSPACE
