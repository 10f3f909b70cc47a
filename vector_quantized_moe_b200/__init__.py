"""Python binding of libvqmoe.so, the B200 (sm_100a) VQ-MoE expert-path library.

Argument marshalling only: every step of the path runs in the library's CUDA
kernels; PyTorch provides device memory and streams. The library is loaded on
first use; every call raises ImportError when it has not been built
(python -m vector_quantized_moe_b200.build). There is no fallback.

Names follow include/vq_moe.h.
"""
from __future__ import annotations

import ctypes
import functools
import os
import re
from typing import Optional

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libvqmoe.so")
HEADER_PATH = os.path.join(os.path.dirname(_HERE), "include", "vq_moe.h")

VQ_OK = 0
VQ_ERR_ARG, VQ_ERR_ALIGN, VQ_ERR_UNSUPPORTED, VQ_ERR_WORKSPACE, VQ_ERR_CUDA, VQ_ERR_DEVICE_CHECK = 1, 2, 3, 4, 5, 6
VQ_F32, VQ_BF16 = 0, 1
VQ_MODE_DECODE, VQ_MODE_PREFILL = 0, 1


class VQError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {_L().vq_status_str(status).decode()}")
        self.status = status


class vq_module(ctypes.Structure):
    _fields_ = [("E", ctypes.c_int32), ("rows", ctypes.c_int32), ("cols", ctypes.c_int32),
                ("d", ctypes.c_int32), ("bits", ctypes.c_int32),
                ("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("codebook", ctypes.c_void_p),
                ("live_bitmap", ctypes.c_void_p), ("live_rank", ctypes.c_void_p), ("live_rows", ctypes.c_int64),
                ("biases", ctypes.c_void_p)]


class vq_moe_layer(ctypes.Structure):
    _fields_ = [("gate", vq_module), ("up", vq_module), ("down", vq_module)]


class vq_norm(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int32), ("weight_dtype", ctypes.c_int32), ("weight", ctypes.c_void_p),
                ("eps", ctypes.c_float), ("weight_offset", ctypes.c_float)]


class vq_q4_module(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int32), ("cols", ctypes.c_int32), ("group", ctypes.c_int32),
                ("words", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("biases", ctypes.c_void_p)]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with `python -m vector_quantized_moe_b200.build`")
    lib = ctypes.CDLL(LIB_PATH)
    P, I32, SZ, I64, F = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t, ctypes.c_int64, ctypes.c_float
    MP = ctypes.POINTER(vq_module)
    LP = ctypes.POINTER(vq_moe_layer)
    NP, QP = ctypes.POINTER(vq_norm), ctypes.POINTER(vq_q4_module)
    sig = {
        "vq_status_str": (ctypes.c_char_p, [ctypes.c_int]),
        "vq_geometry_supported": (ctypes.c_int, [I32, I32]),
        "vq_packed_words": (SZ, [I64, I32, I32]),
        "vq_pack": (ctypes.c_int, [P, I32, I32, I32, I32, P, P, SZ, ctypes.POINTER(SZ)]),
        "vq_pack_scales": (ctypes.c_int, [P, I32, I32, I32, P, P, SZ, ctypes.POINTER(SZ)]),
        "vq_live_rank": (ctypes.c_int, [P, I32, I32, P]),
        "vq_unpack": (ctypes.c_int, [MP, I32, P, P]),
        "vq_dequant": (ctypes.c_int, [MP, I32, P, P]),
        "vq_gemv": (ctypes.c_int, [MP, I32, P, I32, P, I32, P]),
        "vq_gemm_workspace_size": (SZ, [MP, I32]),
        "vq_gemm": (ctypes.c_int, [MP, MP, I32, P, I32, P, P, P, SZ, P]),
        "vq_route": (ctypes.c_int, [P, I32, I32, I32, I32, P, P, P, P, P]),
        "vq_moe_workspace_size": (SZ, [LP, I32, I32, I32]),
        "vq_moe_decode": (ctypes.c_int, [LP, P, I32, P, I32, I32, P, I32, P, SZ, P]),
        "vq_moe_prefill": (ctypes.c_int, [LP, P, I32, P, I32, I32, P, I32, P, SZ, P]),
        "vq_moe_prefill_chunked": (ctypes.c_int, [LP, P, I32, P, I32, I32, I32, P, I32, P, SZ, P]),
        "vq_set_trace_events": (ctypes.c_int, [P, I32]),
        "vq_set_wait_limit": (ctypes.c_int, [I64]),
        "vq_moe_check": (ctypes.c_int, [P, P]),
        "vq_moe_decode_noalloc": (ctypes.c_int, [LP, P, I32, P, I32, I32, P, I32, P]),
        "vq_norm_pre": (ctypes.c_int, [NP, P, I32, I64, I32, P, I64, P]),
        "vq_norm_workspace_size": (SZ, [I32, I32]),
        "vq_norm_pre_backward": (ctypes.c_int, [NP, P, I32, I64, P, I64, P, I64, I32, P, I64, P, P, SZ, P]),
        "vq_norm_post": (ctypes.c_int, [NP, NP, I32, P, I32, I64, P, I32, I32, I64, P, I32, I64, F, F, I32, P, I64, P,
                                        I64, P]),
        "vq_norm_post_backward": (ctypes.c_int, [NP, NP, I32, P, I32, I64, P, I32, I32, I64, P, I32, I64, F, F, I32, P,
                                                 I64, P, I64, P, I64, P, I64, P, I64, P, P, P, SZ, P]),
        "vq_balance_workspace_size": (SZ, [I32, I32]),
        "vq_balance_loss": (ctypes.c_int, [P, P, P, I32, I32, I32, F, P, P, P, P, SZ, P]),
        "vq_balance_loss_backward": (ctypes.c_int, [P, P, P, I32, I32, I32, F, P, P, P]),
        "vq_q4_packed_words": (SZ, [I32, I32]),
        "vq_q4_packed_scales": (SZ, [I32, I32, I32]),
        "vq_q4_pack": (ctypes.c_int, [P, P, P, I32, I32, I32, P, P, P, P]),
        "vq_q4_gemv": (ctypes.c_int, [QP, QP, P, I64, I32, P, I32, I64, P]),
        "vq_fit_workspace_size": (SZ, [I32, I32]),
        "vq_fit": (ctypes.c_int, [P, I32, I32, I32, I32, P, I32, P, I32, P, P, P, P, SZ, P]),
    }
    for name, (res, args) in sig.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    return lib


_lib_handle = None


def _L():
    """The loaded libvqmoe.so (loads it on first use; raises ImportError if missing)."""
    global _lib_handle
    if _lib_handle is None:
        _lib_handle = _load()
    return _lib_handle


def header_functions() -> list:
    """Names of the functions include/vq_moe.h declares."""
    txt = open(HEADER_PATH).read()
    txt = re.sub(r"/\*.*?\*/", "", txt, flags=re.S)
    return sorted(set(re.findall(r"\b(vq_[a-z_0-9]+)\s*\(", txt)))


def _check(status: int, where: str):
    if status != VQ_OK:
        raise VQError(status, where)


def status_str(status: int) -> str:
    return _L().vq_status_str(status).decode()


def geometry_supported(d: int, bits: int) -> bool:
    return bool(_L().vq_geometry_supported(d, bits))


def packed_words(rows: int, ncode: int, bits: int) -> int:
    return int(_L().vq_packed_words(rows, ncode, bits))


# ------------------------------------------------------------------ host packing

def pack(codes: np.ndarray, bits: int, live_bitmap: Optional[np.ndarray] = None) -> np.ndarray:
    """Pack uint16 codes [E, rows, ncode] -> words [live rows, row_words] (vq_pack)."""
    c = np.ascontiguousarray(codes, dtype=np.uint16)
    if c.ndim == 2:
        c = c[None]
    E, rows, ncode = c.shape
    bm = None if live_bitmap is None else np.ascontiguousarray(live_bitmap, dtype=np.uint32)
    rw = packed_words(1, ncode, bits)
    out = np.zeros((E * rows, max(rw, 1)), dtype=np.uint32)
    n = ctypes.c_size_t(0)
    _check(_L().vq_pack(c.ctypes.data, E, rows, ncode, bits, None if bm is None else bm.ctypes.data,
                        out.ctypes.data, out.size, ctypes.byref(n)), "vq_pack")
    return out[: n.value]


def pack_scales(scales: np.ndarray, live_bitmap: Optional[np.ndarray] = None) -> np.ndarray:
    """Keep the live rows of fp16 scales [E, rows, ngroups] (vq_pack_scales)."""
    s = np.ascontiguousarray(scales, dtype=np.uint16)
    E, rows, ng = s.shape
    bm = None if live_bitmap is None else np.ascontiguousarray(live_bitmap, dtype=np.uint32)
    out = np.zeros((E * rows, ng), dtype=np.uint16)
    n = ctypes.c_size_t(0)
    _check(_L().vq_pack_scales(s.ctypes.data, E, rows, ng, None if bm is None else bm.ctypes.data,
                               out.ctypes.data, out.size, ctypes.byref(n)), "vq_pack_scales")
    return out[: n.value]


def live_rank(live_bitmap: np.ndarray, rows: int) -> np.ndarray:
    """Rank table [E, ceil(rows/32)] for a live bitmap (vq_live_rank)."""
    bm = np.ascontiguousarray(live_bitmap, dtype=np.uint32)
    out = np.zeros_like(bm)
    _check(_L().vq_live_rank(bm.ctypes.data, bm.shape[0], rows, out.ctypes.data), "vq_live_rank")
    return out


# ------------------------------------------------------------------ device side

def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


_torch_module = None


def _stream(stream=None) -> int:
    torch = _torch()
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _workspace(n, given, like):
    """(tensor, aligned pointer, bytes) of a workspace of n bytes for a call on `like`: the given one, which has to be
    one piece on like's device, or a new one. The bytes are those behind the aligned pointer, 0 when there are none."""
    ws = given if given is not None else like.new_empty(n + 256, dtype=_torch().uint8)
    if not ws.is_contiguous() or ws.get_device() != like.get_device():
        raise VQError(VQ_ERR_ARG, "workspace")
    base = ws.data_ptr()
    aligned = (base + 255) // 256 * 256
    return ws, aligned, max(0, ws.numel() * ws.element_size() - (aligned - base))


class Module:
    """One VQ module on the device (vq_module). Tensors are kept alive here."""

    def __init__(self, E, rows, cols, d, bits, codes, scales, codebook, live_bitmap=None, live_rank_t=None,
                 biases=None):
        self.E, self.rows, self.cols, self.d, self.bits = E, rows, cols, d, bits
        self.codes, self.scales, self.codebook = codes, scales, codebook
        self.live_bitmap, self.live_rank = live_bitmap, live_rank_t
        self.biases = biases

    @classmethod
    def from_host(cls, E, rows, cols, d, bits, words, scales, codebook, live_bitmap=None, device="cuda",
                  biases=None):
        """Upload packed words [live rows, row_words], fp16 scale bits [live rows, cols/64],
        fp16 codebook bits [2^bits, d], an optional live bitmap [E, ceil(rows/32)] and optional
        fp16 bias bits [live rows, cols/64] (the affine arm)."""
        torch = _torch()
        up = lambda a, dt: torch.from_numpy(np.ascontiguousarray(a).view(dt)).to(device)
        bm = rk = None
        if live_bitmap is not None:
            bm = up(live_bitmap.astype(np.uint32), np.int32)
            rk = up(live_rank(live_bitmap, rows), np.int32)
        return cls(E, rows, cols, d, bits, up(words.astype(np.uint32), np.int32), up(scales, np.int16),
                   up(codebook, np.int16), bm, rk, None if biases is None else up(biases, np.int16))

    def struct(self) -> vq_module:
        return vq_module(self.E, self.rows, self.cols, self.d, self.bits, _ptr(self.codes), _ptr(self.scales),
                         _ptr(self.codebook), _ptr(self.live_bitmap), _ptr(self.live_rank),
                         int(self.scales.shape[0]), _ptr(self.biases))


def unpack(m: Module, expert: int, stream=None):
    """Codes [rows, cols/d] (uint16 bits in an int16 tensor); dead rows 0xFFFF (vq_unpack)."""
    torch = _torch()
    out = torch.empty((m.rows, m.cols // m.d), dtype=torch.int16, device=m.codes.device)
    s = m.struct()
    _check(_L().vq_unpack(ctypes.byref(s), expert, out.data_ptr(), _stream(stream)), "vq_unpack")
    return out


def dequant(m: Module, expert: int, stream=None):
    """Dequantised weights [rows, cols] fp32 (vq_dequant)."""
    torch = _torch()
    out = torch.empty((m.rows, m.cols), dtype=torch.float32, device=m.codes.device)
    s = m.struct()
    _check(_L().vq_dequant(ctypes.byref(s), expert, out.data_ptr(), _stream(stream)), "vq_dequant")
    return out


def _dt(out_dtype):
    torch = _torch()
    return VQ_F32 if out_dtype == torch.float32 else VQ_BF16


def gemv(m: Module, expert: int, x, out_dtype=None, out=None, stream=None):
    """y [T, rows] = x [T, cols] (bf16) . W_expert^T (vq_gemv)."""
    torch = _torch()
    out_dtype = out_dtype or torch.float32
    T = x.shape[0]
    if out is None:
        out = torch.empty((T, m.rows), dtype=out_dtype, device=x.device)
    s = m.struct()
    _check(_L().vq_gemv(ctypes.byref(s), expert, x.data_ptr(), T, out.data_ptr(), _dt(out.dtype), _stream(stream)),
           "vq_gemv")
    return out


def gemm(m0: Module, expert: int, x, m1: Optional[Module] = None, workspace=None, stream=None):
    """The prefill path's tcgen05 GEMM for one expert (vq_gemm): y0 [T, rows] = x . W0_expert^T and,
    with m1, y1 = x . W1_expert^T (fp32). Returns (y0, y1 or None, workspace)."""
    torch = _torch()
    T = x.shape[0]
    y0 = torch.empty((T, m0.rows), dtype=torch.float32, device=x.device)
    y1 = torch.empty((T, m0.rows), dtype=torch.float32, device=x.device) if m1 is not None else None
    s0 = m0.struct()
    s1 = m1.struct() if m1 is not None else None
    n = int(_L().vq_gemm_workspace_size(ctypes.byref(s0), T))
    if n == 0:
        raise VQError(VQ_ERR_ARG, "vq_gemm_workspace_size")
    ws, aligned, nbytes = _workspace(n, workspace, x)
    _check(_L().vq_gemm(ctypes.byref(s0), None if s1 is None else ctypes.byref(s1), expert, x.data_ptr(), T,
                        y0.data_ptr(), _ptr(y1), aligned, nbytes, _stream(stream)), "vq_gemm")
    return y0, y1, ws


def route(logits, top_k: int, renorm: bool = True, stream=None):
    """(ids [T,k] int32, weights [T,k] fp32, offsets [E+1] int32, perm [T*k] int32) (vq_route)."""
    torch = _torch()
    T, E = logits.shape
    dev = logits.device
    ids = torch.empty((T, top_k), dtype=torch.int32, device=dev)
    w = torch.empty((T, top_k), dtype=torch.float32, device=dev)
    offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
    perm = torch.empty(T * top_k, dtype=torch.int32, device=dev)
    _check(_L().vq_route(logits.data_ptr(), T, E, top_k, int(bool(renorm)), ids.data_ptr(), w.data_ptr(),
                         offsets.data_ptr(), perm.data_ptr(), _stream(stream)), "vq_route")
    return ids, w, offsets, perm


def fit(w, d: int, K: int, sample, init, iters: int, workspace=None, stream=None):
    """Data-free VQ fit of one bf16 tensor w [rows, cols] (16-bit bit patterns on the device):
    (scales fp16 bits [rows, cols/64], codebook fp16 bits [K, d], codes uint16 [rows, cols/d] as
    int16 tensors) from `iters` Lloyd steps over the subvectors `sample` starting at the
    subvectors `init` (int32 device tensors) (vq_fit)."""
    torch = _torch()
    rows, cols = w.shape
    dev = w.device
    scales = torch.empty((rows, cols // 64), dtype=torch.int16, device=dev)
    codebook = torch.empty((K, d), dtype=torch.int16, device=dev)
    codes = torch.empty((rows, cols // d), dtype=torch.int16, device=dev)
    n = int(_L().vq_fit_workspace_size(K, d))
    if n == 0:
        raise VQError(1, "vq_fit_workspace_size")
    ws, aligned, nbytes = _workspace(n, workspace, w)
    _check(_L().vq_fit(w.data_ptr(), rows, cols, d, K, sample.data_ptr(), sample.numel(), init.data_ptr(), iters,
                       scales.data_ptr(), codebook.data_ptr(), codes.data_ptr(), aligned, nbytes, _stream(stream)),
           "vq_fit")
    return scales, codebook, codes, ws


def fit_check(workspace, stream=None) -> int:
    """Status of the error word of a vq_fit workspace returned by fit() (vq_moe_check)."""
    _, aligned, nbytes = _workspace(0, workspace, workspace)
    if nbytes < 4:
        raise VQError(VQ_ERR_WORKSPACE, "fit_check")
    return int(_L().vq_moe_check(aligned, _stream(stream)))


# ------------------------------------------------------------------ the block around the experts
#
# norm -> (router) -> experts and 4-bit shared expert -> gate, norm, residual, next norm, and the router's balance
# loss. bf16 arrays may be torch.bfloat16 or their int16 bit patterns; outputs are torch.bfloat16. Rows may be
# windows of wider arrays (a row stride), with consecutive elements inside a row. Every call checks its tensors
# (VQError with VQ_ERR_ARG) before it launches and runs on its tensors' device: on that device's current stream, or on
# `stream` when one is given (the outputs then belong to that stream). Given outputs may not overlap inputs unless said.
# torch's autograd does not see these calls: what they return carries no history, whatever the inputs require, and the
# gradients are calls of their own (*_backward).

_bf16 = _f32 = _codes = _device = _raw_stream = _empty_like = None


def _types():
    """Binds what the calls below use of torch once (they are on a decode step's host path)."""
    global _bf16, _f32, _codes, _device, _raw_stream, _empty_like
    torch = _torch()
    _bf16, _f32, _empty_like = torch.bfloat16, torch.float32, torch.empty_like
    _device, _raw_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream
    _codes = {torch.float32: VQ_F32, torch.bfloat16: VQ_BF16, torch.int16: VQ_BF16}


def _bad(where: str):
    raise VQError(VQ_ERR_ARG, where)


def _on_stream(stream, f, *args):
    """f(*args) with `stream` current: its outputs are allocated on it, its inputs (those of norms and modules too) are
    held until it has run."""
    torch = _torch()
    held = []
    for a in args:
        held += a._held() if isinstance(a, (Norm, Q4Module)) else [a]
    held = [t for t in held if isinstance(t, torch.Tensor) and t.is_cuda]
    if any(t.get_device() != stream.device_index for t in held):
        _bad(f.__name__ + " (stream of another device)")
    with torch.cuda.stream(stream):
        out = f(*args)
    for t in held:
        t.record_stream(stream)
    return out


def _launch(name, dev, *args):
    """Calls the library on device `dev` and its current stream."""
    fn = getattr(_lib_handle, name)
    if dev == _device():
        st = fn(*args, _raw_stream(dev))
    else:
        with _torch().cuda.device(dev):
            st = fn(*args, _raw_stream(dev))
    if st != VQ_OK:
        raise VQError(st, name)


def _row_arg(where, t, T, cols, like=None):
    """(pointer, dtype, row stride) of a [T, cols] array; VQError when t is not one. like: its required dtype code."""
    code = _codes.get(t.dtype)
    if code is None or (like is not None and code != like) or t.shape != (T, cols):
        _bad(where)
    if t.is_contiguous():
        return t.data_ptr(), code, cols
    ld, inner = t.stride()
    if (cols > 1 and inner != 1) or (T > 1 and ld < cols):
        _bad(where)
    return t.data_ptr(), code, ld


def _one_device(where, first, *others) -> int:
    """Index of the one GPU that all tensors (None: skipped) are on."""
    dev = first.get_device()
    if dev < 0:
        _bad(where + " (not on a GPU)")
    for t in others:
        if t is not None and t.get_device() != dev:
            _bad(where + " (tensors on different devices)")
    return dev


def _public(o):
    return {k: v for k, v in vars(o).items() if k[0] != "_"}


class Norm:
    """The weight of a root-mean-square norm (vq_norm): weight [hidden] fp32 or bf16; offset is 1 for checkpoints that
    store weight - 1. A call uses the weight as it is then: another one may be assigned, or new data to it."""

    def __init__(self, weight, eps: float = 1e-6, offset: float = 0.0):
        if _codes is None:
            _types()
        _L()
        self.weight = weight
        self._s = vq_norm(0, 0, None, eps, offset)
        self._ref = ctypes.byref(self._s)
        self._bind()

    def __setattr__(self, name, value):
        object.__setattr__(self, name, value)
        if name[0] != "_":
            self._at = None   # not bound

    def _bind(self):
        w = self.weight
        code = _codes.get(w.dtype)
        if code is None or w.dim() != 1 or w.numel() < 1 or not w.is_contiguous():
            _bad("Norm: weight")
        self.hidden, self._dtype = w.numel(), w.dtype
        self._s.hidden, self._s.weight_dtype, self._s.weight = self.hidden, code, w.data_ptr()
        self._at = w.data_ptr()

    def _now(self):
        """The struct of the weight as it is now."""
        w = self.weight
        if (w.data_ptr() != self._at or w.dtype is not self._dtype or w.numel() != self.hidden
                or not w.is_contiguous()):
            self._at = None
            self._bind()
        return self._ref

    def __reduce__(self):   # a copy has a struct of its own
        return type(self), (self.weight, self._s.eps, self._s.weight_offset), _public(self)

    def _held(self):
        return [self.weight]


def norm_pre(norm: Norm, h, out=None, stream=None):
    """x [T, hidden] bf16 = norm(h), the input of a block from the residual stream h (fp32 or bf16) (vq_norm_pre)."""
    if stream is not None:
        return _on_stream(stream, norm_pre, norm, h, out)
    ref, H, T = norm._now(), norm.hidden, h.shape[0]
    hp, hd, hl = _row_arg("norm_pre: h", h, T, H)
    dev = _one_device("norm_pre", h, norm.weight, out)
    if out is None:
        out = _empty(h, _bf16)
        xp, xl = out.data_ptr(), H
    else:
        xp, _, xl = _row_arg("norm_pre: out", out, T, H, VQ_BF16)
    _launch("vq_norm_pre", dev, ref, hp, hd, hl, T, xp, xl)
    return out


def _empty(like, dtype):
    """A new array of like's shape on its device, rows one after the other (like's own elements are consecutive in a
    row, so that empty_like either keeps them so or, for a window, makes them so; it takes half of new_empty's time)."""
    return _empty_like(like) if like.dtype is dtype else _empty_like(like, dtype=dtype)


@functools.lru_cache(maxsize=1024)
def _norm_ws(H, T):
    return int(_L().vq_norm_workspace_size(H, T))


def norm_pre_backward(norm: Norm, h, dx, dres=None, weight_grad: bool = True, workspace=None, stream=None):
    """(dh, dweight fp32 or None) of norm_pre for the gradient dx (bf16); dres: a gradient that reaches h past the
    norm, added to dh (vq_norm_pre_backward)."""
    if stream is not None:
        return _on_stream(stream, norm_pre_backward, norm, h, dx, dres, weight_grad, workspace)
    ref = norm._now()
    T, H = h.shape[0], norm.hidden
    hp, hd, hl = _row_arg("norm_pre_backward: h", h, T, H)
    xp, _, xl = _row_arg("norm_pre_backward: dx", dx, T, H, VQ_BF16)
    rp, rl = None, 0
    if dres is not None:
        rp, _, rl = _row_arg("norm_pre_backward: dres", dres, T, H, hd)
    dev = _one_device("norm_pre_backward", h, norm.weight, dx, dres, workspace)
    dh = _empty(h, _f32 if hd == VQ_F32 else _bf16)
    dw = wp = dp = None
    nb = 0
    if weight_grad:
        dw = _empty(norm.weight, _f32)
        dp = dw.data_ptr()
        nb = _norm_ws(H, T)
        if nb:
            workspace, wp, nb = _workspace(nb, workspace, h)
    _launch("vq_norm_pre_backward", dev, ref, hp, hd, hl, xp, xl, rp, rl, T, dh.data_ptr(), H, dp, wp, nb)
    return dh, dw


def _gate_arg(where, gate, T, H):
    """(pointer, dtype, columns, row stride) of gate logits [T], [T, 1] or [T, H]."""
    shape = gate.shape
    if len(shape) == 1:
        gate = gate.unsqueeze(1)
        cols = 1
    else:
        cols = shape[1] if len(shape) == 2 else 0
    if cols != 1 and cols != H:
        _bad(where)
    p, d, ld = _row_arg(where, gate, T, cols)
    return p, d, cols, ld


def _norm_ref(where, norm, H):
    ref = norm._now()
    if norm.hidden != H:
        _bad(where)
    return ref


def norm_post(y, h, post: Optional[Norm] = None, gate=None, res_scale: float = 1.0, out_scale: float = 1.0,
              next: Optional[Norm] = None, h_out=None, x_out=None, stream=None):
    """(h_out, x_out) of a block whose output is y [T, hidden] and whose residual stream is h:
    h_out = res_scale * h + out_scale * sigmoid(gate) * post(y) and x_out = next(h_out) in bf16 (None without next).
    gate: logits [T], [T, 1] or [T, hidden]. h_out may be h (vq_norm_post)."""
    if stream is not None:
        return _on_stream(stream, norm_post, y, h, post, gate, res_scale, out_scale, next, h_out, x_out)
    if _codes is None:
        _types()
        _L()
    if y.dim() != 2:
        _bad("norm_post: y")
    T, H = y.shape
    yp, yd, yl = _row_arg("norm_post: y", y, T, H)
    hp, hd, hl = _row_arg("norm_post: h", h, T, H)
    gp = pr = nr = xp = w1 = w2 = None
    gd = gc = gl = xl = 0
    if gate is not None:
        gp, gd, gc, gl = _gate_arg("norm_post: gate", gate, T, H)
    if post is not None:
        pr, w1 = _norm_ref("norm_post: post", post, H), post.weight
    if next is not None:
        nr, w2 = _norm_ref("norm_post: next", next, H), next.weight
    dev = _one_device("norm_post", y, h, gate, h_out, x_out, w1, w2)
    if next is not None:
        if x_out is None:
            x_out = _empty(h, _bf16)
            xp, xl = x_out.data_ptr(), H
        else:
            xp, _, xl = _row_arg("norm_post: x_out", x_out, T, H, VQ_BF16)
    elif x_out is not None:
        _bad("norm_post: x_out without next")
    if h_out is None:
        h_out = _empty(h, _f32 if hd == VQ_F32 else _bf16)
        op, ol = h_out.data_ptr(), H
    else:
        op, _, ol = _row_arg("norm_post: h_out", h_out, T, H, hd)
    _launch("vq_norm_post", dev, pr, nr, H, yp, yd, yl, gp, gd, gc, gl, hp, hd, hl, res_scale, out_scale, T, op, ol, xp, xl)
    return h_out, x_out


def norm_post_backward(y, h_out, dh_out, dx_out=None, post: Optional[Norm] = None, gate=None, res_scale: float = 1.0,
                       out_scale: float = 1.0, next: Optional[Norm] = None, workspace=None, stream=None):
    """(dy, dgate, dh, dpost, dnext) of norm_post from its y, gate and h_out and the gradients dh_out (may be None: 0)
    and dx_out (with next). Gradients of bf16 arrays are bf16, dpost and dnext fp32; None for what the call did not
    have (vq_norm_post_backward)."""
    if stream is not None:
        return _on_stream(stream, norm_post_backward, y, h_out, dh_out, dx_out, post, gate, res_scale, out_scale, next,
                          workspace)
    if _codes is None:
        _types()
        _L()
    if y.dim() != 2:
        _bad("norm_post_backward: y")
    T, H = y.shape
    yp, yd, yl = _row_arg("norm_post_backward: y", y, T, H)
    hp, hd, hl = _row_arg("norm_post_backward: h_out", h_out, T, H)
    if (dx_out is None) != (next is None):
        _bad("norm_post_backward: dx_out goes with next")
    ap = xp = gp = pr = nr = wp = w1 = w2 = dgate = dpost = dnext = zp = d1 = d2 = None
    al = xl = gd = gc = gl = nb = 0
    if dh_out is not None:
        ap, _, al = _row_arg("norm_post_backward: dh_out", dh_out, T, H, hd)
    if gate is not None:
        gp, gd, gc, gl = _gate_arg("norm_post_backward: gate", gate, T, H)
    if post is not None:
        pr, w1 = _norm_ref("norm_post_backward: post", post, H), post.weight
    if next is not None:
        nr, w2 = _norm_ref("norm_post_backward: next", next, H), next.weight
        xp, _, xl = _row_arg("norm_post_backward: dx_out", dx_out, T, H, VQ_BF16)
    dev = _one_device("norm_post_backward", y, h_out, gate, dh_out, dx_out, workspace, w1, w2)
    dy = _empty(y, _f32 if yd == VQ_F32 else _bf16)
    dh = _empty(h_out, _f32 if hd == VQ_F32 else _bf16)
    if gate is not None:
        dgate = _empty(gate, _f32 if gd == VQ_F32 else _bf16)
        zp = dgate.data_ptr()
    if post is not None:
        dpost = _empty(w1, _f32)
        d1 = dpost.data_ptr()
    if next is not None:
        dnext = _empty(w2, _f32)
        d2 = dnext.data_ptr()
    if post is not None or next is not None:
        nb = _norm_ws(H, T)
        if nb:
            workspace, wp, nb = _workspace(nb, workspace, y)
    _launch("vq_norm_post_backward", dev, pr, nr, H, yp, yd, yl, gp, gd, gc, gl, hp, hd, hl, res_scale, out_scale, T, ap,
            al, xp, xl, dy.data_ptr(), H, zp, gc, dh.data_ptr(), H, d1, d2, wp, nb)
    return dy, dgate, dh, dpost, dnext


def _mask_arg(where, mask, T):
    torch = _torch()
    if mask.dtype not in (torch.bool, torch.uint8) or mask.shape != (T,) or not mask.is_contiguous():
        _bad(where)
    return mask.data_ptr()


def _logits_arg(where, logits):
    if _codes is None:
        _types()
        _L()
    if logits.dtype is not _f32 or logits.dim() != 2 or not logits.is_contiguous():
        _bad(where)
    return logits.shape


@functools.lru_cache(maxsize=1024)
def _balance_ws(T, E):
    return int(_L().vq_balance_workspace_size(T, E))


def balance_loss(logits, ids, mask=None, coef: float = 1.0, workspace=None, stream=None):
    """(loss fp32 scalar, counts int32 [E + 1], probs fp32 [E]) of router logits [T, E] (fp32) and the ids [T, k]
    that route() chose: counts[e] pairs go to expert e, counts[E] tokens count (mask, bool or bytes [T], leaves others
    out), probs is the mean softmax, loss = coef * sum_e (E counts[e] / (counts[E] k)) probs[e] (vq_balance_loss)."""
    if stream is not None:
        return _on_stream(stream, balance_loss, logits, ids, mask, coef, workspace)
    torch = _torch()
    T, E = _logits_arg("balance_loss: logits", logits)
    if ids.dtype is not torch.int32 or ids.dim() != 2 or ids.shape[0] != T or not ids.is_contiguous():
        _bad("balance_loss: ids")
    mp = None if mask is None else _mask_arg("balance_loss: mask", mask, T)
    dev = _one_device("balance_loss", logits, ids, mask, workspace)
    loss = logits.new_empty(())
    probs = logits.new_empty(E)
    counts = ids.new_empty(E + 1)
    wp, nb = None, _balance_ws(T, E)
    if nb:
        workspace, wp, nb = _workspace(nb, workspace, logits)
    _launch("vq_balance_loss", dev, logits.data_ptr(), ids.data_ptr(), mp, T, E, ids.shape[1], coef, loss.data_ptr(),
            counts.data_ptr(), probs.data_ptr(), wp, nb)
    return loss, counts, probs


def balance_loss_backward(logits, counts, top_k: int, dloss=None, mask=None, coef: float = 1.0, stream=None):
    """dlogits fp32 [T, E] of balance_loss, from the counts it gave for the same mask; dloss: fp32 scalar tensor on
    the device, None for 1 (vq_balance_loss_backward)."""
    if stream is not None:
        return _on_stream(stream, balance_loss_backward, logits, counts, top_k, dloss, mask, coef)
    torch = _torch()
    T, E = _logits_arg("balance_loss_backward: logits", logits)
    if counts.dtype is not torch.int32 or counts.shape != (E + 1,) or not counts.is_contiguous():
        _bad("balance_loss_backward: counts")
    if dloss is not None and (dloss.dtype is not _f32 or dloss.numel() != 1):
        _bad("balance_loss_backward: dloss")
    mp = None if mask is None else _mask_arg("balance_loss_backward: mask", mask, T)
    dev = _one_device("balance_loss_backward", logits, counts, mask, dloss)
    out = torch.empty_like(logits)
    _launch("vq_balance_loss_backward", dev, logits.data_ptr(), counts.data_ptr(), mp, T, E, top_k, coef,
            None if dloss is None else dloss.data_ptr(), out.data_ptr())
    return out


class Q4Module:
    """A dense 4-bit matrix [rows, cols] with group scales on the device, in the kernel's tile layout (vq_q4_module):
    at least vq_q4_packed_words int32 words, vq_q4_packed_scales fp16 scales (or their int16 bits), and as many biases, as
    from_rows makes them. A call checks and uses the arrays that the module has then."""

    def __init__(self, rows, cols, group, words, scales, biases=None):
        if _codes is None:
            _types()
        _L()
        self.rows, self.cols, self.group = rows, cols, group
        self.words, self.scales, self.biases = words, scales, biases
        self._s = vq_q4_module()
        self._ref = ctypes.byref(self._s)

    def __setattr__(self, name, value):
        object.__setattr__(self, name, value)
        if name[0] != "_":
            self._at = None   # not bound

    def _now(self):
        """The struct of the module as it is now."""
        w, s, b = self.words, self.scales, self.biases
        if b is None:
            at = (w.data_ptr(), s.data_ptr(), w.numel(), s.numel())
        else:
            at = (w.data_ptr(), s.data_ptr(), w.numel(), s.numel(), b.data_ptr(), b.numel())
        if at != self._at:
            self._at = None
            self._bind()
            self._at = at
        return self._ref

    def _bind(self):
        rows, cols, group = self.rows, self.cols, self.group
        nw, ns = int(_L().vq_q4_packed_words(rows, cols)), int(_L().vq_q4_packed_scales(rows, cols, group))
        if nw == 0 or ns == 0:
            _bad("Q4Module: rows, cols, group")
        torch = _torch()
        for name, t, n, types in (("words", self.words, nw, (torch.int32, torch.uint32)),
                                  ("scales", self.scales, ns, (torch.int16, torch.float16)),
                                  ("biases", self.biases, ns, (torch.int16, torch.float16))):
            if t is not None and (t.dtype not in types or t.numel() < n or not t.is_contiguous()):
                _bad("Q4Module: " + name)
        self._dev = _one_device("Q4Module", self.words, self.scales, self.biases)
        s = self._s
        s.rows, s.cols, s.group = rows, cols, group
        s.words, s.scales, s.biases = _ptr(self.words), _ptr(self.scales), _ptr(self.biases)

    def __reduce__(self):   # a copy has a struct of its own
        return (type(self), (self.rows, self.cols, self.group, self.words, self.scales, self.biases), _public(self))

    def _held(self):
        return [self.words, self.scales, self.biases]

    @classmethod
    def from_rows(cls, words, scales, biases=None, group: int = 64, stream=None):
        """Lays row-major device arrays out (vq_q4_pack): words int32 [rows, cols / 8] (pack(codes, 4)'s rows), scales
        and biases fp16 (or their int16 bits) [rows, cols / group]. Without biases W = scale * (q - 8), with them
        W = scale * q + bias."""
        if stream is not None:
            return _on_stream(stream, cls.from_rows, words, scales, biases, group)
        torch = _torch()
        if _codes is None:
            _types()
        if words.dtype not in (torch.int32, torch.uint32) or words.dim() != 2 or not words.is_contiguous():
            _bad("Q4Module.from_rows: words")
        rows, cols = words.shape[0], words.shape[1] * 8
        if group not in (32, 64, 128) or cols % group:
            _bad("Q4Module.from_rows: group")
        for name, t in (("scales", scales), ("biases", biases)):
            if t is not None and (t.dtype not in (torch.float16, torch.int16) or t.shape != (rows, cols // group)
                                  or not t.is_contiguous()):
                _bad("Q4Module.from_rows: " + name)
        nw, ns = int(_L().vq_q4_packed_words(rows, cols)), int(_L().vq_q4_packed_scales(rows, cols, group))
        if nw == 0 or ns == 0:
            _bad("Q4Module.from_rows")
        dev = _one_device("Q4Module.from_rows", words, scales, biases)
        w = words.new_empty(nw, dtype=torch.int32)
        s = scales.new_empty(ns, dtype=torch.int16)
        b = None if biases is None else biases.new_empty(ns, dtype=torch.int16)
        _launch("vq_q4_pack", dev, words.data_ptr(), scales.data_ptr(), _ptr(biases), rows, cols, group, w.data_ptr(),
                s.data_ptr(), _ptr(b))
        return cls(rows, cols, group, w, s, b)


def q4_gemv(m: Q4Module, x, up: Optional[Q4Module] = None, out_dtype=None, out=None, stream=None):
    """y [T, rows] = x [T, cols] (bf16) . W^T; with up: silu(x . W^T) * (x . W_up^T) (vq_q4_gemv). out_dtype: float32
    or bfloat16 (the default, or out's)."""
    if stream is not None:
        return _on_stream(stream, q4_gemv, m, x, up, out_dtype, out)
    ref, up_ref = m._now(), None if up is None else up._now()
    T, rows = x.shape[0], m.rows
    xp, _, xl = _row_arg("q4_gemv: x", x, T, m.cols, VQ_BF16)
    if out is None:
        yd = VQ_BF16 if out_dtype is None else _codes.get(out_dtype)
        if yd is None:
            _bad("q4_gemv: out_dtype")
        dev = _one_device("q4_gemv", x)
        out = x.new_empty(T, rows, dtype=out_dtype or _bf16)
        yp, yl = out.data_ptr(), rows
    else:
        if out_dtype is not None and out.dtype != out_dtype:
            _bad("q4_gemv: out_dtype")
        yp, yd, yl = _row_arg("q4_gemv: out", out, T, rows)
        dev = _one_device("q4_gemv", x, out)
    if dev != m._dev or (up is not None and dev != up._dev):
        _bad("q4_gemv (module on another device)")
    _launch("vq_q4_gemv", dev, ref, up_ref, xp, xl, T, yp, yd, yl)
    return out


def set_trace_events(events) -> None:
    """Record the given torch.cuda.Event objects at the stage boundaries of the
    next MoE calls on this thread (vq_set_trace_events); None switches it off."""
    global _trace_keep
    if events is None:
        _trace_keep = None
        _check(_L().vq_set_trace_events(None, 0), "vq_set_trace_events")
        return
    for e in events:
        if e.cuda_event == 0:
            e.record()
    arr = (ctypes.c_void_p * len(events))(*[e.cuda_event for e in events])
    _trace_keep = arr
    _check(_L().vq_set_trace_events(arr, len(events)), "vq_set_trace_events")


_trace_keep = None


def set_wait_limit(polls: Optional[int]) -> None:
    """Bound the barrier waits of the kernels this thread launches (vq_set_wait_limit);
    None restores the default."""
    _check(_L().vq_set_wait_limit(-1 if polls is None else int(polls)), "vq_set_wait_limit")


class MoELayer:
    """A SwiGLU MoE layer of three VQ modules (vq_moe_layer)."""

    def __init__(self, gate: Module, up: Module, down: Module):
        self.gate, self.up, self.down = gate, up, down
        self.hidden, self.inter, self.E = gate.cols, gate.rows, gate.E
        self._s = vq_moe_layer(gate.struct(), up.struct(), down.struct())
        self._ws = {}
        devs = {t.get_device() for m in (gate, up, down)
                for t in (m.codes, m.scales, m.codebook, m.live_bitmap, m.live_rank, m.biases) if t is not None}
        self._dev = devs.pop() if len(devs) == 1 else None   # index of the one GPU that all arrays are on

    def workspace_size(self, T: int, top_k: int, mode: int) -> int:
        return int(_L().vq_moe_workspace_size(ctypes.byref(self._s), T, top_k, mode))

    def workspace(self, T: int, top_k: int, mode: int, device=None):
        """A cached device workspace large enough for (T, top_k, mode)."""
        torch = _torch()
        n = self.workspace_size(T, top_k, mode)
        if n == 0:
            raise VQError(1, "vq_moe_workspace_size")
        cur = self._ws.get(mode)
        if cur is None or cur.numel() < n:
            cur = torch.empty(n + 256, dtype=torch.uint8, device=device or self.gate.codes.device)
            self._ws[mode] = cur
        return cur

    def _run(self, fn, name, mode, x, logits, top_k, renorm, out, out_dtype, workspace, stream):
        torch = _torch()
        T = x.shape[0]
        if out is None:
            out = torch.empty((T, self.hidden), dtype=out_dtype or torch.float32, device=x.device)
        ws = workspace if workspace is not None else self.workspace(T, top_k, mode, x.device)
        _, aligned, nbytes = _workspace(0, ws, x)
        _check(fn(ctypes.byref(self._s), x.data_ptr(), T, logits.data_ptr(), top_k, int(bool(renorm)),
                  out.data_ptr(), _dt(out.dtype), aligned, nbytes, _stream(stream)), name)
        return out

    def check(self, mode: int, stream=None) -> int:
        """Status of the device error word of the cached workspace for `mode` (vq_moe_check)."""
        ws = self._ws.get(mode)
        if ws is None:
            return VQ_OK
        base = (ws.data_ptr() + 255) // 256 * 256
        return int(_L().vq_moe_check(base, _stream(stream)))

    def decode(self, x, logits, top_k: int, renorm: bool = True, out=None, out_dtype=None, workspace=None,
               stream=None):
        """y [T, hidden] for decode-sized batches (vq_moe_decode)."""
        return self._run(_L().vq_moe_decode, "vq_moe_decode", VQ_MODE_DECODE, x, logits, top_k, renorm, out,
                         out_dtype, workspace, stream)

    def prefill(self, x, logits, top_k: int, renorm: bool = True, out=None, out_dtype=None, workspace=None,
                stream=None):
        """y [T, hidden] for prefill-sized batches (vq_moe_prefill, tcgen05 grouped GEMM)."""
        return self._run(_L().vq_moe_prefill, "vq_moe_prefill", VQ_MODE_PREFILL, x, logits, top_k, renorm, out,
                         out_dtype, workspace, stream)

    def prefill_chunked(self, x, logits, top_k: int, chunk: int = 2048, renorm: bool = True, out=None,
                        out_dtype=None, workspace=None, stream=None):
        """y [T, hidden] for a long prompt, `chunk` tokens at a time through one chunk-sized
        workspace (vq_moe_prefill_chunked)."""
        torch = _torch()
        T = x.shape[0]
        if out is None:
            out = torch.empty((T, self.hidden), dtype=out_dtype or torch.float32, device=x.device)
        ws = workspace if workspace is not None else self.workspace(max(1, min(T, chunk)), top_k, VQ_MODE_PREFILL,
                                                                     x.device)
        _, aligned, nbytes = _workspace(0, ws, x)
        _check(_L().vq_moe_prefill_chunked(ctypes.byref(self._s), x.data_ptr(), T, logits.data_ptr(), top_k,
                                            int(bool(renorm)), int(chunk), out.data_ptr(), _dt(out.dtype), aligned,
                                            nbytes, _stream(stream)), "vq_moe_prefill_chunked")
        return out


class MoEBlock:
    """A residual block around a MoE layer, from the residual stream to the residual stream:

        x  = pre(h)                                     (or the x the block before made with its `next` norm)
        y  = experts(x, router(x)) + sigmoid(shared_gate(x)) * shared expert(x)
        h' = res_scale * h + out_scale * post(y),   x' = next(h')

    router: x [T, hidden] bf16 -> logits fp32 [T, E]. shared: (gate, up, down) Q4Modules of a SwiGLU expert that every
    token takes (its hidden activation and its output are bf16; its products decode the weights once for every 16
    tokens, which a long prompt pays for: 4096 tokens, hidden 4096 and 2048 wide, 1.1 ms); shared_gate: x -> logits
    [T, 1], None for 1. post and next may be None. As the calls it makes, it has no part in autograd, and the experts
    have no gradient. Every call has an experts'
    workspace of its own, so calls on several streams, or captured into several graphs, do not meet in one; a given
    `workspace` (256 bytes more than layer.workspace_size) can be asked for its error word (fit_check)."""

    def __init__(self, layer: MoELayer, pre: Norm, router, top_k: int, post: Optional[Norm] = None,
                 next: Optional[Norm] = None, shared=None, shared_gate=None, renorm: bool = True,
                 res_scale: float = 1.0, out_scale: float = 1.0):
        if pre.hidden != layer.hidden or (shared is not None and (shared[0].cols, shared[2].rows) != (layer.hidden,) * 2):
            _bad("MoEBlock: hidden sizes")
        self.layer, self.pre, self.post, self.next = layer, pre, post, next
        self.router, self.shared, self.shared_gate = router, shared, shared_gate
        self.top_k, self.renorm, self.res_scale, self.out_scale = top_k, renorm, res_scale, out_scale

    def decode(self, h, x=None, workspace=None):
        """(h', x', router logits) for decode-sized batches; x' is None without `next`."""
        return self._run(self.layer.decode, VQ_MODE_DECODE, h, x, workspace)

    def prefill(self, h, x=None, workspace=None):
        """The same for prefill-sized batches."""
        return self._run(self.layer.prefill, VQ_MODE_PREFILL, h, x, workspace)

    def _run(self, experts, mode, h, x, workspace):
        dev = _one_device("MoEBlock", h, x, workspace)
        if dev != _device():
            with _torch().cuda.device(dev):
                return self._run(experts, mode, h, x, workspace)
        if dev != getattr(self.layer, "_dev", dev):   # (a layer of the caller's own making knows its device itself)
            _bad("MoEBlock (layer on another device)")
        if h.dim() != 2 or h.shape[1] != self.layer.hidden:   # the experts read rows of hidden elements of x
            _bad("MoEBlock: h")
        if x is None:
            x = norm_pre(self.pre, h)
        elif x.dtype is not _bf16 or x.shape != h.shape or not x.is_contiguous():
            _bad("MoEBlock: x")
        T = x.shape[0]
        logits = self.router(x)
        if logits.dtype is not _f32 or logits.shape != (T, self.layer.E) or not logits.is_contiguous():
            _bad("MoEBlock: router logits")
        _one_device("MoEBlock: router logits", x, logits)
        if workspace is None:
            n = self.layer.workspace_size(T, self.top_k, mode)
            if n == 0:
                _bad("MoEBlock: tokens or top_k")
            workspace = x.new_empty(n + 256, dtype=_torch().uint8)
        y = experts(x, logits, self.top_k, self.renorm, out_dtype=_f32, workspace=workspace)
        if self.shared is not None:
            gate, up, down = self.shared
            s = q4_gemv(down, q4_gemv(gate, x, up))
            norm_post(s, y, gate=None if self.shared_gate is None else self.shared_gate(x), h_out=y)
        h, x = norm_post(y, h, self.post, None, self.res_scale, self.out_scale, self.next)
        return h, x, logits
