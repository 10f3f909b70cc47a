"""What the block operators' binding hands to the library, and what it refuses before it does: weights and modules as
they are at the call. CPU tensors throughout; the library's launch is replaced by a record of its arguments."""
import copy
import types

import pytest
import torch

import vector_quantized_moe_b200 as vq
from helpers import lib_module, small_module

BF16, F32 = torch.bfloat16, torch.float32
ARG, WORKSPACE = 1, 4


@pytest.fixture
def launches(monkeypatch):
    """The launches that a call would make, as (name, args); every tensor passes for one on GPU 0."""
    made = []
    vq.Norm(torch.ones(8))   # binds the library and torch's types
    monkeypatch.setattr(vq, "_one_device", lambda where, first, *others: 0)
    monkeypatch.setattr(vq, "_launch", lambda name, dev, *args: made.append((name, args)))
    return made


def struct(ref):
    """A copy of the struct behind a byref() as it is now."""
    return type(ref._obj).from_buffer_copy(ref._obj)


def address(t):
    return t.data_ptr()


CALLS = {
    "norm_pre": lambda n, v: vq.norm_pre(n, v),
    "norm_pre_backward": lambda n, v: vq.norm_pre_backward(n, v, v),
    "norm_post, post": lambda n, v: vq.norm_post(v, v, n),
    "norm_post, next": lambda n, v: vq.norm_post(v, v, next=n),
    "norm_post_backward, post": lambda n, v: vq.norm_post_backward(v, v, v, post=n),
    "norm_post_backward, next": lambda n, v: vq.norm_post_backward(v, v, v, v, next=n),
}


@pytest.mark.parametrize("call", CALLS)
def test_a_norm_uses_the_weight_it_has_at_the_call(launches, call):
    def weight_of():
        launches.clear()
        CALLS[call](n, v)
        ref = launches[0][1][1 if call.endswith("next") else 0]
        return struct(ref)

    v = torch.zeros((2, 64), dtype=BF16)
    w = torch.nn.Parameter(torch.ones(64))
    n = vq.Norm(w, 1e-5, 1.0)
    first = w.data
    assert weight_of().weight == address(w)
    w.data = torch.full((64,), 2.0)                      # new data of the same parameter
    got = weight_of()
    assert got.weight == address(w) != address(first) and got.weight_dtype == vq.VQ_F32
    n.weight = torch.full((64,), 3.0, dtype=BF16)        # another weight, of another type
    got = weight_of()
    assert got.weight == address(n.weight) and got.weight_dtype == vq.VQ_BF16
    assert (got.hidden, got.weight_offset) == (64, 1.0) and abs(got.eps - 1e-5) < 1e-12
    n.weight = torch.ones(32)                            # of another width: the rows no longer fit
    with pytest.raises(vq.VQError):
        weight_of()
    n.weight = torch.ones(64, dtype=torch.float16)       # of a type that no norm takes
    with pytest.raises(vq.VQError):
        weight_of()


def q4_arrays(rows, cols, group, biased=False):
    words = torch.zeros(vq._L().vq_q4_packed_words(rows, cols), dtype=torch.int32)
    scales = torch.zeros(vq._L().vq_q4_packed_scales(rows, cols, group), dtype=torch.int16)
    return words, scales, scales.clone() if biased else None


@pytest.mark.parametrize("pair", [False, True])
def test_a_4_bit_module_uses_the_arrays_it_has_at_the_call(launches, pair):
    def structs():
        launches.clear()
        vq.q4_gemv(m, x, up)
        return [struct(r) for r in launches[0][1][:2] if r is not None]

    x = torch.zeros((2, 128), dtype=BF16)
    m = vq.Q4Module(64, 128, 64, *q4_arrays(64, 128, 64, True))
    up = vq.Q4Module(64, 128, 64, *q4_arrays(64, 128, 64, True)) if pair else None
    last = up if pair else m
    assert structs()[-1].words == address(last.words)
    old = last.words.data
    last.words.data = last.words.clone()
    assert structs()[-1].words == address(last.words) != address(old)
    for name in ("scales", "biases"):
        setattr(last, name, getattr(last, name).clone())
        assert getattr(structs()[-1], name) == address(getattr(last, name))
    s = structs()[-1]
    assert (s.rows, s.cols, s.group) == (64, 128, 64)
    if not pair:
        last.biases = None
        assert structs()[-1].biases is None


def refused(f, *a, **k):
    with pytest.raises(vq.VQError) as e:
        f(*a, **k)
    assert e.value.status == ARG


@pytest.mark.parametrize("change", [
    dict(words=slice(0, -1)), dict(words=slice(0, 256)), dict(scales=slice(0, 16)), dict(biases=slice(0, -8)),
    dict(words=BF16), dict(scales=BF16), dict(biases=F32), dict(words=slice(None, None, 2)), dict(rows=80), dict(cols=256),
    dict(group=32), dict(rows=0), dict(group=48), dict(cols=96)])
@pytest.mark.parametrize("as_up", [False, True])
@pytest.mark.parametrize("late", [False, True])
def test_a_4_bit_module_that_does_not_hold_its_layout_is_refused(launches, change, as_up, late):
    # before the first call, and after calls that were right
    rows, cols = 64, 128
    m, other = (vq.Q4Module(rows, cols, 64, *q4_arrays(rows, cols, 64, True)) for _ in range(2))
    x = torch.zeros((2, cols), dtype=BF16)
    call = (lambda: vq.q4_gemv(other, x, m)) if as_up else (lambda: vq.q4_gemv(m, x))
    if late:
        call()
    for name, what in change.items():
        old = getattr(m, name)
        if isinstance(what, slice):
            # steps: as many elements as the layout has, but not consecutive
            new = old.repeat(2)[what] if what.step else old[what]
        else:
            new = torch.zeros(old.shape, dtype=what) if isinstance(what, torch.dtype) else what
        setattr(m, name, new)
    launches.clear()
    refused(call)
    refused(call)
    assert not launches


def test_a_4_bit_module_checks_all_its_arrays_devices(monkeypatch):
    seen = []
    monkeypatch.setattr(vq, "_one_device", lambda where, first, *others: seen.extend((first, *others)) or 0)
    monkeypatch.setattr(vq, "_launch", lambda *a: None)
    m = vq.Q4Module(64, 128, 64, *q4_arrays(64, 128, 64, True))
    x = torch.zeros((2, 128), dtype=BF16)
    vq.q4_gemv(m, x)
    assert all(any(t is s for s in seen) for t in (x, m.words, m.scales, m.biases))
    for out in (None, torch.zeros((2, 64), dtype=BF16)):
        m._dev = 1   # a module on another GPU than the tokens
        refused(vq.q4_gemv, m, x, out=out)


def test_an_undersized_module_is_refused_before_any_gpu_is_asked_for():
    m = vq.Q4Module(64, 64, 64, torch.zeros(256, dtype=torch.int32), torch.zeros(16, dtype=torch.int16))
    refused(vq.q4_gemv, m, torch.zeros((2, 64), dtype=BF16))
    with pytest.raises(vq.VQError, match="words"):
        m._now()


@pytest.fixture
def block(launches, monkeypatch):
    """A block on CPU tensors that pass for GPU 0's; its experts record the x they get."""
    E, H, I = 4, 512, 256
    layer = vq.MoELayer(*[lib_module(small_module(E, r, c, 2, 8, seed=i), device="cpu")
                          for i, (r, c) in enumerate(((I, H), (I, H), (H, I)))])
    layer._dev = 0
    seen = []
    layer.decode = layer.prefill = lambda x, *a, **k: seen.append(x) or torch.zeros((x.shape[0], H))
    monkeypatch.setattr(vq, "_device", lambda: 0)
    b = vq.MoEBlock(layer, vq.Norm(torch.ones(H)), lambda x: torch.zeros((x.shape[0], E)), 2)
    b.seen = seen
    return b


@pytest.mark.parametrize("path", ["decode", "prefill"])
def test_experts_get_rows_of_their_own_width_only(block, path):
    run = getattr(block, path)
    run(torch.zeros((3, 512)), torch.zeros((3, 512), dtype=BF16))
    assert len(block.seen) == 1
    for width in (256, 1024):   # h and a given x agree with each other, and a router that looks at neither
        refused(run, torch.zeros((3, width)), torch.zeros((3, width), dtype=BF16))
    refused(run, torch.zeros(512), torch.zeros(512, dtype=BF16))
    block.pre = vq.Norm(torch.ones(256))   # a norm of another width, given later
    refused(run, torch.zeros((3, 256)))
    assert len(block.seen) == 1


@pytest.mark.parametrize("path", ["decode", "prefill"])
def test_experts_on_another_device_are_refused(block, path):
    block.layer._dev = 1
    refused(getattr(block, path), torch.zeros((3, 512)))
    assert not block.seen


class OnGPU:
    """A tensor that says it is on GPU 3."""

    def __init__(self, t):
        self.t = t

    def __getattr__(self, name):
        return getattr(self.t, name)

    def get_device(self):
        return 3


def test_a_layer_knows_the_one_device_of_its_arrays():
    mods = [lib_module(small_module(4, r, c, 2, 8, seed=i), device="cpu")
            for i, (r, c) in enumerate(((256, 512), (256, 512), (512, 256)))]
    assert vq.MoELayer(*mods)._dev == -1
    for name in ("codes", "scales", "codebook"):
        old = getattr(mods[2], name)
        setattr(mods[2], name, OnGPU(old))
        assert vq.MoELayer(*mods)._dev is None
        setattr(mods[2], name, old)


@pytest.mark.parametrize("how", [copy.copy, copy.deepcopy])
def test_copies_are_bound_for_themselves(launches, how):
    v = torch.zeros((2, 64), dtype=BF16)
    n = vq.Norm(torch.ones(64), 1e-5, 1.0)
    n.name = "input"
    vq.norm_pre(n, v)
    c = how(n)
    assert c.name == "input" and c.hidden == 64
    c.weight = torch.full((64,), 2.0)
    launches.clear()
    for each in (c, n, c):
        vq.norm_pre(each, v)
        s = struct(launches[-1][1][0])
        assert s.weight == address(each.weight) and s.weight_offset == 1.0 and abs(s.eps - 1e-5) < 1e-12
    m = vq.Q4Module(64, 128, 64, *q4_arrays(64, 128, 64, True))
    x = torch.zeros((2, 128), dtype=BF16)
    vq.q4_gemv(m, x)
    c = how(m)
    c.scales = m.scales.clone()
    for each in (c, m, c):
        vq.q4_gemv(each, x)
        s = struct(launches[-1][1][0])
        assert (s.words, s.scales, s.biases) == (address(each.words), address(each.scales), address(each.biases))


def test_a_block_around_a_layer_of_another_class(block):
    plain = types.SimpleNamespace(**{k: getattr(block.layer, k) for k in ("hidden", "E", "workspace_size", "decode", "prefill")})
    b = vq.MoEBlock(plain, block.pre, block.router, 2)
    b.decode(torch.zeros((3, 512)))
    assert len(block.seen) == 1
