"""Memory that a call allocates belongs to the stream that its work runs on: the current stream's
allocator may hand out a block that kernels queued there still use, which work on a given other
stream would overwrite.  On the CPU with stand-ins for the tensors, the library and the current stream;
on the GPU with the allocator itself."""
import math
import sys
import types

import pytest
import torch

import selective_state_space_20_amd as sss
from selective_state_space_20_amd import _block, _lib

F32, BF16, I32 = torch.float32, torch.bfloat16, torch.int32


class Gpu:
    """The GPU that tensors are on, and what is current: raw stream handles and GPUs, innermost last."""

    def __init__(self, current, index=0, device=0):
        self.now, self.made, self.index, self.devices = [current], [], index, [device]

    def torch(self):
        gpu = self

        class On:
            def __init__(self, stack, entry):
                self.stack, self.entry = stack, entry

            def __enter__(self):
                self.stack.append(self.entry)

            def __exit__(self, *a):
                self.stack.pop()

        cuda = types.SimpleNamespace(
            stream=lambda s: On(gpu.now, s.cuda_stream),
            device=lambda d: On(gpu.devices, d if isinstance(d, int) else d.index),
            ExternalStream=lambda h, device=None: types.SimpleNamespace(cuda_stream=h if h != 0 else "a new stream"),
            default_stream=lambda i=None: types.SimpleNamespace(cuda_stream=0),
            current_stream=lambda i=None: types.SimpleNamespace(cuda_stream=gpu.now[-1]))
        c = types.SimpleNamespace(_cuda_getCurrentRawStream=lambda i: gpu.now[-1], _cuda_getDevice=lambda: gpu.devices[-1])
        names = {n: getattr(torch, n) for n in ("float32", "bfloat16", "int32", "uint8", "bool", "device")}
        empty = lambda shape, dtype=F32, device=None: self.tensor(shape, dtype, self.now[-1])
        return types.SimpleNamespace(cuda=cuda, _C=c, Tensor=Tensor, empty=empty, **names)

    def tensor(self, shape, dtype=F32, stream=None):
        t = Tensor(self, tuple(shape) if isinstance(shape, (tuple, list)) else (shape,), dtype, stream)
        if stream is not None:
            self.made.append(t)
        return t


class Tensor:
    is_cuda = True

    def __init__(self, gpu, shape, dtype, stream):
        self.gpu, self.shape, self.dtype, self.stream, self.recorded = gpu, shape, dtype, stream, []

    ndim = property(lambda self: len(self.shape))
    device = property(lambda self: torch.device("cuda", self.gpu.index))
    get_device = lambda self: self.gpu.index
    is_contiguous = lambda self: True
    data_ptr = lambda self: 4096 + id(self) % 4096
    numel = lambda self: math.prod(self.shape)
    element_size = lambda self: self.dtype.itemsize
    stride = lambda self: tuple(math.prod(self.shape[i + 1:]) for i in range(len(self.shape)))
    new_empty = lambda self, shape, dtype=None: self.gpu.tensor(shape, dtype or self.dtype, self.gpu.now[-1])
    record_stream = lambda self, s: self.recorded.append(s.cuda_stream)


class Library:
    """Every size is 64 bytes, every call succeeds; the stream is a call's last argument."""

    def __init__(self):
        self.streams, self.calls, self.devices, self.gpu = [], [], [], None

    def __getattr__(self, name):
        if name.endswith("_size"):
            return lambda *a: 64

        def call(*a):
            self.streams.append(a[-1])
            self.calls.append((name, a))
            self.devices.append(self.gpu.devices[-1])
            return 0
        return call


def block_calls(t):
    """{entry point: a call of it that allocates all it can}"""
    x, w, m, v = t((6, 8)), t((8, 4)), t((6, 2)), t((8,))
    cu, conv, state = t((3,), I32), t((6, 3, 8)), t((6, 8, 2))
    A, r = t((8, 2)), t((6,))
    return {
        "conv": lambda **k: sss.causal_conv1d_packed_fwd(x, w, cu_seqlens=cu, conv_state=conv, **k),
        "conv step": lambda **k: sss.causal_conv1d_update(x, w, conv_state=conv, **k),
        "conv gradients": lambda **k: sss.causal_conv1d_bwd(t((2, 6, 8)), w, v, dout=t((2, 6, 8)), **k),
        "scan": lambda **k: sss.selective_scan_packed_fwd(x, x, A, m, m, cu_seqlens=cu, state=state, **k),
        "scan step": lambda **k: sss.selective_state_update_slots(x, x, A, m, m, state=state, **k),
        "gated norm": lambda **k: sss.rms_norm_gated_fwd(x, v, x, return_rstd=True, **k),
        "gated norm gradients": lambda **k: sss.rms_norm_gated_bwd(x, x, v, x, rstd=t((6, 1)), **k),
        "residual norm": lambda **k: sss.rms_norm_residual_fwd(x, v, x, post_weight=v, return_rstd=True, **k),
        "residual norm gradients": lambda **k: sss.rms_norm_residual_bwd(
            x, x, residual_out=x, weight=v, rstd=r, x=x, post_weight=v, scale=v, rstd_post=r, **k),
    }


def dense_calls(t):
    """The same for the calls on equal-length batches."""
    x, m, A, h, v = t((2, 6, 8)), t((2, 6, 4)), t((8, 4)), t((2, 8, 4)), t((8,))
    e, r, rm = t((2, 6, 8)), t((2, 8)), t((2, 4))
    return {
        "dense scan": lambda **k: sss.selective_scan_fwd(x, x, A, m, m, **k),
        "dense scan gradients": lambda **k: sss.selective_scan_bwd(x, x, A, m, m, dy=x, **k),
        "dense scan gradients, bias": lambda **k: sss.selective_scan_bwd(x, x, A, m, m, v, x, h, dy=x, delta_bias=v, **k),
        "dense step": lambda **k: sss.selective_state_update(r, r, A, rm, rm, state=h, **k),
        "dense conv": lambda **k: sss.causal_conv1d_fwd(x, t((8, 4)), v, **k),
        "elementwise scan": lambda **k: sss.elementwise_scan(e, e, e, e, **k),
    }


BLOCK = list(block_calls(lambda *a: None).keys())
MADE = {"conv": 1, "conv step": 1, "conv gradients": 4, "scan": 2, "scan step": 1, "gated norm": 2,
        "gated norm gradients": 4, "residual norm": 4, "residual norm gradients": 6,
        "dense scan": 3, "dense scan gradients": 7, "dense scan gradients, bias": 10, "dense step": 1, "dense conv": 1,
        "elementwise scan": 3}
DENSE = list(dense_calls(lambda *a: None).keys())


def calls(t):
    return {**block_calls(t), **dense_calls(t)}


@pytest.fixture
def gpu(monkeypatch):
    def make(current, index=0, device=0):
        g, lib = Gpu(current, index, device), Library()
        lib.gpu = g
        for m in (_block, _lib):
            monkeypatch.setattr(m, "load", lambda: lib)
        stand_in = g.torch()
        monkeypatch.setitem(sys.modules, "torch", stand_in)
        monkeypatch.setattr(_block, "_torch", stand_in)
        monkeypatch.setattr(_block, "_current_gpu", stand_in._C._cuda_getDevice)
        monkeypatch.setattr(_block, "torch_", lambda: stand_in)
        monkeypatch.setattr(_lib, "_lib", lib)
        return g, lib
    return make


@pytest.mark.parametrize("name", BLOCK + DENSE)
@pytest.mark.parametrize("current, given", [(0, 7), (5, 7), (5, 0)])
def test_memory_of_the_given_stream(gpu, name, current, given):
    g, lib = gpu(current)
    res = calls(g.tensor)[name](stream=given)
    assert lib.streams == [given] and len(g.made) == MADE[name]
    assert [t.stream for t in g.made] == [given] * len(g.made)
    results = res.values() if isinstance(res, dict) else res if isinstance(res, tuple) else [res]
    for t in (t for t in results if t is not None):  # used on the current stream as a rule: not freed under it
        assert current in t.recorded and "a new stream" not in t.recorded
    assert g.now == [current]


@pytest.mark.parametrize("name", BLOCK + DENSE)
@pytest.mark.parametrize("current, given", [(0, None), (5, None), (5, 5)])
def test_memory_of_the_current_stream(gpu, name, current, given):
    g, lib = gpu(current)
    calls(g.tensor)[name](stream=given)
    assert lib.streams == [current] and len(g.made) == MADE[name]
    assert all(t.stream == current and t.recorded == [] for t in g.made)


@pytest.mark.gpu
def test_no_block_that_the_current_stream_may_still_use():
    """A block freed on the current stream with work queued on it is the next that this stream's allocator
    hands out; a call on another stream does not get it, and the queued work keeps its result."""
    x = torch.randn(4096, 2048, device="cuda:0")
    w, z = torch.rand(2048, device="cuda:0"), torch.randn(4096, 2048, device="cuda:0")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for handle, current in ((side.cuda_stream, torch.cuda.current_stream()), (0, side)):
        with torch.cuda.stream(current):
            block = torch.full((4096, 2048), 3.0, device="cuda:0")
            where = block.data_ptr()
            for _ in range(20):
                block.mul_(1.0)
            kept = block + 1.0
            del block
            out = sss.rms_norm_gated_fwd(x, w, z, stream=handle)
            assert out.data_ptr() != where
            torch.cuda.synchronize()
            assert bool((kept == 4.0).all())
            assert torch.equal(out, sss.rms_norm_gated_fwd(x, w, z))
            torch.cuda.synchronize()
