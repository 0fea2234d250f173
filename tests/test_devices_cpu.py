"""Tensors of another device than the current one, or of two devices, are
refused before anything is launched: the library launches on the current
device, whatever device the pointers belong to.  The tensors here say that
they are on a device; the library is a stub that fails when it is called."""
import pytest
import torch

import mixture_experts_layer_mok_gb300 as mok
from mixture_experts_layer_mok_gb300 import _lib, ops, optim

BF16, F32, U8 = torch.bfloat16, torch.float32, torch.uint8


class On(torch.Tensor):
    """A tensor that says it is on cuda:`index`."""
    __torch_function__ = torch._C._disabled_torch_function_impl
    index = 0

    @property
    def is_cuda(self):
        return True

    @property
    def device(self):
        return torch.device("cuda", self.index)

    def get_device(self):
        return self.index


def on(index, *shape, dtype=BF16):
    t = torch.zeros(*shape, dtype=dtype).as_subclass(On)
    t.index = index
    return t


class Launched(Exception):
    pass


class Stub:
    def __getattr__(self, name):
        def call(*a):
            if name.endswith("_bytes") or name.endswith("bytes_ring"):
                return 4096
            raise Launched(name)
        return call


@pytest.fixture
def stub(monkeypatch):
    real = torch.empty
    monkeypatch.setattr(_lib, "load", lambda *a: Stub())
    for module in (mok, ops, optim):
        monkeypatch.setattr(module, "_current_device", lambda: 0, raising=False)
        if hasattr(module, "_raw_stream"):
            monkeypatch.setattr(module, "_raw_stream", lambda at: at, raising=False)
    monkeypatch.setattr(optim, "_capturing", lambda: False)
    empty = lambda *a, device=None, **k: real(*a, **k)  # noqa: E731
    monkeypatch.setattr(ops, "_empty", empty)
    monkeypatch.setattr(torch, "empty", empty)
    zeros, full = torch.zeros, torch.full
    monkeypatch.setattr(optim.torch, "zeros", lambda *a, device=None, **k: zeros(*a, **k))
    monkeypatch.setattr(optim.torch, "full", lambda *a, device=None, **k: full(*a, **k))


def _ops_calls():
    """name -> (call of tensors, the tensors' shapes and types)"""
    M, N, K = 4, 32, 64
    return {
        "rms_norm": (lambda x, w, r: mok.rms_norm(x, w, residual=r), [((M, K), BF16), ((K,), BF16), ((M, K), F32)]),
        "rms_norm_backward": (lambda dy, h, w, rstd, dh: mok.rms_norm_backward(dy, h, w, rstd, d_h=dh),
                              [((M, K), BF16), ((M, K), BF16), ((K,), BF16), ((M,), F32), ((M, K), BF16)]),
        "linear": (lambda x, w, b, r: mok.linear(x, w, bias=b, residual=r),
                   [((M, K), BF16), ((N, K), BF16), ((N,), F32), ((M, N), BF16)]),
        "linear_backward": (lambda dy, x, w, z: mok.linear_backward(dy, x, w, z=z, activation="gelu", bias=True),
                            [((M, N), BF16), ((M, K), BF16), ((N, K), BF16), ((M, N), BF16)]),
        "mxfp8_dequantize": (mok.mxfp8_dequantize, [((M, K), U8), ((M, K // 32), U8)]),
    }


@pytest.mark.parametrize("name", sorted(_ops_calls()))
def test_operators_refuse_other_devices(stub, name):
    call, args = _ops_calls()[name]
    make = lambda index, **other: [on(other.get(f"a{i}", index), *s, dtype=d)  # noqa: E731
                                   for i, (s, d) in enumerate(args)]
    with pytest.raises(Launched):
        call(*make(0))
    with pytest.raises(ValueError, match="cuda:1"):
        call(*make(1))
    for i in range(len(args)):
        with pytest.raises(ValueError, match="cuda:"):
            call(*make(0, **{f"a{i}": 1}))


def test_the_optimiser_refuses_other_devices(stub, monkeypatch):
    f = lambda index=0, n=64: on(index, n, dtype=F32)  # noqa: E731
    with pytest.raises(ValueError):
        mok.AdamW([f(1)])
    with pytest.raises(ValueError):
        mok.AdamW([f(), f(1)])
    state = lambda index: {"m": [f(index)], "v": [f(index)]}  # noqa: E731
    with pytest.raises(ValueError):
        mok.AdamW([f()], buffers=state(1))
    opt = mok.AdamW([f()], buffers=state(0))
    with pytest.raises(Launched):
        opt.step([f()])
    for kw in (dict(grads=[f(1)]), dict(grads=[f()], grad_scale=f(1, 1))):
        with pytest.raises(ValueError):
            opt.step(**kw)
    monkeypatch.setattr(optim, "_current_device", lambda: 1, raising=False)
    with pytest.raises(ValueError, match="current device"):
        opt.step([f()])
    assert opt.step_count == 0


def test_the_layers_calls_refuse_other_devices(stub):
    ids = on(1, 4, 2, dtype=torch.int64)
    x = on(1, 4, 128)
    for call in (lambda: mok.schedule(ids, 8), lambda: mok.schedule_noalloc(ids, 8), lambda: mok.mxfp8_quantize(x),
                 lambda: mok.mxfp8_quantize_t(x), lambda: mok.mxfp8_quantize_dual(x)):
        with pytest.raises(ValueError, match="cuda:1"):
            call()
    sched = mok.Schedule(4, 2, 8, None, _lib.MokSchedule())
    w = lambda i=0: mok.Weights(on(i, 8, 128, 128), on(i, 8, 128, 128), on(i, 8, 128, 128))  # noqa: E731
    rw = lambda i=0: on(i, 4, 2, dtype=F32)  # noqa: E731
    for a in ((x, rw(), w()), (on(0, 4, 128), rw(1), w()), (on(0, 4, 128), rw(), w(1))):
        with pytest.raises(ValueError, match="cuda:1"):
            mok.forward(a[0], a[1], sched, a[2])
    ctx = mok.Context(None, _lib.MokCtx(), 0)
    for a in ((x, on(0, 4, 128)), (on(0, 4, 128), x)):
        with pytest.raises(ValueError, match="cuda:1"):
            mok.backward(a[0], a[1], rw(), sched, ctx, w())


class _Stream:
    device_index, cuda_stream = 1, 0


def test_the_layers_calls_refuse_another_devices_stream(stub):
    with pytest.raises(ValueError, match="stream"):
        mok.mxfp8_quantize(on(0, 4, 128), stream=_Stream())
