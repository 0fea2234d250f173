"""CPU-side checks of the router, the projections grouped by expert and the 4-bit
projections: sizes, refusals before any device work, the Python faces' own
checks, and tensors of other devices."""
import ctypes as C

import pytest
import torch

import mixture_experts_layer_mok_gb300 as mok
from mixture_experts_layer_mok_gb300 import experts
from tests.test_devices_cpu import BF16, F32, U8, Launched, on, stub  # noqa: F401

FAKE, ODD = C.c_void_p(16), C.c_void_p(24)      # never dereferenced: validation fails first
BAD = 1                                           # MOK_ERR_INVALID_ARG
I32, I64 = torch.int32, torch.int64


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__ as g

    g.build()
    from mixture_experts_layer_mok_gb300 import _lib

    return _lib.load()


def test_route_refusals_and_sizes(lib):
    def fwd(x=FAKE, xd=1, b=None, T=4, E=16, k=2, score=0, norm=1, scale=1.0, ids=FAKE, w=FAKE, lse=FAKE, c=None, m=None, ws=None, n=0):
        return lib.mok_route(x, xd, b, T, E, k, score, norm, scale, ids, w, lse, c, m, ws, n, None)

    for bad in (dict(T=-1), dict(T=1 << 31), dict(E=0), dict(E=1025), dict(k=0), dict(k=17), dict(E=100, k=65), dict(xd=2), dict(score=2),
                dict(scale=float("nan")), dict(scale=float("inf")), dict(x=None), dict(ids=None), dict(w=None), dict(lse=None),
                dict(c=FAKE), dict(m=FAKE), dict(c=FAKE, m=FAKE), dict(c=FAKE, m=FAKE, ws=FAKE, n=64), dict(x=ODD), dict(b=ODD),
                dict(ids=ODD), dict(w=ODD), dict(lse=ODD), dict(c=ODD, m=FAKE, ws=FAKE, n=1 << 20)):
        assert fwd(**bad) == BAD, bad
    assert fwd(T=0) == 0
    size = lib.mok_route_workspace_bytes
    assert size(-1, 8) == 0 and size(4, 0) == 0 and size(4, 1025) == 0
    assert size(0, 8) > 0 and size(1, 8) >= 2 * 8 * 4 and size(1 << 30, 1024) < 1 << 24

    def bwd(dw=FAKE, x=FAKE, xd=1, ids=FAKE, dl=None, dm=None, T=4, E=16, k=2, score=0, norm=1, scale=1.0, d=FAKE):
        return lib.mok_route_bwd(dw, x, xd, ids, dl, dm, T, E, k, score, norm, scale, d, None)

    for bad in (dict(T=-1), dict(E=0), dict(k=0), dict(k=17), dict(xd=-1), dict(score=-1), dict(scale=float("inf")), dict(dw=None),
                dict(x=None), dict(ids=None), dict(d=None), dict(dw=ODD), dict(x=ODD), dict(ids=ODD), dict(dl=ODD), dict(dm=ODD),
                dict(d=ODD)):
        assert bwd(**bad) == BAD, bad
    assert bwd(T=0) == 0


def test_grouped_refusals_and_sizes(lib):
    def fwd(x=FAKE, w=FAKE, c=FAKE, b=None, bd=0, act=0, M=4, E=3, N=64, K=64, y=FAKE, yd=0, z=None):
        return lib.mok_grouped_linear(x, w, c, b, bd, act, M, E, N, K, y, yd, z, None)

    for bad in (dict(M=-1), dict(M=(1 << 31) - 1), dict(E=0), dict(E=1025), dict(N=0), dict(N=12), dict(K=0), dict(K=36), dict(act=5),
                dict(act=-1), dict(yd=2), dict(b=FAKE, bd=2), dict(x=None), dict(w=None), dict(c=None), dict(y=None), dict(x=ODD),
                dict(w=ODD), dict(c=ODD), dict(b=ODD), dict(y=ODD), dict(z=ODD), dict(N=1 << 20, K=1 << 20)):
        assert fwd(**bad) == BAD, bad
    assert fwd(M=0) == 0

    def bwd(dy=FAKE, dd=0, x=FAKE, w=FAKE, c=FAKE, z=None, act=0, M=4, E=3, N=64, K=64, dx=FAKE, dw=FAKE, db=None, ws=FAKE, n=1 << 30):
        return lib.mok_grouped_linear_bwd(dy, dd, x, w, c, z, act, M, E, N, K, dx, dw, db, ws, n, None)

    for bad in (dict(M=-1), dict(E=0), dict(N=12), dict(K=36), dict(act=9), dict(dd=2), dict(dy=None), dict(x=None), dict(w=None),
                dict(c=None), dict(act=3), dict(ws=None), dict(n=8), dict(act=3, z=FAKE, n=300), dict(dy=ODD), dict(dx=ODD), dict(dw=ODD),
                dict(db=ODD), dict(z=ODD), dict(c=ODD)):
        assert bwd(**bad) == BAD, bad
    size = lib.mok_grouped_linear_bwd_workspace_bytes
    assert size(4, 3, 12, 0, 0, 0) == 0 and size(-1, 3, 64, 0, 0, 0) == 0 and size(4, 0, 64, 0, 0, 0) == 0
    assert size(4, 3, 64, 9, 0, 0) == 0 and size(4, 3, 64, 0, 2, 0) == 0 and size(0, 3, 64, 3, 0, 1) > 0
    assert size(4096, 3, 64, 3, 0, 0) >= 2 * 4096 * 64 + size(4096, 3, 64, 0, 0, 0) - 512
    assert size(4096, 3, 64, 0, 0, 1) > size(4096, 3, 64, 0, 0, 0)


def test_int4_refusals_and_sizes(lib):
    n = [C.c_size_t() for _ in range(3)]
    sizes = lambda *a: lib.mok_int4_bytes(*a, *(C.byref(v) for v in n))  # noqa: E731
    assert sizes(2, 17, 320, 64) == 0        # 2 row tiles of 16 and 3 blocks of 128 each
    assert [v.value for v in n] == [2 * 2 * 3 * 1024, 2 * 2 * 3 * 16 * 2 * 2, 2 * 2 * 3 * 16 * 2]
    for bad in ((0, 16, 128, 64), (1, 0, 128, 64), (1, 16, 0, 64), (1, 16, 96, 64), (1, 16, 128, 16), (1, 16, 128, 0),
                (1 << 31, 16, 128, 64), (1 << 30, 1 << 20, 1 << 20, 128)):
        assert sizes(*bad) == BAD, bad
    assert lib.mok_int4_bytes(1, 16, 128, 64, None, None, None) == 0

    def quant(w=FAKE, wd=0, e=1, N=16, K=128, g=64, c=FAKE, s=FAKE, z=None):
        return lib.mok_int4_quantize(w, wd, e, N, K, g, c, s, z, None)

    def pack(q=FAKE, qs=FAKE, qz=None, e=1, N=16, K=128, g=64, c=FAKE, s=FAKE, z=None):
        return lib.mok_int4_pack(q, qs, qz, e, N, K, g, c, s, z, None)

    def deq(c=FAKE, s=FAKE, z=None, e=1, N=16, K=128, g=64, out=FAKE):
        return lib.mok_int4_dequantize(c, s, z, e, N, K, g, out, None)

    def lin(x=FAKE, c=FAKE, s=FAKE, z=None, e=1, N=16, K=128, g=64, ids=None, rows=4, each=1, b=None, bd=0, act=0, y=FAKE, yd=0):
        return lib.mok_int4_linear(x, c, s, z, e, N, K, g, ids, rows, each, b, bd, act, y, yd, None)

    for f, more in ((quant, (dict(wd=2), dict(w=None), dict(c=None), dict(s=None), dict(w=ODD), dict(c=ODD), dict(z=ODD))),
                    (pack, (dict(q=None), dict(qs=None), dict(qz=FAKE), dict(z=FAKE), dict(q=ODD), dict(qz=ODD, z=FAKE))),
                    (deq, (dict(c=None), dict(s=None), dict(out=None), dict(out=ODD), dict(c=ODD))),
                    (lin, (dict(rows=-1), dict(rows=65536), dict(each=0), dict(e=2), dict(each=2), dict(act=5), dict(act=-1), dict(yd=2),
                           dict(b=FAKE, bd=3), dict(x=None), dict(c=None), dict(s=None), dict(y=None), dict(x=ODD), dict(c=ODD),
                           dict(s=ODD), dict(z=ODD), dict(ids=ODD), dict(b=ODD), dict(y=ODD)))):
        for bad in more + (dict(e=0), dict(N=0), dict(K=96), dict(g=48)):
            assert f(**bad) == BAD, (f, bad)
    assert lin(rows=0) == 0


def test_python_faces_refuse_cpu_tensors_and_wrong_shapes():
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(3, 32, 64, dtype=torch.bfloat16)
    c, ids = torch.zeros(3, dtype=I32), torch.zeros(4, 2, dtype=I64)
    for call in (lambda: mok.route(x, 2), lambda: mok.route(x, 2, score="top"), lambda: mok.route(None, 2),
                 lambda: mok.route_backward(x, x, ids), lambda: mok.route_backward(x, x, None), lambda: mok.grouped_linear(x, w, c),
                 lambda: mok.grouped_linear(x, w, c, activation="swish"), lambda: mok.grouped_linear_backward(x, x, w, c),
                 lambda: mok.int4_quantize(x), lambda: mok.int4_pack(x, x), lambda: mok.int4_linear(x, w),
                 lambda: mok.int4_dequantize(w)):
        with pytest.raises(ValueError):
            call()




def _calls():
    """name -> (call of tensors, the tensors' shapes and types)"""
    M, N, K, E = 4, 32, 64, 3
    weight = lambda c, s, z: experts.Int4Weight(c, s, z, (E, N, K), 64)  # noqa: E731
    return {
        "route": (lambda x, b: mok.route(x, 2, bias=b, balance=True), [((M, E), F32), ((E,), F32)]),
        "route_backward": (lambda dw, x, i, dl, dm: mok.route_backward(dw, x, i, d_lse=dl, d_mean_score=dm),
                           [((M, 2), F32), ((M, E), BF16), ((M, 2), I64), ((M,), F32), ((E,), F32)]),
        "grouped_linear": (lambda x, w, c, b: mok.grouped_linear(x, w, c, bias=b),
                           [((M, K), BF16), ((E, N, K), BF16), ((E,), I32), ((E, N), F32)]),
        "grouped_linear_backward": (lambda dy, x, w, c, z: mok.grouped_linear_backward(dy, x, w, c, z=z, activation="gelu", bias=True),
                                    [((M, N), BF16), ((M, K), BF16), ((E, N, K), BF16), ((E,), I32), ((M, N), BF16)]),
        "int4_quantize": (lambda w: mok.int4_quantize(w, 64), [((E, N, K), BF16)]),
        "int4_pack": (mok.int4_pack, [((E, N, K // 2), U8), ((E, N, 1), BF16), ((E, N, 1), U8)]),
        "int4_dequantize": (lambda c, s, z: mok.int4_dequantize(weight(c, s, z)), [((64,), U8), ((64,), BF16), ((64,), U8)]),
        "int4_linear": (lambda x, c, s, z, i, b: mok.int4_linear(x, weight(c, s, z), bias=b, experts=i),
                        [((M, K), BF16), ((64,), U8), ((64,), BF16), ((64,), U8), ((M, 2), I64), ((E, N), F32)]),
    }


@pytest.mark.parametrize("name", sorted(_calls()))
def test_operators_refuse_other_devices(stub, monkeypatch, name):  # noqa: F811
    monkeypatch.setattr(experts, "_int4_sizes", lambda *a: (64, 64, 64))
    monkeypatch.setattr(experts, "_workspace", lambda *a: 4096)
    monkeypatch.setattr(experts, "_new", lambda shape, dtype, dev: torch.zeros(shape, dtype=dtype))
    call, args = _calls()[name]
    make = lambda index, **other: [on(other.get(f"a{i}", index), *s, dtype=d)  # noqa: E731
                                   for i, (s, d) in enumerate(args)]
    with pytest.raises(Launched):
        call(*make(0))
    with pytest.raises(ValueError, match="cuda:1"):
        call(*make(1))
    for i in range(len(args)):
        with pytest.raises(ValueError, match="cuda:"):
            call(*make(0, **{f"a{i}": 1}))
