"""CPU-side checks of the operators around the layer: sizes, refusals before
any device work, and the Python faces' own checks."""
import ctypes as C

import pytest
import torch


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__ as g

    g.build()
    from mixture_experts_layer_mok_gb300 import _lib

    return _lib.load()


FAKE, ODD = C.c_void_p(16), C.c_void_p(24)      # never dereferenced: validation fails first
BAD = 1                                           # MOK_ERR_INVALID_ARG


def test_dequantize_refusals(lib):
    f = lib.mok_mxfp8_dequantize
    assert f(FAKE, FAKE, -1, 32, FAKE, None) == BAD and f(FAKE, FAKE, 2, 40, FAKE, None) == BAD
    assert f(None, FAKE, 1, 32, FAKE, None) == BAD and f(ODD, FAKE, 1, 32, FAKE, None) == BAD
    assert f(FAKE, FAKE, 1, 32, ODD, None) == BAD and f(FAKE, FAKE, 1 << 40, 1 << 40, FAKE, None) == BAD
    assert f(None, None, 0, 32, None, None) == 0 and f(None, None, 3, 0, None, None) == 0


def test_norm_refusals_and_sizes(lib):
    def fwd(x=FAKE, xd=0, r=None, rd=0, w=FAKE, wd=0, rows=4, H=64, eps=1e-6, h=None, y=FAKE, q=None, s=None, rstd=FAKE):
        return lib.mok_rms_norm(x, xd, r, rd, w, wd, rows, H, eps, h, y, q, s, rstd, None)

    for bad in (dict(rows=-1), dict(rows=1 << 31), dict(H=0), dict(H=32769), dict(xd=2), dict(wd=-1), dict(r=FAKE, rd=7, h=FAKE),
                dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(y=None), dict(q=FAKE), dict(s=FAKE),
                dict(q=FAKE, s=FAKE, H=40), dict(x=None), dict(w=None), dict(rstd=None), dict(r=FAKE), dict(x=ODD),
                dict(w=ODD), dict(y=ODD), dict(q=ODD, s=FAKE), dict(r=ODD, h=FAKE), dict(r=FAKE, h=ODD)):
        assert fwd(**bad) == BAD, bad
    assert fwd(rows=0) == 0

    def bwd(dy=FAKE, h=FAKE, hd=0, w=FAKE, wd=0, rstd=FAKE, dh=None, rows=4, H=64, dx=FAKE, d16=None, dw=FAKE, ws=FAKE,
            n=1 << 30):
        return lib.mok_rms_norm_bwd(dy, h, hd, w, wd, rstd, dh, rows, H, dx, d16, dw, ws, n, None)

    for bad in (dict(rows=-1), dict(H=0), dict(hd=3), dict(wd=3), dict(d16=FAKE), dict(dw=None), dict(ws=None), dict(dy=None),
                dict(dx=None), dict(n=16), dict(dy=ODD), dict(dh=ODD), dict(dw=ODD)):
        assert bwd(**bad) == BAD, bad
    size = lib.mok_rms_norm_bwd_workspace_bytes
    assert size(-1, 64) == 0 and size(4, 0) == 0 and size(4, 32769) == 0
    # at least one row of partial sums, and no more than the grid of blocks needs
    assert size(0, 64) > 0 and size(4, 64) >= 64 * 4 and size(1 << 20, 8192) < 1 << 25


def test_linear_refusals_and_sizes(lib):
    def fwd(x=FAKE, w=FAKE, b=None, bd=0, r=None, rd=0, act=0, M=4, N=64, K=64, y=FAKE, yd=0, z=None):
        return lib.mok_linear(x, w, b, bd, r, rd, act, M, N, K, y, yd, z, None)

    for bad in (dict(M=-1), dict(M=(1 << 31) - 1), dict(N=0), dict(N=12), dict(K=0), dict(K=36), dict(act=5), dict(act=-1),
                dict(yd=2), dict(b=FAKE, bd=2), dict(r=FAKE, rd=2), dict(x=None), dict(w=None), dict(y=None), dict(x=ODD),
                dict(w=ODD), dict(b=ODD), dict(r=ODD), dict(y=ODD), dict(z=ODD)):
        assert fwd(**bad) == BAD, bad
    assert fwd(M=0) == 0

    def bwd(dy=FAKE, dd=0, x=FAKE, w=FAKE, z=None, act=0, M=4, N=64, K=64, dx=FAKE, dw=FAKE, db=None, ws=FAKE, n=1 << 30):
        return lib.mok_linear_bwd(dy, dd, x, w, z, act, M, N, K, dx, dw, db, ws, n, None)

    for bad in (dict(M=-1), dict(N=12), dict(K=36), dict(act=9), dict(dd=2), dict(dy=None), dict(x=None), dict(w=None),
                dict(act=3), dict(ws=None), dict(n=8), dict(act=3, z=FAKE, n=300), dict(dy=ODD), dict(dx=ODD), dict(dw=ODD),
                dict(db=ODD), dict(z=ODD)):
        assert bwd(**bad) == BAD, bad
    size = lib.mok_linear_bwd_workspace_bytes
    assert size(4, 12, 0, 0, 0) == 0 and size(-1, 64, 0, 0, 0) == 0 and size(4, 64, 9, 0, 0) == 0 and size(4, 64, 0, 2, 0) == 0
    assert size(4, 64, 0, 0, 0) < 1024                     # bf16 dy, no activation: dy is dz
    assert size(4096, 64, 3, 0, 0) >= 2 * 4096 * 64 and size(4096, 64, 0, 1, 0) >= 2 * 4096 * 64
    assert size(4096, 64, 0, 0, 1) > size(4096, 64, 0, 0, 0)


def test_adamw_refusals(lib):
    from mixture_experts_layer_mok_gb300 import _lib

    def step(cfg=None, n=64, num=1, **fields):
        c = dict(param_dtype=1, grad_dtype=1, state=0, lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.0, step=1)
        c.update(cfg or {})
        t = dict(p=16, master=None, g=16, m=16, v=16, m_scale=None, v_scale=None, n=n, index=0)
        t.update(fields)
        return lib.mok_adamw_step(C.byref(_lib.MokAdamwConfig(**c)), (_lib.MokAdamwTensor * 1)(_lib.MokAdamwTensor(**t)), num,
                                  None, None)

    assert lib.mok_adamw_step(None, None, 0, None, None) == BAD
    for bad in (dict(param_dtype=2), dict(grad_dtype=2), dict(state=2), dict(lr=float("nan")), dict(beta1=1.0),
                dict(beta1=-0.1), dict(beta2=1.0), dict(beta2=float("nan")), dict(eps=-1.0), dict(eps=float("inf")),
                dict(weight_decay=float("inf")), dict(step=0)):
        assert step(bad) == BAD, bad
    for bad in (dict(n=-1), dict(p=None), dict(g=None), dict(m=None), dict(v=None), dict(p=24), dict(g=24), dict(m=24),
                dict(v=24), dict(master=16), dict(num=-1)):
        assert step(**bad) == BAD, bad
    assert step(dict(state=1)) == BAD                       # MXFP8 states without scales


def test_forward_refuses_half_given_codes(lib):
    from mixture_experts_layer_mok_gb300 import _lib

    s, ctx = _lib.MokSchedule(T=4, k=2, E=8), _lib.MokCtx()
    w = _lib.MokWeights(E=8, H=128, I=128, I_s=0)
    w.w_gate = w.w_up = w.w_down = 16
    for n in ("gate", "up", "down"):
        setattr(w, "mx_" + n, 16)
        setattr(w, "mx_" + n + "_sc", 16)
    for kw in (dict(mode=1, x_codes=16), dict(mode=2, x_scales=16), dict(mode=0, x_codes=16, x_scales=16),
               dict(mode=1, x_codes=24, x_scales=16)):
        cfg = _lib.MokConfig(**kw)
        assert lib.mok_forward(C.byref(cfg), FAKE, FAKE, C.byref(s), C.byref(w), FAKE, FAKE, 1 << 30, C.byref(ctx),
                               None) == BAD
        assert b"x_codes" in lib.mok_last_error()


def test_python_faces_refuse_cpu_tensors_and_wrong_shapes():
    import mixture_experts_layer_mok_gb300 as mok

    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(32, 64, dtype=torch.bfloat16)
    for call in (lambda: mok.rms_norm(x, x[0]), lambda: mok.rms_norm(None, x[0]), lambda: mok.linear(x, w),
                 lambda: mok.linear(x, w, activation="swish"), lambda: mok.linear_backward(x, x, w),
                 lambda: mok.rms_norm_backward(x, x, x[0], x), lambda: mok.mxfp8_dequantize(x, x),
                 lambda: mok.AdamW([x]), lambda: mok.AdamW([], state="fp16")):
        with pytest.raises(ValueError):
            call()
    opt = mok.AdamW([])
    assert opt.state_dict()["step"] == 0
    with pytest.raises(ValueError):
        opt.step([x])


def test_counted_adamw_refusals(lib):
    from mixture_experts_layer_mok_gb300 import _lib

    def cfg(**kw):
        c = dict(param_dtype=1, grad_dtype=1, state=0, lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.0, step=0)
        return _lib.MokAdamwConfig(**{**c, **kw})

    t = (_lib.MokAdamwTensor * 1)(_lib.MokAdamwTensor(p=16, g=16, m=16, v=24, n=64))
    for c, counter in ((cfg(), None), (cfg(), ODD), (cfg(step=-1), FAKE), (cfg(lr=float("inf")), FAKE), (cfg(beta2=1.0), FAKE)):
        assert lib.mok_adamw_advance(C.byref(c), 0, counter, None) == BAD
        assert lib.mok_adamw_step_counted(C.byref(c), t, 0, None, counter, None) == BAD
    assert lib.mok_adamw_advance(None, 0, FAKE, None) == BAD
    assert lib.mok_adamw_step_counted(C.byref(cfg()), t, 1, None, FAKE, None) == BAD     # v is misaligned


def test_adamw_check_is_the_steps_own(lib):
    from mixture_experts_layer_mok_gb300 import _lib

    def check(num=1, step=1, **kw):
        c = dict(param_dtype=1, grad_dtype=1, lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, step=step)
        t = dict(p=16, g=16, m=16, v=16, n=64)
        c.update({k: v for k, v in kw.items() if k in c})
        t.update({k: v for k, v in kw.items() if k not in c})
        return lib.mok_adamw_check(C.byref(_lib.MokAdamwConfig(**c)), (_lib.MokAdamwTensor * 1)(_lib.MokAdamwTensor(**t)), num)

    assert check() == 0 and check(step=0) == 0 and check(g=24, n=0) == 0
    for bad in (dict(num=-1), dict(step=-1), dict(g=24), dict(p=24), dict(v=None), dict(master=16), dict(lr=float("inf")),
                dict(beta1=1.0), dict(n=-1)):
        assert check(**bad) == BAD, bad


def test_norm_backward_in_both_types_refusals(lib):
    def bwd(dy=FAKE, h=FAKE, hd=0, w=FAKE, wd=0, rstd=FAKE, dh=None, rows=4, H=64, dx=FAKE, other=FAKE, dw=FAKE, ws=FAKE,
            n=1 << 30):
        return lib.mok_rms_norm_bwd_both(dy, h, hd, w, wd, rstd, dh, rows, H, dx, other, dw, ws, n, None)

    for hd in (0, 1):
        for bad in (dict(rows=-1), dict(H=0), dict(wd=3), dict(dw=None), dict(ws=None), dict(dy=None), dict(dx=None), dict(n=16),
                    dict(other=ODD), dict(dh=ODD)):
            assert bwd(hd=hd, **bad) == BAD, bad
    assert bwd(hd=2) == BAD
