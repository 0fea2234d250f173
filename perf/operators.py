"""Cases, plain forms and work counts of the operators around the mixture-of-experts layer.

Three families: the root-mean-square norm with the residual's addition and an
MXFP8 output (forward and backward), the dense projection with bias,
activation and residual in its epilogue (forward and backward), and the AdamW
step over many tensors with 32-bit or MXFP8 states.

``own`` false: ``run`` computes an operator from elementary torch operations
in 32 bits.  ``own`` true: ``run`` makes the package's calls.  ``exact``
restates the definitions in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

BF16, F32 = torch.bfloat16, torch.float32
TYPES = {"bf16": BF16, "f32": F32}
EPS = 1e-6
BETAS, ADAM_EPS, DECAY, LR, FIRST_STEP, SEED = (0.9, 0.95), 1e-8, 0.1, 3e-4, 100, 1234


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one decoded token through a large layer's norm, MXFP8 codes for the next projection
        dict(name="norm_token_mxfp8", op="norm", rows=1, H=7168, x="bf16", residual="bf16", mxfp8=True),
        # the large layer's batch of 65536 tokens: bf16 stream in and out, normalised in bf16
        dict(name="norm_large", op="norm", rows=65536, H=7168, x="bf16", residual="bf16", mxfp8=False),
        # a prefill batch with a 32-bit residual stream, MXFP8 output only
        dict(name="norm_prefill_mxfp8", op="norm", rows=16384, H=4096, x="bf16", residual="f32", mxfp8=True),
        # training: the norm's gradient joined with the stream's own, at the T = 4096 layer's width
        dict(name="norm_backward", op="norm_backward", rows=4096, H=2048, residual="bf16"),
        # one decoded token: output projection, bias and residual added in the epilogue
        dict(name="linear_token", op="linear", M=1, N=7168, K=2048, bias=True, act="none", residual=True, out="bf16",
             save_z=False),
        # the router's logits for 4096 tokens and 256 experts, in 32 bits
        dict(name="linear_router", op="linear", M=4096, N=256, K=7168, bias=True, act="none", residual=False,
             out="f32", save_z=False),
        # a dense block's first projection in training: bias, GELU, pre-activation kept
        dict(name="linear_gelu", op="linear", M=16384, N=8192, K=2048, bias=True, act="gelu", residual=False,
             out="bf16", save_z=True),
        # a ragged batch with an odd token count
        dict(name="linear_ragged", op="linear", M=1003, N=1416, K=2056, bias=False, act="silu", residual=True,
             out="bf16", save_z=False),
        # the gradient of a dense block's first projection
        dict(name="linear_backward", op="linear_backward", M=8192, N=4096, K=2048, bias=True, act="gelu"),
        # the norms, biases and small matrices of a model: many little tensors, where launches count
        dict(name="adamw_many", op="adamw", tensors=96, numel=20000, param="f32", grad="f32", state="fp32",
             master=False),
        # one T = 4096 layer's routed weights (3 x 64 x 1024 x 2048) with 32-bit master copies and states
        dict(name="adamw_master", op="adamw", tensors=3, numel=134217728, param="bf16", grad="bf16", state="fp32",
             master=True),
        # the same weights with MXFP8 states and 32-bit master copies
        dict(name="adamw_mxfp8", op="adamw", tensors=3, numel=134217728, param="bf16", grad="bf16", state="mxfp8",
             master=True),
    ]


def _log_int(rng, lo, hi):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return min(hi, max(lo, n))


def _width(rng, lo, hi, step):
    n = max(lo, _log_int(rng, lo, hi) // step * step)
    return n + step if n == 3072 else n


def draw(rng):
    op = rng.choice(["norm", "norm_backward", "linear", "linear", "linear_backward", "adamw"])
    if op == "norm":
        mx = rng.random() < 0.5
        H = _width(rng, 64, 8192, 32) if mx else _width(rng, 17, 8192, rng.choice([1, 8]))
        return dict(op=op, rows=_log_int(rng, 1, 32768), H=H, x=rng.choice(["bf16", "bf16", "f32"]),
                    residual=rng.choice(["none", "bf16", "f32"]), mxfp8=mx)
    if op == "norm_backward":
        return dict(op=op, rows=_log_int(rng, 1, 16384), H=_width(rng, 17, 8192, rng.choice([1, 8])),
                    residual=rng.choice(["bf16", "f32"]))
    if op == "linear":
        return dict(op=op, M=_log_int(rng, 1, 8192), N=_width(rng, 8, 8192, 8), K=_width(rng, 64, 4096, 8),
                    bias=rng.random() < 0.5, act=rng.choice(["none", "relu", "silu", "gelu", "gelu_tanh"]),
                    residual=rng.random() < 0.5, out=rng.choice(["bf16", "bf16", "f32"]),
                    save_z=rng.random() < 0.3)
    if op == "linear_backward":
        return dict(op=op, M=_log_int(rng, 1, 8192), N=_width(rng, 8, 4096, 8), K=_width(rng, 64, 4096, 8),
                    bias=rng.random() < 0.5, act=rng.choice(["none", "relu", "silu", "gelu", "gelu_tanh"]))
    tensors = _log_int(rng, 1, 120)
    param = rng.choice(["bf16", "f32"])
    return dict(op=op, tensors=tensors, numel=_log_int(rng, 33, 100_000_000 // tensors), param=param,
                grad="f32" if param == "f32" else rng.choice(["bf16", "f32"]),
                state=rng.choice(["fp32", "mxfp8"]), master=param == "bf16" and rng.random() < 0.5)


def _sizes(c):
    """The lengths of an AdamW case's tensors: around `numel`, no two neighbours alike, odd ones among them when
    there are many of them."""
    n, t = c["numel"], c["tensors"]
    return [n] * t if t <= 3 else [max(1, n - (n * (i % 7)) // 9 + (i % 3)) for i in range(t)]


# ---------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, shape, std=1.0, dtype=F32):
    if dtype == F32:
        return torch.randn(shape, generator=g, device="cuda", dtype=F32).mul_(std)
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype).mul_(std)


def _stream(g, rows, H, dtype):
    """A residual stream: unit noise with a few channels that are much larger, as trained models have."""
    s = _normal(g, (rows, H), 1.0, dtype)
    s[:, torch.randint(0, H, (max(1, H // 512),), generator=g, device="cuda")] *= 20.0
    return s


def prepare(c, seed):
    g = _gen(seed)
    st = dict(c=c)
    op = c["op"]
    if op == "norm":
        st["x"] = _normal(g, (c["rows"], c["H"]), 1.0, TYPES[c["x"]])
        st["residual"] = None if c["residual"] == "none" else _stream(g, c["rows"], c["H"], TYPES[c["residual"]])
        st["weight"] = (1.0 + _normal(g, (c["H"],), 0.1)).to(BF16)
    elif op == "norm_backward":
        st["h"] = _stream(g, c["rows"], c["H"], TYPES[c["residual"]])
        st["rstd"] = torch.rsqrt(st["h"].float().square().mean(-1) + EPS)
        st["weight"] = (1.0 + _normal(g, (c["H"],), 0.1)).to(BF16)
        st["dy"] = _normal(g, (c["rows"], c["H"]), 1.0, BF16)
        st["dh"] = _normal(g, (c["rows"], c["H"]), 1.0, TYPES[c["residual"]])
    elif op == "linear":
        st["x"] = _normal(g, (c["M"], c["K"]), 1.0, BF16)
        st["weight"] = _normal(g, (c["N"], c["K"]), 1.0 / math.sqrt(c["K"]), BF16)
        st["bias"] = _normal(g, (c["N"],), 0.1, TYPES[c["out"]]) if c["bias"] else None
        st["residual"] = _normal(g, (c["M"], c["N"]), 1.0, BF16) if c["residual"] else None
    elif op == "linear_backward":
        st["x"] = _normal(g, (c["M"], c["K"]), 1.0, BF16)
        st["weight"] = _normal(g, (c["N"], c["K"]), 1.0 / math.sqrt(c["K"]), BF16)
        st["z"] = _normal(g, (c["M"], c["N"]), 1.0, BF16) if c["act"] != "none" else None
        st["dy"] = _normal(g, (c["M"], c["N"]), 1.0, BF16)
    else:
        _prepare_adamw(st, c, g)
    return st


def _spans(c):
    """[(first element, length)] of the tensors in the flat buffers a program keeps them in: each begins on a block of
    32 elements; and the buffers' length."""
    at, spans = 0, []
    for n in _sizes(c):
        spans.append((at, n))
        at += -(-n // 32) * 32
    return spans, at


def _prepare_adamw(st, c, g):
    spans, total = _spans(c)
    w = _normal(g, (total,), 0.02)
    before = _normal(g, (total,), 1e-3).mul_(torch.rand((total,), generator=g, device="cuda").add_(0.1))
    for first, n in spans:   # the gaps between the tensors hold zeros
        w[first + n:first + -(-n // 32) * 32] = 0
        before[first + n:first + -(-n // 32) * 32] = 0
    flat = dict(params=w.to(TYPES[c["param"]]), grads=_normal(g, (total,), 1e-3, TYPES[c["grad"]]))
    if c["master"]:
        flat["masters"] = w
    m = before * 0.3
    v = before.square_().mul_(0.5)
    if c["state"] == "fp32":
        flat.update(m=m, v=v)
    else:   # codes and scales, as steps before this one left them
        flat["m"], flat["m_scale"] = _mx_encode(m)
        flat["r"], flat["r_scale"] = _mx_encode(v.sqrt_())
    parts = {k: [t[f // 32:f // 32 + -(-n // 32)] if k.endswith("_scale") else t[f:f + n] for f, n in spans]
             for k, t in flat.items()}
    st.update(flat=flat, parts=parts, step=FIRST_STEP, grad_scale=torch.full((1,), 0.5, device="cuda"))
    if own:   # the optimiser that a program keeps, over the same buffers
        import mixture_experts_layer_mok_gb300 as mok

        st["opt"] = mok.AdamW(parts["params"], lr=LR, betas=BETAS, eps=ADAM_EPS, weight_decay=DECAY, state=c["state"],
                              seed=SEED, step=FIRST_STEP, buffers={k: parts[k] for k in parts
                                                                   if k not in ("params", "grads")})


# ---------------------------------------------------------------- MXFP8 in plain form
def _mx_exponent(blocks):
    """Per block the smallest s with amax <= 448 * 2^s, 0 for a block of zeros."""
    amax = blocks.abs().amax(-1, keepdim=True)
    mant, e = torch.frexp(amax)
    s = torch.where(mant <= 0.875, e - 9, e - 8).clamp(-127, 127)
    return torch.where(amax == 0, torch.zeros_like(s), s)


def _pow2(e):
    """2^e for whole e (int32), from the bits of the exponent."""
    return ((e.clamp(-126, 127) + 127) << 23).view(F32)


def _blocks(v):
    n = v.shape[-1]
    pad = -n % 32
    if pad:
        v = torch.cat([v, v.new_zeros(v.shape[:-1] + (pad,))], -1)
    return v.reshape(v.shape[:-1] + (-1, 32))


def _mx_encode(v):
    """fp32 [..., n] -> (E4M3 codes uint8 [..., n], E8M0 scales uint8 [..., ceil(n / 32)]), to nearest."""
    b = _blocks(v)
    s = _mx_exponent(b)
    codes = (b * _pow2(-s)).to(torch.float8_e4m3fn).view(torch.uint8).reshape(v.shape[:-1] + (-1,))
    return codes[..., :v.shape[-1]].contiguous(), (s + 127).to(torch.uint8).squeeze(-1).contiguous()


def _mx_decode(codes, scales):
    """The fp32 values that codes and scales stand for."""
    b = _blocks(codes.view(torch.float8_e4m3fn).to(F32))
    v = b * _pow2(scales.to(torch.int32).unsqueeze(-1) - 127)
    return v.reshape(codes.shape[:-1] + (-1,))[..., :codes.shape[-1]]


def _mix(i, key):
    """32 mixed bits for each flat index: multiply, xor-shift, multiply, xor-shift, modulo 2^32."""
    low = 0xFFFFFFFF
    h = ((i + key) * 0x9E3779B1) & low
    h = h ^ (h >> 15)
    h = (h * 0xB504F333) & low
    return h ^ (h >> 16)


def _mx_stochastic(v, rand16, keep_positive):
    """The values that the state keeps of fp32 v [n]: per block of 32 on the E4M3 grid times a power of two, rounded up
    or down with the probabilities that make it right on average, by 16 random bits each.  keep_positive: a positive
    value is never rounded to zero."""
    n = v.shape[-1]
    b = _blocks(v)
    s = _mx_exponent(b)
    y = b * _pow2(-s)
    a = y.abs()
    small = a < 2.0 ** -6
    t = torch.where(small, a + 2.0 ** -6, a)
    bits = t.view(torch.int32) + (_blocks(rand16) << 4)
    q = (bits & -0x100000).view(F32)
    q = torch.where(small, q - 2.0 ** -6, q)
    if keep_positive:
        q = torch.where((a > 0) & (q == 0), torch.full_like(q, 2.0 ** -9), q)
    return (torch.copysign(q, y) * _pow2(s)).reshape(-1)[:n]


# ---------------------------------------------------------------- one pass
def run(st):
    return (_run_own if own else _run_plain)(st, st["c"])


def _run_own(st, c):
    import mixture_experts_layer_mok_gb300 as mok

    op = c["op"]
    if op == "norm":
        r = mok.rms_norm(st["x"], st["weight"], residual=st["residual"], eps=EPS, bf16=not c["mxfp8"],
                         mxfp8=c["mxfp8"])
        out = dict(y=mok.mxfp8_dequantize(*r.mx) if c["mxfp8"] else r.y, rstd=r.rstd)
        if st["residual"] is not None:
            out["h"] = r.h
        return out
    if op == "norm_backward":
        g = mok.rms_norm_backward(st["dy"], st["h"], st["weight"], st["rstd"], d_h=st["dh"])
        return dict(dx=g["dx"], d_weight=g["d_weight"])
    if op == "linear":
        y, z = mok.linear(st["x"], st["weight"], bias=st["bias"], activation=c["act"], residual=st["residual"],
                          out_dtype=TYPES[c["out"]], save_z=c["save_z"])
        return dict(y=y, z=z) if c["save_z"] else dict(y=y)
    if op == "linear_backward":
        return mok.linear_backward(st["dy"], st["x"], st["weight"], z=st["z"], activation=c["act"], bias=c["bias"])
    st["opt"].step(st["parts"]["grads"], grad_scale=st["grad_scale"])
    flat = st["flat"]
    if c["state"] == "fp32":
        return _step_outputs(flat, flat["m"], flat["v"])
    return _step_outputs(flat, mok.mxfp8_dequantize(flat["m"], flat["m_scale"]),
                         mok.mxfp8_dequantize(flat["r"], flat["r_scale"]))


def _step_outputs(flat, m, v):
    out = dict(params=flat["params"], m=m, v=v)
    if "masters" in flat:
        out["masters"] = flat["masters"]
    return out


def _act(z, act):
    if act == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-z))
        return s * (1.0 + z * (1.0 - s))
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    a, b = math.sqrt(2.0 / math.pi), 0.044715
    t = torch.tanh(a * (z + b * z * z * z))
    return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * a * (1.0 + 3.0 * b * z * z)


def _run_plain(st, c):
    op = c["op"]
    if op == "norm":
        h = st["x"].float()
        if st["residual"] is not None:
            h = h + st["residual"].float()
        rstd = torch.rsqrt(h.square().mean(-1) + EPS)
        y = h * rstd.unsqueeze(-1) * st["weight"].float()
        out = dict(y=_mx_decode(*_mx_encode(y)).to(BF16) if c["mxfp8"] else y.to(BF16), rstd=rstd)
        if st["residual"] is not None:
            out["h"] = h.to(st["residual"].dtype)
        return out
    if op == "norm_backward":
        h, dy = st["h"].float(), st["dy"].float()
        xhat = h * st["rstd"].unsqueeze(-1)
        gy = dy * st["weight"].float()
        dx = (gy - xhat * (gy * xhat).mean(-1, keepdim=True)) * st["rstd"].unsqueeze(-1) + st["dh"].float()
        return dict(dx=dx.to(st["h"].dtype), d_weight=(dy * xhat).sum(0))
    if op == "linear":
        z = st["x"].float() @ st["weight"].float().t()
        if st["bias"] is not None:
            z = z + st["bias"].float()
        y = _act(z, c["act"])
        if st["residual"] is not None:
            y = y + st["residual"].float()
        out = dict(y=y.to(TYPES[c["out"]]))
        if c["save_z"]:
            out["z"] = z.to(BF16)
        return out
    if op == "linear_backward":
        dz = st["dy"].float()
        if c["act"] != "none":
            dz = dz * _act_grad(st["z"].float(), c["act"])
        out = dict(dx=(dz @ st["weight"].float()).to(BF16), d_weight=(dz.t() @ st["x"].float()).to(BF16))
        if c["bias"]:
            out["d_bias"] = dz.sum(0)
        return out
    st["step"] += 1
    flat = st["flat"]
    for i in range(c["tensors"]):
        _adamw_plain({k: t[i] for k, t in st["parts"].items()}, c, i, st["step"], st["grad_scale"])
    if c["state"] == "fp32":
        return _step_outputs(flat, flat["m"], flat["v"])
    return _step_outputs(flat, _mx_decode(flat["m"], flat["m_scale"]).to(BF16),
                         _mx_decode(flat["r"], flat["r_scale"]).to(BF16))


def _adamw_plain(t, c, i, step, grad_scale):
    """Tensor i's step, in place."""
    b1, b2 = BETAS
    mx = c["state"] == "mxfp8"
    g = t["grads"].float() * grad_scale
    p = t["masters"] if c["master"] else t["params"].float()
    m = b1 * (_mx_decode(t["m"], t["m_scale"]) if mx else t["m"]) + (1.0 - b1) * g
    v = b2 * (_mx_decode(t["r"], t["r_scale"]).square() if mx else t["v"]) + (1.0 - b2) * g * g
    r = v.sqrt()
    upd = (m / (1.0 - b1 ** step)) / (r / math.sqrt(1.0 - b2 ** step) + ADAM_EPS)
    p = p * (1.0 - LR * DECAY) - LR * upd
    t["params"].copy_(p)
    if c["master"]:
        t["masters"].copy_(p)
    if not mx:
        t["m"].copy_(m)
        t["v"].copy_(v)
        return
    key = (SEED * 0x9E3779B1 + step * 0xB504F333 + i * 0xBB67AE85) & 0xFFFFFFFF
    rand = _mix(torch.arange(m.numel(), device="cuda"), key)
    m = _mx_stochastic(m, (rand >> 16).to(torch.int32), False)
    r = _mx_stochastic(r, (rand & 0xFFFF).to(torch.int32), True)
    for name, q in (("m", m), ("r", r)):   # each value is on the grid of its block's scale
        codes, scales = _mx_encode(q)
        t[name].copy_(codes)
        t[name + "_scale"].copy_(scales)


# ---------------------------------------------------------------- 64 bits
def exact(c, seed):
    st = prepare(c, seed)
    op = c["op"]
    d = torch.float64
    if op == "norm":
        h = st["x"].to(d) + (0.0 if st["residual"] is None else st["residual"].to(d))
        ms = (h * h).sum(1) / c["H"] + EPS
        out = dict(y=None if c["mxfp8"] else h / ms.sqrt()[:, None] * st["weight"].to(d)[None, :], rstd=ms ** -0.5)
        if st["residual"] is not None:
            out["h"] = h
        return out
    if op == "norm_backward":
        # y_j = w_j h_j r with r the saved factor, d r / d h_k = -r^3 h_k / H
        h, dy, w, r = st["h"].to(d), st["dy"].to(d), st["weight"].to(d), st["rstd"].to(d)[:, None]
        dot = (dy * w * h).sum(1, keepdim=True)
        return dict(dx=st["dh"].to(d) + r * dy * w - r ** 3 * h * dot / c["H"], d_weight=torch.einsum("ij,ij->j", dy, h * r))
    if op == "linear":
        z = torch.einsum("mk,nk->mn", st["x"].to(d), st["weight"].to(d))
        z = z if st["bias"] is None else z + st["bias"].to(d)
        y = _exact_act(z, c["act"])
        y = y if st["residual"] is None else y + st["residual"].to(d)
        return dict(y=y, z=z) if c["save_z"] else dict(y=y)
    if op == "linear_backward":
        dz = st["dy"].to(d)
        if c["act"] != "none":
            z = st["z"].to(d).requires_grad_(True)
            dz, = torch.autograd.grad(_exact_act(z, c["act"]), z, dz)
        out = dict(dx=torch.einsum("mn,nk->mk", dz, st["weight"].to(d)),
                   d_weight=torch.einsum("mn,mk->nk", dz, st["x"].to(d)))
        if c["bias"]:
            out["d_bias"] = torch.einsum("mn->n", dz)
        return out
    return _exact_adamw(st, c)


def _exact_act(z, act):
    if act == "none":
        return z
    if act == "relu":
        return z.clamp(min=0.0)
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return z * torch.special.ndtr(z)
    return z * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3))


def _exact_adamw(st, c):
    d, (b1, b2), t, flat = torch.float64, BETAS, FIRST_STEP + 1, st["flat"]
    mx = c["state"] == "mxfp8"
    used = torch.zeros(flat["params"].numel(), dtype=torch.bool, device="cuda")
    for first, n in _spans(c)[0]:
        used[first:first + n] = True
    g = flat["grads"].to(d) * 0.5
    old = flat["masters" if c["master"] else "params"].to(d)
    m = _exact_values(flat["m"], flat["m_scale"]) if mx else flat["m"].to(d)
    v = _exact_values(flat["r"], flat["r_scale"]) ** 2 if mx else flat["v"].to(d)
    m += (1 - b1) * (g - m)
    v += (1 - b2) * (g * g - v)
    p = old - LR * (DECAY * old + m / (1 - b1 ** t) / ((v / (1 - b2 ** t)).sqrt() + ADAM_EPS))
    zero = torch.zeros((), dtype=d, device="cuda")   # the gaps stay as they were
    p, m, v = (torch.where(used, new, was) for new, was in ((p, old), (m, zero), (v, zero)))
    out = dict(params=p, m=None if mx else m, v=None if mx else v)   # which way a kept value was rounded: no answer
    if c["master"]:
        out["masters"] = p
    return out


def _exact_values(codes, scales):
    x = codes.to(torch.int64)
    e, f = (x >> 3) & 15, (x & 7).to(torch.float64)
    a = torch.where(e == 0, f * 2.0 ** -9, (8.0 + f) * torch.pow(2.0, (e - 10).to(torch.float64)))
    a = torch.where(x >= 128, -a, a)
    return a * torch.pow(2.0, scales.to(torch.float64) - 127.0).repeat_interleave(32)


# ---------------------------------------------------------------- work
def _bytes(t):
    return {"bf16": 2, "f32": 4, "none": 0}[t]


def work(c):
    op = c["op"]
    if op == "norm":
        n = c["rows"] * c["H"]
        out = 33 / 32 if c["mxfp8"] else 2
        return dict(bytes=n * (_bytes(c["x"]) + 2 * _bytes(c["residual"]) + out) + 2 * c["H"] + 4 * c["rows"],
                    flops=6 * n)
    if op == "norm_backward":
        n = c["rows"] * c["H"]
        return dict(bytes=n * (2 + 3 * _bytes(c["residual"])) + 6 * c["H"] + 4 * c["rows"], flops=11 * n)
    if op == "linear":
        M, N, K = c["M"], c["N"], c["K"]
        out = _bytes(c["out"])
        return dict(bytes=2 * (M * K + N * K) + M * N * (out + 2 * c["residual"] + 2 * c["save_z"])
                    + N * out * c["bias"], flops=2 * M * N * K)
    if op == "linear_backward":
        M, N, K = c["M"], c["N"], c["K"]
        act = c["act"] != "none"
        return dict(bytes=2 * (M * N * (1 + act) + 2 * M * K + 2 * N * K) + 4 * N * c["bias"], flops=4 * M * N * K)
    n = sum(_sizes(c))
    state = 4 * (33 / 32) if c["state"] == "mxfp8" else 16
    p = _bytes(c["param"])
    return dict(bytes=n * (_bytes(c["grad"]) + (p + 8 if c["master"] else 2 * p) + state), flops=15 * n)
