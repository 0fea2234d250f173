"""Cases, plain forms and work counts of routed experts taken apart: the router, the products grouped by expert, and
the products with 4-bit weights.

Three families: the choice of each token's experts with its weights (forward, and the gradient of the logits), the
dense projection with one weight for each group of rows (forward and backward), and the projection with 4-bit weights
and group scales, of one matrix or of the experts that each token chose.

``own`` false: ``run`` computes an operator from elementary torch operations in 32 bits.  ``own`` true: ``run`` makes
the package's calls.  ``exact`` restates the definitions in 64 bits.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

BF16, F32 = torch.bfloat16, torch.float32
TYPES = {"bf16": BF16, "f32": F32}


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one decoded token's choice among 256 experts
        dict(name="route_token", op="route", T=1, E=256, k=8, score="softmax", normalize=True, scale=1.0, logits="f32",
             balance=False),
        # the large layer's batch in training, with the loads and mean scores of the balance loss
        dict(name="route_batch", op="route", T=65536, E=256, k=8, score="sigmoid", normalize=True, scale=2.5,
             logits="f32", balance=True),
        # the gradient of the logits with the balance and z losses, scores not renormalised, bf16 logits
        dict(name="route_backward", op="route_backward", T=16384, E=64, k=8, score="softmax", normalize=False, scale=1.0,
             logits="bf16", losses=True),
        # 64 decoded tokens of 8 experts each: two rows an expert, bound by the weights' bytes
        dict(name="grouped_decode", op="grouped", M=512, E=256, N=2048, K=7168, tail=0, bias=False, act="none",
             out="bf16", save_z=False),
        # the T = 4096 layer's first product in training: SiLU, pre-activations kept
        dict(name="grouped_train", op="grouped", M=32768, E=64, N=1024, K=2048, tail=0, bias=False, act="silu",
             out="bf16", save_z=True),
        # a long batch
        dict(name="grouped_large", op="grouped", M=131072, E=64, N=2048, K=4096, tail=0, bias=False, act="none",
             out="bf16", save_z=False),
        # a ragged batch of odd sizes with biases, 32-bit outputs and rows behind the last group
        dict(name="grouped_ragged", op="grouped", M=1999, E=12, N=1416, K=2056, tail=37, bias=True, act="gelu",
             out="f32", save_z=False),
        # the gradients of grouped_train
        dict(name="grouped_backward", op="grouped_backward", M=32768, E=64, N=1024, K=2048, tail=0, bias=False,
             act="silu"),
        # small experts with biases, ragged
        dict(name="grouped_backward_ragged", op="grouped_backward", M=3001, E=20, N=712, K=1032, tail=5, bias=True,
             act="gelu_tanh"),
        # one decoded token: output projection in 4 bits
        dict(name="int4_token", op="int4", T=1, k=0, E=0, N=7168, K=2048, group=128, zeros=False, bias=False, act="none",
             out="bf16"),
        # one decoded token through its 8 of 256 experts' first products
        dict(name="int4_experts", op="int4", T=1, k=8, E=256, N=2048, K=7168, group=32, zeros=True, bias=False,
             act="silu", out="bf16"),
        # 32 sequences' logits over a vocabulary, in 32 bits
        dict(name="int4_vocabulary", op="int4", T=32, k=0, E=0, N=152064, K=4096, group=64, zeros=False, bias=False,
             act="none", out="f32"),
    ]


def _log_int(rng, lo, hi):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return min(hi, max(lo, n))


def _width(rng, lo, hi, step):
    return max(lo, _log_int(rng, lo, hi) // step * step)


def draw(rng):
    op = rng.choice(["route", "route_backward", "grouped", "grouped", "grouped_backward", "int4", "int4"])
    acts = ["none", "relu", "silu", "gelu", "gelu_tanh"]
    if op in ("route", "route_backward"):
        E = _log_int(rng, 4, 512)
        c = dict(op=op, T=_log_int(rng, 1, 65536 if op == "route" else 32768), E=E, k=rng.randint(1, min(E, 12)),
                 score=rng.choice(["softmax", "sigmoid"]), normalize=rng.random() < 0.6, scale=rng.choice([1.0, 2.5]),
                 logits=rng.choice(["f32", "f32", "bf16"]))
        c["balance" if op == "route" else "losses"] = rng.random() < 0.5
        return c
    if op in ("grouped", "grouped_backward"):
        N, K = _width(rng, 8, 4096, 8), _width(rng, 64, 4096, 8)
        E = _log_int(rng, 1, max(2, min(128, (1 << 28) // (N * K))))
        M = _log_int(rng, 1, 32768 if op == "grouped" else 16384)
        c = dict(op=op, M=M, E=E, N=N, K=K, tail=rng.choice([0, 0, M // 9]), bias=rng.random() < 0.5, act=rng.choice(acts))
        if op == "grouped":
            c.update(out=rng.choice(["bf16", "bf16", "f32"]), save_z=rng.random() < 0.3)
        return c
    group = rng.choice([32, 64, 128])
    N, K = _width(rng, 8, 16384, 8), max(group, _log_int(rng, 128, 8192) // group * group)
    c = dict(op=op, T=_log_int(rng, 1, 64), k=0, E=0, N=N, K=K, group=group, zeros=rng.random() < 0.5,
             bias=rng.random() < 0.3, act=rng.choice(acts), out=rng.choice(["bf16", "bf16", "f32"]))
    if rng.random() < 0.5:   # of experts; the plain form holds a 32-bit matrix for each row
        c["E"] = rng.randint(2, max(2, min(128, (1 << 29) // (N * K))))
        c["k"] = rng.randint(1, min(8, c["E"]))
        c["T"] = max(1, min(c["T"] // 4, (1 << 31) // (N * K * c["k"])))
    return c


# ---------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, shape, std=1.0, dtype=F32):
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype).mul_(std)


def _logits(g, c):
    """Unit noise around each expert's own level: some are chosen several times as often as others."""
    level = _normal(g, (c["E"],), 0.5)
    return (_normal(g, (c["T"], c["E"])) + level).to(TYPES[c["logits"]])


def _sizes(c, seed):
    """Rows of each expert: shares that differ by several times, empty experts among many."""
    rng = np.random.RandomState((int(seed) * 7919 + c["M"]) % (1 << 32))
    share = np.exp(0.7 * rng.randn(c["E"]))
    if c["E"] > 4:
        share[rng.randint(c["E"])] = 0.0
    return rng.multinomial(c["M"] - c["tail"], share / share.sum())


def prepare(c, seed):
    g = _gen(seed)
    st = dict(c=c)
    op = c["op"]
    if op == "route":
        st["logits"] = _logits(g, c)
    elif op == "route_backward":
        st["logits"] = _logits(g, c)
        st["experts"] = torch.sort(st["logits"], dim=1, descending=True, stable=True).indices[:, :c["k"]].contiguous()
        st["d_weights"] = _normal(g, (c["T"], c["k"]))
        st["d_lse"] = _normal(g, (c["T"],), 1e-2) if c["losses"] else None
        st["d_mean_score"] = _normal(g, (c["E"],), 1.0) if c["losses"] else None
    elif op in ("grouped", "grouped_backward"):
        E, M, N, K = c["E"], c["M"], c["N"], c["K"]
        sizes = _sizes(c, seed)
        st["x"] = _normal(g, (M, K), 1.0, BF16)
        st["weight"] = _normal(g, (E, N, K), 1.0 / math.sqrt(K), BF16)
        st["counts"] = torch.from_numpy(sizes.astype(np.int32)).cuda()
        # where each row lies among its expert's, for the plain form's padded batch
        expert = np.repeat(np.arange(E), sizes)
        place = np.arange(len(expert)) - np.repeat(np.cumsum(sizes) - sizes, sizes)
        st["expert"], st["place"] = torch.from_numpy(expert).cuda(), torch.from_numpy(place).cuda()
        st["most"] = int(sizes.max())
        if op == "grouped":
            st["bias"] = _normal(g, (E, N), 0.1, TYPES[c["out"]]) if c["bias"] else None
        else:
            st["z"] = _normal(g, (M, N), 1.0, BF16) if c["act"] != "none" else None
            st["dy"] = _normal(g, (M, N), 1.0, BF16)
    else:
        lead = (c["E"],) if c["E"] else ()
        N, K = c["N"], c["K"]
        # codes as round-to-nearest of normal weights leaves them, two to a byte, the even column's in the low half
        q = (_normal(g, lead + (N, K // 2), 2.4, BF16) + 8).round_().clamp_(0, 15).to(torch.uint8)
        q |= (_normal(g, lead + (N, K // 2), 2.4, BF16) + 8).round_().clamp_(0, 15).to(torch.uint8) << 4
        scale = (0.4 / math.sqrt(K) * (1.0 + 0.3 * _normal(g, lead + (N, K // c["group"])).clamp_(-2, 2))).to(BF16)
        zero = None
        if c["zeros"]:
            zero = torch.randint(6, 11, lead + (N, K // c["group"]), generator=g, device="cuda", dtype=torch.uint8)
        st.update(codes=q, scales=scale, zeros=zero)
        st["x"] = _normal(g, (c["T"], K), 1.0, BF16)
        st["bias"] = _normal(g, lead + (N,), 0.1) if c["bias"] else None
        st["experts"] = None
        if c["E"]:
            st["experts"] = torch.rand((c["T"], c["E"]), generator=g, device="cuda").topk(c["k"], 1).indices.contiguous()
        if own:   # the weight as a program keeps it, laid out once
            import mixture_experts_layer_mok_gb300 as mok

            st["weight"] = mok.int4_pack(q, scale, zero)
    return st


# ---------------------------------------------------------------- one pass
def run(st):
    return (_run_own if own else _run_plain)(st, st["c"])


def _run_own(st, c):
    import mixture_experts_layer_mok_gb300 as mok

    op = c["op"]
    if op == "route":
        r = mok.route(st["logits"], c["k"], score=c["score"], normalize=c["normalize"], scale=c["scale"],
                      balance=c["balance"])
        out = dict(experts=r.experts, weights=r.weights, lse=r.lse)
        return dict(out, counts=r.counts, mean_score=r.mean_score) if c["balance"] else out
    if op == "route_backward":
        return mok.route_backward(st["d_weights"], st["logits"], st["experts"], score=c["score"],
                                  normalize=c["normalize"], scale=c["scale"], d_lse=st["d_lse"],
                                  d_mean_score=st["d_mean_score"])
    if op == "grouped":
        y, z = mok.grouped_linear(st["x"], st["weight"], st["counts"], bias=st["bias"], activation=c["act"],
                                  out_dtype=TYPES[c["out"]], save_z=c["save_z"])
        return dict(y=y, z=z) if c["save_z"] else dict(y=y)
    if op == "grouped_backward":
        return mok.grouped_linear_backward(st["dy"], st["x"], st["weight"], st["counts"], z=st["z"],
                                           activation=c["act"], bias=c["bias"])
    return mok.int4_linear(st["x"], st["weight"], bias=st["bias"], activation=c["act"], experts=st["experts"],
                           out_dtype=TYPES[c["out"]])


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


def _scores(logits, score):
    """(scores, log-sum-exp) of the rows."""
    top = logits.max(1, keepdim=True).values
    e = torch.exp(logits - top)
    total = e.sum(1, keepdim=True)
    s = e / total if score == "softmax" else 1.0 / (1.0 + torch.exp(-logits))
    return s, (top + torch.log(total)).squeeze(1)


def _run_plain(st, c):
    op = c["op"]
    if op == "route":
        logits = st["logits"].float()
        experts = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :c["k"]].contiguous()
        s, lse = _scores(logits, c["score"])
        w = torch.gather(s, 1, experts)
        if c["normalize"]:
            w = w / w.sum(1, keepdim=True)
        out = dict(experts=experts, weights=w * c["scale"], lse=lse)
        if c["balance"]:
            chosen = torch.zeros_like(s).scatter_(1, experts, 1.0)
            out.update(counts=chosen.sum(0).to(torch.int32), mean_score=s.mean(0))
        return out
    if op == "route_backward":
        logits = st["logits"].float()
        s, lse = _scores(logits, c["score"])
        g, p = st["d_weights"] * c["scale"], torch.gather(s, 1, st["experts"])
        if c["normalize"]:
            total = p.sum(1, keepdim=True)
            g = (g - (g * p / total).sum(1, keepdim=True)) / total
        ds = torch.zeros_like(s).scatter_(1, st["experts"], g)
        if st["d_mean_score"] is not None:
            ds = ds + st["d_mean_score"] / c["T"]
        d = s * (ds - (s * ds).sum(1, keepdim=True)) if c["score"] == "softmax" else ds * s * (1.0 - s)
        if st["d_lse"] is not None:
            d = d + torch.exp(logits - lse.unsqueeze(1)) * st["d_lse"].unsqueeze(1)
        return d.to(st["logits"].dtype)
    if op == "grouped":
        z = torch.bmm(_padded(st, c, st["x"]), st["weight"].float().transpose(1, 2))
        if st["bias"] is not None:
            z = z + st["bias"].float().unsqueeze(1)
        out = dict(y=_rows(st, c, _act(z, c["act"])).to(TYPES[c["out"]]))
        if c["save_z"]:
            out["z"] = _rows(st, c, z).to(BF16)
        return out
    if op == "grouped_backward":
        dz = st["dy"].float()
        if c["act"] != "none":
            dz = dz * _act_grad(st["z"].float(), c["act"])
        dz = _padded(st, c, dz)
        out = dict(dx=_rows(st, c, torch.bmm(dz, st["weight"].float())).to(BF16),
                   d_weight=torch.bmm(dz.transpose(1, 2), _padded(st, c, st["x"])).to(BF16))
        if c["bias"]:
            out["d_bias"] = dz.sum(1)
        return out
    w = _int4_values(st, c, st["experts"])
    if c["E"]:   # [T, k, N, K]
        z = torch.matmul(w, st["x"].float()[:, None, :, None]).squeeze(-1)
    else:
        z = st["x"].float() @ w.t()
    if st["bias"] is not None:
        z = z + (st["bias"][st["experts"]] if c["E"] else st["bias"])
    return _act(z, c["act"]).to(TYPES[c["out"]])


def _padded(st, c, rows):
    """[E, most, .] in 32 bits: each expert's rows and zeros."""
    out = torch.zeros((c["E"], st["most"], rows.shape[1]), device="cuda")
    out[st["expert"], st["place"]] = rows[:c["M"] - c["tail"]].float()
    return out


def _rows(st, c, padded):
    """The experts' rows one after the other, and zeros behind them."""
    out = torch.zeros((c["M"], padded.shape[2]), device="cuda")
    out[:c["M"] - c["tail"]] = padded[st["expert"], st["place"]]
    return out


def _int4_values(st, c, pick):
    """The fp32 matrix, or the matrices of the chosen experts."""
    codes, scales, zeros = st["codes"], st["scales"], st["zeros"]
    if pick is not None:
        codes, scales, zeros = codes[pick], scales[pick], None if zeros is None else zeros[pick]
    q = torch.stack((codes & 15, codes >> 4), -1).reshape(scales.shape + (c["group"],)).float()
    q = q - (8.0 if zeros is None else zeros.unsqueeze(-1).float())
    return (q * scales.unsqueeze(-1).float()).reshape(codes.shape[:-1] + (c["K"],))


# ---------------------------------------------------------------- 64 bits
def exact(c, seed):
    st = prepare(c, seed)
    op, d = c["op"], torch.float64
    if op == "route":
        l64 = st["logits"].to(d)
        s = torch.softmax(l64, 1) if c["score"] == "softmax" else torch.sigmoid(l64)
        experts = torch.sort(-l64, dim=1, stable=True).indices[:, :c["k"]].contiguous()
        w = s.gather(1, experts) * c["scale"]
        if c["normalize"]:
            w = w / s.gather(1, experts).sum(1)[:, None]
        out = dict(experts=experts, weights=w, lse=torch.logsumexp(l64, 1))
        if c["balance"]:
            out.update(counts=torch.bincount(experts.reshape(-1), minlength=c["E"]).to(torch.int32),
                       mean_score=s.sum(0) / c["T"])
        return out
    if op == "route_backward":
        l64 = st["logits"].to(d).requires_grad_(True)
        s = torch.softmax(l64, 1) if c["score"] == "softmax" else torch.sigmoid(l64)
        w = s.gather(1, st["experts"])
        w = (w / w.sum(1, keepdim=True) if c["normalize"] else w) * c["scale"]
        loss = (w * st["d_weights"].to(d)).sum()
        if c["losses"]:
            loss = loss + (torch.logsumexp(l64, 1) * st["d_lse"].to(d)).sum() + (s.mean(0) * st["d_mean_score"].to(d)).sum()
        return torch.autograd.grad(loss, l64)[0]
    if op in ("grouped", "grouped_backward"):
        return _exact_grouped(st, c)

    def values(e):
        q, s, zero = (t if t is None or e is None else t[e] for t in (st["codes"], st["scales"], st["zeros"]))
        w = torch.empty((c["N"], c["K"]), dtype=d, device="cuda")
        w[:, 0::2], w[:, 1::2] = q % 16, q // 16
        w -= 8.0 if zero is None else zero.to(d).repeat_interleave(c["group"], 1)
        return w * s.to(d).repeat_interleave(c["group"], 1)

    x, b = st["x"].to(d), st["bias"]
    if not c["E"]:
        z = torch.einsum("tk,nk->tn", x, values(None)) + (0.0 if b is None else b.to(d))
        return _exact_act(z, c["act"])
    rows = [[torch.einsum("k,nk->n", x[t], values(e)) + (0.0 if b is None else b[e].to(d)) for e in row]
            for t, row in enumerate(st["experts"].tolist())]
    return _exact_act(torch.stack([torch.stack(r) for r in rows]), c["act"])


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


def _exact_grouped(st, c):
    d, M, N, K = torch.float64, c["M"], c["N"], c["K"]
    ends = np.cumsum(st["counts"].cpu().numpy())
    kw = dict(dtype=d, device="cuda")
    if c["op"] == "grouped":
        y, z = torch.zeros((M, N), **kw), torch.zeros((M, N), **kw)
    else:
        dx, dw, db = torch.zeros((M, K), **kw), torch.zeros((c["E"], N, K), **kw), torch.zeros((c["E"], N), **kw)
    for e, end in enumerate(ends):
        r = slice(int(ends[e - 1]) if e else 0, int(end))
        w, x = st["weight"][e].to(d), st["x"][r].to(d)
        if c["op"] == "grouped":
            z[r] = torch.einsum("mk,nk->mn", x, w) + (0.0 if st["bias"] is None else st["bias"][e].to(d))
            y[r] = _exact_act(z[r], c["act"])
            continue
        g = st["dy"][r].to(d)
        if c["act"] != "none":
            at = st["z"][r].to(d).requires_grad_(True)
            g, = torch.autograd.grad(_exact_act(at, c["act"]), at, g)
        dx[r], dw[e], db[e] = torch.einsum("mn,nk->mk", g, w), torch.einsum("mn,mk->nk", g, x), g.sum(0)
    if c["op"] == "grouped":
        return dict(y=y, z=z) if c["save_z"] else dict(y=y)
    return dict(dx=dx, d_weight=dw, d_bias=db) if c["bias"] else dict(dx=dx, d_weight=dw)


# ---------------------------------------------------------------- work
def _bytes(t):
    return {"bf16": 2, "f32": 4}[t]


def work(c):
    op = c["op"]
    if op == "route":
        T, E, k = c["T"], c["E"], c["k"]
        return dict(bytes=T * (E * _bytes(c["logits"]) + 12 * k + 4) + 8 * E * c["balance"], flops=T * E * 10)
    if op == "route_backward":
        T, E, k = c["T"], c["E"], c["k"]
        return dict(bytes=T * (2 * E * _bytes(c["logits"]) + 12 * k + 4 * c["losses"]) + 4 * E * c["losses"],
                    flops=T * E * 14)
    if op in ("grouped", "grouped_backward"):
        M, N, K = c["M"], c["N"], c["K"]
        rows, used = M - c["tail"], min(c["E"], M - c["tail"])   # experts that have rows, at most
        if op == "grouped":
            return dict(bytes=2 * (rows * K + used * N * K) + M * N * (_bytes(c["out"]) + 2 * c["save_z"]),
                        flops=2 * rows * N * K)
        act = c["act"] != "none"
        return dict(bytes=2 * (rows * N * (1 + act) + rows * K + M * K + used * N * K + c["E"] * N * K)
                    + 4 * c["E"] * N * c["bias"], flops=4 * rows * N * K)
    N, K, rows = c["N"], c["K"], c["T"] * max(1, c["k"])
    used = min(c["E"], rows) if c["E"] else 1
    return dict(bytes=used * N * (K // 2 + K // c["group"] * (2 + c["zeros"])) + 2 * c["T"] * K
                + rows * N * _bytes(c["out"]), flops=2 * rows * N * K)
