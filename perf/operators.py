"""The operators that surround the estimator in a training step, as cases to be timed and compared:

  linear           y = act(x W^T + b) + residual, the clean layer of a block and the recomputation of later blocks
  linear_backward  dx, dW, db of that layer from dy and the stored pre-activation
  embedding        out_t = scale E[ids_t], a zero row for a negative (padding) id
  embedding_grad   G[v] (+)= scale sum over t with ids_t = v of g_t
  adam             one AdamW step over all tensors of a stack, with fp32 or 8-bit moments

`own` False computes them in their plain form (elementary torch operations in fp32); True makes the calls of the package.
8-bit moments: 256-element blocks of a tensor hold m / s_m and sqrt(v) / s_v in e4m3, with s = (largest magnitude in the
block) / 448 in fp32 and s = 0 for a block whose largest magnitude is below 2^-100; a positive sqrt(v) keeps at least the
smallest code.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 256           # elements that share one scale of an 8-bit moment
TOP = 448.0           # largest e4m3 value
LEAST = 2.0 ** -9     # smallest positive one
TINY = 2.0 ** -100    # a block whose largest magnitude is below this is held as zeros
LR, B1, B2, EPS, WD, STEP = 1e-3, 0.9, 0.999, 1e-8, 0.1, 100

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one token of a sequence that is being extended, through the wide layer of a block
        {"name": "linear-token", "op": "linear", "N": 1, "d_in": 2048, "d_out": 8192, "act": "gelu_tanh", "bias": True,
         "residual": False, "keep_z": False, "out": "bf16"},
        # a few sequences extended at once, with the block's residual, out of the wide layer
        {"name": "linear-tokens-24", "op": "linear", "N": 24, "d_in": 8192, "d_out": 2048, "act": "none", "bias": True,
         "residual": True, "keep_z": False, "out": "bf16"},
        # a ragged packed batch through a small model's joint query, key and value projection
        {"name": "linear-qkv-ragged", "op": "linear", "N": 8109, "d_in": 768, "d_out": 2304, "act": "none", "bias": True,
         "residual": False, "keep_z": False, "out": "bf16"},
        # a whole training batch into the wide layer, the pre-activation kept for the backward pass
        {"name": "linear-mlp-in", "op": "linear", "N": 16384, "d_in": 2048, "d_out": 8192, "act": "gelu", "bias": True,
         "residual": False, "keep_z": True, "out": "bf16"},
        # the backward pass of a small model's attention projection, odd token count
        {"name": "linear-backward-proj", "op": "linear_backward", "N": 5001, "d_in": 1024, "d_out": 1024, "act": "none"},
        # the backward pass of the wide layer over a whole training batch
        {"name": "linear-backward-mlp", "op": "linear_backward", "N": 16384, "d_in": 2048, "d_out": 8192, "act": "gelu"},
        # the rows of the tokens that eight sequences are extended by
        {"name": "embedding-tokens-8", "op": "embedding", "N": 8, "V": 4096, "d": 768, "scale": 1.0, "pad": 0,
         "table": "bf16", "out": "bf16"},
        # a whole training batch, fp32 master rows to bf16 activations, scaled by sqrt(d), padded at its end
        {"name": "embedding-batch", "op": "embedding", "N": 65536, "V": 65536, "d": 2048, "scale": 45.25, "pad": 1500,
         "table": "f32", "out": "bf16"},
        # a small batch onto the gradient that a tied output layer has left
        {"name": "embedding-grad-tied", "op": "embedding_grad", "N": 2000, "V": 4096, "d": 768, "scale": 1.0, "pad": 37,
         "grad": "f32", "accumulate": True},
        # a whole training batch over a large vocabulary; most rows get a few tokens, some get thousands
        {"name": "embedding-grad-batch", "op": "embedding_grad", "N": 65536, "V": 65536, "d": 2048, "scale": 45.25, "pad": 1500,
         "grad": "bf16", "accumulate": False},
        # the twelve-block stack with fp32 moments
        {"name": "adam-stack-32", "op": "adam", "blocks": 12, "d": 768, "bits": 32, "grad": "f32"},
        # four wide blocks with 8-bit moments
        {"name": "adam-wide-8", "op": "adam", "blocks": 4, "d": 2048, "bits": 8, "grad": "f32"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_backward", "embedding", "embedding_grad", "adam"])
    if op in ("linear", "linear_backward"):
        cap = 16384 * 2048 * 8192
        d_in, d_out = 16 * _log(rng, 4, 512), 16 * _log(rng, 4, 512)
        N = _log(rng, 1 if op == "linear" else 16, max(16, min(16384, cap // (d_in * d_out))))
        c = {"op": op, "N": N, "d_in": d_in, "d_out": d_out, "act": rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"])}
        if op == "linear":
            c.update(bias=rng.random() < 0.7, residual=rng.random() < 0.5, keep_z=rng.random() < 0.3,
                     out=rng.choice(["bf16", "bf16", "f32"]))
        return c
    if op in ("embedding", "embedding_grad"):
        N, V, d = _log(rng, 1, 65536), _log(rng, 64, 65536), _log(rng, 48, 2048)
        c = {"op": op, "N": N, "V": V, "d": d, "scale": rng.choice([1.0, math.sqrt(d)]), "pad": rng.randrange(0, N // 4 + 1)}
        if op == "embedding":
            c.update(table=rng.choice(["f32", "bf16"]), out=rng.choice(["f32", "bf16"]))
        else:
            c.update(grad=rng.choice(["f32", "bf16"]), accumulate=rng.random() < 0.5)
        return c
    d = 16 * _log(rng, 4, 128)
    return {"op": "adam", "blocks": rng.randint(1, max(1, min(12, (4 * 2048 * 2048) // (d * d)))), "d": d,
            "bits": rng.choice([32, 8]), "grad": rng.choice(["f32", "bf16"])}


# ------------------------------------------------------------------------------------------------ the inputs

def _pad(n, to):
    return -(-n // to) * to


def _spans(case):
    """(elements, columns) of each tensor of the stack, matrices first, and where each begins in the flat buffers: at
    multiples of 256 elements, the matrices before the vectors."""
    d = case["d"]
    mats = [(3 * d, d), (d, d), (4 * d, d), (d, 4 * d)] * case["blocks"]
    vecs = [(3 * d, 1), (d, 1), (4 * d, 1), (d, 1), (d, 1), (d, 1)] * case["blocks"]
    spans, at, split = [], 0, 0
    for k, (r, c) in enumerate(mats + vecs):
        if k == len(mats):
            split = at
        spans.append((at, r, c))
        at += _pad(r * c, BLOCK)
    return spans, split, at


def _to_e4m3(x, least=0.0):
    """(codes, scales) of a flat fp32 buffer of whole blocks; positive values are held as at least `least`."""
    b = x.view(-1, BLOCK)
    top = b.abs().amax(1)
    zero = top < TINY
    scale = torch.where(zero, torch.zeros_like(top), top * (1.0 / TOP))
    inv = torch.where(zero, torch.zeros_like(top), torch.full_like(top, TOP) / top)
    near = b * inv[:, None]
    near = torch.where(near > 0, near.clamp(min=least), near)
    return near.to(torch.float8_e4m3fn).view(-1), scale


def _from_e4m3(code, scale):
    return (code.to(torch.float32).view(-1, BLOCK) * scale[:, None]).view(-1)


def _ids(case, g):
    """Token ids whose frequencies fall off like one over the rank, the batch padded at its end with -1."""
    u = torch.rand(case["N"], device="cuda", generator=g, dtype=torch.float64)
    ids = (torch.exp(u * math.log(case["V"] + 1)) - 1).long().clamp_(0, case["V"] - 1).to(torch.int32)
    if case["pad"]:
        ids[case["N"] - case["pad"]:] = -1
    return ids


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))

    def normal(*shape, std=1.0, dtype=torch.float32):
        return (torch.randn(shape, device="cuda", generator=g) * std).to(dtype)

    op, s = case["op"], {"case": case}
    if op == "linear":
        N, i, o = case["N"], case["d_in"], case["d_out"]
        s.update(x=normal(N, i, dtype=torch.bfloat16), W=normal(o, i, std=i ** -0.5, dtype=torch.bfloat16),
                 b=normal(o, std=0.02) if case["bias"] else None,
                 res=normal(N, o, dtype=DT[case["out"]]) if case["residual"] else None)
    elif op == "linear_backward":
        N, i, o = case["N"], case["d_in"], case["d_out"]
        s.update(x=normal(N, i, dtype=torch.bfloat16), W=normal(o, i, std=i ** -0.5, dtype=torch.bfloat16),
                 dy=normal(N, o, std=1e-3, dtype=torch.bfloat16),
                 z=normal(N, o, dtype=torch.bfloat16) if case["act"] != "none" else None)
    elif op == "embedding":
        s.update(ids=_ids(case, g), E=normal(case["V"], case["d"], std=0.02, dtype=DT[case["table"]]))
        if case["d"] % 8:  # rows begin at 16-byte boundaries
            E = torch.zeros(case["V"], _pad(case["d"], 8), dtype=s["E"].dtype, device="cuda")
            E[:, :case["d"]] = s["E"]
            s["E"] = E[:, :case["d"]]
    elif op == "embedding_grad":
        s.update(ids=_ids(case, g), g=normal(case["N"], _pad(case["d"], 8), std=1e-3, dtype=DT[case["grad"]])[:, :case["d"]],
                 G=normal(case["V"], _pad(case["d"], 8), std=1e-3)[:, :case["d"]] if case["accumulate"] else None)
    else:
        spans, split, total = _spans(case)
        flat = {n: torch.zeros(total, device="cuda") for n in ("W", "G", "m", "r")}
        for at, rows, cols in spans:
            n = rows * cols
            # each output channel has a gradient size of its own
            size = torch.exp(torch.randn(rows, 1, device="cuda", generator=g)) * 1e-3
            flat["W"][at:at + n] = normal(n, std=0.02)
            flat["G"][at:at + n] = (torch.randn(rows, cols, device="cuda", generator=g) * size).view(-1)
            flat["m"][at:at + n] = (torch.randn(rows, cols, device="cuda", generator=g) * (0.25 * size)).view(-1)
            flat["r"][at:at + n] = (torch.rand(rows, cols, device="cuda", generator=g) * (0.2 * size) + 0.2 * size).view(-1)
        s.update(W=flat["W"], Wb=flat["W"].to(torch.bfloat16), G=flat["G"].to(DT[case["grad"]]), split=split,
                 g_scale=torch.tensor([0.5], device="cuda"))
        if case["bits"] == 8:
            s["m"], s["ms"] = _to_e4m3(flat["m"])
            s["v"], s["vs"] = _to_e4m3(flat["r"], LEAST)
        else:
            s["m"], s["v"] = flat["m"], flat["r"].square_()
        if own:
            import zeroth_order_transformer_b200 as z

            def views(t):
                return [t[at:at + r * c] for at, r, c in spans]

            def block_views(t):
                return [t[at // BLOCK:(at + _pad(r * c, BLOCK)) // BLOCK] for at, r, c in spans]

            more = dict(m_scale=block_views(s["ms"]), v_scale=block_views(s["vs"])) if case["bits"] == 8 else {}
            s["opt"] = z.DustOptimizer(views(s["W"]), views(s["G"]), W_bf16=views(s["Wb"]), bits=case["bits"],
                                       decay=[at < split for at, _, _ in spans], m=views(s["m"]), v=views(s["v"]), **more)
    return s


# ------------------------------------------------------------------------------------------------ plain forms

def _act(z, act):
    if act == "relu":
        return z * (z > 0)
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _act_slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))
    if act == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    p = 1 / (1 + torch.exp(-z))
    return p * (1 + z * (1 - p))


def _linear(s):
    c = s["case"]
    z = s["x"].float() @ s["W"].float().t()
    if s["b"] is not None:
        z = z + s["b"]
    y = _act(z, c["act"])
    if s["res"] is not None:
        y = y + s["res"].float()
    y = y.to(DT[c["out"]])
    return {"y": y, "z": z.to(torch.bfloat16)} if c["keep_z"] else {"y": y}


def _linear_backward(s):
    dz = s["dy"].float()
    if s["z"] is not None:
        dz = dz * _act_slope(s["z"].float(), s["case"]["act"])
    return {"dx": (dz @ s["W"].float()).to(torch.bfloat16), "dW": dz.t() @ s["x"].float(), "db": dz.sum(0)}


def _embedding(s):
    ids = s["ids"].long()
    row = s["E"][ids.clamp(min=0)].float() * s["case"]["scale"]
    return {"out": (row * (ids >= 0)[:, None]).to(DT[s["case"]["out"]])}


def _embedding_grad(s):
    c, ids = s["case"], s["ids"].long()
    g = s["g"].float() * (ids >= 0)[:, None] * c["scale"]
    G = s["G"] if c["accumulate"] else torch.zeros(c["V"], c["d"], device=g.device)
    return {"G": G.index_add_(0, ids.clamp(min=0), g)}


def _adam(s):
    g = s["G"].float() * s["g_scale"]
    eight = s["case"]["bits"] == 8
    m0 = _from_e4m3(s["m"], s["ms"]) if eight else s["m"]
    v0 = _from_e4m3(s["v"], s["vs"]).square() if eight else s["v"]
    m = m0 * B1 + g * (1 - B1)
    v = v0 * B2 + g.square() * (1 - B2)
    r = v.sqrt()
    w = s["W"]
    w[:s["split"]] *= 1 - LR * WD
    w -= (m / (1 - B1 ** STEP)) / (r / math.sqrt(1 - B2 ** STEP) + EPS) * LR
    s["Wb"].copy_(w)
    if eight:
        for name, x, least in (("m", m, 0.0), ("v", r, LEAST)):
            code, scale = _to_e4m3(x, least)
            s[name].copy_(code)
            s[name + "s"].copy_(scale)
    else:
        s["m"].copy_(m)
        s["v"].copy_(v)
    return _adam_out(s)


def _adam_out(s):
    out = {k: s[k] for k in ("W", "Wb", "m", "v")}
    return {**out, "ms": s["ms"], "vs": s["vs"]} if s["case"]["bits"] == 8 else out


def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if not own:
        return {"linear": _linear, "linear_backward": _linear_backward, "embedding": _embedding,
                "embedding_grad": _embedding_grad, "adam": _adam}[op](s)
    import zeroth_order_transformer_b200 as z
    if op == "linear":
        got = z.dust_linear(s["x"], s["W"], bias=s["b"], act=c["act"], residual=s["res"], z=c["keep_z"], out_dtype=DT[c["out"]])
        return {"y": got[0], "z": got[1]} if c["keep_z"] else {"y": got}
    if op == "linear_backward":
        dx, dW, db = z.dust_linear_backward(s["dy"], s["x"], s["W"], act=c["act"], z=s["z"])
        return {"dx": dx, "dW": dW, "db": db}
    if op == "embedding":
        return {"out": z.dust_embedding(s["ids"], s["E"], scale=c["scale"], out_dtype=DT[c["out"]])}
    if op == "embedding_grad":
        return {"G": z.dust_embedding_grad(s["ids"], s["g"], c["V"], scale=c["scale"], G=s["G"], accumulate=c["accumulate"])}
    s["opt"].step(z.adam(LR, STEP, B1, B2, EPS, WD), g_scale=s["g_scale"])
    return _adam_out(s)


# ------------------------------------------------------------------------------------------------ what a pass cannot do without

def _rows_touched(case):
    """The expected number of different rows among the batch's ids."""
    p = np.diff(np.log(np.arange(1, case["V"] + 2, dtype=np.float64))) / math.log(case["V"] + 1)
    return float(np.sum(-np.expm1((case["N"] - case["pad"]) * np.log1p(-p))))


def work(case):
    op, size = case["op"], {"bf16": 2, "f32": 4}
    if op == "linear":
        N, i, o = case["N"], case["d_in"], case["d_out"]
        out = N * o * size[case["out"]]
        return {"bytes": 2 * (N * i + o * i) + 4 * o * case["bias"] + out * (1 + case["residual"]) + 2 * N * o * case["keep_z"],
                "flops": 2 * N * i * o}
    if op == "linear_backward":
        N, i, o = case["N"], case["d_in"], case["d_out"]
        return {"bytes": 2 * N * o * (1 + (case["act"] != "none")) + 4 * N * i + 2 * o * i + 4 * o * i + 4 * o,
                "flops": 4 * N * i * o}
    if op == "embedding":
        return {"bytes": 4 * case["N"] + _rows_touched(case) * case["d"] * size[case["table"]] + case["N"] * case["d"] * size[case["out"]],
                "flops": case["N"] * case["d"]}
    if op == "embedding_grad":
        live = case["N"] - case["pad"]
        rows = 2 * _rows_touched(case) if case["accumulate"] else case["V"]
        return {"bytes": 4 * case["N"] + live * case["d"] * size[case["grad"]] + 4 * rows * case["d"], "flops": 2 * live * case["d"]}
    spans, _, _ = _spans(case)
    n = sum(r * c for _, r, c in spans)
    moments = 16 if case["bits"] == 32 else 4 + 16 / BLOCK
    return {"bytes": n * (size[case["grad"]] + 8 + 2 + moments), "flops": 20 * n}


# ------------------------------------------------------------------------------------------------ the definition in 64 bits

def _exact_act(z, act):
    """(act(z), act'(z)) in 64 bits."""
    one = torch.ones_like(z)
    if act == "relu":
        return torch.where(z > 0, z, 0 * one), torch.where(z > 0, one, 0 * one)
    if act == "gelu":
        cdf = 0.5 * torch.erfc(-z / math.sqrt(2.0))
        return z * cdf, cdf + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if act == "silu" or act == "gelu_tanh":
        # both are z p(u) with the logistic p: u = z, and u = 2 sqrt(2 / pi) (z + 0.044715 z^3)
        k = math.sqrt(8 / math.pi)
        u, du = (z, one) if act == "silu" else (k * (z + 0.044715 * z ** 3), k * (1 + 0.134145 * z ** 2))
        p = torch.sigmoid(u)
        return z * p, p + z * p * (1 - p) * du
    return z, one


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "linear":
        z = torch.einsum("ni,oi->no", s["x"].double(), s["W"].double())
        if s["b"] is not None:
            z += s["b"].double()
        y, _ = _exact_act(z, case["act"])
        if s["res"] is not None:
            y = y + s["res"].double()
        return {"y": y, "z": z} if case["keep_z"] else {"y": y}
    if op == "linear_backward":
        dz = s["dy"].double()
        if s["z"] is not None:
            dz = dz * _exact_act(s["z"].double(), case["act"])[1]
        return {"dx": torch.einsum("no,oi->ni", dz, s["W"].double()), "dW": torch.einsum("no,ni->oi", dz, s["x"].double()),
                "db": torch.einsum("no->o", dz)}
    if op == "embedding":
        out = torch.zeros(case["N"], case["d"], dtype=torch.float64, device="cuda")
        live = torch.nonzero(s["ids"] >= 0)[:, 0]
        out[live] = torch.index_select(s["E"], 0, s["ids"][live]).double() * case["scale"]
        return {"out": out}
    if op == "embedding_grad":
        live = torch.nonzero(s["ids"] >= 0)[:, 0]
        G = torch.zeros(case["V"], case["d"], dtype=torch.float64, device="cuda") if s["G"] is None else s["G"].double()
        G.scatter_add_(0, s["ids"][live].long()[:, None].expand(-1, case["d"]), s["g"][live].double() * case["scale"])
        return {"G": G}
    g = s["G"].double() * 0.5
    if case["bits"] == 8:
        m0 = s["m"].double() * s["ms"].double().repeat_interleave(BLOCK)
        v0 = (s["v"].double() * s["vs"].double().repeat_interleave(BLOCK)) ** 2
    else:
        m0, v0 = s["m"].double(), s["v"].double()
    m, v = torch.lerp(g, m0, B1), torch.lerp(g ** 2, v0, B2)
    decay = torch.ones_like(m)
    decay[:s["split"]] -= LR * WD
    w = s["W"].double() * decay - LR * (m / (1 - B1 ** STEP)) / ((v / (1 - B2 ** STEP)).sqrt() + EPS)
    if case["bits"] == 32:
        return {"W": w, "Wb": w, "m": m, "v": v}
    held = {"W": w, "Wb": w}
    for name, x, least in (("m", m, 0.0), ("v", v.sqrt(), LEAST)):
        top = x.view(-1, BLOCK).abs().max(1).values
        scale = torch.where(top < TINY, 0.0, top / TOP)
        near = x.view(-1, BLOCK) / torch.where(scale > 0, scale, 1.0)[:, None]
        # e4m3: three bits after the leading one down to 2^-6, steps of 2^-9 below
        step = torch.exp2(torch.floor(torch.log2(near.abs().clamp(min=2.0 ** -6))) - 3)
        held[name] = (torch.round(torch.where(near > 0, near.clamp(min=least), near) / step) * step).view(-1)
        held[name + "s"] = scale
    return held
