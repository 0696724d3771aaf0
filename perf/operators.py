"""The cases that measure the library's routing from logits (moe_topk), its 4-bit matrix-vector
products (moe_matvec) and its experts with 4-bit group-scaled weights (moe_experts).

``run`` computes a case in plain torch operations, or, where ``own`` is true, through the library.
Sizes are those of the library's workloads (hidden 2048 and 7168, 256 experts, top-8, expert
widths 512 and 2048) and generic ones around them."""

import math

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # One decoded token: 256 experts in 8 groups, the best 4 groups stay (sums of two scores).
        dict(name="topk_n1_sigmoid_groups", op="topk", n=1, E=256, k=8, routing="sigmoid", bias=True, groups=8,
             kept=4, score="top2", norm=True, factor=2.5, logits="f32", pad=0),
        # A decode batch, softmax over 256 experts, BF16 logits of a router product.
        dict(name="topk_n64_softmax_bf16", op="topk", n=64, E=256, k=8, routing="softmax", bias=False, groups=1,
             kept=1, score="max", norm=True, factor=1.0, logits="bf16", pad=0),
        # An odd prefill chunk: 160 experts in 8 groups of 20, the group's best probability, no renormalising,
        # logits that are columns of a wider matrix.
        dict(name="topk_n5001_softmax_groups", op="topk", n=5001, E=160, k=6, routing="softmax", bias=False, groups=8,
             kept=3, score="max", norm=False, factor=16.0, logits="f32", pad=3),
        # The largest: a long prefill chunk, sigmoid scores with a balance bias and groups.
        dict(name="topk_n32768_sigmoid_groups", op="topk", n=32768, E=256, k=8, routing="sigmoid", bias=True, groups=8,
             kept=4, score="top2", norm=True, factor=2.5, logits="f32", pad=0),
        # A small projection of one token: launch latency.
        dict(name="matvec_n1_2048x2048", op="matvec", n=1, out=2048, inp=2048, fmt="int4_g128", zero=False, bias=False,
             x="bf16", y="bf16", pad=0),
        # A projection of hidden 7168 for one token, zero points and groups of 64.
        dict(name="matvec_n1_7168x7168_zero", op="matvec", n=1, out=7168, inp=7168, fmt="int4_g64", zero=True,
             bias=True, x="bf16", y="bf16", pad=0),
        # The output layer over an odd vocabulary for six tokens of a batch, fp32 logits.
        dict(name="matvec_n6_100003x2048_f32", op="matvec", n=6, out=100003, inp=2048, fmt="int4_g32", zero=False,
             bias=False, x="f16", y="f32", pad=64),
        # Sixteen tokens of a decode batch through an NVFP4 projection.
        dict(name="matvec_n16_7168x2048_nvfp4", op="matvec", n=16, out=7168, inp=2048, fmt="nvfp4", zero=False,
             bias=False, x="bf16", y="bf16", pad=0),
        # Experts of one decoded token.
        dict(name="experts_n1_int4_g128", op="experts", n=1, H=2048, E=256, k=8, I=512, S=512, fmt="int4_g128",
             zero=False, dup=0.0),
        # A decode batch of 16 tokens.
        dict(name="experts_n16_int4_g64_zero", op="experts", n=16, H=2048, E=256, k=8, I=512, S=512, fmt="int4_g64",
             zero=True, dup=0.0),
        # 64 tokens of the wide layer, one rank's 64 experts.
        dict(name="experts_n64_h7168", op="experts", n=64, H=7168, E=64, k=8, I=2048, S=2048, fmt="int4_g128",
             zero=False, dup=0.0),
        # 256 rows of a speculative verify step, a quarter of them duplicated.
        dict(name="experts_n256_int4_g32", op="experts", n=256, H=2048, E=256, k=8, I=512, S=512, fmt="int4_g32",
             zero=False, dup=0.25),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["topk", "matvec", "experts"])
    if op == "topk":
        groups, kept = rng.choice([(1, 1), (1, 1), (4, 2), (8, 3), (8, 4), (16, 5)])
        size = rng.randint(max(2, 10 // kept), 256 // groups) if groups > 1 else rng.randint(12, 256)
        E = groups * size
        routing = rng.choice(["softmax", "sigmoid"])
        bias = rng.random() < 0.6
        k = rng.randint(1, min(10, kept * size))
        return dict(op=op, n=_log(rng, 1, 30000), E=E, k=k, routing=routing, bias=bias, groups=groups, kept=kept,
                    score=rng.choice(["top2", "max"]), norm=rng.random() < 0.7,
                    factor=rng.choice([1.0, 2.5, 16.0]), logits=rng.choice(["f32", "bf16", "f16"]),
                    pad=rng.choice([0, 0, 1, 8]))
    fmt = rng.choice(["int4_g32", "int4_g64", "int4_g128"])
    G = int(fmt[6:])
    zero = rng.random() < 0.5
    if op == "matvec":
        if rng.random() < 0.25:
            fmt, G, zero = "nvfp4", 32, False
        return dict(op=op, n=_log(rng, 1, 16), out=_log(rng, 200, 20000), inp=G * max(1, _log(rng, 256, 7168) // G),
                    fmt=fmt, zero=zero, bias=rng.random() < 0.3, x=rng.choice(["bf16", "f16"]),
                    y=rng.choice(["bf16", "f16", "f32"]), pad=rng.choice([0, 0, 8]))
    I = 128 * rng.randint(1, 6)
    return dict(op=op, n=_log(rng, 1, 256), H=128 * rng.randint(4, 20), E=rng.choice([16, 60, 128, 200]),
                k=rng.randint(1, 8), I=I, S=rng.choice([0, I, 128 * rng.randint(1, 6)]), fmt=fmt, zero=zero,
                dup=rng.choice([0.0, 0.25]))


# ---------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 7919 + 11)
    return g


def _weights(g, lead, out, inp, fmt, zero):
    """A 4-bit matrix [*lead, out, inp] of about N(0, 0.02): codes (two per byte, the even element low), scales of
    its groups along inp, and zero points (INT4) or the matrix scale (NVFP4)."""
    if fmt == "nvfp4":
        z = torch.randn(*lead, out, inp, generator=g, device=DEV, dtype=torch.float32) * 2.0
        mag = torch.bucketize(z.abs(), torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEV)).to(torch.uint8)
        q = mag + 8 * ((z < 0) & (mag > 0)).to(torch.uint8)
        s = (32.0 * (0.5 + torch.rand(*lead, out, inp // 16, generator=g, device=DEV))).to(torch.float8_e4m3fn)
        s2 = torch.full((max(1, math.prod(lead)),), 0.01 / 32.0, device=DEV)
        return dict(fmt=fmt, w=q[..., 0::2] | (q[..., 1::2] << 4), scale=s.view(torch.uint8), scale2=s2, zero=None)
    G = int(fmt[6:])
    zp = None
    z = torch.randn(*lead, out, inp, generator=g, device=DEV, dtype=torch.float16) * 2.7
    if zero:
        zp = (8 + torch.randint(-2, 3, (*lead, out, inp // G), generator=g, device=DEV)).to(torch.uint8)
        z = (z.view(*lead, out, inp // G, G) + zp.to(torch.float16)[..., None]).view(*lead, out, inp)
    else:
        z += 8.0
    q = z.round_().clamp_(0, 15).to(torch.uint8)
    s = (0.0074 * (0.5 + torch.rand(*lead, out, inp // G, generator=g, device=DEV))).to(torch.bfloat16)
    return dict(fmt=fmt, w=q[..., 0::2] | (q[..., 1::2] << 4), scale=s, scale2=None, zero=zp)


def _rows(g, n, width, dtype, pad=0):
    """Rows of normalised activations, columns of a matrix `pad` wider."""
    return torch.randn(n, width + pad, generator=g, device=DEV).to(dtype)[:, :width]


def prepare(case, seed):
    c, g = dict(case), _gen(seed)
    s = {"case": c}
    if c["op"] == "topk":
        # A trained router's logits: unit spread over the experts, with an offset for each expert.
        lg = torch.randn(c["n"], c["E"] + c["pad"], generator=g, device=DEV)
        lg += 0.5 * torch.randn(c["E"] + c["pad"], generator=g, device=DEV)
        s["logits"] = lg.to(TYPES[c["logits"]])[:, :c["E"]]
        s["bias"] = (torch.rand(c["E"], generator=g, device=DEV) - 0.5) * 0.2 if c["bias"] else None
        if own:
            from mixture_experts_decode_router_gb300.layer import MoeTopk
            s["op"] = MoeTopk(c["E"], c["k"], routing=c["routing"], bias=s["bias"], num_groups=c["groups"],
                              topk_groups=c["kept"], group_score=c["score"], norm_topk_prob=c["norm"],
                              routed_scaling_factor=c["factor"])
    elif c["op"] == "matvec":
        s["w"] = _weights(g, (), c["out"], c["inp"], c["fmt"], c["zero"])
        s["x"] = _rows(g, c["n"], c["inp"], TYPES[c["x"]], c["pad"])
        s["bias"] = 0.1 * torch.randn(c["out"], generator=g, device=DEV) if c["bias"] else None
        if own:
            from mixture_experts_decode_router_gb300.layer import MoeMatvec
            from mixture_experts_decode_router_gb300.synth import QMatT
            s["op"] = MoeMatvec(QMatT(**s["w"]), bias=s["bias"], out_dtype=TYPES[c["y"]])
    else:
        E, k, H, I, S, n = c["E"], c["k"], c["H"], c["I"], c["S"], c["n"]
        dims = {"gate": (E, I, H), "up": (E, I, H), "down": (E, H, I)}
        if S:
            dims |= {"sh_gate": (1, S, H), "sh_up": (1, S, H), "sh_down": (1, H, S)}
        s["w"] = {m: _weights(g, d[:1], d[1], d[2], c["fmt"], c["zero"]) for m, d in dims.items()}
        x = _rows(g, n, H, torch.bfloat16)
        score = torch.rand(n, E, generator=g, device=DEV)
        distinct = max(1, n - int(round(n * c["dup"])))
        of = torch.arange(n, device=DEV) % distinct
        s["x"] = x[of].contiguous()
        s["idx"] = score[of].topk(k, dim=1).indices.to(torch.int32).contiguous()
        w = torch.rand(n, k, generator=g, device=DEV)[of] + 0.25
        s["rw"] = (2.5 * w / w.sum(1, keepdim=True)).contiguous()
        if own:
            from mixture_experts_decode_router_gb300 import synth
            from mixture_experts_decode_router_gb300.layer import MoeLayer
            cfg = synth.LayerConfig("experts", H, E, k, I, S, synth.ROUTE_SOFTMAX, True, 1.0, c["fmt"], n)
            q = {m: synth.QMatT(**s["w"][m]) if m in s["w"] else None
                 for m in ("gate", "up", "down", "sh_gate", "sh_up", "sh_down")}
            router = torch.zeros(E, H, dtype=torch.bfloat16, device=DEV)
            s["op"] = MoeLayer(synth.LayerWeights(cfg, router, **q, correction_bias=None, shared_gate_w=None), n)
    return s


# ---------------------------------------------------------------- the plain forms

def _matrix(w, pick=None, dtype=torch.float32):
    """The matrix that 4-bit codes and scales stand for (the experts `pick` of a stack)."""
    at = (lambda t: t) if pick is None else (lambda t: t[pick])
    b = at(w["w"])
    q = torch.stack([b & 15, b >> 4], dim=-1).flatten(-2)
    if w["fmt"] == "nvfp4":
        mag = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=b.device, dtype=dtype)
        v = torch.cat([mag, -mag])[q.long()]
        s = at(w["scale"]).view(torch.float8_e4m3fn).to(dtype) * w["scale2"].to(dtype)[0]
    else:
        v = q.to(dtype)
        s = at(w["scale"]).to(dtype)
    v = v.unflatten(-1, (s.shape[-1], -1))
    if w["fmt"] != "nvfp4":
        v -= 8.0 if w["zero"] is None else at(w["zero"]).to(dtype)[..., None]
    return v.mul_(s[..., None]).flatten(-2)


def _topk_plain(s):
    c = s["case"]
    # Scores in 64 bits: the order of near values decides whole numbers.
    lg = s["logits"].double()
    m = lg.amax(1, keepdim=True)
    p = 1 / (1 + torch.exp(-lg)) if c["routing"] == "sigmoid" else torch.exp(lg - m) / torch.exp(lg - m).sum(1, keepdim=True)
    sel = p + s["bias"].double() if s["bias"] is not None else lg
    if c["groups"] > 1:
        val = sel if s["bias"] is not None else p
        by = val.view(len(lg), c["groups"], -1).sort(dim=2, descending=True).values
        score = by[..., :2].sum(2) if c["score"] == "top2" else by[..., 0]
        order = score.sort(dim=1, descending=True, stable=True).indices[:, :c["kept"]]
        keep = torch.zeros_like(score, dtype=torch.bool).scatter_(1, order, True)
        sel = torch.where(keep[..., None], sel.view(len(lg), c["groups"], -1), -math.inf).flatten(1)
    idx = sel.sort(dim=1, descending=True, stable=True).indices[:, :c["k"]]
    w = p.gather(1, idx)
    if c["norm"]:
        w = w / w.sum(1, keepdim=True)
    return idx.to(torch.int32), (w * c["factor"]).float()


def _swiglu(x, gate, up):
    g, u = x @ gate.mT, x @ up.mT
    return g / (1 + torch.exp(-g)) * u


def _experts_plain(s, dtype=torch.float32):
    c, w = s["case"], s["w"]
    x, rw = s["x"].to(dtype), s["rw"].to(dtype)
    n, k, E = c["n"], c["k"], c["E"]
    if n * k <= E:  # the chosen experts' matrices, one for each route
        pick = s["idx"].flatten().long()
        a = _swiglu(x.repeat_interleave(k, 0)[:, None, :], _matrix(w["gate"], pick, dtype), _matrix(w["up"], pick, dtype))
        d = a @ _matrix(w["down"], pick, dtype).mT
        out = (d.view(n, k, -1) * rw[..., None]).sum(1)
    else:  # every expert over every token, weighted by the dense routing matrix
        dense = torch.zeros(n, E, device=x.device, dtype=dtype).scatter_add_(1, s["idx"].long(), rw)
        a = _swiglu(x, _matrix(w["gate"], None, dtype), _matrix(w["up"], None, dtype))
        a *= dense.T[..., None]
        out = torch.bmm(a, _matrix(w["down"], None, dtype).mT).sum(0)
    if c["S"]:
        out = out + (_swiglu(x, _matrix(w["sh_gate"], None, dtype), _matrix(w["sh_up"], None, dtype))
                     @ _matrix(w["sh_down"], None, dtype).mT)[0]
    return out


def run(state):
    s, op = state, state["case"]["op"]
    if own:
        if op == "topk":
            return s["op"].forward(s["logits"])
        if op == "matvec":
            return s["op"].forward(s["x"])
        return s["op"].experts(s["x"], s["idx"], s["rw"])
    if op == "topk":
        return _topk_plain(s)
    if op == "matvec":
        y = s["x"].float() @ _matrix(s["w"]).mT
        return (y if s["bias"] is None else y + s["bias"]).to(TYPES[s["case"]["y"]])
    return _experts_plain(s).to(torch.bfloat16)


# ---------------------------------------------------------------- the definitions in 64 bits

def _decode64(w, e=None):
    """One matrix's values in 64 bits, from a table of each group's 16 values."""
    take = (lambda t: t) if e is None else (lambda t: t[e])
    b = take(w["w"]).long()
    q = torch.empty(*b.shape[:-1], 2 * b.shape[-1], dtype=torch.long, device=b.device)
    q[..., 0::2], q[..., 1::2] = b % 16, b // 16
    if w["fmt"] == "nvfp4":
        level = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], device=b.device).double()
        scale = take(w["scale"]).view(torch.float8_e4m3fn).double() * float(w["scale2"][0])
        table = scale[..., None] * level
    else:
        scale = take(w["scale"]).double()
        mid = torch.full_like(scale, 8.0) if w["zero"] is None else take(w["zero"]).double()
        table = (torch.arange(16, device=b.device).double() - mid[..., None]) * scale[..., None]
    groups = table.shape[-2]
    return torch.gather(table, -1, q.view(*q.shape[:-1], groups, -1)).reshape(q.shape)


def exact(case, seed):
    global own
    was, own = own, False
    s = prepare(case, seed)
    own = was
    c = s["case"]
    if c["op"] == "topk":
        lg = s["logits"].double().cpu().numpy()
        with np.errstate(over="ignore"):
            if c["routing"] == "sigmoid":
                p = 1.0 / (1.0 + np.exp(-lg))
            else:
                p = np.exp(lg - lg.max(1, keepdims=True))
                p = p / p.sum(1, keepdims=True)
        bias = s["bias"].double().cpu().numpy() if s["bias"] is not None else None
        rank = lg if bias is None else p + bias
        if c["groups"] > 1:
            per = (p if bias is None else p + bias).reshape(len(lg), c["groups"], -1)
            best = np.partition(per, per.shape[2] - 2, axis=2)
            total = best[..., -1] + best[..., -2] if c["score"] == "top2" else best[..., -1]
            out = np.argsort(-total, axis=1, kind="stable")[:, c["kept"]:]
            rank = rank.reshape(len(lg), c["groups"], -1).copy()
            np.put_along_axis(rank, out[..., None], -np.inf, axis=1)
            rank = rank.reshape(len(lg), -1)
        idx = np.argsort(-rank, axis=1, kind="stable")[:, :c["k"]]
        w = np.take_along_axis(p, idx, 1)
        return idx.astype(np.int32), c["factor"] * (w / w.sum(1, keepdims=True) if c["norm"] else w)
    if c["op"] == "matvec":
        y = torch.empty(c["n"], c["out"], dtype=torch.float64, device=DEV)
        x = s["x"].double()
        for r in range(0, c["out"], 8192):
            part = {m: v[r:r + 8192] if torch.is_tensor(v) and m != "scale2" else v for m, v in s["w"].items()}
            y[:, r:r + 8192] = torch.einsum("nk,ok->no", x, _decode64(part))
        return y if s["bias"] is None else y + s["bias"].double()
    x, y = s["x"].double(), torch.zeros(c["n"], c["H"], dtype=torch.float64, device=DEV)
    names = [("gate", "up", "down", e) for e in sorted(set(s["idx"].flatten().tolist()))]
    if c["S"]:
        names.append(("sh_gate", "sh_up", "sh_down", 0))
    for gate, up, down, e in names:
        if gate == "gate":
            t, j = torch.nonzero(s["idx"] == e, as_tuple=True)
            weight = s["rw"][t, j].double()
        else:
            t, weight = torch.arange(c["n"], device=DEV), torch.ones(c["n"], dtype=torch.float64, device=DEV)
        g = torch.einsum("th,ih->ti", x[t], _decode64(s["w"][gate], e))
        u = torch.einsum("th,ih->ti", x[t], _decode64(s["w"][up], e))
        d = torch.einsum("ti,hi->th", torch.sigmoid(g) * g * u, _decode64(s["w"][down], e))
        y.index_add_(0, t, weight[:, None] * d)
    return y


# ---------------------------------------------------------------- what a case cannot do without

def _matrix_bytes(out, inp, fmt, zero):
    if fmt == "nvfp4":
        return out * inp // 2 + out * inp // 16 + 4
    return out * inp // 2 + (3 if zero else 2) * out * inp // int(fmt[6:])


def work(case):
    c = case
    n = c["n"]
    if c["op"] == "topk":
        each = 4 if c["logits"] == "f32" else 2
        return {"bytes": n * c["E"] * each + n * c["k"] * 8 + (4 * c["E"] if c["bias"] else 0),
                "flops": n * c["E"] * 4}
    if c["op"] == "matvec":
        y = 4 if c["y"] == "f32" else 2
        return {"bytes": _matrix_bytes(c["out"], c["inp"], c["fmt"], c["zero"]) + n * c["inp"] * 2 + n * c["out"] * y
                + (4 * c["out"] if c["bias"] else 0), "flops": 2 * n * c["out"] * c["inp"]}
    H, I, S, E, k = c["H"], c["I"], c["S"], c["E"], c["k"]
    distinct = max(1, n - int(round(n * c["dup"])))
    touched = E * (1 - (1 - k / E) ** distinct)  # experts that at least one token chose, on average
    each = 2 * _matrix_bytes(I, H, c["fmt"], c["zero"]) + _matrix_bytes(H, I, c["fmt"], c["zero"])
    shared = 2 * _matrix_bytes(S, H, c["fmt"], c["zero"]) + _matrix_bytes(H, S, c["fmt"], c["zero"]) if S else 0
    return {"bytes": int(touched * each + shared + n * H * 4 + n * k * 8), "flops": 6 * n * H * (k * I + S)}
