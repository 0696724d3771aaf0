"""The cases that measure the library's residual addition with RMSNorm (moe_norm), whose output is of 16 or 32 bits,
of 8 bits with scales, or both, and its low-rank adapters of many requests beside a shared projection (moe_lora).

``run`` computes a case in plain torch operations, or, where ``own`` is true, through the library.
Sizes are those of the library's workloads (hidden 2048 and 7168, 1 to 256 tokens) and generic ones around them:
prefill chunks of thousands of rows, adapter ranks 8 to 128, up to a few hundred adapters."""

import math

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2, "none": 0}
GROUP = 128  # elements of a row that share a scale


# ---------------------------------------------------------------- cases

def listed():
    return [
        # One decoded token between two layers: launch latency.
        dict(name="norm_n1_h2048", op="norm", n=1, H=2048, x="bf16", res="bf16", out="bf16", out8="none", pad=0),
        # A decode batch of the wide layer: BF16 rows for the router, 8-bit rows for FP8 projections.
        dict(name="norm_n64_h7168_both", op="norm", n=64, H=7168, x="bf16", res="bf16", out="bf16", out8="group", pad=0),
        # An odd prefill chunk at an odd width with no alignment, an fp32 residual stream, a scale for each row.
        dict(name="norm_n3001_h2047_row", op="norm", n=3001, H=2047, x="f16", res="f32", out="none", out8="row", pad=2),
        # A first norm without a residual.
        dict(name="norm_n2048_h7168_first", op="norm", n=2048, H=7168, x="bf16", res="none", out="bf16", out8="none", pad=0),
        # The largest: a prefill chunk of the wide layer into FP8 projections.
        dict(name="norm_n8192_h7168_group", op="norm", n=8192, H=7168, x="bf16", res="bf16", out="none", out8="group", pad=0),
        # One decoded token with an adapter: launch latency.
        dict(name="lora_n1_2048_r16", op="lora", n=1, inp=2048, out=2048, r=16, L=64, type="bf16", y="bf16", base=True,
             none=0.0, runs=0, pad=0),
        # A decode batch whose requests have adapters of their own, a few of them none.
        dict(name="lora_n16_7168_r16", op="lora", n=16, inp=7168, out=7168, r=16, L=256, type="bf16", y="bf16", base=True,
             none=0.15, runs=0, pad=0),
        # A larger decode batch over a few adapters of higher rank.
        dict(name="lora_n64_7168_r64", op="lora", n=64, inp=7168, out=2048, r=64, L=8, type="bf16", y="bf16", base=True,
             none=0.0, runs=0, pad=0),
        # 256 rows of a speculative verify step, many adapters, fp16, an odd output width, fp32 rows without a base.
        dict(name="lora_n256_2048_r32_f32", op="lora", n=256, inp=2048, out=5003, r=32, L=200, type="f16", y="f32", base=False,
             none=0.1, runs=4, pad=8),
        # An odd prefill chunk of a dozen requests, some without an adapter.
        dict(name="lora_n3001_2048_r16", op="lora", n=3001, inp=2048, out=2048, r=16, L=16, type="bf16", y="bf16", base=True,
             none=0.2, runs=250, pad=0),
        # The largest: a long prefill chunk of the wide layer.
        dict(name="lora_n8192_7168_r64", op="lora", n=8192, inp=7168, out=7168, r=64, L=8, type="bf16", y="bf16", base=True,
             none=0.0, runs=1024, pad=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.45:
        x = rng.choice(["bf16", "bf16", "f16", "f32"])
        out = rng.choice(["bf16", "f16", "f32", "none"])
        out8 = rng.choice(["none", "row", "group", "group"]) if out != "none" else rng.choice(["row", "group"])
        H = rng.choice([64 * rng.randint(2, 120), 64 * rng.randint(2, 120), _log(rng, 100, 8000)])
        return dict(op="norm", n=min(_log(rng, 1, 8000), 40_000_000 // H), H=H, x=x, res=rng.choice(["none", x, x, "f32"]), out=out,
                    out8=out8, pad=rng.choice([0, 0, 1, 8]))
    n = _log(rng, 1, 6000)
    return dict(op="lora", n=n, inp=32 * _log(rng, 8, 224), out=_log(rng, 200, 7168), r=rng.choice([8, 16, 16, 32, 64, 128, 8 * rng.randint(1, 16)]),
                L=_log(rng, 1, 12 if n > 600 else 200), type=rng.choice(["bf16", "bf16", "f16"]), y=rng.choice(["bf16", "f16", "f32"]),
                base=rng.random() < 0.7, none=rng.choice([0.0, 0.0, 0.2]), runs=rng.choice([0, 0, 4, 40, 500]), pad=rng.choice([0, 0, 8]))


# ---------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 7919 + 13)
    return g


def prepare(case, seed):
    c, g = dict(case), _gen(seed)
    s = {"case": c}
    n = c["n"]
    if c["op"] == "norm":
        H, pad = c["H"], c["pad"]
        # A layer's output and a residual stream some times its size, a few channels of it large.
        s["x"] = torch.randn(n, H + pad, generator=g, device=DEV).to(TYPES[c["x"]])[:, :H]
        s["res"] = None
        if c["res"] != "none":
            spread = 2.0 + 30.0 * (torch.rand(H + pad, generator=g, device=DEV) < 0.01)
            s["res"] = (torch.randn(n, H + pad, generator=g, device=DEV) * spread).to(TYPES[c["res"]])[:, :H]
        s["w"] = (1.0 + 0.2 * torch.randn(H, generator=g, device=DEV)).to(torch.bfloat16)
        s["eps"] = 1e-6
        if own:
            from mixture_experts_decode_router_gb300.layer import MoeNorm
            s["op"] = MoeNorm(s["w"], eps=s["eps"], out_dtype=TYPES.get(c["out"]), out8=None if c["out8"] == "none" else c["out8"])
        return s
    K, O, r, L, t = c["inp"], c["out"], c["r"], c["L"], TYPES[c["type"]]
    s["x"] = torch.randn(n, K + c["pad"], generator=g, device=DEV).to(t)[:, :K]
    s["a"] = (torch.randn(L, r, K, generator=g, device=DEV) / math.sqrt(K)).to(t)
    s["b"] = (torch.randn(L, O, r, generator=g, device=DEV) * (0.5 / math.sqrt(r))).to(t)
    s["scale"] = 0.5 + torch.rand(L, generator=g, device=DEV)
    # Requests of about `runs` consecutive rows (0: of one row each), each with an adapter or none (-1).
    at = torch.arange(n, device=DEV)
    if c["runs"]:
        at = (torch.rand(n, generator=g, device=DEV) < 1.0 / c["runs"]).cumsum(0)
    of = torch.randint(0, L, (n + 1,), generator=g, device=DEV)
    of = torch.where(torch.rand(n + 1, generator=g, device=DEV) < c["none"], -1, of)
    s["idx"] = of[at].to(torch.int32)
    s["base"] = torch.randn(n, O, generator=g, device=DEV).to(TYPES[c["y"]]) if c["base"] else None
    if own:
        from mixture_experts_decode_router_gb300.layer import MoeLora
        s["op"] = MoeLora(s["a"], s["b"], s["scale"], out_dtype=TYPES[c["y"]])
    return s


# ---------------------------------------------------------------- the plain forms

def _norm_plain(s):
    c = s["case"]
    h = s["x"].float()
    new = None
    if s["res"] is not None:
        new = (h + s["res"].float()).to(s["res"].dtype)
        h = new.float()
    y = h / torch.sqrt((h * h).mean(1, keepdim=True) + s["eps"]) * s["w"].float()
    q = scale = None
    if c["out8"] != "none":
        n, H = y.shape
        size = GROUP if c["out8"] == "group" else H
        groups = -(-H // size)
        z = torch.zeros(n, groups * size, device=y.device)
        z[:, :H] = y
        z = z.view(n, groups, size)
        scale = (z.abs().amax(2) / 448.0).clamp(min=2.0 ** -126)
        q = (z / scale[..., None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(n, -1)[:, :H].contiguous()
    return None if c["out"] == "none" else y.to(TYPES[c["out"]]), new, q, scale


def _lora_plain(s):
    c = s["case"]
    n, L, r = c["n"], c["L"], c["r"]
    x, idx = s["x"].float(), s["idx"].long()
    if n <= 16:  # each row's own matrices
        pick = idx.clamp(min=0)
        v = (s["a"][pick].float() * x[:, None, :]).sum(2) * (s["scale"][pick] * (idx >= 0))[:, None]
        y = (s["b"][pick].float() * v[:, None, :]).sum(2)
    else:  # every adapter for every row, and the row's own of them
        mine = (idx[:, None] == torch.arange(L, device=x.device)) * s["scale"]
        v = (x @ s["a"].float().view(L * r, -1).T).view(n, L, r) * mine[..., None]
        y = v.view(n, L * r) @ s["b"].float().transpose(1, 2).reshape(L * r, -1)
    return (y if s["base"] is None else y + s["base"].float()).to(TYPES[c["y"]])


def run(state):
    s, op = state, state["case"]["op"]
    if own:
        if op == "norm":
            return s["op"].forward(s["x"], s["res"])
        return s["op"].forward(s["x"], s["idx"], base=s["base"])
    return _norm_plain(s) if op == "norm" else _lora_plain(s)


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    global own
    was, own = own, False
    s = prepare(case, seed)
    own = was
    c = s["case"]
    if c["op"] == "norm":
        h, new = s["x"].double(), None
        if s["res"] is not None:
            new = torch.add(h, s["res"].double()).to(s["res"].dtype)   # (rounded to its type, whose rows are normalised)
            h = new.double()
        mean = torch.einsum("nh,nh->n", h, h) / c["H"]
        y = h * (mean + s["eps"]).rsqrt()[:, None] * s["w"].double()
        q = scale = None
        if c["out8"] != "none":
            size = GROUP if c["out8"] == "group" else c["H"]
            parts = torch.split(y, size, dim=1)
            scale = torch.stack([p.abs().max(dim=1).values for p in parts], 1) / 448.0
            q = torch.cat([(p / scale[:, i:i + 1]).float().to(torch.float8_e4m3fn).double() for i, p in enumerate(parts)], 1)
        return y if c["out"] != "none" else None, new if new is None else new.double(), q, scale
    y = torch.zeros(c["n"], c["out"], dtype=torch.float64, device=DEV) if s["base"] is None else s["base"].double()
    for a in sorted(set(s["idx"].tolist()) - {-1}):
        rows = torch.nonzero(s["idx"] == a).flatten()
        v = torch.einsum("nk,rk->nr", s["x"][rows].double(), s["a"][a].double())
        y[rows] += float(s["scale"][a]) * torch.einsum("nr,or->no", v, s["b"][a].double())
    return y


# ---------------------------------------------------------------- what a case cannot do without

def work(case):
    c = case
    n = c["n"]
    if c["op"] == "norm":
        H = c["H"]
        scales = 0 if c["out8"] == "none" else 4 * (1 if c["out8"] == "row" else -(-H // GROUP))
        row = H * (BYTES[c["x"]] + 2 * BYTES[c["res"]] + BYTES[c["out"]] + (c["out8"] != "none")) + scales
        return {"bytes": n * row + 2 * H, "flops": n * H * 6}
    K, O, r, L = c["inp"], c["out"], c["r"], c["L"]
    requests = max(1.0, n / c["runs"]) if c["runs"] else n
    with_one = n * (1.0 - c["none"])
    distinct = L * (1.0 - (1.0 - 1.0 / L) ** (requests * (1.0 - c["none"])))  # adapters that at least one row has, on average
    y = BYTES[c["y"]]
    return {"bytes": int(distinct * (r * (K + O) * 2 + 4) + with_one * K * 2 + n * O * y * (2 if c["base"] else 1) + 4 * n),
            "flops": int(2 * with_one * r * (K + O)) + 1}
