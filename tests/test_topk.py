"""moe_topk: refusals (CPU), and routing from logits against plain 64-bit numpy (GPU).

Indices are equal.  Weights: fp32 from exp (2 ulp, 4 * 2^-24), its argument's rounding (half an
ulp of at most 32 for the logits here: 32 * 2^-24), a sum of up to 1024 terms (lane chains of 32
and a butterfly of 5, 37 * 2^-24), the same for the k chosen, two quotients and the factor
(3 * 2^-24): below 120 * 2^-24 relative."""

import numpy as np
import pytest
import torch

from mixture_experts_decode_router_gb300 import binding as B
from mixture_experts_decode_router_gb300 import synth
from mixture_experts_decode_router_gb300.layer import MoeLayer, MoeTopk, make_config, routing_word
from tests.moe_helpers import bf16_bits
from oracle import moe_oracle as O

W_TOL = 120 * 2.0 ** -24


# ---------------------------------------------------------------- the definition in 64 bits

def plain(lg, k, routing="softmax", bias=None, groups=1, kept=1, score="top2", norm=True, factor=1.0):
    """Row by row and expert by expert; lg: float64 [n, E]."""
    n, E = lg.shape
    idx, w = np.empty((n, k), np.int64), np.empty((n, k))
    for t in range(n):
        l = lg[t]
        with np.errstate(all="ignore"):
            if routing == "sigmoid":
                p = np.where(np.isnan(l), np.nan, 1.0 / (1.0 + np.exp(-l)))
            else:
                m = np.nanmax(l) if not np.isnan(l).all() else np.nan
                p = np.zeros(E) if m == -np.inf else np.exp(l - m) / np.sum(np.exp(l - m))
            s = l if bias is None else p + bias
        s = np.where(np.isnan(s), -np.inf, s)
        allowed = np.ones(E, bool)
        if groups > 1:
            size = E // groups
            val = s if bias is not None or score == "max" else np.where(np.isnan(p), -np.inf, p)
            by = -np.sort(-val.reshape(groups, size), axis=1)
            gs = by[:, 0] if score == "max" else by[:, :2].sum(1)
            order = np.lexsort((np.arange(groups), -gs))
            allowed = np.repeat(np.isin(np.arange(groups), order[:kept]), size)
        cand = np.nonzero(allowed)[0]
        order = cand[np.lexsort((cand, -s[cand]))][:k]
        idx[t] = order
        q = p[order]
        if norm:
            # Ratios of p, from log p: p itself can underflow in 64 bits where its ratios are
            # ordinary (equal logits of -3e38 have equal weights).
            with np.errstate(all="ignore"):
                lp = l[order] if routing == "softmax" else -np.logaddexp(0.0, -l[order])
                q = np.exp(lp - lp.max()) if np.isfinite(lp.max()) else q
            tot = q.sum()
            q = np.zeros(k) if tot == 0 else q / tot
        w[t] = q * factor
    return idx, w


def test_definition_matches_the_layer_oracle():
    """Without groups and with the modes that the layer's oracle has, they are the same."""
    rng = np.random.default_rng(0)
    lg = rng.normal(size=(20, 24))
    b = rng.uniform(-0.1, 0.1, 24)
    for mode, bias in (("softmax", None), ("sigmoid", b)):
        i0, w0 = O.route(lg, "softmax" if bias is None else "sigmoid_bias", 5, True, 2.5, bias)
        i1, w1 = plain(lg, 5, mode, bias, factor=2.5)
        assert np.array_equal(i0, i1) and np.allclose(w0, w1, rtol=1e-13)


def test_groups_by_hand():
    p = np.array([[.9, .1, .1, .9, .7, .2, .6, .5]])
    lg = np.log(p / (1 - p))
    # Sigmoid scores; groups of two with sums 1.0, 1.0, 0.9, 1.1: the last, then the lower of a tie.
    i, w = plain(lg, 2, "sigmoid", None, 4, 1, "top2")
    assert i.tolist() == [[6, 7]] and np.allclose(w, [[.6 / 1.1, .5 / 1.1]])
    i, _ = plain(lg, 3, "sigmoid", None, 4, 2, "top2")
    assert i.tolist() == [[0, 6, 7]]
    i, _ = plain(lg, 3, "sigmoid", None, 4, 3, "max")        # best scores .9, .9, .7, .6
    assert i.tolist() == [[0, 3, 4]]


# ---------------------------------------------------------------- refusals, on the CPU

FAKE = 0x7f0000000000      # never dereferenced here


def _cfg(**kw):
    c = B.moe_topk_config_t(64, 4, B.MOE_ROUTE_SOFTMAX, 1, 1.0, B.MOE_F32)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def _call(c, logits=FAKE, stride=64, bias=None, n=2, idx=FAKE, w=FAKE):
    return B.moe_topk(c, logits, stride, bias, n, idx, w, 0)


def test_refusals():
    R = B.MOE_ROUTING
    bad = B.MOE_ERR_INVALID_CONFIG
    assert _call(None) == B.MOE_ERR_NULL
    for kw in (dict(num_experts=0), dict(num_experts=1025), dict(top_k=0), dict(top_k=33), dict(top_k=65),
               dict(routing=4), dict(routing=-1), dict(routing=7), dict(norm_topk_prob=2),
               dict(routed_scaling_factor=float("nan")), dict(routed_scaling_factor=float("inf")),
               dict(logits_type=3), dict(logits_type=-1),
               dict(routing=R(0, 5, 2, 0)),            # 64 experts do not divide into 5 groups
               dict(routing=R(0, 8, 0, 0)), dict(routing=R(0, 8, 9, 0)), dict(routing=R(0, 8, 2, 2)),
               dict(routing=R(0, 0, 2, 0)), dict(routing=R(0, 0, 0, 1)),
               dict(routing=R(0, 32, 1, 0))):          # one group of two experts holds no four
        assert _call(_cfg(**kw)) == bad, kw
    assert _call(_cfg(routing=R(0, 64, 8, 0))) == B.MOE_ERR_UNSUPPORTED
    assert _call(_cfg(routing=B.MOE_ROUTE_SIGMOID_BIAS)) == B.MOE_ERR_NULL
    assert _call(_cfg(routing=B.MOE_ROUTE_SOFTMAX_BIAS)) == B.MOE_ERR_NULL
    assert _call(_cfg(), bias=FAKE) == bad
    assert _call(_cfg(routing=B.MOE_ROUTE_SIGMOID), bias=FAKE) == bad
    assert _call(_cfg(routing=B.MOE_ROUTE_SIGMOID_BIAS), bias=FAKE + 2) == B.MOE_ERR_ALIGNMENT
    assert _call(_cfg(), n=-1) == bad
    assert _call(_cfg(), stride=63) == bad
    for kw in (dict(logits=None), dict(idx=None), dict(w=None)):
        assert _call(_cfg(), **kw) == B.MOE_ERR_NULL
    for kw in (dict(logits=FAKE + 2), dict(idx=FAKE + 2), dict(w=FAKE + 1)):
        assert _call(_cfg(), **kw) == B.MOE_ERR_ALIGNMENT
    assert _call(_cfg(logits_type=B.MOE_BF16), logits=FAKE + 1) == B.MOE_ERR_ALIGNMENT
    assert _call(_cfg(), n=0, logits=None, idx=None, w=None) == B.MOE_OK
    # A valid call of an address that is no device or pinned memory.
    assert _call(_cfg()) == B.MOE_ERR_HOST_MEMORY


def test_layer_routing_words():
    """The layer takes the same words, and needs a bias exactly in the modes that have one."""
    c = make_config(synth.WORKLOADS["decode_n16"].with_(num_groups=8, topk_groups=4))
    assert c.routing == B.MOE_ROUTING(B.MOE_ROUTE_SIGMOID_BIAS, 8, 4, B.MOE_GROUP_TOP2)
    assert B.moe_workspace_bytes(c, 16) > 0
    c.routing = B.MOE_ROUTING(B.MOE_ROUTE_SIGMOID_BIAS, 7, 4, 1)      # 256 experts in 7 groups
    assert B.moe_workspace_bytes(c, 16) == 0
    assert routing_word("softmax") == B.MOE_ROUTE_SOFTMAX
    with pytest.raises(ValueError):
        routing_word("softmax", 256, 1)
    with pytest.raises(KeyError):
        routing_word("softmax", 4, 2, "mean")


def test_holder_refusals():
    with pytest.raises(ValueError):
        MoeTopk(8, 2, bias=torch.zeros(7))
    with pytest.raises(ValueError):
        MoeTopk(8, 2, bias=torch.zeros(8, dtype=torch.float64))
    op = MoeTopk(8, 2)
    for bad in (torch.zeros(4, 7), torch.zeros(8), torch.zeros(8, 4).T, torch.zeros(4, 8)):
        with pytest.raises(ValueError):
            op.forward(bad)


# ---------------------------------------------------------------- routing, on the GPU

gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    B.load()


def check(lg, k, routing="softmax", bias=None, groups=1, kept=1, score="top2", norm=True, factor=1.0):
    op = MoeTopk(lg.shape[1], k, routing, bias, groups, kept, score, norm, factor)
    idx, w = op.forward(lg)
    torch.cuda.synchronize()
    ri, rw = plain(lg.double().cpu().numpy(), k, routing, None if bias is None else bias.double().cpu().numpy(),
                   groups, kept, score, norm, factor)
    assert np.array_equal(idx.cpu().numpy(), ri)
    got = w.cpu().numpy().astype(np.float64)
    assert np.array_equal(np.isnan(got), np.isnan(rw))
    ok = ~np.isnan(rw)
    assert np.all(np.abs(got - rw)[ok] <= W_TOL * np.abs(rw)[ok] + 1e-37), np.max(np.abs(got - rw)[ok])
    return idx, w


def draw(n, E, dtype=torch.float32, seed=0, pad=0, spread=1.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(n, E + pad, generator=g, device="cuda") * spread).to(dtype)[:, :E]


def bias_of(E, seed=9):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.rand(E, generator=g, device="cuda") - 0.5) * 0.2


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("routing", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("groups,kept,score", [(1, 1, "top2"), (8, 4, "top2"), (8, 3, "max")])
@pytest.mark.parametrize("norm", [False, True])
def test_modes(lib, dtype, routing, biased, groups, kept, score, norm):
    check(draw(67, 256, dtype), 8, routing, bias_of(256) if biased else None, groups, kept, score, norm, 2.5)


@gpu
@pytest.mark.parametrize("E,k,groups,kept", [
    (1, 1, 1, 1), (2, 1, 2, 1), (3, 3, 3, 3), (5, 2, 1, 1), (31, 31, 1, 1), (32, 32, 32, 32), (33, 8, 3, 2),
    (60, 4, 1, 1), (64, 6, 16, 3), (96, 6, 4, 2), (100, 7, 10, 3), (128, 8, 1, 1), (160, 6, 8, 3), (257, 9, 1, 1),
    (384, 8, 1, 1), (512, 10, 16, 4), (768, 12, 32, 5), (1000, 32, 8, 2), (1024, 32, 1, 1), (1024, 8, 32, 4)])
@pytest.mark.parametrize("routing,biased", [("softmax", False), ("sigmoid", True)])
def test_expert_counts(lib, E, k, groups, kept, routing, biased):
    for score in ("top2", "max"):
        check(draw(9, E, seed=E), k, routing, bias_of(E) if biased else None, groups, kept, score)


@gpu
@pytest.mark.parametrize("n", [1, 2, 3, 4, 5, 31, 32, 33, 607, 4099])
def test_row_counts_and_strides(lib, n):
    """Odd numbers of rows, of strided and of unaligned logits; the rows behind the last stay."""
    for pad, off in ((0, 0), (5, 0), (8, 1)):
        base = draw(n, 128, torch.float32, seed=n, pad=pad + 1)
        full = torch.randn(n, 128 + pad + 1, generator=torch.Generator(device="cuda").manual_seed(n), device="cuda")
        lg = full[:, off:off + 128]
        del base
        check(lg, 6, "sigmoid", bias_of(128), 8, 4)
    op = MoeTopk(128, 6)
    idx = torch.full((n + 2, 6), 77, dtype=torch.int32, device="cuda")
    w = torch.full((n + 2, 6), 7.5, device="cuda")
    op.forward(full[:, :128], idx=idx, w=w)
    assert (idx[n:] == 77).all() and (w[n:] == 7.5).all()
    assert (idx[:n] < 128).all()


@gpu
def test_no_rows(lib):
    idx, w = MoeTopk(16, 4).forward(torch.empty(0, 16, device="cuda"))
    assert idx.shape == w.shape == (0, 4)


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("routing,biased", [("softmax", False), ("softmax", True), ("sigmoid", False),
                                            ("sigmoid", True)])
@pytest.mark.parametrize("groups,kept", [(1, 1), (8, 4)])
def test_ties_go_to_the_lower_index(lib, dtype, routing, biased, groups, kept):
    """Rows of a few distinct logits, rows of one value, and one bias for all."""
    g = torch.Generator(device="cuda").manual_seed(4)
    lg = (torch.randint(0, 4, (50, 256), generator=g, device="cuda") / 4.0).to(dtype)
    lg[7] = 0
    lg[8] = -3.25
    lg[9, 128:] = -0.0
    lg[9, :128] = 0.0
    b = torch.full((256,), 0.125, device="cuda") if biased else None
    check(lg, 8, routing, b, groups, kept, "max")
    check(lg, 8, routing, b, groups, kept, "top2")


@gpu
@pytest.mark.parametrize("ulps", [1, 2, 5, 40])
@pytest.mark.parametrize("groups,kept,score", [(1, 1, "top2"), (8, 4, "top2"), (8, 4, "max")])
def test_near_ties_are_decided_in_64_bits(lib, ulps, groups, kept, score):
    """Logits a few ulps apart, whose fp32 scores tie or change places, with biases that almost
    cancel the scores' differences."""
    rng = np.random.default_rng(ulps)
    base = rng.normal(size=(40, 256)).astype(np.float32)
    src = rng.integers(0, 256, (40, 256))
    near = np.take_along_axis(base, src, 1)
    step = rng.integers(-ulps, ulps + 1, (40, 256)).astype(np.int32)
    lg = torch.tensor((near.view(np.int32) + step).view(np.float32), device="cuda")
    check(lg, 8, "sigmoid", torch.zeros(256, device="cuda"), groups, kept, score)
    check(lg, 8, "softmax", torch.zeros(256, device="cuda"), groups, kept, score)
    check(lg, 8, "softmax", None, groups, kept, score)
    # One row of logits whose biases bring every score to 0.5, give or take rounding.
    row = lg[:1].expand(40, 256).contiguous()
    b = (0.5 - torch.sigmoid(row[0].double())).float()
    check(row, 8, "sigmoid", b, groups, kept, score)


@gpu
@pytest.mark.parametrize("routing,biased", [("softmax", False), ("sigmoid", False), ("sigmoid", True)])
@pytest.mark.parametrize("norm", [False, True])
def test_masked_experts(lib, routing, biased, norm):
    """-inf and the type's lowest value in masked places, up to rows with nothing left."""
    lg = draw(12, 64, seed=3)
    lg = lg.clone()
    lg[0, 10:] = -float("inf")
    lg[1, 2:] = -float("inf")                  # fewer left than the four chosen
    lg[2] = -float("inf")                      # nothing left
    lg[3, 5:] = torch.finfo(torch.float32).min
    lg[4] = torch.finfo(torch.float32).min
    lg[5, ::2] = -float("inf")
    b = bias_of(64) if biased else None
    for groups, kept in ((1, 1), (8, 2)):
        idx, w = check(lg, 4, routing, b, groups, kept, "max", norm)
        assert torch.isfinite(w).all()


@gpu
def test_far_logits(lib):
    """Sigmoid scores that fp32 holds as 0 or 1, whose normalised ratios are ordinary."""
    g = torch.Generator(device="cuda").manual_seed(1)
    for shift in (-200.0, -95.0, 25.0, 80.0):
        lg = torch.randn(9, 64, generator=g, device="cuda") + shift
        op = MoeTopk(64, 4, "sigmoid")
        idx, w = op.forward(lg)
        d = lg.double()
        top = d.sort(dim=1, descending=True, stable=True).indices[:, :4]
        assert torch.equal(idx.long(), top)
        ref = torch.softmax(-torch.nn.functional.softplus(-d).gather(1, top), 1)
        assert ((w.double() - ref).abs() <= (256 * 2.0 ** -24) * ref).all()   # exponents up to 200 add 200 half-ulps


@gpu
def test_nan_ranks_last(lib):
    lg = draw(6, 40, seed=8).clone()
    lg[0, 3] = float("nan")
    lg[1, 4:] = float("nan")
    lg[2] = float("nan")
    idx, w = MoeTopk(40, 4, "sigmoid", bias_of(40)).forward(lg)
    assert 3 not in idx[0].tolist()
    assert sorted(idx[1].tolist()) == [0, 1, 2, 3]
    assert idx[2].tolist() == [0, 1, 2, 3]
    assert torch.isfinite(w[0]).all() and torch.isfinite(w[3:]).all()


@gpu
@pytest.mark.parametrize("groups,kept", [(1, 1), (8, 2)])
@pytest.mark.parametrize("score", ["max", "top2"])
def test_infinite_logits(lib, groups, kept, score):
    """+inf in one, a few, and all places: a sigmoid of 1, and the first by its logit."""
    lg = draw(9, 64, seed=12).clone()
    lg[0, 7] = lg[1, 3] = lg[1, 50] = float("inf")
    lg[2, 10:30] = float("inf")
    lg[3] = float("inf")
    lg[4, 5], lg[4, 6:] = float("inf"), -float("inf")
    for b in (None, bias_of(64)):
        idx, w = check(lg, 4, "sigmoid", b, groups, kept, score)
        assert torch.isfinite(w).all()
    idx, _ = MoeTopk(64, 4).forward(lg)
    order = lg.sort(dim=1, descending=True, stable=True).indices[:, :4]
    assert torch.equal(idx.long(), order)


@gpu
def test_infinite_bias(lib):
    """A bias of -inf keeps an expert out while others are left; +inf takes it first."""
    lg, b = draw(20, 64, seed=13), bias_of(64)
    b[::2] = -float("inf")
    b[5] = float("inf")
    idx, _ = check(lg, 4, "sigmoid", b)
    assert (idx[:, 0] == 5).all() and (idx % 2 == 1).all()


@gpu
def test_two_streams_at_once(lib):
    lg = [draw(500, 256, seed=s) for s in (20, 21)]
    ops = [MoeTopk(256, 8, "sigmoid", bias_of(256), 8, 4), MoeTopk(256, 6)]
    want = [[tuple(t.clone() for t in op.forward(l)) for l in lg] for op in ops]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        got = []
        for st, op in zip(streams, ops):
            with torch.cuda.stream(st):
                got.append([op.forward(l) for l in lg])
        torch.cuda.synchronize()
        for g2, w2 in zip(got, want):
            for (i, w), (ri, rw) in zip(g2, w2):
                assert torch.equal(i, ri) and torch.equal(w, rw)


def test_arguments_that_are_no_tensors():
    """On the CPU: what is no tensor, or of no type that the operators take, is refused before anything runs."""
    op = MoeTopk(64, 4)
    for bad in (None, 3, [[0.0] * 64]):
        with pytest.raises(TypeError):
            op.forward(bad)
    with pytest.raises(TypeError):
        op.forward(torch.zeros(2, 64), idx=1)
    for bad in (torch.zeros(2, 64, dtype=torch.float64), torch.zeros(2, 64, dtype=torch.int32)):
        with pytest.raises(KeyError):
            op.forward(bad)
    for bad in (torch.zeros(64), torch.zeros(2, 63), torch.zeros(2, 128)[:, ::2], torch.zeros(1, 2, 64), torch.zeros(2, 64)):
        with pytest.raises(ValueError):
            op.forward(bad)                # (the last is not on the GPU)


@gpu
def test_given_outputs_are_checked(lib):
    lg = draw(4, 64)
    op = MoeTopk(64, 4)
    good = torch.empty(4, 4, dtype=torch.int32, device="cuda")
    for bad in (good.long(), good[:3], good[:, :3], good.cpu(), torch.empty(4, 8, dtype=torch.int32, device="cuda")[:, ::2]):
        with pytest.raises(ValueError):
            op.forward(lg, idx=bad)
    with pytest.raises(ValueError):
        op.forward(lg, w=good)
    with pytest.raises(ValueError):
        MoeTopk(64, 4, "sigmoid", torch.zeros(64)).forward(lg)      # a bias on the CPU


@gpu
def test_many_rows_past_32_bit_offsets(lib):
    """Rows whose offset in elements passes 2^31: the last rows are those of a small call."""
    stride = 1 << 20
    n = (1 << 11) + 3
    try:
        buf = torch.empty(n * stride, dtype=torch.bfloat16, device="cuda")
    except torch.OutOfMemoryError:
        pytest.skip("needs 4.3 GB")
    lg = buf.view(n, stride)[:, :64]
    small = draw(n, 64, torch.bfloat16, seed=2)
    lg.copy_(small)
    op = MoeTopk(64, 4)
    a, b = op.forward(lg), op.forward(small)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@gpu
def test_another_stream_and_replay(lib):
    lg = [draw(33, 256, seed=s) for s in range(3)]
    op = MoeTopk(256, 8, "sigmoid", bias_of(256), 8, 4)
    want = [tuple(t.clone() for t in op.forward(l)) for l in lg]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        got = op.forward(lg[1])
    st.synchronize()
    assert torch.equal(got[0], want[1][0]) and torch.equal(got[1], want[1][1])
    buf = lg[0].clone()
    idx, w = torch.empty_like(want[0][0]), torch.empty_like(want[0][1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        op.forward(buf, idx=idx, w=w)
    for l, (ri, rw) in zip(lg, want):
        buf.copy_(l)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(idx, ri) and torch.equal(w, rw)


@gpu
def test_pinned_logits(lib):
    lg = draw(7, 64)
    host = lg.cpu().pin_memory()
    op = MoeTopk(64, 4)
    a, b = op.forward(host), op.forward(lg)
    torch.cuda.synchronize()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


# ---------------------------------------------------------------- the layer

@gpu
@pytest.mark.parametrize("routing", ["softmax", "softmax_bias", "sigmoid", "sigmoid_bias"])
@pytest.mark.parametrize("groups,kept,score", [(1, 1, "top2"), (4, 2, "top2"), (8, 3, "max")])
@pytest.mark.parametrize("n", [1, 3, 20])
def test_layer(lib, routing, groups, kept, score, n):
    """moe_route and moe_forward route as moe_topk does on the same logits, and the output is
    that of moe_experts on these routes."""
    cfg = synth.LayerConfig("g", 256, 32, 4, 128, 128, routing, True, 2.5, synth.FMT_BF16, n, num_groups=groups,
                            topk_groups=kept, group_score=score, shared_gate=n > 1)
    lw = synth.make_weights(cfg, "cuda")
    x = synth.make_input(cfg, n, "cuda")
    layer = MoeLayer(lw, n)
    idx, w, lg = layer.route(x)
    mode = routing.split("_")[0]
    op = MoeTopk(32, 4, mode, lw.correction_bias, groups, kept, score, True, 2.5)
    i2, w2 = op.forward(lg)
    ref = O.router_logits(O.bf16_decode(bf16_bits(x)), O.bf16_decode(bf16_bits(lw.router_w)))
    assert np.max(np.abs(lg.cpu().numpy() - ref)) <= 1e-4 * np.sqrt(np.mean(ref ** 2))
    if groups > 1 or routing in ("softmax_bias", "sigmoid"):
        assert torch.equal(idx, i2) and torch.equal(w, w2)
    out, i3, w3 = layer.forward(x)
    assert torch.equal(i3, idx) and torch.equal(w3, w)
    assert torch.equal(out, layer.experts(x, idx, w))
    assert layer.device_error() == 0
    ri, rw = plain(lg.double().cpu().numpy(), 4, mode,
                   None if lw.correction_bias is None else lw.correction_bias.double().cpu().numpy(), groups, kept,
                   score, True, 2.5)
    assert np.array_equal(idx.cpu().numpy(), ri)
    assert np.max(np.abs(w.cpu().numpy() - rw)) <= 1e-5


@gpu
def test_logits_to_experts(lib):
    """A run as a caller makes it: logits of a product of its own, moe_topk, INT4 experts."""
    cfg = synth.LayerConfig("run", 256, 64, 4, 128, 0, synth.ROUTE_SIGMOID_BIAS, True, 2.5, synth.FMT_INT4_G64, 12)
    lw = synth.make_weights(cfg, "cuda")
    x = synth.make_input(cfg, 12, "cuda")
    lg = (x.float() @ lw.router_w.float().T).to(torch.bfloat16)
    idx, w = check(lg, 4, "sigmoid", lw.correction_bias, 8, 3, "top2", True, 2.5)
    out = MoeLayer(lw, 12).experts(x, idx, w)
    from tests.int4_helpers import int4_oracle_layer
    L = int4_oracle_layer(lw)
    xe = O.bf16_decode(bf16_bits(x))
    ref = np.zeros((12, 256))
    for t in range(12):
        for j in range(4):
            e = int(idx[t, j])
            ref[t] += float(w[t, j]) * O.swiglu_mlp(xe[t], L.gate.expert(e), L.up.expert(e), L.down.expert(e))
    from tests.test_int4_experts import close
    close(out.float().cpu().numpy(), ref)


@gpu
@pytest.mark.parametrize("size,scale", [(2, 100.0), (4, 1024.0), (4, 1e4), (8, 1e6), (32, 4096.0)])
@pytest.mark.parametrize("kept", [1, 4])
@pytest.mark.parametrize("routing", ["softmax", "sigmoid"])
def test_group_sums_that_cancel(lib, size, scale, kept, routing):
    """Biases of opposite sign in each group's two best: the rounding of p + bias goes with the terms,
    and what is left of their sum orders the groups."""
    E = 8 * size
    lg = draw(4000, E, seed=size)
    b = torch.full((E,), -scale, device="cuda")
    b[torch.arange(8, device="cuda") * size + torch.arange(8, device="cuda") % size] = scale
    check(lg, min(4, kept * size), routing, b, 8, kept, "top2")


@gpu
@pytest.mark.parametrize("score", ["max", "top2"])
@pytest.mark.parametrize("routing", ["softmax", "sigmoid"])
def test_infinite_biases_in_groups(lib, score, routing):
    """+inf twice in a group (of 2, 4 and 32 experts), in two groups, next to -inf, and groups of -inf alone."""
    inf = float("inf")
    for size in (2, 4, 32):
        E = 8 * size
        lg, base = draw(300, E, seed=30 + size), bias_of(E)
        for at in ({5: (inf, inf)}, {5: (inf, inf), 2: (inf, inf)}, {6: (inf, -inf)}, {3: (-inf, -inf), 1: (inf, inf)}):
            b = base.clone()
            for g, v in at.items():
                b[g * size:g * size + 2] = torch.tensor(v, device="cuda")
            for kept in (1, 4):
                check(lg, 2, routing, b, 8, kept, score)
        b = base.clone()
        b[:5 * size] = -inf                        # three groups are left
        check(lg, 2, routing, b, 8, 4, score)


@gpu
@pytest.mark.parametrize("norm", [False, True])
def test_weights_of_far_logits(lib, norm):
    """Small sigmoids and softmax terms keep their relative accuracy.  Logits are whole numbers, so l - m is
    exact: exp (2 ulp, 4 * 2^-24), 1 + exp (2^-24), a quotient (2^-24), the row's sum (its terms, and 7 additions
    at 64 experts: 11 * 2^-24), the factor (2^-24), and with norm the k chosen and their quotient (6 * 2^-24):
    24 * 2^-24 at most."""
    d = torch.arange(64, device="cuda", dtype=torch.float32)
    lg = torch.stack([-d, -1.25 * d, 20.0 - d, -17.0 - d])
    for routing in ("sigmoid", "softmax"):
        op = MoeTopk(64, 32, routing, norm_topk_prob=norm, routed_scaling_factor=2.5)
        idx, w = op.forward(lg)
        ri, rw = plain(lg.double().cpu().numpy(), 32, routing, norm=norm, factor=2.5)
        assert np.array_equal(idx.cpu().numpy(), ri)
        assert np.max(np.abs(w.double().cpu().numpy() / rw - 1)) <= 24 * 2.0 ** -24
