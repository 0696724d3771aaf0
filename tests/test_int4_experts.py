"""INT4 experts with group scales: the format (CPU), refusals (CPU), and the layer on every
path against the fp64 oracle (GPU).

Output tolerance, per element: 2^-8 |ref| for the BF16 output, and 5e-3 RMS(ref) for the f16
values inside.  At most four roundings to f16 (gate, up and down weights, and SiLU(g) u), each
at most 2^-11 relative, enter sums of independently signed terms, so each moves an output by a
standard deviation of at most 2^-11 / sqrt(3) of its RMS, gate and up through a SwiGLU whose
slope stays below 1.3: sqrt(4) * 1.3 * 2^-11 / sqrt(3) = 7.4e-4, times six.

With a pre-expert norm the experts' input is itself rounded to BF16, as the layer defines it and the
oracle does not: at most 2^-8 relative for each element, which moves g and u by at most
2^-8 / sqrt(3) of their RMS and an output by sqrt(1.3^2 + 1) times that, 3.7e-3, times six
(2.2e-2)."""

import ctypes
import dataclasses

import numpy as np
import pytest
import torch

from mixture_experts_decode_router_gb300 import binding as B
from mixture_experts_decode_router_gb300 import synth
from mixture_experts_decode_router_gb300.layer import MoeLayer, make_config
from oracle import moe_oracle as O
from tests.int4_helpers import int4_oracle_layer
from tests.moe_helpers import bf16_bits, gap_fn_for

FORMATS = sorted(synth.INT4_GROUP)


def cfg_of(fmt="int4_g32", **kw):
    d = dict(name="int4", hidden=256, num_experts=16, top_k=2, inter=128, shared_inter=128,
             routing=synth.ROUTE_SOFTMAX, norm_topk_prob=True, routed_scaling_factor=1.0, expert_fmt=fmt, n_tokens=1)
    d.update(kw)
    return synth.LayerConfig(**d)


def close(got, ref, norm=False):
    rms = float(np.sqrt(np.mean(ref ** 2)))
    bad = np.abs(got - ref) - (2.0 ** -8 * np.abs(ref) + (5e-3 + (2.2e-2 if norm else 0.0)) * rms)
    assert bad.max() <= 0, f"over by {bad.max():.3e} (RMS {rms:.3e})"


# ---------------------------------------------------------------- the format, on the CPU

@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("zero", [False, True])
def test_decode_by_hand(fmt, zero):
    """Every code of one row, decoded element by element in Python integers."""
    G = synth.INT4_GROUP[fmt]
    rng = np.random.default_rng(5)
    packed = rng.integers(0, 256, (3, G), dtype=np.uint8)              # 2 G elements: two groups
    scale = torch.tensor(rng.uniform(0.01, 2, (3, 2)), dtype=torch.bfloat16)
    zp = rng.integers(0, 16, (3, 2), dtype=np.uint8) if zero else None
    w = O.dequant_int4(packed, scale.view(torch.int16).numpy().view(np.uint16), zp, G)
    for o in range(3):
        for i in range(2 * G):
            code = (int(packed[o, i // 2]) >> (4 * (i % 2))) & 15
            z = 8 if zp is None else int(zp[o, i // G])
            assert w[o, i] == (code - z) * float(scale[o, i // G])


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("zero", [False, True])
def test_quantiser_error(fmt, zero):
    """Within a group every value is at most half a step off (plus the scale's own BF16
    rounding of at most 2^-8, times the 15 steps of the range)."""
    G = synth.INT4_GROUP[fmt]
    w = torch.randn(8, 4 * G, generator=torch.Generator().manual_seed(3)) * 0.02
    q, s, z = synth.quant_int4(w, G, zero)
    back = O.dequant_int4(q.numpy(), s.view(torch.int16).numpy().view(np.uint16), None if z is None else z.numpy(), G)
    step = s.float().numpy().repeat(G, axis=1)
    # A rounded zero point can move an end of the range by half a step more.
    assert np.all(np.abs(back - w.numpy()) <= step * (0.5 + 15 * 2.0 ** -8 + (0.5 if zero else 0.0)))


def test_matrix_bytes():
    assert synth.matrix_bytes("int4_g64", 128, 256) == 128 * 128 + 2 * 128 * 4
    assert synth.matrix_bytes("int4_g64", 128, 256, True) == 128 * 128 + 3 * 128 * 4


# ---------------------------------------------------------------- refusals, on the CPU

FAKE = 0x7f0000000000      # never dereferenced here


def _weights(**kw):
    w = B.moe_weights_t()
    w.router_w = FAKE
    for m in ("gate", "up", "down", "sh_gate", "sh_up", "sh_down"):
        getattr(w, m).w = FAKE
        getattr(w, m).scale = FAKE
    for k, v in kw.items():
        setattr(w, k, v)
    return w


def test_refusals():
    out, big = FAKE + 0x100000, 1 << 40

    def call(c, w):
        return B.moe_forward(c, w, FAKE, 1, out, None, None, FAKE, big, 0)

    for fmt, g in synth.INT4_GROUP.items():
        for field in ("hidden", "inter", "shared_inter"):
            c = make_config(cfg_of(fmt, hidden=256, inter=256, shared_inter=256))
            setattr(c, field, 256 + g // 2 if g > 32 else 272)      # not whole groups
            assert call(c, _weights()) == B.MOE_ERR_INVALID_CONFIG
            assert B.moe_workspace_bytes(c, 4) == 0
        c = make_config(cfg_of(fmt))
        w = _weights()
        w.up.scale = None
        assert call(c, w) == B.MOE_ERR_NULL
        w = _weights()
        w.up.scale = FAKE + 2
        assert call(c, w) == B.MOE_ERR_ALIGNMENT
        # Zero points are bytes (any alignment) and optional: the workspace check comes next.
        w = _weights()
        w.up.zero = FAKE + 1
        assert B.moe_forward(c, w, FAKE, 1, out, None, None, FAKE, 16, 0) == B.MOE_ERR_WORKSPACE
    c = make_config(cfg_of())
    c.expert_fmt = 6
    assert call(c, _weights()) == B.MOE_ERR_INVALID_CONFIG
    c = make_config(cfg_of())
    c.router_fmt = B.MOE_W_INT4_G32      # a router is BF16 or NVFP4
    assert call(c, _weights()) == B.MOE_ERR_INVALID_CONFIG


def test_zero_shares_scale2():
    """The zero points sit where scale2 does, and the struct keeps its size."""
    assert B.moe_qmat_t.zero.offset == B.moe_qmat_t.scale2.offset == 16
    assert ctypes.sizeof(B.moe_qmat_t) == 24


# ---------------------------------------------------------------- the layer, on the GPU

gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    B.load()


def check(cfg, n, path="auto", x=None, lw=None):
    lw = synth.make_weights(cfg, "cuda") if lw is None else lw
    L = int4_oracle_layer(lw)
    if x is None:
        x = synth.make_input(cfg, n, "cuda", gap_fn=gap_fn_for(L))
    layer = MoeLayer(lw, n, path)
    out, idx, w = layer.forward(x)
    torch.cuda.synchronize()
    assert layer.device_error() == 0
    ref, ridx, rw, _ = O.moe_forward(L, bf16_bits(x))
    assert np.array_equal(idx.cpu().numpy(), ridx)
    assert np.max(np.abs(w.cpu().numpy() - rw)) <= 1e-5 * max(1.0, cfg.routed_scaling_factor)
    close(out.float().cpu().numpy(), ref, cfg.pre_expert_norm)
    return lw, x, layer, out, idx, w


@gpu
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("zero", [False, True])
@pytest.mark.parametrize("path", ["auto", "token_major", "grouped"])
@pytest.mark.parametrize("n", [1, 2, 5, 17])
def test_layer(lib, fmt, zero, path, n):
    check(cfg_of(fmt, zero_points=zero), n, path)


@gpu
@pytest.mark.parametrize("path", ["auto", "token_major", "grouped"])
@pytest.mark.parametrize("H,I,S,E,k,n", [
    (96, 32, 32, 5, 3, 1),        # the smallest widths: less than one tile, one group
    (96, 32, 32, 5, 3, 6),
    (160, 96, 0, 3, 3, 9),        # no shared expert, every expert chosen
    (416, 288, 160, 40, 8, 33),   # odd tiles of 32
    (1056, 544, 96, 7, 1, 70),    # top-1, many tokens an expert
])
def test_odd_sizes(lib, path, H, I, S, E, k, n):
    check(cfg_of("int4_g32", hidden=H, inter=I, shared_inter=S, num_experts=E, top_k=k, zero_points=True,
                 routing=synth.ROUTE_SIGMOID_BIAS, routed_scaling_factor=2.5), n, path)


@gpu
@pytest.mark.parametrize("n", [1, 3, 24])
def test_norm_and_shared_gate(lib, n):
    check(cfg_of("int4_g64", shared_gate=True, pre_expert_norm=True), n)


@gpu
@pytest.mark.parametrize("n,path", [(2, "auto"), (24, "auto"), (24, "grouped"), (130, "auto")])
def test_rows_do_not_depend_on_the_batch(lib, n, path):
    """A token's output bits with other tokens in the batch, permuted, and with a duplicate."""
    cfg = cfg_of("int4_g64", zero_points=True)
    lw, x, layer, out, _, _ = check(cfg, n, path)
    p = torch.randperm(n, generator=torch.Generator().manual_seed(1)).cuda()
    out2, _, _ = MoeLayer(lw, n, path).forward(x[p].contiguous())
    assert torch.equal(out2, out[p])
    y = x.clone()
    y[0] = x[n - 1]
    out3, _, _ = MoeLayer(lw, n, path).forward(y)
    assert torch.equal(out3[0], out[n - 1]) and torch.equal(out3[1:], out[1:])


@gpu
@pytest.mark.parametrize("path", ["auto", "grouped", "token_major"])
@pytest.mark.parametrize("n", [1, 7])
def test_given_routing(lib, n, path):
    """moe_experts with routes the caller made: an expert twice in one token's row, indices
    outside the layer (dropped), a zero weight, and a row whose every route is dropped."""
    cfg = cfg_of("int4_g32", top_k=4)
    lw = synth.make_weights(cfg, "cuda")
    L = int4_oracle_layer(lw)
    x = synth.make_input(cfg, n, "cuda")
    g = torch.Generator().manual_seed(2)
    idx = torch.randint(0, 16, (n, 4), generator=g)
    idx[0] = torch.tensor([3, 3, 11, -1])
    if n > 1:
        idx[1] = torch.tensor([-5, 16, 1 << 30, -(1 << 31)])
    w = torch.rand(n, 4, generator=g)
    w[-1, 0] = 0
    layer = MoeLayer(lw, n, path)
    out = layer.experts(x, idx.to(torch.int32).cuda(), w.cuda())
    torch.cuda.synchronize()
    assert layer.device_error() == 0
    xe = O.bf16_decode(bf16_bits(x))
    sh = O.swiglu_mlp(xe, L.sh_gate.expert(0), L.sh_up.expert(0), L.sh_down.expert(0))
    ref = sh.copy()
    for t in range(n):
        for j in range(4):
            e = int(idx[t, j])
            if 0 <= e < 16:
                ref[t] += float(w[t, j]) * O.swiglu_mlp(xe[t], L.gate.expert(e), L.up.expert(e), L.down.expert(e))
    close(out.float().cpu().numpy(), ref)


@gpu
@pytest.mark.parametrize("n", [1, 6])
def test_expert_parallel(lib, n):
    """Two ranks' partials and the shared-expert call: slices of stacked scales and zero points."""
    cfg = cfg_of("int4_g32", zero_points=True)
    lw, x, _, _, _, _ = check(cfg, n)
    L = int4_oracle_layer(lw)
    total = np.zeros((n, cfg.hidden))
    for r in ((0, 5), (5, 16)):
        layer = MoeLayer(synth.expert_slice(lw, *r), n, experts=r, exclude_shared=True)
        out, _, _ = layer.forward(x)
        ref, _, _, _ = O.moe_forward(L, bf16_bits(x), experts=r, include_shared=False)
        got = out.float().cpu().numpy()
        close(got, ref) if np.any(ref) else None
        total += got
    layer = MoeLayer(synth.expert_slice(lw, 16, 16), n, experts=(16, 16), accumulate=True)
    out = torch.tensor(total, dtype=torch.bfloat16, device="cuda")
    before = out.float().cpu().numpy()
    layer.forward(x, out=out, routing=False)
    ref = O.moe_forward(L, bf16_bits(x), experts=(0, 0))[0]
    close(out.float().cpu().numpy(), before + ref)


@gpu
@pytest.mark.parametrize("n", [1, 12])
def test_captured_and_replayed(lib, n):
    """Two layers with workspaces of their own in one graph, replayed on new inputs."""
    cfg = cfg_of("int4_g64")
    lw = synth.make_weights(cfg, "cuda")
    xs = [synth.make_input(cfg, n, "cuda", stream=s) for s in range(3)]
    a, b = MoeLayer(lw, n), MoeLayer(lw, n)
    want = [a.forward(x)[0].clone() for x in xs]
    buf, oa, ob = xs[0].clone(), torch.empty_like(want[0]), torch.empty_like(want[0])
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        a.forward(buf, out=oa)
        b.forward(buf, out=ob)
    torch.cuda.current_stream().wait_stream(st)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a.forward(buf, out=oa)
        b.forward(buf, out=ob)
    for x, r in zip(xs, want):
        buf.copy_(x)
        oa.zero_(), ob.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(oa, r) and torch.equal(ob, r)


@gpu
@pytest.mark.parametrize("n", [1, 5, 40])
def test_pinned_input_and_output(lib, n):
    cfg = cfg_of("int4_g32")
    lw, x, layer, out, idx, w = check(cfg, n)
    xh, oh = x.cpu().pin_memory(), torch.empty(n, cfg.hidden, dtype=torch.bfloat16).pin_memory()
    layer.forward(xh, out=oh, idx=torch.empty_like(idx), w=torch.empty_like(w))
    torch.cuda.synchronize()
    assert torch.equal(oh, out.cpu())


@gpu
@pytest.mark.parametrize("n", [1, 2, 6, 30])
def test_route_then_experts_is_forward(lib, n):
    cfg = cfg_of("int4_g64", zero_points=True, shared_gate=True)
    lw, x, layer, out, idx, w = check(cfg, n)
    i2, w2, _ = layer.route(x)
    assert torch.equal(i2, idx) and torch.equal(w2, w)
    assert torch.equal(layer.experts(x, i2, w2), out)


@gpu
@pytest.mark.parametrize("n", [1, 20])
def test_zero_points_in_some_matrices(lib, n):
    """Zero points for up and the shared down alone, and at an odd address."""
    cfg = cfg_of("int4_g32", zero_points=True)
    lw = synth.make_weights(cfg, "cuda")
    for m in ("gate", "down", "sh_gate", "sh_up"):
        setattr(lw, m, dataclasses.replace(getattr(lw, m), zero=None))
    buf = torch.zeros(lw.up.zero.numel() + 1, dtype=torch.uint8, device="cuda")
    odd = buf[1:].view(lw.up.zero.shape)
    odd.copy_(lw.up.zero)
    lw.up = dataclasses.replace(lw.up, zero=odd)
    for path in ("auto", "token_major", "grouped"):
        check(cfg, n, path, lw=lw)


@gpu
@pytest.mark.parametrize("n", [1, 2, 9])
def test_magnitudes(lib, n):
    """Inputs far from 1: activations that f16 would hold as zero or infinity."""
    cfg = cfg_of("int4_g64", shared_inter=0)
    lw = synth.make_weights(cfg, "cuda")
    L = int4_oracle_layer(lw)
    for scale in (2.0 ** -14, 2.0 ** 14):
        x = synth.make_input(cfg, n, "cuda") * scale
        g = torch.Generator().manual_seed(n)
        idx = torch.randint(0, 16, (n, 2), generator=g).to(torch.int32).cuda()
        w = torch.rand(n, 2, generator=g).cuda()
        out = MoeLayer(lw, n).experts(x, idx, w)
        xe = O.bf16_decode(bf16_bits(x))
        ref = np.zeros((n, cfg.hidden))
        for t in range(n):
            for j in range(2):
                e = int(idx[t, j])
                ref[t] += float(w[t, j]) * O.swiglu_mlp(xe[t], L.gate.expert(e), L.up.expert(e), L.down.expert(e))
        close(out.float().cpu().numpy(), ref)


@gpu
def test_many_tokens_of_one_expert(lib):
    """Every token on the same two experts: segments of every length up to the tile, and past it."""
    cfg = cfg_of("int4_g32", zero_points=True)
    lw = synth.make_weights(cfg, "cuda")
    L = int4_oracle_layer(lw)
    for n in (7, 8, 9, 15, 16, 17, 33):
        x = synth.make_input(cfg, n, "cuda")
        idx = torch.tensor([[3, 9]] * n, dtype=torch.int32, device="cuda")
        w = torch.full((n, 2), 0.5, device="cuda")
        out = MoeLayer(lw, n).experts(x, idx, w)
        xe = O.bf16_decode(bf16_bits(x))
        ref = O.swiglu_mlp(xe, L.sh_gate.expert(0), L.sh_up.expert(0), L.sh_down.expert(0))
        for e in (3, 9):
            ref = ref + 0.5 * O.swiglu_mlp(xe, L.gate.expert(e), L.up.expert(e), L.down.expert(e))
        close(out.float().cpu().numpy(), ref)


@gpu
@pytest.mark.parametrize("n,marks", [(1, 5), (4, 5), (5, 6), (9, 6)])
def test_timed_markers(lib, n, marks):
    """The markers that moe.h counts for the streaming kernels, in stream order, and the same bits."""
    cfg = cfg_of("int4_g64")
    lw, x, layer, out, idx, w = check(cfg, n)
    ev = [torch.cuda.Event(enable_timing=True) for _ in range(8)]
    for e in ev:
        e.record()
    got = torch.empty_like(out)
    s, nm = B.moe_forward_timed(layer.c_cfg, layer.c_w, x, n, got, torch.empty_like(idx), torch.empty_like(w), layer.ws,
                                layer.ws_bytes, None, [e.cuda_event for e in ev])
    torch.cuda.synchronize()
    assert s == B.MOE_OK and nm == marks
    assert torch.equal(got, out)
    assert all(ev[i].elapsed_time(ev[i + 1]) >= 0 for i in range(nm - 1))


@gpu
@pytest.mark.parametrize("n", [2, 3, 4])
@pytest.mark.parametrize("held", [(0, 16), (5, 11)])
def test_a_few_tokens_as_each_alone(lib, n, held):
    """Up to four tokens of small experts: the bits of every token alone, with an expert twice in
    a row, indices outside the layer, experts held elsewhere, and the shared expert's gate."""
    cfg = cfg_of("int4_g32", top_k=4, zero_points=True, shared_gate=True)
    lw = synth.expert_slice(synth.make_weights(cfg, "cuda"), *held)
    x = synth.make_input(cfg, n, "cuda")
    g = torch.Generator().manual_seed(n)
    idx = torch.randint(0, 16, (n, 4), generator=g).to(torch.int32)
    idx[0] = torch.tensor([7, 7, -1, 99])
    idx, w = idx.cuda(), torch.rand(n, 4, generator=g).cuda()
    layer, one = MoeLayer(lw, n, experts=held), MoeLayer(lw, 1, experts=held)
    out = layer.experts(x, idx, w)
    for t in range(n):
        assert torch.equal(out[t], one.experts(x[t:t + 1], idx[t:t + 1], w[t:t + 1])[0])
    assert layer.device_error() == 0


@gpu
@pytest.mark.parametrize("n", [1, 3, 40])
def test_accumulate_adds_to_the_output(lib, n):
    cfg = cfg_of("int4_g32", zero_points=True)
    lw, x, _, out, idx, w = check(cfg, n)
    was = torch.randn(n, cfg.hidden, generator=torch.Generator().manual_seed(n)).to(torch.bfloat16).cuda()
    got = MoeLayer(lw, n, accumulate=True).forward(x, out=was.clone())[0]
    L = int4_oracle_layer(lw)
    ref = O.moe_forward(L, bf16_bits(x))[0] + was.double().cpu().numpy()
    close(got.float().cpu().numpy(), ref)


@gpu
@pytest.mark.parametrize("n", [1, 10])
def test_two_streams_at_once(lib, n):
    """Two layers, a workspace each, on two streams; then two streams sharing the weights."""
    cfg = cfg_of("int4_g64")
    lw = synth.make_weights(cfg, "cuda")
    xs = [synth.make_input(cfg, n, "cuda", stream=s) for s in range(2)]
    layers = [MoeLayer(lw, n) for _ in range(2)]
    want = [l.forward(x)[0].clone() for l, x in zip(layers, xs)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        got = []
        for st, l, x in zip(streams, layers, xs):
            with torch.cuda.stream(st):
                got.append([l.forward(x)[0] for _ in range(3)])
        torch.cuda.synchronize()
        assert all(torch.equal(y, r) for ys, r in zip(got, want) for y in ys)


@gpu
@pytest.mark.parametrize("n", [1, 6])
def test_static_workspace(lib, n):
    cfg = cfg_of("int4_g128")
    lw, x, layer, out, idx, w = check(cfg, n)
    got, i2, w2 = torch.empty_like(out), torch.empty_like(idx), torch.empty_like(w)
    assert B.moe_forward_static_ws(layer.c_cfg, layer.c_w, x, n, got, i2, w2) == B.MOE_OK
    torch.cuda.synchronize()
    assert torch.equal(got, out) and torch.equal(i2, idx) and torch.equal(w2, w)
    assert B.moe_static_workspace_check()[:2] == (B.MOE_OK, 0)


@gpu
@pytest.mark.parametrize("n", [1, 2, 9, 40])
def test_a_workspace_as_large_as_it_says(lib, n):
    """A workspace of exactly moe_workspace_bytes in front of a guard: nothing past its end is
    written, and one byte less is refused."""
    cfg = cfg_of("int4_g32", inter=160, shared_inter=96)
    lw, x, layer, out, idx, w = check(cfg, n)
    size = B.moe_workspace_bytes(layer.c_cfg, n)
    buf = torch.zeros(size + 4096, dtype=torch.uint8, device="cuda")
    buf[size:] = 0xA5
    got = torch.empty(n * cfg.hidden + 512, dtype=torch.bfloat16, device="cuda").fill_(3.0)
    s = B.moe_forward(layer.c_cfg, layer.c_w, x, n, got, torch.empty_like(idx), torch.empty_like(w), buf, size)
    torch.cuda.synchronize()
    assert s == B.MOE_OK
    assert torch.equal(got[:n * cfg.hidden].view(n, -1), out) and (got[n * cfg.hidden:] == 3.0).all()
    assert (buf[size:] == 0xA5).all()
    assert B.moe_forward(layer.c_cfg, layer.c_w, x, n, got, idx, w, buf, size - 1) == B.MOE_ERR_WORKSPACE


@gpu
def test_special_values_stay_in_their_row(lib):
    """NaN and infinity in one token's input do not reach another token's output."""
    cfg = cfg_of("int4_g32", n_tokens=9)
    lw, x, layer, out, idx, w = check(cfg, 9)
    y = x.clone()
    y[4, 3] = float("nan")
    y[6, 200] = float("inf")
    got = layer.experts(y, idx, w)
    rest = [0, 1, 2, 3, 5, 7, 8]
    assert torch.equal(got[rest], layer.experts(x, idx, w)[rest])
    assert torch.isnan(got[4]).all()


@gpu
@pytest.mark.parametrize("name,fmt,n", [("decode_n1", "int4_g128", 1), ("decode_n16", "int4_g64", 16),
                                        ("nvfp4_n256", "int4_g32", 256)])
def test_workload_sizes(lib, name, fmt, n):
    cfg = dataclasses.replace(synth.WORKLOADS[name], expert_fmt=fmt, zero_points=fmt == "int4_g64", dup_frac=0.0)
    lw = synth.make_weights(cfg, "cuda")
    L = int4_oracle_layer(lw)
    x = synth.make_input(cfg, n, "cuda", gap_fn=gap_fn_for(L))
    layer = MoeLayer(lw, n)
    out, idx, w = layer.forward(x)
    rows = [0] if n == 1 else [0, n // 2, n - 1]
    ref, ridx, _, _ = O.moe_forward(L, bf16_bits(x), rows=rows)
    assert np.array_equal(idx.cpu().numpy()[rows], ridx)
    close(out.float().cpu().numpy()[rows], ref)
    assert layer.device_error() == 0


@gpu
@pytest.mark.parametrize("n", [1, 9])
def test_infinite_act_beside_large_ones(lib, n):
    """SiLU(g) u past fp32's range, of finite g and u, beside values past fp16's: an output is an infinity of its
    weight's sign and the product's, or NaN where the weight is 0."""
    cfg = cfg_of("int4_g32", shared_inter=0, top_k=1)
    lw = synth.make_weights(cfg, "cuda")
    x = synth.make_input(cfg, n, "cuda") * 2.0 ** 13
    xe = O.bf16_decode(bf16_bits(x))
    L = int4_oracle_layer(lw)
    gs, us = lw.gate.scale.float(), lw.up.scale.float()
    for t in range(n):                                    # row 5 of the token's expert: g about 1e29 and positive
        gs[t, 5] *= 2.0 ** 85 * float(np.sign(L.gate.expert(t)[5] @ xe[t]))
        us[t, 5] *= 2.0 ** 85
    lw.gate = dataclasses.replace(lw.gate, scale=gs.to(torch.bfloat16))
    lw.up = dataclasses.replace(lw.up, scale=us.to(torch.bfloat16))
    L = int4_oracle_layer(lw)
    idx, w = torch.arange(n, dtype=torch.int32, device="cuda")[:, None], torch.ones(n, 1, device="cuda")
    got = MoeLayer(lw, n).experts(x, idx, w).float().cpu().numpy()
    for t in range(n):
        g, u = L.gate.expert(t) @ xe[t], L.up.expert(t) @ xe[t]
        # No fp32 sum of g or u overflows, and only act 5 does.
        assert max(np.abs(L.gate.expert(t)[5]) @ np.abs(xe[t]), np.abs(L.up.expert(t)[5]) @ np.abs(xe[t])) < 1e37
        rest = np.delete(g * u, 5)
        assert g[5] > 0 and abs(g[5] * u[5]) > 1e40 and 1e5 < np.max(np.abs(rest)) < 1e30
        d = L.down.expert(t)[:, 5]
        want = np.full(len(d), np.nan, np.float32)
        want[d != 0] = np.inf * np.sign(d[d != 0]) * np.sign(u[5])
        assert np.array_equal(got[t], want, equal_nan=True)


def experts_ref(lw, x, idx, w):
    """The routed experts' (and an ungated shared one's) output in 64 bits for given routes."""
    L, xe = int4_oracle_layer(lw), O.bf16_decode(bf16_bits(x))
    ref = np.zeros((len(xe), lw.cfg.hidden))
    if lw.sh_gate is not None:
        ref += O.swiglu_mlp(xe, L.sh_gate.expert(0), L.sh_up.expert(0), L.sh_down.expert(0))
    for t in range(len(xe)):
        for j in range(idx.shape[1]):
            e = int(idx[t, j])
            ref[t] += float(w[t, j]) * O.swiglu_mlp(xe[t], L.gate.expert(e), L.up.expert(e), L.down.expert(e))
    return ref


def routes(n, k=2, E=16):
    g = torch.Generator().manual_seed(n)
    return torch.randint(0, E, (n, k), generator=g).to(torch.int32).cuda(), torch.rand(n, k, generator=g).cuda()


@gpu
@pytest.mark.parametrize("path,n", [("grouped", 1), ("grouped", 9), ("auto", 170)])
@pytest.mark.parametrize("shared", [0, 128])
def test_act_past_f16_on_the_grouped_path(lib, path, n, shared):
    """SiLU(g) u that f16 would hold as zero or infinity, with x and the scales inside its range."""
    cfg = cfg_of("int4_g64", shared_inter=shared, zero_points=True)
    lw = synth.make_weights(cfg, "cuda")
    for scale in (2.0 ** -10, 2.0 ** 13):
        x = synth.make_input(cfg, n, "cuda") * scale
        idx, w = routes(n)
        layer = MoeLayer(lw, n, path)
        got, ref = layer.experts(x, idx, w).float().cpu().numpy(), experts_ref(lw, x, idx, w)
        for t in range(n):
            close(got[t], ref[t])
        assert layer.device_error() == 0


@gpu
@pytest.mark.parametrize("n,path", [(1, "grouped"), (2, "grouped"), (40, "grouped"), (170, "auto")])
def test_a_workspace_of_the_grouped_path(lib, n, path):
    """A workspace of exactly moe_workspace_bytes in front of a guard: nothing past its end is written; one made for
    more tokens serves fewer, on whichever path they run."""
    cfg = cfg_of("int4_g32", inter=160, shared_inter=96, zero_points=True)
    lw, x, layer, out, idx, w = check(cfg, n, path)
    size = B.moe_workspace_bytes(layer.c_cfg, n)
    buf = torch.zeros(size + 4096, dtype=torch.uint8, device="cuda")
    buf[size:] = 0xA5
    got = torch.empty_like(out)
    assert B.moe_forward(layer.c_cfg, layer.c_w, x, n, got, torch.empty_like(idx), torch.empty_like(w), buf, size) == B.MOE_OK
    torch.cuda.synchronize()
    assert torch.equal(got, out) and (buf[size:] == 0xA5).all()
    for m in range(1, n, max(1, n // 7)):
        assert B.moe_workspace_bytes(layer.c_cfg, m) <= size
        assert B.moe_forward(layer.c_cfg, layer.c_w, x, m, got, None, None, buf, size) == B.MOE_OK
        torch.cuda.synchronize()
        if path == "grouped":
            assert torch.equal(got[:m], out[:m])
    assert (buf[size:] == 0xA5).all() and B.moe_workspace_check(buf, size) == (B.MOE_OK, 0)


@gpu
@pytest.mark.parametrize("path,n", [("grouped", 1), ("grouped", 9), ("auto", 170)])
@pytest.mark.parametrize("norm", [False, True])
def test_inputs_past_f16_on_the_grouped_path(lib, path, n, norm):
    """Rows of x that f16 would hold as zero or infinity, beside ordinary ones."""
    cfg = cfg_of("int4_g64", pre_expert_norm=norm)
    for scale in (2.0 ** -40, 2.0 ** -14, 2.0 ** 14, 2.0 ** 40):
        lw = synth.make_weights(cfg, "cuda")
        x = synth.make_input(cfg, n, "cuda")
        if norm:
            lw.pre_expert_norm_w = (lw.pre_expert_norm_w.float() * scale).to(torch.bfloat16)
            xe = x.float() * torch.rsqrt((x.float() ** 2).mean(1, keepdim=True) + cfg.rms_norm_eps)
            xr = (xe * lw.pre_expert_norm_w.float()).to(torch.bfloat16)
        else:
            x[::2] *= scale
            xr = x
        idx, w = routes(n)
        layer = MoeLayer(lw, n, path)
        got, ref = layer.experts(x, idx, w).float().cpu().numpy(), experts_ref(lw, xr, idx, w)
        for t in range(n):
            close(got[t], ref[t], norm)
        assert layer.device_error() == 0


@gpu
@pytest.mark.parametrize("path", ["auto", "grouped"])
def test_infinite_and_nan_inputs(lib, path):
    """An infinity stays one, and reaches only its own token, on either path."""
    cfg = cfg_of("int4_g32", shared_inter=0)
    lw = synth.make_weights(cfg, "cuda")
    x = synth.make_input(cfg, 9, "cuda")
    idx, w = routes(9)
    layer = MoeLayer(lw, 9, path)
    want = layer.experts(x, idx, w)
    y = x.clone()
    y[4, 3], y[6, 200] = float("nan"), float("inf")
    got = layer.experts(y, idx, w)
    rest = [0, 1, 2, 3, 5, 7, 8]
    assert torch.equal(got[rest], want[rest])
    assert torch.isnan(got[4]).all() and not torch.isfinite(got[6]).any()


def scaled(q, factor):
    return dataclasses.replace(q, scale=(q.scale.float() * factor).to(torch.bfloat16))


@gpu
@pytest.mark.parametrize("path,n", [("grouped", 1), ("grouped", 9), ("auto", 170)])
@pytest.mark.parametrize("zero", [False, True])
@pytest.mark.parametrize("gate,up,down", [
    (1.0, 2.0 ** -24, 1.0), (1.0, 2.0 ** 30, 2.0 ** -30), (1.0, 2.0 ** -40, 2.0 ** 40), (1.0, 1.0, 2.0 ** 24),
    (2.0 ** -30, 2.0 ** 30, 1.0)])
def test_scales_far_from_one(lib, path, n, zero, gate, up, down):
    """Group scales that f16 would hold as zero or infinity, on the grouped path (past 160 tokens of this layer AUTO's)."""
    cfg = cfg_of("int4_g32", zero_points=zero)
    lw = synth.make_weights(cfg, "cuda")
    for m, f in (("gate", gate), ("up", up), ("down", down)):
        setattr(lw, m, scaled(getattr(lw, m), f))
        setattr(lw, "sh_" + m, scaled(getattr(lw, "sh_" + m), f))
    x = synth.make_input(cfg, n, "cuda")
    idx, w = routes(n)
    layer = MoeLayer(lw, n, path)
    out = layer.experts(x, idx, w)
    close(out.float().cpu().numpy(), experts_ref(lw, x, idx, w))
    assert layer.device_error() == 0


@gpu
@pytest.mark.parametrize("path", ["auto", "grouped"])
def test_scales_apart_in_a_row(lib, path):
    """Groups of one row whose scales are 2^16 apart: the small ones count where x is small beside the large."""
    cfg = cfg_of("int4_g32", shared_inter=0)
    lw = synth.make_weights(cfg, "cuda")
    s = lw.up.scale.float()
    s[..., 1::2] *= 2.0 ** -16
    lw.up = dataclasses.replace(lw.up, scale=s.to(torch.bfloat16))
    x = synth.make_input(cfg, 12, "cuda").view(12, -1, 2, 32).clone()
    x[:, :, 0] *= 2.0 ** -10
    x[:, :, 1] *= 2.0 ** 6
    x = x.view(12, -1)
    idx, w = routes(12)
    close(MoeLayer(lw, 12, path).experts(x, idx, w).float().cpu().numpy(), experts_ref(lw, x, idx, w))


@gpu
@pytest.mark.parametrize("zero", [False, True])
def test_expert_parallel_on_the_grouped_path(lib, zero):
    """Ranks that hold some experts, none, or all but the shared one, with scales far from one."""
    n, cfg = 9, cfg_of("int4_g32", zero_points=zero, shared_gate=True)
    lw = synth.make_weights(cfg, "cuda")
    for m in ("up", "sh_up"):
        setattr(lw, m, scaled(getattr(lw, m), 2.0 ** 30))
    L = int4_oracle_layer(lw)
    x = synth.make_input(cfg, n, "cuda", gap_fn=gap_fn_for(L))
    for r in ((0, 5), (5, 16), (7, 8)):
        layer = MoeLayer(synth.expert_slice(lw, *r), n, "grouped", experts=r, exclude_shared=True)
        out, _, _ = layer.forward(x)
        ref, _, _, _ = O.moe_forward(L, bf16_bits(x), experts=r, include_shared=False)
        got = out.float().cpu().numpy()
        close(got, ref) if np.any(ref) else np.testing.assert_array_equal(got, 0)
        assert layer.device_error() == 0
    layer = MoeLayer(synth.expert_slice(lw, 16, 16), n, "grouped", experts=(16, 16), accumulate=True)
    out = torch.zeros(n, cfg.hidden, dtype=torch.bfloat16, device="cuda")
    layer.forward(x, out=out, routing=False)
    close(out.float().cpu().numpy(), O.moe_forward(L, bf16_bits(x), experts=(0, 0))[0])
    assert layer.device_error() == 0


@gpu
@pytest.mark.parametrize("path,n", [("auto", 3), ("auto", 20), ("grouped", 20), ("token_major", 2)])
@pytest.mark.parametrize("hidden,inter", [(256, 128), (512, 256), (96, 160)])
def test_scales_at_a_4_byte_offset(lib, path, n, hidden, inter):
    """Scale arrays that are aligned to 4 bytes alone: the same bits."""
    cfg = cfg_of("int4_g32", hidden=hidden, inter=inter, shared_inter=inter)
    lw = synth.make_weights(cfg, "cuda")
    x = synth.make_input(cfg, n, "cuda")
    idx, w = routes(n)
    want = MoeLayer(lw, n, path).experts(x, idx, w)
    for m in ("gate", "up", "down", "sh_gate", "sh_up", "sh_down"):
        q = getattr(lw, m)
        buf = torch.empty(q.scale.numel() + 2, dtype=torch.bfloat16, device="cuda")
        moved = buf[2:].view(q.scale.shape)
        moved.copy_(q.scale)
        assert moved.data_ptr() % 16 == 4
        setattr(lw, m, dataclasses.replace(q, scale=moved))
    assert torch.equal(MoeLayer(lw, n, path).experts(x, idx, w), want)


@gpu
def test_experts_without_tokens_on_the_grouped_path(lib):
    """NaN and infinite scales of experts that no token chose reach nothing, and those of one that some chose, those."""
    cfg = cfg_of("int4_g32", shared_inter=0)
    lw = synth.make_weights(cfg, "cuda")
    x = synth.make_input(cfg, 9, "cuda")
    idx, w = torch.tensor([[1, 4]] * 8 + [[4, 9]], dtype=torch.int32, device="cuda"), torch.ones(9, 2, device="cuda")
    want = MoeLayer(lw, 9, "grouped").experts(x, idx, w)
    s = lw.up.scale.clone()
    s[[0, 2, 3, 5]] = float("nan")
    s[9, :, 0] = float("inf")
    lw.up = dataclasses.replace(lw.up, scale=s)
    got = MoeLayer(lw, 9, "grouped").experts(x, idx, w)
    assert torch.equal(got[:8], want[:8]) and not torch.isfinite(got[8]).any()


@gpu
def test_infinite_act_on_the_grouped_path(lib):
    """One value of SiLU(g) u past fp32's range beside values past fp16's, one expert and one row of down's each: the
    infinity's sign, or NaN where its weight is 0."""
    cfg = cfg_of("int4_g32", shared_inter=0, top_k=1)
    lw = synth.make_weights(cfg, "cuda")
    n = 9
    x = synth.make_input(cfg, n, "cuda") * 2.0 ** 13
    xe = O.bf16_decode(bf16_bits(x))
    L = int4_oracle_layer(lw)
    gs, us = lw.gate.scale.float(), lw.up.scale.float()
    for t in range(n):
        gs[t, 5] *= 2.0 ** 85 * float(np.sign(L.gate.expert(t)[5] @ xe[t]))
        us[t, 5] *= 2.0 ** 85
    lw.gate = dataclasses.replace(lw.gate, scale=gs.to(torch.bfloat16))
    lw.up = dataclasses.replace(lw.up, scale=us.to(torch.bfloat16))
    L = int4_oracle_layer(lw)
    idx, w = torch.arange(n, dtype=torch.int32, device="cuda")[:, None], torch.ones(n, 1, device="cuda")
    got = MoeLayer(lw, n, "grouped").experts(x, idx, w).float().cpu().numpy()
    for t in range(n):
        d, u5 = L.down.expert(t)[:, 5], float(L.up.expert(t)[5] @ xe[t])
        want = np.full(len(d), np.nan, np.float32)
        want[d != 0] = np.inf * np.sign(d[d != 0]) * np.sign(u5)
        assert np.array_equal(got[t], want, equal_nan=True)


@gpu
@pytest.mark.parametrize("n", [9, 170])
def test_the_grouped_path_captured_and_replayed(lib, n):
    """In a graph, replayed on inputs of other magnitudes, between layers that share the weights."""
    cfg = cfg_of("int4_g64", zero_points=True)
    lw = synth.make_weights(cfg, "cuda")
    xs = [synth.make_input(cfg, n, "cuda", stream=s) * f for s, f in ((0, 1.0), (1, 2.0 ** 20), (2, 2.0 ** -20))]
    a, b = MoeLayer(lw, n, "grouped"), MoeLayer(lw, n, "grouped")
    want = [a.forward(x)[0].clone() for x in xs]
    buf, oa, ob = xs[0].clone(), torch.empty_like(want[0]), torch.empty_like(want[0])
    b.forward(buf, out=ob)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a.forward(buf, out=oa)
        b.forward(buf, out=ob)
    for x, r in zip(xs, want):
        buf.copy_(x)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(oa, r) and torch.equal(ob, r)
