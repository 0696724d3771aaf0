"""The Python holders' calls: what they take, what they refuse, the memory and the streams they use."""

import dataclasses
import gc
import weakref

import pytest
import torch

from mixture_experts_decode_router_gb300 import binding as B
from mixture_experts_decode_router_gb300 import synth
from mixture_experts_decode_router_gb300.layer import MoeLayer, MoeMatvec, MoeTopk

gpu = pytest.mark.gpu


def cfg_of(fmt="int4_g32", **kw):
    d = dict(name="holders", hidden=128, num_experts=8, top_k=2, inter=64, shared_inter=64,
             routing=synth.ROUTE_SOFTMAX, norm_topk_prob=True, routed_scaling_factor=1.0, expert_fmt=fmt, n_tokens=3)
    d.update(kw)
    return synth.LayerConfig(**d)


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    B.load()


# ---------------------------------------------------------------- the layer's tensors

def refusals_of_a_layer(dev):
    """Every tensor that moe_experts or moe_forward would read or write as something else."""
    layer = MoeLayer(synth.make_weights(cfg_of(), dev), 3)
    def t(shape, dtype):
        return torch.zeros(shape, dtype=dtype, device=dev)
    x, idx, w = t((3, 128), torch.bfloat16), t((3, 2), torch.int32), t((3, 2), torch.float32)
    xs = [x.half(), x.float(), x[:, :64], x[:, :64].contiguous(), t((3, 256), torch.bfloat16)[:, ::2], x[0],
          t((128, 3), torch.bfloat16).T, torch.zeros((), dtype=torch.bfloat16, device=dev)]
    routes = [idx.long(), w, idx[:2], idx[:, :1], t((3, 1), torch.int32), t((3, 4), torch.int32)[:, ::2], t((2, 3), torch.int32),
              t((3, 3), torch.int32), t((5,), torch.int32)]
    weights = [w.double(), idx, w.half(), w[:2], w[:, :1], t((3, 4), torch.float32)[:, ::2], t((3, 3), torch.float32)]
    outs = [x.float(), x[:2], t((3, 256), torch.bfloat16)[:, ::2], x[:, :64].contiguous()]
    for bad in xs:
        with pytest.raises(ValueError):
            layer.experts(bad, idx, w)
        with pytest.raises(ValueError):
            layer.forward(bad)
    for bad in routes:
        with pytest.raises(ValueError):
            layer.experts(x, bad, w)
        with pytest.raises(ValueError):
            layer.forward(x, idx=bad)
    for bad in weights:
        with pytest.raises(ValueError):
            layer.experts(x, idx, bad)
        with pytest.raises(ValueError):
            layer.forward(x, w=bad)
    for bad in outs:
        with pytest.raises(ValueError):
            layer.forward(x, out=bad)
    for bad in (None, 3, [[0.0] * 128]):
        with pytest.raises(TypeError):
            layer.forward(bad)
    return layer, x, idx, w


def test_layer_refusals():
    """On the CPU, where nothing can run: a ValueError of the call, before the library is called."""
    layer, x, idx, w = refusals_of_a_layer("cpu")
    with pytest.raises(ValueError):
        layer.experts(x, idx, w)               # nothing of this is on a GPU
    with pytest.raises(ValueError):
        layer.forward(x)


@gpu
def test_layer_refusals_on_the_gpu(lib):
    layer, x, idx, w = refusals_of_a_layer("cuda")
    for kw in (dict(idx=idx.cpu()), dict(w=w.cpu()), dict(out=x.cpu()), dict(idx=idx.cpu().pin_memory())):
        with pytest.raises(ValueError):
            layer.forward(x, **kw)
    with pytest.raises(ValueError):
        layer.experts(x, idx.cpu(), w)
    assert layer.device_error() == 0


@gpu
@pytest.mark.parametrize("fmt", ["bf16", "fp8_b128", "nvfp4", "int4_g32"])
def test_forms_that_hold_the_same_elements(lib, fmt):
    """Larger buffers, flat routes, and x of more than two dimensions are taken as before."""
    cfg = cfg_of(fmt)
    lw = synth.make_weights(cfg, "cuda")
    layer, x = MoeLayer(lw, 3), synth.make_input(cfg, 3, "cuda")
    out, idx, w = layer.forward(x)
    assert torch.equal(layer.experts(x.view(3, 1, 128), idx.view(-1), w.view(-1)), layer.experts(x, idx, w))
    big = torch.zeros(5, 128, dtype=torch.bfloat16, device="cuda")
    bi, bw = torch.zeros(5, 2, dtype=torch.int32, device="cuda"), torch.zeros(5, 2, device="cuda")
    layer.forward(x, out=big, idx=bi, w=bw)
    assert torch.equal(big[:3], out) and torch.equal(bi[:3], idx) and torch.equal(bw[:3], w)
    assert not big[3:].any() and not bi[3:].any() and not bw[3:].any()
    # One row of a wider matrix is contiguous.
    wide = torch.zeros(1, 200, dtype=torch.bfloat16, device="cuda")
    wide[:, :128] = x[:1]
    assert torch.equal(layer.forward(wide[:, :128])[0], layer.forward(x[:1])[0])
    assert layer.forward(x[:0])[0].shape == (0, 128)


@gpu
@pytest.mark.parametrize("fmt", ["bf16", "int4_g32"])
def test_addresses_of_outputs_and_routes(lib, fmt):
    """out, idx and w may be device addresses, as the C functions take them; they come back as they were given."""
    cfg = cfg_of(fmt)
    layer = MoeLayer(synth.make_weights(cfg, "cuda"), 3)
    x = synth.make_input(cfg, 3, "cuda")
    out, idx, w = layer.forward(x)
    o2, i2, w2 = torch.zeros_like(out), torch.zeros_like(idx), torch.zeros_like(w)
    got = layer.forward(x, out=o2.data_ptr(), idx=i2.data_ptr(), w=w2.data_ptr())
    assert got == (o2.data_ptr(), i2.data_ptr(), w2.data_ptr())
    assert torch.equal(o2, out) and torch.equal(i2, idx) and torch.equal(w2, w)
    assert torch.equal(layer.experts(x, idx.data_ptr(), w.data_ptr()), layer.experts(x, idx, w))


def test_what_is_neither_a_tensor_nor_an_address():
    layer = MoeLayer(synth.make_weights(cfg_of(), "cpu"), 3)
    x = torch.zeros(3, 128, dtype=torch.bfloat16)
    for bad in ("idx", 1.5, [0], True):
        with pytest.raises((TypeError, ValueError)):
            layer.forward(x, idx=bad)
        with pytest.raises((TypeError, ValueError)):
            layer.experts(x, bad, bad)


@gpu
@pytest.mark.parametrize("fmt", ["bf16", "int4_g32"])
@pytest.mark.parametrize("n", [1, 3])
def test_pinned_x_without_outputs(lib, fmt, n):
    """What a call with x in pinned memory returns is on the current GPU."""
    cfg = cfg_of(fmt)
    layer = MoeLayer(synth.make_weights(cfg, "cuda"), n)
    x = synth.make_input(cfg, n, "cuda")
    want = layer.forward(x)
    host = x.cpu().pin_memory()
    for got, ref in zip(layer.forward(host), want):
        assert got.is_cuda and torch.equal(got, ref)
    assert torch.equal(layer.experts(host, *want[1:]), layer.experts(x, *want[1:]))
    torch.cuda.synchronize()


def test_experts_of_an_accumulating_layer():
    """There is nothing to add to: refused (the output would be added to what its memory held)."""
    layer = MoeLayer(synth.make_weights(cfg_of(), "cpu"), 3, accumulate=True)
    x, idx, w = torch.zeros(3, 128, dtype=torch.bfloat16), torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, 2)
    with pytest.raises(ValueError, match="accumulate"):
        layer.experts(x, idx, w)
    with pytest.raises(ValueError, match="accumulate"):
        layer.forward(x)


# ---------------------------------------------------------------- what the holders hold

@gpu
@pytest.mark.parametrize("fmt", ["bf16", "int4_g32"])
@pytest.mark.parametrize("n", [1, 3])
def test_a_new_workspace_config_or_weights(lib, fmt, n):
    """A workspace, config or weight struct assigned after construction is the one that the next call uses."""
    cfg = cfg_of(fmt)
    a, b = (synth.make_weights(cfg.with_(seed=s), "cuda") for s in (1, 2))
    layer, other, x = MoeLayer(a, n), MoeLayer(b, n), synth.make_input(cfg, n, "cuda")
    want = layer.forward(x)
    old = layer.ws
    layer.ws = torch.zeros_like(old)
    old.zero_()
    assert torch.equal(layer.forward(x)[0], want[0])
    assert not old.any() and layer.ws.any()
    was = layer.c_cfg, layer.c_w                            # (held: the calls before could read them still)
    layer.c_cfg = type(was[0]).from_buffer_copy(was[0])
    layer.c_cfg.routed_scaling_factor = 2.0
    assert torch.equal(layer.forward(x)[2], 2 * want[2])
    layer.c_cfg, layer.c_w = was[0], other.c_w
    assert torch.equal(layer.forward(x)[0], other.forward(x)[0])
    layer.c_w = was[1]
    assert torch.equal(layer.forward(x)[0], want[0])


@gpu
def test_a_new_workspace_of_another_size(lib):
    cfg = cfg_of()
    layer, x = MoeLayer(synth.make_weights(cfg, "cuda"), 3), synth.make_input(cfg, 3, "cuda")
    for bad in (torch.zeros(16, dtype=torch.uint8, device="cuda"), layer.ws.cpu(), torch.zeros(2 * layer.ws_bytes, dtype=torch.uint8, device="cuda")[::2]):
        good, layer.ws = layer.ws, bad
        with pytest.raises(ValueError):
            layer.forward(x)
        layer.ws = good
    layer.forward(x)
    assert layer.device_error() == 0


def test_a_matrix_keeps_what_it_points_to():
    """The weights and the bias are those of construction: assigning others would leave the struct's addresses behind."""
    w, s, _ = synth.quant_int4(torch.randn(16, 64), 32)
    q = synth.QMatT("int4_g32", w, s)
    op = MoeMatvec(q, bias=torch.zeros(16))
    assert op.weights is q and op.bias.shape == (16,)
    for name in ("weights", "bias"):
        with pytest.raises(AttributeError):
            setattr(op, name, None)
    at, held = op.c_w.scale, s.data_ptr()
    q.scale = torch.zeros_like(s)          # the tensors that the struct points to live on
    del s
    assert at == held and any(t is not None and t.data_ptr() == at for t in op._held[2])


def test_a_bias_assigned_later_is_checked():
    op = MoeTopk(8, 2, "sigmoid", torch.zeros(8))
    for bad in (torch.zeros(7), torch.zeros(8, dtype=torch.float64), torch.zeros(16)[::2], torch.zeros(8, 1)):
        op.bias = bad
        with pytest.raises(ValueError, match="bias is contiguous"):
            op.forward(torch.zeros(3, 8))      # (before what says that the logits are on no GPU)


# ---------------------------------------------------------------- a stream given by argument

def calls_on_a_stream():
    """name -> (call of a stream or None, its first output's shape and type)."""
    cfg = cfg_of(hidden=1024, n_tokens=64)
    layer = MoeLayer(synth.make_weights(cfg, "cuda"), 64)
    x = synth.make_input(cfg, 64, "cuda")
    _, idx, w = layer.forward(x)
    q, s, _ = synth.quant_int4(torch.randn(1024, 1024, device="cuda"), 32)
    lg = torch.randn(64, 8, device="cuda")
    mv, tk = MoeMatvec(synth.QMatT("int4_g32", q, s)), MoeTopk(8, 2)
    out, pair = ((64, 1024), torch.bfloat16), ((64, 2), torch.int32)
    return {"forward": (lambda st: layer.forward(x, stream=st), out), "experts": (lambda st: (layer.experts(x, idx, w, stream=st),), out),
            "route": (lambda st: layer.route(x, stream=st), pair), "topk": (lambda st: tk.forward(lg, stream=st), pair),
            "matvec": (lambda st: (mv.forward(x, stream=st),), out)}


CALLS = ["forward", "experts", "route", "topk", "matvec"]


@gpu
@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("raw", [False, True])
def test_outputs_of_another_stream(lib, name, raw):
    """Outputs of a call on another stream are that stream's memory: dropped while it runs, they are not handed out on
    the current stream; dropped while the current stream reads them, not on the other."""
    call, (shape, dtype) = calls_on_a_stream()[name]
    want = call(None)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    given = st.cuda_stream if raw else st
    got = call(given)
    torch.cuda.current_stream().wait_stream(st)
    assert all(torch.equal(g, r) for g, r in zip(got, want))
    at = {t.data_ptr() for t in call(given)}                # dropped at once
    assert not at & {torch.empty(shape, dtype=dtype, device="cuda").data_ptr() for _ in range(3)}
    torch.cuda.synchronize()
    got = call(given)
    torch.cuda.current_stream().wait_stream(st)
    torch.cuda._sleep(40_000_000)                           # 20 ms
    kept = got[0].clone()
    at = got[0].data_ptr()
    del got
    with torch.cuda.stream(st):
        assert torch.empty(shape, dtype=dtype, device="cuda").data_ptr() != at
    torch.cuda.synchronize()
    assert torch.equal(kept, want[0])
    # The current stream, given by name, is no other stream.
    assert all(torch.equal(g, r) for g, r in zip(call(torch.cuda.current_stream()), want))


# ---------------------------------------------------------------- weights

def bad_int4(q):
    """Arrays that the int4_g32 kernels would read past, or as something else."""
    s, z = q.scale, torch.zeros(q.scale.shape, dtype=torch.uint8)
    return [dict(scale=s[..., :1].contiguous()), dict(scale=s.half()), dict(scale=s.float()), dict(scale=None),
            dict(scale=s[..., :1, :].contiguous()), dict(scale=s.transpose(-1, -2).contiguous().transpose(-1, -2)),
            dict(zero=z[..., :1].contiguous()), dict(zero=z.to(torch.int32)), dict(zero=z.to(torch.bfloat16)),
            dict(scale2=torch.ones(1)), dict(w=q.w.view(torch.int32)), dict(w=q.w.to(torch.int16)), dict(fmt="int4_g64"),
            dict(fmt="int4_g128")]


def test_a_matrix_of_other_arrays():
    w, s, z = synth.quant_int4(torch.randn(16, 128), 32, True)
    good = synth.QMatT("int4_g32", w, s, zero=z)
    for q in (good, dataclasses.replace(good, zero=None), dataclasses.replace(good, w=w.view(torch.int8), zero=z.view(torch.int8)),
              synth.QMatT("int4_g32", w[None], s[None], zero=z[None])):
        MoeMatvec(q)
    for bad in bad_int4(good):
        with pytest.raises(ValueError):
            MoeMatvec(dataclasses.replace(good, **bad))
    b, f = torch.zeros(16, 64, dtype=torch.uint8), torch.zeros(16, 8, dtype=torch.uint8)
    nv = synth.QMatT("nvfp4", b, f, torch.ones(1))
    for q in (nv, dataclasses.replace(nv, scale=f.view(torch.float8_e4m3fn)), dataclasses.replace(nv, scale2=torch.tensor(1.0))):
        MoeMatvec(q)
    for bad in (dict(scale=f[:, :4].contiguous()), dict(scale=f.to(torch.bfloat16)), dict(scale2=None), dict(scale2=torch.ones(16)),
                dict(scale2=torch.ones(1, dtype=torch.float64)), dict(zero=f), dict(scale=None), dict(w=b.to(torch.int32)),
                dict(scale=torch.zeros(16, 8, dtype=torch.float8_e5m2))):
        with pytest.raises(ValueError):
            MoeMatvec(dataclasses.replace(nv, **bad))


@pytest.mark.parametrize("name", ["gate", "down", "sh_up", "sh_down"])
def test_a_layer_of_other_arrays(name):
    """INT4 stacks whose arrays are not those of the layer's sizes, experts and format."""
    lw = synth.make_weights(cfg_of(zero_points=True), "cpu")
    good = getattr(lw, name)
    MoeLayer(lw, 3)
    fewer = [] if name.startswith("sh_") else [dict(w=good.w[:7], scale=good.scale[:7], zero=good.zero[:7])]
    for bad in bad_int4(good) + fewer:
        setattr(lw, name, dataclasses.replace(good, **bad))
        with pytest.raises(ValueError):
            MoeLayer(lw, 3)
    setattr(lw, name, None)
    with pytest.raises(ValueError):
        MoeLayer(lw, 3)


def test_a_layer_without_some_of_its_arrays():
    """What a call does not read is not asked for: no shared expert, none of the experts, one rank's slice."""
    lw = synth.make_weights(cfg_of(zero_points=True), "cpu")
    for held in ((0, 8), (2, 5), (8, 8)):
        MoeLayer(synth.expert_slice(lw, *held), 3, experts=held)
    with pytest.raises(ValueError):
        MoeLayer(synth.expert_slice(lw, 2, 5), 3, experts=(2, 6))
    none = synth.expert_slice(lw, 8, 8)
    none.gate = none.up = none.down = None
    MoeLayer(none, 3, experts=(8, 8))
    lw.sh_gate = lw.sh_up = lw.sh_down = None
    MoeLayer(lw, 3, exclude_shared=True)
    with pytest.raises(ValueError):
        MoeLayer(lw, 3)


def test_a_matrix_struct_by_position():
    """moe_qmat_t takes its addresses in order, as the C struct does, and by name."""
    q = B.moe_qmat_t(1 << 40, 2, 3)
    assert (q.w, q.scale, q.scale2, q.zero) == (1 << 40, 2, 3, 3)
    q = B.moe_qmat_t(w=1, zero=4)
    assert (q.w, q.scale, q.scale2, q.zero) == (1, None, 4, 4)
    q = B.moe_qmat_t()
    assert (q.w, q.scale, q.scale2, q.zero) == (None,) * 4
    w = B.moe_weights_t()
    w.gate = B.moe_qmat_t(5, 6, 7)
    assert (w.gate.w, w.gate.scale, w.gate.scale2) == (5, 6, 7)


@gpu
@pytest.mark.parametrize("name", CALLS)
def test_outputs_of_the_default_stream_from_another(lib, name):
    """stream=0 is the default stream: called from another, the outputs are the default stream's memory."""
    call, (shape, dtype) = calls_on_a_stream()[name]
    want = call(None)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        got = call(0)
        at = got[0].data_ptr()
    torch.cuda.synchronize()
    assert all(torch.equal(g, r) for g, r in zip(got, want))
    del got
    torch.cuda.synchronize()
    assert at in {t.data_ptr() for t in [torch.empty(shape, dtype=dtype, device="cuda") for _ in range(64)]}


# ---------------------------------------------------------------- moe_route

def test_route_refusals():
    """On the CPU: what moe_route would read as something else, or past its end, is refused before the library is called."""
    layer = MoeLayer(synth.make_weights(cfg_of(), "cpu"), 3)
    x = torch.zeros(3, 128, dtype=torch.bfloat16)
    for bad in (x.half(), x.float(), x[:, :64].contiguous(), torch.zeros(3, 256, dtype=torch.bfloat16)[:, ::2], x[0]):
        with pytest.raises(ValueError, match="contiguous bfloat16"):
            layer.route(bad)
    with pytest.raises(ValueError, match="on the current device"):
        layer.route(x)


@gpu
@pytest.mark.parametrize("n", [1, 3])
def test_route_of_pinned_x(lib, n):
    """Its outputs are on the layer's GPU, wherever x is."""
    cfg = cfg_of()
    layer = MoeLayer(synth.make_weights(cfg, "cuda"), n)
    x = synth.make_input(cfg, n, "cuda")
    for got, want in zip(layer.route(x.cpu().pin_memory()), layer.route(x)):
        assert got.is_cuda and torch.equal(got, want)
    torch.cuda.synchronize()
    with pytest.raises(ValueError):
        layer.route(x.cpu())


@gpu
@pytest.mark.parametrize("name", ["forward", "experts", "topk", "matvec"])
def test_a_forked_stream_in_a_capture(lib, name):
    """A call on a stream that joins the capture, its outputs made and some dropped there, replayed."""
    call, _ = calls_on_a_stream()[name]
    want = [t.clone() for t in call(None)]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        st.wait_stream(torch.cuda.current_stream())
        call(st)
        got = call(st)
        torch.cuda.current_stream().wait_stream(st)
    for _ in range(3):
        for t in got:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("fmt", ["bf16", "int4_g32"])
def test_a_layer_keeps_what_it_points_to(fmt):
    """Matrices replaced in the weights after construction: the ones that the struct points to live on."""
    lw = synth.make_weights(cfg_of(fmt, shared_gate=True, pre_expert_norm=True), "cpu")
    layer = MoeLayer(lw, 3)
    refs = [weakref.ref(t) for t in (lw.up.w, lw.sh_down.w, lw.router_w, lw.shared_gate_w, lw.pre_expert_norm_w)]
    lw.up = lw.sh_down = lw.router_w = lw.shared_gate_w = lw.pre_expert_norm_w = None
    gc.collect()
    assert all(r() is not None for r in refs)
    del layer
    gc.collect()
    assert all(r() is None for r in refs)
