"""moe_matvec: refusals (CPU), and products of 4-bit matrices against plain 64-bit numpy (GPU).

Tolerance, per element: half a step of the output's type (2^-8 bf16, 2^-11 fp16, 2^-24 fp32, of
the result), and the fp32 sums: a product passes at most 64 + K / 64 additions, each off by at
most 2^-23 of the partial sum, which sum |w x| bounds."""

import numpy as np
import pytest
import torch

from mixture_experts_decode_router_gb300 import binding as B
from mixture_experts_decode_router_gb300 import synth
from mixture_experts_decode_router_gb300.layer import MoeMatvec
from oracle import moe_oracle as O

FMTS = sorted(synth.INT4_GROUP) + ["nvfp4"]
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}

# ---------------------------------------------------------------- refusals, on the CPU

FAKE = 0x7f0000000000      # never dereferenced here


def _call(fmt=B.MOE_W_INT4_G64, out=64, inp=256, x_type=B.MOE_BF16, out_type=B.MOE_BF16, acc=0, w=FAKE, scale=FAKE,
          second=None, bias=None, x=FAKE, xs=256, n=2, y=FAKE + 0x100000, ys=64):
    c = B.moe_matvec_config_t(out, inp, fmt, x_type, out_type, acc)
    q = B.moe_qmat_t()
    q.w, q.scale, q.scale2 = w, scale, second
    return B.moe_matvec(c, q, bias, x, xs, n, y, ys, 0)


def test_refusals():
    bad = B.MOE_ERR_INVALID_CONFIG
    q = B.moe_qmat_t()
    assert B.moe_matvec(None, q, None, FAKE, 32, 1, FAKE, 32, 0) == B.MOE_ERR_NULL
    assert B.moe_matvec(B.moe_matvec_config_t(), None, None, FAKE, 32, 1, FAKE, 32, 0) == B.MOE_ERR_NULL
    assert _call(out=(1 << 28) + 1, ys=(1 << 28) + 1) == B.MOE_ERR_UNSUPPORTED
    assert _call(inp=57344 + 64, xs=57344 + 64) == B.MOE_ERR_UNSUPPORTED
    for kw in (dict(out=0), dict(inp=0), dict(inp=48, xs=48), dict(inp=96, xs=96), dict(fmt=6), dict(fmt=-1),
               dict(x_type=B.MOE_F32), dict(x_type=3), dict(out_type=3), dict(acc=2), dict(n=-1), dict(xs=255),
               dict(xs=248), dict(ys=63)):
        assert _call(**kw) == bad, kw
    for fmt in (B.MOE_W_BF16, B.MOE_W_FP8_B128):
        assert _call(fmt=fmt) == B.MOE_ERR_UNSUPPORTED
    for kw in (dict(w=None), dict(scale=None), dict(x=None), dict(y=None), dict(fmt=B.MOE_W_NVFP4)):
        assert _call(**kw) == B.MOE_ERR_NULL, kw
    for kw in (dict(w=FAKE + 8), dict(scale=FAKE + 2), dict(x=FAKE + 8), dict(xs=260), dict(y=FAKE + 0x100001),
               dict(out_type=B.MOE_F32, y=FAKE + 0x100002), dict(bias=FAKE + 2),
               dict(fmt=B.MOE_W_NVFP4, second=FAKE + 2)):
        assert _call(**kw) == B.MOE_ERR_ALIGNMENT, kw
    assert _call(y=FAKE + 512) == B.MOE_ERR_ALIAS          # inside x's second row
    assert _call(n=0, x=None, y=None) == B.MOE_OK
    assert _call() == B.MOE_ERR_HOST_MEMORY                # no device or pinned memory there


def test_holder_refusals():
    w, s, z = synth.quant_int4(torch.randn(16, 64), 32)
    q = synth.QMatT("int4_g32", w, s)
    with pytest.raises(ValueError):
        MoeMatvec(q, bias=torch.zeros(15))
    with pytest.raises(ValueError):
        MoeMatvec(synth.QMatT("int4_g32", torch.stack([w, w]), torch.stack([s, s])))
    op = MoeMatvec(q, accumulate=True)
    for bad in (torch.zeros(2, 32), torch.zeros(64), torch.zeros(64, 64).T):
        with pytest.raises(ValueError):
            op.forward(bad.to(torch.bfloat16))
    with pytest.raises(KeyError):
        op.forward(torch.zeros(2, 64))                     # fp32 x
    with pytest.raises(ValueError):
        op.forward(torch.zeros(2, 64, dtype=torch.bfloat16))   # not on the GPU


# ---------------------------------------------------------------- products, on the GPU

gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    B.load()


def matrix(out, inp, fmt, zero=False, seed=0):
    """(QMatT on the GPU, decoded float64) of random codes and scales."""
    rng = np.random.default_rng(seed)
    w = rng.integers(0, 256, (out, inp // 2), dtype=np.uint8)
    if fmt == "nvfp4":
        sc = rng.integers(0x28, 0x48, (out, inp // 16), dtype=np.uint8)
        s2 = 0.0173
        ref = O.dequant_nvfp4(w, sc, float(np.float32(s2)))
        return synth.QMatT(fmt, torch.tensor(w).cuda(), torch.tensor(sc).cuda(),
                           torch.tensor([s2], dtype=torch.float32).cuda()), ref
    G = synth.INT4_GROUP[fmt]
    sc = torch.tensor(rng.uniform(0.005, 0.02, (out, inp // G)) * rng.choice([-1, 1], (out, inp // G)), dtype=torch.bfloat16)
    z = rng.integers(0, 16, (out, inp // G), dtype=np.uint8) if zero else None
    ref = O.dequant_int4(w, sc.view(torch.int16).numpy().view(np.uint16), z, G)
    return synth.QMatT(fmt, torch.tensor(w).cuda(), sc.cuda(), zero=torch.tensor(z).cuda() if zero else None), ref


def close(y, x, w, bias=None, was=None):
    K = w.shape[1]
    xd = x.double().cpu().numpy()
    ref = xd @ w.T
    mag = np.abs(xd) @ np.abs(w).T
    for more in (bias, was):
        if more is not None:
            m = more.double().cpu().numpy()
            ref, mag = ref + m, mag + np.abs(m)
    err = np.abs(y.double().cpu().numpy() - ref)
    tol = HALF[y.dtype] * np.abs(ref) * (1 + 1e-3) + (64 + K / 64) * 2.0 ** -23 * mag
    if y.dtype == torch.float16:
        tol = tol + 2.0 ** -25                             # half a step of its subnormals
    assert np.all(err <= tol), f"{np.max(err - tol):.3e} over, at {np.unravel_index(np.argmax(err - tol), err.shape)}"


def rows(n, K, dtype=torch.bfloat16, seed=1, pad=0, spread=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(n, K + pad, generator=g, device="cuda") * spread).to(dtype)[:, :K]


@gpu
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("zero", [False, True])
@pytest.mark.parametrize("xt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("yt", [torch.bfloat16, torch.float16, torch.float32])
def test_types(lib, fmt, zero, xt, yt):
    if zero and fmt == "nvfp4":
        pytest.skip("NVFP4 has no zero points")
    q, w = matrix(96, 384, fmt, zero)
    for n in (1, 5):
        x = rows(n, 384, xt)
        close(MoeMatvec(q, out_dtype=yt).forward(x), x, w)


@gpu
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("out,K", [(1, 128), (7, 128), (16, 256), (17, 128), (33, 640), (129, 1152), (511, 2048),
                                   (2050, 384), (64, 7168), (5, 11008)])
@pytest.mark.parametrize("n", [1, 3, 8, 9])
def test_sizes(lib, fmt, out, K, n):
    q, w = matrix(out, K, fmt, fmt == "int4_g64", seed=out + K)
    x = rows(n, K, seed=n)
    close(MoeMatvec(q, out_dtype=torch.float32).forward(x), x, w)


@gpu
@pytest.mark.parametrize("K", [32, 64, 96, 160, 224, 288, 2080])
@pytest.mark.parametrize("fmt", ["int4_g32", "nvfp4"])
def test_short_and_ragged_reductions(lib, K, fmt):
    """Reductions that end inside a kernel's step."""
    q, w = matrix(50, K, fmt, fmt == "int4_g32", seed=K)
    for n in (1, 4, 16):
        x = rows(n, K, seed=n)
        close(MoeMatvec(q, out_dtype=torch.float32).forward(x), x, w)


@gpu
@pytest.mark.parametrize("n", [2, 7, 15, 16, 17, 31, 33, 64, 130])
def test_row_counts(lib, n):
    q, w = matrix(130, 512, "int4_g128")
    x = rows(n, 512, seed=n)
    y = MoeMatvec(q).forward(x)
    close(y, x, w)
    # A row's bits are those of a call with that row alone, and of any other order.
    op = MoeMatvec(q)
    for t in (0, n // 2, n - 1):
        assert torch.equal(op.forward(x[t:t + 1]), y[t:t + 1])
    p = torch.randperm(n, generator=torch.Generator().manual_seed(0)).cuda()
    assert torch.equal(op.forward(x[p].contiguous()), y[p])


@gpu
@pytest.mark.parametrize("yt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fmt", ["int4_g32", "nvfp4"])
def test_strides_bias_accumulate(lib, yt, fmt):
    q, w = matrix(75, 256, fmt)
    x = rows(6, 256, pad=24)
    b = torch.randn(75, device="cuda")
    buf = torch.randn(8, 91, device="cuda").to(yt)
    was = buf.clone()
    out = buf[1:7, 3:78]
    MoeMatvec(q, bias=b, out_dtype=yt, accumulate=True).forward(x, out=out)
    torch.cuda.synchronize()
    close(out, x, w, b, was[1:7, 3:78])
    buf[1:7, 3:78] = was[1:7, 3:78]
    assert torch.equal(buf, was)                            # nothing around the output is written
    close(MoeMatvec(q, bias=b, out_dtype=yt).forward(x), x, w, b)


@gpu
@pytest.mark.parametrize("fmt", FMTS)
def test_large_and_small_values(lib, fmt):
    """BF16 rows far outside fp16's range, next to ordinary ones; fp16 rows near its ends."""
    q, w = matrix(64, 512, fmt, fmt == "int4_g32")
    x = rows(5, 512)
    x = x * torch.tensor([1e30, 1e-30, 1.0, 1e5, 1e-6], device="cuda").to(torch.bfloat16)[:, None]
    y = MoeMatvec(q, out_dtype=torch.float32).forward(x)
    close(y, x, w)
    x = rows(2, 512, torch.float16) * torch.tensor([2e4, 1e-5], device="cuda").to(torch.float16)[:, None]
    close(MoeMatvec(q, out_dtype=torch.float32).forward(x.clamp(-6e4, 6e4)), x.clamp(-6e4, 6e4), w)


@gpu
@pytest.mark.parametrize("fmt", FMTS)
def test_special_values_stay_in_their_row(lib, fmt):
    q, w = matrix(40, 256, fmt)
    x = rows(10, 256)
    op = MoeMatvec(q, out_dtype=torch.float32)
    want = op.forward(x)
    y = x.clone()
    y[3, 17] = float("nan")
    y[5, 200] = float("inf")
    got = op.forward(y)
    keep = [0, 1, 2, 4, 6, 7, 8, 9]
    assert torch.equal(got[keep], want[keep])
    assert torch.isnan(got[3]).all()
    assert not torch.isfinite(got[5][torch.tensor(w[:, 200] != 0)]).any()


@gpu
@pytest.mark.parametrize("fmt", ["int4_g128", "nvfp4"])
@pytest.mark.parametrize("n", [1, 3, 12])
def test_the_longest_rows(lib, fmt, n):
    """Rows of x of which few fit in shared memory beside the kernel's rings."""
    for K in (16384, 57344):
        q, w = matrix(19, K, fmt)
        x = rows(n, K, seed=n)
        y = MoeMatvec(q, out_dtype=torch.float32).forward(x)
        close(y, x, w)
        assert torch.equal(MoeMatvec(q, out_dtype=torch.float32).forward(x[n - 1:]), y[n - 1:])


@gpu
def test_more_rows_than_a_grid_has(lib):
    """More rows of x than 65535 rows of blocks of eight or sixteen."""
    q, w = matrix(3, 32, "int4_g32")
    n = 65535 * 16 + 5
    x = rows(n, 32)
    y = MoeMatvec(q, out_dtype=torch.float32).forward(x)
    close(y, x, w)


@gpu
def test_two_streams_at_once(lib):
    qs = [matrix(300, 1024, f, seed=i)[0] for i, f in enumerate(("int4_g64", "nvfp4"))]
    ops, x = [MoeMatvec(q) for q in qs], rows(7, 1024)
    want = [op.forward(x).clone() for op in ops]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        got = []
        for st, op in zip(streams, ops):
            with torch.cuda.stream(st):
                got.append([op.forward(x) for _ in range(3)])
        torch.cuda.synchronize()
        assert all(torch.equal(y, r) for ys, r in zip(got, want) for y in ys)


@gpu
def test_weights_elsewhere(lib):
    w, s, _ = synth.quant_int4(torch.randn(16, 64), 32)
    x = rows(2, 64)
    with pytest.raises(ValueError):
        MoeMatvec(synth.QMatT("int4_g32", w, s)).forward(x)              # weights on the CPU
    with pytest.raises(ValueError):
        MoeMatvec(synth.QMatT("int4_g32", w.cuda(), s))
    with pytest.raises(ValueError):
        MoeMatvec(synth.QMatT("int4_g32", w.cuda(), s.cuda())).forward(x, out=torch.empty(2, 16, dtype=torch.bfloat16))


@gpu
def test_no_rows(lib):
    q, _ = matrix(16, 64, "int4_g32")
    assert MoeMatvec(q).forward(torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")).shape == (0, 16)


@gpu
def test_rows_past_32_bit_offsets(lib):
    """A matrix of more than 2^32 bytes' worth of codes would be large; strided rows of x and out
    pass 2^31 elements at little cost."""
    q, w = matrix(24, 64, "int4_g32")
    n, stride = 5, 1 << 29
    try:
        xb = torch.empty(n * stride, dtype=torch.bfloat16, device="cuda")
        yb = torch.empty(n * stride, dtype=torch.bfloat16, device="cuda")
    except torch.OutOfMemoryError:
        pytest.skip("needs 10.8 GB")
    x, y = xb.view(n, stride)[:, :64], yb.view(n, stride)[:, :24]
    x.copy_(rows(n, 64))
    MoeMatvec(q).forward(x, out=y)
    close(y.contiguous(), x.contiguous(), w)


@gpu
@pytest.mark.parametrize("n", [1, 6, 16])
def test_another_stream_replay_and_pinned(lib, n):
    q, w = matrix(200, 512, "int4_g64", True)
    op = MoeMatvec(q)
    xs = [rows(n, 512, seed=s).contiguous() for s in range(3)]
    want = [op.forward(x).clone() for x in xs]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        got = op.forward(xs[1])
    st.synchronize()
    assert torch.equal(got, want[1])
    buf, out = xs[0].clone(), torch.empty_like(want[0])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        op.forward(buf, out=out)
    for x, r in zip(xs, want):
        buf.copy_(x)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, r)
    host = xs[2].cpu().pin_memory()
    got = op.forward(host)
    torch.cuda.synchronize()
    assert torch.equal(got, want[2])


@gpu
def test_projection_before_the_layer(lib):
    """A run as a decoder makes it: a projection, then the layer's INT4 experts on its rows."""
    from mixture_experts_decode_router_gb300.layer import MoeLayer
    from tests.int4_helpers import int4_oracle_layer
    from tests.moe_helpers import bf16_bits
    from tests.test_int4_experts import cfg_of, close as close_layer
    q, w = matrix(256, 512, "int4_g128")
    x = rows(6, 512)
    h = MoeMatvec(q).forward(x)
    close(h, x, w)
    lw = synth.make_weights(cfg_of("int4_g64"), "cuda")
    out, idx, rw = MoeLayer(lw, 6).forward(h)
    L = int4_oracle_layer(lw)
    ref, ridx, _, _ = O.moe_forward(L, bf16_bits(h))
    assert np.array_equal(idx.cpu().numpy(), ridx)
    close_layer(out.float().cpu().numpy(), ref)


@gpu
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("n", [1, 5])
def test_infinity_beside_large_values(lib, fmt, n):
    """A row with an infinity and values past fp16's range: the infinity's sign, or NaN where its weight is 0."""
    q, w = matrix(70, 4096, fmt, seed=3)
    x = rows(n, 4096, spread=1e6)
    x[n - 1, 300] = float("inf")
    y = MoeMatvec(q, out_dtype=torch.float32).forward(x)
    at = w[:, 300]
    want = torch.tensor(np.where(at == 0, np.nan, np.sign(at) * np.inf), dtype=torch.float32, device="cuda")
    assert torch.equal(torch.isnan(y[n - 1]), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(y[n - 1]), torch.nan_to_num(want))
    close(y[:n - 1], x[:n - 1], w)
