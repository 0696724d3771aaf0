"""moe_norm: refusals (CPU), and residual addition with RMSNorm against plain 64-bit torch (GPU).

h is fp32's x + residual, rounded to the residual's type: exactly that.  y's relative error: a row's
squares are added in chains of at most 64, 5 shuffles and 16 warps, all terms positive (86 roundings,
halved by the root), and ten more roundings at most follow (the mean, eps, root, quotient, three
products, the weight's offset): 53 x 2^-24, taken as 64.  An output adds half a step of its type,
a scale two roundings.  A code is the E4M3 of some value that near to y / scale."""

import ctypes

import pytest
import torch

from mixture_experts_decode_router_gb300 import binding as B
from mixture_experts_decode_router_gb300.layer import MoeNorm

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
HALF = {BF: 2.0 ** -8, HF: 2.0 ** -11, F32: 2.0 ** -24}
TINY = {BF: 2.0 ** -134, HF: 2.0 ** -25, F32: 2.0 ** -150}      # half a step of the subnormals
REL = 64 * 2.0 ** -24

# ---------------------------------------------------------------- refusals, on the CPU

FAKE = 0x7f0000000000      # never dereferenced here
MB = 1 << 20


def _call(hidden=64, x_type=B.MOE_BF16, residual_type=B.MOE_BF16, weight_type=B.MOE_BF16, out_type=B.MOE_BF16, scale_group=128,
          eps=1e-6, offset=0.0, x=FAKE, xs=64, res=FAKE + MB, rs=64, w=FAKE + 2 * MB, n=2, ro=FAKE + 3 * MB, ros=64, out=FAKE + 4 * MB,
          ys=64, q=FAKE + 5 * MB, qs=64, scale=FAKE + 6 * MB):
    c = B.moe_norm_config_t(hidden, x_type, residual_type, weight_type, out_type, scale_group, eps, offset)
    return B.moe_norm(c, x, xs, res, rs, w, n, ro, ros, out, ys, q, qs, scale, 0)


def test_refusals():
    assert B.moe_norm(None, FAKE, 64, None, 64, None, 1, None, 64, FAKE + MB, 64, None, 64, None, 0) == B.MOE_ERR_NULL
    for kw in (dict(hidden=0), dict(n=-1), dict(x_type=3), dict(x_type=-1), dict(residual_type=B.MOE_F16), dict(residual_type=7),
               dict(weight_type=3), dict(out_type=3), dict(scale_group=64), dict(eps=-1e-6), dict(eps=float("nan")),
               dict(eps=float("inf")), dict(offset=float("inf")), dict(offset=float("nan")), dict(xs=63), dict(rs=0), dict(ros=63),
               dict(ys=-64), dict(qs=1), dict(res=None), dict(ys=1 << 41)):
        assert _call(**kw) == B.MOE_ERR_INVALID_CONFIG, kw
    assert _call(hidden=32769, xs=32769, rs=32769, ros=32769, ys=32769, qs=32769) == B.MOE_ERR_UNSUPPORTED
    for kw in (dict(x=None), dict(out=None, q=None), dict(scale=None)):
        assert _call(**kw) == B.MOE_ERR_NULL, kw
    for kw in (dict(x=FAKE + 1), dict(res=FAKE + MB + 1), dict(w=FAKE + 2 * MB + 1), dict(ro=FAKE + 3 * MB + 1), dict(out=FAKE + 4 * MB + 1),
               dict(scale=FAKE + 6 * MB + 2), dict(out_type=B.MOE_F32, out=FAKE + 4 * MB + 2)):
        assert _call(**kw) == B.MOE_ERR_ALIGNMENT, kw
    # Overlaps: x has 256 bytes, as residual and the outputs of 16 bits.
    for kw in (dict(out=FAKE + 254), dict(ro=FAKE), dict(ro=FAKE + MB + 2), dict(ro=FAKE + MB, ros=66), dict(out=FAKE + MB), dict(q=FAKE + 255),
               dict(q=FAKE + 4 * MB), dict(scale=FAKE + 3 * MB), dict(out=FAKE, x_type=B.MOE_F16, residual_type=B.MOE_F16),
               dict(out=FAKE + 2 * MB), dict(out=FAKE + 3 * MB), dict(scale=FAKE + 5 * MB + 124)):
        assert _call(**kw) == B.MOE_ERR_ALIAS, kw
    assert _call(n=0, x=None, out=None, q=None) == B.MOE_OK
    # What is left are the addresses themselves, which are none of CUDA's.
    for kw in (dict(), dict(ro=FAKE + MB), dict(out=FAKE), dict(res=None, ro=None, residual_type=9), dict(out=None, out_type=9),
               dict(q=None, scale=None, scale_group=9), dict(w=None, weight_type=9), dict(ro=None), dict(q=FAKE + 5 * MB + 3)):
        assert _call(**kw) == B.MOE_ERR_HOST_MEMORY, kw


def test_config_layout():
    assert ctypes.sizeof(B.moe_norm_config_t) == 32


def test_holder_refusals():
    w = torch.ones(64)
    for bad in (torch.ones(2, 64), torch.ones(64, dtype=torch.float64), torch.ones(128)[::2], None, 3):
        with pytest.raises(ValueError):
            MoeNorm(bad)
    for kw in (dict(out8="column"), dict(out_dtype=None)):
        with pytest.raises(ValueError):
            MoeNorm(w, **kw)
    op = MoeNorm(w, out8="group")
    x = torch.zeros(2, 64)
    for args in ((torch.zeros(2, 32),), (torch.zeros(64),), (torch.zeros(64, 64).T,), (x, torch.zeros(3, 64)), (x, x.half()),
                 (x, x, x.half()), (x, None, x), (x, None, None, x), (x, None, None, None, x), (x, None, None, None, None, x)):
        with pytest.raises(ValueError):
            op.forward(*args)
    with pytest.raises(KeyError):
        op.forward(x.double())
    with pytest.raises(ValueError):
        op.forward(x)                                       # not on the GPU
    with pytest.raises(TypeError):
        op.forward(None)


# ---------------------------------------------------------------- on the GPU

gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    B.load()


def rows(n, H, dtype=BF, seed=1, pad=0, spread=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(n, H + pad, generator=g, device="cuda") * spread).to(dtype)[:, :H]


def weights(H, dtype=BF, seed=9):
    return (1 + 0.3 * torch.randn(H, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")).to(dtype)


def e4m3(v):
    """To nearest even, magnitudes past 448 to it."""
    return v.clamp(-448, 448).float().to(torch.float8_e4m3fn).double()


def check(op, x, res, got, eps=1e-6, offset=0.0):
    """Everything that a call returned."""
    out, ro, q, s = got
    h = x.float()
    if res is not None:
        h = (h + res.float()).to(res.dtype)
        assert torch.equal(ro, h)
    else:
        assert ro is None
    h = h.double()
    y = h / torch.sqrt(h.square().mean(1, keepdim=True) + eps) * (op.weight.double() + offset)
    if op.out_dtype is None:
        assert out is None
    else:
        assert out.dtype == op.out_dtype and out.shape == x.shape
        err = (out.double() - y).abs()
        tol = y.abs() * (REL + HALF[op.out_dtype] * (1 + REL)) + TINY[op.out_dtype]
        assert bool((err <= tol).all()), float((err - tol).max())
    if op.out8 is None:
        assert q is None and s is None
        return
    n, H = x.shape
    size = 128 if op.out8 == "group" else H
    G = -(-H // size)
    assert q.dtype == torch.float8_e4m3fn and q.shape == x.shape and s.shape == (n, G)
    z = torch.zeros(n, G * size, dtype=torch.float64, device="cuda")
    z[:, :H] = y
    want = (z.view(n, G, size).abs().amax(2) / 448).clamp(min=2.0 ** -126)
    assert bool(((s.double() - want).abs() <= want * (REL + 2.0 ** -23)).all())
    by = s.double().repeat_interleave(size, 1)[:, :H]
    v, slack = (y / by).abs(), REL + 2 * 2.0 ** -24             # (the reciprocal and a product)
    qa = q.double().abs()
    assert bool((e4m3(v * (1 - slack)) <= qa).all()) and bool((qa <= e4m3(v * (1 + slack))).all())
    assert bool((q.double() * y >= 0).all())


@gpu
@pytest.mark.parametrize("x,r", [(BF, None), (BF, BF), (BF, F32), (HF, None), (HF, HF), (HF, F32), (F32, None), (F32, F32)])
@pytest.mark.parametrize("out", [None, BF, HF, F32])
@pytest.mark.parametrize("out8", [None, "group", "row"])
@pytest.mark.parametrize("w", [BF, HF, F32])
def test_types(lib, x, r, out, out8, w):
    if out is None and out8 is None:
        pytest.skip("no output")
    for n, H in ((3, 320), (5, 333)):
        op = MoeNorm(weights(H, w), out_dtype=out, out8=out8)
        xv, rv = rows(n, H, x), None if r is None else rows(n, H, r, seed=2, spread=3.0)
        check(op, xv, rv, op.forward(xv, rv))


@gpu
@pytest.mark.parametrize("H", [1, 2, 7, 8, 9, 127, 128, 129, 255, 256, 257, 1000, 1024, 2047, 2048, 4104, 7168, 8191, 8200, 16384, 16392,
                               20001, 32767, 32768])
@pytest.mark.parametrize("n", [1, 2, 9])
def test_sizes(lib, H, n):
    for x, r, out8 in ((BF, BF, "group"), (F32, None, "row"), (HF, F32, "group")):
        op = MoeNorm(weights(H), out_dtype=x, out8=out8)
        xv, rv = rows(n, H, x, seed=H), None if r is None else rows(n, H, r, seed=2)
        check(op, xv, rv, op.forward(xv, rv))


@gpu
@pytest.mark.parametrize("H", [64, 250, 2048, 7168])
@pytest.mark.parametrize("n", [151, 1217, 5003])
def test_many_rows(lib, H, n):
    for out, out8 in ((BF, None), (None, "group"), (None, "row")):
        op = MoeNorm(weights(H), out_dtype=out, out8=out8)
        xv, rv = rows(n, H, seed=n), rows(n, H, seed=2)
        check(op, xv, rv, op.forward(xv, rv))


@gpu
@pytest.mark.parametrize("H", [96, 250, 2048])
def test_a_row_alone(lib, H):
    """A row's result is the same in calls of few rows, in any order."""
    op = MoeNorm(weights(H), out8="group")
    x, r = rows(40, H), rows(40, H, seed=2)
    got = op.forward(x, r)
    p = torch.randperm(40, generator=torch.Generator().manual_seed(0)).cuda()
    for a, b in zip(got, op.forward(x[p].contiguous(), r[p].contiguous())):
        assert torch.equal(a[p].view(torch.uint8), b.view(torch.uint8))
    for a, b in zip(got, op.forward(x[17:18], r[17:18])):
        assert torch.equal(a[17:18].view(torch.uint8), b.view(torch.uint8))


@gpu
@pytest.mark.parametrize("pad", [1, 3, 8])
@pytest.mark.parametrize("at", [0, 1, 8])
def test_strides_and_offsets(lib, pad, at):
    """Rows inside wider matrices, at any element: what lies around them stays as it was."""
    n, H = 6, 264
    op = MoeNorm(weights(H), out8="group")
    W = H + pad + at
    x, r = rows(n, W)[:, at:at + H], rows(n, W, seed=2)[:, at:at + H]
    bufs = [torch.full((n + 2, W), 7.0, device="cuda").to(t) for t in (BF, BF, F32)]
    codes = bufs[2].to(torch.float8_e4m3fn)
    was = [b.clone() for b in bufs[:2]] + [codes.clone()]
    views = [b[1:n + 1, at:at + H] for b in (bufs[0], bufs[1], codes)]
    s = torch.empty(n, 3, device="cuda")
    got = op.forward(x, r, residual_out=views[0], out=views[1], out8=views[2], scale=s)
    assert all(g.data_ptr() == v.data_ptr() for g, v in zip((got[1], got[0], got[2], got[3]), views + [s]))
    check(op, x, r, tuple(g.contiguous() for g in got))
    for b, w in zip((bufs[0], bufs[1], codes), was):
        b.view(torch.uint8).view(n + 2, W, -1)[1:n + 1, at:at + H] = w.view(torch.uint8).view(n + 2, W, -1)[1:n + 1, at:at + H]
        assert torch.equal(b.view(torch.uint8), w.view(torch.uint8))


@gpu
@pytest.mark.parametrize("r", [None, BF, F32])
@pytest.mark.parametrize("out", [HF, F32])
@pytest.mark.parametrize("H,W,n", [(1, 3, 40), (5, 9, 7), (40, 43, 300), (264, 267, 9), (1001, 1003, 1300), (2040, 2055, 5), (4097, 4099, 1), (8203, 8205, 3)])
def test_every_alignment(lib, H, W, n, out, r):
    """Rows of an odd stride begin at every address there is; NaN beside x, residual and weight stays there, what is
    beside the outputs stays as it was."""
    def inside(t, fill, dtype, at):
        b = torch.full((n + 2, W), fill, device="cuda").to(dtype)
        v = b[1:n + 1, at:at + H]
        if t is not None:
            v.copy_(t)
        return b, v

    nan = float("nan")
    w = torch.full((H + 8,), nan, device="cuda", dtype=BF)
    w[3:3 + H] = weights(H)
    for out8 in ("group", "row"):
        op = MoeNorm(w[3:3 + H], out_dtype=out, out8=out8)
        x = inside(rows(n, H), nan, BF, 1)[1]
        rb, res = inside(rows(n, H, r, seed=2), nan, r, 2) if r else (None, None)
        ob, y = inside(None, 7.0, out, W - H)
        qb, q = inside(None, 7.0, torch.float8_e4m3fn, 0)
        was = None if res is None else res.clone()
        got = op.forward(x, res, residual_out=res, out=y, out8=q)
        check(op, x, was, tuple(g if g is None else g.contiguous() for g in got))
        y.fill_(7.0)
        q.copy_(torch.full((n, H), 7.0, device="cuda").to(q.dtype))
        assert bool((ob == 7).all()) and bool((qb.float() == 7).all())
        if res is not None:
            res.fill_(nan)
            assert bool(rb.isnan().all())


@gpu
@pytest.mark.parametrize("H", [100, 2048, 7168])
def test_in_place(lib, H):
    op = MoeNorm(weights(H))
    x, r = rows(33, H), rows(33, H, seed=2)
    want = op.forward(x, r)
    x2, r2 = x.clone(), r.clone()
    got = op.forward(x2, r2, residual_out=r2, out=x2)
    assert got[0] is x2 and got[1] is r2
    assert torch.equal(x2, want[0]) and torch.equal(r2, want[1])
    with pytest.raises(B.MoeError):
        op.forward(x2, r2, residual_out=x2)
    with pytest.raises(B.MoeError):
        op.forward(x2[:32], out=torch.as_strided(x2, (32, H), (H, 1), 1))


@gpu
def test_offset_weight_and_eps(lib):
    H = 512
    w = weights(H) - 1
    for eps in (0.0, 1e-6, 0.5):
        op = MoeNorm(w, eps=eps, out_dtype=F32, weight_offset=1.0)
        x = rows(4, H)
        check(op, x, None, op.forward(x), eps=eps, offset=1.0)


@gpu
def test_no_weight_through_the_c_call(lib):
    x = rows(3, 200)
    out = torch.empty_like(x)
    c = B.moe_norm_config_t(200, B.MOE_BF16, B.MOE_BF16, 9, B.MOE_BF16, 0, 1e-6, 0.0)
    assert B.moe_norm(c, x, 200, None, 0, None, 3, None, 0, out, 200, None, 0, None) == B.MOE_OK
    assert torch.equal(out, MoeNorm(torch.ones(200, device="cuda")).forward(x)[0])


@gpu
@pytest.mark.parametrize("H", [96, 2048, 7168])
@pytest.mark.parametrize("t", [BF, F32])
def test_values_whose_squares_leave_fp32(lib, H, t):
    x = rows(6, H, t) * torch.tensor([1e30, 1e-30, 1.0, 3e37, 2e-37, 1e19], device="cuda").to(t)[:, None]
    for eps in (0.0, 1e-6, 1e-35):
        op = MoeNorm(weights(H), eps=eps, out_dtype=F32, out8="group")
        check(op, x, None, op.forward(x), eps=eps)


@gpu
@pytest.mark.parametrize("eps", [0.0, 1e-6])
@pytest.mark.parametrize("H", [33, 2048])
def test_rows_of_zeros(lib, eps, H):
    x = rows(4, H)
    x[1] = 0
    for out8 in ("row", "group"):
        out, _, q, s = MoeNorm(weights(H), eps=eps, out8=out8).forward(x)
        assert not out[1].any() and not q[1].float().any() and bool((s[1] == 2.0 ** -126).all())
        assert bool(torch.isfinite(out).all())


@gpu
@pytest.mark.parametrize("x,r,w", [(BF, BF, BF), (HF, None, BF), (BF, None, HF), (HF, HF, HF), (HF, F32, BF), (F32, None, F32), (BF, BF, F32)])
@pytest.mark.parametrize("out8", ["group", "row"])
@pytest.mark.parametrize("n,H", [(64, 7168), (700, 333), (40, 16392)])
def test_scales_and_codes(lib, x, r, w, out8, n, H):
    """The scale is the quotient max |y| / 448 of y as the fp32 output shows it.  Codes are those of h (w + offset) against its
    largest in 64 bits: of 16-bit h and weights all of them, whose products are exact (rows of 16 bits have many quotients at the
    borders of E4M3); else those of a number within 2^-22 (two rounded products, the quotient's rounding and this test's, 2^-24
    each).  Where weights are so small that products are subnormal (off by 2^-150, scales at least 2^-126), 2^-23 besides; and
    where the scale is the smallest there is, the row's root counts (REL)."""
    for wv in (weights(H, w), torch.ones(H, device="cuda", dtype=w)):
        for f in (0, -80, -117, -118, -119, -120, -121, -133):
            wf = (wv.float() * 2.0 ** f).to(w)
            if f < 0 and w == HF:
                continue
            for out in (F32, None):
                op = MoeNorm(wf, eps=0.0, out_dtype=out, out8=out8)
                xv, rv = rows(n, H, x, seed=H), None if r is None else rows(n, H, r, seed=2, spread=3.0)
                y, h, q, s = op.forward(xv, rv)
                h = xv if h is None else h
                size = 128 if out8 == "group" else H
                G = -(-H // size)
                if out is not None:
                    z = torch.zeros(n, G * size, dtype=torch.float64, device="cuda")
                    z[:, :H] = y
                    # (64 bits hold more than twice 24 and two: rounded to 32 they are the quotient rounded once.)
                    want = (z.view(n, G, size).abs().amax(2) / 448).float().clamp(min=2.0 ** -126)
                    assert torch.equal(s, want)
                z = torch.zeros(n, G * size, dtype=torch.float64, device="cuda")
                z[:, :H] = h.double() * wf.double()
                z = z / torch.sqrt(h.double().square().mean(1, keepdim=True))
                z = z.view(n, G, size)
                v = (z / (z.abs().amax(2, keepdim=True) / 448).clamp(min=2.0 ** -126)).reshape(n, -1)[:, :H]
                if h.dtype != F32 and w != F32 and f == 0:
                    assert torch.equal(q.double(), e4m3(v))
                else:
                    slack, least = (2.0 ** -22, 0.0) if f > -100 else (REL, 2.0 ** -23)
                    qa = q.double().abs()
                    assert bool((e4m3((v.abs() * (1 - slack) - least).clamp(min=0)) <= qa).all())
                    assert bool((qa <= e4m3(v.abs() * (1 + slack) + least)).all()) and bool((q.double() * v >= 0).all())


@gpu
@pytest.mark.parametrize("out8", ["group", "row"])
@pytest.mark.parametrize("big", [1.5, 3.0, -1.5])
@pytest.mark.parametrize("out", [F32, None])
def test_results_past_fp32(lib, out8, big, out):
    """An element that the weight takes past fp32 makes its group's scale an infinity, and every value that it stands for NaN."""
    x = torch.ones(3, 300, device="cuda")
    x[1, 5] = big
    w = torch.full((300,), 3e38, device="cuda")
    y, _, q, s = MoeNorm(w, eps=0.0, out_dtype=out, out8=out8).forward(x)
    if out is not None:
        assert y[1, 5].item() == float("inf") * big and int(y.isinf().sum()) == 1
    stands = q.float() * (s.repeat_interleave(128, 1)[:, :300] if out8 == "group" else s)
    last = 128 if out8 == "group" else 300
    assert s[1, 0].item() == float("inf") and bool(stands[1, :last].isnan().all())
    assert bool(stands[1, last:].isfinite().all()) and bool(stands[[0, 2]].isfinite().all())


@gpu
def test_as_many_rows_as_there_can_be(lib):
    """2^31 - 1 rows: the blocks that take eight rows each are still counted right."""
    n = (1 << 31) - 1
    try:
        x = torch.empty(n, 1, dtype=BF, device="cuda").fill_(2.0)
        out = torch.empty(n, 1, dtype=BF, device="cuda")
    except torch.OutOfMemoryError:
        pytest.skip("needs 9 GB")
    x[-1], x[n // 2], x[0] = -3.0, -0.5, 0.0
    MoeNorm(torch.full((1,), 4.0, device="cuda")).forward(x, out=out)
    for at, want in ((-1, -4.0), (n // 2, -4.0), (0, 0.0), (1, 4.0), (-2, 4.0)):
        assert out[at].item() == want
    assert all(bool((part[part != -4] == 4).all()) for part in out[1:].split(1 << 28))


@gpu
@pytest.mark.parametrize("H", [96, 2048])
def test_special_values_stay_in_their_row(lib, H):
    x, r = rows(8, H), rows(8, H, seed=2)
    for out8 in ("row", "group"):
        op = MoeNorm(weights(H), out8=out8)
        want = op.forward(x, r)
        y = x.clone()
        y[2, 5], y[4, 50], y[6, 7] = float("nan"), float("inf"), -float("inf")
        out, ro, q, s = op.forward(y, r)
        keep = [0, 1, 3, 5, 7]
        for a, b in zip((out, ro, q, s), want):
            assert torch.equal(a[keep].view(torch.uint8), b[keep].view(torch.uint8))
        assert bool(torch.isnan(out[2]).all())
        for row, at in ((4, 50), (6, 7)):
            assert bool(torch.isnan(out[row, at])) and int(torch.isnan(out[row]).sum()) == 1 and not out[row].nan_to_num(0.0).any()
            stands = q[row].float() * (s[row].repeat_interleave(128)[:H] if out8 == "group" else s[row])
            first = 128 * (at // 128) if out8 == "group" else 0
            last = min(H, first + 128) if out8 == "group" else H
            assert bool(torch.isnan(stands[first:last]).all()) and not stands[:first].any() and not stands[last:].any()
        assert bool(torch.isnan(q[2].float()).all()) and bool(torch.isnan(s[2]).all())


@gpu
def test_tiny_values_have_their_own_scale(lib):
    """A weight that takes y below fp32's normal range: scales stop at 2^-126, and the codes at 0."""
    H = 256
    op = MoeNorm(torch.full((H,), 1e-37, device="cuda"), out_dtype=None, out8="group")
    x = rows(3, H)
    check(op, x, None, op.forward(x))


@gpu
def test_two_streams_at_once(lib):
    ops = [MoeNorm(weights(2048), out8="group"), MoeNorm(weights(7168), out8="row")]
    xs = [rows(50, 2048), rows(50, 7168)]
    want = [op.forward(x, x) for op, x in zip(ops, xs)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        got = []
        for st, op, x in zip(streams, ops, xs):
            with torch.cuda.stream(st):
                got.append([op.forward(x, x) for _ in range(3)])
        torch.cuda.synchronize()
        for calls, w in zip(got, want):
            for c in calls:
                assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(c, w))


@gpu
@pytest.mark.parametrize("n", [1, 9])
def test_another_stream_replay_and_pinned(lib, n):
    H = 2048
    op = MoeNorm(weights(H), out8="group")
    xs = [rows(n, H, seed=s) for s in range(3)]
    rs = [rows(n, H, seed=s + 10) for s in range(3)]
    want = [op.forward(x, r) for x, r in zip(xs, rs)]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = op.forward(xs[1], rs[1], stream=st)
    st.synchronize()
    same = lambda a, b: all(torch.equal(u.view(torch.uint8), v.view(torch.uint8)) for u, v in zip(a, b))
    assert same(got, want[1])
    x, r = xs[0].clone(), rs[0].clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = op.forward(x, r)
    for i in (2, 0, 1):
        x.copy_(xs[i])
        r.copy_(rs[i])
        g.replay()
        torch.cuda.synchronize()
        assert same(held, want[i])
    hx, hr = xs[2].cpu().pin_memory(), rs[2].cpu().pin_memory()
    host = torch.empty(n, H, dtype=BF).pin_memory()
    got = op.forward(hx, hr, out=host)
    torch.cuda.synchronize()
    assert same([host.cuda(), *got[1:]], want[2])


@gpu
def test_elsewhere_and_no_rows(lib):
    op, x = MoeNorm(weights(64)), rows(2, 64)
    for args in ((x.cpu(),), (x, x.cpu()), (x, x, x.cpu()), (x, None, None, x.cpu())):
        with pytest.raises(ValueError):
            op.forward(*args)
    with pytest.raises(ValueError):
        MoeNorm(torch.ones(64)).forward(x)                  # the weight on the CPU
    out, ro, q, s = MoeNorm(weights(64), out8="group").forward(x[:0], x[:0])
    assert out.shape == ro.shape == q.shape == (0, 64) and s.shape == (0, 1)
    op.weight.data = torch.ones(32, device="cuda", dtype=BF)
    with pytest.raises(ValueError):
        op.forward(x)


@gpu
def test_rows_past_32_bit_offsets(lib):
    n, stride, H = 5, 1 << 29, 72
    try:
        xb = torch.empty(n * stride, dtype=BF, device="cuda")
        yb = torch.empty(n * stride, dtype=BF, device="cuda")
    except torch.OutOfMemoryError:
        pytest.skip("needs 10.8 GB")
    x, y = xb.view(n, stride)[:, :H], yb.view(n, stride)[:, :H]
    x.copy_(rows(n, H))
    op = MoeNorm(weights(H))
    op.forward(x, out=y)
    check(op, x.contiguous(), None, (y.contiguous(), None, None, None))
