"""moe_lora: refusals (CPU), and low-rank adapters of rows against plain 64-bit torch (GPU).

Tolerance, per element: v = A x has fp32 sums of at most K / 16 + 64 additions, each off by at most
2^-23 of the sum of |a x|, and one product with the scale; it enters the second product in parts that
are off by at most 2^-16 of it (2^-24 for fp32 outputs; fp16 parts besides by 2^-39 of the row's
largest v); that product passes at most 64 additions, 2^-23 each of the sum of |b v|; base's addition
is one more, and the output is off by half a step of its type."""

import ctypes

import pytest
import torch

from mixture_experts_decode_router_gb300 import binding as B
from mixture_experts_decode_router_gb300.layer import MoeLora

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
HALF = {BF: 2.0 ** -8, HF: 2.0 ** -11, F32: 2.0 ** -24}

# ---------------------------------------------------------------- refusals, on the CPU

FAKE = 0x7f0000000000      # never dereferenced here
MB = 1 << 20


def _config(inp=64, feats=48, rank=16, L=4, x_type=B.MOE_BF16, out_type=B.MOE_BF16):
    return B.moe_lora_config_t(inp, feats, rank, L, x_type, out_type)


def _call(a=FAKE, b=FAKE + MB, scale=None, x=FAKE + 2 * MB, xs=64, idx=FAKE + 3 * MB, n=3, base=FAKE + 4 * MB, bs=48, out=FAKE + 5 * MB, os=48,
          ws=FAKE + 6 * MB, ws_bytes=1 << 30, **kw):
    return B.moe_lora(_config(**kw), a, b, scale, x, xs, idx, n, base, bs, out, os, ws, ws_bytes, 0)


def test_refusals():
    assert B.moe_lora(None, FAKE, FAKE, None, FAKE, 64, FAKE, 1, None, 0, FAKE, 48, FAKE, 1 << 20, 0) == B.MOE_ERR_NULL
    for kw in (dict(inp=0), dict(inp=60), dict(feats=0), dict(rank=0), dict(rank=12), dict(L=0), dict(x_type=B.MOE_F32), dict(x_type=3),
               dict(out_type=3), dict(out_type=-1), dict(n=-1), dict(xs=56), dict(bs=47), dict(os=0), dict(os=1 << 41)):
        assert _call(**kw) == B.MOE_ERR_INVALID_CONFIG, kw
    for kw in (dict(rank=136), dict(L=1025), dict(inp=(1 << 20) + 8, xs=(1 << 20) + 8),
               dict(feats=(1 << 28) + 1, bs=(1 << 28) + 1, os=(1 << 28) + 1)):
        assert _call(**kw) == B.MOE_ERR_UNSUPPORTED, kw
    for kw in (dict(a=None), dict(b=None), dict(x=None), dict(idx=None), dict(out=None), dict(ws=None)):
        assert _call(**kw) == B.MOE_ERR_NULL, kw
    for kw in (dict(a=FAKE + 8), dict(b=FAKE + MB + 8), dict(scale=FAKE + 2), dict(x=FAKE + 2 * MB + 8), dict(xs=68), dict(idx=FAKE + 3 * MB + 2),
               dict(base=FAKE + 4 * MB + 1), dict(out=FAKE + 5 * MB + 1), dict(out_type=B.MOE_F32, out=FAKE + 5 * MB + 2),
               dict(ws=FAKE + 6 * MB + 8)):
        assert _call(**kw) == B.MOE_ERR_ALIGNMENT, kw
    for kw in (dict(out=FAKE + 2 * MB + 382), dict(out=FAKE + 4 * MB + 2), dict(out=FAKE + 4 * MB, os=50), dict(out=FAKE + 4 * MB - 286)):
        assert _call(**kw) == B.MOE_ERR_ALIAS, kw
    need = B.moe_lora_workspace_bytes(_config(), 5000)
    assert _call(n=5000, ws_bytes=need - 1) == B.MOE_ERR_WORKSPACE and _call(ws_bytes=255) == B.MOE_ERR_WORKSPACE
    assert _call(n=0, x=None, idx=None, out=None, ws=None) == B.MOE_OK
    # What is left are the addresses themselves, which are none of CUDA's.
    for kw in (dict(), dict(base=None, bs=0), dict(base=FAKE + 5 * MB), dict(out=FAKE + 5 * MB + 2), dict(scale=FAKE + 4)):
        assert _call(**kw) == B.MOE_ERR_HOST_MEMORY, kw


def test_outputs_over_other_arguments():
    """The adapters have 8 and 6 KB, scales 16 bytes, indexes 20000, out 480 KB; the workspace its size."""
    need = B.moe_lora_workspace_bytes(_config(), 5000)
    ws = FAKE + 6 * MB
    for kw in (dict(out=FAKE), dict(out=FAKE + 8190), dict(out=FAKE + MB + 6142), dict(scale=FAKE + 5 * MB), dict(scale=FAKE + 5 * MB + 479996),
               dict(out=FAKE + 3 * MB), dict(out=FAKE + 3 * MB + 19998), dict(out=ws + need - 2), dict(ws=FAKE + 5 * MB - 16), dict(a=ws), dict(b=ws + 16),
               dict(scale=ws + need - 4), dict(idx=ws), dict(x=ws), dict(base=ws)):
        assert _call(**{**dict(n=5000, ws_bytes=need), **kw}) == B.MOE_ERR_ALIAS, kw
    # A workspace of 256 bytes is not used.
    for kw in (dict(ws=FAKE), dict(ws=FAKE + 5 * MB), dict(out=FAKE + 8192, ws=FAKE + 8192)):
        assert _call(**kw) == B.MOE_ERR_HOST_MEMORY, kw
    for kw in (dict(out=FAKE + 8192), dict(out=FAKE + 3 * MB + 20000), dict(scale=FAKE + 5 * MB + 480000), dict(base=ws + (need + 255) // 256 * 256)):
        assert _call(**{**dict(n=5000, ws_bytes=need), **kw}) == B.MOE_ERR_HOST_MEMORY, kw


def test_refusals_of_the_checked_call():
    def call(errors, n=3):
        return B.moe_lora_checked(_config(), FAKE, FAKE + MB, None, FAKE + 2 * MB, 64, FAKE + 3 * MB, n, None, 0, FAKE + 5 * MB, 48, FAKE + 6 * MB,
                                  1 << 30, errors, 0)
    assert call(None) == B.MOE_ERR_NULL and call(FAKE + 7 * MB + 8) == B.MOE_ERR_ALIGNMENT
    assert call(FAKE + 7 * MB) == B.MOE_ERR_HOST_MEMORY and call(FAKE + 7 * MB, 0) == B.MOE_OK and call(FAKE + 7 * MB, -1) == B.MOE_ERR_INVALID_CONFIG


def test_workspace_bytes():
    assert ctypes.sizeof(B.moe_lora_config_t) == 24
    assert B.moe_lora_workspace_bytes(None, 1) == 0 and B.moe_lora_workspace_bytes(_config(), -1) == 0
    assert B.moe_lora_workspace_bytes(_config(rank=20), 1) == 0
    sizes = [B.moe_lora_workspace_bytes(_config(), n) for n in (0, 1, 100, 1000, 10000, 1 << 20, (1 << 31) - 1)]
    assert sizes == sorted(sizes) and sizes[0] >= 256 and all(s % 256 == 0 for s in sizes)


@pytest.mark.parametrize("L", [1, 7, 8, 9, 100, 182, 183, 255, 256, 1024])
@pytest.mark.parametrize("inp,feats,rank", [(64, 48, 16), (2048, 2048, 16), (4096, 4096, 32), (7168, 7168, 64), (4096, 4096, 128)])
def test_a_workspace_for_many_rows_serves_fewer(L, inp, feats, rank):
    c = _config(inp, feats, rank, L)
    sizes = [B.moe_lora_workspace_bytes(c, n) for n in range(1100)]
    assert sizes == sorted(sizes)


def test_holder_refusals():
    a, b = torch.zeros(3, 16, 64, dtype=BF), torch.zeros(3, 40, 16, dtype=BF)
    for bad in ((a[0], b), (a, b[:2]), (a, b.half()), (a.float(), b.float()), (a[:, :8], b), (a.transpose(1, 2), b), (a, b, torch.ones(4)),
                (a, b, torch.ones(3).half())):
        with pytest.raises(ValueError):
            MoeLora(*bad)
    with pytest.raises(B.MoeError):
        MoeLora(torch.zeros(3, 12, 64, dtype=BF), torch.zeros(3, 40, 12, dtype=BF))
    op = MoeLora(a, b)
    x, idx = torch.zeros(2, 64, dtype=BF), torch.zeros(2, dtype=torch.int32)
    for args in ((x.half(), idx), (x[:, :32], idx), (x[0], idx), (torch.zeros(64, 2, dtype=BF).T, idx), (x, idx, torch.zeros(2, 40)),
                 (x, idx, torch.zeros(3, 40, dtype=BF)), (x, idx, None, torch.zeros(2, 41, dtype=BF)), (x, idx.long()), (x, idx[:1]),
                 (x, idx)):
        with pytest.raises(ValueError):
            op.forward(*args)
    with pytest.raises(TypeError):
        op.forward(x, None)


# ---------------------------------------------------------------- on the GPU

gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    B.load()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rows(n, K, dtype=BF, seed=1, pad=0, spread=1.0):
    return (torch.randn(n, K + pad, generator=gen(seed), device="cuda") * spread).to(dtype)[:, :K]


def adapters(L, r, K, O, dtype=BF, seed=5):
    g = gen(seed)
    a = (torch.randn(L, r, K, generator=g, device="cuda") / K ** 0.5).to(dtype)
    b = (torch.randn(L, O, r, generator=g, device="cuda") / r ** 0.5).to(dtype)
    return a, b, 0.5 + torch.rand(L, generator=g, device="cuda")


def choose(n, L, seed=3, none=0.2):
    g = gen(seed)
    idx = torch.randint(0, L, (n,), generator=g, device="cuda")
    return torch.where(torch.rand(n, generator=g, device="cuda") < none, -1, idx).to(torch.int32)


def reference(op, x, idx, base):
    """(result, tolerance) in 64 bits."""
    a, b, scale = op.a, op.b, op.scale
    L, r, K = a.shape
    n, O = x.shape[0], b.shape[1]
    y = torch.zeros(n, O, dtype=torch.float64, device="cuda") if base is None else base.double()
    mag, off = y.abs(), torch.zeros_like(y)
    part = 2.0 ** -24 if op.out_dtype == F32 else 2.0 ** -16
    y = y.clone()
    for e in range(L):
        at = torch.nonzero(idx == e).flatten()
        if len(at) == 0:
            continue
        s = 1.0 if scale is None else float(scale[e])
        xd, ad, bd = x[at].double(), a[e].double(), b[e].double()
        v, vm = xd @ ad.T * s, xd.abs() @ ad.abs().T * abs(s)
        ve = vm * ((64 + K / 16) * 2.0 ** -23 + 2.0 ** -24) + v.abs() * part
        if x.dtype == HF:
            ve += v.abs().amax(1, keepdim=True) * 2.0 ** -39
        bv = v.abs() @ bd.abs().T
        y[at] += v @ bd.T
        mag[at] += bv
        off[at] += ve @ bd.abs().T + 64 * 2.0 ** -23 * bv
    tol = off + 2.0 ** -24 * mag
    tol = tol + HALF[op.out_dtype] * (y.abs() + tol)
    if op.out_dtype == HF:
        tol = tol + 2.0 ** -25
    return y, tol


def check(op, x, idx, base, out):
    y, tol = reference(op, x, idx, base)
    err = (out.double() - y).abs()
    assert out.dtype == op.out_dtype and bool((err <= tol).all()), float((err - tol).max())
    rest = (idx < 0) | (idx >= op.a.shape[0])
    want = torch.zeros_like(out) if base is None else base
    assert torch.equal(out[rest], want[rest])


@gpu
@pytest.mark.parametrize("t", [BF, HF])
@pytest.mark.parametrize("y", [BF, HF, F32])
@pytest.mark.parametrize("r", [8, 16, 24, 32, 40, 64, 72, 104, 128])
@pytest.mark.parametrize("n", [1, 13, 700])
def test_types_and_ranks(lib, t, y, r, n):
    a, b, s = adapters(5, r, 256, 104, t)
    op = MoeLora(a, b, s, out_dtype=y)
    x, idx, base = rows(n, 256, t), choose(n, 5), rows(n, 104, y, seed=8)
    if n == 1:
        idx[0] = 3
    check(op, x, idx, base, op.forward(x, idx, base))


@gpu
@pytest.mark.parametrize("K,O", [(8, 1), (8, 40), (16, 3), (24, 33), (32, 32), (40, 31), (88, 65), (256, 255), (1032, 129), (2048, 2048),
                                 (7168, 130), (64, 7168), (5000, 1001)])
@pytest.mark.parametrize("n", [1, 6, 40, 600])
def test_sizes(lib, K, O, n):
    a, b, s = adapters(3, 16, K, O, seed=K)
    for y in (BF, F32):
        op = MoeLora(a, b, s, out_dtype=y)
        x, idx, base = rows(n, K, seed=n), choose(n, 3, seed=n, none=0.1), rows(n, O, y, seed=8)
        check(op, x, idx, base, op.forward(x, idx, base))
        check(op, x, idx, None, op.forward(x, idx))


@gpu
@pytest.mark.parametrize("n", [1, 2, 7, 8, 9, 16, 17, 31, 64, 65, 127, 128, 129, 255, 256, 257, 511, 512, 513, 1024, 2049, 5000])
@pytest.mark.parametrize("L", [1, 2, 64])
def test_row_counts(lib, n, L):
    a, b, s = adapters(L, 16, 128, 72)
    op = MoeLora(a, b, s)
    x, base = rows(n, 128, seed=n), rows(n, 72, seed=8)
    for idx in (choose(n, L, seed=n, none=0.0), choose(n, L, seed=n, none=0.5), torch.full((n,), L - 1, dtype=torch.int32, device="cuda"),
                torch.full((n,), -1, dtype=torch.int32, device="cuda"), torch.sort(choose(n, L, seed=n)).values):
        check(op, x, idx, base, op.forward(x, idx, base))


@gpu
@pytest.mark.parametrize("y", [BF, F32])
@pytest.mark.parametrize("O", [1024, 2080, 1003])
@pytest.mark.parametrize("rest", [1, 3, 8, 15, 16, 17, 31, 32, 33, 48, 49, 80, 97, 113, 127, 128])
def test_runs_that_end_inside_a_tile(lib, y, O, rest):
    """Rows of an adapter behind whole tiles of 128, over several tiles of outputs, together in memory and not."""
    a, b, s = adapters(4, 16, 192, O)
    op = MoeLora(a, b, s, out_dtype=y)
    idx = torch.cat([torch.full((m,), e, dtype=torch.int32, device="cuda")
                     for e, m in enumerate((128 + rest, rest, 256 + rest, 384 + rest))])
    n = len(idx)
    x, base = rows(n, 192, seed=rest), rows(n, O, y, seed=8)
    check(op, x, idx, base, op.forward(x, idx, base))
    p = torch.randperm(n, generator=torch.Generator().manual_seed(rest)).cuda()
    check(op, x, idx[p], base, op.forward(x, idx[p], base))
    got = op.forward(x, idx)
    check(op, x, idx, None, got)


@gpu
@pytest.mark.parametrize("n", [17, 32, 33, 200, 257, 500, 511, 512, 513, 767, 1023, 1024])
@pytest.mark.parametrize("L", [1, 7, 219])
@pytest.mark.parametrize("how", ["one", "none", "skewed", "blocks", "few"])
def test_how_rows_share_adapters(lib, n, L, how):
    """Rows of one adapter, of none, most of one, runs of eight and nine, and a few rows between many without."""
    a, b, s = adapters(L, 16, 96, 131)
    g, t = torch.Generator(device="cuda").manual_seed(n + L), torch.arange(n, device="cuda")
    idx = torch.randint(0, L, (n,), generator=g, device="cuda")
    some = torch.rand(n, generator=g, device="cuda")
    if how == "one":
        idx = torch.full_like(idx, L - 1)
    elif how == "none":
        idx = torch.where(t % 2 == 0, -1, L)
    elif how == "skewed":
        idx = torch.where(some < 0.8, L // 2, idx)
    elif how == "blocks":
        idx = t // torch.where(t < n // 2, 8, 9) % (L + 1)
    else:
        idx = torch.where(some < 0.9, 1 << 20, idx)
    idx, x = idx.to(torch.int32), rows(n, 96)
    op = MoeLora(a, b, s)
    base = rows(n, 131, seed=8)
    check(op, x, idx, base, op.forward(x, idx, base))
    check(op, x, idx, None, op.forward(x, idx))
    out = base.clone()
    op.forward(x, idx, out, out=out)
    check(op, x, idx, base, out)


@gpu
@pytest.mark.parametrize("n", [5, 300, 900])
def test_indexes_outside(lib, n):
    """-1, the number of adapters, and the ends of int32 are no adapter."""
    a, b, s = adapters(4, 16, 64, 40)
    op = MoeLora(a, b, s)
    x, base = rows(n, 64), rows(n, 40, seed=8)
    idx = choose(n, 4, none=0.0)
    for i, v in enumerate((-1, 4, -2 ** 31, 2 ** 31 - 1)):
        idx[i::5] = v
    check(op, x, idx, base, op.forward(x, idx, base))
    check(op, x, idx, None, op.forward(x, idx))
    keep = base.clone()
    assert op.forward(x, idx, keep, out=keep) is keep
    check(op, x, idx, base, keep)


@gpu
@pytest.mark.parametrize("n", [40, 700])
@pytest.mark.parametrize("L", [300, 1024])
def test_many_adapters(lib, n, L):
    a, b, s = adapters(L, 8, 64, 40)
    op = MoeLora(a, b, s)
    x, idx, base = rows(n, 64), choose(n, L), rows(n, 40, seed=8)
    check(op, x, idx, base, op.forward(x, idx, base))


@gpu
@pytest.mark.parametrize("n", [3, 100, 900])
def test_without_scales(lib, n):
    a, b, _ = adapters(4, 16, 64, 40)
    op = MoeLora(a, b, out_dtype=F32)
    x, idx = rows(n, 64), choose(n, 4)
    check(op, x, idx, None, op.forward(x, idx))
    assert torch.equal(op.forward(x, idx), MoeLora(a, b, torch.ones(4, device="cuda"), out_dtype=F32).forward(x, idx))


@gpu
@pytest.mark.parametrize("y", [BF, F32])
@pytest.mark.parametrize("n", [6, 600])
@pytest.mark.parametrize("at,wide", [(0, 88), (1, 91), (2, 90), (4, 96), (3, 89)])
def test_strides_and_offsets(lib, y, n, at, wide):
    """Rows inside wider matrices: what lies around the output stays as it was."""
    a, b, s = adapters(3, 16, 64, 75)
    op = MoeLora(a, b, s, out_dtype=y)
    x, idx = rows(n, 64, pad=24), choose(n, 3)
    base = rows(n, wide, y, seed=8)[:, at:at + 75]
    buf = rows(n + 2, wide, y, seed=9)
    was, out = buf.clone(), buf[1:n + 1, at:at + 75]
    assert op.forward(x, idx, base, out=out).data_ptr() == out.data_ptr()
    check(op, x, idx, base, out)
    buf[1:n + 1, at:at + 75] = was[1:n + 1, at:at + 75]
    assert torch.equal(buf, was)
    # In place.
    op.forward(x, idx, out, out=out)
    check(op, x, idx, was[1:n + 1, at:at + 75], out)
    buf[1:n + 1, at:at + 75] = was[1:n + 1, at:at + 75]
    assert torch.equal(buf, was)


@gpu
@pytest.mark.parametrize("n", [12, 700])
@pytest.mark.parametrize("t", [BF, HF])
def test_large_and_small_values(lib, n, t):
    """v far outside fp16's range, or below it, in rows next to ordinary ones."""
    a, b, s = adapters(3, 32, 256, 64, t)
    s = s * torch.tensor([1e8, 1.0, 1e-8], device="cuda")
    op = MoeLora(a, b, s, out_dtype=F32)
    f = torch.tensor([1e25, 1e-20, 1.0] if t == BF else [3e3, 1e-4, 1.0], device="cuda").repeat(n)[:n, None]
    x, idx = (rows(n, 256) * f).to(t), choose(n, 3)
    check(op, x, idx, None, op.forward(x, idx))


@gpu
@pytest.mark.parametrize("r", [8, 16])
@pytest.mark.parametrize("t", [BF, HF])
@pytest.mark.parametrize("n", [12, 700])
def test_special_values_stay_in_their_row(lib, n, t, r):
    a, b, s = adapters(2, r, 64, 40, t)
    op = MoeLora(a, b, s, out_dtype=F32)
    x, idx = rows(n, 64, t), choose(n, 2, none=0.0)
    want = op.forward(x, idx)
    y = x.clone()
    y[3, 5], y[6, 9] = float("nan"), float("inf")
    got = op.forward(y, idx)
    keep = [i for i in range(n) if i not in (3, 6)]
    assert torch.equal(got[keep], want[keep])
    assert bool(torch.isnan(got[3]).all())
    # v is an infinity wherever A's element is not 0; the sum over the rank is one, or NaN where signs differ.
    e = int(idx[6])
    v = (a[e].double() @ y[6].double()) * float(s[e])
    ref = (b[e].double() * v).sum(1)
    assert torch.equal(torch.isnan(got[6]), torch.isnan(ref))
    assert torch.equal(got[6].double().nan_to_num(0.0, 1.0, -1.0), ref.nan_to_num(0.0, 1.0, -1.0))


@gpu
@pytest.mark.parametrize("n", [4, 30, 700])
def test_other_adapters_are_not_read(lib, n):
    """An adapter that no row has may hold anything."""
    a, b, s = adapters(4, 24, 72, 40)
    op = MoeLora(a, b, s)
    x, base = rows(n, 72), rows(n, 40, seed=8)
    idx = 2 * choose(n, 2, none=0.0)
    want = op.forward(x, idx, base)
    for e in (1, 3):
        a[e], b[e], s[e] = float("nan"), float("inf"), float("nan")
    assert torch.equal(op.forward(x, idx, base), want)
    check(op, x, idx, base, want)


@gpu
@pytest.mark.parametrize("n", [16, 300, 800])
def test_the_same_call_twice(lib, n):
    a, b, s = adapters(6, 32, 512, 200)
    op = MoeLora(a, b, s, out_dtype=F32)
    x, idx = rows(n, 512), choose(n, 6)
    want = op.forward(x, idx)
    for _ in range(5):
        assert torch.equal(op.forward(x, idx), want)


@gpu
def test_two_streams_at_once(lib):
    ops = [MoeLora(*adapters(6, 16, 512, 200)), MoeLora(*adapters(3, 64, 256, 300))]
    xs = [rows(900, 512), rows(2000, 256)]
    ids = [choose(900, 6), choose(2000, 3)]
    want = [op.forward(x, i) for op, x, i in zip(ops, xs, ids)]
    streams = [torch.cuda.Stream() for _ in range(4)]
    torch.cuda.synchronize()
    for _ in range(20):
        got = []
        for k, st in enumerate(streams):
            with torch.cuda.stream(st):                     # (two streams on each holder)
                got.append([ops[k % 2].forward(xs[k % 2], ids[k % 2]) for _ in range(3)])
        torch.cuda.synchronize()
        assert all(torch.equal(y, want[k % 2]) for k, ys in enumerate(got) for y in ys)


@gpu
@pytest.mark.parametrize("n", [1, 20, 700])
def test_another_stream_replay_and_pinned(lib, n):
    a, b, s = adapters(5, 16, 256, 104)
    op = MoeLora(a, b, s)
    xs = [rows(n, 256, seed=k) for k in range(3)]
    ids = [choose(n, 5, seed=k, none=0.1) for k in range(3)]
    base = rows(n, 104, seed=8)
    want = [op.forward(x, i, base) for x, i in zip(xs, ids)]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = op.forward(xs[1], ids[1], base, stream=st)
    st.synchronize()
    assert torch.equal(got, want[1])
    x, idx = xs[0].clone(), ids[0].clone()
    graphs = []
    for _ in range(2):                                      # two graphs, whose replays overlap
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            held = op.forward(x, idx, base)
        graphs.append((g, held))
    for k in (2, 0, 1):
        x.copy_(xs[k])
        idx.copy_(ids[k])
        torch.cuda.synchronize()
        for (g, _), side in zip(graphs, (torch.cuda.current_stream(), st)):
            with torch.cuda.stream(side):
                g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(held, want[k]) for _, held in graphs)
    host = torch.empty(n, 104, dtype=BF).pin_memory()
    op.forward(xs[2].cpu().pin_memory(), ids[2], base.cpu().pin_memory(), out=host)
    torch.cuda.synchronize()
    check(op, xs[2], ids[2], base, host.cuda())             # (many rows: not by the same kernels)


@gpu
def test_elsewhere_and_no_rows(lib):
    a, b, s = adapters(3, 16, 64, 40)
    op, x, idx = MoeLora(a, b, s), rows(2, 64), choose(2, 3)
    base = rows(2, 40)
    for args in ((x.cpu(), idx), (x, idx.cpu()), (x, idx.cpu().pin_memory()), (x, idx, base.cpu()), (x, idx, None, base.cpu())):
        with pytest.raises(ValueError):
            op.forward(*args)
    with pytest.raises(ValueError):
        MoeLora(a.cpu(), b.cpu()).forward(x, idx)
    with pytest.raises(ValueError):
        MoeLora(a, b.cpu())
    assert op.forward(x[:0], idx[:0]).shape == (0, 40) and op.forward(x[:0], idx[:0], base[:0]).shape == (0, 40)
    a.data = a[:, :8].contiguous()
    with pytest.raises(ValueError):
        op.forward(x, idx)


@gpu
@pytest.mark.parametrize("n", [5, 600])
def test_rows_past_32_bit_offsets(lib, n):
    K, O, stride = 64, 40, (1 << 31) // (n - 1) // 8 * 8 + 8
    try:
        xb = torch.empty(n * stride, dtype=BF, device="cuda")
        yb = torch.empty(n * stride, dtype=BF, device="cuda")
    except torch.OutOfMemoryError:
        pytest.skip("needs 10 GB")
    a, b, s = adapters(3, 16, K, O)
    op, idx = MoeLora(a, b, s), choose(n, 3)
    x, y = xb.view(n, stride)[:, :K], yb.view(n, stride)[:, :O]
    x.copy_(rows(n, K))
    op.forward(x, idx, out=y)
    check(op, x.contiguous(), idx, None, y.contiguous())


@gpu
def test_matrices_past_32_bit_offsets(lib):
    """The last adapters' matrices begin past 2^31 elements."""
    L, r, K, O = 1024, 128, 16384, 16392
    try:
        a = torch.zeros(L, r, K, dtype=BF, device="cuda")
        b = torch.zeros(L, O, r, dtype=BF, device="cuda")
    except torch.OutOfMemoryError:
        pytest.skip("needs 9 GB")
    small = adapters(2, r, K, O)
    a[-2:], b[-2:] = small[0], small[1]
    op = MoeLora(a, b)
    for n in (5, 600):
        x = rows(n, K)
        idx = choose(n, 2, none=0.0)
        got = op.forward(x, idx + (L - 2))
        check(MoeLora(small[0], small[1]), x, idx, None, got)
    assert not op.forward(x, idx).any()


@gpu
@pytest.mark.parametrize("n", [1, 6, 40])
def test_a_step_between_two_layers(lib, n):
    """A run as a decoder makes it: the norm with the residual, a projection with adapters beside it, the residual and the norm
    again, then the layer."""
    import numpy as np

    from mixture_experts_decode_router_gb300 import synth
    from mixture_experts_decode_router_gb300.layer import MoeLayer, MoeMatvec, MoeNorm
    from oracle import moe_oracle as O
    from tests.int4_helpers import int4_oracle_layer
    from tests.moe_helpers import bf16_bits
    from tests.test_int4_experts import cfg_of, close as close_layer
    from tests.test_matvec import close as close_matvec, matrix
    from tests.test_norm import check as check_norm
    H = 256
    first, second = MoeNorm(rows(1, H, seed=20)[0] + 1), MoeNorm(rows(1, H, seed=21)[0] + 1, out8="group")
    q, w = matrix(H, H, "int4_g64")
    lora = MoeLora(*adapters(4, 16, H, H))
    x, stream, idx = rows(n, H), rows(n, H, seed=2), choose(n, 4)
    old = stream.clone()
    h = first.forward(x, stream, residual_out=stream)
    check_norm(first, x, old, h)
    p = MoeMatvec(q).forward(h[0])
    close_matvec(p, h[0], w)
    y = lora.forward(h[0], idx, p.clone())
    check(lora, h[0], idx, p, y)
    old = stream.clone()
    z = second.forward(y, stream, residual_out=stream)
    check_norm(second, y, old, z)
    lw = synth.make_weights(cfg_of("int4_g64", hidden=H), "cuda")
    out, chosen, _ = MoeLayer(lw, n).forward(z[0])
    ref, ridx, _, _ = O.moe_forward(int4_oracle_layer(lw), bf16_bits(z[0]))
    assert np.array_equal(chosen.cpu().numpy(), ridx)
    close_layer(out.float().cpu().numpy(), ref)
