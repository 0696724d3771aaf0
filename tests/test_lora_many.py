"""moe_lora's kernels for many rows (sort, shrink, sum, expand), against the 64 bits of test_lora.py and with its
tolerances.  A call takes them where its workspace is more than the 256 bytes of the kernel for few rows; every
case here asserts that."""

import pytest
import torch

from mixture_experts_decode_router_gb300 import binding as B
from mixture_experts_decode_router_gb300.layer import MoeLora
from tests.test_lora import BF, F32, HF, adapters, check, choose, lib, rows  # noqa: F401 (lib is a fixture)

pytestmark = pytest.mark.gpu


def holder(n, a, b, scale=None, **kw):
    """A holder whose calls of n rows are sorted."""
    op = MoeLora(a, b, scale, **kw)
    assert B.moe_lora_workspace_bytes(op.c_cfg, n) > 256
    return op


@pytest.mark.parametrize("y", [BF, HF, F32])
@pytest.mark.parametrize("each", [1, 4, 8, 9, 16, 17, 33])
def test_short_runs_of_one_tile_of_outputs(lib, y, each):
    """Blocks of the expansion take several adapters' few rows one after another, with base's rows on their way."""
    L, K, O = 640, 64, 128
    n = L * each if each > 1 else 2 * L
    a, b, s = adapters(L, 16, K, O)
    op = holder(n, a, b, s, out_dtype=y)
    idx = (torch.arange(n, device="cuda") % L if each > 1 else torch.arange(n, device="cuda")).to(torch.int32)
    x, base = rows(n, K), rows(n, O, y, seed=8)
    want = op.forward(x, idx, base)
    check(op, x, idx, base, want)
    for _ in range(4):
        assert torch.equal(op.forward(x, idx, base), want)
    out = base.clone()
    op.forward(x, idx, out, out=out)
    assert torch.equal(out, want)


@pytest.mark.parametrize("y,O", [(BF, 256), (F32, 256), (BF, 131)])
@pytest.mark.parametrize("r", [16, 64])
def test_nothing_is_written_while_an_error_is_pending(lib, y, O, r):
    """The word that a wait that gave up would leave, set by hand: out stays as it was (base, in place), until the holder
    is asked."""
    n = 1500
    a, b, s = adapters(5, r, 256, O)
    op = holder(n, a, b, s, out_dtype=y)
    x, idx, base = rows(n, 256), choose(n, 5), rows(n, O, y, seed=8)
    want = op.forward(x, idx, base)
    check(op, x, idx, base, want)
    assert op.device_error() == 0
    errors = op._held[3]
    errors[8:12] = torch.tensor([33, 0, 0, 0], dtype=torch.uint8, device="cuda")
    out = torch.full_like(base, 7)
    assert op.forward(x, idx, base, out=out) is out and bool((out == 7).all())
    keep = base.clone()
    op.forward(x, idx, keep, out=keep)
    assert torch.equal(keep, base)
    assert op.device_error() == 33 and op.device_error() == 0
    assert torch.equal(op.forward(x, idx, base), want)
    # What is no code of these waits says nothing (a holder that was made within a capture, before its first replay).
    errors[8:12] = 255
    assert torch.equal(op.forward(x, idx, base), want) and op.device_error() == 0
    # A workspace's own word is the last call's.
    c, need = op.c_cfg, B.moe_lora_workspace_bytes(op.c_cfg, n)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    assert B.moe_lora(c, a, b, s, x, 256, idx, n, base, O, out, O, ws, need) == B.MOE_OK
    assert torch.equal(out, want) and B.moe_workspace_check(ws, need) == (B.MOE_OK, 0)


# Outputs in whole aligned pieces of 16 bytes (the expansion's aligned form), and not.
WIDE, ODD = 160, 104


@pytest.mark.parametrize("t", [BF, HF])
@pytest.mark.parametrize("y", [BF, HF, F32])
@pytest.mark.parametrize("r", [8, 16, 24, 32, 40, 64, 72, 104, 128])
@pytest.mark.parametrize("O", [WIDE, ODD])
def test_types_and_ranks(lib, t, y, r, O):
    n = 1100
    a, b, s = adapters(5, r, 256, O, t)
    op = holder(n, a, b, s, out_dtype=y)
    x, idx, base = rows(n, 256, t), choose(n, 5), rows(n, O, y, seed=8)
    check(op, x, idx, base, op.forward(x, idx, base))


@pytest.mark.parametrize("t", [BF, HF])
@pytest.mark.parametrize("y", [BF, HF, F32])
@pytest.mark.parametrize("r", [8, 24, 64, 72, 128])
@pytest.mark.parametrize("O", [640, 651])
def test_blocks_of_several_units_and_tiles(lib, t, y, r, O):
    """Over 304 runs: blocks of the expansion take two or three units of five or six tiles of outputs each, so that its ring,
    its accumulators and base's copies go round; adapters of 2 to 33 rows, some of none."""
    L, K = 640, 72
    each = torch.tensor([5, 2, 33, 16, 0, 17, 9], device="cuda").repeat(L)[:L]
    idx = torch.repeat_interleave(torch.arange(L, device="cuda"), each)
    idx = idx[torch.randperm(len(idx), generator=torch.Generator().manual_seed(r)).cuda()].to(torch.int32)
    idx[::50] = -1
    n = len(idx)
    a, b, s = adapters(L, r, K, O, t)
    op = holder(n, a, b, s, out_dtype=y)
    x, base = rows(n, K, t), rows(n, O, y, seed=8)
    want = op.forward(x, idx, base)
    check(op, x, idx, base, want)
    out = base.clone()
    op.forward(x, idx, out, out=out)
    assert torch.equal(out, want)
    check(op, x, idx, None, op.forward(x, idx))


@pytest.mark.parametrize("K,O", [(8, 1), (8, 40), (16, 3), (24, 33), (32, 32), (40, 31), (88, 65), (256, 255), (1032, 129), (2048, 2048),
                                 (7168, 130), (64, 7168), (5000, 1001)])
@pytest.mark.parametrize("n", [1025, 2049])
def test_sizes(lib, K, O, n):
    for r, y in ((16, BF), (16, F32), (48, BF), (48, F32)):
        a, b, s = adapters(3, r, K, O, seed=K)
        op = holder(n, a, b, s, out_dtype=y)
        x, idx, base = rows(n, K, seed=n), choose(n, 3, seed=n, none=0.1), rows(n, O, y, seed=8)
        check(op, x, idx, base, op.forward(x, idx, base))
        check(op, x, idx, None, op.forward(x, idx))


@pytest.mark.parametrize("n", [1025, 1151, 1152, 1153, 4095, 20001])
@pytest.mark.parametrize("L", [1, 2, 64, 1024])
def test_row_counts(lib, n, L):
    """Up to eight stretches of K, and above some 5000 rows fewer."""
    for r, O in ((16, 72), (40, 96)):
        a, b, s = adapters(L, r, 704, O)
        op = holder(n, a, b, s)
        x, base = rows(n, 704, seed=n), rows(n, O, seed=8)
        for idx in (choose(n, L, seed=n, none=0.0), choose(n, L, seed=n, none=0.5), torch.full((n,), L - 1, dtype=torch.int32, device="cuda"),
                    torch.full((n,), -1, dtype=torch.int32, device="cuda"), torch.sort(choose(n, L, seed=n)).values):
            check(op, x, idx, base, op.forward(x, idx, base))


@pytest.mark.parametrize("t,y,r", [(HF, HF, 16), (HF, F32, 64), (BF, HF, 72)])
@pytest.mark.parametrize("O", [1024, 1003])
@pytest.mark.parametrize("rest", [1, 15, 16, 17, 33, 97, 127, 128])
def test_runs_that_end_inside_a_tile(lib, t, y, r, O, rest):
    a, b, s = adapters(4, r, 192, O, t)
    idx = torch.cat([torch.full((m,), e, dtype=torch.int32, device="cuda")
                     for e, m in enumerate((384 + rest, rest, 256 + rest, 384 + rest))])
    n = len(idx)
    op = holder(n, a, b, s, out_dtype=y)
    x, base = rows(n, 192, t, seed=rest), rows(n, O, y, seed=8)
    check(op, x, idx, base, op.forward(x, idx, base))
    p = torch.randperm(n, generator=torch.Generator().manual_seed(rest)).cuda()
    check(op, x, idx[p], base, op.forward(x, idx[p], base))


@pytest.mark.parametrize("r", [16, 64])
@pytest.mark.parametrize("O", [WIDE, ODD])
def test_indexes_outside(lib, r, O):
    n = 2500
    a, b, s = adapters(4, r, 64, O)
    op = holder(n, a, b, s)
    x, base = rows(n, 64), rows(n, O, seed=8)
    idx = choose(n, 4, none=0.0)
    for i, v in enumerate((-1, 4, -2 ** 31, 2 ** 31 - 1)):
        idx[i::5] = v
    check(op, x, idx, base, op.forward(x, idx, base))
    check(op, x, idx, None, op.forward(x, idx))
    keep = base.clone()
    assert op.forward(x, idx, keep, out=keep) is keep
    check(op, x, idx, base, keep)


@pytest.mark.parametrize("O", [WIDE, ODD])
@pytest.mark.parametrize("y", [BF, F32])
def test_without_scales(lib, O, y):
    n = 1500
    a, b, _ = adapters(4, 32, 64, O)
    op = holder(n, a, b, out_dtype=y)
    x, idx = rows(n, 64), choose(n, 4)
    check(op, x, idx, None, op.forward(x, idx))
    assert torch.equal(op.forward(x, idx), MoeLora(a, b, torch.ones(4, device="cuda"), out_dtype=y).forward(x, idx))


@pytest.mark.parametrize("y", [BF, HF, F32])
@pytest.mark.parametrize("O", [75, 160])
@pytest.mark.parametrize("at,pad", [(0, 0), (0, 16), (1, 16), (2, 15), (4, 20), (3, 14), (8, 16)])
def test_strides_and_offsets(lib, y, O, at, pad):
    """Rows inside wider matrices, base and out at like and at other addresses: what lies around the output stays."""
    n, wide = 1100, O + pad
    at = min(at, pad)
    a, b, s = adapters(3, 24, 64, O)
    op = holder(n, a, b, s, out_dtype=y)
    x, idx = rows(n, 64, pad=24), choose(n, 3)
    buf = rows(n + 2, wide, y, seed=9)
    was, out = buf.clone(), buf[1:n + 1, at:at + O]
    for base in (rows(n, wide, y, seed=8)[:, at:at + O], rows(n, O, y, seed=8), rows(n, O, y, seed=8, pad=13), None):
        assert op.forward(x, idx, base, out=out).data_ptr() == out.data_ptr()
        check(op, x, idx, base, out)
        buf[1:n + 1, at:at + O] = was[1:n + 1, at:at + O]
        assert torch.equal(buf, was)
    op.forward(x, idx, out, out=out)
    check(op, x, idx, was[1:n + 1, at:at + O], out)
    buf[1:n + 1, at:at + O] = was[1:n + 1, at:at + O]
    assert torch.equal(buf, was)


@pytest.mark.parametrize("t", [BF, HF])
@pytest.mark.parametrize("r", [16, 72])
@pytest.mark.parametrize("O", [WIDE, ODD])
def test_large_and_small_values(lib, t, r, O):
    n = 1500
    a, b, s = adapters(3, r, 256, O, t)
    s = s * torch.tensor([1e8, 1.0, 1e-8], device="cuda")
    op = holder(n, a, b, s, out_dtype=F32)
    f = torch.tensor([1e25, 1e-20, 1.0] if t == BF else [3e3, 1e-4, 1.0], device="cuda").repeat(n)[:n, None]
    x, idx = (rows(n, 256) * f).to(t), choose(n, 3)
    check(op, x, idx, None, op.forward(x, idx))


@pytest.mark.parametrize("r", [8, 16, 40])
@pytest.mark.parametrize("t", [BF, HF])
@pytest.mark.parametrize("O", [WIDE, ODD])
def test_special_values_stay_in_their_row(lib, t, r, O):
    n = 1500
    a, b, s = adapters(2, r, 64, O, t)
    op = holder(n, a, b, s, out_dtype=F32)
    x, idx = rows(n, 64, t), choose(n, 2, none=0.0)
    want = op.forward(x, idx)
    y = x.clone()
    y[3, 5], y[6, 9], y[n - 1, 0] = float("nan"), float("inf"), -float("inf")
    got = op.forward(y, idx)
    keep = [i for i in range(n) if i not in (3, 6, n - 1)]
    assert torch.equal(got[keep], want[keep])
    assert bool(torch.isnan(got[3]).all())
    for row in (6, n - 1):
        e = int(idx[row])
        v = (a[e].double() @ y[row].double()) * float(s[e])
        ref = (b[e].double() * v).sum(1)
        assert torch.equal(torch.isnan(got[row]), torch.isnan(ref))
        assert torch.equal(got[row].double().nan_to_num(0.0, 1.0, -1.0), ref.nan_to_num(0.0, 1.0, -1.0))


@pytest.mark.parametrize("r", [8, 24, 72])
@pytest.mark.parametrize("O", [WIDE, ODD])
def test_other_adapters_are_not_read(lib, r, O):
    """Nor base's rows that others have, nor the rest of x's last rows."""
    n = 1500
    a, b, s = adapters(4, r, 72, O)
    op = holder(n, a, b, s)
    x, base = rows(n, 72), rows(n, O, seed=8)
    idx = 2 * choose(n, 2, none=0.0)
    want = op.forward(x, idx, base)
    for e in (1, 3):
        a[e], b[e], s[e] = float("nan"), float("inf"), float("nan")
    assert torch.equal(op.forward(x, idx, base), want)
    check(op, x, idx, base, want)


@pytest.mark.parametrize("r", [16, 64])
@pytest.mark.parametrize("O", [WIDE, ODD])
@pytest.mark.parametrize("n", [1100, 6000])
def test_the_same_call_twice(lib, n, r, O):
    a, b, s = adapters(6, r, 1024, O)
    op = holder(n, a, b, s, out_dtype=F32)
    x, idx = rows(n, 1024), choose(n, 6)
    want = op.forward(x, idx)
    check(op, x, idx, None, want)
    for _ in range(5):
        assert torch.equal(op.forward(x, idx), want)


def test_two_streams_at_once(lib):
    ops = [holder(1300, *adapters(6, 16, 512, 200)), holder(2000, *adapters(3, 64, 256, 320))]
    xs = [rows(1300, 512), rows(2000, 256)]
    ids = [choose(1300, 6), choose(2000, 3)]
    want = [op.forward(x, i) for op, x, i in zip(ops, xs, ids)]
    for op, x, i, w in zip(ops, xs, ids, want):
        check(op, x, i, None, w)
    streams = [torch.cuda.Stream() for _ in range(4)]
    torch.cuda.synchronize()
    for _ in range(10):
        got = []
        for k, st in enumerate(streams):
            with torch.cuda.stream(st):                     # (two streams on each holder)
                got.append([ops[k % 2].forward(xs[k % 2], ids[k % 2]) for _ in range(3)])
        torch.cuda.synchronize()
        assert all(torch.equal(y, want[k % 2]) for k, ys in enumerate(got) for y in ys)
    assert all(op.device_error() == 0 for op in ops)


@pytest.mark.parametrize("r,O", [(16, WIDE), (16, ODD), (64, WIDE)])
def test_another_stream_and_replay(lib, r, O):
    n = 1500
    op = holder(n, *adapters(5, r, 256, O))
    xs = [rows(n, 256, seed=k) for k in range(3)]
    ids = [choose(n, 5, seed=k, none=0.1) for k in range(3)]
    base = rows(n, O, seed=8)
    want = [op.forward(x, i, base) for x, i in zip(xs, ids)]
    for x, i, w in zip(xs, ids, want):
        check(op, x, i, base, w)
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


@pytest.mark.parametrize("where", ["x", "out", "base", "all"])
@pytest.mark.parametrize("r", [16, 72])
@pytest.mark.parametrize("t,y,O", [(BF, BF, 1024), (HF, F32, 104), (BF, HF, 131)])
def test_pinned_memory(lib, where, r, t, y, O):
    """Pinned x: runs of eight rows by the kernel for few rows.  Pinned base or out: the form for any rows, whatever their
    alignment."""
    n = 1500
    op = holder(n, *adapters(5, r, 256, O, t), out_dtype=y)
    x, idx, base = rows(n, 256, t), choose(n, 5, none=0.3), rows(n, O, y, seed=8)
    idx[:40] = -1
    pin = lambda v, name: v.cpu().pin_memory() if where in (name, "all") else v   # noqa: E731
    out = pin(torch.zeros(n, O, dtype=y, device="cuda"), "out")
    op.forward(pin(x, "x"), idx, pin(base, "base"), out=out)
    torch.cuda.synchronize()
    check(op, x, idx, base, out.cuda())
    keep = pin(base, "out").clone()
    keep = keep if keep.is_cuda else keep.pin_memory()
    op.forward(pin(x, "x"), idx, keep, out=keep)            # in place
    torch.cuda.synchronize()
    check(op, x, idx, base, keep.cuda())


@pytest.mark.parametrize("O", [40, 64])
def test_rows_past_32_bit_offsets(lib, O):
    n, K = 1100, 64
    stride = (1 << 31) // (n - 1) // 8 * 8 + 8
    try:
        xb = torch.empty(n * stride, dtype=BF, device="cuda")
        yb = torch.empty(n * stride, dtype=BF, device="cuda")
        bb = torch.empty(n * stride, dtype=BF, device="cuda")
    except torch.OutOfMemoryError:
        pytest.skip("needs 15 GB")
    op, idx = holder(n, *adapters(3, 40, K, O)), choose(n, 3)
    x, y, base = (v.view(n, stride)[:, :w] for v, w in ((xb, K), (yb, O), (bb, O)))
    x.copy_(rows(n, K))
    base.copy_(rows(n, O, seed=8))
    op.forward(x, idx, base, out=y)
    check(op, x.contiguous(), idx, base.contiguous(), y.contiguous())


def test_made_within_a_capture(lib):
    n = 1500
    a, b, s = adapters(5, 16, 256, WIDE)
    x, idx, base = rows(n, 256), choose(n, 5), rows(n, WIDE, seed=8)
    want = holder(n, a, b, s).forward(x, idx, base)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        op = holder(n, a, b, s)
        held = op.forward(x, idx, base)
    assert torch.equal(op.forward(x, idx, base), want)      # before the word was ever cleared
    for _ in range(2):
        held.fill_(7)
        g.replay()
        assert torch.equal(held, want) and op.device_error() == 0
