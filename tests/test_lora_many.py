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
    # A workspace's own word is the last call's.
    c, need = op.c_cfg, B.moe_lora_workspace_bytes(op.c_cfg, n)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    assert B.moe_lora(c, a, b, s, x, 256, idx, n, base, O, out, O, ws, need) == B.MOE_OK
    assert torch.equal(out, want) and B.moe_workspace_check(ws, need) == (B.MOE_OK, 0)
