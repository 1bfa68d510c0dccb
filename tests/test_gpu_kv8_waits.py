"""Waits of the cache's attention that run out: one CTA copies none of its blocks (woq_tune_fault, with the
bound cut to one millisecond), so its own waits for them end.  The status says so, every row of the output
either keeps what it held or is right, and zero-filling the workspace restores a working state.  Nothing
traps, faults or waits without a bound."""
import pytest
import torch

from tests import kv8_model as M
from tests import test_gpu_kv8 as base
from tests.test_gpu_kv8 import DEV, Cache, gen, ints

pytestmark = pytest.mark.gpu

WAIT_US = 1000
woq = None


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    global woq
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import weight_only_quantised_gb300 as w
    woq = base.woq = w
    torch.cuda.set_device(0)
    yield
    woq.woq_tune_fault(0, 0, 0)


def one(dim, fmt):
    c = Cache(fmt=fmt, heads=4, dim=dim, max_tokens=9000, pages=150)
    g = gen(dim)
    c.prompt(0, g, 8990)
    return c, g, [0]


def many(dim, fmt):
    """More items than CTAs: shares that end inside an item."""
    c = Cache(fmt=fmt, heads=8, dim=dim, seqs=24, max_tokens=3000, pages=160)
    g = gen(dim)
    for s in range(24):
        c.prompt(s, g, 2999 if s == 9 else 90 + (37 * s) % 200)
    return c, g, list(range(24))


@pytest.mark.parametrize("cta", [0, 1, 40])
@pytest.mark.parametrize("make,dim,fmt,rows,group", [(one, 128, 0, 1, 5), (one, 128, 1, 8, 5), (one, 128, 0, 8, 16), (one, 256, 0, 1, 4),
                                                     (one, 64, 1, 3, 4), (many, 128, 1, 1, 4), (many, 128, 0, 3, 4), (many, 256, 1, 2, 4)])
def test_a_copy_that_never_comes(make, dim, fmt, rows, group, cta):
    c, g, seqs = make(dim, fmt)
    c.draft(seqs, g, rows)
    n, hq = len(seqs), c.heads * group
    ws = torch.zeros(woq.woq_kv8_attention_workspace(c.cfg, n, rows, hq), dtype=torch.uint8, device=DEV)
    # a launch that ends well leaves its parts in the workspace: of other queries
    c.attend(seqs, rows, group, g, ws=ws)
    q = (torch.randn((n * rows, hq, dim), generator=g) * 1.5).to(torch.bfloat16)
    out = torch.full((n * rows + 1, hq, dim), 7.0, dtype=torch.bfloat16, device=DEV)
    woq.woq_tune_fault(1, cta, WAIT_US)
    try:
        woq.woq_kv8_attention(c.cfg, c.buf, 0, ints(seqs), rows, q.to(DEV), hq, out[:-1], ws, 0.1)
        torch.cuda.synchronize()
    finally:
        woq.woq_tune_fault(0, 0, 0)
    assert woq.woq_read_status(c.buf, clear=True) == woq.WOQ_DEVERR_TIMEOUT
    got = out.cpu()
    kept = (got == 7).all(-1)  # rows x query heads
    assert kept[-1].all() and kept[:-1].any()
    for e, s in enumerate(seqs):
        ref, bound = M.attention(c.model[0][s], fmt, q[e * rows:(e + 1) * rows], [(2 << m) - 1 for m in range(rows)], 0.1)
        right = ((got[e * rows:(e + 1) * rows].double() - ref).abs() <= bound).all(-1)
        assert (right | kept[e * rows:(e + 1) * rows]).all(), f"entry {e}: a row that is neither right nor as it was"
    woq.woq_workspace_init(ws)
    c.attend(seqs, rows, group, g, ws=ws, q=q, scale=0.1)
