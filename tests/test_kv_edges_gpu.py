"""The 4-bit key/value cache and its attention on a B200 where they are easily wrong."""
import math

import pytest
import torch

from test_kv_gpu import check, fill_cache, q4  # noqa: F401  (q4: the fixture)

pytestmark = pytest.mark.gpu


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("rows,length", [(2, 500), (14, 500), (150, 500), (130, 30000)])
def test_rows_that_are_nan_have_a_nan_log_sum_exp(q4, rows, length):
    """A NaN in a query: every score of its row is one (both kernels, and parts that are joined)."""
    g = torch.Generator().manual_seed(rows)
    c, table = fill_cache(q4, g, [length], 2, 128, 64, 64)
    q = torch.randn(rows, 4, 128, generator=g).half().cuda()
    bad = torch.zeros(rows, 4, dtype=torch.bool)
    for row, head in ((0, 1), (rows // 2, 3), (rows - 1, 0)):
        q[row, head, 5] = math.nan
        bad[row, head] = True
    out, lse = q4.kv_attention(q, c, table.cuda(), ints([length]), ints([0, rows]), return_lse=True)
    assert torch.equal(torch.isnan(lse).cpu(), bad) and torch.equal(torch.isnan(out).all(-1).cpu(), bad)
    assert torch.isfinite(lse).cpu()[~bad].all() and torch.isfinite(out).cpu()[~bad].all()


@pytest.mark.parametrize("name", ["k_state", "v_state"])
@pytest.mark.parametrize("rows,length", [(300, 300), (1000, 1000)])
def test_a_first_key_that_could_not_be_held_makes_every_log_sum_exp_nan(q4, rows, length, name):
    """Row 0 of a whole prompt attends to that key alone."""
    g = torch.Generator().manual_seed(rows)
    c, table = fill_cache(q4, g, [length], 2, 128, 64, 64)
    getattr(c, name)[int(table[0, 0]), 1, 0, 1, 0] = math.nan
    q = torch.randn(rows, 4, 128, generator=g).half().cuda()
    out, lse = q4.kv_attention(q, c, table.cuda(), ints([length]), ints([0, rows]), return_lse=True)
    assert torch.isnan(lse[:, 2:]).all() and torch.isnan(out[:, 2:]).all()
    assert torch.isfinite(lse[:, :2]).all() and torch.isfinite(out[:, :2]).all()



@pytest.mark.parametrize("rows,length", [(1, 300), (3, 40000), (12, 3000), (300, 700), (130, 30000)])
def test_waits_that_run_out_while_copies_are_on_their_way(q4, rows, length):
    """Limits around a copy's own time: any of the warps' waits may run out (a probe of a barrier blocks for a while
    itself, so none has to).  Every call returns, with the right result or with its status, and the next one is right."""
    g = torch.Generator().manual_seed(rows)
    c, table = fill_cache(q4, g, [length], 2, 64, 64, 64)
    q = torch.randn(rows, 4, 64, generator=g).half()
    args = (q.cuda(), c, table.cuda(), ints([length]), ints([0, rows]))
    want = q4.kv_attention(*args)
    try:
        for limit in (1, 300, 1000, 2000, 5000) * 4:
            q4.set_wait_limit_ns(limit)
            out = q4.kv_attention(*args)
            torch.cuda.synchronize()
            status = q4.last_device_status()
            assert status in (0, 2)
            assert status or torch.equal(out, want)
            q4.reset_workspaces()
            q4.clear_device_status()
    finally:
        q4.set_wait_limit_ns(0)
        q4.reset_workspaces()
        q4.clear_device_status()
    check(q4, c, table, [length], [rows], q, implicit=False)
