"""The bounded waits of the prompt kernel of windowed attention: faults that the device reports cost
no wait, and a wait that runs out ends the call with a status."""
import pytest
import torch

import query_aware_kv_gb300 as q
from test_gpu_window import BIG, check, make, ok

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def seeded():
    torch.manual_seed(0)


@pytest.mark.parametrize("n", [3, 300])
@pytest.mark.parametrize("entry", [-1, 2 ** 31 - 1])
def test_unmapped_pages_are_reported_without_a_wait(n, entry):
    """Every page of a long row unmapped: each is reported as it is fetched, and no wait of the
    call runs out (its limit is a second)."""
    cache = make([16000], 4, 2, 16, seed=1)
    ws = q.window_workspace(cache, n)
    qq = torch.randn((1, n, 4, 128), device="cuda").half()
    q.window_prefill(cache, qq, 4, BIG, ws)
    ok(ws)
    mapped = cache.block_table.clone()
    cache.block_table.fill_(entry)
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record()
    q.window_prefill(cache, qq, 4, BIG, ws)
    end.record()
    rc, detail = q.read_status(ws)
    assert rc == q.QUEST_ERR_BAD_PAGE and detail[0] == 0
    assert start.elapsed_time(end) < 300
    q.workspace_init(ws)
    cache.block_table.copy_(mapped)
    out, lse = q.window_prefill(cache, qq, 4, 999, ws)
    ok(ws)
    check(cache, qq, out, lse, 4, 999, True)


@pytest.mark.parametrize("lens,n,pps", [([3000, 40], 3, 0), ([3000, 40], 300, 0), ([3000, 700], 150, 16),
                                        ([100], 90, 0), ([4, 0], 2, 0)], ids=str)
def test_a_wait_that_runs_out_ends_the_call(lens, n, pps):
    """The last tile of values never comes: every wait ends at its limit (5 ms), the call reports it,
    and the next call on the same workspace and memory is right."""
    cache = make(lens, 8, 2, 16, seed=2)
    o = q.opts(pages_per_split=pps, wait_limit_ns=5_000_000, debug_flags=q.QUEST_DEBUG_WITHHOLD_VALUES)
    ws = q.window_workspace(cache, n, o)
    qq = torch.randn((len(lens), n, 8, 128), device="cuda").half()
    for _ in range(2):
        start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        start.record()
        q.window_prefill(cache, qq, 4, 2000, ws, o)
        end.record()
        rc, _ = q.read_status(ws)
        assert rc == q.QUEST_ERR_TIMEOUT
        assert 4 < start.elapsed_time(end) < 500
        q.workspace_init(ws)
    o = q.opts(pages_per_split=pps)
    out, lse = q.window_prefill(cache, qq, 4, 2000, ws, o)
    ok(ws)
    check(cache, qq, out, lse, 4, 2000, True)


def test_a_short_limit_is_no_limit_on_work():
    """A limit that bounds waits, far below the call's own time, changes nothing."""
    cache = make([9000] * 4, 32, 8, 16, seed=3)
    o = q.opts(wait_limit_ns=2_000_000)
    ws = q.window_workspace(cache, 2000, o)
    qq = torch.randn((4, 2000, 32, 128), device="cuda").half()
    want, want_lse = q.window_prefill(cache, qq, 4, BIG, ws)
    out, lse = q.window_prefill(cache, qq, 4, BIG, ws, o)
    ok(ws)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
