"""The bounded waits of the prompt kernel of windowed attention: faults that the device reports cost
no wait."""
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
