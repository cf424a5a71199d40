"""Page operators on tables that are not as they should be: reported, and nothing else is touched."""
import pytest
import torch

from chunked_prefill_paged_cpa_gb300 import ops
from pages_support import Pool
from test_gpu_pages import Device

pytestmark = pytest.mark.gpu


# rows, columns, pages of the pool: one cluster with the tables, one cluster and the tables behind it, three launches
@pytest.mark.parametrize("rows,columns,pages", [(6, 8, 60), (40, 300, 4000), (300, 500, 140_000)])
def test_compact_reports_an_entry_with_a_free_page_below_the_live_ones(cuda_device, rows, columns, pages):
    """The entry stays, the page is filled as if the entry were not there, the status word is raised."""
    g = torch.Generator().manual_seed(rows)
    lens = torch.randint(16, columns * 8, (rows - 2,), generator=g).tolist()
    pool = Pool.random(lens, rows, columns, pages, 4)
    pool.release([0, 2])
    live = sum(r > 0 for r in pool.refs)
    holes = [x for x, r in enumerate(pool.refs) if r == 0 and x < live]
    assert len(holes) > 2
    d = Device(pool, cuda_device)
    stale = [holes[0], holes[-1], holes[len(holes) // 2]]
    for c, x in zip((0, 3, columns - 1), stale):
        d.table[rows - 1, c] = x
    moves, m = pool.compact()
    d.compact()
    assert d.counts.tolist() == [len(moves), m] and d.pairs() == moves
    assert [int(d.table[rows - 1, c]) for c in (0, 3, columns - 1)] == stale
    assert d.status() == ops.CPA_ERR_DEVICE
    d.table[rows - 1] = -1
    d.same(pool)
    d.compact()
    assert d.status() == ops.CPA_OK


def test_extend_rows_that_need_more_pages_than_32_bits_count(cuda_device):
    """2048 rows that all claim the same 2^24 tokens need 2^31 pages: too few are free, and nothing changes."""
    rows, columns, tokens = 4096, 1 << 20, 1 << 24
    table = torch.full((rows, columns), -1, dtype=torch.int32, device=cuda_device)
    refs = torch.zeros(64, dtype=torch.int32, device=cuda_device)
    starts = torch.zeros(rows + 1, dtype=torch.int32, device=cuda_device)
    starts[1::2] = tokens  # (the rows between them have a negative count)
    lens = torch.full((rows,), tokens, dtype=torch.int32, device=cuda_device)
    slots = torch.zeros(tokens, dtype=torch.int64, device=cuda_device)
    src, dst = (torch.full((rows,), -7, dtype=torch.int32, device=cuda_device) for _ in range(2))
    counts = torch.zeros(2, dtype=torch.int32, device=cuda_device)
    ws = ops.pages_workspace_for(64, device=cuda_device)
    ops.extend_sequences(starts, lens, table, refs, slots, src, dst, counts, ws)
    assert counts.tolist() == [0, -2 ** 31 + 1]
    assert (slots == -1).all() and (refs == 0).all() and (src == -7).all() and (dst == -7).all()
    assert int(table.max()) == int(table.min()) == -1
    st = ops.CpaDesc(1, 1, 64, 16, 1, 1, 1, 0, ws.data_ptr(), ws.shape[0])
    assert ops.cpa_read_device_status(st, ops._stream(None)) == ops.CPA_ERR_DEVICE
