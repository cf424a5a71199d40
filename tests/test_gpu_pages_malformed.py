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
