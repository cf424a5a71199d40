"""Listed pages that cannot be read: entries that are no candidates, candidates without a page in the table.  Whatever kernel a
step takes, their keys get no weight, every other key its own, and the status word is raised."""
import pytest
import torch

from chunked_prefill_paged_cpa_gb300 import ops
from select_support import limit_of, make_batch, reference
from test_gpu_selected import call, workspace
from window_support import tolerance

pytestmark = pytest.mark.gpu

# (q_lens, seq_lens, query heads, kv heads, budget, local): single tokens alone, in one CTA and over clusters; more pages than
# a cluster takes; single tokens and chunks in one queue, whole pairs and split ones; enough pairs that none is split; single
# tokens beside chunks; fp32 tiles whose keys are split and four to a CTA
STEPS = {
    "tokens": ([1] * 5, [500, 700, 300, 40, 1000], 8, 2, 6, 2),
    "tokens over clusters": ([1, 1], [1500, 1100], 4, 2, 60, 4),
    "one token, long list": ([1], [40000], 4, 1, 1100, 4),
    "queue": ([1, 40, 1, 300, 1], [500, 700, 90, 900, 2000], 8, 2, 20, 2),
    "one chunk": ([130], [20011], 8, 2, 100, 4),
    "whole pairs": ([700, 3], [1500, 600], 64, 8, 24, 1),
    "beside": ([1] * 30 + [200] + [1] * 34, [600 + 9 * i for i in range(65)], 16, 8, 28, 4),
}
# which entries of a list of n: one at either end, the first tile of 128 keys, every third, all
HOLES = {
    "first": lambda n: [0],
    "last": lambda n: [n - 1],
    "tile": lambda n: list(range(min(n, 8))),
    "third": lambda n: list(range(1, n, 3)),
    "all": lambda n: list(range(n)),
}


def verify(b, seen):
    """The call on ``b`` against the formula over the pages that ``seen`` lists."""
    ws = workspace(b)
    out = call(b, ws)
    want, size = reference(dict(b, selected=seen.to(out.device)))
    err = (out.double() - want).abs()
    assert (err <= tolerance(b, want, size)).all(), err.max()   # (NaN is not below)
    args = b["k_cache"], b["q"].shape[1], b["table"].shape[1], ws
    assert ops.device_status(*args) == ops.CPA_ERR_DEVICE
    assert ops.device_status(*args) == ops.CPA_OK


@pytest.mark.parametrize("mode", ["bf16", "f16", "bf16-e4m3", "f16-e4m3", "f32"])
@pytest.mark.parametrize("step", STEPS)
def test_entries_that_are_no_candidates(cuda_device, step, mode):
    q_lens, seq_lens, hq, hkv, budget, local = STEPS[step]
    for i, (holes, d) in enumerate(zip(HOLES, (64, 128, 64, 128, 64))):
        b = make_batch(q_lens, seq_lens, hq, hkv, d, mode, budget, local, 40 + i, cuda_device)
        told, seen = b["selected"].cpu(), b["selected"].cpu()
        for u, (_, t, _, x) in enumerate(b["units"]):
            limit = limit_of(x, local)
            if u % 3 == 2 or limit == 0:   # some units as they were
                continue
            for k, at in enumerate(HOLES[holes](min(limit, budget))):
                told[t, u % hkv, at] = (-1, limit, 1 << 30, -(1 << 31), limit + 1)[(u + k) % 5]
                seen[t, u % hkv, at] = limit   # (a page that the unit sees in any case)
        verify(dict(b, selected=told.to(cuda_device)), seen)


@pytest.mark.parametrize("mode", ["bf16", "f16-e4m3", "f32"])
@pytest.mark.parametrize("step", STEPS)
def test_candidates_without_a_page(cuda_device, step, mode):
    q_lens, seq_lens, hq, hkv, budget, local = STEPS[step]
    b = make_batch(q_lens, seq_lens, hq, hkv, 64, mode, budget, local, 60, cuda_device)
    table, seen, pages = b["table"].cpu(), b["selected"].cpu(), b["k_cache"].shape[0]
    gone = {}   # of every sequence some of its first unit's first list: columns before all its units' own pages
    for i, (s, t, _, x) in enumerate(b["units"]):
        limit = limit_of(x, local)
        k = min(limit, budget)
        if s not in gone:
            gone[s] = set(seen[t, 0, :k:2].tolist())
        for h in range(hkv):
            for at in range(k):
                if int(seen[t, h, at]) in gone[s]:
                    seen[t, h, at] = limit
    for s, columns in gone.items():
        for k, c in enumerate(sorted(columns)):
            table[s, c] = (-1, pages, 1 << 30, -(1 << 31))[(s + k) % 4]
    verify(dict(b, table=table.to(cuda_device)), seen)
