"""Page summaries, their copies and the selection of pages: whole numbers, equal to the definition's on the host."""
import numpy as np
import pytest
import torch

from chunked_prefill_paged_cpa_gb300 import ops
from select_support import DTYPES, PAGE, limit_of, random_table, select, starts_of, summarise, units

pytestmark = pytest.mark.gpu

MODES = ["bf16", "f16", "f32", "e4m3"]


def random_cache(pages, hkv, d, mode, seed, device):
    g = torch.Generator().manual_seed(seed)
    # scales that differ from page to page and head to head
    x = torch.randn(pages, hkv, PAGE, d, generator=g) * torch.exp(2 * torch.randn(pages, hkv, 1, 1, generator=g))
    if mode == "e4m3":
        return (x * 16).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).to(device)
    return x.to(DTYPES[mode]).to(device)


def step_tensors(q_lens, seq_lens, pages, seed, device, columns=None):
    table = random_table(seq_lens, pages, seed, columns)
    return table, (table.to(device), starts_of(q_lens).to(device), torch.tensor(seq_lens, dtype=torch.int32, device=device))


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("hkv,d", [(1, 64), (3, 128), (8, 128), (2, 64)])
def test_summaries(cuda_device, mode, hkv, d):
    """Only the pages that the step completes change: single tokens at every place of a page, chunks that complete none, one
    and several, a sequence without tokens."""
    q_lens = [1] * 17 + [0, 5, 16, 40, 17, 15, 100, 33]
    seq_lens = [32 + i for i in range(17)] + [64, 7, 16, 40, 48, 31, 130, 80]
    pages = sum(-(-n // PAGE) for n in seq_lens) + 3
    cache = random_cache(pages, hkv, d, mode, 1, cuda_device)
    table, where = step_tensors(q_lens, seq_lens, pages, 2, cuda_device)
    rows = torch.randint(0, 256, (pages, hkv, 2 * d + 16), dtype=torch.uint8, generator=torch.Generator().manual_seed(3))
    summaries = rows.to(cuda_device)
    ops.summarise_pages(cache, *where, summaries)
    want = summarise(cache, table, q_lens, seq_lens, rows.numpy())
    assert np.array_equal(summaries.cpu().numpy(), want)
    # and a sequence's whole again
    ops.summarise_pages(cache, where[0], starts_of(seq_lens).to(cuda_device), where[2], summaries)
    assert np.array_equal(summaries.cpu().numpy(), summarise(cache, table, seq_lens, seq_lens, want))


@pytest.mark.parametrize("mode", MODES)
def test_summaries_of_odd_keys(cuda_device, mode):
    """NaN, infinities, zeros of both signs, the smallest and the largest magnitudes, halves between two codes."""
    d, hkv = 64, 2
    cache = random_cache(16, hkv, d, mode, 4, cuda_device)
    if mode == "e4m3":
        cache[0, 0, 3, 5], cache[1, 1, 0, 0], cache[2] = 0x7F, 0xFF, 0x80
        cache[3], cache[4] = 1, 0x7E                   # the smallest and the largest value everywhere
    else:
        tiny = torch.finfo(cache.dtype).tiny
        cache[0, 0, 3, 5], cache[1, 1, 0, 0], cache[2, 0, 15, 63], cache[3], cache[4] = float("nan"), float("inf"), -float("inf"), -0.0, 0.0
        cache[5], cache[6], cache[7], cache[8] = tiny, torch.finfo(cache.dtype).max, -torch.finfo(cache.dtype).max, tiny / 4
        cache[9] = 1.0
        cache[9, 0, 0, :63] = (torch.arange(63, device=cuda_device) + 0.5).to(cache.dtype)
        cache[9, 0, 1, 63] = 127.0
    table = torch.arange(16, dtype=torch.int32).view(1, 16)
    where = (table.to(cuda_device), starts_of([256]).to(cuda_device), torch.tensor([256], dtype=torch.int32, device=cuda_device))
    summaries = ops.summaries_for(cache)
    ops.summarise_pages(cache, *where, summaries)
    assert np.array_equal(summaries.cpu().numpy(), summarise(cache, table, [256], [256], np.zeros(summaries.shape, np.uint8)))


def test_summaries_of_many_sequences_and_large_pools(cuda_device):
    """4096 sequences; a page whose bytes lie beyond 32 bits."""
    q_lens, seq_lens = [1] * 4096, [16 * (1 + i % 3) - (i % 7 == 0) for i in range(4096)]
    pages = sum(-(-n // PAGE) for n in seq_lens)
    cache = random_cache(pages, 1, 64, "bf16", 5, cuda_device)
    table, where = step_tensors(q_lens, seq_lens, pages, 6, cuda_device)
    summaries = ops.summaries_for(cache)
    ops.summarise_pages(cache, *where, summaries)
    assert np.array_equal(summaries.cpu().numpy(), summarise(cache, table, q_lens, seq_lens, np.zeros(summaries.shape, np.uint8)))
    pages = 2 ** 33 // (8 * PAGE * 128 * 2) + 10
    cache = torch.empty(pages, 8, PAGE, 128, dtype=torch.bfloat16, device=cuda_device)
    far = pages - 3
    cache[far].normal_()
    table = torch.tensor([[far]], dtype=torch.int32)
    summaries = torch.zeros(pages, 8, 272, dtype=torch.uint8, device=cuda_device)
    ops.summarise_pages(cache, table.to(cuda_device), starts_of([1]).to(cuda_device), torch.tensor([16], dtype=torch.int32, device=cuda_device), summaries)
    want = summarise(cache[far:far + 1], torch.tensor([[0]]), [1], [16], np.zeros((1, 8, 272), np.uint8))
    assert np.array_equal(summaries[far:far + 1].cpu().numpy(), want)
    assert int(summaries.sum(dtype=torch.int64)) == int(want.astype(np.int64).sum())


def test_summaries_copied(cuda_device):
    g = torch.Generator().manual_seed(7)
    for hkv, d in ((1, 64), (8, 128), (3, 64)):
        rows = torch.randint(0, 256, (50, hkv, 2 * d + 16), dtype=torch.uint8, generator=g)
        order = torch.randperm(50, generator=g).to(torch.int32)
        src, dst = order[:20], order[20:40]
        for n in (None, 0, 7, 20, 99):
            summaries = rows.to(cuda_device)
            count = None if n is None else torch.tensor([n], dtype=torch.int32, device=cuda_device)
            ops.copy_summaries(src.to(cuda_device), dst.to(cuda_device), summaries, num_pairs=count)
            want, k = rows.clone(), 20 if n is None else min(n, 20)
            want[dst[:k].long()] = rows[src[:k].long()]
            assert torch.equal(summaries.cpu(), want)
    ws = torch.zeros(256, dtype=torch.uint8, device=cuda_device)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=cuda_device)  # noqa: E731
    before = summaries.clone()
    ops.copy_summaries(i32(-1, 3, 50), i32(4, 50, 1), summaries, workspace=ws)
    assert torch.equal(summaries, before) and int(ws[0]) == 1


def run_select(q, rows, where, table, q_lens, seq_lens, budget, sinks, local, device, **kw):
    hkv = rows.shape[1]
    selected = torch.full((q.shape[0], hkv, budget), -7, dtype=torch.int32, device=device)
    ops.select_pages(q, torch.as_tensor(rows).to(device), *where, selected, sink_pages=sinks, local_pages=local, **kw)
    want = select(q, rows, table, q_lens, seq_lens, budget, sinks, local, np.full(selected.shape, -7, np.int32))
    got = selected.cpu().numpy()
    assert np.array_equal(got, want)
    return got


def random_rows(pages, hkv, d, seed):
    g = torch.Generator().manual_seed(seed)
    codes = torch.randint(-127, 128, (pages, hkv, 2 * d), dtype=torch.int8, generator=g).view(torch.uint8)
    scale = torch.exp(torch.randn(pages, hkv, 1, generator=g))
    return torch.cat([codes, scale.view(torch.uint8), torch.zeros(pages, hkv, 12, dtype=torch.uint8)], 2).numpy()


@pytest.mark.parametrize("mode", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("hq,hkv,d", [(4, 4, 64), (4, 2, 128), (8, 2, 64), (16, 2, 128)])
def test_selection(cuda_device, mode, hq, hkv, d):
    q_lens = [1, 1, 1, 1, 2, 300, 1, 70, 1, 257, 33]
    seq_lens = [1, 16, 17, 1000, 40, 900, 2000, 70, 33, 1300, 4000]
    pages = sum(-(-n // PAGE) for n in seq_lens) + 2
    rows = random_rows(pages, hkv, d, 1)
    table, where = step_tensors(q_lens, seq_lens, pages, 2, cuda_device)
    q = torch.randn(sum(q_lens), hq, d, generator=torch.Generator().manual_seed(3)).to(DTYPES[mode]).to(cuda_device)
    for budget, sinks, local in ((1, 0, 1), (4, 1, 2), (9, 4, 1), (16, 30, 3), (64, 2, 1), (300, 1, 4)):
        run_select(q, rows, where, table, q_lens, seq_lens, budget, sinks, local, cuda_device)


def test_ties_go_to_the_lower_page(cuda_device):
    """Equal pages, queries of zeros and of what is not finite, scores of both zeros, infinite scales."""
    lens, hkv, d = [1700, 1700, 1700, 1700, 33 * 16], 2, 64
    pages = sum(-(-n // PAGE) for n in lens)
    rows = random_rows(pages, hkv, d, 4)
    rows[:, 0] = rows[0, 0]                       # all pages alike in head 0
    rows[::3, 1] = rows[1, 1]                     # some in head 1
    inf = np.array([np.inf], np.float32).view(np.uint8)
    rows[5:pages:17, 1, 2 * d:2 * d + 4] = inf
    rows[7:pages:13, 1, 2 * d:2 * d + 4] = 0      # a scale of zero: scores of both zeros
    table, where = step_tensors([1] * 5, lens, pages, 5, cuda_device)
    q = torch.randn(5, 4, d, generator=torch.Generator().manual_seed(6)).to(cuda_device)
    q[1], q[2, 0, 3], q[2, 3, 5], q[3] = 0, float("nan"), float("inf"), q[3] * 2.0 ** -110
    for budget, sinks in ((1, 0), (10, 0), (40, 3), (90, 0)):
        got = run_select(q, rows, where, table, [1] * 5, lens, budget, sinks, 2, cuda_device)
        assert got[1, 0].tolist() == list(range(budget))


def test_scores_past_the_largest_number(cuda_device):
    """Scales whose products are infinite: both infinities order like numbers."""
    rows = random_rows(200, 1, 64, 7)
    rows[::2, 0, 128:132] = np.array([3e38], np.float32).view(np.uint8)
    table, where = step_tensors([1], [200 * 16], 200, 8, cuda_device)
    q = torch.randn(1, 1, 64, generator=torch.Generator().manual_seed(9)).to(cuda_device)
    for budget in (1, 30, 60, 150, 190):
        run_select(q, rows, where, table, [1], [200 * 16], budget, 0, 1, cuda_device)


@pytest.mark.parametrize("length,columns", [(100003, None), (500, 20000), (30000, 260000)])
def test_long_contexts_and_wide_tables(cuda_device, length, columns):
    """Candidates over the CTAs of a cluster; columns that no context reaches."""
    pages = -(-length // PAGE) + 1
    rows = random_rows(pages, 2, 128, 10)
    for q_lens in ([1], [40]):
        table, where = step_tensors(q_lens, [length], pages, 11, cuda_device, columns)
        q = torch.randn(q_lens[0], 8, 128, generator=torch.Generator().manual_seed(12)).bfloat16().to(cuda_device)
        for budget, local in ((1, 1), (128, 4), (3333, 2)):
            run_select(q, rows, where, table, q_lens, [length], budget, 1, local, cuda_device)


@pytest.mark.parametrize("d", [64, 128])
def test_fewer_pages_than_a_cluster_has_warps(cuda_device, d):
    """CTAs and warps without a page beside others with some."""
    for length in (100, 300, 520, 900, 2300):
        pages = -(-length // PAGE)
        rows = random_rows(pages, 1, d, length)
        table, where = step_tensors([1], [length], pages, 30, cuda_device, 20000)
        q = torch.randn(1, 4, d, generator=torch.Generator().manual_seed(31)).bfloat16().to(cuda_device)
        for budget in (1, 3, 17):
            for _ in range(5):
                run_select(q, rows, where, table, [1], [length], budget, 1, 2, cuda_device)


def test_summaries_beyond_32_bit_offsets(cuda_device):
    rows = random_rows(100, 8, 128, 27)
    far = 2 ** 32 // (8 * 272) + 10
    table, where = step_tensors([1, 30], [1000, 500], 100, 28, cuda_device)
    pool = torch.empty(far + 100, 8, 272, dtype=torch.uint8, device=cuda_device)
    pool[far:] = torch.as_tensor(rows).to(cuda_device)
    q = torch.randn(31, 16, 128, generator=torch.Generator().manual_seed(29)).bfloat16().to(cuda_device)
    got = torch.full((31, 8, 5), -7, dtype=torch.int32, device=cuda_device)
    ops.select_pages(q, pool, torch.where(where[0] >= 0, where[0] + far, -1), *where[1:], got, sink_pages=1, local_pages=2)
    want = select(q, rows, table, [1, 30], [1000, 500], 5, 1, 2, np.full(got.shape, -7, np.int32))
    assert np.array_equal(got.cpu().numpy(), want)


def test_many_rows(cuda_device):
    """More units than the GPU holds at a time; 4000 sequences."""
    lens = [40 + 7 * (i % 90) for i in range(4000)]
    rows = random_rows(64, 1, 64, 13)
    table = torch.randint(0, 64, (4000, 48), generator=torch.Generator().manual_seed(14), dtype=torch.int32)   # pages shared by many
    where = (table.to(cuda_device), starts_of([1] * 4000).to(cuda_device), torch.tensor(lens, dtype=torch.int32, device=cuda_device))
    q = torch.randn(4000, 2, 64, generator=torch.Generator().manual_seed(15)).half().to(cuda_device)
    run_select(q, rows, where, table, [1] * 4000, lens, 8, 1, 2, cuda_device)


@pytest.mark.parametrize("hq", [1, 8])
def test_units_of_long_chunks(cuda_device, hq):
    """Many units per chunk, chunks that begin and end anywhere, short last units of one token and of all but one."""
    size = 256 // hq
    q_lens = [3 * size + 1, 1, 5 * size - 1, 2 * size, size + 1, 1, 2000, size - 1]
    seq_lens = [q + o for q, o in zip(q_lens, [700, 90, 0, 1300, 15, 800, 333, 2000])]
    pages = sum(-(-n // PAGE) for n in seq_lens)
    rows = random_rows(pages, 1, 64, 24)
    table, where = step_tensors(q_lens, seq_lens, pages, 25, cuda_device)
    q = torch.randn(sum(q_lens), hq, 64, generator=torch.Generator().manual_seed(26)).bfloat16().to(cuda_device)
    run_select(q, rows, where, table, q_lens, seq_lens, 6, 1, 2, cuda_device)


def test_bad_entries_raise_the_status_word(cuda_device):
    rows = random_rows(60, 2, 64, 16)
    table, where = step_tensors([1, 1], [500, 400], 60, 17, cuda_device)
    table[0, 3], table[1, 4], table[1, 7] = -1, 60, 1 << 30
    where = (table.to(cuda_device), *where[1:])
    ws = torch.zeros(256, dtype=torch.uint8, device=cuda_device)
    q = torch.randn(2, 4, 64, generator=torch.Generator().manual_seed(18)).bfloat16().to(cuda_device)
    for budget in (5, 20, 23):
        run_select(q, rows, where, table, [1, 1], [500, 400], budget, 0, 1, cuda_device, workspace=ws)
        assert int(ws[0]) == 1
        ws.zero_()
    # a length past the table: no more than the table's columns
    where = (where[0], where[1], torch.tensor([500, 100000], dtype=torch.int32, device=cuda_device))
    selected = torch.zeros(2, 2, 5, dtype=torch.int32, device=cuda_device)
    ops.select_pages(q, torch.as_tensor(rows).to(cuda_device), *where, selected, workspace=ws)
    assert int(ws[0]) == 1 and int(selected.max()) < table.shape[1]
    cache = random_cache(60, 2, 64, "bf16", 19, cuda_device)
    summaries = ops.summaries_for(cache)
    ws.zero_()
    ops.summarise_pages(cache, *where, summaries, workspace=ws)   # (none of the table's pages is completed)
    assert int(ws[0]) == 1 and not summaries.any()
    ws.zero_()
    ops.summarise_pages(cache, where[0], starts_of([500, 300]).to(cuda_device), torch.tensor([500, 400], dtype=torch.int32, device=cuda_device), summaries, workspace=ws)
    assert int(ws[0]) == 1
    assert np.array_equal(summaries.cpu().numpy(), summarise(cache, table, [500, 300], [500, 400], np.zeros(summaries.shape, np.uint8)))


def test_the_score_is_a_bound(cuda_device):
    """What the whole numbers stand for: no key of a page has a larger logit than its bounds allow, but for the codes'
    roundings.  A code is off by half a step: hi and lo by scale / 2 and 2^-22 of themselves each, q by a / 254 and the same;
    d products of |q| <= a and |hi| <= 127 scale: |score * a / 127 - bound| <= d (a scale / 2 + 127 scale a / 254 + ...) < 1.02 d a scale."""
    d, n = 64, 40
    cache = random_cache(n, 1, d, "f32", 20, cuda_device)
    table, where = torch.arange(n, dtype=torch.int32).view(1, n), None
    where = (table.to(cuda_device), starts_of([n * PAGE]).to(cuda_device), torch.tensor([n * PAGE], dtype=torch.int32, device=cuda_device))
    summaries = ops.summaries_for(cache)
    ops.summarise_pages(cache, *where, summaries)
    rows = summaries.cpu().numpy()[:, 0]
    codes, scale = rows[:, :2 * d].view(np.int8).astype(np.float64), rows[:, 2 * d:2 * d + 4].copy().view(np.float32)[:, 0].astype(np.float64)
    q = torch.randn(d, generator=torch.Generator().manual_seed(21)).double().numpy()
    a = np.abs(q).max()
    c = np.rint(q * 127 / a)
    score = scale * (codes[:, :d] @ np.maximum(c, 0) + codes[:, d:] @ np.minimum(c, 0)) * a / 127
    logits = (cache[:, 0].double().cpu().numpy() @ q).max(1)
    assert (logits <= score + 1.02 * d * a * scale).all()


@pytest.mark.parametrize("budget,local", [(4, 1), (24, 2)])
def test_capture(cuda_device, budget, local):
    """Append, summaries, selection and attention captured together and replayed on a second step's tokens."""
    dev, hq, hkv, d, lens0 = cuda_device, 8, 2, 64, [100, 47, 640, 31, 15]
    pages, g = 200, torch.Generator().manual_seed(22)
    table = random_table([n + 80 for n in lens0], pages, 23).to(dev)
    caches = [torch.full((pages, hkv, PAGE, d), float("nan"), dtype=torch.bfloat16, device=dev) for _ in range(2)]
    summaries = ops.summaries_for(caches[0])
    ws = ops.workspace_for(caches[0], hq, table.shape[1], 5, 1000)
    said = [torch.randn(2, n + 2 * 40, hkv, d, generator=g).bfloat16().to(dev) for n in lens0]

    def tokens(q_lens, at):
        slots = torch.cat([table[s, (p := torch.arange(a, a + q, device=dev)) // PAGE].long() * PAGE + p % PAGE for s, (q, a) in enumerate(zip(q_lens, at))])
        new = [torch.cat([said[s][i, a:a + q] for s, (q, a) in enumerate(zip(q_lens, at))]) for i in range(2)]
        return new, slots

    new, slots = tokens(lens0, [0] * 5)
    ops.kv_append(*new, slots, *caches)
    ops.summarise_pages(caches[0], table, starts_of(lens0).to(dev), torch.tensor(lens0, dtype=torch.int32, device=dev), summaries)
    q_lens = [1, 40, 1, 2, 1]
    T = sum(q_lens)
    at = {"q": torch.zeros(T, hq, d, dtype=torch.bfloat16, device=dev), "k": torch.zeros(T, hkv, d, dtype=torch.bfloat16, device=dev),
          "v": torch.zeros(T, hkv, d, dtype=torch.bfloat16, device=dev), "slots": torch.full((T,), -1, device=dev),
          "lens": torch.tensor([n + q for n, q in zip(lens0, q_lens)], dtype=torch.int32, device=dev)}
    starts, out = starts_of(q_lens).to(dev), torch.zeros(T, hq, d, dtype=torch.bfloat16, device=dev)
    selected = torch.full((T, hkv, budget), -1, dtype=torch.int32, device=dev)

    def step():
        where = (table, starts, at["lens"])
        ops.kv_append(at["k"], at["v"], at["slots"], *caches, ws)
        ops.summarise_pages(caches[0], *where, summaries, workspace=ws)
        ops.select_pages(at["q"], summaries, *where, selected, sink_pages=1, local_pages=local, workspace=ws)
        ops.selected_attention_forward(at["q"], *caches, *where, d ** -0.5, ws, selected, local, out=out)

    step()          # no token is written: the slots are -1
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    for n in range(2):
        before = [a + n * q for a, q in zip(lens0, q_lens)]
        seq_lens = [a + q for a, q in zip(before, q_lens)]
        new, new_slots = tokens(q_lens, before)
        at["k"].copy_(new[0]), at["v"].copy_(new[1]), at["slots"].copy_(new_slots)
        at["lens"].copy_(torch.tensor(seq_lens, dtype=torch.int32))
        at["q"].copy_(torch.randn(T, hq, d, generator=g))
        graph.replay()
        rows = summaries.cpu().numpy()
        want = select(at["q"], rows, table.cpu(), q_lens, seq_lens, budget, 1, local, np.full(selected.shape, -1, np.int32))
        assert np.array_equal(selected.cpu().numpy(), want)
        # every complete page's summary is there
        full = summarise(caches[0], table.cpu(), seq_lens, seq_lens, rows)
        assert np.array_equal(full, rows)
        for s, t, count, x in units(q_lens, seq_lens, 4):
            limit = limit_of(x, local)
            pos, j = x + torch.arange(count, device=dev), torch.arange(seq_lens[s], device=dev)
            for h in range(hkv):
                listed = torch.zeros(-(-seq_lens[s] // PAGE), dtype=torch.bool, device=dev)
                listed[selected[t, h, :min(limit, budget)].long()] = True
                mask = (j <= pos[:, None]) & ((j >= limit * PAGE) | listed[j // PAGE])
                k, v = (said[s][i, :seq_lens[s], h].double() for i in range(2))
                for i in range(4 * h, 4 * h + 4):
                    p = torch.softmax((d ** -0.5 * at["q"][t:t + count, i].double() @ k.T).masked_fill(~mask, float("-inf")), -1)
                    err = (out[t:t + count, i].double() - p @ v).abs()
                    # the output's rounding, the weights', fp32 arithmetic (window_support.tolerance)
                    assert (err <= 2.0 ** -8 * (p @ v).abs() + (2.0 ** -8 + 2.0 ** -13) * (p @ v.abs())).all()
    assert ops.device_status(caches[0], hq, table.shape[1], ws) == ops.CPA_OK
