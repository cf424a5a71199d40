"""The page operators on the GPU against their definitions, one step at a time; all values are whole numbers or copied bits."""
import pytest
import torch

from chunked_prefill_paged_cpa_gb300 import ops
from pages_support import PAGE, Pool
from window_support import visible

pytestmark = pytest.mark.gpu


def i32(x, dev):
    return torch.tensor(x, dtype=torch.int32, device=dev)


class Device:
    """A Pool's state on the GPU, and its workspace."""

    def __init__(self, pool, dev):
        self.dev = dev
        self.table, self.lens, self.refs = pool.to(dev)
        self.ws = ops.pages_workspace_for(len(pool.refs), device=dev)
        self.src, self.dst = (torch.full((max(len(pool.refs), len(pool.lens)),), -7, dtype=torch.int32, device=dev) for _ in range(2))
        self.counts = torch.zeros(2, dtype=torch.int32, device=dev)

    def same(self, pool):
        pool.check()
        assert self.refs.tolist() == pool.refs
        assert self.table.tolist() == pool.table
        assert self.lens.tolist() == pool.lens

    def status(self):
        return ops.cpa_read_device_status(ops.CpaDesc(1, 1, 64, 16, 1, 1, 1, 0, self.ws.data_ptr(), self.ws.shape[0]),
                                          ops._stream(None))

    def fork(self, parents, children):
        ops.fork_sequences(i32(parents, self.dev), i32(children, self.dev), self.table, self.lens, self.refs, self.ws)

    def extend(self, q_lens, tokens=None):
        starts = torch.zeros(len(q_lens) + 1, dtype=torch.int32)
        starts[1:] = torch.cumsum(torch.tensor(q_lens, dtype=torch.int32), 0)
        slots = torch.full((sum(q_lens) if tokens is None else tokens,), -9, dtype=torch.int64, device=self.dev)
        ops.extend_sequences(starts.to(self.dev), self.lens, self.table, self.refs, slots, self.src, self.dst, self.counts, self.ws)
        return slots

    def pairs(self):
        n = int(self.counts[0])
        assert (self.src[n:] == -7).all() and (self.dst[n:] == -7).all()  # nothing behind the list
        out = list(zip(self.src[:n].tolist(), self.dst[:n].tolist()))
        self.src.fill_(-7), self.dst.fill_(-7)
        return out

    def release(self, rows, window=0, sinks=0):
        ops.release_pages(None if rows is None else i32(rows, self.dev), self.table, self.lens, self.refs, self.ws, window, sinks)

    def compact(self):
        ops.compact_pages(self.table, self.refs, self.src, self.dst, self.counts, self.ws)


# ---- copies

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32, torch.uint8])
@pytest.mark.parametrize("hkv,d", [(1, 64), (3, 64), (8, 128), (5, 128)])
@pytest.mark.parametrize("pairs", [1, 7, 300])
def test_copy(cuda_device, dtype, hkv, d, pairs):
    g = torch.Generator(cuda_device).manual_seed(pairs + hkv)
    shape = (2 * pairs + 3, hkv, PAGE, d)
    bits = [torch.randint(0, 256, (*shape[:3], d * dtype.itemsize), generator=g, device=cuda_device, dtype=torch.uint8) for _ in range(2)]
    caches = [b.clone().view(dtype) for b in bits]
    order = torch.randperm(shape[0], generator=g, device=cuda_device).int()
    src, dst = order[:pairs].contiguous(), order[pairs:2 * pairs].contiguous()
    ops.copy_pages(src, dst, *caches)
    for b, c in zip(bits, caches):
        b[dst.long()] = b[src.long()]
        assert torch.equal(c.view(torch.uint8), b)


def test_copy_counts_on_the_device(cuda_device):
    c0 = torch.arange(40, device=cuda_device).view(40, 1, 1, 1).expand(40, 2, PAGE, 64).float().contiguous()
    src, dst = torch.arange(10, device=cuda_device).int(), torch.arange(20, 30, device=cuda_device).int()
    for n in (-3, 0, 4, 10, 99):
        k, v = c0.clone(), c0.clone() + 1
        ops.copy_pages(src, dst, k, v, num_pairs=i32([n, 77], cuda_device))
        m = min(max(n, 0), 10)
        assert k[:, 0, 0, 0].tolist() == list(range(20)) + list(range(m)) + list(range(20 + m, 40))
        assert torch.equal(v, k + 1)


def test_copy_skips_and_reports_bad_pages(cuda_device):
    k = torch.arange(8, device=cuda_device).view(8, 1, 1, 1).expand(8, 2, PAGE, 64).bfloat16().contiguous()
    v, ws = k.clone(), ops.pages_workspace_for(8, device=cuda_device)
    ops.copy_pages(i32([0, -1, 2, 8, 3], cuda_device), i32([4, 5, 8, 6, 7], cuda_device), k, v, workspace=ws)
    assert k[:, 1, 3, 5].tolist() == [0, 1, 2, 3, 0, 5, 6, 3] and torch.equal(k, v)
    st = ops.CpaDesc(1, 1, 64, 16, 1, 1, 1, 0, ws.data_ptr(), ws.shape[0])
    assert ops.cpa_read_device_status(st, ops._stream(None)) == ops.CPA_ERR_DEVICE
    ops.copy_pages(i32([], cuda_device), i32([], cuda_device), k, v)  # no pairs


# ---- tables

@pytest.mark.parametrize("rows,forks,columns", [(1, 1, 1), (3, 5, 70), (40, 100, 300), (1, 400, 1100)])
def test_fork(cuda_device, rows, forks, columns):
    g = torch.Generator().manual_seed(rows)
    lens = torch.randint(0, columns * PAGE + 1, (rows,), generator=g).tolist()
    pool = Pool.random(lens, rows + forks, columns, rows * columns + 5, 3, shared=0.5)
    d = Device(pool, cuda_device)
    parents = torch.randint(0, rows, (forks,), generator=g).tolist()
    children = (rows + torch.randperm(forks, generator=g)).tolist()
    assert not pool.fork(parents, children)
    d.fork(parents, children)
    d.same(pool)
    assert d.status() == ops.CPA_OK


def test_fork_refuses_rows_it_cannot_fork(cuda_device):
    pool = Pool.random([30, 40, 50], 9, 5, 20, 1)
    d = Device(pool, cuda_device)
    # a held row, a child named twice, a child that is a parent, itself, rows that are none; the last one is good
    parents = [0, 1, 2, 1, 6, 0, -1, 9, 2]
    children = [1, 3, 3, 6, 5, 0, 7, 7, 4]
    assert pool.fork(parents, children)
    d.fork(parents, children)
    d.same(pool)
    assert pool.lens[4] == 50 and d.status() == ops.CPA_ERR_DEVICE


@pytest.mark.parametrize("seed", range(6))
def test_extend(cuda_device, seed):
    """Rows that share pages, take no, one or many tokens, on pools of one piece of the search and of several."""
    g = torch.Generator().manual_seed(seed)
    r = lambda lo, hi: int(torch.randint(lo, hi + 1, (1,), generator=g))  # noqa: E731
    rows, columns = [1, 5, 40, 300, 1500, 64][seed], [6, 30, 200, 12, 8, 600][seed]
    pages = [40, 100, 20_000, 9_000, 300_000, 40_000][seed]
    parents = max(1, rows // 3)
    lens = [r(1, columns * PAGE // 2) for _ in range(parents)]
    pool = Pool.random(lens, rows, columns, pages, seed)
    d = Device(pool, cuda_device)
    kids = list(range(parents, rows))
    who = [r(0, parents - 1) for _ in kids]
    if kids:
        pool.fork(who, kids)
        d.fork(who, kids)
    for step in range(3):
        q = [r(0, 3) if r(0, 9) else r(0, columns * PAGE - n - 20 * (2 - step)) if columns * PAGE - n > 50 else 0 for n in pool.lens]
        q = [max(0, min(x, columns * PAGE - n)) for x, n in zip(q, pool.lens)]
        pool.lens = [n + x for n, x in zip(pool.lens, q)]
        d.lens.copy_(i32(pool.lens, cuda_device))
        slots, pairs, taken = pool.extend(q)
        got = d.extend(q)
        if slots is None:
            assert got.tolist() == [-1] * len(got) and d.counts.tolist() == [0, -taken]
            assert d.status() == ops.CPA_ERR_DEVICE
            d.same(pool)
            break
        assert d.counts.tolist() == [len(pairs), taken]
        assert got.tolist() == slots
        assert d.pairs() == pairs
        d.same(pool)
        assert d.status() == ops.CPA_OK
        slots_seen = [x for x in slots if x >= 0]
        assert len(set(slots_seen)) == len(slots_seen)  # no two tokens in one place


def test_extend_last_writer_keeps_the_shared_page(cuda_device):
    pool = Pool.random([20, 32], 6, 4, 30, 2)
    d = Device(pool, cuda_device)
    for p in (pool, d):
        p.fork([0, 0, 1], [2, 3, 4])
    # rows 0 and 3 write to the shared page, row 2 does not: both copy; then row 2 alone holds it and writes in place
    for q in ([1, 0, 0, 2, 0, 0], [0, 1, 1, 0, 1, 0]):
        pool.lens = [n + x for n, x in zip(pool.lens, q)]
        d.lens.copy_(i32(pool.lens, cuda_device))
        slots, pairs, taken = pool.extend(q)
        assert d.extend(q).tolist() == slots and d.pairs() == pairs and d.counts.tolist() == [len(pairs), taken]
        d.same(pool)
    assert taken == 2 and not pairs


def test_extend_after_rows_were_set_back(cuda_device):
    """Rows whose length went back hold pages behind it; where others hold them too, new tokens do not go there."""
    pool = Pool.random([150, 64, 40, 500], 12, 40, 120, 6)
    d = Device(pool, cuda_device)
    for p in (pool, d):
        p.fork([0, 0, 1, 2, 3, 3], [4, 5, 6, 7, 8, 9])
    #      set back inside a page, to a page's edge, to nothing, not at all
    lens = [20, 48, 0, 500, 150, 32, 64, 40, 17, 400, 0, 0]
    pool.lens = list(lens)
    for q in ([40, 20, 30, 1, 1, 1, 0, 3, 300, 90, 5, 0], [1] * 12):
        pool.lens = [n + x for n, x in zip(pool.lens, q)]
        d.lens.copy_(i32(pool.lens, cuda_device))
        slots, pairs, taken = pool.extend(q)
        assert slots is not None
        assert d.extend(q).tolist() == slots and d.counts.tolist() == [len(pairs), taken] and d.pairs() == pairs
        d.same(pool)
        assert len(set(slots)) == len(slots)
    assert d.status() == ops.CPA_OK


def test_extend_a_row_without_its_partly_filled_page(cuda_device):
    pool = Pool.random([20, 20], 2, 30, 60, 6)
    for r in range(2):
        pool.refs[pool.table[r][1]] = 0
        pool.table[r][1] = -1
    d = Device(pool, cuda_device)
    pool.lens = [21, 320]
    d.lens.copy_(i32(pool.lens, cuda_device))
    slots, pairs, taken = pool.extend([1, 300])
    assert d.extend([1, 300]).tolist() == slots and d.counts.tolist() == [0, taken] and not pairs
    d.same(pool)


def test_extend_too_few_pages_changes_nothing(cuda_device):
    pool = Pool.random([16, 20], 4, 5, 6, 2)
    d = Device(pool, cuda_device)
    for p in (pool, d):
        p.fork([1], [2])
    pool.lens = [40, 21, 21, 16]
    d.lens.copy_(i32(pool.lens, cuda_device))
    slots, _, taken = pool.extend([24, 1, 1, 16])
    assert slots is None
    assert d.extend([24, 1, 1, 16]).tolist() == [-1] * 42 and d.counts.tolist() == [0, -taken]
    assert d.status() == ops.CPA_ERR_DEVICE
    d.same(pool)


def test_extend_malformed_rows_take_nothing(cuda_device):
    """Lengths below q_len or past the row, an entry past the pool, tokens behind the last row."""
    pool = Pool.random([20, 20, 20, 20], 5, 3, 20, 2)
    d = Device(pool, cuda_device)
    d.lens.copy_(i32([21, 1, 49, 21, 1], cuda_device))
    d.table[3, 1] = 20
    slots = d.extend([1, 2, 1, 1, 1], tokens=9).tolist()
    assert slots[0] == pool.table[0][1] * PAGE + 4 and slots[5] == min(x for x, r in enumerate(pool.refs) if r == 0) * PAGE
    assert slots[1:5] == [-1] * 4 and slots[6:] == [-1] * 3
    assert d.counts.tolist() == [0, 1] and d.status() == ops.CPA_ERR_DEVICE


def test_extend_without_rows_or_tokens(cuda_device):
    pool = Pool.random([20], 1, 3, 20, 2)
    d = Device(pool, cuda_device)
    assert d.extend([0]).numel() == 0 and d.counts.tolist() == [0, 0]
    slots = torch.full((3,), 5, dtype=torch.int64, device=cuda_device)
    ops.extend_sequences(i32([0], cuda_device), d.lens[:0], d.table[:0], d.refs, slots, d.src, d.dst, d.counts, d.ws)
    assert slots.tolist() == [-1] * 3 and d.counts.tolist() == [0, 0]
    d.same(pool)


@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (1, 1), (16, 16), (17, 17), (100, 4), (33, 50), (4000, 4), (5, 4000)])
def test_release(cuda_device, window, sinks):
    lens = [1, 15, 16, 17, 160, 161, 175, 700, 1000, 1600, 33, 90]
    pool = Pool.random(lens, 14, 101, 400, 5, shared=0.6)
    d = Device(pool, cuda_device)
    before = [list(r) for r in pool.table]
    rows = [3, 9, 8, 7, 7, 11, 0, 2, 13, 10, 4]
    pool.release(rows, window, sinks)
    d.release(rows, window, sinks)
    d.same(pool)
    if window:  # what is gone is what no later query sees, and every page of that kind
        for r in set(rows) - {13}:
            n = lens[r]
            seen = visible(torch.tensor([n, n + 1, n + 40]), torch.arange(n), window, sinks).any(0)
            for c in range(-(-n // PAGE)):
                keep = bool(seen[c * PAGE:(c + 1) * PAGE].any()) or (c + 1) * PAGE > n
                assert (pool.table[r][c] >= 0) == keep and before[r][c] >= 0
    d.release(None, window, sinks)
    pool.release(range(14), window, sinks)
    d.same(pool)
    assert d.status() == ops.CPA_OK
    if window == 0:
        assert sum(pool.refs) == 0


def test_release_reports(cuda_device):
    pool = Pool.random([20, 20], 3, 3, 20, 2)
    d = Device(pool, cuda_device)
    d.release([-1, 3, 0])
    pool.release([0])
    d.same(pool)
    assert d.status() == ops.CPA_ERR_DEVICE
    d.table[2, 0], d.table[2, 1] = 25, pool.refs.index(0)
    d.release([2])
    assert d.table[2].tolist() == [-1] * 3 and d.refs.tolist() == pool.refs and d.status() == ops.CPA_ERR_DEVICE


@pytest.mark.parametrize("pages", [1, 2, 15, 16, 17, 4095, 4096, 4097, 9000, 16_384, 16_385, 70_001, 131_072, 131_073, 200_001])
@pytest.mark.parametrize("fill", [0.0, 0.3, 0.9, 1.0])
def test_compact(cuda_device, pages, fill):
    g = torch.Generator().manual_seed(pages)
    columns = 40 if pages < 100_000 else 1000
    rows = -(-pages // columns) + 2
    pool = Pool(rows, columns, pages)
    held = [x for x, y in enumerate(torch.rand(pages, generator=g).tolist()) if y < fill]
    order = torch.randperm(len(held), generator=g).tolist()
    for i, o in enumerate(order):
        pool.table[i // columns][i % columns] = held[o]
        if i % 5 == 0:  # a second holder
            pool.table[rows - 1][i // 5 % columns] = held[o]
    pool.refs = [0] * pages
    for r in pool.table:
        for x in r:
            if x >= 0:
                pool.refs[x] += 1
    d = Device(pool, cuda_device)
    moves, m = pool.compact()
    d.compact()
    assert d.counts.tolist() == [len(moves), m]
    assert d.pairs() == moves
    d.same(pool)
    assert d.status() == ops.CPA_OK
    d.compact()  # packed already
    assert d.counts.tolist() == [0, m] and d.pairs() == []
    d.same(pool)


def test_compact_a_large_table(cuda_device):
    """A small pool under more entries than the pool's cluster takes with it: rows that share everything."""
    pool = Pool.random([4000] * 3, 120, 260, 900, 5)
    d = Device(pool, cuda_device)
    for p in (pool, d):
        p.fork([r % 3 for r in range(117)], list(range(3, 120)))
        p.release([0, 3], 0, 0)
        p.release([1] + list(range(4, 120, 3)), 0, 0)
    moves, m = pool.compact()
    d.compact()
    assert d.counts.tolist() == [len(moves), m] and d.pairs() == moves and moves
    d.same(pool)
    assert d.status() == ops.CPA_OK


def test_compact_reports_entries_without_a_page(cuda_device):
    pool = Pool.random([30, 30], 3, 4, 12, 2)
    d = Device(pool, cuda_device)
    free = [x for x, r in enumerate(pool.refs) if r == 0]
    d.table[2, 0], d.table[2, 1] = 12, free[-1]
    pool.compact()
    d.compact()
    assert d.table[2].tolist() == [12, free[-1], -1, -1] and d.table[:2].tolist() == pool.table[:2]
    assert d.status() == ops.CPA_ERR_DEVICE


# ---- together

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("window,sinks", [(40, 4), (300, 20)])
def test_serving_with_shared_prefixes(cuda_device, dtype, window, sinks):
    """Prompts are filled, forked and decoded with a window; pages that slid out are given back, a sequence ends, the pool is packed on
    the way.  Every step's output is that of sequences that share nothing, computed in 64 bits from what was appended."""
    dev, hq, hkv, d, pages, rows = cuda_device, 4, 2, 64, 200, 7
    g = torch.Generator(dev).manual_seed(9)
    pool = Pool(rows, 40, pages)
    s = Device(pool, dev)
    k_cache = torch.full((pages, hkv, PAGE, d), float("nan"), dtype=dtype, device=dev)
    v_cache = k_cache.clone()
    said = [([], []) for _ in range(rows)]  # every row's keys and values

    def copies():
        ops.copy_pages(s.src, s.dst, k_cache, v_cache, num_pairs=s.counts, workspace=s.ws)

    def step(q):
        live = [r for r in range(rows) if q[r]]
        s.lens += i32(q, dev)
        slots = s.extend(q)
        assert int(s.counts[1]) >= 0
        copies()
        T = sum(q)
        draw = lambda h: torch.randn(T, h, d, generator=g, device=dev).to(dtype)  # noqa: E731
        x, k, v = draw(hq), draw(hkv), draw(hkv)
        starts = i32([0] + [sum(q[r] for r in live[:i + 1]) for i in range(len(live))], dev)
        table, lens = s.table[live].contiguous(), s.lens[live].contiguous()
        ws = ops.workspace_for(k_cache, hq, table.shape[1], len(live), T)
        out = ops.append_window_attention_forward(x, k, v, slots, k_cache, v_cache, table, starts, lens, d ** -0.5, ws, window, sinks)
        at = 0
        for r in live:
            said[r][0].append(k[at:at + q[r]])
            said[r][1].append(v[at:at + q[r]])
            kk, vv = (torch.cat(z).double() for z in said[r])
            n = kk.shape[0]
            mask = visible(torch.arange(n - q[r], n, device=dev), torch.arange(n, device=dev), window, sinks)
            for h in range(hq):
                logits = d ** -0.5 * x[at:at + q[r], h].double() @ kk[:, h // 2].T
                p = torch.softmax(logits.masked_fill(~mask, float("-inf")), -1)
                want, size = p @ vv[:, h // 2], p @ vv[:, h // 2].abs()
                half = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
                weights = half if dtype == torch.bfloat16 else 0.0
                err = (out[at:at + q[r], h].double() - want).abs()
                assert (err <= half * want.abs() + (weights + 2.0 ** -13) * size).all()
            at += q[r]

    step([70, 250, 33, 0, 0, 0, 0])
    s.fork([0, 0, 1, 2], [3, 4, 5, 6])
    for a, b in ((0, 3), (0, 4), (1, 5), (2, 6)):
        said[b] = tuple(list(z) for z in said[a])
    step([1] * 7)
    step([1, 5, 1, 40, 1, 1, 1])
    s.release(None, window, sinks)
    step([1] * 7)
    s.release([3, 1])
    said[3], said[1] = ([], []), ([], [])
    s.compact()
    copies()
    live = int(s.counts[1])
    assert (s.refs[:live] > 0).all() and (s.refs[live:] == 0).all()
    k_cache[live:], v_cache[live:] = float("nan"), float("nan")
    step([1, 0, 30, 0, 2, 1, 1])
    s.fork([6], [3])
    said[3] = tuple(list(z) for z in said[6])
    s.release(None, window, sinks)
    step([1, 100, 1, 1, 1, 1, 1])
    assert s.status() == ops.CPA_OK
    have = torch.bincount(s.table[s.table >= 0].long(), minlength=pages)
    assert torch.equal(have.int(), s.refs)


def test_captured_and_replayed(cuda_device):
    """Fork, extend, copy, release and compact in one graph: replays on the restored state give the same state."""
    pool = Pool.random([100, 37, 64, 9], 8, 12, 80, 4)
    d = Device(pool, cuda_device)
    kc = torch.randn(80, 2, PAGE, 64, device=cuda_device).bfloat16()
    vc = kc.clone()
    start = [t.clone() for t in (d.table, d.lens, d.refs, kc, vc)]
    q = [1] * 8
    starts, slots = i32(range(9), cuda_device), torch.zeros(8, dtype=torch.int64, device=cuda_device)
    parents, kids, done = i32([0, 0, 1, 2], cuda_device), i32([4, 5, 6, 7], cuda_device), i32([1, 4], cuda_device)

    def flow():
        ops.fork_sequences(parents, kids, d.table, d.lens, d.refs, d.ws)
        d.lens.add_(1)
        ops.extend_sequences(starts, d.lens, d.table, d.refs, slots, d.src, d.dst, d.counts, d.ws)
        ops.copy_pages(d.src, d.dst, kc, vc, num_pairs=d.counts, workspace=d.ws)
        ops.release_pages(done, d.table, d.lens, d.refs, d.ws)
        ops.release_pages(None, d.table, d.lens, d.refs, d.ws, 20, 4)
        ops.compact_pages(d.table, d.refs, d.src, d.dst, d.counts, d.ws)
        ops.copy_pages(d.src, d.dst, kc, vc, num_pairs=d.counts, workspace=d.ws)

    def restore():
        for t, x in zip((d.table, d.lens, d.refs, kc, vc), start):
            t.copy_(x)

    flow()
    torch.cuda.synchronize()
    want = [t.clone() for t in (d.table, d.lens, d.refs, kc, vc, slots, d.counts)]
    restore()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        flow()
    for _ in range(2):
        restore()
        d.ws[256:].random_(0, 256)
        graph.replay()
        torch.cuda.synchronize()
        for t, x in zip((d.table, d.lens, d.refs, kc, vc, slots, d.counts), want):
            assert torch.equal(t, x)
    assert q and d.status() == ops.CPA_OK


def test_tensors_that_are_refused(cuda_device):
    pool = Pool.random([30, 30], 4, 6, 40, 3)
    d = Device(pool, cuda_device)
    rows = i32([0, 1], cuda_device)
    with pytest.raises(ValueError):
        ops.fork_sequences(rows, rows[:1], d.table, d.lens, d.refs, d.ws)
    with pytest.raises(ValueError):
        ops.fork_sequences(rows, rows, d.table[:, ::2], d.lens, d.refs, d.ws)
    with pytest.raises(TypeError):
        ops.release_pages(rows.long(), d.table, d.lens, d.refs, d.ws)
    with pytest.raises(ValueError):
        ops.release_pages(rows, d.table, d.lens[:3], d.refs, d.ws)
    with pytest.raises(ValueError):  # lists too short
        ops.compact_pages(d.table, d.refs, d.src[:19], d.dst, d.counts, d.ws)
    with pytest.raises(ops.CpaError):  # references off a 16-byte boundary
        ops.compact_pages(d.table, d.refs[1:], d.src, d.dst, d.counts, d.ws)
    with pytest.raises(ops.CpaError):  # a workspace for fewer pages
        ops.compact_pages(d.table, d.refs, d.src, d.dst, d.counts, d.ws[:256])
    with pytest.raises(ops.CpaError):
        ops.release_pages(rows, d.table, d.lens, d.refs, d.ws, window=-5)
    with pytest.raises(ops.CpaError):  # sinks without a window
        ops.release_pages(rows, d.table, d.lens, d.refs, d.ws, sinks=3)
    d.same(pool)
    assert d.status() == ops.CPA_OK


def test_on_another_stream(cuda_device):
    """The whole flow on a stream of its own, with the host's stream idle."""
    pool = Pool.random([100, 37], 4, 12, 40, 4)
    d = Device(pool, cuda_device)
    kc = torch.randn(40, 2, PAGE, 64, device=cuda_device)
    vc, before = kc.clone(), kc.clone()
    starts, slots = i32(range(5), cuda_device), torch.zeros(4, dtype=torch.int64, device=cuda_device)
    parents, kids, gone = i32([0, 1], cuda_device), i32([2, 3], cuda_device), i32([0], cuda_device)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    ops.fork_sequences(parents, kids, d.table, d.lens, d.refs, d.ws, stream=s)
    with torch.cuda.stream(s):
        d.lens.add_(1)
    ops.extend_sequences(starts, d.lens, d.table, d.refs, slots, d.src, d.dst, d.counts, d.ws, stream=s)
    ops.copy_pages(d.src, d.dst, kc, vc, num_pairs=d.counts, workspace=d.ws, stream=s)
    ops.release_pages(gone, d.table, d.lens, d.refs, d.ws, stream=s)
    s.synchronize()
    pool.fork([0, 1], [2, 3])
    pool.lens = [n + 1 for n in pool.lens]
    want, pairs, _ = pool.extend([1] * 4)
    pool.release([0])
    d.same(pool)
    assert slots.tolist() == want and pairs
    for a, b in pairs:
        assert torch.equal(kc[b], before[a]) and torch.equal(vc[b], before[a])
