"""Packing a step on the device against the definition on the host."""
import pytest
import torch

from chunked_prefill_paged_cpa_gb300 import batch, ops
from select_support import PAGE, random_table

pytestmark = pytest.mark.gpu


def outputs(n, cols, tokens, device):
    i32 = lambda *s: torch.full(s, -9, dtype=torch.int32, device=device)  # noqa: E731
    return {"starts": i32(n + 1), "lens": i32(n), "table": i32(n, cols), "positions": i32(tokens),
            "slots": torch.full((tokens,), -9, dtype=torch.int64, device=device), "counts": i32(2)}


def expected(o, requests, took, table, lens, num_pages):
    """The outputs after the call, and whether the status word is raised."""
    o = {k: v.cpu().clone() for k, v in o.items()}
    n = t = 0
    bad = False
    live = []
    for row, q in zip(requests, took):
        ok = 0 <= row < table.shape[0] and q >= 0 and q <= int(lens[row]) <= table.shape[1] * PAGE
        bad |= not ok
        if ok and q:
            live.append((row, q))
    T = sum(q for _, q in live)
    if T > o["slots"].shape[0]:
        o["counts"][:] = torch.tensor([0, -min(T, 2 ** 31 - 1)])
        return o, True
    o["starts"][0] = 0
    for row, q in live:
        length = int(lens[row])
        held = -(-length // PAGE)
        o["starts"][n + 1], o["lens"][n], o["table"][n, :held] = t + q, length, table[row, :held]
        for p in range(length - q, length):
            page = int(table[row, p // PAGE])
            ok = 0 <= page < num_pages
            bad |= not ok
            o["positions"][t], o["slots"][t] = p, page * PAGE + p % PAGE if ok else -1
            t += 1
        n += 1
    o["counts"][:] = torch.tensor([n, t])
    return o, bad


def check(device, requests, took, table, lens, tokens, num_pages, listed=True):
    n = len(took)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=device)  # noqa: E731
    o = outputs(n, table.shape[1], tokens, device)
    want, bad = expected(o, requests, took, table, lens, num_pages)
    ws = torch.zeros(256, dtype=torch.uint8, device=device)
    ops.pack_step(i32(requests) if listed else None, i32(took), table.to(device), lens.to(device), o["starts"], o["lens"], o["table"], o["positions"],
                  o["slots"], o["counts"], num_pages=num_pages, workspace=ws)
    for k in want:
        assert torch.equal(o[k].cpu(), want[k]), k
    assert bool(ws[:4].any()) == bad
    return o


def pool(lengths, seed, columns=None):
    pages = sum(-(-n // PAGE) for n in lengths) + 4
    return random_table(lengths, pages, seed, columns), torch.tensor(lengths, dtype=torch.int32), pages


def test_small_steps(cuda_device):
    table, lens, pages = pool([1, 16, 17, 200, 33, 64, 5], 1)
    check(cuda_device, [3], [1], table, lens, 1, pages)
    check(cuda_device, [6, 0, 3, 2], [5, 1, 100, 0], table, lens, 110, pages)
    check(cuda_device, [5, 5, 1], [64, 1, 16], table, lens, 81, pages)
    check(cuda_device, list(range(7)), [0] * 7, table, lens, 4, pages)
    check(cuda_device, list(range(7)), [0, 3, 17, 0, 1, 0, 5], table, lens, 26, pages, listed=False)
    check(cuda_device, [], [], table, lens, 0, pages)


@pytest.mark.parametrize("n,rows,longest", [(300, 400, 900), (4096, 4096, 100), (1000, 1500, 12000), (2, 3, 70000)])
def test_large_steps(cuda_device, n, rows, longest):
    g = torch.Generator().manual_seed(n)
    lengths = torch.randint(1, longest, (rows,), generator=g).tolist()
    table, lens, pages = pool(lengths, 2)
    requests = torch.randperm(rows, generator=g)[:n].tolist()
    took = [min(lengths[r], 0 if i % 5 == 2 else 300 if i % 50 == 7 else 1) for i, r in enumerate(requests)]
    check(cuda_device, requests, took, table, lens, sum(took) + 3, pages)


def test_a_whole_prompt_and_a_wide_table(cuda_device):
    table, lens, pages = pool([20000, 3], 3, columns=9000)
    check(cuda_device, [1, 0], [3, 20000], table, lens, 20003, pages)


def test_what_cannot_be_packed(cuda_device):
    """Rows outside the table, negative counts, counts above lengths, lengths above the table: left out; more tokens than there
    is room for: nothing; entries that are no pages: slot -1."""
    table, lens, pages = pool([50, 60, 70, 80], 4)
    check(cuda_device, [0, 9, 2], [3, 1, 4], table, lens, 20, pages)
    check(cuda_device, [-1, 1, 2], [3, 1, 4], table, lens, 20, pages)
    check(cuda_device, [0, 1, 2], [-3, 1, 4], table, lens, 20, pages)
    check(cuda_device, [0, 1, 2], [51, 1, 4], table, lens, 200, pages)
    lens[1] = table.shape[1] * PAGE + 1
    check(cuda_device, [0, 1, 2], [1, 1, 4], table, lens, 20, pages)
    lens[1] = 60
    check(cuda_device, [0, 1, 2], [10, 10, 1], table, lens, 20, pages)
    lens[:] = 2 ** 30    # (far above the table: every request is refused before its tokens count)
    check(cuda_device, [0, 1, 2], [2 ** 30] * 3, table, lens, 20, pages)
    lens[:] = torch.tensor([50, 60, 70, 80])
    table[0, 3], table[2, 4] = -1, pages
    check(cuda_device, [0, 1, 2], [10, 1, 40], table, lens, 60, pages)
    check(cuda_device, [0, 1, 2], [1, 1, 1], table, lens, 3, pages)
    table[1, 0] = -1     # (an entry of earlier tokens is copied as it is)
    check(cuda_device, [1], [1], table, lens, 3, pages)


def test_sums_past_32_bits(cuda_device):
    """4096 requests of 2^20 tokens: nothing is written but the count, which stops at 2^31 - 1."""
    n, cols = 4096, 2 ** 16
    table = torch.zeros(1, cols, dtype=torch.int32, device=cuda_device)
    i32 = lambda x, k: torch.full((k,), x, dtype=torch.int32, device=cuda_device)  # noqa: E731
    o = outputs(n, cols, 10, cuda_device)
    ops.pack_step(i32(0, n), i32(2 ** 20, n), table, i32(2 ** 20, 1), o["starts"], o["lens"], o["table"], o["positions"], o["slots"], o["counts"])
    assert o["counts"].tolist() == [0, -(2 ** 31 - 1)]
    assert all(int(o[k].max()) == -9 for k in ("starts", "lens", "table", "positions", "slots"))


def test_equals_the_host_metadata(cuda_device):
    """What the batch module builds on the host."""
    lengths, q_lens = [100, 33, 640, 16], [1, 33, 200, 1]
    table, lens, pages = pool(lengths, 5)
    m = batch.build_metadata(q_lens, lengths, [table[s].tolist() for s in range(4)], PAGE, pages, max_pages=table.shape[1])
    o = check(cuda_device, [0, 1, 2, 3], q_lens, table, lens, sum(q_lens), pages)
    assert torch.equal(o["starts"].cpu(), m.query_start_loc) and torch.equal(o["lens"].cpu(), m.seq_lens)
    assert torch.equal(o["slots"].cpu(), m.slot_mapping)
    for s, n in enumerate(lengths):
        assert torch.equal(o["table"][s, :-(-n // PAGE)].cpu(), m.block_table[s, :-(-n // PAGE)])


def test_capture(cuda_device):
    table, lens, pages = pool([100, 200, 300], 6)
    o = outputs(3, table.shape[1], 40, cuda_device)
    took, dev_lens, dev_table = torch.tensor([1, 0, 20], dtype=torch.int32, device=cuda_device), lens.to(cuda_device), table.to(cuda_device)
    args = (None, took, dev_table, dev_lens, o["starts"], o["lens"], o["table"], o["positions"], o["slots"], o["counts"])
    ops.pack_step(*args)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        ops.pack_step(*args)
    took.copy_(torch.tensor([7, 30, 0], dtype=torch.int32))
    fresh = outputs(3, table.shape[1], 40, cuda_device)
    for k in o:
        o[k].copy_(fresh[k])
    graph.replay()
    want, _ = expected(fresh, [0, 1, 2], [7, 30, 0], table, lens, pages)
    for k in want:
        assert torch.equal(o[k].cpu(), want[k]), k
