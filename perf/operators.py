"""Cases of the sliding-window attention and of the paged cache's page operators, with their plain forms.

Four kinds of case ("kind"):

* ``attention``: one step of attention with a sliding window and sinks over a packed batch (decodes, then chunks) and a
  cache of 16-token pages.  The row at position p sees key j when j <= p and (j < sinks or j > p - window).
* ``copy``: pages of the cache copied to other pages, from a list of (source, destination) pairs on the device.
* ``branch``: sequences forked (a child shares its parent's pages), every row extended by a few tokens (free pages taken,
  shared pages that are written to replaced by copies), and the copies carried out.
* ``trim``: pages that slid out of the window released, finished sequences released, the pool compacted, the moves carried
  out.

``run`` computes them from elementary torch operations, or, where ``own`` is true, through the package's entry points.
"""
import torch

own = False

PAGE = 16
E4M3_SCALE = 2.0 ** -6      # K and V of an 8-bit cache are codes of x / 2^-6
BLOCK = 256                 # query rows of a chunk that the plain form takes together

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ---------------------------------------------------------------------------------------------------------------- cases

def _attention(name, decodes, lo, hi, chunks, chunk, offset, window, sinks, hq, hkv, d, dtype="bf16", cache="same", append=False, trimmed=False):
    c = {"kind": "attention", "decodes": decodes, "lo": lo, "hi": hi, "chunks": chunks, "chunk": chunk, "offset": offset, "window": window,
         "sinks": sinks, "hq": hq, "hkv": hkv, "d": d, "dtype": dtype, "cache": cache, "append": append, "trimmed": trimmed}
    return dict(c, name=name) if name else c


def _copy(name, pages, pairs, hkv, d, dtype="bf16", cache="same"):
    c = {"kind": "copy", "pages": pages, "pairs": pairs, "hkv": hkv, "d": d, "dtype": dtype, "cache": cache}
    return dict(c, name=name) if name else c


def _branch(name, rows, forks, lo, hi, new, spare, hkv, d, dtype="bf16"):
    c = {"kind": "branch", "rows": rows, "forks": forks, "lo": lo, "hi": hi, "new": new, "spare": spare, "hkv": hkv, "d": d, "dtype": dtype}
    return dict(c, name=name) if name else c


def _trim(name, rows, finished, lo, hi, window, sinks, hkv, d, dtype="bf16"):
    c = {"kind": "trim", "rows": rows, "finished": finished, "lo": lo, "hi": hi, "window": window, "sinks": sinks, "hkv": hkv, "d": d, "dtype": dtype}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one user's next token: the latency of a single call
        _attention("decode_one", 1, 1500, 1500, 0, 0, 0, 1024, 4, 32, 8, 128),
        # a full batch of single tokens, the long window of a long-context deployment: the cache's bandwidth
        _attention("decode_batch", 256, 2048, 8192, 0, 0, 0, 4096, 4, 32, 8, 128, trimmed=True),
        # the same kind of batch over the 8-bit cache, shorter window
        _attention("decode_e4m3", 256, 2048, 8192, 0, 0, 0, 1024, 64, 32, 8, 128, cache="e4m3", trimmed=True),
        # the default hybrid step: 32 decodes beside a 480-token chunk of an 8192-token prompt, appended in the same call
        _attention("hybrid_append", 32, 512, 4096, 1, 480, 3840, 1024, 4, 32, 8, 128, append=True),
        # a whole long prompt in one step, binary16: the tensor cores
        _attention("prefill_long", 0, 0, 0, 1, 8192, 0, 2048, 4, 32, 8, 128, dtype="f16"),
        # the high-resolution configuration: fp32, few heads, an odd chunk and an odd window
        _attention("hybrid_f32", 7, 100, 2000, 1, 333, 500, 250, 3, 8, 2, 64, dtype="f32", append=True),
        # a handful of pages swapped by a scheduler, 8-bit cache: the latency of a single call
        _copy("copy_few", 1024, 8, 8, 128, cache="e4m3"),
        # a large defragmentation or a migrated batch of prefixes: bandwidth
        _copy("copy_many", 10240, 4096, 8, 128),
        # four prompts sampled twice
        _branch("branch_few", 4, 4, 100, 1000, 1, 512, 8, 128),
        # a batch of 64 prompts branched into 256 candidates of four tokens each, a large pool
        _branch("branch_many", 64, 192, 512, 4096, 4, 4096, 8, 128),
        # a small batch slides by some pages and one sequence ends
        _trim("trim_few", 6, 1, 200, 1200, 256, 4, 2, 64),
        # a large batch slides, 16 sequences end, and the pool is packed
        _trim("trim_many", 96, 16, 512, 4096, 1024, 4, 8, 128),
    ]


def _log(rng, lo, hi):
    """An integer from lo to hi, spread over its logarithm."""
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    """One more case: most are attention, the others one of the page operators' flows."""
    hkv, d = rng.choice([1, 2, 4, 8]), rng.choice([64, 128])
    kind = rng.choice(["attention", "attention", "attention", "copy", "branch", "trim"])
    if kind == "copy":
        pages = _log(rng, 300, 8000)
        return _copy(None, pages, _log(rng, 1, pages // 2), hkv, d, rng.choice(["bf16", "f16", "f32"]), rng.choice(["same", "same", "e4m3"]))
    if kind == "branch":
        rows = _log(rng, 1, 64)
        lo = _log(rng, 17, 600)
        return _branch(None, rows, _log(rng, 1, 128), lo, lo + _log(rng, 30, 2500), _log(rng, 1, 40), _log(rng, 900, 4000), hkv, d, rng.choice(["bf16", "f32"]))
    if kind == "trim":
        rows = _log(rng, 3, 96)
        lo = _log(rng, 40, 800)
        return _trim(None, rows, rng.randrange(0, rows // 2 + 1), lo, lo + _log(rng, 30, 2500), _log(rng, 1, 2048), rng.choice([0, 1, 4, 16, 37]), hkv, d, rng.choice(["bf16", "f32"]))
    g = rng.choice([x for x in (1, 2, 4, 8) if x * hkv <= 32])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    form = rng.choice(["decode", "chunk", "hybrid"])
    decodes = 0 if form == "chunk" else _log(rng, 1, 40 if dtype == "f32" else 100)
    chunk = 0 if form == "decode" else _log(rng, 2, 400 if dtype == "f32" else 1000)
    lo = _log(rng, 1, 3000)
    cache = rng.choice(["same", "same", "e4m3"]) if dtype != "f32" else "same"
    return _attention(None, decodes, lo, lo + _log(rng, 20, 4000), 0 if form == "decode" else rng.choice([1, 1, 2, 3]), chunk, rng.choice([0, _log(rng, 1, 4000)]),
                      _log(rng, 1, 8000), rng.choice([0, 1, 4, rng.randrange(5, 100)]), hkv * g, hkv, d, dtype, cache, cache == "same" and rng.random() < 0.5, rng.random() < 0.5)


# --------------------------------------------------------------------------------------------------------------- inputs

def _lengths(case, n, g):
    return torch.randint(case["lo"], case["hi"] + 1, (n,), generator=g).tolist() if n else []


def _normal(shape, dtype, gen):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def _cache(case, pages, gen):
    """K and V of every page, N(0, 1); an 8-bit cache as codes."""
    shape = (pages, case["hkv"], PAGE, case["d"])
    out = []
    for _ in range(2):
        if case.get("cache") == "e4m3":
            x = torch.empty(shape, dtype=torch.uint8, device="cuda")
            for p in range(0, pages, 4096):
                y = torch.randn(x[p:p + 4096].shape, generator=gen, device="cuda")
                x[p:p + 4096] = (y / E4M3_SCALE).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        else:
            x = torch.empty(shape, dtype=DTYPES[case["dtype"]], device="cuda")
            for p in range(0, pages, 4096):
                x[p:p + 4096].normal_(generator=gen)
        out.append(x)
    return out


def _int(x, dtype=torch.int32):
    return torch.as_tensor(x, dtype=dtype).cuda()


def _sequences(case, seed):
    """(new tokens, length) of every sequence of an attention case."""
    g = torch.Generator().manual_seed(seed)
    seqs = [(1, n) for n in _lengths(case, case["decodes"], g)]
    return seqs + [(case["chunk"], case["offset"] + case["chunk"])] * case["chunks"], g


def _visible(case, q_len, length):
    """Positions that the sequence's new rows see between them: [0, a) and [b, length)."""
    first = length - q_len
    b = max(0, first - case["window"] + 1)
    return min(case["sinks"], b), b


def _prepare_attention(case, seed):
    seqs, g = _sequences(case, seed)
    gen = torch.Generator("cuda").manual_seed(seed)
    tokens = sum(q for q, _ in seqs)
    columns = max(-(-n // PAGE) for _, n in seqs) + 1
    table = torch.full((len(seqs), columns), -1, dtype=torch.int32)
    held = torch.zeros((len(seqs), columns), dtype=torch.bool)
    for s, (q, n) in enumerate(seqs):
        held[s, :-(-n // PAGE)] = True
        if case["trimmed"]:  # the pages that no row sees any more were given back
            a, b = _visible(case, q, n)
            held[s, -(-a // PAGE):b // PAGE] = False
    most = -(-case["hi"] // PAGE)  # pages of a decode at most: the pool's size does not depend on the seed
    if case["trimmed"]:
        most = min(most, -(-case["sinks"] // PAGE) + case["window"] // PAGE + 2)
    pages = case["decodes"] * most + case["chunks"] * -(-(case["offset"] + case["chunk"]) // PAGE) + 1
    need = int(held.sum())
    table[held] = torch.randperm(pages, generator=g)[:need].to(torch.int32)
    starts, slots = [0], []
    for s, (q, n) in enumerate(seqs):
        pos = torch.arange(n - q, n)
        slots.append(table[s, pos // PAGE].long() * PAGE + pos % PAGE)
        starts.append(starts[-1] + q)
    dtype = DTYPES[case["dtype"]]
    k_cache, v_cache = _cache(case, pages, gen)
    state = {"case": case, "k_cache": k_cache, "v_cache": v_cache, "table": table.cuda(), "starts": _int(starts), "lengths": _int([n for _, n in seqs]),
             "q": _normal((tokens, case["hq"], case["d"]), dtype, gen), "out": torch.empty((tokens, case["hq"], case["d"]), dtype=dtype, device="cuda"),
             "k": _normal((tokens, case["hkv"], case["d"]), dtype, gen), "v": _normal((tokens, case["hkv"], case["d"]), dtype, gen), "slots": torch.cat(slots).cuda()}
    if own:  # the workspace that a user's program holds from step to step
        from chunked_prefill_paged_cpa_gb300 import ops
        state["workspace"] = ops.workspace_for(k_cache, case["hq"], columns, len(seqs), tokens, act_dtype=dtype)
    return state


def _prepare_copy(case, seed):
    g, gen = torch.Generator().manual_seed(seed), torch.Generator("cuda").manual_seed(seed)
    k_cache, v_cache = _cache(case, case["pages"], gen)
    order = torch.randperm(case["pages"], generator=g)[:2 * case["pairs"]].to(torch.int32).cuda()
    return {"case": case, "k_cache": k_cache, "v_cache": v_cache, "src": order[:case["pairs"]].contiguous(), "dst": order[case["pairs"]:].contiguous()}


def _prepare_pool(case, seed):
    """Page references, block table and lengths of a branch or trim case, and the working copy that the calls change."""
    g, gen = torch.Generator().manual_seed(seed), torch.Generator("cuda").manual_seed(seed)
    rows, forks, new = case["rows"], case.get("forks", 0), case.get("new", 0)
    lengths = _lengths(case, rows, g)
    counts = [-(-n // PAGE) for n in lengths]
    columns = -(-(case["hi"] + new) // PAGE) + 3
    table = torch.full((rows + forks, columns), -1, dtype=torch.int32)
    pages = rows * -(-case["hi"] // PAGE) + case.get("spare", 8)  # enough for any seed's lengths
    order, at = torch.randperm(pages, generator=g).to(torch.int32), 0
    for r, n in enumerate(counts):
        table[r, :n] = order[at:at + n]
        at += n
        if case["kind"] == "trim" and r % 3 == 2:  # every third sequence was branched from the one before it after its first pages
            m = min(n, counts[r - 1]) // 2
            table[r, :m] = table[r - 1, :m]
    refs = torch.bincount(table[table >= 0].long(), minlength=pages).to(torch.int32)
    saved = torch.cat([refs, table.flatten(), torch.tensor(lengths + [0] * forks, dtype=torch.int32)]).cuda()
    live = saved.clone()
    k_cache, v_cache = _cache(case, pages, gen)
    state = {"case": case, "k_cache": k_cache, "v_cache": v_cache, "saved": saved, "live": live, "refs": live[:pages],
             "table": live[pages:pages + table.numel()].view(table.shape), "lengths": live[pages + table.numel():]}
    if case["kind"] == "branch":
        state |= {"parents": torch.randint(0, rows, (forks,), generator=g).to(torch.int32).cuda(), "children": _int(range(rows, rows + forks)),
                  "starts": _int(range(0, (rows + forks) * new + 1, new)), "slots": torch.full(((rows + forks) * new,), -1, dtype=torch.int64, device="cuda")}
        most = rows + forks
    else:
        state |= {"every": _int(range(rows)), "done": torch.randperm(rows, generator=g)[:case["finished"]].to(torch.int32).cuda()}
        most = pages
    state |= {"src": torch.full((most,), -1, dtype=torch.int32, device="cuda"), "dst": torch.full((most,), -1, dtype=torch.int32, device="cuda"),
              "counts": torch.zeros(2, dtype=torch.int32, device="cuda")}
    if own:
        from chunked_prefill_paged_cpa_gb300 import ops
        state["workspace"] = ops.pages_workspace_for(pages, device="cuda")
    return state


def prepare(case, seed):
    return {"attention": _prepare_attention, "copy": _prepare_copy, "branch": _prepare_pool, "trim": _prepare_pool}[case["kind"]](case, seed)


# ----------------------------------------------------------------------------------------------------------- plain forms

def _values(codes, scale):
    if codes.dtype == torch.uint8:
        return codes.view(torch.float8_e4m3fn).float() * scale
    return codes.float()


def _attend(case, q, pos, table, k_cache, v_cache):
    """q [n, b, hq, d]: blocks of consecutive rows of one sequence each, pos [n, b] their positions, table [n, columns]."""
    n, b = pos.shape
    w, sinks, hkv, d = case["window"], case["sinks"], case["hkv"], case["d"]
    count = min(w + b - 1, table.shape[1] * PAGE)
    start = (pos[:, :1] - w + 1).clamp(min=0)
    near = start + torch.arange(count, device=pos.device)
    far = torch.arange(min(sinks, table.shape[1] * PAGE), device=pos.device).expand(n, -1)
    keys = torch.cat([far, near], 1)
    seen = keys[:, None] <= pos[:, :, None]
    seen &= torch.cat([(far < start)[:, None].expand(-1, b, -1), (near[:, None] > pos[:, :, None] - w) | ((near < sinks)[:, None])], 2)
    keys = keys.clamp(max=table.shape[1] * PAGE - 1)
    page, off = table.gather(1, keys // PAGE).clamp(min=0).long(), keys % PAGE
    k = _values(k_cache[page, :, off], E4M3_SCALE).permute(0, 2, 3, 1)
    v = _values(v_cache[page, :, off], E4M3_SCALE).permute(0, 2, 1, 3)
    rows = q.float().reshape(n, b, hkv, -1, d).permute(0, 2, 3, 1, 4)
    s = (rows.reshape(n, hkv, -1, d) @ k).reshape(n, hkv, -1, b, keys.shape[1]) * d ** -0.5
    s = s.masked_fill(~seen[:, None, None], float("-inf"))
    e = torch.exp(s - s.amax(-1, keepdim=True))
    e = e / e.sum(-1, keepdim=True)
    o = (e.reshape(n, hkv, -1, keys.shape[1]) @ v).reshape(n, hkv, -1, b, d)
    return o.permute(0, 3, 1, 2, 4).reshape(n, b, -1, d)


def _plain_attention(st):
    case, q, table, lengths = st["case"], st["q"], st["table"].long(), st["lengths"].long()
    k_cache, v_cache, out = st["k_cache"], st["v_cache"], st["out"]
    if case["append"]:
        page, off = st["slots"] // PAGE, st["slots"] % PAGE
        k_cache[page, :, off] = st["k"]
        v_cache[page, :, off] = st["v"]
    nd, nc, c = case["decodes"], case["chunks"], case["chunk"]
    if nd:
        out[:nd] = _attend(case, q[:nd, None], lengths[:nd, None] - 1, table[:nd], k_cache, v_cache)[:, 0].to(q.dtype)
    if nc:
        block = min(BLOCK, c)
        nb = -(-c // block)
        row = torch.arange(nb * block, device=q.device).clamp(max=c - 1)  # the last block is filled with the last row
        pos = (lengths[nd:, None] - c + row).reshape(nc * nb, block)
        rows = q[nd:].reshape(nc, c, -1, case["d"])[:, row].reshape(nc * nb, block, -1, case["d"])
        o = _attend(case, rows, pos, table[nd:].repeat_interleave(nb, 0), k_cache, v_cache)
        out[nd:] = o.reshape(nc, nb * block, -1, case["d"])[:, :c].reshape(nc * c, -1, case["d"]).to(q.dtype)


def _plain_fork(refs, table, lengths, parents, children):
    taken = table[parents]
    table[children] = taken
    lengths[children] = lengths[parents]
    refs.index_add_(0, taken.clamp(min=0).flatten(), (taken >= 0).int().flatten())


def _plain_extend(refs, table, lengths, starts, slots, src, dst, counts, new):
    rows, pages, dev = table.shape[0], refs.shape[0], table.device
    took = (starts[1:] - starts[:-1]).long()
    end = lengths.long()
    first = (end - took) // PAGE
    cols = first[:, None] + torch.arange(-(-new // PAGE) + 1, device=dev)
    used = (cols <= ((end - 1) // PAGE)[:, None]) & (took > 0)[:, None]
    entry = table.gather(1, cols).long()
    row, head = torch.arange(rows, device=dev), entry[:, 0].clamp(min=0)
    writes = (took > 0) & ((end - took) % PAGE != 0) & (entry[:, 0] >= 0)
    shared = writes & (refs[head] > 1)
    writers = torch.zeros(pages, dtype=torch.int32, device=dev).index_add_(0, head, writes.int())
    last = torch.full((pages,), -1, dtype=torch.int64, device=dev).scatter_reduce_(0, head, torch.where(writes, row, -1), "amax")
    copies = shared & ~((writers[head] == refs[head]) & (last[head] == row))  # the last writer of a page that all its holders write to keeps it
    need = used & (entry < 0)
    need[:, 0] |= copies
    free = refs == 0
    place = torch.where(free, torch.cumsum(free, 0) - 1, pages)
    lowest = torch.zeros(pages + 1, dtype=torch.int64, device=dev).scatter_(0, place, torch.arange(pages, device=dev))
    given = lowest[(torch.cumsum(need.flatten(), 0) - 1).clamp(min=0)].view_as(need)
    refs.index_add_(0, head, -copies.int())
    refs.index_add_(0, given.flatten(), need.flatten().int())
    table.scatter_(1, cols, torch.where(need, given, entry).int())
    place = torch.where(copies, torch.cumsum(copies, 0) - 1, rows)
    src.copy_(torch.full((rows + 1,), -1, dtype=torch.int32, device=dev).scatter_(0, place, head.int())[:rows])
    dst.copy_(torch.full((rows + 1,), -1, dtype=torch.int32, device=dev).scatter_(0, place, given[:, 0].int())[:rows])
    counts.copy_(torch.stack([copies.sum(), need.sum()]))
    token = torch.arange(slots.shape[0], device=dev)
    seq = torch.searchsorted(starts, token.int(), right=True) - 1
    pos = (end - took)[seq] + token - starts[seq]
    slots.copy_(table[seq, pos // PAGE].long() * PAGE + pos % PAGE)


def _plain_copy(cache, src, dst):
    cache[dst] = cache[src]


def _plain_release(refs, table, rows, first, end):
    """Columns first .. end - 1 (per row) of the rows given."""
    col = torch.arange(table.shape[1], device=table.device)
    held = table[rows]
    drop = (held >= 0) & (col >= first) & (col < end)
    refs.index_add_(0, held.clamp(min=0).flatten(), -drop.int().flatten())
    table[rows] = torch.where(drop, -1, held)


def _plain_compact(refs, table, src, dst, counts):
    live = refs > 0
    m = live.sum()
    index = torch.arange(refs.shape[0], device=refs.device)
    holes, movers = index[~live & (index < m)], index[live & (index >= m)]
    to = index.int()
    to[movers] = holes.int()
    table.copy_(torch.where(table >= 0, to[table.clamp(min=0)], table))
    refs[holes] = refs[movers]
    refs[movers] = 0
    src.fill_(-1)[:movers.shape[0]] = movers
    dst.fill_(-1)[:movers.shape[0]] = holes
    counts.copy_(torch.stack([(live & (index >= m)).sum(), m]))
    return movers, holes


# ------------------------------------------------------------------------------------------------------------------ run

def _run_attention(st):
    case = st["case"]
    if own:
        from chunked_prefill_paged_cpa_gb300 import ops
        scales = {"k_scale": E4M3_SCALE, "v_scale": E4M3_SCALE} if case["cache"] == "e4m3" else {}
        rest = (st["k_cache"], st["v_cache"], st["table"], st["starts"], st["lengths"], case["d"] ** -0.5, st["workspace"], case["window"], case["sinks"])
        if case["append"]:
            ops.append_window_attention_forward(st["q"], st["k"], st["v"], st["slots"], *rest, out=st["out"], **scales)
        else:
            ops.window_attention_forward(st["q"], *rest, out=st["out"], **scales)
    else:
        _plain_attention(st)
    return {"out": st["out"], "k_cache": st["k_cache"], "v_cache": st["v_cache"]} if case["append"] else {"out": st["out"]}


def _run_copy(st):
    if own:
        from chunked_prefill_paged_cpa_gb300 import ops
        ops.copy_pages(st["src"], st["dst"], st["k_cache"], st["v_cache"])
    else:
        _plain_copy(st["k_cache"], st["src"], st["dst"])
        _plain_copy(st["v_cache"], st["src"], st["dst"])
    if st["k_cache"].dtype == torch.uint8:  # the codes as the values that they stand for
        return {"k_cache": st["k_cache"].view(torch.float8_e4m3fn), "v_cache": st["v_cache"].view(torch.float8_e4m3fn)}
    return {"k_cache": st["k_cache"], "v_cache": st["v_cache"]}


def _pool_outputs(st):
    return {x: st[x] for x in ("refs", "table", "lengths", "src", "dst", "counts", "slots", "k_cache", "v_cache") if x in st}


def _run_branch(st):
    refs, table, lengths, new = st["refs"], st["table"], st["lengths"], st["case"]["new"]
    st["live"].copy_(st["saved"])
    if own:
        from chunked_prefill_paged_cpa_gb300 import ops
        ops.fork_sequences(st["parents"], st["children"], table, lengths, refs, st["workspace"])
        lengths += new
        ops.extend_sequences(st["starts"], lengths, table, refs, st["slots"], st["src"], st["dst"], st["counts"], st["workspace"])
        ops.copy_pages(st["src"], st["dst"], st["k_cache"], st["v_cache"], num_pairs=st["counts"], workspace=st["workspace"])
    else:
        _plain_fork(refs, table, lengths, st["parents"], st["children"])
        lengths += new
        _plain_extend(refs, table, lengths, st["starts"], st["slots"], st["src"], st["dst"], st["counts"], new)
        named = st["src"] >= 0  # the list is filled up with its first pair, and with a page's copy to itself where it is empty
        src, dst = torch.where(named, st["src"], st["src"][:1]).clamp(min=0), torch.where(named, st["dst"], st["dst"][:1]).clamp(min=0)
        _plain_copy(st["k_cache"], src, dst)
        _plain_copy(st["v_cache"], src, dst)
    return _pool_outputs(st)


def _run_trim(st):
    refs, table, lengths, case = st["refs"], st["table"], st["lengths"], st["case"]
    st["live"].copy_(st["saved"])
    if own:
        from chunked_prefill_paged_cpa_gb300 import ops
        ops.release_pages(st["every"], table, lengths, refs, st["workspace"], window=case["window"], sinks=case["sinks"])
        ops.release_pages(st["done"], table, lengths, refs, st["workspace"])
        ops.compact_pages(table, refs, st["src"], st["dst"], st["counts"], st["workspace"])
        ops.copy_pages(st["src"], st["dst"], st["k_cache"], st["v_cache"], num_pairs=st["counts"], workspace=st["workspace"])
    else:
        end = ((lengths - case["window"] + 1).clamp(min=0) // PAGE)[:, None]
        _plain_release(refs, table, st["every"], -(-case["sinks"] // PAGE), end)
        _plain_release(refs, table, st["done"], 0, table.shape[1])
        lengths[st["done"]] = 0
        src, dst = _plain_compact(refs, table, st["src"], st["dst"], st["counts"])
        _plain_copy(st["k_cache"], src, dst)
        _plain_copy(st["v_cache"], src, dst)
    return _pool_outputs(st)


def run(state):
    return {"attention": _run_attention, "copy": _run_copy, "branch": _run_branch, "trim": _run_trim}[state["case"]["kind"]](state)


# ----------------------------------------------------------------------------------------------------------------- work

def _element(case):
    return 1 if case.get("cache") == "e4m3" else DTYPES[case["dtype"]].itemsize


def work(case):
    page = 2 * PAGE * case["hkv"] * case["d"] * _element(case)  # K and V of one page
    if case["kind"] == "attention":
        # sequence lengths at the middle of their range; each key that some row sees is read once, q read, out written
        seqs = [(1, (case["lo"] + case["hi"]) // 2)] * case["decodes"] + [(case["chunk"], case["offset"] + case["chunk"])] * case["chunks"]
        keys = pairs = 0
        for q, n in seqs:
            a, b = _visible(case, q, n)
            keys += a + n - b
            pos = torch.arange(n - q, n, dtype=torch.int64)
            low = (pos - case["window"] + 1).clamp(min=0)
            pairs += int((pos - low + 1 + low.clamp(max=case["sinks"])).sum())
        tokens = sum(q for q, _ in seqs)
        wide = DTYPES[case["dtype"]].itemsize
        moved = keys * page // PAGE + 2 * tokens * case["hq"] * case["d"] * wide + sum(-(-n // PAGE) for _, n in seqs) * 4
        if case["append"]:
            moved += 2 * tokens * case["hkv"] * case["d"] * wide + tokens * page // PAGE
        return {"bytes": moved, "flops": 4 * case["d"] * case["hq"] * pairs}
    if case["kind"] == "copy":
        return {"bytes": 2 * page * case["pairs"] + 8 * case["pairs"], "flops": 0}
    mean = (case["lo"] + case["hi"]) // 2 // PAGE + 1
    if case["kind"] == "branch":
        rows = case["rows"] + case["forks"]
        # children's rows written and their parents' read, a reference for each page; about every fork makes one copy
        words = 4 * case["forks"] * mean + 3 * rows * (2 + case["new"])
        return {"bytes": 4 * words + 2 * page * case["forks"] * (PAGE - 1) // PAGE, "flops": 0}
    kept = (case["rows"] - case["finished"]) * min(mean, -(-case["window"] // PAGE) + -(-case["sinks"] // PAGE) + 1)
    total = case["rows"] * -(-case["hi"] // PAGE) + 8
    moves = max(0, kept * (total - kept)) // max(1, total)  # live pages that lie above the packed part
    return {"bytes": 4 * (2 * case["rows"] * mean + 2 * total) + 2 * page * moves, "flops": 0}


# ---------------------------------------------------------------------------------------------------------------- exact

def exact(case, seed):
    """The attention in 64 bits, sequence by sequence; copied pages by each page's origin.  The pools' operators compute whole numbers only."""
    if case["kind"] == "copy":
        st = _prepare_copy(case, seed)
        origin = list(range(case["pages"]))
        for a, b in zip(st["src"].tolist(), st["dst"].tolist()):
            origin[b] = a
        x = [st[c].view(torch.float8_e4m3fn) if st[c].dtype == torch.uint8 else st[c] for c in ("k_cache", "v_cache")]
        return {"k_cache": x[0].double()[origin], "v_cache": x[1].double()[origin]}
    if case["kind"] != "attention":
        return None
    seqs, _ = _sequences(case, seed)
    st = _prepare_attention(case, seed)
    if case["append"]:
        flat = [st[c].transpose(1, 2).contiguous().view(-1, case["hkv"], case["d"]) for c in ("k_cache", "v_cache")]
        flat[0][st["slots"]], flat[1][st["slots"]] = st["k"], st["v"]
    else:
        flat = [st[c].transpose(1, 2).reshape(-1, case["hkv"], case["d"]) for c in ("k_cache", "v_cache")]
    group = case["hq"] // case["hkv"]
    out = torch.empty(st["q"].shape, dtype=torch.float64, device="cuda")
    token = 0
    for s, (q_len, n) in enumerate(seqs):
        for row in range(0, q_len, 512):
            rows = min(512, q_len - row)
            p = n - q_len + row + torch.arange(rows, device="cuda")
            low = max(0, n - q_len + row - case["window"] + 1)
            j = torch.cat([torch.arange(min(case["sinks"], low), device="cuda"), torch.arange(low, n - q_len + row + rows, device="cuda")])
            at = st["table"][s][j // PAGE].long() * PAGE + j % PAGE
            kk, vv = (x[at].view(torch.float8_e4m3fn).double() * E4M3_SCALE if x.dtype == torch.uint8 else x[at].double() for x in flat)
            mask = (j[None] <= p[:, None]) & ((j[None] < case["sinks"]) | (j[None] > p[:, None] - case["window"]))
            here = st["q"][token + row:token + row + rows].double()
            for h in range(case["hkv"]):
                logits = torch.einsum("rgd,jd->grj", here[:, h * group:(h + 1) * group], kk[:, h]) / case["d"] ** 0.5
                logits = torch.where(mask, logits, -torch.inf)
                weight = torch.softmax(logits, -1)
                out[token + row:token + row + rows, h * group:(h + 1) * group] = torch.einsum("grj,jd->rgd", weight, vv[:, h])
        token += q_len
    return {"out": out, "k_cache": None, "v_cache": None} if case["append"] else {"out": out}
