"""Cases of the attention over selected pages, the operators that select them, and the packing of a step, with their plain forms.

A page holds 16 tokens.  A *unit* is the tokens of a step that share a selection: a decode's one token, and of a chunk runs of
256 / (query heads per kv head) tokens counted from its first.  With x the position of a unit's first token and
L = max(0, x // 16 + 1 - local), the unit sees pages from L on (each row up to its own position) and the pages selected among
0 .. L - 1, which are full.  Kinds of case ("kind"):

* ``summarise``: rows of the pages' summaries copied along with moved pages, then the pages that a step's tokens complete
  summarised: per kv head the largest and the smallest key element by element, as whole numbers of at most 127 times a scale.
* ``select``: for every unit and kv head the ``budget`` pages whose bounds allow the largest logits, summed over the unit's rows.
* ``attend``: attention of the packed batch (decodes, then chunks) over the selected pages.
* ``step``: append, summarise, select and attend, as one layer of a step makes them.
* ``pack``: a step's metadata from the list of requests, their new tokens, their lengths and their rows of the page table.

``run`` computes them from elementary torch operations, or, where ``own`` is true, through the package's entry points.
"""
import torch

own = False

PAGE = 16
E4M3_SCALE = 2.0 ** -6      # K and V of an 8-bit cache are codes of x / 2^-6
BLOCK = 64                  # units that the plain form takes together

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ---------------------------------------------------------------------------------------------------------------- cases

def _case(name, kind, **values):
    return dict(kind=kind, **values) | ({"name": name} if name else {})


def _batch(name, kind, decodes, lo, hi, chunks, chunk, offset, budget, sinks, local, hq, hkv, d, dtype="bf16", cache="same"):
    return _case(name, kind, decodes=decodes, lo=lo, hi=hi, chunks=chunks, chunk=chunk, offset=offset, budget=budget, sinks=sinks, local=local,
                 hq=hq, hkv=hkv, d=d, dtype=dtype, cache=cache)


def _summarise(name, decodes, lo, hi, chunks, chunk, offset, moved, hkv, d, dtype="bf16", cache="same"):
    return _case(name, "summarise", decodes=decodes, lo=lo, hi=hi, chunks=chunks, chunk=chunk, offset=offset, moved=moved, hkv=hkv, d=d, dtype=dtype,
                 cache=cache)


def _pack(name, rows, requests, lo, hi, new, columns):
    return _case(name, "pack", rows=rows, requests=requests, lo=lo, hi=hi, new=new, columns=columns)


def listed():
    return [
        # one user's next token deep in a long document: the latency of a single call
        _batch("attend_one", "attend", 1, 100000, 100000, 0, 0, 0, 128, 1, 4, 32, 8, 128),
        # a full batch of single tokens over long contexts, 2048 keys of each selected: the cache's bandwidth
        _batch("attend_batch", "attend", 128, 8192, 32768, 0, 0, 0, 128, 1, 4, 32, 8, 128),
        # a larger batch over the 8-bit cache, half the budget
        _batch("attend_e4m3", "attend", 256, 4096, 16384, 0, 0, 0, 64, 1, 4, 32, 8, 128, cache="e4m3"),
        # a long prompt's next chunk, binary16: the tensor cores
        _batch("attend_chunk", "attend", 0, 0, 0, 1, 2048, 30720, 128, 1, 4, 32, 8, 128, dtype="f16"),
        # the high-resolution configuration: fp32, few heads, an odd chunk beside decodes
        _batch("attend_f32", "attend", 7, 100, 2000, 1, 333, 500, 16, 1, 2, 8, 2, 64, dtype="f32"),
        # the selection for one user's next token deep in a long document: latency
        _batch("select_one", "select", 1, 100000, 100000, 0, 0, 0, 128, 1, 4, 32, 8, 128),
        # the selection for a full batch of single tokens: the summaries' bandwidth
        _batch("select_batch", "select", 256, 4096, 16384, 0, 0, 0, 64, 1, 4, 32, 8, 128),
        # eight prompts prefilled, a pool packed before: the keys' bandwidth
        _summarise("summarise_prompt", 0, 0, 0, 8, 8192, 0, 1024, 8, 128),
        # a full batch's next tokens, of which one in sixteen completes a page, 8-bit cache: latency
        _summarise("summarise_step", 256, 512, 4096, 0, 0, 0, 16, 8, 128, cache="e4m3"),
        # one layer of a hybrid step: decodes beside a chunk of a long prompt
        _batch("step_hybrid", "step", 64, 4096, 16384, 1, 512, 15872, 64, 1, 4, 32, 8, 128),
        # a handful of requests
        _pack("pack_few", 16, 8, 100, 2000, 1, 256),
        # a large server's step: many decodes, some chunks, long tables
        _pack("pack_many", 2048, 1024, 512, 32000, 300, 2048),
    ]


def _log(rng, lo, hi):
    """An integer from lo to hi, spread over its logarithm."""
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    """One more case: most are batches (attend, select, step), the others summaries and packing."""
    kind = rng.choice(["attend", "attend", "attend", "select", "select", "step", "summarise", "pack"])
    if kind == "pack":
        requests = _log(rng, 1, 1000)
        lo = _log(rng, 1, 2000)
        hi = lo + _log(rng, 30, 20000)
        return _pack(None, requests + rng.randrange(0, 200), requests, lo, hi, _log(rng, 1, 300), -(-hi // PAGE) + rng.randrange(0, 50))
    hkv, d = rng.choice([1, 2, 4, 8]), rng.choice([64, 128])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    cache = rng.choice(["same", "same", "e4m3"]) if dtype != "f32" else "same"
    form = rng.choice(["decode", "decode", "chunk", "hybrid"])
    decodes = 0 if form == "chunk" else _log(rng, 1, 60 if dtype == "f32" else 128)
    chunks = 0 if form == "decode" else rng.choice([1, 1, 2, 3])
    chunk = _log(rng, 2, 400 if dtype == "f32" else 1000) if chunks else 0
    offset = rng.choice([0, _log(rng, 1, 12000)]) if chunks else 0
    lo = _log(rng, 1, 6000)
    hi = lo + _log(rng, 20, 10000)
    if kind == "summarise":
        return _summarise(None, decodes, lo, hi, chunks, chunk, offset, _log(rng, 1, 200), hkv, d, dtype, cache)
    g = rng.choice([x for x in (1, 2, 4, 8) if x * hkv <= 32])
    return _batch(None, kind, decodes, lo, hi, chunks, chunk, offset, _log(rng, 1, 128), rng.choice([0, 1, 1, 2]), rng.choice([1, 2, 4, rng.randrange(3, 9)]),
                  hkv * g, hkv, d, dtype, cache)


# --------------------------------------------------------------------------------------------------------------- inputs

def _normal(shape, dtype, gen):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def _cache(case, pages, gen):
    """K and V of every page, N(0, 1); an 8-bit cache as codes."""
    shape = (pages, case["hkv"], PAGE, case["d"])
    out = []
    for _ in range(2):
        if case["cache"] == "e4m3":
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


def _random_summaries(case, pages, gen):
    """Summaries of pages of N(0, 1) keys: bounds about +-1.77, the largest magnitude about 4."""
    d = case["d"]
    out = torch.zeros((pages, case["hkv"], 2 * d + 16), dtype=torch.uint8, device="cuda")
    for p in range(0, pages, 4096):
        rows = out[p:p + 4096]
        bounds = torch.randn(rows.shape[:2] + (2, d), generator=gen, device="cuda") * 0.5 + torch.tensor([[1.77], [-1.77]], device="cuda")
        scale = bounds.abs().amax((2, 3)) / 127 * (1 + 0.2 * torch.rand(rows.shape[:2], generator=gen, device="cuda"))
        rows[:, :, :2 * d] = (bounds / scale[:, :, None, None]).round().to(torch.int8).view(torch.uint8).flatten(2)
        rows[:, :, 2 * d:2 * d + 4] = scale[:, :, None].contiguous().view(torch.uint8)
    return out


def _int(x, dtype=torch.int32):
    return torch.as_tensor(x, dtype=dtype).cuda()


def _sequences(case, seed):
    """(new tokens, length) of every sequence of a batch."""
    g = torch.Generator().manual_seed(seed)
    n = case["decodes"]
    seqs = [(1, x) for x in torch.randint(case["lo"], case["hi"] + 1, (n,), generator=g).tolist()] if n else []
    return seqs + [(case["chunk"], case["offset"] + case["chunk"])] * case["chunks"], g


def _tables(case, seed):
    """Block table, starts, lengths and slots of a batch, whose pages are drawn from a pool."""
    seqs, g = _sequences(case, seed)
    columns = max(-(-n // PAGE) for _, n in seqs) + 1
    table = torch.full((len(seqs), columns), -1, dtype=torch.int32)
    held = torch.arange(columns)[None] < torch.tensor([-(-n // PAGE) for _, n in seqs])[:, None]
    # the pool's size does not depend on the seed
    pages = case["decodes"] * -(-case["hi"] // PAGE) + case["chunks"] * -(-(case["offset"] + case["chunk"]) // PAGE) + 1 + 2 * case.get("moved", 0)
    order = torch.randperm(pages, generator=g).to(torch.int32)
    table[held] = order[:int(held.sum())]
    starts, slots = [0], []
    for s, (q, n) in enumerate(seqs):
        pos = torch.arange(n - q, n)
        slots.append(table[s, pos // PAGE].long() * PAGE + pos % PAGE)
        starts.append(starts[-1] + q)
    return {"case": case, "table": table.cuda(), "starts": _int(starts), "lengths": _int([n for _, n in seqs]), "slots": torch.cat(slots).cuda()}, pages, order


def _prepare_batch(case, seed):
    st, pages, _ = _tables(case, seed)
    gen = torch.Generator("cuda").manual_seed(seed)
    kind, dtype = case["kind"], DTYPES[case["dtype"]]
    tokens = st["slots"].shape[0]
    st["q"] = _normal((tokens, case["hq"], case["d"]), dtype, gen)
    st["selected"] = torch.full((tokens, case["hkv"], case["budget"]), -1, dtype=torch.int32, device="cuda")
    if kind == "select":
        st["summaries"] = _random_summaries(case, pages, gen)
        return st
    st["k_cache"], st["v_cache"] = _cache(case, pages, gen)
    st["out"] = torch.empty((tokens, case["hq"], case["d"]), dtype=dtype, device="cuda")
    if kind == "step":
        st["k"], st["v"] = (_normal((tokens, case["hkv"], case["d"]), dtype, gen) for _ in range(2))
        st["summaries"] = torch.zeros((pages, case["hkv"], 2 * case["d"] + 16), dtype=torch.uint8, device="cuda")
        for p in range(0, pages, 4096):  # earlier steps left every page's summary
            at = torch.arange(p, min(p + 4096, pages), device="cuda")
            st["summaries"][at] = _summary_rows(_values(st["k_cache"][at], 1.0))
    else:
        for rows, _, _, first in _units(case, st["lengths"]):  # distinct pages in rising order, as many as there are
            for i in range(0, rows.shape[0], BLOCK):
                limit = first[i:i + BLOCK, None, None]
                keys = torch.rand((limit.shape[0], case["hkv"], st["table"].shape[1]), generator=gen, device="cuda")
                keys.masked_fill_(torch.arange(keys.shape[2], device="cuda") >= limit, 2.0)
                st["selected"][rows[i:i + BLOCK, 0]] = _listed_pages(keys.argsort(-1), limit, case["budget"])
    if own:  # the workspace that a user's program holds from step to step
        from chunked_prefill_paged_cpa_gb300 import ops
        st["workspace"] = ops.workspace_for(st["k_cache"], case["hq"], st["table"].shape[1], st["table"].shape[0], tokens, act_dtype=dtype)
    return st


def _prepare_summarise(case, seed):
    st, pages, order = _tables(case, seed)
    gen = torch.Generator("cuda").manual_seed(seed)
    st["k_cache"], _ = _cache(case, pages, gen)
    st["summaries"] = _random_summaries(case, pages, gen)
    spare = order[pages - 2 * case["moved"]:].cuda()  # pages that no sequence holds
    st["src"], st["dst"] = spare[:case["moved"]].contiguous(), spare[case["moved"]:].contiguous()
    return st


def _prepare_pack(case, seed):
    g = torch.Generator().manual_seed(seed)
    rows, n, columns = case["rows"], case["requests"], case["columns"]
    lengths = torch.randint(case["lo"], case["hi"] + 1, (rows,), generator=g)
    listed_rows = torch.randperm(rows, generator=g)[:n]
    # most requests take one token, every eighth up to ``new``, every sixteenth sits the step out
    took = torch.where(torch.arange(n) % 8 == 3, torch.randint(1, case["new"] + 1, (n,), generator=g), torch.ones(n, dtype=torch.int64))
    took = torch.where(torch.arange(n) % 16 == 9, 0, torch.minimum(took, lengths[listed_rows]))
    held = torch.arange(columns)[None] < ((lengths + PAGE - 1) // PAGE)[:, None]
    table = torch.full((rows, columns), -1, dtype=torch.int32)
    table[held] = torch.randperm(int(held.sum()), generator=g).to(torch.int32)
    tokens = n * case["new"]  # the step's buffers hold any such step
    st = {"case": case, "requests": _int(listed_rows), "took": _int(took), "table": table.cuda(), "lengths": _int(lengths)}
    for name, size, dtype in (("starts", n + 1, torch.int32), ("seq_lens", n, torch.int32), ("positions", tokens, torch.int32), ("slots", tokens, torch.int64),
                              ("counts", 2, torch.int32)):
        st[name] = torch.full((size,), -1, dtype=dtype, device="cuda")
    st["block_table"] = torch.full((n, columns), -1, dtype=torch.int32, device="cuda")
    return st


def prepare(case, seed):
    return {"summarise": _prepare_summarise, "pack": _prepare_pack}.get(case["kind"], _prepare_batch)(case, seed)


# ----------------------------------------------------------------------------------------------------------- plain forms

def _values(codes, scale):
    if codes.dtype == torch.uint8:
        return codes.view(torch.float8_e4m3fn).float() * scale
    return codes.float()


def _units(case, lengths):
    """Groups of units of one size: (packed tokens [u, rows], positions [u, rows], sequences [u], L [u]).  A chunk's last unit is
    filled up with its last token."""
    nd, c, dev = case["decodes"], case["chunk"], lengths.device
    size = 256 * case["hkv"] // case["hq"]
    groups = []
    if nd:
        seq = torch.arange(nd, device=dev)
        groups.append((seq[:, None], lengths[:nd, None].long() - 1, seq))
    if case["chunks"]:
        per = -(-c // size)
        row = torch.arange(per * size, device=dev).clamp(max=c - 1).view(per, size)[:, :min(size, c)]
        seq = torch.arange(case["chunks"], device=dev)
        token = (nd + seq[:, None, None] * c + row).flatten(0, 1)
        pos = (lengths[nd:, None, None].long() - c + row).flatten(0, 1)
        groups.append((token, pos, (nd + seq).repeat_interleave(per)))
    return [(t, x, s, (x[:, 0] // PAGE + 1 - case["local"]).clamp(min=0)) for t, x, s in groups]


def _listed_pages(order, limit, budget):
    """The first min(budget, limit) of each row's pages in rising order, then -1; the list has ``budget`` entries."""
    kept = order[..., :budget]
    kept = torch.where(torch.arange(kept.shape[-1], device=order.device) < limit, kept, 1 << 30).sort(-1).values
    kept = torch.where(kept == 1 << 30, -1, kept).int()
    return torch.nn.functional.pad(kept, (0, budget - kept.shape[-1]), value=-1)


def _summary_rows(keys):
    """keys [n, hkv, 16, d] in 32 bits: the summaries' rows."""
    hi, lo = keys.amax(2), keys.amin(2)
    most = keys.abs().amax((2, 3))
    fine = torch.isfinite(keys).all(3).all(2)
    used = fine & (most >= 2.0 ** -100)
    whole = torch.full_like(most, 127.0)
    inverse = torch.where(used, whole / torch.where(used, most, 1.0), 0.0)
    scale = torch.where(used, most / whole, torch.where(fine, 0.0, torch.inf))
    codes = torch.where(used[..., None], torch.cat([hi, lo], 2) * inverse[..., None], 0.0).round().to(torch.int8)
    return torch.cat([codes.view(torch.uint8), scale[..., None].contiguous().view(torch.uint8), torch.zeros(scale.shape + (12,), dtype=torch.uint8, device=keys.device)], 2)


def _plain_summarise(st):
    first, end = (st["lengths"] - (st["starts"][1:] - st["starts"][:-1])) // PAGE, st["lengths"] // PAGE
    column = torch.arange(st["table"].shape[1], device=first.device)
    pages = st["table"][(column >= first[:, None]) & (column < end[:, None])].long()
    for i in range(0, pages.shape[0], 2048):
        at = pages[i:i + 2048]
        st["summaries"][at] = _summary_rows(_values(st["k_cache"][at], 1.0))


def _unit_codes(q):
    """q [u, rows, hkv, g, d]: whole numbers [u, hkv, 2 d], by which the largest and the smallest keys are multiplied."""
    x = q.float()
    most = x.abs().amax((1, 3, 4))
    used = torch.isfinite(x).all(4).all(3).all(1) & (most >= 2.0 ** -100)
    inverse = torch.full_like(most, 127.0) / torch.where(used, most, 1.0)
    c = torch.where(used[:, None, :, None, None], x * inverse[:, None, :, None, None], 0.0).round()
    up, down = c.clamp(min=0).sum((1, 3)).long(), (-c).clamp(min=0).sum((1, 3)).long()
    top = torch.maximum(up, down).amax(2)
    shift = sum((top >= 128 << k).long() for k in range(16))[..., None]  # the least that leaves 7 bits
    half = (1 << shift) >> 1
    return torch.cat([((up + half) >> shift).clamp(max=127), -((down + half) >> shift).clamp(max=127)], 2)


def _plain_select(st):
    case, d = st["case"], st["case"]["d"]
    for token, _, seq, limit in _units(case, st["lengths"]):
        for i in range(0, token.shape[0], BLOCK):
            rows, top = token[i:i + BLOCK], limit[i:i + BLOCK, None, None]
            whole = _unit_codes(st["q"][rows].unflatten(2, (case["hkv"], -1))).float()
            score = torch.empty(whole.shape[:2] + (st["table"].shape[1],), device=whole.device)
            for c in range(0, score.shape[2], 512):
                page = st["table"][seq[i:i + BLOCK], c:c + 512].clamp(min=0).long()
                found = st["summaries"][page]
                codes = found[..., :2 * d].view(torch.int8).float()
                scale = found[..., 2 * d:2 * d + 4].contiguous().view(torch.float32)[..., 0]
                products = (codes.permute(0, 2, 1, 3) @ whole[..., None])[..., 0]  # whole numbers below 2^24
                scale = scale.transpose(1, 2)
                score[:, :, c:c + 512] = torch.where(torch.isinf(scale), torch.inf, torch.where(torch.isinf(scale), 0.0, scale) * products)
            column = torch.arange(score.shape[2], device=score.device)
            score = torch.where(column < case["sinks"], torch.inf, score + 0.0)
            score = torch.where(column < top, score, -torch.inf)
            st["selected"][rows[:, 0]] = _listed_pages(score.sort(dim=-1, descending=True, stable=True).indices, top, case["budget"])


def _plain_attend(st):
    case, q, out = st["case"], st["q"], st["out"]
    hkv, d, dev = case["hkv"], case["d"], q.device
    head = torch.arange(hkv, device=dev)[:, None]
    for token, pos, seq, limit in _units(case, st["lengths"]):
        near = -(-token.shape[1] // PAGE) + case["local"]  # pages from L to the unit's last row, and one more
        for i in range(0, token.shape[0], BLOCK):
            rows, x, top = token[i:i + BLOCK], pos[i:i + BLOCK], limit[i:i + BLOCK]
            u, r = rows.shape
            column = torch.cat([st["selected"][rows[:, 0]].long(), (top[:, None, None] + torch.arange(near, device=dev)).expand(-1, hkv, -1)], 2)
            inside = (column >= 0) & (column < st["table"].shape[1])
            page = torch.where(inside, st["table"][seq[i:i + BLOCK, None, None], torch.where(inside, column, 0)], 0).clamp(min=0).long()
            place = (column[..., None] * PAGE + torch.arange(PAGE, device=dev)).flatten(2)
            seen = inside.repeat_interleave(PAGE, 2)[:, :, None] & (place[:, :, None] <= x[:, None, :, None])
            k = _values(st["k_cache"][page, head], E4M3_SCALE).flatten(2, 3)
            v = _values(st["v_cache"][page, head], E4M3_SCALE).flatten(2, 3)
            unread = ~seen.any(2)[..., None]
            k, v = k.masked_fill(unread, 0.0), v.masked_fill(unread, 0.0)
            f = q[rows].float().unflatten(2, (hkv, -1)).permute(0, 2, 1, 3, 4).flatten(2, 3)
            s = (f @ k.transpose(2, 3)).unflatten(2, (r, -1)) * d ** -0.5
            s = s.masked_fill(~seen[:, :, :, None], -torch.inf)
            e = torch.exp(s - s.amax(-1, keepdim=True))
            e = e / e.sum(-1, keepdim=True)
            o = (e.flatten(2, 3) @ v).unflatten(2, (r, -1)).permute(0, 2, 1, 3, 4).flatten(2, 3)
            out[rows] = o.to(out.dtype)


def _plain_append(st):
    page, off = st["slots"] // PAGE, st["slots"] % PAGE
    for cache, rows in ((st["k_cache"], st["k"]), (st["v_cache"], st["v"])):
        if cache.dtype == torch.uint8:
            rows = (rows.float() / E4M3_SCALE).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        cache[page, :, off] = rows


def _plain_pack(st):
    live = st["took"] > 0
    rows, took = st["requests"][live].long(), st["took"][live]
    n, dev = rows.shape[0], rows.device
    length = st["lengths"][rows]
    end = torch.cumsum(took, 0).int()
    st["starts"][0] = 0
    st["starts"][1:n + 1] = end
    st["seq_lens"][:n] = length
    column = torch.arange(st["table"].shape[1], device=dev)
    st["block_table"][:n] = torch.where(column < ((length + PAGE - 1) // PAGE)[:, None], st["table"][rows], st["block_table"][:n])
    seq = torch.repeat_interleave(torch.arange(n, device=dev), took)
    tokens = seq.shape[0]
    pos = length[seq] - took[seq] + torch.arange(tokens, device=dev) - (end - took)[seq]
    st["positions"][:tokens] = pos
    st["slots"][:tokens] = st["table"][rows[seq], pos // PAGE].long() * PAGE + pos % PAGE
    st["counts"][0], st["counts"][1] = n, tokens


# ------------------------------------------------------------------------------------------------------------------ run

def _summary_views(st):
    """The summaries' codes and scales, without a copy."""
    d = st["case"]["d"]
    return {"codes": st["summaries"][..., :2 * d].view(torch.int8), "scales": st["summaries"][..., 2 * d:2 * d + 4].view(torch.float32)}


def _run_batch(st):
    case, kind = st["case"], st["case"]["kind"]
    where = (st["table"], st["starts"], st["lengths"])
    if own:
        from chunked_prefill_paged_cpa_gb300 import ops
        scales = {"k_scale": E4M3_SCALE, "v_scale": E4M3_SCALE} if case["cache"] == "e4m3" else {}
        if kind == "step":
            ops.kv_append(st["k"], st["v"], st["slots"], st["k_cache"], st["v_cache"], st["workspace"], **scales)
            ops.summarise_pages(st["k_cache"], *where, st["summaries"], workspace=st["workspace"])
        if kind != "attend":
            ops.select_pages(st["q"], st["summaries"], *where, st["selected"], sink_pages=case["sinks"], local_pages=case["local"], workspace=st.get("workspace"))
        if kind != "select":
            ops.selected_attention_forward(st["q"], st["k_cache"], st["v_cache"], *where, case["d"] ** -0.5, st["workspace"], st["selected"],
                                           local_pages=case["local"], out=st["out"], **scales)
    else:
        if kind == "step":
            _plain_append(st)
            _plain_summarise(st)
        if kind != "attend":
            _plain_select(st)
        if kind != "select":
            _plain_attend(st)
    outputs = {}
    if kind == "step":
        outputs = {x: st[x].view(torch.float8_e4m3fn) if st[x].dtype == torch.uint8 else st[x] for x in ("k_cache", "v_cache")} | _summary_views(st)
    if kind != "attend":
        outputs["selected"] = st["selected"]
    if kind != "select":
        outputs["out"] = st["out"]
    return outputs


def _run_summarise(st):
    if own:
        from chunked_prefill_paged_cpa_gb300 import ops
        ops.copy_summaries(st["src"], st["dst"], st["summaries"])
        ops.summarise_pages(st["k_cache"], st["table"], st["starts"], st["lengths"], st["summaries"])
    else:
        st["summaries"][st["dst"]] = st["summaries"][st["src"]]
        _plain_summarise(st)
    return _summary_views(st)


def _run_pack(st):
    if own:
        from chunked_prefill_paged_cpa_gb300 import ops
        ops.pack_step(st["requests"], st["took"], st["table"], st["lengths"], st["starts"], st["seq_lens"], st["block_table"], st["positions"], st["slots"],
                      st["counts"])
    else:
        _plain_pack(st)
    return {x: st[x] for x in ("starts", "seq_lens", "block_table", "positions", "slots", "counts")}


def run(state):
    return {"summarise": _run_summarise, "pack": _run_pack}.get(state["case"]["kind"], _run_batch)(state)


# ----------------------------------------------------------------------------------------------------------------- work

def _mean(case):
    """(new tokens, length) of every sequence, decodes at the middle of their range."""
    return [(1, (case["lo"] + case["hi"]) // 2)] * case["decodes"] + [(case["chunk"], case["offset"] + case["chunk"])] * case["chunks"]


def work(case):
    if case["kind"] == "pack":
        n, mean = case["requests"] * 15 // 16, (case["lo"] + case["hi"]) // 2
        tokens = n + n // 8 * ((case["new"] + 1) // 2 - 1)
        # the table's held entries read and written, three words of a request read, two written, position and slot of a token
        return {"bytes": n * (8 * -(-mean // PAGE) + 20) + 12 * tokens, "flops": 0}
    hkv, d = case["hkv"], case["d"]
    element = 1 if case["cache"] == "e4m3" else DTYPES[case["dtype"]].itemsize
    wide = DTYPES[case["dtype"]].itemsize
    row = 2 * d + 16
    summarised = bytes_moved = flops = 0
    if case["kind"] in ("summarise", "step"):
        for q, n in _mean(case):
            summarised += q // PAGE if q > 1 else 1 / PAGE
        bytes_moved += int(summarised * hkv * (PAGE * d * element + row))
    if case["kind"] == "summarise":
        return {"bytes": bytes_moved + 2 * case["moved"] * hkv * row + 8 * case["moved"], "flops": 0}
    tokens, size = sum(q for q, _ in _mean(case)), 256 * hkv // case["hq"]
    if case["kind"] == "step":
        bytes_moved += 2 * tokens * hkv * d * (wide + element)
    for q, n in _mean(case):
        starts = range(0, q, size)
        first = [max(0, (n - q + t) // PAGE + 1 - case["local"]) for t in starts]
        if case["kind"] != "attend":
            # every candidate's summary once, its table entry; a list for every unit
            bytes_moved += max(first) * (hkv * row + 4) + sum(4 * hkv * case["budget"] for _ in starts)
            flops += sum(4 * d * hkv * x for x in first)
        if case["kind"] != "select":
            # what a chunk's units see of the chunk and before, each page once
            far = min(max(first), sum(min(case["budget"], x) for x in first))
            bytes_moved += 2 * hkv * d * element * min(n, far * PAGE + n - first[0] * PAGE)
            for t, x in zip(starts, first):
                rows = min(size, q - t)
                seen = min(case["budget"], x) * PAGE + (n - q + t - x * PAGE)
                flops += 4 * d * case["hq"] * (rows * seen + rows * (rows + 1) // 2)
            bytes_moved += sum(4 * hkv * min(case["budget"], x) for x in first)
    bytes_moved += tokens * case["hq"] * d * wide * (1 if case["kind"] == "select" else 2)
    return {"bytes": bytes_moved, "flops": flops}


# ---------------------------------------------------------------------------------------------------------------- exact

def _wide(cache, page):
    """Pages of a cache in 64 bits, as the attention reads them."""
    x = cache[page]
    return x.view(torch.float8_e4m3fn).double() * E4M3_SCALE if x.dtype == torch.uint8 else x.double()


def _exact_bounds(keys):
    """keys [n, hkv, 16, d] in 64 bits: whole numbers [n, hkv, 2, d] and scales (the keys here are finite and not tiny)."""
    most = keys.abs().flatten(2).max(2).values
    step = (127 * torch.ones_like(most) / most).float().double()
    bounds = torch.stack([keys.max(2).values, keys.min(2).values], 2)
    return torch.round((bounds * step[:, :, None, None]).float().double()), (most / (127 * torch.ones_like(most))).float().double()


def _exact_choice(case, rows, bounds, scales, limit):
    """rows [hkv, n, d] of one unit, bounds [pages, hkv, 2, d], scales [pages, hkv]: the chosen pages of every kv head."""
    step = 127 * torch.ones_like(rows[:, 0, 0]) / rows.abs().flatten(1).max(1).values
    c = torch.round((rows * step.float().double()[:, None, None]).float().double())
    above, below = torch.relu(c).sum(1), torch.relu(-c).sum(1)
    power = torch.ones_like(above[:, :1])
    for _ in range(16):
        power = torch.where(torch.maximum(above, below).max(1, keepdim=True).values >= 128 * power, 2 * power, power)
    above, below = (torch.clamp(torch.floor(x / power + torch.where(power > 1, 0.5, 0.0)), max=127.0) for x in (above, below))
    score = (torch.einsum("jhd,hd->hj", bounds[:limit, :, 0], above) - torch.einsum("jhd,hd->hj", bounds[:limit, :, 1], below)) * scales[:limit].T
    score = score.float()
    score[:, :min(case["sinks"], limit)] = torch.inf
    return [torch.argsort(s, descending=True, stable=True)[:case["budget"]] for s in score]


def exact(case, seed):
    """The attention in 64 bits, unit by unit; whole numbers and copies have no such value."""
    if case["kind"] in ("select", "pack"):
        return None
    st = prepare(case, seed)
    if case["kind"] == "summarise":
        # (the scales' own rounding to 32 bits is part of their definition: codes are made with it)
        scales = st["summaries"][..., 2 * case["d"]:2 * case["d"] + 4].clone().view(torch.float32).double()
        scales[st["dst"].long()] = scales[st["src"].long()]
        for s, (q, n) in enumerate(_sequences(case, seed)[0]):
            page = st["table"][s, (n - q) // PAGE:n // PAGE].long()
            if page.numel():
                keys = st["k_cache"][page]
                keys = keys.view(torch.float8_e4m3fn).double() if keys.dtype == torch.uint8 else keys.double()
                scales[page, :, 0] = keys.abs().flatten(2).max(2).values / 127
        return {"codes": None, "scales": scales}
    if case["kind"] == "step":
        at, off = st["slots"] // PAGE, st["slots"] % PAGE
        for cache, new in ((st["k_cache"], st["k"]), (st["v_cache"], st["v"])):
            if cache.dtype == torch.uint8:
                new = (new.double() / E4M3_SCALE).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            cache[at, :, off] = new
    hkv, group, size = case["hkv"], case["hq"] // case["hkv"], 256 * case["hkv"] // case["hq"]
    q64, token = st["q"].double(), 0
    out = torch.empty(st["q"].shape, dtype=torch.float64, device="cuda")
    for s, (q_len, n) in enumerate(_sequences(case, seed)[0]):
        page = st["table"][s, :-(-n // PAGE)].long()
        k, v = _wide(st["k_cache"], page), _wide(st["v_cache"], page)
        if case["kind"] == "step":
            full = n // PAGE
            bounds, scales = _exact_bounds(k[:full] / (E4M3_SCALE if case["cache"] == "e4m3" else 1.0)) if full else (None, None)
        for t in range(0, q_len, size):
            rows = min(size, q_len - t)
            x = n - q_len + t + torch.arange(rows, device="cuda")
            limit = max(0, (n - q_len + t) // PAGE + 1 - case["local"])
            mine = q64[token + t:token + t + rows].unflatten(1, (hkv, group)).permute(1, 0, 2, 3)
            if case["kind"] == "step":
                chosen = _exact_choice(case, mine.flatten(1, 2), bounds, scales, limit) if limit else [torch.empty(0, dtype=torch.int64, device="cuda")] * hkv
            else:
                chosen = [row[:min(case["budget"], limit)].long() for row in st["selected"][token + t]]
            tail = torch.arange(limit, (n - q_len + t + rows - 1) // PAGE + 1, device="cuda")
            columns = torch.stack([torch.cat([c, tail]) for c in chosen])
            head = torch.arange(hkv, device="cuda")[:, None]
            kk, vv = (z[columns, head].flatten(1, 2) for z in (k, v))
            place = (columns[..., None] * PAGE + torch.arange(PAGE, device="cuda")).flatten(1)
            logits = torch.einsum("hrgd,hjd->hrgj", mine, kk) / case["d"] ** 0.5
            logits = torch.where(place[:, None, None] <= x[:, None, None], logits, -torch.inf)
            o = torch.einsum("hrgj,hjd->hrgd", torch.softmax(logits, -1), vv)
            out[token + t:token + t + rows] = o.permute(1, 0, 2, 3).flatten(1, 2)
        token += q_len
    if case["kind"] == "step":
        return {"k_cache": None, "v_cache": None, "codes": None, "scales": None, "selected": None, "out": out}
    return {"out": out}
