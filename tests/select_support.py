"""Page summaries, the selection of pages and the attention over them as their definitions say, on the host or in 64 bits."""
import numpy as np
import torch

PAGE = 16
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SCALE8 = 2.0 ** -6   # per-tensor scale of the 8-bit caches
TINY = np.float32(2.0 ** -100)


def units(q_lens, seq_lens, group):
    """(sequence, packed first token, tokens, position of the first token) of every unit."""
    out, t = [], 0
    size = 256 // group
    for s, (q, n) in enumerate(zip(q_lens, seq_lens)):
        out += [(s, t + i, min(size, q - i), n - q + i) for i in range(0, q, size)]
        t += q
    return out


def limit_of(x, local):
    return max(0, x // PAGE + 1 - local)


def starts_of(q_lens):
    return torch.tensor([0] + np.cumsum(q_lens).tolist(), dtype=torch.int32)


def random_table(seq_lens, pages, seed, columns=None):
    """Block table of sequences of these lengths over a pool, -1 behind."""
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    table = torch.full((len(seq_lens), columns or max(-(-n // PAGE) for n in seq_lens) + 2), -1, dtype=torch.int32)
    at = 0
    for s, n in enumerate(seq_lens):
        k = -(-n // PAGE)
        table[s, :k] = order[at:at + k]
        at += k
    return table


# ------------------------------------------------------------------------------------------------ summaries and selection

def summary_row(keys):
    """One page's row of one kv head, uint8: keys float32 [16, d]."""
    d = keys.shape[1]
    row = np.zeros(2 * d + 16, dtype=np.uint8)
    if not np.isfinite(keys).all():
        row[2 * d:2 * d + 4] = np.array([np.inf], np.float32).view(np.uint8)
        return row
    most = np.abs(keys).max()
    if most < TINY:
        return row
    factor, scale = np.float32(127) / most, most / np.float32(127)
    for at, bound in ((0, keys.max(0)), (d, keys.min(0))):
        row[at:at + d] = np.rint(bound * factor).astype(np.int8).view(np.uint8)
    row[2 * d:2 * d + 4] = np.array([scale], np.float32).view(np.uint8)
    return row


def key_values(cache):
    """A cache's values in fp32, without the 8-bit cache's scale."""
    return (cache.view(torch.float8_e4m3fn) if cache.dtype == torch.uint8 else cache).float().cpu().numpy()


def summarise(cache, table, q_lens, seq_lens, rows):
    """``rows`` (numpy uint8 [pages, hkv, 2 d + 16]) after the step's complete pages were summarised."""
    keys, rows = key_values(cache), rows.copy()
    for s, (q, n) in enumerate(zip(q_lens, seq_lens)):
        for c in range((n - q) // PAGE if q else 0, n // PAGE if q else 0):
            page = int(table[s, c])
            if 0 <= page < rows.shape[0]:
                for g in range(rows.shape[1]):
                    rows[page, g] = summary_row(keys[page, g])
    return rows


def unit_codes(q):
    """A and B of one unit and kv head: q float32 [rows, d]."""
    if not np.isfinite(q).all() or np.abs(q).max() < TINY:
        return np.zeros(2 * q.shape[1], dtype=np.int64)
    c = np.rint(q * (np.float32(127) / np.abs(q).max())).astype(np.int64)
    up, down = np.maximum(c, 0).sum(0), np.maximum(-c, 0).sum(0)
    h = 0
    while max(up.max(), down.max()) >> h > 127:
        h += 1
    half = (1 << h) // 2
    return np.concatenate([np.minimum(127, (up + half) >> h), -np.minimum(127, (down + half) >> h)])


def select(q, rows, table, q_lens, seq_lens, budget, sinks, local, selected):
    """``selected`` (int32 numpy [T, hkv, budget]) after the selection."""
    qn, selected, hkv = q.float().cpu().numpy(), selected.copy(), rows.shape[1]
    d = qn.shape[2]
    codes, scales = rows[:, :, :2 * d].view(np.int8).astype(np.int64), rows[:, :, 2 * d:2 * d + 4].copy().view(np.float32)[..., 0]
    group = qn.shape[1] // hkv
    for s, t, n, x in units(q_lens, seq_lens, group):
        limit = limit_of(x, local)
        entries = np.asarray(table[s, :limit])
        bad = (entries < 0) | (entries >= rows.shape[0])
        page = np.where(bad, 0, entries)
        for g in range(hkv):
            mine = qn[t:t + n, g * group:(g + 1) * group]
            if x != seq_lens[s] - q_lens[s]:   # not the first unit: a short one's last token counts for those it lacks
                mine = np.concatenate([mine, np.repeat(mine[-1:], 256 // group - n, 0)])
            whole = unit_codes(mine.reshape(-1, d))
            with np.errstate(over="ignore", invalid="ignore"):
                score = scales[page, g] * (codes[page, g] @ whole).astype(np.float32)
            score[~(scales[page, g] < np.inf)] = np.inf
            score[:sinks] = np.inf
            key = score.astype(np.float64)
            key[bad] = -np.inf   # behind all others (the scores here are finite or +infinity)
            best = np.sort(np.argsort(-key, kind="stable")[:budget])
            selected[t, g] = -1
            selected[t, g, :best.size] = best
    return selected


# ---------------------------------------------------------------------------------------------------------- the attention

def make_batch(q_lens, seq_lens, hq, hkv, d, mode, budget, local, seed, device, spare=5, rising=True, columns=None):
    """One step's tensors over random lists.  ``mode`` as in window_support.  Every (page, kv head) that no unit sees, the free
    pages and the slots past each sequence hold NaN; the lists' rows behind their n entries, and those of other tokens than a
    unit's first, hold numbers that are no pages."""
    act, e4m3 = DTYPES[mode.split("-")[0]], mode.endswith("e4m3")
    g = torch.Generator().manual_seed(seed)
    T = sum(q_lens)
    need = sum(-(-n // PAGE) for n in seq_lens)
    table = random_table(seq_lens, need + spare, seed, columns)
    selected = torch.full((T, hkv, budget), 1 << 30, dtype=torch.int32)
    us = units(q_lens, seq_lens, hq // hkv)
    seen = [torch.zeros(hkv, -(-n // PAGE), dtype=torch.bool) for n in seq_lens]
    for s, t, n, x in us:
        limit = limit_of(x, local)
        k = min(limit, budget)
        for h in range(hkv):
            pages = torch.randperm(limit, generator=g)[:k]
            selected[t, h, :k] = pages.sort().values if rising else pages
            seen[s][h, pages] = True
        seen[s][:, limit:(x + n - 1) // PAGE + 1] = True
    shape = (need + spare, hkv, PAGE, d)
    caches = [torch.full(shape, 0x7F, dtype=torch.uint8) if e4m3 else torch.full(shape, float("nan"), dtype=act) for _ in range(2)]
    dense = []
    for s, n in enumerate(seq_lens):
        values = []
        keep = seen[s].repeat_interleave(PAGE, 1)[:, :n]
        h, pos = keep.nonzero(as_tuple=True)
        for c in caches:
            x = torch.randn(hkv, n, d, generator=g).to(act)
            if e4m3:
                x = (x.float() / SCALE8).clamp(-448, 448).to(torch.float8_e4m3fn)
                c[table[s, pos // PAGE].long(), h, pos % PAGE] = x.view(torch.uint8)[h, pos]
                values.append(x.double() * SCALE8)
            else:
                c[table[s, pos // PAGE].long(), h, pos % PAGE] = x[h, pos]
                values.append(x.double())
        dense.append([v.to(device) for v in values])
    b = dict(q=torch.randn(T, hq, d, generator=g).to(act), k_cache=caches[0], v_cache=caches[1], table=table, starts=starts_of(q_lens),
             lens=torch.tensor(seq_lens, dtype=torch.int32), selected=selected)
    b = {k: t.to(device) for k, t in b.items()}
    b.update(dense=dense, q_lens=list(q_lens), seq_lens=list(seq_lens), budget=budget, local=local, mode=mode, units=us,
             scales={"k_scale": SCALE8, "v_scale": SCALE8} if e4m3 else {}, scale=d ** -0.5)
    return b


def reference(b):
    """(out, bound) in 64 bits: the formula, and for each output sum_j p_j |v_j|, the size of what the roundings act on."""
    q = b["q"].double()
    out, size = torch.empty_like(q), torch.empty_like(q)
    for s, t, n, x in b["units"]:
        k, v = b["dense"][s]
        limit = limit_of(x, b["local"])
        pos = x + torch.arange(n, device=q.device)
        j = torch.arange(k.shape[1], device=q.device)
        group = q.shape[1] // k.shape[0]
        for h in range(k.shape[0]):
            listed = torch.zeros(-(-k.shape[1] // PAGE), dtype=torch.bool, device=q.device)
            listed[b["selected"][t, h, :min(limit, b["budget"])].long()] = True
            mask = (j <= pos[:, None]) & ((j >= limit * PAGE) | listed[j // PAGE])
            for i in range(h * group, (h + 1) * group):
                p = torch.softmax((b["scale"] * q[t:t + n, i] @ k[h].T).masked_fill(~mask, float("-inf")), -1)
                out[t:t + n, i] = p @ v[h]
                size[t:t + n, i] = p @ v[h].abs()
    return out, size
