"""Inputs and the plain 64-bit form of attention with a sliding window and sinks."""
import torch

PAGE = 16
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SCALE8 = 2.0 ** -6   # per-tensor scale of the 8-bit caches


def visible(positions, keys, window, sinks):
    """[rows, keys] matrix: which keys the rows at these positions see."""
    p, j = positions[:, None], keys[None]
    return (j <= p) & ((j < sinks) | (j > p - window))


def make_batch(q_lens, seq_lens, hq, hkv, d, mode, window, sinks, seed, device, spare=5, poison=True):
    """One step's tensors.  ``mode``: "bf16", "f16", "f32", or "bf16-e4m3" / "f16-e4m3" (8-bit caches).

    Pages that no row sees have no entry in the block table (-1); every cache position that no row of its sequence sees,
    the free pages and the slots past each sequence hold NaN."""
    act = DTYPES[mode.split("-")[0]]
    e4m3 = mode.endswith("e4m3")
    g = torch.Generator().manual_seed(seed)
    S, T = len(q_lens), sum(q_lens)
    cols = max(-(-n // PAGE) for n in seq_lens) + 2
    table = torch.full((S, cols), -1, dtype=torch.int32)
    kv, seen_pages = [], []
    for s, (q, n) in enumerate(zip(q_lens, seq_lens)):
        seen = visible(torch.arange(n - q, n)[:1], torch.arange(n), window, sinks)[0]
        seen |= torch.arange(n) >= n - q                   # and everything from the first row on
        pages = torch.zeros(-(-n // PAGE), dtype=torch.bool)
        pages[torch.arange(n)[seen] // PAGE] = True
        seen_pages.append(pages if poison else torch.ones_like(pages))
        kv.append((torch.randn(n, hkv, d, generator=g), torch.randn(n, hkv, d, generator=g), seen))
    need = sum(int(p.sum()) for p in seen_pages)
    order = torch.randperm(need + spare, generator=g)[:need].to(torch.int32)
    at = 0
    for s, p in enumerate(seen_pages):
        k = int(p.sum())
        table[s, :p.numel()][p] = order[at:at + k]
        at += k
    shape = (need + spare, hkv, PAGE, d)
    if e4m3:
        caches = [torch.full(shape, 0x7F, dtype=torch.uint8) for _ in range(2)]
    else:
        caches = [torch.full(shape, float("nan"), dtype=act) for _ in range(2)]
    dense, new_k, new_v, slots = [], [], [], []
    for s, (q, n) in enumerate(zip(q_lens, seq_lens)):
        pos = torch.arange(n)
        keep = kv[s][2] if poison else torch.ones(n, dtype=torch.bool)
        page, off = table[s, pos // PAGE][keep].long(), (pos % PAGE)[keep]
        values = []
        for c, x in zip(caches, kv[s][:2]):
            if e4m3:  # the codes of the rows as the append is given them
                codes = (x.to(act).float() / SCALE8).clamp(-448, 448).to(torch.float8_e4m3fn)
                c[page, :, off] = codes.view(torch.uint8)[keep]
                values.append(codes.double() * SCALE8)
            else:
                c[page, :, off] = x.to(act)[keep]
                values.append(x.to(act).double())
        dense.append([v.to(device) for v in values])
        new_k.append(kv[s][0][n - q:].to(act))
        new_v.append(kv[s][1][n - q:].to(act))
        p = torch.arange(n - q, n)
        slots.append(table[s, p // PAGE].long() * PAGE + p % PAGE)
    starts = torch.zeros(S + 1, dtype=torch.int32)
    starts[1:] = torch.cumsum(torch.tensor(q_lens, dtype=torch.int32), 0)
    b = dict(q=torch.randn(T, hq, d, generator=g).to(act), k=torch.cat(new_k), v=torch.cat(new_v),
             slots=torch.cat(slots), k_cache=caches[0], v_cache=caches[1], table=table, starts=starts,
             lens=torch.tensor(seq_lens, dtype=torch.int32))
    b = {k: t.to(device) for k, t in b.items()}
    b.update(dense=dense, q_lens=list(q_lens), seq_lens=list(seq_lens), window=window, sinks=sinks, mode=mode,
             scales={"k_scale": SCALE8, "v_scale": SCALE8} if e4m3 else {}, scale=d ** -0.5)
    return b


def reference(b):
    """(out, bound) in 64 bits: the formula, and for each output sum_j p_j |v_j|, the size of what the roundings act on."""
    q = b["q"].double()
    out, size = torch.empty_like(q), torch.empty_like(q)
    t = 0
    for (k, v), ql, n in zip(b["dense"], b["q_lens"], b["seq_lens"]):
        pos = torch.arange(n - ql, n, device=q.device)
        mask = visible(pos, torch.arange(n, device=q.device), b["window"], b["sinks"])
        group = q.shape[1] // k.shape[1]
        for h in range(q.shape[1]):
            s = b["scale"] * q[t:t + ql, h] @ k[:, h // group].T
            p = torch.softmax(s.masked_fill(~mask, float("-inf")), -1)
            out[t:t + ql, h] = p @ v[:, h // group]
            size[t:t + ql, h] = p @ v[:, h // group].abs()
        t += ql
    return out, size


# Half a step of each type, relative to the value.
HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}


def tolerance(b, want, size):
    """|error| at most, per output.  The output's own rounding; the rounding of each softmax weight to the type that the
    tensor cores multiply (16-bit steps: the caches' type, binary16 for 8-bit caches): half a step of p_j |v_j| summed;
    and the fp32 arithmetic of the scores: a score is a sum of d products, off by at most (d + 2) 2^-24 sum |q k| scale,
    which is below 2^-14 for N(0, 1) inputs (sum |q k| scale < 0.64 d^0.5 * 1.5 = 11 for d = 128, 130 * 11 * 2^-24 < 2^-13.5;
    the sum's random walk stays far below the bound), the weights' sums are off by less, and binary16 weights below 2^-14
    are off by at most 2^-25 of the largest each: 2^-13 of the size covers them for contexts up to 4096."""
    act, _, cache = b["mode"].partition("-")
    p = HALF["f16"] if cache else (HALF[act] if act != "f32" else 0.0)
    return HALF[act] * want.abs() + (p + 2.0 ** -13) * size
