"""A pool of pages on the host: the page operators one step at a time, as their definitions say."""
import torch

PAGE = 16


class Pool:
    """``table`` [rows][columns] (-1: none), ``lens``, ``refs`` as plain lists."""

    def __init__(self, rows, columns, pages):
        self.table = [[-1] * columns for _ in range(rows)]
        self.lens = [0] * rows
        self.refs = [0] * pages

    @classmethod
    def random(cls, lengths, rows, columns, pages, seed, shared=0.0):
        """Rows of the given lengths on random pages; with probability ``shared`` a row begins with pages of the row before."""
        g = torch.Generator().manual_seed(seed)
        p = cls(rows, columns, pages)
        order, at = torch.randperm(pages, generator=g).tolist(), 0
        for r, n in enumerate(lengths):
            k = -(-n // PAGE)
            m = 0
            if r and torch.rand(1, generator=g).item() < shared:
                m = min(k, sum(x >= 0 for x in p.table[r - 1])) // 2
            for c in range(k):
                if c < m:
                    p.table[r][c] = p.table[r - 1][c]
                else:
                    p.table[r][c] = order[at]
                    at += 1
                p.refs[p.table[r][c]] += 1
            p.lens[r] = n
        return p

    def fork(self, parents, children):
        rows, bad = len(self.table), False
        good = []
        for i, (a, b) in enumerate(zip(parents, children)):
            ok = 0 <= a < rows and 0 <= b < rows and b not in parents and list(children).count(b) == 1
            if ok and all(x < 0 for x in self.table[b]):
                good.append((a, b))
            else:
                bad = True
        for a, b in good:
            self.table[b] = list(self.table[a])
            self.lens[b] = self.lens[a]
            for x in self.table[a]:
                if x >= 0:
                    self.refs[x] += 1
        return bad

    def extend(self, q_lens):
        """Slots, pairs, pages taken; None where the pool is too small (then nothing changed)."""
        free = [x for x, r in enumerate(self.refs) if r == 0]
        keep = [list(r) for r in self.table], list(self.refs)
        pairs, taken = [], 0
        held = list(self.refs)  # before the call
        first = [self.table[s][(self.lens[s] - q) // PAGE] if q and (self.lens[s] - q) % PAGE else -1 for s, q in enumerate(q_lens)]
        for s, q in enumerate(q_lens):
            n = self.lens[s]
            if q == 0:
                continue
            for c in range((n - q) // PAGE, (n - 1) // PAGE + 1):
                x = self.table[s][c]
                write = x < 0
                if not write and held[x] > 1 and c * PAGE < n - q:
                    # the last of the rows that write to it so keeps it, if all its references are theirs
                    last = len(first) - 1 - first[::-1].index(x)
                    if not (s == last and first.count(x) == held[x]):
                        write = True
                        self.refs[x] -= 1
                        pairs.append((x, free[taken] if taken < len(free) else -1))
                elif not write and held[x] > 1:
                    write = True
                    self.refs[x] -= 1
                if write:
                    if taken < len(free):
                        self.table[s][c] = free[taken]
                        self.refs[free[taken]] = 1
                    taken += 1
        if taken > len(free):
            self.table, self.refs = keep
            return None, [], taken
        slots = []
        for s, q in enumerate(q_lens):
            for pos in range(self.lens[s] - q, self.lens[s]):
                slots.append(self.table[s][pos // PAGE] * PAGE + pos % PAGE)
        return slots, pairs, taken

    def release(self, rows, window=0, sinks=0):
        for r in rows:
            for c, x in enumerate(self.table[r]):
                gone = window == 0 or (c * PAGE >= sinks and (c + 1) * PAGE <= self.lens[r] - window + 1)
                if x >= 0 and gone:
                    self.table[r][c] = -1
                    self.refs[x] -= 1
            if window == 0:
                self.lens[r] = 0

    def compact(self):
        live = [x for x, r in enumerate(self.refs) if r > 0]
        m = len(live)
        holes = [x for x in range(m) if self.refs[x] <= 0]
        movers = [x for x in live if x >= m]
        to = dict(zip(movers, holes))
        self.table = [[to.get(x, x) for x in r] for r in self.table]
        for a, b in to.items():
            self.refs[b], self.refs[a] = self.refs[a], 0
        return list(to.items()), m

    def check(self):
        """Every reference is counted."""
        have = [0] * len(self.refs)
        for r in self.table:
            for x in r:
                if x >= 0:
                    have[x] += 1
        assert have == self.refs

    def to(self, device):
        i = dict(dtype=torch.int32, device=device)
        return torch.tensor(self.table, **i), torch.tensor(self.lens, **i), torch.tensor(self.refs, **i)
