"""README's step over selected pages, run as it stands: prompts, single tokens, idle rows, a sequence that ends, a pool that is packed."""
import os
import re

import numpy as np
import pytest
import torch

from chunked_prefill_paged_cpa_gb300 import ops
from select_support import limit_of, select, summarise, units
from window_support import HALF

pytestmark = pytest.mark.gpu


def block():
    with open(os.path.join(os.path.dirname(__file__), "..", "README.md")) as f:
        return next(b for b in re.findall(r"```python\n(.*?)```", f.read(), re.S) if "select_pages" in b)


def test_step(cuda_device):
    dev, hq, hkv, d, pages, rows, cols, budget = cuda_device, 4, 2, 64, 120, 6, 40, 3
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    g = torch.Generator(dev).manual_seed(4)
    layers = [tuple(torch.full((pages, hkv, 16, d), float("nan"), dtype=torch.bfloat16, device=dev) for _ in range(2)) for _ in range(2)]
    layers = [(k, v, ops.summaries_for(k)) for k, v in layers]
    most = 700
    at = dict(ops=ops, torch=torch, layers=layers, scale=d ** -0.5, table=torch.full((rows, cols), -1, dtype=torch.int32, device=dev),
              lens=i32([0] * rows), refs=i32([0] * pages), pws=ops.pages_workspace_for(pages, dev), ws=ops.workspace_for(layers[0][0], hq, cols, rows, most),
              src=i32([0] * pages), dst=i32([0] * pages), counts=i32([0, 0]), packed_counts=i32([0, 0]), packed_starts=i32([0] * (rows + 1)),
              packed_lens=i32([0] * rows), packed_table=torch.full((rows, cols), -1, dtype=torch.int32, device=dev))
    said = [([], []) for _ in range(rows)]
    # (tokens of each row, rows that end)
    steps = [([300, 33, 100, 0, 200, 0], []), ([1, 1, 1, 0, 1, 0], []), ([1, 15, 0, 0, 40, 0], [0]), ([5, 1, 28, 90, 1, 0], [2]), ([12, 1, 0, 1, 130, 3], []),
             ([1, 0, 64, 7, 1, 1], [])]
    code = block()
    for q_lens, finished in steps:
        T, live = sum(q_lens), [r for r in range(rows) if q_lens[r]]
        draw = lambda h: torch.randn(T, h, d, generator=g, device=dev).bfloat16()  # noqa: E731
        at.update(q_lens=i32(q_lens), finished=i32(finished), starts=i32([sum(q_lens[:r]) for r in range(rows + 1)]), n=len(live), T=T,
                  slots=torch.zeros(T, dtype=torch.int64, device=dev), positions=torch.zeros(T, dtype=torch.int32, device=dev), q=draw(hq), k=draw(hkv),
                  v=draw(hkv), out=torch.full((T, hq, d), float("nan"), dtype=torch.bfloat16, device=dev),
                  selected=torch.full((T, hkv, budget), -1, dtype=torch.int32, device=dev))
        cut = code.index("ops.release_pages")   # between the layers and the pool's upkeep, the summaries are looked at
        exec(code[:cut], at)
        ql = [q_lens[r] for r in live]
        t = 0
        for r in live:
            said[r][0].append(at["k"][t:t + q_lens[r]])
            said[r][1].append(at["v"][t:t + q_lens[r]])
            t += q_lens[r]
        n = [sum(x.shape[0] for x in said[r][0]) for r in live]
        table = at["packed_table"][:len(live)].cpu()
        kept = layers[1][2].cpu().numpy()
        assert np.array_equal(summarise(layers[1][0], table, n, n, kept), kept)   # every full page's is there
        want = select(at["q"], kept, table, ql, n, budget, 1, 4, np.full(at["selected"].shape, -1, np.int32))
        assert np.array_equal(at["selected"].cpu().numpy(), want)
        for s, t, m, x in units(ql, n, hq // hkv):
            kk, vv = (torch.cat(y).double() for y in said[live[s]])
            limit = limit_of(x, 4)
            pos, j = x + torch.arange(m, device=dev), torch.arange(n[s], device=dev)
            for h in range(hq):
                listed = torch.zeros(-(-n[s] // 16), dtype=torch.bool, device=dev)
                listed[at["selected"][t, h // 2, :min(limit, budget)].long()] = True
                mask = (j <= pos[:, None]) & ((j >= limit * 16) | listed[j // 16])
                p = torch.softmax((at["scale"] * at["q"][t:t + m, h].double() @ kk[:, h // 2].T).masked_fill(~mask, float("-inf")), -1)
                exact, size = p @ vv[:, h // 2], p @ vv[:, h // 2].abs()
                # the output's rounding, the weights' rounding, fp32 arithmetic (window_support.tolerance)
                err = (at["out"][t:t + m, h].double() - exact).abs()
                assert (err <= HALF["bf16"] * exact.abs() + (HALF["bf16"] + 2.0 ** -13) * size).all()
        exec(code[cut:], at)
        for r in finished:
            said[r] = ([], [])
        assert at["lens"].tolist() == [sum(x.shape[0] for x in s[0]) for s in said]
    assert ops.device_status(layers[0][0], hq, cols, at["pws"]) == ops.CPA_OK
    assert ops.device_status(layers[0][0], hq, cols, at["ws"]) == ops.CPA_OK
