"""README's serving loop, run as it stands: prompts, forks, a sequence that ends and leaves its row idle."""
import os
import re

import pytest
import torch

from chunked_prefill_paged_cpa_gb300 import ops
from window_support import HALF, visible

pytestmark = pytest.mark.gpu


def loop():
    with open(os.path.join(os.path.dirname(__file__), "..", "README.md")) as f:
        return next(b for b in re.findall(r"```python\n(.*?)```", f.read(), re.S) if "fork_sequences" in b)


def test_serving_loop(cuda_device):
    dev, hq, hkv, d, pages, rows, cols, window, sinks = cuda_device, 4, 2, 64, 100, 8, 20, 40, 4
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    g = torch.Generator(dev).manual_seed(3)
    # two layers; their caches start with NaN everywhere
    layers = [tuple(torch.full((pages, hkv, 16, d), float("nan"), dtype=torch.bfloat16, device=dev) for _ in range(2)) for _ in range(2)]
    at = dict(ops=ops, torch=torch, layers=layers, window=window, sinks=sinks, scale=d ** -0.5,
              table=torch.full((rows, cols), -1, dtype=torch.int32, device=dev), lens=i32([0] * rows), refs=i32([0] * pages),
              pws=ops.pages_workspace_for(pages, dev), ws=ops.workspace_for(layers[0][0], hq, cols, rows, 300),
              src=i32([0] * pages), dst=i32([0] * pages), counts=i32([0, 0]))
    said = [([], []) for _ in range(rows)]
    # (forks, tokens of each row, rows that end): the prompts; samples of two of them; six rows while two are idle; one that
    # takes an idle row's place
    steps = [([], [70, 33, 100, 0, 0, 0, 0, 0], []), ([(0, 3), (0, 4), (1, 5), (2, 6), (2, 7)], [1] * 8, [1, 4]),
             ([], [1, 0, 1, 1, 0, 1, 1, 1], []), ([(6, 1)], [1, 1, 5, 1, 0, 1, 30, 1], [0]), ([], [0, 2, 1, 1, 0, 1, 1, 1], [])]
    for forks, q_lens, finished in steps:
        T = sum(q_lens)
        for a, b in forks:
            said[b] = tuple(list(x) for x in said[a])
        draw = lambda h: torch.randn(T, h, d, generator=g, device=dev).bfloat16()  # noqa: E731
        at.update(parents=i32([a for a, _ in forks]), children=i32([b for _, b in forks]), q_lens=i32(q_lens), finished=i32(finished),
                  starts=i32([sum(q_lens[:r]) for r in range(rows + 1)]), slots=torch.zeros(T, dtype=torch.int64, device=dev),
                  live=torch.tensor([r for r in range(rows) if q_lens[r]], device=dev), q=draw(hq), k=draw(hkv), v=draw(hkv),
                  out=torch.full((T, hq, d), float("nan"), dtype=torch.bfloat16, device=dev))
        exec(loop(), at)
        t = 0
        for r, ql in enumerate(q_lens):
            if not ql:
                continue
            said[r][0].append(at["k"][t:t + ql])
            said[r][1].append(at["v"][t:t + ql])
            kk, vv = (torch.cat(x).double() for x in said[r])
            n = kk.shape[0]
            mask = visible(torch.arange(n - ql, n, device=dev), torch.arange(n, device=dev), window, sinks)
            for h in range(hq):
                p = torch.softmax((at["scale"] * at["q"][t:t + ql, h].double() @ kk[:, h // 2].T).masked_fill(~mask, float("-inf")), -1)
                want, size = p @ vv[:, h // 2], p @ vv[:, h // 2].abs()
                # the output's rounding, the weights' rounding, fp32 arithmetic (window_support.tolerance)
                err = (at["out"][t:t + ql, h].double() - want).abs()
                assert (err <= HALF["bf16"] * want.abs() + (HALF["bf16"] + 2.0 ** -13) * size).all()
            t += ql
        for r in finished:
            said[r] = ([], [])
        held = torch.bincount(at["table"][at["table"] >= 0].long(), minlength=pages)
        assert torch.equal(held.int(), at["refs"])
        assert at["lens"].tolist() == [sum(x.shape[0] for x in s[0]) for s in said]
    assert ops.device_status(layers[0][0], hq, cols, at["pws"]) == ops.CPA_OK
    assert ops.device_status(layers[0][0], hq, cols, at["ws"]) == ops.CPA_OK
