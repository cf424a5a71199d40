"""The windowed calls refuse malformed arguments on the host, before any launch (no GPU)."""
import ctypes

import pytest
import torch

from chunked_prefill_paged_cpa_gb300 import ops
from oracle import dense


@pytest.fixture(scope="module", autouse=True)
def lib():
    return ops.load(build_if_missing=True)


def _desc(**kw):
    d = ops.CpaDesc(32, 8, 128, 16, 1000, 64, ops.CPA_BF16, 10, None, 0)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


P = ctypes.c_void_p(4096)


def forward(window, sinks, d=None, seqs=2, scale=0.1, **null):
    a = dict(q=P, kc=P, vc=P, bt=P, qsl=P, sl=P, out=P) | null
    return ops.cpa_window_attention_forward(a["q"], a["kc"], a["vc"], a["bt"], a["qsl"], a["sl"], seqs, scale, window,
                                            sinks, a["out"], None, d or _desc())


def fused(window, sinks, d=None, seqs=2, k=P, v=P, slots=P):
    return ops.cpa_append_window_attention_forward(P, k, v, slots, P, P, P, P, P, seqs, 0.1, window, sinks, P, None,
                                                   d or _desc())


@pytest.mark.parametrize("call", [forward, fused])
def test_window_and_sinks(call):
    big = dict(workspace=4096, workspace_bytes=1 << 30)
    assert call(0, 4) == ops.CPA_ERR_ARG
    assert call(-1, 0) == ops.CPA_ERR_ARG
    assert call(16, -1) == ops.CPA_ERR_ARG
    assert call(16, 0) == ops.CPA_ERR_WORKSPACE
    assert call(2 ** 31 - 1, 2 ** 31 - 1) == ops.CPA_ERR_WORKSPACE
    # positions beyond 2^30
    assert call(16, 0, _desc(max_pages_per_seq=(1 << 26) + 1, **big)) == ops.CPA_ERR_UNSUPPORTED
    # the checks of the plain call
    assert call(16, 0, _desc(head_dim=96)) == ops.CPA_ERR_UNSUPPORTED
    assert call(16, 0, _desc(page_size=32)) == ops.CPA_ERR_UNSUPPORTED
    assert call(16, 0, _desc(**big), seqs=11) == ops.CPA_ERR_ARG
    assert call(16, 0, _desc(num_tokens=0), seqs=0) == ops.CPA_OK


def test_pointers():
    for name in ("q", "kc", "vc", "bt", "qsl", "sl", "out"):
        assert forward(16, 0, **{name: None}) == ops.CPA_ERR_ARG
    assert forward(16, 0, q=ctypes.c_void_p(4104)) == ops.CPA_ERR_ARG
    assert forward(16, 0, _desc(workspace=4096, workspace_bytes=1 << 30), scale=-1.0) == ops.CPA_ERR_ARG
    for name in ("k", "v", "slots"):
        assert fused(16, 0, **{name: None}) == ops.CPA_ERR_ARG


def test_tensors_the_library_cannot_take():
    """Checked before anything of the library is called: types, shapes, devices."""
    kc = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    q = torch.zeros(1, 4, 64, dtype=torch.bfloat16)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    ws = torch.zeros(1 << 20, dtype=torch.uint8)
    with pytest.raises(TypeError):   # queries of another type than the caches
        ops.window_attention_forward(q.float(), kc, kc.clone(), i32(1, 4), i32(2), i32(1), 0.1, ws, 8)
    with pytest.raises(ValueError):  # tensors on the host
        ops.window_attention_forward(q, kc, kc.clone(), i32(1, 4), i32(2), i32(1), 0.1, ws, 8)


def test_plain_visibility():
    """The dense oracle's windowed visibility, by counting."""
    seen = dense.visibility(3, 10, window=4, sinks=2)
    assert seen.tolist()[0] == [j in (0, 1, 4, 5, 6, 7) for j in range(10)]
    assert seen.tolist()[2] == [j in (0, 1, 6, 7, 8, 9) for j in range(10)]
    assert (dense.visibility(3, 10, window=10) == dense.visibility(3, 10)).all()
