"""Refusals of the selection, the attention over selected pages and the packing, before any launch (no GPU); the host's forms by hand."""
import ctypes

import numpy as np
import pytest
import torch

from chunked_prefill_paged_cpa_gb300 import ops
from select_support import select, starts_of, summarise, unit_codes, units


@pytest.fixture(scope="module", autouse=True)
def lib():
    return ops.load(build_if_missing=True)


P = ctypes.c_void_p(4096)
ODD = ctypes.c_void_p(4098)
OFF8 = ctypes.c_void_p(4104)
BIG = dict(workspace=4096, workspace_bytes=1 << 30)


def desc(**kw):
    d = ops.CpaDesc(32, 8, 128, 16, 1000, 64, ops.CPA_BF16, 10, None, 0)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def attend(d=None, n=2, scale=0.1, pages=4, local=1, **x):
    a = dict(q=P, kc=P, vc=P, bt=P, qsl=P, sl=P, sel=P, out=P) | x
    return ops.cpa_selected_attention_forward(a["q"], a["kc"], a["vc"], a["bt"], a["qsl"], a["sl"], n, scale, a["sel"], pages, local, a["out"], None,
                                              d or desc(**BIG))


def choose(d=None, n=2, pages=4, sinks=1, local=1, **x):
    a = dict(q=P, sum=P, bt=P, qsl=P, sl=P, sel=P) | x
    return ops.cpa_select_pages(a["q"], a["sum"], a["bt"], a["qsl"], a["sl"], n, pages, sinks, local, a["sel"], None, d or desc())


def summary(d=None, n=2, **x):
    a = dict(kc=P, bt=P, qsl=P, sl=P, sum=P) | x
    return ops.cpa_summarise_pages(a["kc"], a["bt"], a["qsl"], a["sl"], n, a["sum"], d or desc(), None)


def pack(d=None, n=2, rows=4, **x):
    a = dict(req=P, new=P, bt=P, tl=P, qsl=P, sl=P, out=P, pos=P, slots=P, counts=P) | x
    return ops.cpa_pack_step(a["req"], a["new"], n, a["bt"], a["tl"], rows, a["qsl"], a["sl"], a["out"], a["pos"], a["slots"], a["counts"], d or desc(), None)


def test_attention_refuses():
    assert attend(pages=-1) == attend(local=0) == attend(local=-5) == ops.CPA_ERR_ARG
    assert attend(pages=(1 << 26) + 1) == ops.CPA_ERR_UNSUPPORTED
    for name in ("q", "kc", "vc", "bt", "qsl", "sl", "sel", "out"):
        assert attend(**{name: None}) == ops.CPA_ERR_ARG, name
    assert attend(sel=ODD) == attend(q=OFF8) == attend(scale=-1.0) == ops.CPA_ERR_ARG
    assert attend(desc()) == attend(desc(workspace=4096, workspace_bytes=512)) == ops.CPA_ERR_WORKSPACE
    assert attend(desc(**BIG, head_dim=96)) == attend(desc(**BIG, max_pages_per_seq=(1 << 26) + 1)) == ops.CPA_ERR_UNSUPPORTED
    assert attend(n=11) == ops.CPA_ERR_ARG
    assert attend(desc(num_tokens=0), n=0, sel=None) == ops.CPA_OK


def test_selection_refuses():
    assert choose(pages=-1) == choose(sinks=-1) == choose(local=0) == choose(n=-1) == choose(n=11) == ops.CPA_ERR_ARG
    for name in ("q", "sum", "bt", "qsl", "sl", "sel"):
        assert choose(**{name: None}) == ops.CPA_ERR_ARG, name
    assert choose(sum=OFF8) == choose(q=OFF8) == choose(sel=ODD) == choose(bt=ODD) == ops.CPA_ERR_ARG
    assert choose(desc(max_pages_per_seq=0)) == ops.CPA_ERR_ARG
    assert choose(desc(max_pages_per_seq=262145)) == choose(desc(num_pages=1 << 27)) == choose(desc(page_size=32)) == ops.CPA_ERR_UNSUPPORTED
    assert choose(desc(num_pages=1 << 26, num_kv_heads=32)) == ops.CPA_ERR_UNSUPPORTED
    assert choose(desc(num_tokens=5000), n=4097) == ops.CPA_ERR_UNSUPPORTED
    assert choose(desc(workspace=4100, workspace_bytes=256)) == choose(desc(workspace=4096, workspace_bytes=64)) == ops.CPA_ERR_WORKSPACE
    assert choose(pages=0, sel=None) == choose(desc(num_tokens=0)) == choose(n=0) == ops.CPA_OK


def test_summaries_refuse():
    for name in ("kc", "bt", "qsl", "sl", "sum"):
        assert summary(**{name: None}) == ops.CPA_ERR_ARG, name
    assert summary(kc=OFF8) == summary(sum=OFF8) == summary(qsl=ODD) == summary(n=-1) == ops.CPA_ERR_ARG
    assert summary(n=4097) == summary(desc(head_dim=80)) == summary(desc(max_pages_per_seq=(1 << 26) + 1)) == ops.CPA_ERR_UNSUPPORTED
    assert summary(desc(max_pages_per_seq=1 << 22), n=512) == ops.CPA_ERR_UNSUPPORTED
    assert summary(desc(workspace=4096, workspace_bytes=64)) == ops.CPA_ERR_WORKSPACE
    assert summary(n=0) == ops.CPA_OK
    copy = lambda s, d, n, m, at, ds: ops.cpa_copy_summaries(s, d, n, m, at, ds, None)  # noqa: E731
    assert copy(P, P, None, -1, P, desc()) == copy(None, P, None, 1, P, desc()) == copy(P, P, None, 1, None, desc()) == ops.CPA_ERR_ARG
    assert copy(P, P, ODD, 1, P, desc()) == copy(P, P, None, 1, OFF8, desc()) == ops.CPA_ERR_ARG
    assert copy(P, P, None, 1, P, desc(head_dim=80)) == ops.CPA_ERR_UNSUPPORTED
    assert copy(None, None, None, 0, None, desc()) == ops.CPA_OK
    assert ops.cpa_summary_bytes(desc()) == 1000 * 8 * 272 and ops.cpa_summary_bytes(desc(head_dim=64)) == 1000 * 8 * 144
    assert ops.cpa_summary_bytes(desc(head_dim=96)) == 0


def test_packing_refuses():
    for name in ("new", "bt", "tl", "qsl", "sl", "out", "pos", "slots", "counts"):
        assert pack(**{name: None}) == ops.CPA_ERR_ARG, name
        assert pack(**{name: ODD}) == ops.CPA_ERR_ARG, name
    assert pack(req=ODD) == pack(n=-1) == pack(rows=-1) == pack(req=None, n=5) == ops.CPA_ERR_ARG
    assert pack(desc(num_pages=0)) == pack(desc(max_pages_per_seq=0)) == pack(desc(num_tokens=-1)) == ops.CPA_ERR_ARG
    assert pack(n=4097, rows=5000) == pack(desc(page_size=32)) == pack(desc(num_pages=1 << 27)) == pack(desc(num_tokens=1 << 30)) == ops.CPA_ERR_UNSUPPORTED
    assert pack(desc(workspace=4096, workspace_bytes=64)) == ops.CPA_ERR_WORKSPACE


def test_tensors_the_library_cannot_take():
    """Checked before anything of the library is called: types, shapes, devices."""
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    kc, q, ws = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16), torch.zeros(1, 4, 64, dtype=torch.bfloat16), torch.zeros(1 << 20, dtype=torch.uint8)
    sums = torch.zeros(4, 2, 144, dtype=torch.uint8)
    with pytest.raises(ValueError):  # on the host
        ops.selected_attention_forward(q, kc, kc.clone(), i32(1, 4), i32(2), i32(1), 0.1, ws, i32(1, 2, 4))
    with pytest.raises(ValueError):
        ops.select_pages(q, sums, i32(1, 4), i32(2), i32(1), i32(1, 2, 4))
    with pytest.raises(TypeError):
        ops.select_pages(q.double(), sums, i32(1, 4), i32(2), i32(1), i32(1, 2, 4))
    with pytest.raises(ValueError):
        ops.summarise_pages(kc, i32(1, 4), i32(2), i32(1), sums)
    with pytest.raises(ValueError):
        ops.copy_summaries(i32(1), i32(1), sums)
    with pytest.raises(ValueError):
        ops.pack_step(None, i32(1), i32(1, 4), i32(1), i32(2), i32(1), i32(1, 4), i32(3), torch.zeros(3, dtype=torch.int64), i32(2))


def test_the_host_forms_by_hand():
    """Two tokens of a chunk, two heads, four full pages of keys along one axis."""
    assert units([1, 70, 64], [5, 100, 64], 4) == [(0, 0, 1, 4), (1, 1, 64, 30), (1, 65, 6, 94), (2, 71, 64, 0)]
    cache = torch.zeros(5, 1, 16, 64)
    for page, (a, b) in enumerate([(1.0, -1.0), (4.0, 3.0), (2.0, -8.0), (0.5, 0.25)]):
        cache[page, 0, :, 0] = torch.linspace(a, b, 16)
    table = torch.tensor([[0, 1, 2, 3, 4]], dtype=torch.int32)
    rows = summarise(cache, table, [66], [66], np.zeros((5, 1, 144), np.uint8))
    assert rows[:, 0, 0].view(np.int8).tolist() == [127, 127, 32, 127, 0]         # 2 * 127 / 8 = 31.75
    assert rows[:, 0, 64].view(np.int8).tolist() == [-127, 95, -127, 64, 0]       # 3 * 127 / 4 = 95.25, 63.5 to even
    assert np.allclose(rows[:, 0, 128:132].copy().view(np.float32)[:, 0], [1 / 127, 4 / 127, 8 / 127, 0.5 / 127, 0])
    q = torch.zeros(2, 1, 64)
    q[0, 0, 0], q[1, 0, 0] = 1.0, -1.0
    assert unit_codes(q[:1, 0].numpy())[0] == 127 and unit_codes(q[:, 0].numpy())[[0, 64]].tolist() == [127, -127]
    none = np.full((2, 1, 2), -1, np.int32)
    # position 65 alone: the largest product is page 1's, then page 2's; of its negative page 2's, then page 0's
    assert select(q[:1], rows, table, [1], [66], 2, 0, 1, none[:1])[0, 0].tolist() == [1, 2]
    assert select(q[1:], rows, table, [1], [66], 2, 0, 1, none[:1])[0, 0].tolist() == [0, 2]
    # both as a unit: bounds 1 + 1, 4 - 3, 2 + 8, 0.5 - 0.25
    assert select(q, rows, table, [2], [66], 1, 0, 1, none[..., :1])[0, 0].tolist() == [2]
    assert select(q, rows, table, [2], [66], 2, 0, 2, none)[0, 0].tolist() == [0, 2]
    assert select(q, rows, table, [2], [66], 2, 2, 1, none)[0, 0].tolist() == [0, 1]   # sinks first
    assert starts_of([1, 3]).tolist() == [0, 1, 4]
