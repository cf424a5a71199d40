"""The page operators' checks on the host (no GPU: nothing is launched), and the host pool that the GPU tests compare with."""
import ctypes

import pytest
import torch

from chunked_prefill_paged_cpa_gb300 import ops
from pages_support import Pool


@pytest.fixture(scope="module", autouse=True)
def lib():
    return ops.load(build_if_missing=True)


P = ctypes.c_void_p(4096)
ODD = ctypes.c_void_p(4098)


def desc(**kw):
    d = ops.CpaDesc(8, 2, 128, 16, 1000, 64, ops.CPA_BF16, 10, 4096, 1 << 20)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


CALLS = {
    "fork": lambda d, table=P, refs=P, n=2, rows=4, x=P: ops.cpa_fork_sequences(x, P, n, table, P, rows, refs, d, None),
    "extend": lambda d, table=P, refs=P, n=2, rows=4, x=P: ops.cpa_extend_sequences(x, P, n, table, refs, P, P, P, P, d, None),
    "release": lambda d, table=P, refs=P, n=2, rows=4, x=P: ops.cpa_release_pages(P, n, table, x, rows, 0, 0, refs, d, None),
    "compact": lambda d, table=P, refs=P, n=2, rows=4, x=P: ops.cpa_compact_pages(table, n, refs, P, P, x, d, None),
}


@pytest.mark.parametrize("call", CALLS.values(), ids=CALLS.keys())
def test_table_operators_refuse(call):
    assert call(desc(num_pages=0)) == ops.CPA_ERR_ARG
    assert call(desc(max_pages_per_seq=0)) == ops.CPA_ERR_ARG
    assert call(desc(page_size=32)) == ops.CPA_ERR_UNSUPPORTED
    assert call(desc(num_pages=1 << 27)) == ops.CPA_ERR_UNSUPPORTED
    assert call(desc(max_pages_per_seq=(1 << 26) + 1)) == ops.CPA_ERR_UNSUPPORTED
    assert call(desc(), table=None) == ops.CPA_ERR_ARG
    assert call(desc(), table=ODD) == ops.CPA_ERR_ARG
    assert call(desc(), refs=None) == ops.CPA_ERR_ARG
    assert call(desc(), refs=ctypes.c_void_p(4104)) == ops.CPA_ERR_ARG
    assert call(desc(), n=-1) == ops.CPA_ERR_ARG
    assert call(desc(), x=None) == ops.CPA_ERR_ARG
    assert call(desc(), x=ODD) == ops.CPA_ERR_ARG
    assert call(desc(workspace=None)) == ops.CPA_ERR_WORKSPACE
    assert call(desc(workspace=4100)) == ops.CPA_ERR_WORKSPACE
    assert call(desc(workspace_bytes=ops.cpa_pages_workspace_bytes(1000) - 1)) == ops.CPA_ERR_WORKSPACE


def test_sizes():
    assert CALLS["fork"](desc(), n=5, rows=4) == ops.CPA_ERR_ARG
    assert CALLS["fork"](desc(), n=4097, rows=5000) == ops.CPA_ERR_UNSUPPORTED
    assert CALLS["fork"](desc(), n=0) == ops.CPA_OK
    assert CALLS["extend"](desc(), n=4097) == ops.CPA_ERR_UNSUPPORTED
    assert CALLS["release"](desc(), n=0) == ops.CPA_OK
    rel = lambda w, s, rows=P, n=2: ops.cpa_release_pages(rows, n, P, P, 4, w, s, P, desc(), None)  # noqa: E731
    assert rel(-1, 0) == rel(16, -1) == rel(0, 4) == ops.CPA_ERR_ARG
    assert rel(0, 0, rows=None, n=5) == ops.CPA_ERR_ARG


def test_workspace_bytes():
    f = ops.cpa_pages_workspace_bytes
    assert f(0) == f(-4) == f(1 << 27) == 0
    assert f(1) == 512 and f(100_000) >= 256 + 400_000 and f(100_000) % 256 == 0


def test_copy_refuses():
    f = ops.cpa_copy_pages
    assert f(P, P, None, -1, P, P, desc(), None) == ops.CPA_ERR_ARG
    assert f(P, P, None, 0, None, None, desc(), None) == ops.CPA_OK
    assert f(None, P, None, 1, P, P, desc(), None) == ops.CPA_ERR_ARG
    assert f(P, None, None, 1, P, P, desc(), None) == ops.CPA_ERR_ARG
    assert f(P, P, ODD, 1, P, P, desc(), None) == ops.CPA_ERR_ARG
    assert f(P, P, None, 1, ctypes.c_void_p(4104), P, desc(), None) == ops.CPA_ERR_ARG
    assert f(P, P, None, 1, P, None, desc(), None) == ops.CPA_ERR_ARG
    assert f(P, P, None, 1, P, P, desc(head_dim=80), None) == ops.CPA_ERR_UNSUPPORTED
    assert f(P, P, None, 1, P, P, desc(workspace_bytes=64), None) == ops.CPA_ERR_WORKSPACE


def test_binding_checks_its_tensors():
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    ws = torch.zeros(4096, dtype=torch.uint8)
    with pytest.raises(ValueError):  # on the host
        ops.compact_pages(i32(2, 4), i32(16), i32(16), i32(16), i32(2), ws)
    with pytest.raises(TypeError):
        ops.release_pages(None, i32(2, 4), i32(2), torch.zeros(16), ws)
    with pytest.raises(ValueError):
        ops.copy_pages(i32(2), i32(2), torch.zeros(4, 2, 16, 64), torch.zeros(4, 2, 16, 64))


def test_the_host_pool_by_hand():
    """20 tokens on two pages, forked twice: the copies of the second page, by hand."""
    p = Pool(3, 3, 8)
    p.table[0][:2], p.lens[0] = [5, 1], 20
    p.refs[5] = p.refs[1] = 1
    assert not p.fork([0, 0], [1, 2])
    assert p.refs[5] == p.refs[1] == 3
    p.lens = [21, 21, 21]
    slots, pairs, taken = p.extend([1, 1, 1])
    assert pairs == [(1, 0), (1, 2)] and taken == 2 and slots == [4, 36, 20]
    assert p.table == [[5, 0, -1], [5, 2, -1], [5, 1, -1]] and p.refs == [1, 1, 1, 0, 0, 3, 0, 0]
    p.release([1], 3, 0)      # position 21 sees 19, 20, 21: page 0 is out
    assert p.table[1] == [-1, 2, -1] and p.refs[5] == 2
    moves, m = p.compact()
    assert m == 4 and moves == [(5, 3)] and p.refs == [1, 1, 1, 2, 0, 0, 0, 0]
    p.release([0, 1, 2])
    assert sum(p.refs) == 0
    p.check()
