"""Attention over selected pages against the formula in 64 bits, its edges and its refusals on the device."""
import pytest
import torch

from chunked_prefill_paged_cpa_gb300 import ops
from select_support import make_batch, reference
from window_support import tolerance

pytestmark = pytest.mark.gpu

MODES = ["bf16", "f16", "bf16-e4m3", "f16-e4m3", "f32"]


def call(b, ws=None, **kw):
    if ws is None:
        ws = workspace(b)
    return ops.selected_attention_forward(b["q"], b["k_cache"], b["v_cache"], b["table"], b["starts"], b["lens"], b["scale"], ws,
                                          b["selected"], b["local"], **b["scales"], **kw)


def workspace(b):
    return ops.workspace_for(b["k_cache"], b["q"].shape[1], b["table"].shape[1], len(b["q_lens"]), b["q"].shape[0], act_dtype=b["q"].dtype)


def check(b, **kw):
    ws = workspace(b)
    out = call(b, ws, **kw)
    want, size = reference(b)
    err = (out.double() - want).abs()
    assert (err <= tolerance(b, want, size)).all(), err.max()   # (NaN is not below)
    assert ops.device_status(b["k_cache"], b["q"].shape[1], b["table"].shape[1], ws) == ops.CPA_OK
    return out


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("hq,hkv,d", [(4, 4, 64), (4, 2, 128), (8, 2, 64), (16, 2, 128), (1, 1, 128)])
def test_single_tokens(cuda_device, mode, hq, hkv, d):
    """Lengths about the pages' edges; lists of fewer, as many and more pages than there are."""
    lens = [1, 2, 15, 16, 17, 31, 32, 33, 64, 65, 100, 500, 1000]
    for budget, local in ((0, 1), (1, 1), (3, 2), (8, 1), (70, 4)):
        check(make_batch([1] * len(lens), lens, hq, hkv, d, mode, budget, local, 3 + budget, cuda_device))


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("hq,hkv,d", [(2, 2, 128), (4, 2, 64), (8, 2, 128), (8, 1, 64)])
def test_chunks(cuda_device, mode, hq, hkv, d):
    """Chunks of less than a unit, of several and with a part of one; from odd positions; beside single tokens."""
    q_lens = [1, 2, 300, 1, 257, 16, 1, 64, 33]
    seq_lens = [700, 2, 300, 17, 900, 1016, 1, 95, 1500]
    for budget, local in ((0, 1), (2, 1), (9, 3), (200, 2)):
        check(make_batch(q_lens, seq_lens, hq, hkv, d, mode, budget, local, 5 + budget, cuda_device))


@pytest.mark.parametrize("mode", ["bf16", "f16-e4m3", "f32"])
def test_lists_in_any_order(cuda_device, mode):
    check(make_batch([1, 70, 1], [600, 800, 333], 8, 2, 64, mode, 12, 2, 7, cuda_device, rising=False))


@pytest.mark.parametrize("mode", MODES)
def test_long_contexts(cuda_device, mode):
    """One token, a few tokens and a chunk far from the first page."""
    check(make_batch([1], [60001], 8, 2, 128, mode, 128, 4, 1, cuda_device))
    check(make_batch([1, 1, 1], [20000, 31, 16016], 8, 8, 64, mode, 64, 1, 2, cuda_device))
    check(make_batch([130], [20011], 8, 2, 128, mode, 100, 4, 3, cuda_device))


@pytest.mark.parametrize("mode", ["bf16", "bf16-e4m3"])
def test_few_rows_with_long_lists(cuda_device, mode):
    """More pages than a cluster of the single tokens' kernel takes: the step kernel's splits.  (18 K keys: the weights' sums
    have 18 K / 256 terms per lane, off by less than 2^-17: inside the tolerance's 2^-13.)"""
    check(make_batch([1], [40000], 4, 1, 64, mode, 1100, 4, 4, cuda_device))


@pytest.mark.parametrize("act", ["bf16", "f16"])
def test_many_single_tokens_beside_a_chunk(cuda_device, act):
    """8-bit cache: single tokens on their own kernel beside the chunk's."""
    lens = [100 + 37 * i for i in range(64)] + [1100]
    check(make_batch([1] * 64 + [200], lens, 16, 8, 128, act + "-e4m3", 28, 4, 5, cuda_device))


@pytest.mark.parametrize("q_lens", [[1, 1, 1], [1, 20, 1]])
@pytest.mark.parametrize("what,value", [("k", float("nan")), ("k", float("inf")), ("v", float("nan")), ("v", -float("inf")), ("q", float("inf"))])
def test_fp32_keeps_what_is_not_finite(cuda_device, q_lens, what, value):
    """One element that the first sequence's row sees: NaN in its outputs (of V: in that dim), nothing elsewhere."""
    b = make_batch(q_lens, [500, 700, 300], 4, 2, 64, "f32", 6, 2, 17, cuda_device)
    good = call(b)
    page = b["table"][0, b["selected"][0, 1, 3]]
    if what == "q":
        b["q"][0, 2, 5] = value
    else:
        b["k_cache" if what == "k" else "v_cache"][page, 1, 7, 5] = value
    out = call(b)
    hit = torch.zeros_like(out, dtype=torch.bool)
    if what == "q":
        hit[0, 2] = True
    elif what == "k":
        hit[0, 2:4] = True
    else:
        hit[0, 2:4, 5] = True
    assert out[hit].isnan().all() and torch.equal(out[~hit], good[~hit])


def test_many_fp32_single_tokens(cuda_device):
    """More rows than are resident at once, and more sequences than the single tokens' kernel takes."""
    check(make_batch([1] * 90, [40 + 13 * i for i in range(90)], 16, 8, 128, "f32", 5, 1, 18, cuda_device))
    b = make_batch([1] * 4100, [17 + i % 60 for i in range(4100)], 1, 1, 64, "f32", 2, 1, 19, cuda_device)
    check(b)


def test_large_fp32_steps(cuda_device):
    """Enough tiles for four to a CTA."""
    check(make_batch([700, 1, 90], [1500, 300, 90], 32, 8, 64, "f32", 10, 2, 6, cuda_device))


def test_wide_lists_are_rows_apart(cuda_device):
    """A list far longer than the candidates, a table far wider than the context."""
    check(make_batch([1, 40], [300, 200], 4, 2, 64, "bf16", 3000, 1, 8, cuda_device, columns=5000))


def test_every_page_selected_is_causal_attention(cuda_device):
    b = make_batch([1, 50, 1], [400, 300, 17], 8, 2, 128, "bf16", 40, 1, 9, cuda_device)
    b["selected"].copy_(torch.arange(40, device=cuda_device).int())
    for c in ("k_cache", "v_cache"):
        b[c].nan_to_num_(0.0)
    full = ops.attention_forward(b["q"], b["k_cache"], b["v_cache"], b["table"], b["starts"], b["lens"], b["scale"], workspace(b))
    # two roundings of the weights and of the output; values below 6
    assert (call(b).double() - full.double()).abs().max() <= 4 * 2.0 ** -8 * 6


@pytest.mark.parametrize("mode", ["bf16", "bf16-e4m3", "f32"])
def test_bad_list_entries_raise_the_status_word(cuda_device, mode):
    """An entry that is no candidate is not read; rows of other sequences are as before."""
    for q_lens in ([1, 1, 1], [1, 40, 1]):
        b = make_batch(q_lens, [500, 700, 300], 8, 2, 64, mode, 6, 2, 10, cuda_device)
        good, ws = call(b), workspace(b)
        for bad in (-1, limit := (500 - 1) // 16 + 1 - 2, 1 << 30, -(1 << 31)):
            b["selected"][0, 0, 2] = bad
            out = call(b, ws)
            assert torch.equal(out[1:].view(torch.uint8), good[1:].view(torch.uint8)), (bad, limit)
            assert ops.device_status(b["k_cache"], 8, b["table"].shape[1], ws) == ops.CPA_ERR_DEVICE
            assert ops.device_status(b["k_cache"], 8, b["table"].shape[1], ws) == ops.CPA_OK


@pytest.mark.parametrize("mode", ["bf16", "f16-e4m3", "f32"])
def test_capture_and_other_streams(cuda_device, mode):
    """Captured, then replayed on new inputs; on a stream that is not the current one."""
    a, b = (make_batch([1, 60, 1, 1], [800, 460, 90, 33], 8, 2, 64, mode, 7, 2, seed, cuda_device) for seed in (11, 12))
    names = ("q", "k_cache", "v_cache", "table", "selected")
    ws, out = workspace(a), torch.zeros_like(a["q"])
    call(a, ws, out=out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(a, ws, out=out)
    for x in names:
        a[x].copy_(b[x])
    graph.replay()
    want, size = reference(b)
    assert ((out.double() - want).abs() <= tolerance(b, want, size)).all()
    side = torch.cuda.Stream()
    out2 = torch.zeros_like(out)
    torch.cuda.synchronize()
    call(b, workspace(b), out=out2, stream=side)
    side.synchronize()
    assert torch.equal(out2.view(torch.uint8), out.view(torch.uint8))


def test_results_do_not_vary(cuda_device):
    b = make_batch([1] * 20 + [300], [900 + 31 * i for i in range(20)] + [2000], 32, 8, 128, "bf16", 16, 3, 13, cuda_device)
    first = call(b)
    for _ in range(3):
        assert torch.equal(call(b).view(torch.int16), first.view(torch.int16))


@pytest.mark.parametrize("mode", ["bf16", "bf16-e4m3", "f32"])
def test_pages_beyond_32_bit_offsets(cuda_device, mode):
    """A pool of more than 2^32 bytes in each cache, the batch's pages at its end, for every kernel."""
    for q_lens in ([1, 1, 1], [1, 40, 1]):
        b = make_batch(q_lens, [500, 700, 300], 16, 8, 128, mode, 6, 2, 16, cuda_device)
        pages = b["k_cache"].shape[0]
        far = 2 ** 32 // (b["k_cache"][0].numel() * b["k_cache"].element_size()) + 10
        for c in ("k_cache", "v_cache"):
            pool = torch.empty(far + pages, *b[c].shape[1:], dtype=b[c].dtype, device=cuda_device)
            pool[far:] = b[c]
            b[c] = pool
        b["table"] = torch.where(b["table"] >= 0, b["table"] + far, -1)
        check(b)


def test_rows_behind_the_last_token_are_left(cuda_device):
    b = make_batch([1, 33, 1], [100, 200, 300], 8, 2, 64, "bf16", 4, 1, 14, cuda_device)
    big = torch.full((b["q"].shape[0] + 9, 8, 64), 7.0, dtype=torch.bfloat16, device=cuda_device)
    call(b, out=big[:b["q"].shape[0]])
    assert (big[b["q"].shape[0]:] == 7.0).all()
