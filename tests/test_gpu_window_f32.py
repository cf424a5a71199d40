"""fp32 windowed attention: what is not finite stays so, and fp32's precision in every shape of the kernel."""
import pytest
import torch

from test_gpu_window import check, status, window_call, workspace
from window_support import make_batch, reference, visible

from chunked_prefill_paged_cpa_gb300 import ops

pytestmark = pytest.mark.gpu

# (q_lens, seq_lens, query heads, kv heads): a tile's keys split over warps and CTAs (chunks, single tokens alone), and
# enough tiles for four to a CTA
SHAPES = {"split": ([40, 1], [300, 290], 8, 2), "tokens": ([1, 1, 1], [300, 40, 290], 8, 2), "rows": ([700], [760], 32, 8)}
# the NaN that fp32 arithmetic on the GPU gives, the same with a sign, torch's, one with its lowest bit alone; both infinities
BITS = {"gpu nan": 0x7FFFFFFF, "-gpu nan": -1, "nan": 0x7FC00000, "low nan": 0x7F800001, "inf": 0x7F800000, "-inf": -0x800000}


@pytest.mark.parametrize("bits", BITS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("shape", SHAPES)
def test_not_finite_where_a_row_sees_it(cuda_device, shape, d, bits):
    """One element of q, of K or of V: the rows that see it are not finite, the other heads keep their bits."""
    q_lens, seq_lens, hq, hkv = SHAPES[shape]
    window, sinks, group = 200, 4, hq // hkv
    b = make_batch(q_lens, seq_lens, hq, hkv, d, "f32", window, sinks, 7, cuda_device, poison=False)
    ws = workspace(b)
    good = window_call(b, ws)
    check(b, good)
    raw = lambda t: t.view(torch.int32)  # noqa: E731
    x = dict(b, q=b["q"].clone())
    raw(x["q"])[0, 1, 5] = BITS[bits]
    got = window_call(x, ws)
    assert not torch.isfinite(got[0, 1]).any()
    got[0, 1] = good[0, 1]
    assert torch.equal(raw(got), raw(good))
    n, q = seq_lens[0], q_lens[0]
    for pos in (1, n - 1 - q // 2):  # a sink; a key inside the windows
        page, off = int(b["table"][0, pos // 16]), pos % 16
        sees = visible(torch.arange(n - q, n), torch.tensor([pos]), window, sinks)[:, 0].to(cuda_device)
        for c in ("k_cache", "v_cache"):
            x = dict(b, **{c: b[c].clone()})
            raw(x[c])[page, 0, off, 5] = BITS[bits]
            got = window_call(x, ws)
            of_head = got[:q, :group][sees]
            assert of_head.numel() and not torch.isfinite(of_head if c == "k_cache" else of_head[:, :, 5]).any()
            assert torch.equal(raw(got[:, group:]), raw(good[:, group:]))  # the other kv heads'
            assert torch.equal(raw(got[q:]), raw(good[q:]))                # the other sequences'
            if c == "k_cache":
                assert torch.equal(raw(got[:q, :group][~sees]), raw(good[:q, :group][~sees]))
    assert status(b, ws) == ops.CPA_OK


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("shape", SHAPES)
def test_precision(cuda_device, shape, d):
    """A score is off by 2^-21 of its d products at most, each with a sign of its own: 2^-21 scale sqrt(sum (q k)^2) = 2^-21
    for N(0, 1) inputs; P V's products the same, and the sums of some hundred terms add about as much: 2^-19 is four
    times one of these.  One product of the three left out would cost 2^-12."""
    q_lens, seq_lens, hq, hkv = SHAPES[shape]
    b = make_batch(q_lens, seq_lens, hq, hkv, d, "f32", 200, 4, 90, cuda_device)
    want, _ = reference(b)
    err = (window_call(b, workspace(b)).double() - want).norm() / want.norm()
    assert err < 2.0 ** -19


@pytest.mark.parametrize("q_lens,seq_lens", [([0], [1]), ([0, 0, 0], [5, 0, 9])])
def test_the_append_is_done_behind_a_batch_without_rows(cuda_device, q_lens, seq_lens):
    """A malformed step (tokens, and no row that owns one): nothing is computed, and what follows on the stream finds every
    new row in the cache."""
    tokens, hkv, d = 60_000, 8, 128
    g = torch.Generator(cuda_device).manual_seed(1)
    draw = lambda h: torch.randn(tokens, h, d, generator=g, device=cuda_device)  # noqa: E731
    q, k, v = draw(hkv), draw(hkv), draw(hkv)
    pages = tokens // 16
    caches = [torch.full((pages, hkv, 16, d), float("nan"), device=cuda_device) for _ in range(2)]
    slots = torch.randperm(tokens, generator=g, device=cuda_device)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=cuda_device)  # noqa: E731
    table = torch.arange(len(q_lens) * 8, device=cuda_device).int().view(-1, 8)
    ws = ops.workspace_for(caches[0], hkv, 8, len(q_lens), tokens)
    out = torch.full_like(q, 7)
    for _ in range(3):
        for c in caches:
            c.fill_(float("nan"))
        ops.append_window_attention_forward(q, k, v, slots, *caches, table, i32([0] * (len(q_lens) + 1)), i32(seq_lens), 0.1, ws, 40, 4,
                                            out=out)
        got = [c + 0 for c in caches]  # right behind the call
        for c, x in zip(got, (k, v)):
            assert torch.equal(c[slots // 16, :, slots % 16], x)
        assert (out == 7).all()
