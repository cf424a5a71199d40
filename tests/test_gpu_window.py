"""Attention with a sliding window and sinks on the GPU, against the formula in 64 bits."""
import pytest
import torch

from chunked_prefill_paged_cpa_gb300 import ops
from window_support import make_batch, reference, tolerance

pytestmark = pytest.mark.gpu

MODES = ["bf16", "f16", "f32", "bf16-e4m3", "f16-e4m3"]
# (window, sinks): one key; sinks alone; page edges; odd; past a tile; past every context; all sinks
WINDOWS = [(1, 0), (1, 1), (16, 0), (17, 4), (100, 33), (128, 16), (129, 130), (1000, 4), (5000, 0), (3, 5000)]
# decodes of one key up to several pages, chunks from scratch, one-page chunks, chunks with an unaligned prefix
MIXED = ([1, 1, 1, 37, 130, 1, 2, 300], [1, 17, 700, 37, 900, 2049, 50, 300])


def workspace(b):
    return ops.workspace_for(b["k_cache"], b["q"].shape[1], b["table"].shape[1], len(b["q_lens"]),
                             b["q"].shape[0], act_dtype=b["q"].dtype)


def window_call(b, ws, append=False, out=None):
    rest = (b["k_cache"], b["v_cache"], b["table"], b["starts"], b["lens"], b["scale"], ws, b["window"], b["sinks"])
    if append:
        return ops.append_window_attention_forward(b["q"], b["k"], b["v"], b["slots"], *rest, out=out, **b["scales"])
    return ops.window_attention_forward(b["q"], *rest, out=out, **b["scales"])


def check(b, got, what=""):
    want, size = reference(b)
    err = (got.double() - want).abs()
    assert torch.isfinite(got).all(), f"{what}: non-finite output"
    over = err > tolerance(b, want, size)
    assert not over.any(), f"{what}: {int(over.sum())} outputs off, worst {float(err[over].max()):.3e}"


def status(b, ws):
    return ops.device_status(b["k_cache"], b["q"].shape[1], b["table"].shape[1], ws)


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("window,sinks", WINDOWS)
def test_mixed_batch(cuda_device, mode, window, sinks):
    b = make_batch(*MIXED, 8, 2, 128, mode, window, sinks, 11 + window, cuda_device)
    ws = workspace(b)
    out = window_call(b, ws)
    assert status(b, ws) == ops.CPA_OK
    check(b, out, f"{mode} {window} {sinks}")


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 3), (4, 2), (12, 3), (8, 1), (32, 8)])
def test_heads(cuda_device, mode, d, hq, hkv):
    b = make_batch([1, 70, 1, 1], [333, 200, 16, 1500], hq, hkv, d, mode, 77, 5, 500 + hq, cuda_device)
    ws = workspace(b)
    check(b, window_call(b, ws), f"{mode} {hq}/{hkv} {d}")
    assert status(b, ws) == ops.CPA_OK


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("seed", range(4))
def test_ragged(cuda_device, mode, seed):
    """Random lengths, windows and sinks, several chunks in one step."""
    g = torch.Generator().manual_seed(900 + seed)
    r = lambda lo, hi: int(torch.randint(lo, hi + 1, (1,), generator=g))  # noqa: E731
    q_lens = [r(1, 400) if r(0, 2) == 0 else 1 for _ in range(9)]
    seq_lens = [q + r(0, 2500) for q in q_lens]
    b = make_batch(q_lens, seq_lens, 8, 2, 64, mode, r(1, 700), r(0, 60), 950 + seed, cuda_device)
    ws = workspace(b)
    check(b, window_call(b, ws), f"{mode} {q_lens} {seq_lens}")
    assert status(b, ws) == ops.CPA_OK


@pytest.mark.parametrize("mode", MODES)
def test_append_in_the_same_call(cuda_device, mode):
    """The cache's bytes and the output's bits are those of the two separate calls."""
    b = make_batch(*MIXED, 8, 2, 128, mode, 150, 4, 31, cuda_device)
    whole = [b["k_cache"].clone(), b["v_cache"].clone()]
    page, off = b["slots"] // 16, b["slots"] % 16
    for c in ("k_cache", "v_cache"):
        b[c][page, :, off] = 0x7F if b[c].dtype == torch.uint8 else float("nan")
    k1, v1 = b["k_cache"].clone(), b["v_cache"].clone()
    ops.kv_append(b["k"], b["v"], b["slots"], k1, v1, **b["scales"])
    out1 = window_call(dict(b, k_cache=k1, v_cache=v1), workspace(b))
    out2 = window_call(b, workspace(b), append=True)
    raw = lambda t: t.view(torch.uint8)  # noqa: E731
    for got, sep, want in ((b["k_cache"], k1, whole[0]), (b["v_cache"], v1, whole[1])):
        assert torch.equal(raw(got), raw(sep)) and torch.equal(raw(got), raw(want))
    assert torch.equal(raw(out1), raw(out2))
    check(b, out2, mode)


@pytest.mark.parametrize("mode", ["bf16", "f32", "bf16-e4m3"])
def test_long_context_costs_only_its_window(cuda_device, mode):
    """Decodes and a chunk far behind their sinks: only the visible pages exist."""
    b = make_batch([1, 40, 1], [100_000, 70_000, 65_537], 4, 1, 64, mode, 200, 20, 7, cuda_device)
    ws = workspace(b)
    check(b, window_call(b, ws), mode)
    assert status(b, ws) == ops.CPA_OK


@pytest.mark.parametrize("mode", ["bf16", "bf16-e4m3"])
def test_split_over_the_context(cuda_device, mode):
    """One long decode and one short chunk with a long window: both split over many CTAs and merged."""
    b = make_batch([1, 20], [4090, 4000], 8, 1, 128, mode, 3900, 40, 8, cuda_device)
    ws = workspace(b)
    check(b, window_call(b, ws), mode)


def test_many_sequences(cuda_device):
    g = torch.Generator().manual_seed(3)
    lens = torch.randint(1, 60, (4096,), generator=g).tolist()
    b = make_batch([1] * 4096, lens, 4, 2, 64, "bf16", 21, 3, 4, cuda_device)
    ws = workspace(b)
    check(b, window_call(b, ws))


@pytest.mark.parametrize("mode", ["bf16", "f32", "f16-e4m3"])
def test_jumps_of_the_logits_at_the_windows_edge(cuda_device, mode):
    """Large keys just outside the window (they must not move the softmax) and just inside."""
    b = make_batch([1, 90], [500, 400], 4, 2, 64, mode, 100, 7, 21, cuda_device, poison=False)
    q0 = b["q"][0, 0].double() * 4
    for s, n in enumerate(b["seq_lens"]):
        for pos in (7, n - b["q_lens"][s] - 100, n - 100, n - 101):
            page, off = int(b["table"][s, pos // 16]), pos % 16
            row = q0.to(b["q"].dtype).double()
            if b["k_cache"].dtype == torch.uint8:
                codes = (row / 2.0 ** -6).clamp(-448, 448).to(torch.float8_e4m3fn)
                b["k_cache"][page, :, off] = codes.view(torch.uint8)
                b["dense"][s][0][pos] = codes.double() * 2.0 ** -6
            else:
                b["k_cache"][page, :, off] = row.to(b["k_cache"].dtype)
                b["dense"][s][0][pos] = row.to(b["k_cache"].dtype).double()
    want, size = reference(b)
    got = window_call(b, workspace(b)).double()
    # these scores reach |s| = 4 sum |q|^2 scale < 64: the fp32 bound of the scores grows by 64 / 11 < 8
    tol = tolerance(b, want, size) + 7 * 2.0 ** -13 * size
    assert ((got - want).abs() <= tol).all()


def test_bad_page_inside_the_window_is_reported(cuda_device):
    b = make_batch([1], [300], 4, 2, 64, "bf16", 50, 4, 5, cuda_device)
    ws = workspace(b)
    b["table"][0, 300 // 16] = 1 << 20
    window_call(b, ws)
    assert status(b, ws) == ops.CPA_ERR_DEVICE
    assert status(b, ws) == ops.CPA_OK


@pytest.mark.parametrize("mode", ["bf16", "f32"])
def test_captured_and_replayed(cuda_device, mode):
    b = make_batch(*MIXED, 8, 2, 64, mode, 60, 4, 41, cuda_device)
    ws, out = workspace(b), torch.empty_like(b["q"])
    eager = window_call(b, ws, append=True).clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        window_call(b, ws, append=True, out=out)
    for _ in range(3):
        out.zero_()
        ws[256:].random_(0, 256)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager)
    b["q"].mul_(-1)
    graph.replay()
    torch.cuda.synchronize()
    check(b, out, "replayed on new queries")


def test_on_another_stream(cuda_device):
    b = make_batch(*MIXED, 8, 2, 64, "bf16", 60, 4, 43, cuda_device)
    want = window_call(b, workspace(b))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    ws = workspace(b)
    s.wait_stream(torch.cuda.current_stream())
    got = ops.window_attention_forward(b["q"], b["k_cache"], b["v_cache"], b["table"], b["starts"], b["lens"],
                                       b["scale"], ws, 60, 4, stream=s)
    s.synchronize()
    assert torch.equal(got, want)


# ---- steps of single tokens alone

TOKENS = [1, 2, 15, 16, 17, 40, 130, 700, 2049, 4000]


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("window,sinks", WINDOWS)
def test_single_tokens(cuda_device, mode, window, sinks):
    b = make_batch([1] * len(TOKENS), TOKENS, 8, 2, 128, mode, window, sinks, 60 + window, cuda_device)
    ws = workspace(b)
    check(b, window_call(b, ws), f"{mode} {window} {sinks}")
    assert status(b, ws) == ops.CPA_OK


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (6, 3), (4, 1), (8, 1), (32, 8), (16, 2)])
def test_single_tokens_heads(cuda_device, mode, d, hq, hkv):
    b = make_batch([1] * 3, [333, 5, 1500], hq, hkv, d, mode, 400, 5, 510 + hq, cuda_device)
    ws = workspace(b)
    check(b, window_call(b, ws), f"{mode} {hq}/{hkv} {d}")
    assert status(b, ws) == ops.CPA_OK


@pytest.mark.parametrize("mode", MODES)
def test_single_tokens_appended(cuda_device, mode):
    b = make_batch([1] * len(TOKENS), TOKENS, 8, 2, 64, mode, 150, 4, 31, cuda_device)
    whole = [b["k_cache"].clone(), b["v_cache"].clone()]
    page, off = b["slots"] // 16, b["slots"] % 16
    for c in ("k_cache", "v_cache"):
        b[c][page, :, off] = 0x7F if b[c].dtype == torch.uint8 else float("nan")
    check(b, window_call(b, workspace(b), append=True), mode)
    for got, want in zip((b["k_cache"], b["v_cache"]), whole):
        assert torch.equal(got.view(torch.uint8), want.view(torch.uint8))


@pytest.mark.parametrize("mode", ["bf16", "f32", "f16-e4m3"])
@pytest.mark.parametrize("seqs", [1, 7, 500])
def test_single_tokens_far_into_their_sequences(cuda_device, mode, seqs):
    g = torch.Generator().manual_seed(seqs)
    lens = torch.randint(1, 60_000 if seqs < 100 else 3000, (seqs,), generator=g).tolist()
    b = make_batch([1] * seqs, lens, 4, 1, 64, mode, 1800, 20, 7, cuda_device)
    ws = workspace(b)
    check(b, window_call(b, ws), mode)
    assert status(b, ws) == ops.CPA_OK


@pytest.mark.parametrize("mode", ["bf16", "f32", "bf16-e4m3"])
def test_single_tokens_captured_and_replayed(cuda_device, mode):
    b = make_batch([1] * len(TOKENS), TOKENS, 8, 2, 64, mode, 60, 4, 41, cuda_device)
    ws, out = workspace(b), torch.empty_like(b["q"])
    eager = window_call(b, ws, append=True).clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        window_call(b, ws, append=True, out=out)
    for _ in range(2):
        out.zero_()
        ws[256:].random_(0, 256)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager)


@pytest.mark.parametrize("mode", ["bf16", "f32", "bf16-e4m3"])
def test_single_tokens_a_bad_page_is_reported(cuda_device, mode):
    """... and the other rows are right."""
    b = make_batch([1, 1, 1], [300, 300, 300], 4, 2, 64, mode, 50, 4, 5, cuda_device)
    ws, good = workspace(b), None
    good = window_call(b, ws).clone()
    b["table"][1, 300 // 16] = -5
    got = window_call(b, ws)
    assert status(b, ws) == ops.CPA_ERR_DEVICE
    assert torch.equal(got[0], good[0]) and torch.equal(got[2], good[2])


@pytest.mark.parametrize("mode", ["bf16", "f32"])
def test_the_same_sequence_twice_in_one_step(cuda_device, mode):
    """Two tokens of one sequence as two rows of the batch: both are appended before either is computed."""
    b = make_batch([1, 1], [100, 101], 4, 2, 64, mode, 30, 4, 6, cuda_device, poison=False)
    b["table"][0] = b["table"][1]
    b["dense"][0] = [x[:100] for x in b["dense"][1]]
    kv = [x.to(b["q"].dtype) for x in b["dense"][1]]
    b["k"], b["v"] = kv[0][99:101].contiguous(), kv[1][99:101].contiguous()
    b["slots"][0] = int(b["table"][1, 99 // 16]) * 16 + 99 % 16
    page, off = b["slots"] // 16, b["slots"] % 16
    b["k_cache"][page, :, off] = float("nan")
    b["v_cache"][page, :, off] = float("nan")
    check(b, window_call(b, workspace(b), append=True), mode)


# ---- fp32: tiles of few rows and of many

@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(2, 2), (4, 2), (8, 2), (16, 2)])
def test_f32_chunks(cuda_device, d, hq, hkv):
    """Chunks of one row to many tiles, tails of every kind."""
    b = make_batch([17, 1, 130, 5, 1, 64], [300, 250, 130, 77, 1, 640], hq, hkv, d, "f32", 90, 19, 70 + hq, cuda_device)
    ws = workspace(b)
    check(b, window_call(b, ws), f"{hq}/{hkv} {d}")
    assert status(b, ws) == ops.CPA_OK


@pytest.mark.parametrize("window,sinks", [(1, 0), (300, 7), (5000, 0)])
@pytest.mark.parametrize("d", [64, 128])
def test_f32_many_rows(cuda_device, d, window, sinks):
    """Enough tiles for four to a CTA (19200 rows and more of 32 heads)."""
    b = make_batch([1, 601, 33, 3, 250, 1], [40, 700, 33, 500, 1100, 900], 32, 8, d, "f32", window, sinks, 80 + window, cuda_device)
    ws = workspace(b)
    check(b, window_call(b, ws), f"{d} {window} {sinks}")
    assert status(b, ws) == ops.CPA_OK


def test_f32_precision(cuda_device):
    """Far closer to the formula than tf32 products could be: 2^-11 of the operands' half step against 2^-21."""
    b = make_batch([200, 1], [900, 1000], 8, 2, 128, "f32", 700, 4, 90, cuda_device)
    want, size = reference(b)
    err = (window_call(b, workspace(b)).double() - want).norm() / want.norm()
    assert err < 2.0 ** -19


@pytest.mark.parametrize("seqs", [33, 1025, 3000])
def test_f32_finds_its_sequence(cuda_device, seqs):
    """Many sequences, some of several tokens."""
    g = torch.Generator().manual_seed(seqs)
    q = torch.where(torch.rand(seqs, generator=g) < 0.1, torch.randint(2, 20, (seqs,), generator=g), 1).tolist()
    lens = [x + int(y) for x, y in zip(q, torch.randint(0, 60, (seqs,), generator=g))]
    b = make_batch(q, lens, 2, 1, 64, "f32", 21, 3, 4, cuda_device)
    check(b, window_call(b, workspace(b)))


@pytest.mark.parametrize("mode", ["bf16-e4m3", "f16-e4m3"])
@pytest.mark.parametrize("append", [False, True])
def test_many_single_tokens_beside_chunks_8_bit(cuda_device, mode, append):
    """Enough single tokens for a kernel beside the chunks' one; results as for any other step, and what comes next on the stream
    sees all of them."""
    g = torch.Generator().manual_seed(12)
    seqs = 60
    q = [1] * seqs
    q[7], q[30], q[59] = 33, 200, 2
    lens = [x + int(y) for x, y in zip(q, torch.randint(0, 3000, (seqs,), generator=g))]
    b = make_batch(q, lens, 16, 8, 128, mode, 1200, 30, 13, cuda_device)
    ws, out = workspace(b), torch.empty_like(b["q"])
    for _ in range(3):
        out.fill_(float("nan"))
        window_call(b, ws, append=append, out=out)
        after = out + 0  # an ordinary kernel right behind the call
        check(b, after, mode)
    assert status(b, ws) == ops.CPA_OK
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        window_call(b, ws, append=append, out=out)
        copied = out + 0
    out.fill_(float("nan"))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(copied, after)


# ---- what the documentation allows and little else reaches

@pytest.mark.parametrize("mode", ["bf16", "f16", "bf16-e4m3"])
@pytest.mark.parametrize("hq,hkv,window", [(8, 2, 20_000), (4, 1, 2 ** 40)])
def test_few_tokens_with_a_very_long_window(cuda_device, mode, hq, hkv, window):
    b = make_batch([1, 1], [30_000, 21_001], hq, hkv, 64, mode, min(window, 2 ** 30), 100, 14, cuda_device)
    ws = workspace(b)
    b["window"] = window
    out = window_call(b, ws, append=True)
    b["window"] = min(window, 2 ** 30)
    check(b, out, mode)
    assert status(b, ws) == ops.CPA_OK


@pytest.mark.parametrize("mode", ["bf16", "f32", "bf16-e4m3"])
@pytest.mark.parametrize("q_lens", [[1, 1, 1], [1, 40, 1]])
def test_pages_beyond_32_bit_offsets(cuda_device, mode, q_lens):
    """The same step with its pages at the end of a cache of more than 2^32 elements: the same bits."""
    b = make_batch(q_lens, [700, 300, 90], 16, 8, 128, mode, 250, 20, 15, cuda_device)
    want = window_call(b, workspace(b))
    n = b["k_cache"].shape[0]
    first = 2 ** 32 // (8 * 16 * 128) + 5
    far = dict(b)
    for c in ("k_cache", "v_cache"):
        far[c] = torch.empty((first + n, *b[c].shape[1:]), dtype=b[c].dtype, device=cuda_device)
        far[c][first:] = b[c]
    far["table"] = torch.where(b["table"] >= 0, b["table"] + first, -1)
    far["slots"] = b["slots"] + first * 16
    ws = workspace(far)
    got = window_call(far, ws, append=True)
    assert status(far, ws) == ops.CPA_OK
    assert torch.equal(got, want)
    src = torch.arange(first, first + n, dtype=torch.int32, device=cuda_device)
    ops.copy_pages(src, src - first, far["k_cache"], far["v_cache"])
    assert torch.equal(far["k_cache"][:n].view(torch.uint8), b["k_cache"].view(torch.uint8))


def test_rows_behind_the_last_sequence_stay(cuda_device):
    """Tokens that no sequence owns: their output is left as it was."""
    for mode in MODES:
        for q in ([1, 1], [1, 30]):
            b = make_batch(q, [80, 90], 4, 2, 64, mode, 30, 4, 16, cuda_device)
            T = sum(q)
            pad = torch.randn(5, 4, 64, device=cuda_device).to(b["q"].dtype)
            long = dict(b, q=torch.cat([b["q"], pad]))
            out = torch.full_like(long["q"], 7)
            ws = workspace(long)
            ops.window_attention_forward(long["q"], long["k_cache"], long["v_cache"], long["table"], long["starts"],
                                         long["lens"], long["scale"], ws, 30, 4, out=out, **long["scales"])
            check(b, out[:T], mode)
            assert (out[T:] == 7).all()


def test_tensors_that_are_refused(cuda_device):
    b = make_batch([1, 1], [80, 90], 4, 2, 64, "bf16", 30, 4, 16, cuda_device)
    ws = workspace(b)
    good = dict(b)

    def call(**kw):
        return window_call(dict(good, **kw), kw.pop("ws", ws))

    wide = torch.zeros((2, 2 * b["table"].shape[1]), dtype=torch.int32, device=cuda_device)
    for kw in (dict(table=wide[:, ::2]), dict(lens=b["lens"][:1]), dict(starts=b["starts"][:2]), dict(v_cache=b["v_cache"][1:]),
               dict(k_cache=b["k_cache"].transpose(1, 2)), dict(q=b["q"][:, :, :32]), dict(table=b["table"].cpu()),
               dict(q=b["q"].expand(2, 4, 64)[:, ::2]), dict(ws=ws.view(torch.int32))):
        with pytest.raises((ValueError, TypeError)):
            call(**kw)
    for kw in (dict(lens=b["lens"].long()), dict(q=b["q"].half())):
        with pytest.raises(TypeError):
            call(**kw)
    for kw in (dict(window=0), dict(window=-2 ** 40), dict(sinks=-1), dict(ws=ws[256:512]), dict(scale=float("nan"))):
        with pytest.raises(ops.CpaError):
            call(**kw)
    with pytest.raises(ValueError):
        window_call(good, ws, out=torch.empty_like(b["q"])[:1])
    check(b, call())


@pytest.mark.parametrize("mode", ["bf16-e4m3", "f16-e4m3", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
def test_single_tokens_of_many_rows(cuda_device, mode, d):
    """More rows than the SMs hold at a time."""
    g = torch.Generator().manual_seed(17)
    lens = torch.randint(1, 300, (1500,), generator=g).tolist()
    b = make_batch([1] * 1500, lens, 8, 4, d, mode, 130, 9, 18, cuda_device)
    ws = workspace(b)
    check(b, window_call(b, ws), mode)
    assert status(b, ws) == ops.CPA_OK
