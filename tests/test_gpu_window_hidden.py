"""What no row of a 256-row group of a chunk sees may hold anything: the group's outputs keep their bits."""
import pytest
import torch

from test_gpu_window import check, status, window_call, workspace
from window_support import make_batch

from chunked_prefill_paged_cpa_gb300 import ops

pytestmark = pytest.mark.gpu


def poison(b, mode, seq, first):
    """NaN in every K and V of the sequence from position ``first`` on."""
    n = b["seq_lens"][seq]
    pos = torch.arange(first, n, device=b["table"].device)
    page, off = b["table"][seq, pos // 16].long(), pos % 16
    x = dict(b, k_cache=b["k_cache"].clone(), v_cache=b["v_cache"].clone())
    for c in ("k_cache", "v_cache"):
        x[c][page, :, off] = 0x7F if mode.endswith("e4m3") else float("nan")
    return x


@pytest.mark.parametrize("mode", ["bf16", "f16", "f32", "bf16-e4m3", "f16-e4m3"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("group", [1, 2, 4, 8])
@pytest.mark.parametrize("prefix,window,sinks", [(0, 5000, 0), (37, 100, 5), (3000, 700, 33)])
def test_later_tokens_of_the_chunk(cuda_device, mode, d, group, prefix, window, sinks):
    """The tokens behind a group, in the group's last tile of keys and past it."""
    q_len = 300
    b = make_batch([1, q_len, 20], [90, prefix + q_len, 20], 2 * group, 2, d, mode, window, sinks, 3 + group, cuda_device)
    ws = workspace(b)
    good = window_call(b, ws)
    check(b, good)
    tokens = 256 // group  # of a group
    for k in range(1, -(-q_len // tokens)):
        got = window_call(poison(b, mode, 1, prefix + k * tokens), ws)
        assert torch.equal(got[:1 + k * tokens], good[:1 + k * tokens]), f"group {k - 1} of {tokens} tokens"
        assert torch.equal(got[1 + q_len:], good[1 + q_len:])
    assert status(b, ws) == ops.CPA_OK
