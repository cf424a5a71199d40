"""A chunk's short last unit, and the same tokens as a sequence of their own."""
import pytest
import torch

from select_support import make_batch, reference, select
from test_gpu_select import random_rows, run_select, step_tensors
from test_gpu_selected import call, workspace
from window_support import tolerance

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("group,tail", [(4, 36), (4, 1), (1, 255), (8, 7)])
def test_every_token_counts_once_in_a_sequence_of_its_own(cuda_device, group, tail):
    """The tail described as a second sequence on the same pages: its lists are those of the plain sum over its rows, and the
    full units' lists are as in the whole chunk."""
    size, hkv, d, n = 256 // group, 2, 64, 5000
    chunk = 2 * size + tail
    pages = -(-n // 16)
    rows = random_rows(pages, hkv, d, 41)
    table, whole = step_tensors([chunk], [n], pages, 42, cuda_device)
    q = torch.randn(chunk, hkv * group, d, generator=torch.Generator().manual_seed(43)).bfloat16().to(cuda_device)
    one = run_select(q, rows, whole, table, [chunk], [n], 32, 1, 2, cuda_device)
    two_table = table.expand(2, -1).contiguous()
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=cuda_device)  # noqa: E731
    where = (two_table.to(cuda_device), i32(0, 2 * size, chunk), i32(n - tail, n))
    two = run_select(q, rows, where, two_table, [2 * size, tail], [n - tail, n], 32, 1, 2, cuda_device)   # (equal to the host's, which weighs no first unit)
    assert (one[:2 * size] == two[:2 * size]).all()
    alone = select(q[2 * size:], rows, table, [tail], [n], 32, 1, 2, two[2 * size:])
    assert (alone == two[2 * size:]).all()


@pytest.mark.parametrize("mode", ["bf16", "f16-e4m3", "f32"])
def test_attention_is_the_same_in_both_descriptions(cuda_device, mode):
    b = make_batch([1, 100, 1], [500, 1500, 90], 8, 2, 64, mode, 20, 2, 44, cuda_device)
    want, size = reference(b)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=cuda_device)  # noqa: E731
    split = dict(b, table=b["table"][[0, 1, 1, 2]].contiguous(), starts=i32(0, 1, 65, 101, 102), lens=i32(500, 1464, 1500, 90), q_lens=[1, 64, 36, 1])
    out = call(split, workspace(split))
    assert ((out.double() - want).abs() <= tolerance(b, want, size)).all()
