"""Mixed steps over lists whose single tokens run on their own kernel beside the step kernel of the chunks."""
import pytest
import torch

from select_support import make_batch
from test_gpu_selected import call, check

pytestmark = pytest.mark.gpu

# single tokens and chunks in mixed order, so that a sequence's number is not its token's
ORDER = {
    "chunk between": [1] * 20 + [200] + [1] * 44,
    "chunks first and last": [130] + [1] * 62 + [2, 70],
    "alternating": [1, 3] * 33,
}


@pytest.mark.parametrize("mode", ["bf16", "f16", "bf16-e4m3", "f16-e4m3"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("order", ORDER)
def test_single_tokens_beside_chunks(cuda_device, order, d, mode):
    q_lens = ORDER[order]
    budget, local, hq, hkv = 28, 4, 16 if d == 64 else 32, 8
    seq_lens = [600 + 29 * (i * 7 % 60) + q for i, q in enumerate(q_lens)]
    # the rule: 96 pages of single tokens, every sequence counted as one, for each SM
    sms = torch.cuda.get_device_properties(cuda_device).multi_processor_count
    assert len(q_lens) * hkv * (budget + local) >= 96 * sms and 1 in q_lens and max(q_lens) > 1
    b = make_batch(q_lens, seq_lens, hq, hkv, d, mode, budget, local, 50, cuda_device)
    first = check(b)
    for _ in range(3):   # side by side in any order
        assert torch.equal(call(b).view(torch.int16), first.view(torch.int16))


@pytest.mark.parametrize("group", [1, 2, 8])
def test_other_groups(cuda_device, group):
    q_lens = [1] * 40 + [300 // group + 5] + [1] * 25
    seq_lens = [700 + 11 * i for i in range(66)]
    sms = torch.cuda.get_device_properties(cuda_device).multi_processor_count
    assert len(q_lens) * 8 * 32 >= 96 * sms
    check(make_batch(q_lens, seq_lens, 8 * group, 8, 64, "bf16", 30, 2, 51 + group, cuda_device))
