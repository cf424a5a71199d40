"""Chunks over lists of hundreds and thousands of pages: tile pairs split as far as they are, and whole ones."""
import pytest

from select_support import make_batch
from test_gpu_selected import check

pytestmark = pytest.mark.gpu

# The tolerance's 2^-13 of the size, which stands for fp32 arithmetic, at these lengths: a tile pair is split into up to eight
# units, so a row's weights are summed in at most 2100 pages / 8 = 263 tiles of 16 steps and 263 sums of tiles, and P V in 263
# k-steps of 16 keys, each off by a step of the accumulator (2^-23): 2^-14.9 of the size.  The scores, d = 64: 66 2^-24 times
# sum |q k| scale < 8: 2^-15.  Together below 2^-13.9.  (Whole pairs: 300 pages in 38 tiles, 300 k-steps: the same.)


@pytest.mark.parametrize("mode", ["bf16", "f16", "bf16-e4m3", "f32"])
@pytest.mark.parametrize("budget", [512, 2048])
def test_a_short_chunk(cuda_device, budget, mode):
    """One pair of one kv head; the last of its eight units holds the chunk's own tokens."""
    check(make_batch([64], [16 * 2100 + 7], 4, 1, 64, mode, budget, 4, 80, cuda_device))


@pytest.mark.parametrize("mode", ["bf16", "f16-e4m3"])
def test_a_few_pairs(cuda_device, mode):
    """Two pairs of eight kv heads each, the second with one tile; a single token beside them."""
    check(make_batch([1, 70], [9000, 8 * 1024 + 33], 32, 8, 64, mode, 400, 2, 81, cuda_device))


@pytest.mark.parametrize("mode", ["f16", "bf16-e4m3"])
def test_whole_pairs(cuda_device, mode):
    """As many pairs as CTAs and more: none is split."""
    check(make_batch([1300], [16 * 400 + 1300], 32, 8, 64, mode, 300, 2, 82, cuda_device))
