"""fp32 attention over a window, and over selected pages, is as precise over thousands of keys as over few."""
import pytest

import select_support
import window_support
from test_gpu_selected import call
from test_gpu_window import window_call, workspace

pytestmark = pytest.mark.gpu

# (q_lens, query heads, kv heads): enough tiles for four to a CTA, where one warp sums up all of a row's keys; a tile's keys
# split over warps and CTAs; a CTA per single token; few single tokens
SHAPES = {"rows": ([700, 1, 30], 32, 8), "split": ([40, 1], 8, 2), "many tokens": ([1] * 100, 32, 8), "few tokens": ([1] * 5, 8, 2)}

# The bound, for the relative 2-norm of the error.  The tensor cores cut a sum off below its 24 bits, towards zero: 2^-24 of it
# on average, each time that products are added.  Three products of every 8 keys are added to a sum of at most 64 keys that
# begins with nothing (half of it is there on average): 24 * 2^-25 = 2^-20.4, all of one sign.  The sums of 64 keys are added
# rounded to nearest, 2^-25 with either sign, 64 times at 4096 keys: 2^-22.  A score's two sums of d / 16 products lose as
# much of the score, which is about 1: 8 * 2^-25 = 2^-22; the operands' halves leave out 2^-21 (test_gpu_selected_f32.py).
# The larger two together are 2^-19.7.  Added to one sum throughout, 4096 keys would lose 2^-15.4.
BOUND = 2.0 ** -19


def relative_error(out, want):
    return float((out.double() - want).norm() / want.norm())


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("shape", SHAPES)
def test_window(cuda_device, shape, d):
    q_lens, hq, hkv = SHAPES[shape]
    b = window_support.make_batch(q_lens, [5600 + 3 * i for i in range(len(q_lens))], hq, hkv, d, "f32", 4096, 4, 90, cuda_device)
    assert relative_error(window_call(b, workspace(b)), window_support.reference(b)[0]) < BOUND


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("shape", SHAPES)
def test_selected_pages(cuda_device, shape, d):
    q_lens, hq, hkv = SHAPES[shape]
    b = select_support.make_batch(q_lens, [5600 + 3 * i for i in range(len(q_lens))], hq, hkv, d, "f32", 252, 4, 91, cuda_device)
    assert relative_error(call(b), select_support.reference(b)[0]) < BOUND
