"""fp32 attention over selected pages keeps fp32's precision in every shape of its two kernels."""
import pytest

from select_support import make_batch, reference
from test_gpu_selected import call

pytestmark = pytest.mark.gpu


def relative_error(b):
    want, _ = reference(b)
    return float((call(b).double() - want).norm() / want.norm())


# The bound: a score is off by 2^-21 of its d products at most, each with a sign of its own: 2^-21 scale sqrt(sum (q k)^2) =
# 2^-21 for N(0, 1) inputs; P V's products the same, and the sums of some hundred terms add about as much: 2^-19 is four times
# one of these.  Outputs and errors are means over the same keys, so the ratio of their norms does not shrink with the keys:
# one product of the three left out would cost 2^-12.

@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(2, 2), (4, 2), (8, 2), (16, 2)])
@pytest.mark.parametrize("budget,local", [(5, 1), (10, 2), (20, 2), (60, 4)])
def test_single_tokens(cuda_device, budget, local, hq, hkv, d):
    """Pages for clusters of one, two, four and eight CTAs; groups of 1 to 8 heads."""
    assert relative_error(make_batch([1] * 5, [1100, 1500, 90, 1037, 1216], hq, hkv, d, "f32", budget, local, 70, cuda_device)) < 2.0 ** -19


@pytest.mark.parametrize("d", [64, 128])
def test_many_single_tokens(cuda_device, d):
    """More rows than are resident at once."""
    assert relative_error(make_batch([1] * 100, [500 + 9 * i for i in range(100)], 32, 8, d, "f32", 12, 2, 71, cuda_device)) < 2.0 ** -19


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("q_lens,seq_lens,hq,hkv", [([40, 1], [900, 1200], 8, 2), ([1, 17, 1, 3], [700, 600, 90, 1100], 2, 2), ([700, 1, 30], [1500, 800, 600], 32, 8)])
def test_steps_with_chunks(cuda_device, q_lens, seq_lens, hq, hkv, d):
    """A tile's keys split over warps and CTAs; enough tiles for four to a CTA."""
    assert relative_error(make_batch(q_lens, seq_lens, hq, hkv, d, "f32", 14, 2, 72, cuda_device)) < 2.0 ** -19
