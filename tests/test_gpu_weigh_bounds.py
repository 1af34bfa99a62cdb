"""Bounds of the new tokens that are smaller than a sequence is, at and around the most that the kernel
for few rows is chosen for, steer the weights' kernels and change no sum beyond its bound."""
import pytest

import paged
from test_gpu_paged import both

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("most_q", [1, 63, 64, 65, 99])
@pytest.mark.parametrize("ql,kl", [([100], [900]), ([300], [300]), ([100, 3, 70], [100, 800, 2000])])
def test_bounds_below_the_lengths(gdn_lib, ql, kl, most_q):
    x = paged.cache(ql, kl, 16, 4, 32, seed=most_q)
    both(gdn_lib, x, ql, kl, most=max(kl), most_q=most_q)
