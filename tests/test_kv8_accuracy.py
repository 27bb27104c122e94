"""The size of the decode's error over the 8-bit cache as a whole, beside the bounds per value.

Relative to the output's norm, in the mean square.  bf16's rounding of the output: off evenly within half a step, 2^-8 of
the power of two below a value, so 2^-8 / sqrt 3 of it; values spread evenly over an octave's logarithm have a mean square of
1.5 / ln 2 = 2.164 of that power's: 1.53e-3, and at most 2^-8 / sqrt 3 = 2.26e-3 where all lie at the octaves' beginnings;
1.7e-3 is taken.  A weight's hi part leaves evenly up to half a step, 2^-4 of a power of two: 2^-4 / sqrt 3 / sqrt 2.164 =
0.0245 of the weight in the mean square.  Its lo part leaves of that, in the same way, 0.0245 (e4m3) or, with a step
twice as wide, 0.049 (e5m2): 6.0e-4 or 1.2e-3 of the weight.  Weights' errors are independent, as the values are that
they weigh: the output's is at most that part of it.  Queries and lse add less than 2^-16."""
import math

import pytest
import torch

from tests._kv8_reference import attention
from tests.test_kv8_decode import SCALE, decode, inputs

gpu = pytest.mark.gpu


@gpu
@pytest.mark.parametrize("h_q,s_q,weights", [(16, 1, 6.0e-4), (32, 1, 6.0e-4), (20, 3, 6.0e-4), (128, 1, 1.2e-3), (96, 2, 1.2e-3)])
@pytest.mark.parametrize("spread", [0.0, 0.5])
def test_error_of_the_whole(h_q, s_q, weights, spread):
    q, cache, scales, bt, sl = inputs([2000, 700, 3000, 129, 64, 1500], s_q, h_q, seed=70)
    scales = scales * torch.exp(spread * torch.randn(scales.shape, generator=torch.Generator().manual_seed(71))).cuda()
    x = (q, cache, scales, bt, sl)
    out, lse = decode(*x, causal=s_q > 1)
    o, l, _, lb = attention(*x, SCALE, s_q > 1)
    err = float((out.double() - o).norm() / o.norm())
    assert err <= math.hypot(1.7e-3, weights), f"{err:.3e}"
    # a score is a sum of 576 products in 32 bits, off by 2^-17 of their magnitudes' sum, which is many times the score:
    # the bound per value counts that
    assert ((lse.double() - l).abs() <= lb).all()
