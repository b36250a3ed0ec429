"""clip_gradients on gradients so many and so large that their squares leave
float32's range together."""
import math

import pytest
import torch

import speculative_decoding_verification_71_gb300 as svp
from speculative_decoding_verification_71_gb300 import build as svbuild

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    svbuild.build()
    svp.load_library()


@pytest.mark.parametrize("dtype,n,value", [(BF16, 2_700_000_001, 2.0 ** 57), (F32, 1_400_000_001, 1.4 * 2.0 ** 57)],
                         ids=["bf16", "f32"])
def test_many_squares_past_the_range_together(dtype, n, value):
    """More than 5 GB of one value: each thread's sums of a piece, of 64 values at
    most, are below 2^120, all of a CTA's pieces are above 2^128.  The sums over
    hundreds of terms are off by 1e-6 of themselves at most, as elsewhere; halving
    is exact but for the factor's own 4 steps."""
    t = torch.full((n,), value, dtype=dtype, device=DEV)
    value = t[0].double().item()
    want = math.sqrt(n) * value
    got = svp.clip_gradients([t]).item()
    assert abs(got - want) <= 1e-6 * want, (got, want)
    norm = svp.clip_gradients([t], want / 2)
    assert norm.item() == got
    low, high = t.min().item(), t.max().item()
    half = 2.0 ** -8 if dtype == BF16 else 2.0 ** -24
    assert low == high and abs(low - value / 2) <= value / 2 * (1e-6 + 4 * 2.0 ** -24 + half)
