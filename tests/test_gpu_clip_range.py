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


@pytest.mark.parametrize("kind", ["l2", "max"])
@pytest.mark.parametrize("place", [False, True])
def test_the_factor_is_rounded_once(kind, place):
    """Gradients of one power of two: their squares' sum is exact, so the factor
    max_norm / (norm + 1e-6) is known, and the scaled gradients show it.  To float32 it
    is off by half a step, and a product with a power of two is exact."""
    for n in (1, 3, 7, 1000, 4099, 100003, 5_000_001):
        for e in (-11, 0, 3):
            norm = 2.0 ** e * (math.sqrt(n) if kind == "l2" else 1.0)
            for share in (0.001, 0.3, 0.77, 0.9999):
                most = torch.tensor(norm * share).item()          # as float32
                t = torch.full((n,), 2.0 ** e, device=DEV)
                out = None if place else [torch.empty_like(t)]
                got = svp.clip_gradients([t], most, kind=kind, out=out).item()
                assert abs(got - norm) <= 2.0 ** -24 * norm
                scaled = (t if place else out[0]) / 2.0 ** e
                want = most / (norm + 1e-6)
                assert (scaled.double() - want).abs().max().item() <= 2.0 ** -24 * want * (1 + 1e-6), (n, e, share)
