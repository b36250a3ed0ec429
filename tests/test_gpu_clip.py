"""clip_gradients against its definition in 64 bits.

The norm: squares and their sums in float32 over at most a few hundred terms a
thread, then pairwise and in 64 bits: 1e-6 of itself, the root halves it; one
rounding to float32 more.  A scaled gradient: the factor is off by the norm's
error and two roundings, the product by one, and a bfloat16 by half a step.
"""
import math

import numpy as np
import pytest
import torch

import speculative_decoding_verification_71_gb300 as svp
from speculative_decoding_verification_71_gb300 import build as svbuild

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16
INF, NAN = float("inf"), float("nan")
NORM_TOL = 1e-6
STEP = {F32: 2.0 ** -24, BF16: 2.0 ** -8}


@pytest.fixture(scope="module", autouse=True)
def _built():
    svbuild.build()
    svp.load_library()


def make(sizes, dtypes, seed=0, scale=1.0, offsets=None):
    g = torch.Generator().manual_seed(seed)
    out = []
    for i, n in enumerate(sizes):
        t = torch.randn(n, generator=g) * scale
        by = offsets[i % len(offsets)] if offsets else 0
        out.append(torch.empty(n + by, dtype=dtypes[i % len(dtypes)], device=DEV)[by:].copy_(t))
    return out


def norm64(grads, kind):
    if kind == "max":
        return max([float(t.double().abs().max()) if t.numel() else 0.0 for t in grads], default=0.0)
    return math.sqrt(math.fsum(float(t.double().square().sum()) for t in grads))


def check(grads, max_norm, kind="l2", out=None):
    before = [t.double().clone() for t in grads]
    want = norm64(grads, kind)
    got = svp.clip_gradients(grads, max_norm, kind=kind, out=out)
    torch.cuda.synchronize()
    assert got.shape == () and got.dtype == F32
    assert abs(got.item() - want) <= NORM_TOL * want, (got.item(), want)
    scale = 1.0 if max_norm is None else min(1.0, max_norm / (want + 1e-6))
    for i, (a, t) in enumerate(zip(before, grads)):
        o = t if out is None else out[i]
        if out is not None and o is not t:
            assert torch.equal(t.double(), a)
        if scale == 1.0:
            assert torch.equal(o.double(), a)
            continue
        ref = a * scale
        tol = ref.abs() * ((NORM_TOL + 4 * 2.0 ** -24) + STEP[o.dtype] * (1 + 2e-6)) + 1e-45
        assert ((o.double() - ref).abs() <= tol).all(), i
    return got


SIZES = [
    [1], [0], [0, 7], [3, 5], [8], [1000], [4096, 4096], [100003], [1 << 20], [33, 0, 100001, 1, 2, 70000],
    [2000 * 64, 64 * 2000], [17] * 300, [1] * 1500, [1 << 22, 5, 1 << 21, 13],
]


@pytest.mark.parametrize("dtypes", [(F32,), (BF16,), (BF16, F32)], ids=["f32", "bf16", "mixed"])
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{max(s)}")
@pytest.mark.parametrize("kind", ["l2", "max"])
def test_norm_and_scaling(sizes, dtypes, kind):
    grads = make(sizes, dtypes, seed=len(sizes))
    want = norm64(grads, kind)
    check(grads, None, kind)
    check(grads, want * 2 + 1, kind)            # within bounds: nothing is written
    check(grads, max(want * 0.3, 1e-3), kind)
    check(grads, max(want * 0.01, 1e-5), kind)


@pytest.mark.parametrize("offsets", [(1,), (0, 1, 2, 3), (7, 2, 5)])
@pytest.mark.parametrize("dtypes", [(F32,), (BF16,), (BF16, F32)], ids=["f32", "bf16", "mixed"])
def test_tensors_at_any_alignment(dtypes, offsets):
    grads = make([5, 100003, 1, 20000, 31, 64], dtypes, seed=3, offsets=offsets)
    check(grads, None)
    check(grads, norm64(grads, "l2") * 0.5)
    out = make([5, 100003, 1, 20000, 31, 64], dtypes, seed=4, offsets=offsets[::-1])
    check(grads, norm64(grads, "l2") * 0.5, out=out)


@pytest.mark.parametrize("share", [0.1, 5.0])
def test_into_other_tensors(share):
    sizes = [5, 100003, 0, 20000, 31, 1 << 20]
    grads = make(sizes, (BF16, F32), seed=5)
    want = norm64(grads, "l2")
    check(grads, want * share, out=[torch.full_like(t, 3.0) for t in grads])
    check(grads, want * share, out=[torch.full_like(t, 3.0, dtype=F32) for t in grads])
    check(grads, want * share, out=grads)
    check(grads, want * share, "max", out=[torch.full_like(t, 3.0, dtype=F32) for t in grads])


def test_tensors_end_to_end_keep_to_themselves():
    """Tensors that share 16-byte vectors with their neighbours, of which every
    other one is not given."""
    sizes = [3, 1, 17, 5, 100, 33, 7, 2, 5000, 11]
    for dtype in (F32, BF16):
        flat = torch.randn(sum(sizes), device=DEV, dtype=F32).to(dtype)
        before = flat.clone()
        parts = list(flat.split(sizes))
        check(parts[::2], 0.01)
        for a, b in zip(parts[1::2], list(before.split(sizes))[1::2]):
            assert torch.equal(a, b)


def test_layouts_without_gaps():
    g = [torch.randn(30, 50, device=DEV).t(), torch.randn(4, 6, 5, device=DEV).permute(2, 0, 1), torch.randn((), device=DEV),
         torch.randn(2, 3, 8, 8, device=DEV).to(memory_format=torch.channels_last)]
    check(g, 1.0)
    check(g, 0.5, out=[torch.empty_like(t) for t in g])
    check([t for t in (None, *g) if t is not None], None)
    norm = svp.clip_gradients([None, *g, None])
    assert abs(norm.item() - norm64(g, "l2")) < 1e-5
    with pytest.raises(ValueError, match="gaps"):
        svp.clip_gradients([torch.zeros(4, 8, device=DEV)[:, :4]])
    with pytest.raises(ValueError, match="gaps"):
        svp.clip_gradients([torch.zeros(1, device=DEV).expand(5)])
    with pytest.raises(ValueError, match="laid out"):
        svp.clip_gradients(g[:1], 1.0, out=[torch.empty(50, 30, device=DEV)])
    with pytest.raises(ValueError, match="laid out"):
        svp.clip_gradients([torch.zeros(4, device=DEV)], 1.0, out=[torch.zeros(4, device=DEV, dtype=BF16)])
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        svp.clip_gradients([torch.zeros(4, device=DEV, dtype=torch.float16)])
    a = torch.zeros(64, device=DEV)
    for bad in ([a, a], [a[:40], a[30:]]):
        with pytest.raises(svp.SpecVerifyError, match="INVALID_ARG"):
            svp.clip_gradients(bad, 1.0)
        assert svp.clip_gradients(bad).item() == 0.0      # only read: each counts as often as it is there


@pytest.mark.parametrize("scale", [1e-30, 1e-22, 1e-10, 1e10, 1e17, 1e22, 1e30])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_squares_past_the_range(dtype, scale):
    """Norms that float32 holds, of values whose squares it does not."""
    grads = make([50000, 3, 700001], (dtype,), seed=6, scale=scale)
    check(grads, None)
    check(grads, None, "max")
    one = make([1], (dtype,), seed=1, scale=scale)
    check([*one, *make([100000], (dtype,), seed=2, scale=scale * 1e-6)], None)
    check(grads, norm64(grads, "l2") * 0.5) if scale > 1e-9 else None


def test_zeros_and_denormals():
    assert svp.clip_gradients([torch.zeros(1000, device=DEV)], 1.0).item() == 0.0
    t = torch.full((1000,), 1e-42, device=DEV)
    want = math.sqrt(1000) * float(t[0].double())
    assert abs(svp.clip_gradients([t]).item() - want) <= 1e-3 * want
    assert svp.clip_gradients([t], kind="max").item() == t[0].item()


@pytest.mark.parametrize("bad", [NAN, INF, -INF])
@pytest.mark.parametrize("kind", ["l2", "max"])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_a_norm_that_is_not_finite_scales_nothing(dtype, kind, bad):
    for n, at in ((9, 0), (100003, 100002), (1 << 20, 777777)):
        grads = make([5, n], (dtype,), seed=7)
        grads[1][at] = bad
        before = [t.clone() for t in grads]
        norm = svp.clip_gradients(grads, 0.1, kind=kind).item()
        assert math.isnan(norm) if math.isnan(bad) else norm == INF
        same = lambda a, b: torch.equal(a.view(torch.int32 if dtype == F32 else torch.int16), b.view(torch.int32 if dtype == F32 else torch.int16))
        assert all(same(a, b) for a, b in zip(grads, before))
        out = [torch.zeros_like(t) for t in grads]
        svp.clip_gradients(grads, 0.1, kind=kind, out=out)
        assert all(torch.equal(a.nan_to_num(3.0), b.nan_to_num(3.0)) for a, b in zip(out, before))


def test_more_elements_than_31_bits_count():
    t = torch.zeros((1 << 31) + 1000, dtype=BF16, device=DEV)
    t[-1], t[0], t[1 << 30] = 3.0, 4.0, 12.0
    assert svp.clip_gradients([t], 6.5).item() == 13.0
    assert (t[-1].item(), t[0].item(), t[1 << 30].item()) == (1.5, 2.0, 6.0)


def test_streams_and_graphs():
    grads = make([100003, 64, 1 << 20], (BF16, F32), seed=8)
    out = [torch.empty_like(t, dtype=F32) for t in grads]
    want = svp.clip_gradients(grads, 3.0, out=out).clone()
    ref = [t.clone() for t in out]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for o in out:
        o.zero_()
    side.wait_stream(torch.cuda.current_stream())
    assert torch.equal(svp.clip_gradients(grads, 3.0, out=out, stream=side).cpu(), want.cpu())
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, ref))
    graphs, results = [], []
    for _ in range(2):
        o = [torch.empty_like(t, dtype=F32) for t in grads]
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            results.append((svp.clip_gradients(grads, 3.0, out=o), o))
        graphs.append(g)
    grads[0].mul_(2.0)                          # a replay reads what is there then
    want = svp.clip_gradients(grads, 3.0, out=out)
    streams = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for g, s in zip(graphs, streams):
        with torch.cuda.stream(s):
            g.replay()
    torch.cuda.synchronize()
    for norm, o in results:
        assert torch.equal(norm, want) and all(torch.equal(a, b) for a, b in zip(o, out))


def test_more_tensors_than_a_table_holds():
    """Tables of 512 tensors: the norm of all, scaled copies of each."""
    sizes = [(i * 37) % 300 for i in range(1200)]
    grads = make(sizes, (BF16, F32, BF16), seed=11)
    want = norm64(grads, "l2")
    check(grads, None)
    check(grads, want * 0.3, out=[torch.empty_like(t, dtype=F32) for t in grads])
    check(grads, want * 0.3, "max", out=[torch.empty_like(t) for t in grads])
    check(grads, want * 0.3)


def test_contiguous_tensors_whose_strides_differ():
    t = torch.randn(8, 1, device=DEV).t()                 # one row: contiguous with any first stride
    o = torch.empty(1, 8, device=DEV)
    check([t], 0.1, out=[o])
