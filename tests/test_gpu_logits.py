"""process_logits against the rule in 64 bits, token by token.

Tolerance, from the arithmetic: the rule takes at most five fp32 operations
(divide or multiply, f * n, two subtractions, the bias), each rounding by
2^-24 of at most A = max(|z| r, |z| / r) + f n + p + |bias|: 6 * 2^-24 A
(and the oracle's value the same to 2^-50).  A bf16 result is the rounding
of such an fp32 value: it lies between the roundings of the oracle's value
less and plus that tolerance, with nothing added.  What passes the type's
range is infinite.  A logit to which nothing applies keeps
its bits.
"""
import numpy as np
import pytest
import torch

import speculative_decoding_verification_71_gb300 as svp
from speculative_decoding_verification_71_gb300 import build as svbuild

pytestmark = pytest.mark.gpu
DEV = "cuda"
NAMES = ("history", "prompt_len", "history_len", "tokens", "draft_len", "repetition", "presence", "frequency",
         "bias_ids", "bias_values", "mask")


@pytest.fixture(scope="module", autouse=True)
def _built():
    svbuild.build()
    svp.load_library()


def reference(z, a, k):
    """(values, magnitude A, touched) [B, R, V] in 64 bits; rows that are left alone are NaN with touched 2."""
    B, R, V = z.shape
    out = z.double().numpy().copy()
    mag = np.zeros((B, R, V))
    kind = np.zeros((B, R, V), int)        # 0 untouched, 1 computed, 2 row left alone, 3 masked
    f = lambda name, b, default: float(a[name][b]) if a.get(name) is not None else default
    for b in range(B):
        rows = R
        if a.get("draft_len") is not None:
            kb = int(a["draft_len"][b])
            rows = kb + R - k if 0 <= kb <= k else 0
        prompt, said = [], []
        if a.get("history") is not None:
            h = a["history"][b].tolist()
            n = max(0, min(len(h), int(a["history_len"][b]) if a.get("history_len") is not None else len(h)))
            p = int(a["prompt_len"][b]) if a.get("prompt_len") is not None else 0
            prompt, said = h[:min(p, n)], h[max(0, min(p, n)):n]
        bias = {}
        if a.get("bias_ids") is not None:
            bias = dict(zip(a["bias_ids"][b].tolist(), a["bias_values"][b].double().tolist()))
        r, pres, freq = f("repetition", b, 1.0), f("presence", b, 0.0), f("frequency", b, 0.0)
        for i in range(R):
            if i >= rows:
                kind[b, i] = 2
                continue
            gen = said + (a["tokens"][b, :i].tolist() if a.get("tokens") is not None else [])
            counts = {}
            for t in gen:
                counts[t] = counts.get(t, 0) + 1
            for t in (set(prompt) | set(gen) | set(bias)):
                if not 0 <= t < V:
                    continue
                x, n = out[b, i, t], counts.get(t, 0)
                if n or t in prompt:
                    x = x / r if x > 0 else x * r
                top = abs(x)
                if n:
                    x = x - freq * n - pres
                    top += freq * n + pres
                x += bias.get(t, 0.0)
                out[b, i, t], mag[b, i, t], kind[b, i, t] = x, top + abs(bias.get(t, 0.0)), 1
            if a.get("mask") is not None:
                bits = np.unpackbits(a["mask"][b, i].numpy().view(np.uint8), bitorder="little")[:V]
                out[b, i, bits == 0] = -np.inf
                kind[b, i, bits == 0] = 3
    with np.errstate(over="ignore"):
        out = np.where(np.isinf(out.astype(np.float32)), out.astype(np.float32), out)
    return out, mag, kind


def rules(B, R, k, V, seed, H=0, drafts=True, ragged=True, penalties=True, n_bias=0, mask=None):
    g = torch.Generator().manual_seed(seed)
    tok = lambda *s: (torch.rand(*s, generator=g) ** 3 * V).to(torch.int32).clamp_(max=V - 1)
    a = {}
    if H:
        a["history"] = tok(B, H)
        a["history_len"] = torch.randint(0, H + 1, (B,), generator=g).to(torch.int32)
        a["history_len"][0] = H
        a["prompt_len"] = (a["history_len"] * torch.rand(B, generator=g)).to(torch.int32)
    if drafts and k:
        a["tokens"] = tok(B, k)
    if ragged and k:
        a["draft_len"] = torch.randint(0, k + 1, (B,), generator=g).to(torch.int32)
        a["draft_len"][0] = k
    if penalties:
        a["repetition"] = 1.0 + torch.rand(B, generator=g)
        a["presence"] = torch.rand(B, generator=g)
        a["frequency"] = torch.rand(B, generator=g)
    if n_bias:
        a["bias_ids"] = tok(B, n_bias)
        a["bias_values"] = torch.randn(B, n_bias, generator=g) * 5
    if mask is not None:
        W = (V + 31) // 32
        bits = torch.rand(B, R, W * 32, generator=g) < mask
        a["mask"] = torch.from_numpy(np.packbits(bits.numpy(), axis=-1, bitorder="little").view(np.int32).copy())
    return a


def gpu(a, **over):
    a = {n: (v.to(DEV) if v is not None else None) for n, v in a.items()}
    a.update(over)
    return a


def close(got, z, ref, mag, kind):
    got64, dtype = got.double().numpy(), got.dtype
    assert np.array_equal(np.isnan(got64[kind == 1]), np.isnan(ref[kind == 1]))
    same = kind == 0
    view = torch.int16 if dtype == torch.bfloat16 else torch.int32
    assert np.array_equal(got.view(view).numpy()[same], z.view(view).numpy()[same]), "an untouched logit changed"
    assert (got64[kind == 3] == -np.inf).all()
    t = (kind == 1) & np.isfinite(ref)
    tol = 6 * 2.0 ** -24 * mag
    if dtype == torch.bfloat16:
        low, high = (torch.from_numpy((ref + d)[t]).to(torch.bfloat16).double().numpy() for d in (-tol, tol))
        assert ((low <= got64[t]) & (got64[t] <= high)).all()
    else:
        assert (np.abs(got64 - ref)[t] <= tol[t]).all(), (np.abs(got64 - ref)[t] - tol[t]).max()
    inf = (kind == 1) & np.isinf(ref)
    assert np.array_equal(got64[inf], ref[inf])


def check(z, a, k, sentinel=-77.0, shift=0, in_place=False, **over):
    B, R, V = z.shape
    ref, mag, kind = reference(z, a, k)
    dev = torch.empty(z.numel() + 16, dtype=z.dtype, device=DEV)[shift:shift + z.numel()].view(B, R, V)
    dev.copy_(z)
    if in_place:
        out = dev
    else:
        out = torch.full((z.numel() + 16,), sentinel, dtype=z.dtype, device=DEV)
        out = out[shift + over.pop("out_shift", 0):][:z.numel()].view(B, R, V)
    over.pop("out_shift", None)
    res = svp.process_logits(dev, out=out, **gpu(a, **over))
    assert res is out
    torch.cuda.synchronize()
    got = out.cpu()
    close(got, z, ref, mag, kind)
    left = kind[:, :, 0] == 2
    want = z[torch.from_numpy(left)] if in_place else torch.full_like(z, sentinel)[torch.from_numpy(left)]
    assert torch.equal(got[torch.from_numpy(left)].nan_to_num(1e9), want.nan_to_num(1e9)), "a row past the drafts was written"
    if not in_place:
        assert torch.equal(dev.cpu().nan_to_num(1e9), z.nan_to_num(1e9)), "the input changed"
    return got


def logits(B, R, V, dtype, seed):
    return (torch.randn(B, R, V, generator=torch.Generator().manual_seed(seed)) * 4).to(dtype)


CASES = [  # B, k, V, dtype, rules
    (1, 0, 1, torch.float32, dict(H=3, n_bias=1)),
    (1, 0, 7, torch.bfloat16, dict(H=1, mask=0.5)),
    (3, 2, 33, torch.bfloat16, dict(H=40, n_bias=5, mask=0.7)),
    (2, 31, 129, torch.float32, dict(H=300, mask=0.9)),
    (5, 3, 1000, torch.bfloat16, dict(H=2000)),
    (4, 3, 4099, torch.float32, dict(H=100, n_bias=300, mask=0.99)),
    (4, 7, 4099, torch.bfloat16, dict(H=5000, n_bias=17, mask=0.5)),
    (2, 3, 20001, torch.bfloat16, dict(n_bias=64)),
    (2, 3, 50004, torch.float32, dict(H=30000)),
    (2, 3, 151936, torch.bfloat16, dict(H=1500, n_bias=3, mask=0.02)),
    (200, 1, 8192, torch.bfloat16, dict(H=64, mask=0.9)),       # larger slices: many sequences
    (1300, 0, 2050, torch.float32, dict(H=20, n_bias=2)),
    (2, 3, 30000, torch.bfloat16, dict(penalties=False, drafts=False, mask=0.6)),   # a mask alone
    (2, 3, 999, torch.bfloat16, dict(H=50, penalties=False)),                        # nothing to do: a copy
]


@pytest.mark.parametrize("in_place", [False, True], ids=["apart", "in_place"])
@pytest.mark.parametrize("B,k,V,dtype,r", CASES, ids=[f"{c[0]}x{c[1] + 1}x{c[2]}-{str(c[3])[6:]}" for c in CASES])
def test_matches_the_rule(B, k, V, dtype, r, in_place):
    a = rules(B, k + 1, k, V, seed=V + B, **r)
    check(logits(B, k + 1, V, dtype, V), a, k, in_place=in_place)


# How a call is cut depends on the numbers of CTAs that its slices make: vectors
# a thread (2, 4), passes a slice (2, for fp32), rows a CTA (all of them, or two).
MANY = [  # B, k, V, dtype, rules
    (130, 7, 5001, torch.bfloat16, dict(H=50, n_bias=3)),       # 2 vectors
    (120, 3, 9001, torch.float32, dict(H=64)),                  # 2
    (256, 3, 9001, torch.bfloat16, dict(H=64, n_bias=2)),       # 4
    (256, 3, 9001, torch.float32, dict(H=64, n_bias=2)),        # 4
    (600, 0, 10001, torch.float32, dict(H=64)),                 # 4, two passes, the second with tokens
    (500, 1, 9001, torch.float32, dict(H=64, n_bias=3)),        # 4, two passes, two rows
    (620, 4, 8300, torch.bfloat16, dict(H=20)),                 # 4, five rows to a CTA
    (256, 3, 9001, torch.bfloat16, dict(H=9000)),               # a list of thousands, above 48 KB of shared memory
    (512, 1, 9001, torch.float32, dict(H=9000)),                # ... and two passes
]


@pytest.mark.parametrize("mask", [None, 0.6], ids=["no_mask", "mask"])
@pytest.mark.parametrize("B,k,V,dtype,r", MANY, ids=[f"{c[0]}x{c[1] + 1}x{c[2]}-{str(c[3])[6:]}-{c[4]['H']}" for c in MANY])
def test_batches_of_many_sequences(B, k, V, dtype, r, mask):
    a = rules(B, k + 1, k, V, seed=V + B, mask=mask, **r)
    if r["H"] > 1000:      # a few whole histories, the others short: the reference goes token by token
        a["history_len"][3:] %= 60
        a["prompt_len"] = a["history_len"] // 3
    check(logits(B, k + 1, V, dtype, V), a, k, in_place=mask is not None and B % 4 == 0)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_draft_rows(dtype):
    # R = k: row i follows i drafts, rows i >= k_b are the padding
    B, k, V = 6, 4, 3001
    a = rules(B, k, k, V, seed=5, H=80, n_bias=4, mask=0.8)
    a["draft_len"][1] = 0
    check(logits(B, k, V, dtype, 6), a, k)


@pytest.mark.parametrize("in_place", [False, True], ids=["apart", "in_place"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_draft_rows_without_drafts(dtype, in_place):
    # a mask and biases on draft rows, full drafts among them, before any is drawn
    B, k, V = 6, 4, 3001
    a = rules(B, k, k, V, seed=55, drafts=False, penalties=False, n_bias=4, mask=0.6)
    a["draft_len"] = torch.tensor([k, 0, 1, k, k - 1, 2], dtype=torch.int32)
    z = logits(B, k, V, dtype, 56)
    dev = z.to(DEV)
    out = dev if in_place else torch.full_like(dev, -77.0)
    svp.process_logits(dev, out=out, k=k, **gpu(a))
    got, (ref, mag, kind) = out.cpu(), reference(z, a, k)
    close(got, z, ref, mag, kind)
    left = torch.from_numpy(kind[:, :, 0] == 2)
    assert left.sum() == 4 + 3 + 1 + 2 and torch.equal(got[left], z[left] if in_place else torch.full_like(z, -77.0)[left])


def test_target_rows_without_drafts():
    B, k, V = 4, 3, 700
    a = rules(B, k + 1, k, V, seed=57, drafts=False, H=30, mask=0.6)
    a["draft_len"] = torch.tensor([k, 0, k + 1, 2], dtype=torch.int32)    # one is out of range
    z = logits(B, k + 1, V, torch.float32, 58)
    got = check(z, a, k)
    said = svp.process_logits(z.to(DEV), k=k, out=torch.full_like(z, -77.0, device=DEV), **gpu(a))
    assert torch.equal(said.cpu(), got)


def test_k_has_to_fit_the_rows_and_the_drafts():
    z = torch.zeros(2, 3, 64, device=DEV)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device=DEV)
    for k in (0, 1, 4, -1):
        with pytest.raises(ValueError):
            svp.process_logits(z, draft_len=i32(2), k=k)
        with pytest.raises(ValueError):
            svp.process_logits(z, k=k)
    with pytest.raises(ValueError):
        svp.process_logits(z, tokens=i32(2, 2), k=3)               # tokens says two
    for k in (2.0, True, "2"):
        with pytest.raises(TypeError):
            svp.process_logits(z, draft_len=i32(2), k=k)
    assert svp.process_logits(z, tokens=i32(2, 3), draft_len=i32(2), k=3).shape == z.shape


@pytest.mark.parametrize("shift,out_shift", [(1, 0), (3, 0), (0, 1), (5, 2)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_bases_off_the_16_byte_boundary(dtype, shift, out_shift):
    B, k, V = 2, 2, 1531
    a = rules(B, k + 1, k, V, seed=8, H=60, n_bias=6, mask=0.6)
    check(logits(B, k + 1, V, dtype, 9), a, k, shift=shift, out_shift=out_shift)
    check(logits(B, k + 1, V, dtype, 9), a, k, shift=shift, in_place=True)


def test_a_drafted_token_counts_from_the_next_row_on():
    V, k = 64, 3
    z = torch.full((1, k + 1, V), 2.0)
    a = {"tokens": torch.tensor([[9, 9, 40]], dtype=torch.int32), "frequency": torch.tensor([0.25]),
         "presence": torch.tensor([0.5]), "repetition": torch.tensor([2.0])}
    got = check(z, a, k)
    assert got[0, :, 9].tolist() == [2.0, 1.0 - 0.75, 1.0 - 1.0, 1.0 - 1.0]
    assert got[0, :, 40].tolist() == [2.0, 2.0, 2.0, 1.0 - 0.75]


def test_prompt_tokens_are_repeated_but_not_generated():
    z = torch.tensor([[[3.0, -3.0, 3.0, -3.0]]])
    a = {"history": torch.tensor([[0, 1, 1, 2]], dtype=torch.int32), "prompt_len": torch.tensor([3], dtype=torch.int32),
         "repetition": torch.tensor([1.5]), "presence": torch.tensor([10.0])}
    assert check(z, a, 0)[0, 0].tolist() == [2.0, -4.5, -8.0, -3.0]


def test_lengths_ids_and_drafts_out_of_range():
    B, k, V, H = 5, 3, 500, 20
    a = rules(B, k + 1, k, V, seed=12, H=H, n_bias=8)
    a["history"][:, ::3] = -1
    a["history"][:, 1::5] = V
    a["history"][:, 2::7] = 2 ** 31 - 1
    a["bias_ids"][:, 0] = -5
    a["bias_ids"][:, 1] = V + 3
    a["tokens"][:, 1] = -1
    a["history_len"] = torch.tensor([-4, 0, 1, H, H + 9], dtype=torch.int32)
    a["prompt_len"] = torch.tensor([0, 5, 3, H + 7, -2], dtype=torch.int32)
    a["draft_len"] = torch.tensor([k, -1, k + 1, 0, 2], dtype=torch.int32)
    check(logits(B, k + 1, V, torch.bfloat16, 13), a, k)


def test_history_with_strided_rows_and_without_lengths():
    B, V = 3, 700
    a = rules(B, 1, 0, V, seed=14, H=30)
    del a["history_len"], a["prompt_len"]
    wide = torch.full((B, 101), 5, dtype=torch.int32, device=DEV)
    wide[:, 7:37] = a["history"].to(DEV)
    check(logits(B, 1, V, torch.float32, 15), a, 0, history=wide[:, 7:37])


def test_the_last_of_a_tokens_biases_counts():
    z = torch.zeros(1, 1, 300, dtype=torch.float32)
    ids = torch.tensor([[7] * 200 + [8] + [7] * 99], dtype=torch.int32)
    vals = torch.arange(300, dtype=torch.float32)[None]
    got = check(z, {"bias_ids": ids, "bias_values": vals}, 0)
    assert got[0, 0, 7] == 299.0 and got[0, 0, 8] == 200.0


def test_the_bias_is_added_after_the_penalties():
    z = torch.tensor([[[2.0, -2.0, 2.0]]])
    a = {"history": torch.tensor([[0, 1]], dtype=torch.int32), "prompt_len": torch.tensor([2], dtype=torch.int32),
         "repetition": torch.tensor([2.0]), "bias_ids": torch.tensor([[0, 1, 2]], dtype=torch.int32),
         "bias_values": torch.tensor([[3.0, 3.0, 3.0]])}
    assert check(z, a, 0)[0, 0].tolist() == [4.0, -1.0, 5.0]


def test_counts_beyond_16_bits():
    z = torch.full((1, 1, 40), 1.0)
    h = torch.full((1, 70001), 11, dtype=torch.int32)
    got = check(z, {"history": h, "frequency": torch.tensor([0.5])}, 0)
    assert got[0, 0, 11] == 1.0 - 0.5 * 70001


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_masked_places_may_hold_anything(dtype):
    V = 1003
    z = logits(1, 3, V, dtype, 20)
    low = torch.finfo(dtype).min
    z[0, 0, ::3] = float("nan")
    z[0, 0, 1::3] = float("inf")
    z[0, 1, ::2] = -float("inf")
    z[0, 1, 1::2] = low
    a = rules(1, 3, 2, V, seed=21, H=900, mask=0.5)
    a["draft_len"] = None
    a["mask"][0, 2] = 0                      # a row that allows nothing
    got = check(z, a, 2)
    assert (got[0, 2] == -float("inf")).all()


def test_nan_and_infinite_logits_go_through_the_rule():
    V = 64
    z = torch.zeros(1, 1, V)
    z[0, 0, :4] = torch.tensor([float("nan"), float("inf"), -float("inf"), torch.finfo(torch.float32).min])
    a = {"history": torch.arange(8, dtype=torch.int32)[None], "repetition": torch.tensor([2.0]),
         "presence": torch.tensor([1.0])}
    got = svp.process_logits(z.to(DEV), **gpu(a)).cpu()[0, 0]
    assert torch.isnan(got[0]) and got[1] == float("inf") and got[2] == -float("inf")
    assert got[3] == -float("inf")           # twice the lowest value
    assert (got[4:8] == -1.0).all() and (got[8:] == 0).all()


def test_another_stream_and_repeated_calls_give_the_same_bits():
    B, k, V = 16, 3, 20011
    z = logits(B, k + 1, V, torch.bfloat16, 30).to(DEV)
    a = gpu(rules(B, k + 1, k, V, seed=31, H=700, n_bias=20, mask=0.9, ragged=False))
    want = svp.process_logits(z, **a)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(5):
        got = svp.process_logits(z, stream=s, **a)
        s.synchronize()
        assert torch.equal(got.view(torch.int16), want.view(torch.int16))


def test_a_captured_call_replays():
    z = logits(4, 1, 5000, torch.float32, 33).to(DEV)
    a = gpu(rules(4, 1, 0, 5000, seed=34, H=50, mask=0.9))
    want = svp.process_logits(z, **a)
    out = torch.zeros_like(z)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        svp.process_logits(z, out=out, **a)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


@pytest.mark.slow
def test_more_than_2_31_logits():
    B, V = 16800, 128256                      # 2.15e9 logits: the last rows lie past 32-bit offsets
    z = torch.zeros(B, 1, V, dtype=torch.bfloat16, device=DEV)
    tail = logits(2, 1, V, torch.bfloat16, 40)
    z[-2:] = tail.to(DEV)
    h = torch.zeros(B, 64, dtype=torch.int32, device=DEV)
    a = rules(2, 1, 0, V, seed=41, H=64)
    h[-2:] = a["history"].to(DEV)
    pres = torch.ones(B, device=DEV)
    a = {"history": a["history"], "presence": torch.ones(2)}
    out = svp.process_logits(z, history=h, presence=pres)
    torch.cuda.synchronize()
    close(out[-2:].cpu(), tail, *reference(tail, a, 0))
    assert (out[0, 0, 1:] == 0).all() and out[0, 0, 0] == -1


def test_refusals():
    z = torch.zeros(2, 3, 64, device=DEV)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device=DEV)
    with pytest.raises(TypeError):
        svp.process_logits(z.half())
    with pytest.raises(ValueError):
        svp.process_logits(z[0])
    with pytest.raises(ValueError):
        svp.process_logits(z.transpose(1, 2))
    with pytest.raises(ValueError):
        svp.process_logits(z.cpu())
    with pytest.raises(ValueError):
        svp.process_logits(z, tokens=i32(2, 5))                   # 3 rows for 5 drafts
    with pytest.raises(TypeError):
        svp.process_logits(z, tokens=i32(2, 2).long())
    with pytest.raises(ValueError):
        svp.process_logits(z, history=i32(3, 8))
    with pytest.raises(ValueError):
        svp.process_logits(z, history=i32(8, 2).t())
    with pytest.raises(ValueError):
        svp.process_logits(z, prompt_len=i32(2))
    with pytest.raises(ValueError):
        svp.process_logits(z, bias_ids=i32(2, 4))
    with pytest.raises(ValueError):
        svp.process_logits(z, mask=i32(2, 3, 3))
    with pytest.raises(ValueError):
        svp.process_logits(z, mask=i32(2, 1, 2))
    with pytest.raises(ValueError):
        svp.process_logits(z, out=torch.zeros(2, 3, 65, device=DEV))
    both = torch.zeros(2 * 3 * 64 + 4, device=DEV)
    with pytest.raises(svp.SpecVerifyError):                       # overlapping, not in place
        svp.process_logits(both[:384].view(2, 3, 64), out=both[4:].view(2, 3, 64))
    big = torch.zeros(1, 33, 8, device=DEV)
    with pytest.raises(svp.SpecVerifyError):                       # 32 drafts
        svp.process_logits(big, tokens=i32(1, 32))
