"""Host-side checks of the logit operators' C entry points: each bad call is
refused before anything is launched (no GPU needed)."""
import ctypes

import pytest

import speculative_decoding_verification_71_gb300 as svp
from speculative_decoding_verification_71_gb300 import build as svbuild

BAD = svp.SV_ERR_INVALID_ARG
P = lambda a: ctypes.c_void_p(a)


@pytest.fixture(scope="module")
def lib():
    svbuild.build()
    return svp.load_library()


def _logits(lib, **over):
    a = dict(B=2, R=4, V=100, dtype=svp.SV_BF16, logits=P(1 << 20), out=P(1 << 24), history_max=0, history_stride=0,
             history=None, prompt_len=None, history_len=None, k=3, tokens=None, draft_len=None, repetition=None,
             presence=None, frequency=None, n_bias=0, bias_ids=None, bias_values=None, mask=None, stream=None)
    a.update(over)
    return lib.sv_process_logits(*a.values())


@pytest.mark.parametrize("over", [
    dict(B=0), dict(R=0), dict(V=0), dict(dtype=2), dict(logits=None), dict(out=None), dict(k=-1), dict(k=32),
    dict(n_bias=-1), dict(n_bias=2), dict(n_bias=2, bias_ids=P(16)), dict(history_max=5), dict(history_max=-1),
    dict(history_max=5, history=P(16), history_stride=4), dict(history_max=1 << 30, history=P(16), history_stride=1 << 30),
    dict(tokens=P(16), R=3, k=4 - 2 + 3), dict(draft_len=P(16), R=6), dict(out=P((1 << 20) + 16)),
    dict(out=P((1 << 20) - 16)), dict(logits=P((1 << 20) + 1)), dict(out=P((1 << 24) + 1)),
    dict(dtype=svp.SV_F32, logits=P((1 << 20) + 2)), dict(V=1 << 30), dict(B=1 << 20, R=1 << 11, k=1 << 4),
], ids=lambda o: ",".join(o))
def test_process_logits_refuses(lib, over):
    assert _logits(lib, **over) == BAD


def _top(lib, **over):
    a = dict(n_seq=2, t_len=3, V=100, dtype=svp.SV_BF16, target=P(1 << 20), n_rows=None, K=5, T=1.0, ids=P(16),
             logp=P(16), lse=P(16), stream=None)
    a.update(over)
    return lib.spec_kd_top(*a.values())


@pytest.mark.parametrize("over", [
    dict(n_seq=0), dict(t_len=0), dict(V=0), dict(dtype=9), dict(target=None), dict(K=0), dict(K=257), dict(T=0.0),
    dict(T=float("nan")), dict(T=float("inf")), dict(T=1e-35), dict(ids=None), dict(logp=None), dict(lse=None),
    dict(target=P((1 << 20) + 1)), dict(V=1 << 30), dict(n_seq=1 << 20, t_len=1 << 11),
], ids=lambda o: ",".join(o))
def test_kd_top_refuses(lib, over):
    assert _top(lib, **over) == BAD


def _loss(lib, **over):
    a = dict(n_seq=2, t_len=3, V=100, dtype=svp.SV_BF16, K=5, ids=P(16), logp=P(16), draft=P(1 << 20), weights=P(16),
             T=1.0, mode=svp.SV_KD_TOP_TAIL, row_kl=P(16), loss=P(16), grad=P(1 << 24), stream=None)
    a.update(over)
    return lib.spec_kd_top_loss(*a.values())


@pytest.mark.parametrize("over", [
    dict(n_seq=0), dict(t_len=0), dict(V=0), dict(V=524289), dict(dtype=-1), dict(K=0), dict(K=257), dict(ids=None),
    dict(logp=None), dict(draft=None), dict(weights=None), dict(row_kl=None), dict(loss=None), dict(T=-1.0),
    dict(T=float("nan")), dict(mode=2), dict(mode=-1), dict(grad=P(1 << 20)), dict(grad=P((1 << 20) + 64)),
    dict(grad=P((1 << 24) + 1)), dict(draft=P((1 << 20) + 1)), dict(n_seq=1 << 20, t_len=1 << 11),
], ids=lambda o: ",".join(o))
def test_kd_top_loss_refuses(lib, over):
    assert _loss(lib, **over) == BAD
