"""Host-side checks of the policy operators' entry points: each bad call is
refused before anything is launched (no GPU needed)."""
import ctypes

import pytest
import torch

import speculative_decoding_verification_71_gb300 as svp
from speculative_decoding_verification_71_gb300 import build as svbuild

BAD, OK = svp.SV_ERR_INVALID_ARG, svp.SV_OK
P = lambda a: ctypes.c_void_p(a)
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    svbuild.build()
    return svp.load_library()


ROWS = [dict(n_seq=0), dict(t_len=0), dict(V=0), dict(dtype=2), dict(logits=None), dict(tokens=None), dict(T=0.0),
        dict(T=-1.0), dict(T=NAN), dict(T=INF), dict(T=1e-35), dict(logits=P((1 << 20) + 1)), dict(V=524289),
        dict(n_seq=1 << 20, t_len=1 << 11), dict(logp=None)]
GRAD = [dict(grad=P((1 << 20) + 64)), dict(grad=P((1 << 20) - 64)), dict(grad=P((1 << 24) + 1))]


def _logp(lib, **over):
    a = dict(n_seq=2, t_len=3, V=100, dtype=svp.SV_BF16, logits=P(1 << 20), tokens=P(16), T=1.0, logp=P(16),
             entropy=None, lse=P(16), stream=None)
    a.update(over)
    return lib.sv_token_logp(*a.values())


@pytest.mark.parametrize("over", ROWS + [dict(lse=None)], ids=lambda o: ",".join(o))
def test_token_logp_refuses(lib, over):
    assert _logp(lib, **over) == BAD


def _logp_grad(lib, **over):
    a = dict(n_seq=2, t_len=3, V=100, dtype=svp.SV_BF16, logits=P(1 << 20), tokens=P(16), logp=P(16), lse=P(16),
             entropy=None, d_logp=P(16), d_entropy=None, T=1.0, grad=P(1 << 24), stream=None)
    a.update(over)
    return lib.sv_token_logp_grad(*a.values())


@pytest.mark.parametrize("over", ROWS + GRAD + [dict(lse=None), dict(d_logp=None), dict(grad=None), dict(entropy=P(16)),
                                                dict(d_entropy=P(16))], ids=lambda o: ",".join(o))
def test_token_logp_grad_refuses(lib, over):
    assert _logp_grad(lib, **over) == BAD


def _policy(lib, **over):
    a = dict(n_seq=2, t_len=3, V=100, dtype=svp.SV_BF16, logits=P(1 << 20), tokens=P(16), adv=P(16), per_token=0,
             weights=P(16), old=P(16), ref=P(16), T=1.0, low=0.2, high=0.2, dual=0.0, kl=0.1, ent=0.0, logp=P(16),
             entropy=None, row_loss=P(16), loss=P(16), grad=P(1 << 24), stream=None)
    a.update(over)
    return lib.sv_policy_loss(*a.values())


@pytest.mark.parametrize("over", ROWS + GRAD + [
    dict(adv=None), dict(weights=None), dict(row_loss=None), dict(loss=None), dict(ref=None), dict(per_token=2),
    dict(low=-0.1), dict(low=1.5), dict(low=NAN), dict(high=-0.1), dict(high=INF), dict(dual=1.0), dict(dual=-2.0),
    dict(dual=NAN), dict(dual=INF), dict(kl=NAN), dict(kl=INF), dict(ent=NAN)], ids=lambda o: ",".join(o))
def test_policy_loss_refuses(lib, over):
    assert _policy(lib, **over) == BAD


def _preference(lib, **over):
    a = dict(n_seq=2, t_len=3, V=100, dtype=svp.SV_BF16, logits=P(1 << 20), tokens=P(16), ref=P(16), weights=P(16),
             T=1.0, beta=0.1, kind=0, smoothing=0.0, average=0, logp=P(16), margin=P(16), loss=P(16), grad=P(1 << 24),
             work=P(256), stream=None)
    a.update(over)
    return lib.sv_preference_loss(*a.values())


@pytest.mark.parametrize("over", ROWS + GRAD + [
    dict(ref=None), dict(weights=None), dict(margin=None), dict(loss=None), dict(work=None), dict(work=P(260)),
    dict(beta=0.0), dict(beta=-1.0), dict(beta=NAN), dict(beta=INF), dict(kind=3), dict(kind=-1), dict(smoothing=-0.1),
    dict(smoothing=0.5), dict(smoothing=NAN), dict(smoothing=0.1, kind=1), dict(smoothing=0.1, kind=2),
    dict(average=2), dict(n_seq=1 << 28, t_len=1)], ids=lambda o: ",".join(o))
def test_preference_loss_refuses(lib, over):
    assert _preference(lib, **over) == BAD


def test_preference_work_is_zero_for_bad_sizes(lib):
    assert lib.sv_preference_work(0, 3) == 0 and lib.sv_preference_work(2, 0) == 0
    assert lib.sv_preference_work(2, 3) >= 12


def _clip(lib, n=2, at=(1 << 20, 1 << 22), sizes=(100, 50), dtypes=(1, 0), kind=0, max_norm=1.0, outs=None,
          out_dtypes=None, norm=P(64), work=P(1 << 16)):
    arr = lambda kind_, v: None if v is None else (kind_ * max(len(v), 1))(*v)
    return lib.sv_clip_gradients(n, arr(ctypes.c_void_p, at), arr(ctypes.c_longlong, sizes), arr(ctypes.c_int, dtypes),
                                 kind, max_norm, arr(ctypes.c_void_p, outs), arr(ctypes.c_int, out_dtypes), norm, work,
                                 None)


@pytest.mark.parametrize("over", [
    dict(n=-1), dict(at=None), dict(sizes=None), dict(dtypes=None), dict(kind=2), dict(kind=-1), dict(max_norm=0.0),
    dict(max_norm=-1.0), dict(max_norm=NAN), dict(norm=None), dict(work=None), dict(sizes=(100, -1)),
    dict(sizes=(100, 1 << 41)), dict(dtypes=(1, 2)), dict(at=(1 << 20, 0)), dict(at=((1 << 20) + 1, 1 << 22)),
    dict(at=(1 << 20, (1 << 22) + 2)), dict(outs=(1 << 24, 1 << 25)), dict(out_dtypes=(1, 0)),
    dict(outs=(1 << 24, 1 << 25), out_dtypes=(1, 1)),                     # bfloat16 from float32
    dict(outs=(1 << 24, 0), out_dtypes=(1, 0)), dict(outs=(1 << 24, 1 << 25), out_dtypes=(3, 0)),
    dict(at=(1 << 20, 1 << 20), sizes=(100, 50)),                          # the same tensor twice
    dict(at=(1 << 20, (1 << 20) + 196), sizes=(100, 50)),                  # the second begins inside the first
    dict(at=((1 << 20) + 8, 1 << 20), sizes=(1, 50)),                      # the first lies inside the second
    dict(outs=(1 << 24, 1 << 24), out_dtypes=(1, 0)), dict(outs=(1 << 22, 1 << 25), out_dtypes=(1, 0)),
    dict(outs=(1 << 20, 1 << 25), out_dtypes=(0, 0)),                      # float32 over its own bfloat16
    dict(norm=P((1 << 20) + 4)), dict(work=P((1 << 20) - 8)), dict(norm=P((1 << 16) + 8)), dict(norm=P(66)),
    dict(work=P((1 << 16) + 4))], ids=lambda o: ",".join(o))
def test_clip_gradients_refuses(lib, over):
    assert _clip(lib, **over) == BAD


def test_the_binding_refuses_on_the_host(lib):
    z, t, r = torch.zeros(2, 3, 8), torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2)
    for call in (lambda: svp.token_logp(z, t), lambda: svp.policy_loss(z, t, r, r), lambda: svp.preference_loss(z, t, r, r[:1]),
                 lambda: svp.token_logp_grad(z, t, z[..., 0], z[..., 0], z[..., 0])):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()
    with pytest.raises(TypeError):
        svp.token_logp(z.double(), t)
    with pytest.raises(TypeError):
        svp.token_logp([1.0], t)
    with pytest.raises(ValueError, match="three dimensions"):
        svp.token_logp(z[0], t)
    with pytest.raises(ValueError, match="CUDA tensors"):
        svp.clip_gradients([z])
    for bad, error in ((z, TypeError), ([], ValueError), ([None], ValueError), ([1.0], TypeError)):
        with pytest.raises(error):
            svp.clip_gradients(bad)
    with pytest.raises(ValueError, match="max_norm"):
        svp.clip_gradients([z], max_norm=0.0)
    with pytest.raises(ValueError, match="max_norm"):
        svp.clip_gradients([z], max_norm=NAN)
    with pytest.raises(ValueError, match="max_norm"):
        svp.clip_gradients([z], out=[z])
    with pytest.raises(ValueError, match="kind"):
        svp.clip_gradients([z], kind="l1")
    with pytest.raises(ValueError, match="each of grads"):
        svp.clip_gradients([z, z], 1.0, out=[z])


def test_dense_layouts():
    z = torch.zeros(4, 6, 5)
    assert svp._is_dense(z) and svp._is_dense(z.transpose(0, 2)) and svp._is_dense(z[1:3]) and svp._is_dense(z[0, 0, 0])
    assert svp._is_dense(torch.zeros(0, 3)) and svp._is_dense(torch.zeros(3, 1, 2).transpose(0, 1))
    assert not svp._is_dense(z[:, :3]) and not svp._is_dense(z[..., ::2]) and not svp._is_dense(torch.zeros(1).expand(5))
