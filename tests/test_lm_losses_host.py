"""The language-model losses' argument checks: every refusal is answered on the
host, before any CUDA call, with a status and a message; the Python binding
refuses tensors of the wrong type, shape, layout or device."""
import ctypes as C

import pytest
import torch

from sinkhorn_point_cloud_gb300 import binding, build

BAD, UNSUP, OK = binding.SOT_ERR_INVALID_ARG, binding.SOT_ERR_UNSUPPORTED, binding.SOT_OK
F32, F16, BF16, I32, I64 = binding.SOT_F32, binding.SOT_F16, binding.SOT_BF16, binding.SOT_I32, binding.SOT_I64
P = C.c_void_p(64)  # never dereferenced: the checks fail first
ODD = C.c_void_p(65)
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


def logprob(lib, x=P, T=4, V=10, ld=10, dt=BF16, tau=1.0, target=P, ty=I64, logp=P, lse=P):
    return lib.sot_token_logprob(x, T, V, ld, dt, tau, target, ty, logp, lse, None)


def logprob_grad(lib, x=P, T=4, V=10, ld=10, dt=BF16, tau=1.0, target=P, ty=I64, lse=P, g=P, grad=P, ldg=10):
    return lib.sot_token_logprob_grad(x, T, V, ld, dt, tau, target, ty, lse, g, grad, ldg, None)


def distill(lib, x=P, T=4, V=10, ld=10, dt=BF16, tau=1.0, ids=P, ty=I32, teacher=P, tt=F32, K=3, tail=0, w=P, loss=P,
            grad=P, ldg=10):
    return lib.sot_distill_topk(x, T, V, ld, dt, tau, ids, ty, teacher, tt, K, tail, w, loss, grad, ldg, None)


def policy(lib, x=P, T=4, V=10, ld=10, dt=BF16, tau=1.0, target=P, ty=I64, old=P, ref=P, adv=P, w=P, lo=0.2, hi=0.2,
           kc=0.1, loss=P, logp=P, kl=P, grad=P, ldg=10):
    return lib.sot_policy_loss(x, T, V, ld, dt, tau, target, ty, old, ref, adv, w, lo, hi, kc, loss, logp, kl, grad, ldg,
                               None)


def preference(lib, logp=P, ref=P, target=None, ty=I64, off=P, n=2, T=9, beta=0.1, ls=0.0, avg=0, scale=1.0, loss=P,
               margin=P, grad=P):
    return lib.sot_preference_loss(logp, ref, target, ty, off, n, T, beta, ls, avg, scale, loss, margin, grad, None)


def balance(lib, x=P, T=4, E=8, ld=8, dt=F32, ids=P, ty=I32, K=2, mask=None, cb=1.0, cz=0.0, counts=P, loss=P, grad=P,
            ldg=8):
    return lib.sot_balance_loss(x, T, E, ld, dt, ids, ty, K, mask, cb, cz, counts, loss, grad, ldg, None)


@pytest.mark.parametrize("call", [logprob, logprob_grad, distill, policy])
def test_rows_of_logits_refused(lib, call):
    for kw in (dict(T=-1), dict(V=0), dict(V=-3), dict(ld=9), dict(dt=I32), dict(dt=7), dict(dt=-1), dict(x=None),
               dict(x=ODD), dict(T=1 << 31), dict(ld=1 << 30), dict(tau=0.0), dict(tau=-1.0), dict(tau=INF),
               dict(tau=NAN), dict(tau=1e-45), dict(ty=F32), dict(ty=9)):
        assert call(lib, **kw) == BAD, kw
        assert lib.sot_last_error()
    assert call(lib, T=0, x=None) == OK


@pytest.mark.parametrize("call", [logprob_grad, distill, policy])
def test_gradient_rows_refused(lib, call):
    assert call(lib, ldg=9) == BAD
    assert call(lib, grad=ODD) == BAD
    assert call(lib, ldg=1 << 30) == BAD


def test_missing_arrays_refused(lib):
    assert logprob(lib, target=None) == BAD
    assert logprob(lib, logp=None, lse=None) == BAD
    for kw in (dict(target=None), dict(lse=None), dict(g=None), dict(grad=None)):
        assert logprob_grad(lib, **kw) == BAD, kw
    for kw in (dict(ids=None), dict(teacher=None), dict(loss=None, grad=None), dict(ids=ODD), dict(teacher=ODD)):
        assert distill(lib, **kw) == BAD, kw
    for kw in (dict(target=None), dict(old=None), dict(adv=None), dict(loss=None, logp=None, kl=None, grad=None)):
        assert policy(lib, **kw) == BAD, kw
    for kw in (dict(logp=None), dict(off=None), dict(loss=None, margin=None, grad=None), dict(off=C.c_void_p(68))):
        assert preference(lib, **kw) == BAD, kw
    for kw in (dict(x=None), dict(ids=None), dict(counts=None), dict(loss=None)):
        assert balance(lib, **kw) == BAD, kw


def test_values_refused(lib):
    for kw in (dict(K=0), dict(K=1025), dict(tt=I32), dict(tail=1, tau=2.0)):
        assert distill(lib, **kw) == BAD, kw
    for kw in (dict(lo=-0.1), dict(lo=1.1), dict(hi=-0.1), dict(hi=INF), dict(lo=NAN), dict(kc=NAN), dict(ref=None)):
        assert policy(lib, **kw) == BAD, kw
    for kw in (dict(n=-1), dict(T=-1), dict(beta=NAN), dict(scale=INF), dict(ls=-0.1), dict(ls=0.6),
               dict(target=P, ty=F32)):
        assert preference(lib, **kw) == BAD, kw
    for kw in (dict(K=0), dict(K=1 << 30, T=4), dict(cb=INF), dict(cz=NAN), dict(ty=F32), dict(dt=I64), dict(ldg=7),
               dict(ld=7)):
        assert balance(lib, **kw) == BAD, kw


def test_sizes_without_a_kernel(lib):
    assert distill(lib, V=1 << 27, ld=1 << 27, ldg=1 << 27, dt=F32, tail=1) == UNSUP
    assert b"do not fit" in lib.sot_last_error()
    assert balance(lib, E=1025, ld=1025, ldg=1025) == UNSUP


def test_binding_refuses_wrong_tensors():
    x = torch.zeros(3, 8)
    t = torch.zeros(3, dtype=torch.int64)
    with pytest.raises(ValueError, match="CUDA"):
        binding.sot_token_logprob(x, t)
    with pytest.raises(TypeError, match="float32, float16 or bfloat16"):
        binding.sot_token_logprob(x.double(), t)
    with pytest.raises(TypeError):
        binding.sot_token_logprob([1.0], t)
    with pytest.raises(ValueError, match="rows, columns"):
        binding.sot_policy_loss(torch.zeros(2, 3, 8), t, t, t)
    with pytest.raises(ValueError, match="CUDA"):
        binding.sot_preference_loss(torch.zeros(4), torch.zeros(3, dtype=torch.int64))
    with pytest.raises(ValueError, match="CUDA"):
        binding.sot_balance_loss(x, torch.zeros(3, 2, dtype=torch.int32))
