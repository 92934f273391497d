"""The argument checks of the language-model operators around the losses: every refusal is answered on the
host, before any CUDA call, with a status and a message; the Python binding refuses tensors of the wrong
type, shape, layout or device."""
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


def topk(lib, x=P, T=4, V=10, ld=10, dt=BF16, tau=1.0, target=P, ty=I64, K=3, logp=P, lse=P, ent=P, ids=P, top=P):
    return lib.sot_token_topk(x, T, V, ld, dt, tau, target, ty, K, logp, lse, ent, ids, top, None)


def topk_grad(lib, x=P, T=4, V=10, ld=10, dt=BF16, tau=1.0, target=P, ty=I64, lse=P, ent=P, gl=P, gh=P, ids=P, K=3, gt=P,
              grad=P, ldg=10):
    return lib.sot_token_topk_grad(x, T, V, ld, dt, tau, target, ty, lse, ent, gl, gh, ids, K, gt, grad, ldg, None)


def embed(lib, table=P, V=10, D=6, ld=6, ty=BF16, ids=P, ity=I64, T=4, scale=1.0, out=P, ldo=6, oty=BF16):
    return lib.sot_embed(table, V, D, ld, ty, ids, ity, T, scale, out, ldo, oty, None)


def embed_grad(lib, g=P, T=4, D=6, ld=6, ty=BF16, ids=P, ity=I64, V=10, scale=1.0, acc=0, grad=P, ldg=6, gty=F32):
    return lib.sot_embed_grad(g, T, D, ld, ty, ids, ity, V, scale, acc, grad, ldg, gty, None)


def routed(lib, x=P, T=4, H=16, ld=16, dt=BF16, router=P, bias=None, E=8, gu=P, dn=P, F=8, K=2, renorm=1, scale=1.0, out=P,
           ldo=16, logits=P, ids=P, w=P):
    return lib.sot_routed_layer(x, T, H, ld, dt, router, bias, E, gu, dn, F, K, renorm, scale, out, ldo, logits, ids, w, None)


@pytest.mark.parametrize("call", [topk, topk_grad])
def test_rows_of_logits_refused(lib, call):
    for kw in (dict(T=-1), dict(V=0), dict(ld=9), dict(dt=I32), dict(dt=7), dict(x=None), dict(x=ODD), dict(T=1 << 31),
               dict(ld=1 << 30), dict(tau=0.0), dict(tau=-1.0), dict(tau=INF), dict(tau=NAN), dict(ty=F32), dict(K=-1),
               dict(K=1025), dict(target=ODD)):
        assert call(lib, **kw) == BAD, kw
        assert lib.sot_last_error()
    assert call(lib, T=0, x=None) == OK


def test_scores_missing_arrays_refused(lib):
    assert topk(lib, target=None) == BAD  # logp without a target
    assert topk(lib, logp=None, lse=None, ent=None, ids=None, top=None) == BAD
    assert topk(lib, logp=None, lse=None, ent=None, K=0) == BAD
    for kw in (dict(lse=None), dict(grad=None), dict(ent=None), dict(ids=None), dict(target=None), dict(ldg=9),
               dict(grad=ODD), dict(ldg=1 << 30)):
        assert topk_grad(lib, **kw) == BAD, kw
    big = dict(V=1 << 28, ld=1 << 28)
    assert topk(lib, **big) == UNSUP and b"do not fit" in lib.sot_last_error()


def test_embedding_refused(lib):
    for call, rows in ((embed, "T"), (embed_grad, "T")):
        for kw in (dict(T=-1), dict(T=1 << 31), dict(D=0), dict(V=0), dict(ld=5), dict(ld=1 << 30), dict(ty=I32), dict(ity=F32),
                   dict(ids=None), dict(ids=ODD), dict(scale=INF), dict(scale=NAN)):
            assert call(lib, **kw) == BAD, (call.__name__, kw)
            assert lib.sot_last_error()
    for kw in (dict(table=None), dict(table=ODD), dict(out=None), dict(out=ODD), dict(ldo=5), dict(oty=I64)):
        assert embed(lib, **kw) == BAD, kw
    for kw in (dict(g=None), dict(g=ODD), dict(grad=None), dict(grad=ODD), dict(ldg=5), dict(gty=9), dict(V=0x7fffffff)):
        assert embed_grad(lib, **kw) == BAD, kw
    assert embed(lib, T=0, out=None, ids=None, table=None) == OK
    assert embed_grad(lib, T=0, g=None, ids=None, grad=None, acc=1) == OK


def test_routed_layer_refused(lib):
    for kw in (dict(T=-1), dict(H=0), dict(E=0), dict(F=0), dict(K=0), dict(K=9), dict(ld=15), dict(ldo=15), dict(dt=I32),
               dict(x=None), dict(x=ODD), dict(router=None), dict(gu=None), dict(dn=ODD), dict(out=None), dict(logits=None),
               dict(ids=None), dict(w=None), dict(scale=NAN)):
        assert routed(lib, **kw) == BAD, kw
        assert lib.sot_last_error()
    for kw in (dict(T=129), dict(E=1025), dict(E=64, K=33), dict(F=(1 << 20) + 1)):
        assert routed(lib, **kw) == UNSUP, kw
    assert routed(lib, T=0, x=None, out=None) == OK


def test_binding_refuses_wrong_tensors():
    x, t = torch.zeros(3, 8), torch.zeros(3, dtype=torch.int64)
    with pytest.raises(ValueError, match="CUDA"):
        binding.sot_token_topk(x, 2, target=t)
    with pytest.raises(TypeError, match="float32, float16 or bfloat16"):
        binding.sot_token_topk(x.double(), 2)
    with pytest.raises(ValueError, match="CUDA"):
        binding.sot_token_topk_grad(x, t.float())
    with pytest.raises(ValueError, match="CUDA"):
        binding.sot_embed(x, t)
    with pytest.raises(ValueError, match="rows, columns"):
        binding.sot_embed(torch.zeros(2, 3, 4), t)
    with pytest.raises(ValueError, match="CUDA"):
        binding.sot_embed_grad(x, t, 5)
    with pytest.raises(ValueError, match="CUDA"):
        binding.sot_routed_layer(x, torch.zeros(4, 8), torch.zeros(4, 8, 8), torch.zeros(4, 8, 4), 2)
