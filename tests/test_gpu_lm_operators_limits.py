"""The language-model operators around the losses where their ranges end: gradients of rows far from zero, the most
alternatives, the longest rows that have any, and the routed layer's fullest shared memory.  Tolerances are those of
test_gpu_lm_operators.py unless a test derives its own."""
import numpy as np
import pytest

import lm_operators_ref as R
from test_gpu_lm_operators import (ATOL, GTOL, HALF_ULP, LOWEST, RTOL, TINY, check_routed, grad_close,  # noqa: F401
                                   host, near, normal, put, routed_inputs, sot)

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


# ---- gradients of rows far from zero --------------------------------------------------------------------------------
# p comes from x / tau - lse, where the stored lse, its product and x / tau are each good to 2^-24 of the lse: 2^-22 with the
# difference's own rounding, beside the lse's ATOL.  With e that error, p is off by expm1(e) of itself, and the entropy's
# term p (log p + H) by that much of p (|log p| + H + 1) and by e p once more.
FAR = [("f32", 600.0), ("f32", -600.0), ("f32", 706.0), ("f32", 712.0), ("f32", -712.0), ("f32", 3e4), ("f32", -3e4),
       ("f32", 1e6), ("bf16", 500.0), ("bf16", 3e4), ("bf16", -3e4), ("f16", 600.0), ("f16", 3e4), ("f16", -3e4)]


@pytest.mark.parametrize("tau", [1.0, 0.7])
@pytest.mark.parametrize("dtype,offset", FAR)
def test_gradient_of_far_rows(sot, dtype, offset, tau):
    rng = np.random.default_rng(int(abs(offset)))
    T, V, K = 5, 3001, 6
    step = abs(offset) * HALF_ULP[dtype] * 2  # of the type, there
    rows = offset + max(2.0, 2.0 * step) * rng.standard_normal((T, V))
    x = put(rows, dtype, 3, 1)
    tg = torch.from_numpy(rng.integers(0, V, T)).cuda()
    tg[1] = -100
    _, lse, ent, ids, _ = sot.sot_token_topk(x, K, target=tg, temperature=tau)
    f = lambda *n: torch.from_numpy(rng.standard_normal(n).astype(np.float32)).cuda()  # noqa: E731
    gl, gh, gt = f(T), f(T), f(T, K)
    e = 2.0 ** -22 * host(lse.abs())[:, None] + ATOL
    assert e.max() < 0.5
    for a, b, c in ((gl, gh, gt), (None, gh, None), (gl, None, None), (None, None, gt)):
        ref, size = R.token_topk_grad(host(x), tg.cpu().numpy(), ids.cpu().numpy(), tau, None if a is None else host(a),
                                      None if b is None else host(b), None if c is None else host(c))
        got = host(sot.sot_token_topk_grad(x, lse, entropy=ent, target=tg, grad_logp=a, grad_entropy=b, ids=ids, grad_top=c,
                                           temperature=tau))
        assert np.isfinite(got).all() and (got[1] == 0).all()
        over = np.abs(got - ref) - HALF_ULP[dtype] * np.abs(ref) - (GTOL + 2.0 * np.expm1(e)) * size - TINY[dtype]
        assert over.max() <= 0, over.max()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_gradient_of_a_row_at_the_lowest_value(sot, dtype):
    """Every column at the type's lowest value.  In fp16 the lse still tells the columns apart from one alone; in the
    wider types it is the value itself, log V below its rounding, so that p = 1 for each column."""
    V = 5000
    x = put(np.full((2, V), LOWEST[dtype]), dtype)
    tg = torch.tensor([4, 4990]).cuda()
    _, lse, ent, ids, _ = sot.sot_token_topk(x, 7, target=tg)
    assert (ids.cpu().numpy() == np.arange(7)).all()
    near(ent, np.full(2, np.log(V)), ATOL * (1 + np.log(V)))
    one = torch.ones(2, device="cuda")
    got = host(sot.sot_token_topk_grad(x, lse, entropy=ent, target=tg, grad_logp=one, grad_entropy=one, ids=ids,
                                       grad_top=torch.ones(2, 7, device="cuda")))
    p, l = np.full(2, 1.0 / V), np.full(2, -np.log(V))
    if dtype != "f16":
        assert np.array_equal(host(lse), np.full(2, host(x)[0, 0]))
        p, l = np.ones(2), np.zeros(2)
    into = np.zeros((2, V))
    into[:, :7] += 1
    into[[0, 1], [4, 4990]] += 1
    ref = into - p[:, None] * 8 - (p * (l + host(ent)))[:, None]
    e = 2.0 ** -22 * abs(LOWEST["f16"]) if dtype == "f16" else 2.0 ** -22
    # (no entropy's term but its error is left in fp16: log p + H = 0)
    tol = HALF_ULP[dtype] * np.abs(ref) + (p * (8 + np.abs(l) + host(ent) + 1))[:, None] * (GTOL + 2 * np.expm1(e))
    assert (np.abs(got - ref) <= tol).all(), (np.abs(got - ref) - tol).max()


# ---- the most alternatives ------------------------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,V,K", [(3, 1500, 1024), (2, 50021, 1024), (40, 1024, 1024), (3, 900, 1023), (1, 131073, 1000)])
def test_gradient_of_many_alternatives(sot, T, V, K, dtype):
    rng = np.random.default_rng(V)
    x = put(normal(T, V, seed=V, scale=3.0), dtype, 3, 1)
    tg = torch.from_numpy(rng.integers(0, V, T)).cuda()
    _, lse, ent, ids, _ = sot.sot_token_topk(x, K, target=tg)
    if T > 1:
        tg[1] = ids[1, min(V, K) - 1]  # the target among the entries
    f = lambda *n: torch.from_numpy(rng.standard_normal(n).astype(np.float32)).cuda()  # noqa: E731
    gl, gh, gt = f(T), f(T), f(T, K)
    ref, size = R.token_topk_grad(host(x), tg.cpu().numpy(), ids.cpu().numpy(), 1.0, host(gl), host(gh), host(gt))
    kw = dict(entropy=ent, target=tg, grad_logp=gl, grad_entropy=gh, ids=ids, grad_top=gt)
    got = sot.sot_token_topk_grad(x, lse, **kw)
    # (the sum of K gradients: K / 64 additions in a thread's chain and a tree of 8 more, 2^-24 of their size each)
    grad_close(got, ref, size * (1 + (K / 64 + 8) * 2.0 ** -24 / GTOL), dtype)
    again = x.clone()
    assert torch.equal(sot.sot_token_topk_grad(again, lse, grad=again, **kw), got)


@pytest.mark.parametrize("dtype,V", [("f32", 7_300_001), ("bf16", 14_500_003)])
@pytest.mark.parametrize("K", [513, 1024])
def test_alternatives_of_the_longest_rows(sot, dtype, V, K):
    """Ordinary logits, few distinct ones (ties over all slices), and all large ones in one slice."""
    rng = np.random.default_rng(K)
    rows = rng.standard_normal((3, V), np.float32).astype(np.float64)
    rows[1] = np.round(rows[1] * 4) / 4
    rows[2, V // 2:V // 2 + 5000] += 9.0
    x = put(rows, dtype, 3, 1)
    _, rl, re, ri, rt = R.token_topk(host(x), None, K, 1.0)
    _, lse, ent, ids, top = sot.sot_token_topk(x, K)
    assert np.array_equal(ids.cpu().numpy(), ri)
    # eight CTAs a row, 256 threads with two sums each: chains of V / 4096 additions, 2^-24 each
    tol = ATOL + V / 4096 * 2.0 ** -24
    near(lse, rl, tol + RTOL * np.abs(rl))
    near(ent, re, tol * (1 + np.log(V)))
    near(top, rt, tol + RTOL * np.abs(rt))


# ---- the routed layer's fullest shared memory --------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("T,H,E,F,K", [(128, 64, 1024, 24, 32), (128, 96, 32, 72, 32), (128, 64, 1000, 16, 8), (15, 72, 1024, 32, 32),
                                       (14, 72, 1024, 32, 1), (1, 64, 1024, 64, 32), (128, 136, 257, 40, 31)])
def test_routed_layer_at_its_limits(sot, T, H, E, F, K, dtype):
    args = routed_inputs(T, H, E, F, dtype, seed=E + T)
    a = check_routed(sot, args, K, dtype)
    for v, w in zip(sot.sot_routed_layer(*args[:4], K, bias=args[4]), a):
        assert torch.equal(v, w)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("K", [1, 4, 32])
def test_routed_layer_with_all_tokens_at_the_same_experts(sot, K, dtype):
    """128 tokens of each chosen expert among 1024: the widest tokens' side beside the fullest lists."""
    x, router, gu, dn, bias = routed_inputs(128, 200, 1024, 40, dtype, seed=K)
    bias.fill_(0.0)
    which = torch.arange(K, device="cuda") * 31 + 7
    bias[which] = 14.0 + torch.arange(K, device="cuda") % 2
    _, _, ids, _ = check_routed(sot, (x, router, gu, dn, bias), K, dtype)
    assert torch.equal(ids.sort(1).values.long(), which.expand(128, K))


# ---- whole numbers beyond 32 bits -----------------------------------------------------------------------------------------
def test_numbers_beyond_32_bits_are_refused(sot):
    """Not taken for what is left of them: 2^32 + 5 rows are not five."""
    x, ids = torch.ones(1, 1, dtype=torch.bfloat16, device="cuda"), torch.tensor([7], device="cuda")
    for V in ((1 << 32) + 5, 1 << 31):
        with pytest.raises(ValueError, match="V must satisfy"):
            sot.sot_embed_grad(x, ids, V)
    with pytest.raises(ValueError, match="K must satisfy"):
        sot.sot_token_topk(x, (1 << 32) + 3)
    table = torch.empty((1 << 32) + 5, 1, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="V must satisfy"):
        sot.sot_embed(table, ids)
    with pytest.raises(ValueError, match="V must satisfy"):
        sot.sot_embed_grad(x, ids, (1 << 32) + 5, grad=table)
