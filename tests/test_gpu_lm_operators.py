"""The language-model operators around the losses on the GPU against plain 64-bit forms
(lm_operators_ref.py), at the sizes and masks where they can go wrong.

Tolerances.  Log-sum-exp and log-probabilities: 2^-16 and 2^-23 of the logits' size, as derived for the
losses (a thread's chain is at most 256 additions, 2^-24 each, and exp2 is good to 2^-22).  Entropy: log S - A / S with
the same relative error, 2^-16, of each sum, where log S and A / S are at most log V.  A gradient: 2^-14 of
the size of its terms (the lse's and the entropy's errors enter as factors of p) and half an ulp of its type.
Embedding: one product, 2^-24, and half an ulp; its gradient: 2^-24 for each addition of a chain (32 in a chunk, then one a
chunk) of the size of the terms.  Routed layer: 2^-24 for each addition of a chain of products (under 256, and the tree) in
each of the two products, 2^-16 in all, h rounded to the type (half an ulp) on the tensor cores, and half an ulp
of the output; softmax weights 2^-20."""
import numpy as np
import pytest

import lm_operators_ref as R

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

ATOL, RTOL, GTOL = 2.0 ** -16, 2.0 ** -23, 2.0 ** -14
HALF_ULP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f32": 2.0 ** -126, "f16": 2.0 ** -24, "bf16": 2.0 ** -126}
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
LOWEST = {"f32": -3.4028235e38, "f16": -65504.0, "bf16": -3.3895314e38}


@pytest.fixture(scope="module")
def sot():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import sinkhorn_point_cloud_gb300 as s
    from sinkhorn_point_cloud_gb300 import build
    build.build()
    return s


def host(t):
    return t.detach().double().cpu().numpy()


def put(rows, dtype, pad=0, shift=0):
    """A host array on the GPU as a view with `pad` columns of NaN between its rows, `shift` elements into its memory."""
    T, V = rows.shape
    full = torch.full((T * (V + pad) + shift,), float("nan"), dtype=TYPES[dtype])
    view = full[shift:].view(T, V + pad)
    view[:, :V] = torch.as_tensor(np.asarray(rows)).to(TYPES[dtype])
    return full.cuda()[shift:].view(T, V + pad)[:, :V]


def normal(*n, seed=0, scale=1.0):
    return scale * np.random.default_rng(seed).standard_normal(n)


def near(got, ref, tol):
    """Within tol (an array or number) where the reference is finite, and the same infinities and NaN."""
    got, ref = host(got), np.asarray(ref, np.float64)
    assert got.shape == ref.shape
    assert np.array_equal(np.isnan(got), np.isnan(ref)), "NaN in other places"
    far = np.isinf(ref)
    assert np.array_equal(got[far], ref[far]) and np.isfinite(got[np.isfinite(ref)]).all()
    ok = np.isfinite(ref)
    over = (np.abs(got - ref) - np.broadcast_to(tol, ref.shape))[ok]
    assert over.size == 0 or over.max() <= 0, f"off by {over.max()} more than the bound"


# ---- scores -----------------------------------------------------------------------------------------------------------
def check_scores(sot, x, K, tau=1.0, target=None):
    xh, th = host(x), None if target is None else target.cpu().numpy()
    with np.errstate(all="ignore"):
        rp, rl, re, ri, rt = R.token_topk(xh, th, K, tau)
    logp, lse, ent, ids, top = sot.sot_token_topk(x, K, target=target, temperature=tau)
    assert ids.dtype == torch.int32 and tuple(ids.shape) == (x.shape[0], K) == tuple(top.shape)
    assert np.array_equal(ids.cpu().numpy(), ri)
    fin = np.where(np.isfinite(xh) & (np.abs(xh) < 1e30), np.abs(xh), 0.0)
    size = fin.max(axis=1) / tau
    near(lse, rl, ATOL + RTOL * np.maximum(size, np.where(np.isfinite(rl), np.abs(rl), 0)))
    near(ent, re, ATOL * (1 + np.log(x.shape[1])))
    near(top, rt, ATOL + RTOL * np.where(np.isfinite(rt), np.abs(rt), 0))
    if target is None:
        assert logp is None
    else:
        near(logp, rp, ATOL + RTOL * np.where(np.isfinite(rp), np.abs(rp), 0))
    return logp, lse, ent, ids, top


SIZES = [(1, 1), (3, 2), (5, 7), (4, 31), (17, 1000), (5, 4099), (700, 515), (2, 32768), (160, 9001), (3, 50021), (2, 131073)]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,V", SIZES)
def test_scores(sot, T, V, dtype):
    for K, pad, shift, tau, it in ((1, 0, 0, 1.0, torch.int64), (min(V, 20), 3, 1, 0.7, torch.int32),
                                   (min(V + 3, 90), 8, 0, 3.0, torch.int64), (0, 5, 3, 1.0, torch.int32)):
        x = put(normal(T, V, seed=V, scale=3.0), dtype, pad, shift)
        tg = torch.from_numpy(np.random.default_rng(1).integers(0, V, T)).to(it).cuda()
        if T > 2:
            tg[1], tg[2] = -100, V  # left out
        check_scores(sot, x, K, tau, tg)
    check_scores(sot, x, min(V, 5))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,V,K", [(2, 40000, 1024), (200, 5000, 1024), (3, 1500, 1024), (4, 131072, 128), (1, 600001, 300),
                                   (300, 2000, 256), (2, 900, 1024)])
def test_many_alternatives(sot, T, V, K, dtype):
    check_scores(sot, put(normal(T, V, seed=K, scale=3.0), dtype, 1), K)


@pytest.mark.parametrize("dtype,V", [("f32", 17000), ("bf16", 34001), ("f16", 33000)])
def test_many_long_rows(sot, V, dtype):
    """More rows than a GPU holds at a time, ordinary ones between ties, masks, bad rows and rows left out."""
    rng = np.random.default_rng(V)
    kinds = normal(12, V, seed=V, scale=2.0)
    few = rng.random(V) < 0.001
    few[V // 2] = True
    kinds[1] = 1.5
    kinds[2, ~few] = -np.inf
    kinds[3, ~few] = LOWEST[dtype]
    kinds[4] = -np.inf
    kinds[5, 7] = np.nan
    kinds[6, V - 1] = np.inf
    kinds[7] = rng.integers(0, 3, V)
    kinds[8] = np.linspace(-4, 4, V)
    kinds[9, ::2] = -np.inf
    which = rng.integers(0, 12, 1000)
    which[:12] = np.arange(12)
    x = put(kinds, dtype, 3, 1)[torch.from_numpy(which).cuda()]  # (rows are whole here)
    wide = torch.full((1000, V + 3), float("nan"), dtype=TYPES[dtype], device="cuda")
    wide[:, :V] = x
    tg = torch.full((12,), V // 2, dtype=torch.int64)
    tg[11] = -1
    for view, K in ((x, 1), (wide[:, :V], 33), (x, 128), (x, 129)):
        with np.errstate(all="ignore"):
            rp, rl, re, ri, rt = R.token_topk(host(view[:12]), tg.numpy(), K, 0.9)
            # (the type's lowest value over 0.9 lies beyond the range of a float: -inf there)
            rp, rl, rt = (np.where(np.abs(v) > 3.4028235e38, -np.inf, v) for v in (rp, rl, rt))
        logp, lse, ent, ids, top = sot.sot_token_topk(view, K, target=tg[torch.from_numpy(which)].cuda(), temperature=0.9)
        assert np.array_equal(ids.cpu().numpy(), ri[which])
        near(lse, rl[which], ATOL + RTOL * np.where(np.isfinite(rl), np.abs(rl), 0)[which])
        near(ent, re[which], ATOL * (1 + np.log(V)))
        near(top, rt[which], ATOL + RTOL * np.where(np.isfinite(rt), np.abs(rt), 0)[which])
        near(logp, rp[which], ATOL + RTOL * np.where(np.isfinite(rp), np.abs(rp), 0)[which])


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,V,Ks", [(40, 300, (17, 65, 250)), (40, 1000, (32, 100, 250)), (40, 1600, (120, 200)),
                                    (40, 4090, (65, 129, 256)), (200, 5000, (64, 65, 200)), (200, 9001, (97, 257)),
                                    (1300, 300, (9, 17, 65, 250)), (1300, 1000, (32, 100, 250)), (1300, 1600, (120, 200)),
                                    (1300, 4090, (16, 65, 129, 256)), (160, 70001, (96, 97, 128, 200)), (2, 70001, (65, 128, 400))])
def test_alternatives_of_all_kinds_of_rows(sot, T, V, Ks, dtype):
    """Ordinary rows, few distinct values, large ones side by side, masks that leave fewer than K, values far apart."""
    rng = np.random.default_rng(V)
    kinds = normal(9, V, seed=V, scale=2.0)
    kinds[1] = np.round(kinds[1])
    kinds[2] = np.round(kinds[2] * 4) / 4
    kinds[3, :V // 3] += 20.0
    kinds[4, rng.permutation(V)[:V - Ks[0] // 2]] = -np.inf
    kinds[5, rng.permutation(V)[:V - Ks[-1] - 1]] = LOWEST[dtype]
    kinds[6] = np.where(kinds[6] > 0, np.exp(4 * kinds[6]).clip(0, 6e4), -np.exp(-4 * kinds[6]).clip(0, 6e4))
    kinds[7] = np.where(np.arange(V) % 8 == 3, 3.0, kinds[7])
    kinds[8, :] = 0.0
    kinds[8, V - 20:] = np.arange(20)
    which = np.arange(T) % 9
    x = put(kinds, dtype, 5, 1)
    many = torch.full((T, V + 5), float("nan"), dtype=x.dtype, device="cuda")
    many[:, 2:V + 2] = x[torch.from_numpy(which).cuda()] if T > 9 else x[:T]
    for K in Ks:
        with np.errstate(all="ignore"):
            _, rl, _, ri, rt = R.token_topk(host(x), None, K, 1.0)
        _, lse, _, ids, top = sot.sot_token_topk(many[:, 2:V + 2], K)
        assert np.array_equal(ids.cpu().numpy(), ri[which])
        near(lse, rl[which], ATOL + RTOL * np.abs(rl)[which])
        near(top, rt[which], ATOL + RTOL * np.where(np.isfinite(rt), np.abs(rt), 0)[which])


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("V", [300, 5000, 70001])
def test_equal_logits_go_by_column(sot, V, dtype):
    rng = np.random.default_rng(V)
    rows = np.stack([np.full(V, 1.5), np.zeros(V), rng.integers(0, 3, V) * 1.0, np.where(rng.random(V) < 0.5, 0.0, -0.0),
                     np.arange(V) % 7 * 0.25, np.where(np.arange(V) == V - 1, 2.0, 1.0), np.where(rng.random(V) < 0.01, 4.0, -3.0)])
    x = put(rows, dtype, 5, 1)
    for K in (1, 33, 200):
        check_scores(sot, x, K)
    big = put(np.tile(rows, (40, 1)), dtype)  # many rows
    check_scores(sot, big, 40)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("V", [200, 4100, 66000])
def test_sorted_rows(sot, V, dtype):
    ramp = np.linspace(-8, 8, V)
    x = put(np.stack([ramp, ramp[::-1], np.roll(ramp, V // 3)]), dtype)
    for K in (1, 64, 150):
        check_scores(sot, x, K)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("V", [100, 5000, 70001])
def test_masks_and_bad_rows(sot, V, dtype):
    rng = np.random.default_rng(V)
    base = normal(10, V, seed=V, scale=2.0)
    few = rng.random(V) < 0.02
    few[V // 2] = True
    rows = base.copy()
    rows[0, ~few] = -np.inf            # fewer than K columns left
    rows[1, ~few] = LOWEST[dtype]      # masked by the type's lowest value
    rows[2] = -np.inf                  # nothing left
    rows[3] = LOWEST[dtype]            # every column at the lowest value
    rows[4, 3] = np.nan
    rows[5, V - 1] = np.inf
    rows[6] = -np.inf
    rows[6, V - 1] = 5.0               # one column left
    rows[7, ::2] = -np.inf             # half of them
    rows[8] = np.nan
    rows[9, ~few] = -1e4
    x = put(rows, dtype, 3, 1)
    tg = torch.full((10,), V // 2, dtype=torch.int64, device="cuda")
    for K in (1, 50):
        check_scores(sot, x, K, target=tg)
    check_scores(sot, x, 0, target=tg)


@pytest.mark.parametrize("offset,dtype", [(3e4, "f32"), (-3e4, "f32"), (1e9, "f32"), (-2e30, "f32"), (2e30, "bf16"), (-6e4, "f16"),
                                          (500.0, "bf16")])
def test_far_rows(sot, offset, dtype):
    rows = np.asarray(torch.from_numpy(normal(3, 9000, scale=2.0) * max(1.0, abs(offset) * 1e-3) + offset).to(TYPES[dtype]).double())
    x = put(rows, dtype)
    rp, rl, re, ri, rt = R.token_topk(rows, None, 10, 1.0)
    _, lse, ent, ids, top = sot.sot_token_topk(x, 10)
    assert np.array_equal(ids.cpu().numpy(), ri)
    near(lse, rl, ATOL + RTOL * np.abs(rl))
    near(top, rt, ATOL + RTOL * np.abs(rt))
    near(ent, re, ATOL * (1 + np.log(9000)))


def test_small_entropies_keep_their_digits(sot):
    """A row where one column has nearly everything: no cancellation against the lse."""
    rows = np.full((4, 3000), -5.0)
    rows[:, 7] = [8.0, 15.0, 25.0, 60.0]
    _, _, re, _, _ = R.token_topk(rows, None, 0, 1.0)
    _, _, ent, _, _ = sot.sot_token_topk(put(rows, "f32"), 0)
    # the weight of the largest logit is 1 exactly; what is added to it rounds to 2^-24 each, 47 in a thread's
    # chain and 5 in the tree, and A's terms are good to 2^-16
    near(ent, re, 2.0 ** -16 * re + 52 * 2.0 ** -24)


def test_scores_of_no_rows_and_row_strides(sot):
    out = sot.sot_token_topk(torch.zeros(0, 9, device="cuda"), 3, target=torch.zeros(0, dtype=torch.int64, device="cuda"))
    assert [tuple(v.shape) for v in out] == [(0,), (0,), (0,), (0, 3), (0, 3)]
    x = torch.randn(1, 40, device="cuda").expand(1, 40)
    check_scores(sot, x, 4)


def grad_close(got, ref, size, dtype):
    got = host(got)
    bound = HALF_ULP[dtype] * np.abs(ref) + GTOL * size + TINY[dtype]
    assert not np.isnan(got).any()
    assert (np.abs(got - ref) - bound).max() <= 0, (np.abs(got - ref) - bound).max()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,V", [(1, 1), (3, 2), (5, 7), (17, 1000), (5, 4099), (3, 50021), (2, 131073)])
def test_scores_gradient(sot, T, V, dtype):
    rng = np.random.default_rng(V)
    for pad, shift, tau, K in ((0, 0, 1.0, min(V, 9)), (3, 1, 0.7, min(V, 300)), (8, 0, 2.0, 0)):
        x = put(normal(T, V, seed=V, scale=3.0), dtype, pad, shift)
        tg = torch.from_numpy(rng.integers(0, V, T)).cuda()
        if T > 2:
            tg[1] = -100
        _, lse, ent, ids, _ = sot.sot_token_topk(x, K, target=tg, temperature=tau)
        if K > 3:
            ids[:, 2] = -1  # an entry that is not used
        f = lambda *n: torch.from_numpy(rng.standard_normal(n).astype(np.float32)).cuda()  # noqa: E731
        gl, gh, gt = f(T), f(T), f(T, K)
        if T > 4:
            gl[3] = gh[3] = 0
            gt[3] = 0
        for a, b, c in ((gl, gh, gt), (None, gh, None), (gl, None, None), (None, None, gt)):
            if c is not None and K == 0:
                c = None
            if a is None and b is None and c is None:
                continue
            ref = R.token_topk_grad(host(x), tg.cpu().numpy(), ids.cpu().numpy(), tau, None if a is None else host(a),
                                    None if b is None else host(b), None if c is None else host(c))
            got = sot.sot_token_topk_grad(x, lse, entropy=ent, target=tg, grad_logp=a, grad_entropy=b, ids=ids, grad_top=c,
                                          temperature=tau)
            assert got.dtype == x.dtype
            grad_close(got, *ref, dtype)
        into = torch.empty(T, V + 5, dtype=TYPES[dtype], device="cuda")[:, :V]
        kw = dict(entropy=ent, target=tg, grad_logp=gl, grad_entropy=gh, temperature=tau)
        whole = sot.sot_token_topk_grad(x, lse, **kw)
        assert torch.equal(sot.sot_token_topk_grad(x, lse, grad=into, **kw), whole)
        again = x.clone()
        assert torch.equal(sot.sot_token_topk_grad(again, lse, grad=again, **kw), whole)  # in place of the logits


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_scores_gradient_of_masks(sot, dtype):
    V = 5000
    rows = normal(5, V, scale=2.0)
    rows[0, 100:] = -np.inf
    rows[1, 100:] = LOWEST[dtype]
    rows[2] = -np.inf
    rows[3, 5] = np.nan
    rows[4] = LOWEST[dtype]
    x = put(rows, dtype)
    tg = torch.full((5,), 4, device="cuda")
    _, lse, ent, ids, _ = sot.sot_token_topk(x, 7, target=tg)
    one = torch.ones(5, device="cuda")
    got = host(sot.sot_token_topk_grad(x, lse, entropy=ent, target=tg, grad_logp=one, grad_entropy=one, ids=ids,
                                       grad_top=torch.ones(5, 7, device="cuda")))
    assert np.isnan(got[2]).all() and np.isnan(got[3]).all()
    xh = host(x)
    ref, size = R.token_topk_grad(xh[:2], np.array([4, 4]), ids[:2].cpu().numpy(), 1.0, np.ones(2), np.ones(2), np.ones((2, 7)))
    assert (np.abs(got[:2] - ref) <= HALF_ULP[dtype] * np.abs(ref) + GTOL * size + TINY[dtype]).all()
    assert (got[0, 100:] == 0).all() and (got[1, 100:] == 0).all()


def test_scores_gradient_by_differences(sot):
    """The gradient of sum(a logp + b entropy + c top) by central differences of the operator's own definition."""
    rng = np.random.default_rng(0)
    x = put(rng.standard_normal((2, 23)) * 2, "f32")
    tg = torch.tensor([3, 8]).cuda()
    a, b, c = rng.standard_normal(2), rng.standard_normal(2), rng.standard_normal((2, 4))
    _, lse, ent, ids, _ = sot.sot_token_topk(x, 4, target=tg, temperature=0.8)
    f = lambda v: torch.from_numpy(v.astype(np.float32)).cuda()  # noqa: E731
    got = host(sot.sot_token_topk_grad(x, lse, entropy=ent, target=tg, grad_logp=f(a), grad_entropy=f(b), ids=ids, grad_top=f(c),
                                       temperature=0.8))

    def total(v):
        lp, _, h, _, top = R.token_topk(v, tg.cpu().numpy(), 4, 0.8)
        return (a * lp + b * h).sum() + (c * top).sum()
    xh, step = host(x), 1e-5
    for i in range(2):
        for j in range(23):
            up, down = xh.copy(), xh.copy()
            up[i, j] += step
            down[i, j] -= step
            assert abs(got[i, j] - (total(up) - total(down)) / (2 * step)) < 1e-4


# ---- embedding --------------------------------------------------------------------------------------------------------
EMBED = [(1, 1, 1), (5, 3, 7), (40, 100, 33), (3, 50, 4096), (700, 1000, 128), (33, 77, 1001), (2000, 300, 72), (17, 9, 2056)]


@pytest.mark.parametrize("src,dst", [("f32", "f32"), ("bf16", "bf16"), ("f16", "f16"), ("f32", "bf16"), ("f16", "f32"),
                                     ("bf16", "f16")])
@pytest.mark.parametrize("T,V,D", EMBED)
def test_embed(sot, T, V, D, src, dst):
    rng = np.random.default_rng(D)
    for pad, shift, it in ((0, 0, torch.int64), (3, 1, torch.int32), (8, 0, torch.int32)):
        table = put(rng.standard_normal((V, D)), src, pad, shift)
        ids = rng.integers(0, V, T)
        if T > 3:
            ids[1], ids[2] = -1, V
        scale = np.float32(D ** 0.5)
        i = torch.from_numpy(ids).to(it).cuda()
        ref = R.embed(host(table), ids, float(scale))
        out = sot.sot_embed(table, i, scale=float(scale), dtype=TYPES[dst])
        near(out, ref, (HALF_ULP[dst] + 2.0 ** -24) * np.abs(ref) + TINY[dst])
        into = torch.full((T, D + pad), 7.0, dtype=TYPES[dst], device="cuda")
        assert torch.equal(sot.sot_embed(table, i, scale=float(scale), out=into[:, :D]), out)
        assert (into[:, D:] == 7.0).all()  # what lies between the rows stays


@pytest.mark.parametrize("src,dst", [("f32", "f32"), ("bf16", "bf16"), ("f16", "f16"), ("bf16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("T,V,D", EMBED + [(3000, 5, 40), (70000, 40, 8), (4000, 300000, 16), (33, 131072, 24)])
def test_embed_grad(sot, T, V, D, src, dst):
    rng = np.random.default_rng(T)
    for pad, shift, it, hot in ((0, 0, torch.int64, 0.0), (3, 1, torch.int32, 0.6), (8, 0, torch.int32, 1.0)):
        g = put(rng.standard_normal((T, D)), src, pad, shift)
        ids = np.where(rng.random(T) < hot, V // 2, rng.integers(0, V, T))
        if T > 3:
            ids[rng.random(T) < 0.1] = -1
            ids[2] = V
        i = torch.from_numpy(ids).to(it).cuda()
        ref, size = R.embed_grad(host(g), ids, V, 0.5)
        chain = 2.0 ** -24 * (34 + T / 16)
        got = sot.sot_embed_grad(g, i, V, scale=0.5, dtype=TYPES[dst])
        near(got, ref, HALF_ULP[dst] * np.abs(ref) + chain * size + TINY[dst])
        assert torch.equal(sot.sot_embed_grad(g, i, V, scale=0.5, dtype=TYPES[dst]), got)  # the same bits again
        old = torch.full((V, D + pad), 0.25, dtype=TYPES[dst], device="cuda")
        sot.sot_embed_grad(g, i, V, scale=0.5, grad=old[:, :D], accumulate=True)
        ref2 = ref + 0.25
        near(old[:, :D], ref2, HALF_ULP[dst] * np.abs(ref2) + chain * size + 2.0 ** -24 * (0.25 + size) + TINY[dst])
        named = np.zeros(V, bool)
        named[ids[(ids >= 0) & (ids < V)]] = True
        assert (host(old)[~named] == 0.25).all() and (old[:, D:] == 0.25).all()  # nothing else is touched


@pytest.mark.parametrize("src,dst", [("f32", "f32"), ("bf16", "bf16"), ("f16", "f32"), ("f32", "f16")])
@pytest.mark.parametrize("T", [63, 64, 65, 512, 513, 1000, 1024, 1025])
def test_embed_grad_of_rows_with_many_tokens(sot, T, src, dst):
    """One row with every token, two with half each, one with two thirds among ordinary ones, at widths that end inside
    a thread's columns and a tile."""
    rng = np.random.default_rng(T)
    V = 50
    for D, pad, shift in ((8, 0, 0), (1003, 2, 1), (1500, 4, 0), (2057, 0, 1)):
        g = put(rng.standard_normal((T, D)), src, pad, shift)
        for ids in (np.full(T, V - 1), np.arange(T) % 2 * 7, np.where(rng.random(T) < 0.67, 3, rng.integers(-2, V + 2, T))):
            i = torch.from_numpy(ids).cuda()
            ref, size = R.embed_grad(host(g), ids, V, 1.0)
            chain = 2.0 ** -24 * (64 + 16 + T / 16)  # up to 63 tokens in a chain, or a sixteenth of a row's and sixteen sums
            got = sot.sot_embed_grad(g, i, V, dtype=TYPES[dst])
            near(got, ref, HALF_ULP[dst] * np.abs(ref) + chain * size + TINY[dst])
            assert torch.equal(sot.sot_embed_grad(g, i, V, dtype=TYPES[dst]), got)
            old = torch.full((V, D + 3), 0.5, dtype=TYPES[dst], device="cuda")
            sot.sot_embed_grad(g, i, V, grad=old[:, :D], accumulate=True)
            near(old[:, :D], ref + 0.5, HALF_ULP[dst] * np.abs(ref + 0.5) + chain * size + 2.0 ** -24 * (0.5 + size) + TINY[dst])
            assert (old[:, D:] == 0.5).all()


def test_embed_without_tokens(sot):
    g, ids = torch.zeros(0, 24, device="cuda"), torch.zeros(0, dtype=torch.int64, device="cuda")
    grad = torch.full((9, 24), 3.0, device="cuda")
    assert tuple(sot.sot_embed(grad, ids).shape) == (0, 24)
    sot.sot_embed_grad(g, ids, 9, grad=grad, accumulate=True)
    assert (grad == 3).all()
    assert (sot.sot_embed_grad(g, ids, 9, grad=grad) == 0).all()
    none = torch.full((50,), -7, dtype=torch.int32, device="cuda")
    assert (sot.sot_embed_grad(torch.ones(50, 24, device="cuda"), none, 9) == 0).all()


def test_embed_beyond_32_bits(sot):
    """A table of more than 2^32 bytes and 2^31 elements: the last rows are found and written."""
    V, D = (1 << 31) // 4096 + 5, 4096
    table = torch.zeros(V, D, dtype=torch.bfloat16, device="cuda")
    table[-1], table[-5] = 2.0, 3.0
    ids = torch.tensor([V - 1, V - 5, 0], device="cuda")
    out = sot.sot_embed(table, ids)
    assert (out[0] == 2).all() and (out[1] == 3).all() and (out[2] == 0).all()
    sot.sot_embed_grad(out, ids, V, grad=table)
    assert (table[-1] == 2).all() and (table[-5] == 3).all() and float(table.sum(dtype=torch.float64)) == 5.0 * D


# ---- routed layer -----------------------------------------------------------------------------------------------------
def routed_inputs(T, H, E, F, dtype, seed=0, bias=True):
    rng = np.random.default_rng(seed)
    f = lambda *n, s=1.0: (s * torch.from_numpy(rng.standard_normal(n))).to(TYPES[dtype]).cuda()  # noqa: E731
    b = torch.from_numpy((0.3 * rng.standard_normal(E)).astype(np.float32)).cuda() if bias else None
    return f(T, H), f(E, H, s=H ** -0.5), f(E, 2 * F, H, s=H ** -0.5), f(E, H, F, s=F ** -0.5), b


def check_routed(sot, args, K, dtype, renorm=True, scale=1.0, **kw):
    x, router, gu, dn, bias = args
    with np.errstate(invalid="ignore"):
        ro, rl, ri, rw, size = R.routed(host(x), host(router), host(gu), host(dn), K, None if bias is None else host(bias), renorm,
                                        scale)
    out, logits, ids, w = sot.sot_routed_layer(x, router, gu, dn, K, bias=bias, renorm=renorm, scale=scale, **kw)
    assert np.array_equal(ids.cpu().numpy(), ri)
    near(logits, rl, 2.0 ** -23 * np.where(np.isfinite(rl), np.abs(rl), 0) + 2.0 ** -40)
    near(w, rw, 2.0 ** -20 * abs(scale))
    size = np.where(np.isfinite(ro), size, 0)
    near(out, ro, HALF_ULP[dtype] * np.where(np.isfinite(ro), np.abs(ro), 0) + (2.0 ** -16 + 2.0 ** -20 + (HALF_ULP[dtype] if dtype != "f32" else 0)) * size
         + TINY[dtype])
    return out, logits, ids, w


ROUTED = [(1, 8, 1, 8, 1), (1, 256, 16, 128, 4), (3, 40, 5, 24, 2), (7, 1032, 9, 520, 3), (16, 256, 4, 64, 4), (33, 512, 64, 192, 8),
          (64, 128, 300, 64, 8), (128, 264, 8, 136, 2), (100, 64, 3, 72, 1), (5, 64, 40, 8, 32), (128, 64, 1, 64, 1)]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,H,E,F,K", ROUTED + [(3, 33, 6, 17, 2), (2, 7, 4, 3, 4), (9, 100, 5, 50, 2)])
def test_routed_layer(sot, T, H, E, F, K, dtype):
    args = routed_inputs(T, H, E, F, dtype, seed=H)
    check_routed(sot, args, K, dtype)
    check_routed(sot, args[:4] + (None,), K, dtype, renorm=False, scale=2.5)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_routed_layer_one_expert_for_all(sot, dtype):
    """Every token chooses the same experts, and then each its own."""
    args = routed_inputs(96, 128, 12, 136, dtype)
    args[4].fill_(0.0)
    args[4][7], args[4][2] = 50.0, 40.0
    _, _, ids, _ = check_routed(sot, args, 2, dtype)
    assert (ids.cpu().numpy() == [7, 2]).all()


def test_routed_layer_removed_experts_and_bad_tokens(sot):
    x, router, gu, dn, bias = routed_inputs(6, 64, 8, 32, "bf16")
    bias.fill_(-float("inf"))
    bias[3], bias[5] = 0.0, 0.1
    _, _, ids, w = check_routed(sot, (x, router, gu, dn, bias), 4, "bf16")
    assert (ids[:, 2:] == -1).all() and (w[:, 2:] == 0).all()
    x[2, 5] = float("nan")
    x[4, 6] = float("inf")
    out, _, ids, w = sot.sot_routed_layer(x, router, gu, dn, 4, bias=bias)
    good = [0, 1, 3, 5]
    assert torch.isnan(out[2]).all() and (ids[2] == -1).all() and torch.isnan(w[2]).all()
    assert torch.isfinite(out[good]).all() and (ids[good, 0] >= 0).all()
    bias.fill_(-float("inf"))
    out, _, ids, w = sot.sot_routed_layer(x[:2], router, gu, dn, 4, bias=bias)
    assert (out == 0).all() and (ids == -1).all() and (w == 0).all()


def test_routed_layer_equal_scores_go_to_the_lower_expert(sot):
    x, router, gu, dn, bias = routed_inputs(9, 72, 20, 40, "f16")
    router[:] = router[0]
    _, _, ids, _ = check_routed(sot, (x, router, gu, dn, None), 5, "f16")
    assert (ids.cpu().numpy() == np.arange(5)).all()


def test_routed_layer_strides(sot):
    x, router, gu, dn, bias = routed_inputs(11, 80, 6, 48, "bf16")
    wide = torch.full((11, 99), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 3:83] = x
    into = torch.full((11, 90), 7.0, dtype=torch.bfloat16, device="cuda")
    a = sot.sot_routed_layer(x, router, gu, dn, 2, bias=bias)[0]
    out, _, _, _ = check_routed(sot, (wide[:, 3:83], router, gu, dn, bias), 2, "bf16", out=into[:, 5:85])
    assert (into[:, :5] == 7).all() and (into[:, 85:] == 7).all()
    assert (a.double() - out.double()).abs().max() < 0.05


def test_routed_layer_without_tokens(sot):
    x, router, gu, dn, bias = routed_inputs(1, 64, 8, 32, "bf16")
    assert [tuple(v.shape) for v in sot.sot_routed_layer(x[:0], router, gu, dn, 2)] == [(0, 64), (0, 8), (0, 2), (0, 2)]


# ---- together ---------------------------------------------------------------------------------------------------------
def test_decoding_then_training(sot):
    """Decode with embedding, routed layer and scores, distil on the alternatives, and carry the gradient back to the table."""
    V, H, E, F, T = 3001, 64, 8, 48, 24
    x, router, gu, dn, bias = routed_inputs(T, H, E, F, "bf16", seed=4)
    table = torch.from_numpy(normal(V, H, seed=5)).to(torch.bfloat16).cuda()
    ids = torch.from_numpy(np.random.default_rng(6).integers(0, V, T)).cuda()
    h = sot.sot_embed(table, ids, scale=H ** 0.5)
    y, r, chosen, _ = sot.sot_routed_layer(h, router, gu, dn, 2, bias=bias)
    logits = (0.02 * (h + y) @ table.T).contiguous()
    target = logits.argmax(1)
    logp, lse, ent, best, top = sot.sot_token_topk(logits, 16, target=target)
    assert torch.equal(best[:, 0].long(), target) and torch.equal(top[:, 0], logp)
    loss, grad = sot.sot_distill_topk(logits, best, top, tail=True, weight=torch.ones(T, device="cuda"))
    # the student is its own teacher: the loss is 0, and so is the gradient, to the rounding of the entries
    assert loss.abs().max() < 1e-5 and grad.float().abs().max() < 1e-4
    counts, _, _ = sot.sot_balance_loss(r, chosen)
    assert int(counts.sum()) == 2 * T
    g = sot.sot_token_topk_grad(logits, lse, entropy=ent, target=target, grad_logp=torch.ones(T, device="cuda"))
    assert torch.equal(g, sot.sot_token_logprob_grad(logits, target, lse, torch.ones(T, device="cuda"))) or \
        (g.float() - sot.sot_token_logprob_grad(logits, target, lse, torch.ones(T, device="cuda")).float()).abs().max() < 2.0 ** -8
    dh = (g.float() @ table.float() * 0.02).bfloat16()
    dt = sot.sot_embed_grad(dh, ids, V, scale=H ** 0.5, dtype=torch.float32)
    ref, size = R.embed_grad(host(dh), ids.cpu().numpy(), V, 8.0)
    near(dt, ref, 2.0 ** -18 * size)


def test_captured_and_replayed(sot):
    """Calls captured into a graph answer for new inputs, beside eager calls on another stream."""
    T, V, H, E, F = 6, 5000, 64, 8, 32
    x, router, gu, dn, bias = routed_inputs(T, H, E, F, "bf16")
    table = torch.from_numpy(normal(V, H)).to(torch.bfloat16).cuda()
    ids = torch.zeros(T, dtype=torch.int64, device="cuda")

    def step():
        h = sot.sot_embed(table, ids)
        y, _, chosen, _ = sot.sot_routed_layer(h, router, gu, dn, 2, bias=bias)
        logits = h @ table.T
        _, lse, ent, best, _ = sot.sot_token_topk(logits, 9)
        g = sot.sot_token_topk_grad(logits, lse, entropy=ent, grad_entropy=torch.ones_like(lse))
        return y, chosen, best, ent, g, sot.sot_embed_grad(y, ids, V)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for seed in range(3):
        ids.copy_(torch.from_numpy(np.random.default_rng(seed).integers(0, V, T)))
        torch.cuda.synchronize()
        graph.replay()
        with torch.cuda.stream(side):
            ref = step()
        torch.cuda.synchronize()
        for a, b in zip(got, ref):
            assert torch.equal(a, b)


def test_streams(sot):
    """A call on a given stream allocates and runs there."""
    s = torch.cuda.Stream()
    x = torch.randn(5, 4000, device="cuda")
    torch.cuda.synchronize()
    a = sot.sot_token_topk(x, 3, stream=s)
    e = sot.sot_embed(x, torch.arange(5, device="cuda"), stream=s)
    s.synchronize()
    b = sot.sot_token_topk(x, 3)
    assert torch.equal(a[3], b[3]) and torch.equal(a[4], b[4]) and torch.equal(e, x)
