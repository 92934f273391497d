"""The language-model losses on the GPU against plain 64-bit forms (lm_ref.py), at the
sizes and masks where they can go wrong, and their gradients against differences.

Tolerances.  A probability is exp2 of a rounded product: the hardware's exp2 is
good to 2^-22 of its value, the difference x - m and its product with
log2(e)/tau to 2^-24 each of their size, at most 2^-23 |t| with |t| < 64 for any
term that matters, 2^-17 in all; a row's sum of positive terms adds at most
2^-24 per term of a thread's chain (under 256) and of the trees: below 2^-16.
So a log-sum-exp is within ATOL = 2^-16 of the truth, and usually far nearer;
a gradient is within 2^-14 of the size of the terms that make it up, plus half
an ulp of its type (and half of the type's smallest value)."""
import numpy as np
import pytest

import lm_ref as R

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

ATOL = 2.0 ** -16
RTOL = 2.0 ** -23
GTOL = 2.0 ** -14
HALF_ULP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f32": 2.0 ** -126, "f16": 2.0 ** -24, "bf16": 2.0 ** -126}
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


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


def rows(T, V, dtype, pad=0, seed=0, spread=3.0):
    """Logits on the GPU, `pad` columns of NaN between the rows."""
    g = torch.Generator().manual_seed(seed)
    full = torch.full((T, V + pad), float("nan"), dtype=TYPES[dtype])
    full[:, :V] = (torch.randn(T, V, generator=g) * spread).to(TYPES[dtype])
    return full.cuda()[:, :V]


def targets(T, V, seed=1, dtype=torch.int64):
    return torch.randint(0, V, (T,), generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def close_grad(got, ref, size, dtype):
    got = host(got)
    bound = HALF_ULP[dtype] * np.abs(ref) + GTOL * size + TINY[dtype]
    over = np.abs(got - ref) - bound
    assert not np.isnan(got).any()
    assert over.max() <= 0, (over.max(), np.unravel_index(over.argmax(), over.shape))


def close(got, ref, scale=1.0, size=None):
    got = host(got)
    size = np.abs(ref) if size is None else size
    assert np.array_equal(np.isfinite(got), np.isfinite(ref))
    ok = np.isfinite(ref)
    assert np.all(np.abs(got - ref)[ok] <= scale * ATOL + RTOL * np.broadcast_to(size, ref.shape)[ok]), \
        np.abs(got - ref)[ok].max()


SIZES = [(1, 1), (3, 2), (5, 7), (2, 8), (4, 31), (3, 1000), (17, 4099), (2, 32768), (3, 50021), (2, 131073)]
BIG = [("bf16", 2, 400001), ("f32", 2, 262145), ("f16", 1, 800000)]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,V", SIZES)
def test_token_logprob(sot, T, V, dtype):
    for pad, tau, it in ((0, 1.0, torch.int64), (3, 0.7, torch.int32), (8, 3.0, torch.int64)):
        x, tg = rows(T, V, dtype, pad, seed=V), targets(T, V, dtype=it)
        if T > 2:
            tg[1] = -100
            tg[2] = V  # out of range: left out as well
        logp, lse = sot.sot_token_logprob(x, tg, temperature=tau)
        rp, rl = R.token_logprob(host(x), tg.cpu().numpy(), tau)
        close(lse, rl, size=np.abs(host(x)).max() / tau)
        close(logp, rp, size=np.abs(host(x)).max() / tau)
        g = torch.randn(T, generator=torch.Generator().manual_seed(2)).cuda()
        if T > 3:
            g[3] = 0.0
        grad = sot.sot_token_logprob_grad(x, tg, lse, g, temperature=tau)
        close_grad(grad, *R.token_grad(host(x), tg.cpu().numpy(), tau, host(g)), dtype)


@pytest.mark.parametrize("dtype,T,V", BIG)
def test_widest_rows(sot, dtype, T, V):
    x, tg = rows(T, V, dtype, 1, seed=V), targets(T, V)
    logp, lse = sot.sot_token_logprob(x, tg)
    rp, rl = R.token_logprob(host(x), tg.cpu().numpy(), 1.0)
    close(logp, rp)
    close(lse, rl)
    adv, old = torch.ones(T).cuda(), logp.clone()
    loss, _, _, grad = sot.sot_policy_loss(x, tg, old, adv, weight=torch.ones(T).cuda())
    close_grad(grad, *R.token_grad(host(x), tg.cpu().numpy(), 1.0, -np.ones(T)), dtype)


def policy_inputs(T, V, dtype, pad, tau, seed):
    x, tg = rows(T, V, dtype, pad, seed), targets(T, V, seed + 1)
    rng = np.random.default_rng(seed)
    lp, _ = R.token_logprob(host(x), tg.cpu().numpy(), tau)
    # ratios away from the clip's two corners, on both sides of each
    ratio = rng.choice([0.5, 0.7, 0.9, 1.1, 1.4, 2.0], T) * rng.uniform(0.98, 1.02, T)
    f = lambda v: torch.from_numpy(np.asarray(v, np.float32)).cuda()  # noqa: E731
    w = rng.uniform(0.1, 1.0, T)
    w[rng.random(T) < 0.2] = 0.0
    return x, tg, f(lp - np.log(ratio)), f(rng.standard_normal(T)), f(lp + 0.3 * rng.standard_normal(T)), f(w)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,V", SIZES)
def test_policy_loss(sot, T, V, dtype):
    for pad, tau, kc in ((0, 1.0, 0.05), (5, 0.8, 0.0)):
        x, tg, old, adv, ref, w = policy_inputs(T, V, dtype, pad, tau, seed=V + T)
        if T > 4:
            tg[4] = -1
        ref = ref if kc else None
        loss, logp, kl, grad = sot.sot_policy_loss(x, tg, old, adv, ref_logp=ref, weight=w, temperature=tau, kl_coef=kc)
        rl, rp, rk, d = R.policy(host(x), tg.cpu().numpy(), host(old), host(adv), None if ref is None else host(ref),
                                 host(w), tau, 0.2, 0.2, kc)
        big = np.abs(host(x)).max() / tau
        close(logp, rp, size=big)
        close(kl, rk, scale=4.0)
        close(loss, rl, scale=8.0)
        rg, size = R.token_grad(host(x), tg.cpu().numpy(), tau, d)
        # d itself moves by (|A| r + kc e^u) times the error of logp: at most a few ATOL
        close_grad(grad, rg, size + 8.0, dtype)
        only, _, _, none = sot.sot_policy_loss(x, tg, old, adv, ref_logp=ref, weight=w, temperature=tau, kl_coef=kc,
                                               grad=False)
        assert none is None and torch.equal(only, loss)


def distill_inputs(T, V, K, dtype, pad, tail, seed):
    x = rows(T, V, dtype, pad, seed)
    rng = np.random.default_rng(seed)
    ids = np.stack([rng.permutation(V)[:K] if V >= K else np.concatenate([rng.permutation(V), -np.ones(K - V, int)])
                    for _ in range(T)])
    z = 2.0 * rng.standard_normal((T, K)) + 3.0
    if tail:
        z = z - np.log(np.exp(z).sum(1, keepdims=True)) + np.log(rng.uniform(0.5, 0.95, (T, 1)))
    ids[rng.random((T, K)) < 0.1] = -1
    if T > 2:
        ids[1] = -1      # no entry at all
        ids[2, 0] = V    # out of range
    if T > 3 and K > 1:
        z[3, 1] = -np.inf
    w = rng.uniform(0.5, 1.5, T)
    if T > 4:
        w[4] = 0.0
    return x, ids, z, w


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,V", SIZES)
@pytest.mark.parametrize("K", [1, 8, 100])
def test_distill_topk(sot, T, V, K, dtype):
    for tail, tau, pad, it, tt in ((False, 1.0, 0, torch.int32, "f32"), (False, 2.0, 3, torch.int64, "bf16"),
                                   (True, 1.0, 1, torch.int32, "f32"), (True, 1.0, 0, torch.int64, "f16")):
        x, ids, z, w = distill_inputs(T, V, K, dtype, pad, tail, seed=V + K)
        zt = torch.from_numpy(z.astype(np.float32)).to(TYPES[tt]).cuda()
        wt = torch.from_numpy(w.astype(np.float32)).cuda()
        loss, grad = sot.sot_distill_topk(x, torch.from_numpy(ids).to(it).cuda(), zt, weight=wt, temperature=tau, tail=tail)
        rl, rg, size = R.distill(host(x), ids, host(zt), host(wt), tau, tail)
        # the terms of a KL divergence are as large as the log-probabilities
        close(loss, rl, scale=4.0 * tau * tau, size=tau * tau * 64.0)
        close_grad(grad, rg, size, dtype)
        only, none = sot.sot_distill_topk(x, torch.from_numpy(ids).to(it).cuda(), zt, weight=wt, temperature=tau, tail=tail,
                                          grad=False)
        assert none is None and torch.equal(only, loss)


def test_distill_tail_of_a_confident_student(sot):
    """The student's mass outside the entries far below the rounding of its total."""
    T, V, K = 4, 5003, 6
    x = rows(T, V, "f32", 0, 7, spread=1.0)
    ids = np.stack([np.arange(K) * 11 + t for t in range(T)])
    lift = torch.tensor([10.0, 20.0, 40.0, 100.0])
    for t in range(T):
        x[t, torch.from_numpy(ids[t]).cuda()] += lift[t].item()
    z = np.log(np.full((T, K), 0.9 / K))
    zt = torch.from_numpy(z.astype(np.float32)).cuda()
    w = torch.ones(T).cuda()
    loss, grad = sot.sot_distill_topk(x, torch.from_numpy(ids).int().cuda(), zt, weight=w, tail=True)
    rl, rg, size = R.distill(host(x), ids, host(zt), host(w), 1.0, True)
    close(loss, rl, scale=4.0, size=200.0)
    close_grad(grad, rg, size, "f32")


def test_distill_entries_cover_the_vocabulary(sot):
    T, V = 3, 40
    x = rows(T, V, "f32", 0, 9)
    ids = np.stack([np.random.default_rng(t).permutation(V) for t in range(T)])
    z = R.log_softmax(np.random.default_rng(5).standard_normal((T, V)), 1.0)[0]
    zt = torch.from_numpy(z.astype(np.float32)).cuda()
    loss, grad = sot.sot_distill_topk(x, torch.from_numpy(ids).int().cuda(), zt, weight=torch.ones(T).cuda(), tail=True)
    rl, rg, size = R.distill(host(x), ids, host(zt), np.ones(T), 1.0, True)
    close(loss, rl, scale=4.0, size=16.0)
    close_grad(grad, rg, size, "f32")


def test_most_entries(sot):
    T, V, K = 2, 9001, 1024
    x, ids, z, w = distill_inputs(T, V, K, "bf16", 0, True, 3)
    zt, wt = torch.from_numpy(z.astype(np.float32)).cuda(), torch.from_numpy(w.astype(np.float32)).cuda()
    loss, grad = sot.sot_distill_topk(x, torch.from_numpy(ids).int().cuda(), zt, weight=wt, tail=True)
    rl, rg, size = R.distill(host(x), ids, host(zt), host(wt), 1.0, True)
    close(loss, rl, scale=4.0, size=64.0)
    close_grad(grad, rg, size, "bf16")


def test_weights_default_to_the_mean(sot):
    T, V = 6, 300
    x, tg, old, adv, ref, _ = policy_inputs(T, V, "f32", 0, 1.0, 4)
    mean = torch.full((T,), 1.0 / T).cuda()
    for a, b in zip(sot.sot_policy_loss(x, tg, old, adv, ref, None, kl_coef=0.1),
                    sot.sot_policy_loss(x, tg, old, adv, ref, mean, kl_coef=0.1)):
        assert torch.equal(a, b)
    ids, z = torch.arange(5, dtype=torch.int32).expand(T, 5).contiguous().cuda(), torch.randn(T, 5).cuda()
    for a, b in zip(sot.sot_distill_topk(x, ids, z), sot.sot_distill_topk(x, ids, z, weight=mean)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_masked_and_extreme_logits(sot, dtype):
    """Columns at -inf and at the type's lowest and largest values; rows of one value;
    rows left out that hold NaN."""
    V = 777
    x = rows(8, V, dtype, 0, 11)
    low, high = torch.finfo(TYPES[dtype]).min, torch.finfo(TYPES[dtype]).max
    x[0, 5:700] = float("-inf")
    x[1, 100:] = low
    x[2] = low                 # every column at the lowest value: uniform
    x[3] = 0.0
    x[4, :10] = high           # ten columns share the mass
    x[5] = float("nan")        # left out
    x[6, 1:] = float("-inf")   # a single column left
    tg = torch.tensor([2, 7, 500, 0, 3, 1, 0, 9]).cuda()
    w = torch.ones(8).cuda()
    w[5] = 0.0
    out = tg.clone()
    out[5] = -100
    logp, lse = sot.sot_token_logprob(x, out)
    xh = host(x)
    xh[5] = 0.0
    rp, rl = R.token_logprob(xh, out.cpu().numpy(), 1.0)
    big = np.abs(np.where(np.isfinite(xh), xh, 0)).max(1)
    close(logp, rp, size=np.maximum(np.abs(rp), 1.0))
    close(lse, rl, size=np.maximum(big, 1.0))
    adv = torch.ones(8).cuda()
    loss, _, _, grad = sot.sot_policy_loss(x, tg, logp, adv, weight=w)
    rg, size = R.token_grad(xh, tg.cpu().numpy(), 1.0, -host(w))
    close_grad(grad, rg, size, dtype)
    ids = torch.tensor([[0, 1, 2]] * 8, dtype=torch.int32).cuda()
    ids[6, 1:] = -1
    ids[1] = torch.tensor([50, 60, 70])
    z = torch.log(torch.tensor([[0.5, 0.2, 0.1]] * 8)).cuda()
    for tail in (False, True):
        loss, grad = sot.sot_distill_topk(x, ids, z, weight=w, tail=tail)
        rl, rg, size = R.distill(xh, ids.cpu().numpy(), host(z), host(w), 1.0, tail)
        close(loss, rl, scale=4.0, size=np.where(np.isfinite(rl), np.maximum(np.abs(rl), 128.0), 0))
        fine = np.isfinite(rg).all(1)
        close_grad(grad[torch.from_numpy(fine).cuda()], rg[fine], size[fine], dtype)


def test_a_target_at_minus_infinity(sot):
    x = rows(2, 50, "f32", 0, 3)
    x[0, 4] = float("-inf")
    logp, _ = sot.sot_token_logprob(x, torch.tensor([4, 4]).cuda())
    assert logp[0].item() == float("-inf") and np.isfinite(logp[1].item())
    ids = torch.tensor([[4, 5]] * 2, dtype=torch.int32).cuda()
    loss, _ = sot.sot_distill_topk(x, ids, torch.zeros(2, 2).cuda(), weight=torch.ones(2).cuda())
    assert loss[0].item() == float("inf") and np.isfinite(loss[1].item())


def test_rows_with_nothing_left_are_nan(sot):
    x = rows(2, 50, "bf16", 0, 3)
    x[0] = float("-inf")
    logp, lse = sot.sot_token_logprob(x, torch.tensor([4, 4]).cuda())
    assert np.isnan(logp[0].item()) and np.isfinite(logp[1].item())
    x[0] = 0.0
    x[0, 3] = float("nan")
    logp, lse = sot.sot_token_logprob(x, torch.tensor([4, 4]).cuda())
    assert np.isnan(logp[0].item()) and np.isnan(lse[0].item()) and np.isfinite(logp[1].item())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [1000, 4099, 50021])
def test_gradient_in_place_and_in_a_strided_array(sot, V, dtype):
    T = 5
    x, tg, old, adv, ref, w = policy_inputs(T, V, dtype, 0, 1.0, 21)
    args = dict(ref_logp=ref, weight=w, kl_coef=0.1)
    want = sot.sot_policy_loss(x, tg, old, adv, **args)[3]
    out = torch.full((T, V + 5), 7.0, dtype=x.dtype, device="cuda")
    got = sot.sot_policy_loss(x, tg, old, adv, grad=out[:, :V], **args)[3]
    assert torch.equal(got, want) and bool((out[:, V:] == 7.0).all())
    wide = torch.full((T, V + 3), 7.0, dtype=x.dtype, device="cuda")
    wide[:, :V] = x
    want = sot.sot_policy_loss(wide[:, :V], tg, old, adv, **args)[3]  # the same alignment: the same sums
    sot.sot_policy_loss(wide[:, :V], tg, old, adv, grad=wide[:, :V], **args)
    assert torch.equal(wide[:, :V], want) and bool((wide[:, V:] == 7.0).all())
    ids, z = torch.arange(9, dtype=torch.int32).expand(T, 9).contiguous().cuda(), torch.randn(T, 9).cuda()
    want = sot.sot_distill_topk(x, ids, z, weight=w)[1]
    y = x.clone()
    sot.sot_distill_topk(y, ids, z, weight=w, grad=y)
    assert torch.equal(y, want)
    logp, lse = sot.sot_token_logprob(x, tg)
    want = sot.sot_token_logprob_grad(x, tg, lse, adv)
    y = x.clone()
    sot.sot_token_logprob_grad(y, tg, lse, adv, grad=y)
    assert torch.equal(y, want)


def test_views_that_start_off_a_16_byte_boundary(sot):
    T, V = 4, 3001
    base = torch.randn(T * V + 16).to(torch.bfloat16).cuda()
    for shift in range(8):
        x = base[shift:shift + T * V].view(T, V)
        tg = targets(T, V)
        logp, lse = sot.sot_token_logprob(x, tg)
        rp, rl = R.token_logprob(host(x), tg.cpu().numpy(), 1.0)
        close(logp, rp)
        out = torch.full((T * V + 16,), 7.0, dtype=torch.bfloat16, device="cuda")
        g = out[3:3 + T * V].view(T, V)
        sot.sot_token_logprob_grad(x, tg, lse, torch.ones(T).cuda(), grad=g)
        close_grad(g, *R.token_grad(host(x), tg.cpu().numpy(), 1.0, np.ones(T)), "bf16")
        assert bool((out[:3] == 7.0).all()) and bool((out[3 + T * V:] == 7.0).all())


def test_row_offsets_beyond_32_bits(sot):
    T, V, ld = 5, 1000, (1 << 29) + 8
    store = torch.empty(4 * ld + V, dtype=torch.bfloat16, device="cuda")
    x = store.as_strided((T, V), (ld, 1))
    y = rows(T, V, "bf16", 0, 2)
    x.copy_(y)
    tg = targets(T, V)
    logp, lse = sot.sot_token_logprob(x, tg)
    rp, _ = R.token_logprob(host(y), tg.cpu().numpy(), 1.0)
    close(logp, rp)
    want = sot.sot_token_logprob_grad(y, tg, lse, torch.ones(T).cuda())
    sot.sot_token_logprob_grad(x, tg, lse, torch.ones(T).cuda(), grad=x)
    assert torch.equal(x, want)
    x.copy_(y)
    sot.sot_policy_loss(x, tg, logp, -torch.ones(T).cuda(), weight=torch.ones(T).cuda(), grad=x)
    close_grad(x, *R.token_grad(host(y), tg.cpu().numpy(), 1.0, np.ones(T)), "bf16")


def wide_reference(x, tg, tau, d):
    """Log-probabilities and their gradient in 64 bits for whole batches, on the GPU."""
    y = x.double() / tau
    lse = torch.logsumexp(y, 1)
    p = torch.exp(y - lse[:, None])
    logp = y.gather(1, tg[:, None])[:, 0] - lse
    grad, size = -p, p.clone()
    one = torch.ones_like(lse)[:, None]
    grad.scatter_add_(1, tg[:, None], one)
    size.scatter_add_(1, tg[:, None], one)
    return host(logp), host(lse), host(grad * (d / tau)[:, None]), host(size * (d.abs() / tau)[:, None])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,V", [(400, 1003), (400, 2040), (300, 4096), (200, 6001), (160, 17000), (170, 50021), (160, 107003),
                                 (100, 140001), (30, 300001), (60, 9000), (153, 30000)])
def test_every_way_of_cutting_rows(sot, T, V, dtype):
    """Batches on both sides of each choice: a warp, a CTA or a cluster a row, few rows and many."""
    x, tg = rows(T, V, dtype, 0, seed=V), targets(T, V)
    d = torch.randn(T, generator=torch.Generator().manual_seed(5)).double().cuda()
    rp, rl, rg, size = wide_reference(x, tg, 0.9, d)
    logp, lse = sot.sot_token_logprob(x, tg, temperature=0.9)
    close(logp, rp, size=np.abs(host(x)).max() / 0.9)
    close(lse, rl, size=np.abs(host(x)).max() / 0.9)
    # at old = logp the policy's gradient is -A w times the log-probability's
    loss, lp, _, grad = sot.sot_policy_loss(x, tg, logp, -torch.ones(T).cuda(), weight=d.float(), temperature=0.9)
    close(lp, rp, size=np.abs(host(x)).max() / 0.9)
    close_grad(grad, rg, size, dtype)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,V", [(3, 5003), (200, 5003), (200, 1500), (4, 40000)])
def test_sharp_and_offset_logits(sot, T, V, dtype):
    """Rows far from zero and rows whose logits span hundreds: the sums' first stabiliser does
    not serve them."""
    x, tg = rows(T, V, dtype, 0, seed=3, spread=1.0), targets(T, V)
    scale = torch.tensor([1.0, 60.0, 10.0, 1.0])[torch.arange(T) % 4].cuda()[:, None]
    shift = torch.tensor([300.0, 0.0, -200.0, -900.0])[torch.arange(T) % 4].cuda()[:, None]
    x.copy_((x.float() * scale + shift).to(x.dtype))
    d = torch.ones(T).double().cuda()
    rp, rl, rg, size = wide_reference(x, tg, 1.0, d)
    logp, lse = sot.sot_token_logprob(x, tg)
    close(lse, rl, size=np.abs(rl) + np.abs(rp))
    close(logp, rp, size=np.abs(rl) + np.abs(rp))
    grad = sot.sot_policy_loss(x, tg, logp, -torch.ones(T).cuda(), weight=torch.ones(T).cuda())[3]
    # a log-probability of size |rl| + |rp| moves by its rounding
    wide = 1.0 + 2.0 ** -8 * (np.abs(rl) + np.abs(rp))[:, None]
    close_grad(grad, rg, size * wide, dtype)


@pytest.mark.parametrize("T,V,K", [(5, 2000, 300), (200, 2000, 300), (200, 3000, 40), (160, 120001, 64), (2, 200000, 8)])
def test_tail_of_many_shapes(sot, T, V, K):
    x = rows(T, V, "f32", 0, 6)
    rng = np.random.default_rng(K)
    ids = np.stack([np.sort(rng.permutation(V)[:K]) for _ in range(T)])
    ids[:, 0] = 0
    ids[:, -1] = V - 1
    z = torch.log_softmax(torch.randn(T, K, generator=torch.Generator().manual_seed(1)), 1) - 0.2
    zt, w = z.cuda(), torch.ones(T).cuda()
    loss, grad = sot.sot_distill_topk(x, torch.from_numpy(ids).cuda(), zt, weight=w, tail=True)
    rl, rg, size = R.distill(host(x), ids, host(zt), host(w), 1.0, True)
    close(loss, rl, scale=4.0, size=64.0)
    close_grad(grad, rg, size, "f32")


def test_empty_batches(sot):
    x = torch.zeros(0, 10, device="cuda")
    tg = torch.zeros(0, dtype=torch.int64, device="cuda")
    z = torch.zeros(0, device="cuda")
    logp, lse = sot.sot_token_logprob(x, tg)
    assert logp.shape == (0,)
    assert sot.sot_policy_loss(x, tg, z, z)[3].shape == (0, 10)
    loss, margin, grad = sot.sot_preference_loss(torch.ones(3, device="cuda"), torch.zeros(1, dtype=torch.int64, device="cuda"))
    assert loss.shape == (0,) and bool((grad == 0).all())
    counts, loss, grad = sot.sot_balance_loss(x, torch.zeros(0, 2, dtype=torch.int32, device="cuda"))
    assert bool((counts == 0).all()) and bool((loss == 0).all())


def test_other_stream_and_repeated_runs(sot):
    T, V = 64, 20011
    x, tg, old, adv, ref, w = policy_inputs(T, V, "bf16", 0, 1.0, 31)
    want = sot.sot_policy_loss(x, tg, old, adv, ref, w, kl_coef=0.1)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    got = sot.sot_policy_loss(x, tg, old, adv, ref, w, kl_coef=0.1, stream=st)
    st.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    with torch.cuda.stream(st):
        again = sot.sot_policy_loss(x, tg, old, adv, ref, w, kl_coef=0.1)
    st.synchronize()
    for a, b in zip(want, again):
        assert torch.equal(a, b)
    r = rows(500, 60, "f32", 0, 5)
    ids = r.topk(4, 1).indices.int().contiguous()
    first = sot.sot_balance_loss(r, ids, z_coef=0.1)
    for a, b in zip(first, sot.sot_balance_loss(r, ids, z_coef=0.1)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("what", ["policy", "distill", "tail", "balance"])
def test_gradient_against_differences(sot, what):
    """Along the unit direction of the gradient the loss grows by |grad| per step; the
    five-point difference with step h is within h^4 / 30 of the loss's fifth derivative
    (at most a few times |grad| here: the losses are smooth on the scale of 1) and, with
    losses good to 2^-18, within 2^-17 / h."""
    T, V = 3, 41
    x = rows(T, V, "f32", 0, 13, spread=1.5)
    tg = targets(T, V)
    w = torch.ones(T).cuda()
    logp, _ = sot.sot_token_logprob(x, tg)
    old, ref = logp - 0.05, logp + 0.4
    adv = torch.tensor([1.0, -0.7, 0.4]).cuda()
    ids = torch.tensor([[1, 5, 9, 30], [0, 2, 40, 7], [3, 4, 8, -1]], dtype=torch.int32).cuda()
    z = torch.log(torch.tensor([[0.4, 0.2, 0.1, 0.1], [0.3, 0.1, 0.2, 0.05], [0.3, 0.3, 0.1, 0.9]])).cuda()

    def f(y, grad=False):
        if what == "policy":
            out = sot.sot_policy_loss(y, tg, old, adv, ref, w, kl_coef=0.3, clip_low=0.9, clip_high=5.0, grad=grad)
            return out[0].double().sum().item(), out[3]
        if what == "balance":
            out = sot.sot_balance_loss(y, ids, balance_coef=2.0, z_coef=0.1, grad=grad)
            return out[1].double().sum().item(), out[2]
        out = sot.sot_distill_topk(y, ids, z, weight=w, tail=what == "tail", grad=grad)
        return out[0].double().sum().item(), out[1]

    _, g = f(x, True)
    norm = g.double().norm().item()
    d = (g.double() / norm).float()
    h = 0.125
    at = {k: f(x + k * h * d)[0] for k in (-2, -1, 1, 2)}
    slope = (8 * (at[1] - at[-1]) - (at[2] - at[-2])) / (12 * h)
    assert abs(slope - norm) <= 4 * norm * h ** 4 + 2.0 ** -17 / h, (slope, norm)


@pytest.mark.parametrize("average", [False, True])
@pytest.mark.parametrize("with_ref", [False, True])
def test_preference_loss(sot, average, with_ref):
    rng = np.random.default_rng(3)
    lens = [0, 1, 1, 0, 5, 700, 33, 32, 257, 256]
    off = np.concatenate([[3], 3 + np.cumsum(lens)])  # tokens before and after belong to no pair
    T = off[-1] + 7
    logp, ref = -3 * rng.random(T), -3 * rng.random(T)
    logp[off[4]:off[5]] = -500.0  # a margin far out on the sigmoid
    tg = rng.integers(0, 100, T)
    tg[rng.random(T) < 0.2] = -100
    f = lambda v: torch.from_numpy(np.asarray(v, np.float32)).cuda()  # noqa: E731
    lp, rf = f(logp), f(ref) if with_ref else None
    for use in (None, tg):
        for ls, scale in ((0.0, None), (0.1, 2.0)):
            got = sot.sot_preference_loss(lp, torch.from_numpy(off).cuda(), ref_logp=rf,
                                          target=None if use is None else torch.from_numpy(use).cuda(), beta=0.3,
                                          label_smoothing=ls, average=average, scale=scale)
            want = R.preference(host(lp), None if rf is None else host(rf), use, off, 0.3, ls, average,
                                1 / 5 if scale is None else scale)
            for a, b in zip(got, want):  # sums in 64 bits: a few roundings of 32 bits at the end
                assert np.all(np.abs(host(a) - b) <= 2.0 ** -20 * np.abs(b) + 2.0 ** -22), np.abs(host(a) - b).max()


def test_preference_offsets_are_clamped(sot):
    lp = -torch.rand(20).cuda()
    for off in ([-5, 3, 40], [18, 5, 2], [30, 40, 50], [0, 1 << 40, 1 << 41]):
        loss, margin, grad = sot.sot_preference_loss(lp, torch.tensor(off).cuda())
        torch.cuda.synchronize()
        assert loss.shape == (1,) and grad.shape == (20,)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,E,K", [(1, 1, 1), (1, 8, 2), (3, 2, 2), (50, 7, 3), (257, 32, 4), (100, 33, 1), (64, 64, 8),
                                   (301, 100, 6), (97, 256, 8), (40, 500, 10), (1000, 60, 6), (17, 1024, 12)])
def test_balance_loss(sot, T, E, K, dtype):
    scale = 256.0 * T if dtype == "f16" else 1.0
    for pad, it, share in ((0, torch.int32, None), (3, torch.int64, 0.3), (8, torch.int32, 1.0)):
        x = rows(T, E, dtype, pad, seed=E, spread=1.5)
        if E > 4:
            x[:, 3] = float("-inf")  # an expert that is switched off
        ids = torch.stack([torch.randperm(E, generator=torch.Generator().manual_seed(t))[:K] for t in range(T)]).to(it)
        ids[::5, 0] = -1
        if T > 2:
            ids[2, 0] = E
        mask = None if share is None else torch.rand(T, generator=torch.Generator().manual_seed(1)) >= share
        cb, cz = 0.5 * scale, 0.01 * scale
        counts, loss, grad = sot.sot_balance_loss(x, ids.cuda(), mask=None if mask is None else mask.cuda(),
                                                  balance_coef=cb, z_coef=cz)
        rc, rl, rg, size = R.balance(host(x), ids.numpy(), None if mask is None else mask.numpy(), cb, cz)
        assert np.array_equal(counts.cpu().numpy(), rc)
        assert np.all(np.abs(host(loss) - rl) <= ATOL * np.maximum(np.abs(rl), scale * 0.01))
        close_grad(grad, rg, size, dtype)
        c2, l2, none = sot.sot_balance_loss(x, ids.cuda(), mask=None if mask is None else mask.cuda(), balance_coef=cb,
                                            z_coef=cz, grad=False)
        assert none is None and torch.equal(c2, counts) and torch.equal(l2, loss)


def test_balance_loss_many_tokens(sot):
    T, E, K = 30011, 128, 8
    x = rows(T, E, "bf16", 0, 3)
    ids = x.float().topk(K, 1).indices.int().contiguous()
    mask = torch.rand(T, generator=torch.Generator().manual_seed(1)).cuda() > 0.1
    counts, loss, grad = sot.sot_balance_loss(x, ids, mask=mask, balance_coef=float(T), z_coef=0.01)
    rc, rl, rg, size = R.balance(host(x), ids.cpu().numpy(), mask.cpu().numpy(), float(T), 0.01)
    assert np.array_equal(counts.cpu().numpy(), rc)
    assert np.all(np.abs(host(loss) - rl) <= ATOL * np.abs(rl))
    close_grad(grad, rg, size, "bf16")


def test_preference_from_logits_to_gradient(sot):
    """The chain a training step runs: log-probabilities, paired loss, gradient of the logits."""
    T, V = 90, 501
    x, tg = rows(T, V, "f32", 0, 17), targets(T, V)
    tg[:5] = -100
    off = torch.tensor([0, 20, 45, 60, 90]).cuda()
    ref, _ = R.token_logprob(host(x) * 0.9, tg.cpu().numpy(), 1.0)
    rf = torch.from_numpy(ref.astype(np.float32)).cuda()
    logp, lse = sot.sot_token_logprob(x, tg)
    loss, margin, d = sot.sot_preference_loss(logp, off, ref_logp=rf, target=tg, beta=0.2)
    grad = sot.sot_token_logprob_grad(x, tg, lse, d)
    rp, _ = R.token_logprob(host(x), tg.cpu().numpy(), 1.0)
    rl, rm, rd = R.preference(rp, host(rf), tg.cpu().numpy(), off.cpu().numpy(), 0.2, 0.0, False, 0.5)
    close(margin, rm, scale=45.0)
    close(loss, rl, scale=10.0)
    rg, size = R.token_grad(host(x), tg.cpu().numpy(), 1.0, rd)
    close_grad(grad, rg, size + 0.1, "f32")


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,E", [(40, 60), (40, 64), (3000, 60), (3000, 256), (1500, 520), (700, 1024)])
@pytest.mark.parametrize("empty", [True, False])
def test_balance_loss_of_offset_logits(sot, T, E, dtype, empty):
    """Neighbouring rows far from zero in different directions, so that their sums of
    exponentials leave the range of a float, and rows with few experts left.  Some rows have none
    left: they make the losses NaN and touch no other row's gradient, or (empty = False) are masked."""
    x = rows(T, E, dtype, 0, seed=E + T, spread=2.0)
    off = torch.tensor([0, 30, -30, 17, -45, 200, -200, 3000, -26, 16, -3000], dtype=x.dtype).cuda()
    x += off[torch.arange(T).cuda() % 11, None]
    x[3::7, 1:] = float("-inf")
    x[4::9, : E // 2] = float("-inf")
    ids = torch.stack([torch.randperm(E, generator=torch.Generator().manual_seed(t))[:2] for t in range(T)]).int()
    mask = torch.arange(T) % 13 != 5
    some = torch.isfinite(x).any(1).cpu()
    if not empty:
        mask &= some
    scale = 256.0 * T
    counts, loss, grad = sot.sot_balance_loss(x, ids.cuda(), mask=mask.cuda(), balance_coef=scale, z_coef=1e-5 * scale)
    with np.errstate(invalid="ignore"):
        rc, rl, rg, size = R.balance(host(x), ids.numpy(), mask.numpy(), scale, 1e-5 * scale)
    assert np.array_equal(counts.cpu().numpy(), rc)
    assert np.array_equal(np.isnan(host(loss)), np.isnan(rl))
    assert np.isnan(rl).any() == bool((mask & ~some).any())
    if not np.isnan(rl).any():
        assert np.all(np.abs(host(loss) - rl) <= ATOL * np.abs(rl))
    fine = (some | ~mask).numpy()
    close_grad(grad[torch.from_numpy(fine).cuda()], rg[fine], size[fine], dtype)


@pytest.mark.parametrize("V", [1384698, 1566394])
def test_tail_marks_near_the_default_shared_memory(sot, V):
    """Rows whose marks fill a CTA's shared memory to just below what needs no special leave."""
    T, K = 2, 8
    x = rows(T, V, "f32", 0, 3)
    rng = np.random.default_rng(V)
    ids = np.stack([np.sort(rng.permutation(V)[:K]) for _ in range(T)])
    z = torch.log_softmax(torch.randn(T, K, generator=torch.Generator().manual_seed(1)), 1) - 0.2
    zt, w = z.cuda(), torch.ones(T).cuda()
    loss, grad = sot.sot_distill_topk(x, torch.from_numpy(ids).cuda(), zt, weight=w, tail=True)
    rl, rg, size = R.distill(host(x), ids, host(zt), host(w), 1.0, True)
    close(loss, rl, scale=4.0, size=64.0)
    close_grad(grad, rg, size, "f32")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,V", [(3, 100), (200, 1000), (3, 5003), (200, 5003), (2, 60000)])
@pytest.mark.parametrize("level", [-10.0, -19.0, -26.0])
def test_small_probabilities_of_low_logits(sot, T, V, dtype, level):
    """Rows whose exponentials sum to as little as 2^-40: probabilities down to 2^-115 are still there."""
    g = torch.Generator().manual_seed(V)
    x = (level - 80.0 * torch.rand(T, V, generator=g)).to(TYPES[dtype]).cuda()
    x[:, 0] = level
    tg = torch.ones(T, dtype=torch.int64).cuda()
    ones, zero = torch.ones(T).cuda(), torch.zeros(T).cuda()
    lp, _ = R.token_logprob(host(x), tg.cpu().numpy(), 1.0)
    old = torch.from_numpy(lp.astype(np.float32)).cuda()
    _, _, _, grad = sot.sot_policy_loss(x, tg, old, ones, weight=ones)
    rg, size = R.token_grad(host(x), tg.cpu().numpy(), 1.0, -np.exp(lp - host(old)))
    close_grad(grad, rg, size, dtype)
    ids = torch.tensor([[5, 2, 70]] * T).cuda()
    z = torch.tensor([[-1.0, -2.0, -80.0]] * T).cuda()
    for tail in (False, True):
        _, grad = sot.sot_distill_topk(x, ids, z, weight=ones, tail=tail)
        _, rg, size = R.distill(host(x), ids.cpu().numpy(), host(z), host(ones), 1.0, tail)
        close_grad(grad, rg, size, dtype)
    if V <= 1000:
        ids = torch.zeros(T, 1, dtype=torch.int32)
        _, _, grad = sot.sot_balance_loss(x, ids.cuda(), balance_coef=1.0, z_coef=1.0)
        _, _, rg, size = R.balance(host(x), ids.numpy(), None, 1.0, 1.0)
        # (a balance row of sum 2^-10 loses what lies below 2^-116)
        close_grad(grad, rg, size + 2.0 ** -102, dtype)


def test_tail_of_masked_rows_is_nan(sot):
    """A row in use whose logits are all -inf gives NaN, with and without used entries."""
    for V in (1, 7, 700, 40000):
        x = torch.full((3, V), float("-inf")).cuda()
        ids = torch.tensor([[0], [-1], [V - 1]]).cuda()
        _, grad = sot.sot_distill_topk(x, ids, torch.full((3, 1), -0.5).cuda(), weight=torch.ones(3).cuda(), tail=True)
        assert torch.isnan(grad).all()


LEVELS = {"f32": [-1e4, -1e9, 3e9, -1e10, -1e20, 1e30, -1.7e38, -3.4028234663852886e38], "f16": [-65504.0, 3e4],
          "bf16": [-1e4, -1e9, -1e10, -1.7e38, -3.3895313892515355e38]}


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("V", [6, 100, 1000, 5003, 60000])
@pytest.mark.parametrize("tau", [1.0, 2.0, 0.7])
def test_rows_at_one_level(sot, V, dtype, tau):
    """Rows whose columns all hold one value however large, and rows where half of them are far below it."""
    levels = LEVELS[dtype]
    T = 2 * len(levels)
    x = torch.empty(T, V, dtype=TYPES[dtype])
    for i, c in enumerate(levels):
        x[2 * i:2 * i + 2] = c
        if c > -3e38 and dtype != "f16":
            x[2 * i + 1, V // 2:] = c * 1.5 if c < 0 else c / 1.5
    x = x.cuda()
    n = (x == x[:, :1]).sum(1).double().cpu().numpy()
    tg, ones = torch.ones(T, dtype=torch.int64).cuda(), torch.ones(T).cuda()
    p = np.where(host(x) == host(x)[:, :1], 1.0 / n[:, None], 0.0)
    lp = torch.from_numpy(-np.log(n).astype(np.float32)).cuda()

    logp, lse = sot.sot_token_logprob(x, tg, temperature=tau)
    close(logp, -np.log(n), scale=4.0)
    with np.errstate(over="ignore"):
        want = (host(x)[:, 0] / tau + np.log(n)).astype(np.float32).astype(np.float64)
    close(lse, want, size=2.0 * np.where(np.isfinite(want), np.abs(want), 0.0))
    # the gradient from the stored lse knows p to 2^-24 |lse| only, and stays below 1
    grad = host(sot.sot_token_logprob_grad(x, tg, lse, ones, temperature=tau))
    assert (np.abs(grad) * tau <= 1.0 + 2.0 ** -7).all()

    _, _, _, grad = sot.sot_policy_loss(x, tg, lp, ones, weight=ones, temperature=tau)
    ref = p.copy()
    ref[:, 1] -= 1.0
    close_grad(grad, ref / tau, (p + 1.0) / tau, dtype)
    ids, z = torch.tensor([[1, 4]] * T).cuda(), torch.tensor([[-1.0, -2.0]] * T).cuda()
    q = np.exp([-1.0, -2.0])
    loss, grad = sot.sot_distill_topk(x, ids, z, weight=ones, temperature=tau)
    qn = np.exp(np.array([-1.0, -2.0]) / tau) / np.exp(np.array([-1.0, -2.0]) / tau).sum()
    ref = tau * p
    ref[:, [1, 4]] -= tau * qn
    close_grad(grad, ref, tau * (p + 1.0), dtype)
    if tau == 1.0:
        loss, grad = sot.sot_distill_topk(x, ids, z, weight=ones, tail=True)
        rest = p.copy()
        rest[:, [1, 4]] = 0.0
        pr = rest.sum(1, keepdims=True)
        used = pr[:, 0] > 0  # the others' rest is one that does not show in 64 bits either
        ref = p - (1.0 - q.sum()) * rest / np.where(pr > 0, pr, 1.0)
        ref[:, [1, 4]] -= q
        close_grad(grad[torch.from_numpy(used).cuda()], ref[used], p[used] + 2.0, dtype)
        if V <= 1000 and dtype != "f16":
            cid = torch.zeros(T, 1, dtype=torch.int32)
            counts, _, grad = sot.sot_balance_loss(x, cid.cuda(), balance_coef=1.0)
            f = np.zeros(V)
            f[0] = V
            dot = p @ f
            close_grad(grad, p * (f - dot[:, None]) / T, p * (f + dot[:, None]) / T, dtype)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("V", [6, 100, 1000, 5003, 60000])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
@pytest.mark.parametrize("masked", [False, True])
def test_one_bad_logit_spoils_its_row(sot, V, dtype, bad, masked):
    T = 200
    x = rows(T, V, dtype, 3, seed=V)
    if masked:
        x[::2] = torch.finfo(x.dtype).min
    x[::2, V // 3] = bad
    tg, ones = torch.zeros(T, dtype=torch.int64).cuda(), torch.ones(T).cuda()
    spoilt = torch.arange(T).cuda() % 2 == 0
    logp, lse = sot.sot_token_logprob(x, tg)
    assert torch.equal(torch.isnan(logp), spoilt) and torch.equal(torch.isnan(lse), spoilt)
    loss, _, _, grad = sot.sot_policy_loss(x, tg, torch.nan_to_num(logp), ones, weight=ones)
    assert torch.equal(torch.isnan(loss), spoilt) and torch.equal(torch.isnan(grad).any(1), spoilt)
    ids, z = torch.tensor([[1, 4]] * T).cuda(), torch.tensor([[-1.0, -2.0]] * T).cuda()
    for tail in (False, True):
        loss, grad = sot.sot_distill_topk(x, ids, z, weight=ones, tail=tail)
        assert torch.equal(torch.isnan(loss), spoilt) and torch.equal(torch.isnan(grad).any(1), spoilt)
    if V <= 1000:
        _, _, grad = sot.sot_balance_loss(x, ids.int(), z_coef=1.0)
        assert torch.equal(torch.isnan(grad).any(1), spoilt)
