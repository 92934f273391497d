"""The language-model losses at their edges: values that are not finite, calls from several host threads, in captured
graphs, in place and under other default types.  Tolerances are those of test_gpu_lm_losses.py unless a test derives
its own; values that are not finite have to be the same ones."""
import threading

import numpy as np
import pytest

import lm_ref as R
from test_gpu_lm_losses import (ATOL, GTOL, RTOL, SIZES, TYPES, close_grad, host, policy_inputs, rows, sot,  # noqa: F401
                                targets)

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

INF, NAN = float("inf"), float("nan")


def f32(v):
    return torch.from_numpy(np.asarray(v, np.float32)).cuda()


def alike(got, ref, bound):
    """Within `bound` where the reference is finite, the same infinity or NaN where it is not."""
    got, ref = host(got), np.asarray(ref, np.float64)
    assert np.array_equal(np.isnan(got), np.isnan(ref)), (got, ref)
    ends = np.isinf(got) | np.isinf(ref)
    assert np.array_equal(got[ends], ref[ends]), (got, ref)
    ok = np.isfinite(ref)
    over = np.abs(got[ok] - ref[ok]) - np.broadcast_to(bound, ref.shape)[ok]
    assert over.size == 0 or over.max() <= 0, over.max()


@pytest.mark.parametrize("default", [torch.bfloat16, torch.float16, torch.float64])
def test_outputs_are_float32_under_any_default_type(sot, default):
    """torch's default type says nothing about the outputs: they are float32, and the same bits."""
    T, V = 700, 50
    x, tg, old, adv, ref, w = policy_inputs(T, V, "bf16", 0, 1.0, 3)
    ids = torch.arange(5, dtype=torch.int32).expand(T, 5).contiguous().cuda()
    z = torch.randn(T, 5, generator=torch.Generator().manual_seed(1)).cuda()
    off = torch.arange(0, T + 1, 2).cuda()
    off = off[:off.numel() // 2 * 2 - 1].contiguous()
    pts, eps = torch.rand(1, 40, 3, generator=torch.Generator().manual_seed(2)).cuda(), 0.1

    def calls():
        out = list(sot.sot_token_logprob(x, tg))
        out.append(sot.sot_token_logprob_grad(x, tg, out[1], adv))
        out += sot.sot_distill_topk(x, ids, z, weight=w)
        out += sot.sot_policy_loss(x, tg, old, adv, ref, w, kl_coef=0.1)
        out += sot.sot_preference_loss(out[0], off)
        out += sot.sot_balance_loss(x, ids, z_coef=0.1)
        f, g = sot.sot_potentials(pts, pts, eps=eps, iters=10)
        got = sot.sot_plan_coo_operands(pts, pts, None, None, f, g, eps)
        return out + [got[k] for k in ("xc", "lwx", "yc", "lwy", "Mr", "Mc")]
    want = calls()
    before = torch.get_default_dtype()
    torch.set_default_dtype(default)
    try:
        got = calls()
    finally:
        torch.set_default_dtype(before)
    for a, b in zip(got, want):
        assert a.dtype == b.dtype and torch.equal(a, b)


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("bad,tt", [(NAN, "f32"), (INF, "f32"), (NAN, "bf16"), (INF, "f16")])
@pytest.mark.parametrize("T,V,K", [(6, 50, 4), (200, 3000, 70), (6, 50021, 40), (200, 5003, 8)])
def test_a_bad_teacher_value_spoils_its_row(sot, T, V, K, bad, tt, tail):
    x = rows(T, V, "bf16", 0, V)
    rng = np.random.default_rng(V)
    ids = torch.from_numpy(np.stack([rng.permutation(V)[:K] for _ in range(T)])).cuda()
    z = torch.log_softmax(torch.randn(T, K, generator=torch.Generator().manual_seed(1)), 1).sub(0.3).to(TYPES[tt]).cuda()
    w = torch.ones(T).cuda()
    ids[1, 0] = -1  # unused: what it holds does not count
    w[2] = 0.0      # left out
    want = sot.sot_distill_topk(x, ids, z, weight=w, tail=tail)
    z[1, 0] = bad
    z[2, 1] = bad
    spoilt = torch.arange(T).cuda() % 3 == 0
    z[spoilt, torch.arange(T).cuda()[spoilt] % K] = bad
    loss, grad = sot.sot_distill_topk(x, ids, z, weight=w, tail=tail)
    only, _ = sot.sot_distill_topk(x, ids, z, weight=w, tail=tail, grad=False)
    for got in (loss, only):
        assert torch.isnan(got[spoilt]).all() and torch.equal(got[~spoilt], want[0][~spoilt])
    assert torch.isnan(grad[spoilt]).all() and torch.equal(grad[~spoilt], want[1][~spoilt])


@pytest.mark.parametrize("V", [60, 40000])
def test_a_bad_teacher_value_where_nothing_else_is_left(sot, V):
    """Every column outside the entries masked: the rest takes no part, the row's loss and gradient are NaN all the same."""
    x = torch.full((3, V), -INF).cuda()
    ids = torch.tensor([[3, 20, 41]] * 3).cuda()
    x[:, ids[0]] = 0.5
    z = torch.tensor([[-1.0, -2.0, -3.0], [-1.0, NAN, -3.0], [-1.0, -2.0, INF]]).cuda()
    for tail in (False, True):
        loss, grad = sot.sot_distill_topk(x, ids, z, weight=torch.ones(3).cuda(), tail=tail)
        assert torch.isfinite(loss[0]) and torch.isfinite(grad[0]).all()
        assert torch.isnan(loss[1:]).all() and torch.isnan(grad[1:]).all()


@pytest.mark.parametrize("average", [False, True])
@pytest.mark.parametrize("smoothing", [0.0, 0.1])
@pytest.mark.parametrize("at", [0, 31, 300, -1])
def test_preference_with_a_token_of_no_probability(sot, average, smoothing, at):
    """A log-probability of -inf leaves the losses and gradients that the definition gives."""
    rng = np.random.default_rng(5)
    lens = rng.integers(301, 700, 12)
    off = np.concatenate([[0], np.cumsum(lens)])
    T, P, beta, scale = off[-1], 6, 0.3, 0.5
    logp, ref = (-3 * rng.random(T)).astype(np.float32), (-3 * rng.random(T)).astype(np.float32)
    tg = rng.integers(0, 100, T)

    def put(a, seq, value):
        a[off[seq + 1] - 1 if at < 0 else off[seq] + at] = value
    put(logp, 3, -INF)   # pair 1: in the rejected answer
    put(logp, 4, -INF)   # pair 2: in the chosen one
    put(logp, 6, -INF)   # pair 3: in both
    put(logp, 7, -INF)
    put(logp, 8, -INF)   # pair 4: at a token that takes no part
    put(tg, 8, -100)
    put(ref, 10, -INF)   # pair 5: the reference model rules a chosen token out
    loss, margin, grad = sot.sot_preference_loss(f32(logp), torch.from_numpy(off).cuda(), ref_logp=f32(ref),
                                                 target=torch.from_numpy(tg).cuda(), beta=beta, label_smoothing=smoothing,
                                                 average=average, scale=scale)
    with np.errstate(all="ignore"):
        rl, rm, rd = R.preference(np.where(np.isinf(logp), 0.0, logp), np.where(np.isinf(ref), 0.0, ref), tg, off, beta,
                                  smoothing, average, scale)
    far = INF if smoothing else 0.0
    for p, m, l, sn in ((1, INF, far, 0.0), (2, -INF, INF, 1.0), (3, NAN, NAN, NAN), (5, INF, far, 0.0)):
        rm[p], rl[p] = m, l
        d = scale * beta * (smoothing * (1 - sn) - (1 - smoothing) * sn)
        for h, s in ((0, d), (1, -d)):
            i = np.arange(off[2 * p + h], off[2 * p + h + 1])
            i = i[tg[i] >= 0]
            rd[i] = s / (len(i) if average else 1)
    # sums in 64 bits: a few roundings of 32 bits at the end
    for got, want in ((loss, rl), (margin, rm), (grad, rd)):
        alike(got, want, 2.0 ** -20 * np.abs(want) + 2.0 ** -22)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,V,K", [(5, 3000, 33), (5, 3000, 64), (5, 3000, 256), (5, 50021, 33), (5, 50021, 256),
                                   (200, 5003, 64), (5, 9000, 1024)])
def test_an_entry_on_a_masked_column_in_any_place(sot, T, V, K, dtype):
    """A used entry whose column is masked makes the row's loss +inf wherever it stands, and the gradient
    stays what the definition gives."""
    x = rows(T, V, dtype, 0, V)
    rng = np.random.default_rng(K)
    ids = np.stack([rng.permutation(V)[:K] for _ in range(T)])
    place = [0, K // 2, K - 33, K - 1]  # row 4, 9, ... is whole
    for t in range(T):
        if t % 5 < 4:
            x[t, ids[t, place[t % 5]]] = -INF
    z = torch.log_softmax(torch.randn(T, K, generator=torch.Generator().manual_seed(1)), 1).sub(0.3).cuda()
    w = torch.ones(T).cuda()
    for tail in (False, True):
        loss, grad = sot.sot_distill_topk(x, torch.from_numpy(ids).cuda(), z, weight=w, tail=tail)
        rl, rg, size = R.distill(host(x), ids, host(z), host(w), 1.0, tail)
        assert np.array_equal(np.isinf(rl), np.arange(T) % 5 < 4)
        alike(loss, rl, 4.0 * ATOL + RTOL * 64.0)
        close_grad(grad, rg, size, dtype)


@pytest.mark.parametrize("T,V", [(4, 1000), (200, 5003), (4, 50021)])
def test_kl_term_far_from_the_reference(sot, T, V):
    """The KL term's gradient is kl_coef (1 - exp d) however negative d is, its value +inf where exp d leaves the
    range, and with kl_coef = 0 it takes no part."""
    x, tg = rows(T, V, "f32", 0, V), targets(T, V)
    lp, _ = R.token_logprob(host(x), tg.cpu().numpy(), 1.0)
    far = np.array([-1e4, -1e8, -INF, -60.0])[np.arange(T) % 4]
    ref = np.where(far > -100, lp + far, far).astype(np.float32)
    old, adv, w = f32(lp), f32(np.full(T, 0.5)), torch.ones(T).cuda()
    loss, logp, kl, grad = sot.sot_policy_loss(x, tg, old, adv, f32(ref), w, kl_coef=0.05)
    with np.errstate(all="ignore"):
        rl, _, rk, d = R.policy(host(x), tg.cpu().numpy(), host(old), host(adv), ref, np.ones(T), 1.0, 0.2, 0.2, 0.05)
    alike(kl, rk, 4.0 * ATOL + 2.0 * RTOL * np.abs(rk))
    alike(loss, rl, 8.0 * ATOL + 4.0 * RTOL * np.abs(rl))
    rg, size = R.token_grad(host(x), tg.cpu().numpy(), 1.0, d)
    # d = -A r + 0.05: both are as large as 10 times their sum at most, and r moves by the error of logp
    close_grad(grad, rg, 2.0 * size, "f32")
    above = f32(lp + 200.0)  # exp 200 is out of range
    assert torch.equal(sot.sot_policy_loss(x, tg, old, adv, above, w, kl_coef=0.05)[2], torch.full((T,), INF).cuda())
    want = sot.sot_policy_loss(x, tg, old, adv, None, w)
    for r in (f32(ref), above):
        got = sot.sot_policy_loss(x, tg, old, adv, r, w, kl_coef=0.0)
        for i in (0, 1, 3):
            assert torch.equal(got[i], want[i])


@pytest.mark.parametrize("V", [1000, 50021])
def test_kl_of_a_masked_token(sot, V):
    """The token's own probability is 0, the reference's is not: the estimate of the KL term is +inf."""
    x, tg = rows(2, V, "f32", 0, V), targets(2, V)
    x[0, tg[0]] = -INF
    lp = f32([-3.0, -4.0])
    loss, logp, kl, _ = sot.sot_policy_loss(x, tg, lp, torch.ones(2).cuda(), lp, torch.ones(2).cuda(), kl_coef=0.1, grad=False)
    assert logp[0].item() == -INF and kl[0].item() == INF and loss[0].item() == INF
    assert bool(torch.isfinite(torch.stack([loss, logp, kl])[:, 1]).all())


@pytest.mark.parametrize("T,V", [(4, 1000), (200, 5003), (4, 50021)])
def test_no_advantage_gives_no_policy_term(sot, T, V):
    """Advantage 0: the ratio does not count, also where it leaves the range of a float."""
    x, tg = rows(T, V, "f32", 0, V), targets(T, V)
    lp, _ = R.token_logprob(host(x), tg.cpu().numpy(), 1.0)
    old = f32(lp - np.array([0.1, 90.0, 200.0, -200.0])[np.arange(T) % 4])
    zero, w = torch.zeros(T).cuda(), torch.ones(T).cuda()
    loss, logp, _, grad = sot.sot_policy_loss(x, tg, old, zero, weight=w)
    assert bool((loss == 0).all()) and bool((grad == 0).all())
    ref = f32(lp + 0.2)
    loss, _, kl, grad = sot.sot_policy_loss(x, tg, old, zero, ref, w, kl_coef=0.5)
    rl, _, rk, d = R.policy(host(x), tg.cpu().numpy(), host(old), np.zeros(T), host(ref), np.ones(T), 1.0, 0.2, 0.2, 0.5)
    alike(loss, rl, 8.0 * ATOL)
    rg, size = R.token_grad(host(x), tg.cpu().numpy(), 1.0, d)
    # exp d - 1 with d near 0.2 moves by the error of logp, ATOL, times exp d: 2^-13.5 of its value
    close_grad(grad, rg, 4.0 * size, "f32")
    x[0, 0] = NAN
    loss, _, _, grad = sot.sot_policy_loss(x, tg, old, zero, weight=w)
    assert np.isnan(loss[0].item()) and torch.isnan(grad[0]).all() and bool((grad[1:] == 0).all())


def test_wide_tails_from_two_host_threads(sot):
    """Two threads whose rows need different amounts of the same kernel's shared memory.  (Straight through the C
    interface, so that the calls overlap; rows of weight 0, so that the GPU keeps up.)"""
    from sinkhorn_point_cloud_gb300 import binding
    lib, runs = binding.load(), 20000
    ids, z, w = torch.tensor([[1, 70, 500, 9000]]).cuda(), torch.full((1, 4), -2.0).cuda(), torch.zeros(1).cuda()
    refused = []

    def work(x, loss, st):
        V = x.shape[1]
        args = (x.data_ptr(), 1, V, V, binding.SOT_F32, 1.0, ids.data_ptr(), binding.SOT_I64, z.data_ptr(), binding.SOT_F32, 4,
                1, w.data_ptr(), loss.data_ptr(), None, 0, st.cuda_stream)
        for _ in range(runs):
            if lib.sot_distill_topk(*args):
                refused.append(lib.sot_last_error())
    arrays = [(torch.zeros(1, V).cuda(), torch.ones(1).cuda(), torch.cuda.Stream()) for V in (1500000, 3000000)]
    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=a) for a in arrays]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not refused, (len(refused), refused[0])
    assert all(loss.item() == 0.0 for _, loss, _ in arrays)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,E", [(40, 60), (40, 64), (3000, 60), (3000, 256)])
def test_z_loss_out_of_range(sot, T, E, dtype):
    """A row whose squared log-sum-exp leaves the range of a float makes the z loss +inf, and no loss at all where
    its coefficient is 0."""
    x = rows(T, E, dtype, 0, seed=E + T)
    x[T // 2] = 1e25
    x[T // 3] = -1e30
    ids = x.float().topk(2, 1).indices.int().contiguous()
    counts, loss, grad = sot.sot_balance_loss(x, ids, balance_coef=float(T), z_coef=0.0)
    rc, rl, rg, size = R.balance(host(x), ids.cpu().numpy(), None, float(T), 0.0)
    alike(loss, rl, ATOL * np.abs(rl))
    close_grad(grad, rg, size, dtype)
    loss = sot.sot_balance_loss(x, ids, balance_coef=float(T), z_coef=0.01)[1]
    alike(loss, [rl[0], INF], ATOL * np.abs(rl))
    x[1, 0] = NAN
    for cz in (0.0, 0.01):
        assert torch.isnan(sot.sot_balance_loss(x, ids, balance_coef=float(T), z_coef=cz)[1]).all()


@pytest.mark.parametrize("T,E", [(40, 60), (3000, 256)])
@pytest.mark.parametrize("bad", [NAN, INF, -INF])
def test_balance_losses_of_a_row_without_a_sum(sot, T, E, bad):
    x = rows(T, E, "f32", 0, seed=E)
    ids = x.topk(2, 1).indices.int().contiguous()
    if bad == -INF:
        x[1] = bad
    else:
        x[1, 5] = bad
    for cz in (0.0, 0.01):
        assert torch.isnan(sot.sot_balance_loss(x, ids, z_coef=cz)[1]).all()


def test_a_transposed_teacher_is_refused(sot):
    x, ids = rows(3, 50, "f32"), torch.arange(5).expand(3, 5).contiguous().cuda()
    with pytest.raises(ValueError, match="teacher"):
        sot.sot_distill_topk(x, ids, torch.zeros(5, 3).cuda())
    assert sot.sot_distill_topk(x, ids, torch.zeros(3, 5).cuda())[0].shape == (3,)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,V", SIZES)
def test_policy_gradient_of_every_column(sot, T, V, dtype):
    """Clipped, weighted and with a KL term.  The coefficient d of a row moves by w (|A| r + kc e^u) times the error of
    logp (ATOL and the logits' rounding) and the rounding of the exponentials (under 2^-20 of their value); at a column
    this counts with p_v + [v = target]."""
    for pad, tau, kc in ((0, 1.0, 0.05), (5, 0.8, 0.3)):
        x, tg, old, adv, ref, w = policy_inputs(T, V, dtype, pad, tau, seed=V + T)
        grad = sot.sot_policy_loss(x, tg, old, adv, ref_logp=ref, weight=w, temperature=tau, kl_coef=kc)[3]
        _, lp, _, d = R.policy(host(x), tg.cpu().numpy(), host(old), host(adv), host(ref), host(w), tau, 0.2, 0.2, kc)
        rg, size = R.token_grad(host(x), tg.cpu().numpy(), tau, d)
        terms = host(w) * (np.abs(host(adv)) * np.exp(lp - host(old)) + kc * np.exp(host(ref) - lp))
        _, unit = R.token_grad(host(x), tg.cpu().numpy(), tau, np.ones(T))
        moved = terms * (ATOL + RTOL * np.abs(host(x)).max() / tau + 2.0 ** -20)
        close_grad(grad, rg, size + unit * moved[:, None] / GTOL, dtype)


@pytest.mark.parametrize("off", [[-5, 3, 40], [18, 5, 2], [30, 40, 50], [0, 1 << 40, 1 << 41], [4, 4, 9, 90, -3]])
@pytest.mark.parametrize("average", [False, True])
def test_clamped_offsets_give_the_losses_of_what_is_left(sot, off, average):
    T = 20
    lp = -torch.rand(T, generator=torch.Generator().manual_seed(4)).cuda()
    loss, margin, grad = sot.sot_preference_loss(lp, torch.tensor(off).cuda(), beta=0.3, average=average)
    held = np.clip(np.array(off, np.float64), 0, T).astype(int)
    rl, rm, rd = R.preference(host(lp), None, None, held, 0.3, 0.0, average, 1.0 / (len(off) // 2))
    alike(loss, rl, 2.0 ** -20 * np.abs(rl) + 2.0 ** -22)
    alike(margin, rm, 2.0 ** -20 * np.abs(rm) + 2.0 ** -22)
    if np.all(np.diff(held) >= 0):
        alike(grad, rd, 2.0 ** -20 * np.abs(rd) + 2.0 ** -22)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,E,pad", [(40, 64, 0), (40, 60, 1), (300, 33, 0), (6000, 64, 0), (6000, 61, 3), (2000, 500, 0)])
def test_balance_gradient_in_place(sot, T, E, pad, dtype):
    x = rows(T, E + pad, dtype, 0, seed=E)
    x[T // 2] -= 300.0  # a row that is read twice
    v = x[:, :E]
    ids = v.float().topk(3, 1).indices.int().contiguous()
    mask = torch.rand(T, generator=torch.Generator().manual_seed(1)).cuda() > 0.2
    args = dict(mask=mask, balance_coef=float(T), z_coef=0.1)
    counts, loss, _ = sot.sot_balance_loss(v, ids, grad=False, **args)
    out = x.clone()[:, :E]  # the same strides and alignment
    sot.sot_balance_loss(v, ids, grad=out, **args)
    beside = x[:, E:].clone()
    c2, l2, g2 = sot.sot_balance_loss(v, ids, grad=v, **args)
    assert g2 is v and torch.equal(c2, counts) and torch.equal(l2, loss)
    assert torch.equal(v, out) and torch.equal(x[:, E:], beside)


def everything(sot, s):
    """One of each call on the tensors of `s`."""
    out = list(sot.sot_token_logprob(s["x"], s["tg"]))
    pref = sot.sot_preference_loss(out[0], s["off"], beta=0.3)
    out += [*pref, sot.sot_token_logprob_grad(s["x"], s["tg"], out[1], pref[2])]
    out += sot.sot_policy_loss(s["x"], s["tg"], s["old"], s["adv"], s["ref"], s["w"], kl_coef=0.1)
    for tail in (False, True):
        out += sot.sot_distill_topk(s["x"], s["ids"], s["z"], weight=s["w"], tail=tail)
    for r, c in ((s["r"], s["c"]), (s["r"][:50], s["c"][:50])):  # with scratch and without
        out += sot.sot_balance_loss(r, c, z_coef=0.1)
    return out


def some_inputs(seed, T=40, V=9001):
    x, tg, old, adv, ref, w = policy_inputs(T, V, "bf16", 0, 1.0, seed)
    g = torch.Generator().manual_seed(seed)
    r = rows(4000, 128, "bf16", 0, seed)
    return dict(x=x, tg=tg, old=old, adv=adv, ref=ref, w=w, off=torch.tensor([0, 9, 17, 30, 40]).cuda(),
                ids=torch.stack([torch.randperm(V, generator=g)[:20] for _ in range(T)]).cuda(),
                z=torch.log_softmax(torch.randn(T, 20, generator=g), 1).sub(0.2).cuda(), r=r,
                c=r.float().topk(4, 1).indices.int().contiguous())


def test_in_a_captured_graph(sot):
    s, t = some_inputs(1), some_inputs(2)
    want = [[o.clone() for o in everything(sot, v)] for v in (s, t)]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        everything(sot, s)
    torch.cuda.current_stream().wait_stream(st)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = everything(sot, s)
    for v, w in ((s, want[0]), (t, want[1]), (t, want[1])):
        for k in s:
            s[k].copy_(v[k])
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, w):
            assert torch.equal(a, b)


def test_from_two_host_threads(sot):
    inputs = [some_inputs(3), some_inputs(4)]
    want = [everything(sot, s) for s in inputs]
    torch.cuda.synchronize()
    wrong = []

    def work(s, w):
        try:
            st = torch.cuda.Stream()
            with torch.cuda.stream(st):
                for _ in range(30):
                    got = everything(sot, s)
                st.synchronize()
            if not all(torch.equal(a, b) for a, b in zip(got, w)):
                wrong.append("results differ")
        except Exception as e:  # noqa: BLE001
            wrong.append(e)
    threads = [threading.Thread(target=work, args=a) for a in zip(inputs, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong[0]


@pytest.mark.parametrize("T,V", [(400, 2040), (300, 4096), (200, 6001), (160, 107003), (160, 140001), (30, 300001), (60, 9000),
                                 (153, 30000)])
def test_losses_alone_are_the_same_bits(sot, T, V):
    """A loss does not depend on whether its gradient is asked for, whichever way the rows are cut."""
    x, tg, old, adv, ref, w = policy_inputs(T, V, "bf16", 0, 1.0, V)
    a = sot.sot_policy_loss(x, tg, old, adv, ref, w, kl_coef=0.1)
    b = sot.sot_policy_loss(x, tg, old, adv, ref, w, kl_coef=0.1, grad=False)
    for i in range(3):
        assert torch.equal(a[i], b[i])
    ids = (torch.arange(20) * (V // 20)).expand(T, 20).contiguous().cuda()
    z = torch.log_softmax(torch.randn(T, 20, generator=torch.Generator().manual_seed(1)), 1).sub(0.2).cuda()
    for tail in (False, True):
        loss = sot.sot_distill_topk(x, ids, z, weight=w, tail=tail)[0]
        assert torch.equal(loss, sot.sot_distill_topk(x, ids, z, weight=w, tail=tail, grad=False)[0])


def test_the_widest_tail(sot):
    """Marks that fill nearly all of the shared memory that a tail row may take."""
    V, K = 6300000, 4
    x = rows(1, V, "f32", 0, 3)
    ids = torch.tensor([[0, 70, 3000001, V - 1]])
    z, w = torch.log(torch.tensor([[0.3, 0.2, 0.1, 0.1]])).cuda(), torch.ones(1).cuda()
    loss, grad = sot.sot_distill_topk(x, ids.cuda(), z, weight=w, tail=True)
    rl, rg, size = R.distill(host(x), ids.numpy(), host(z), host(w), 1.0, True)
    alike(loss, rl, 4.0 * ATOL + RTOL * 64.0)
    close_grad(grad, rg, size, "f32")


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,V", [(12, 900), (12, 50021), (200, 5003)])
@pytest.mark.parametrize("tau", [1.0, 2.0, 0.75])
def test_policy_of_a_token_on_a_masked_column(sot, T, V, dtype, tau):
    """Tokens whose logit is a mask's finite value, with old and reference log-probabilities from sot_token_logprob: the
    ratio is exp of what their rounding left, and 1 beyond 2^24, where neighbouring floats lie 2 and more apart."""
    levels = {"f32": [-300.0, -1e4, -1e9, -1.7e38], "f16": [-300.0, -1e4, -65504.0, -32752.0],
              "bf16": [-300.0, -1e4, -1e9, -1.7e38]}[dtype]
    x, tg = rows(T, V, dtype, 0, V), targets(T, V)
    at = torch.arange(T).cuda()
    x[at, tg] = torch.tensor(levels, dtype=x.dtype).cuda()[at % 4]
    lp, _ = R.token_logprob(host(x), tg.cpu().numpy(), tau)
    logp, _ = sot.sot_token_logprob(x, tg, temperature=tau)
    alike(logp, lp, ATOL + RTOL * np.abs(lp))
    adv, w = f32(np.where(np.arange(T) % 3 == 0, -1.0, 0.5)), torch.ones(T).cuda()
    loss, again, kl, grad = sot.sot_policy_loss(x, tg, logp, adv, logp, w, temperature=tau, kl_coef=0.1)
    assert torch.equal(again, logp)
    u = np.where(np.abs(lp) < 2.0 ** 24, lp - host(logp), 0.0)
    alike(loss, -host(adv) * np.exp(u), 8.0 * ATOL)
    alike(kl, np.expm1(-u) + u, 4.0 * ATOL)
    rg, size = R.token_grad(host(x), tg.cpu().numpy(), tau, -host(adv) * np.exp(u) - 0.1 * np.expm1(-u))
    # the coefficient moves by (|A| + 0.1) times the error of u, ATOL: 0.3 GTOL of it
    close_grad(grad, rg, 2.0 * size, dtype)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,V", [(16, 100), (16, 60000), (200, 5003)])
@pytest.mark.parametrize("tau", [1.0, 2.0, 0.75])
def test_distillation_of_rows_far_from_zero(sot, T, V, dtype, tau):
    """A row's loss does not change with the level of its logits: all columns at one masked value, half of them far
    below it, or usual logits moved far away."""
    levels = {"f32": [-1e4, -1e9, -1.7e38, -3.4028234663852886e38], "f16": [-1e4, -32752.0, -65504.0, 3e4],
              "bf16": [-1e4, -1e9, -1.7e38, -3.3895313892515355e38]}[dtype]
    x = rows(T, V, dtype, 0, V)
    for t in range(T):
        c, kind = levels[t % 4], t // 4 % 4
        if kind == 0:
            x[t] = c
        elif kind == 1 and abs(c) < 3e4:
            x[t] = x[t] + c
        elif kind == 2:
            x[t] = c
            x[t, V // 2:] = -INF
        elif kind == 3 and abs(c) < 3e38 and dtype != "f16":
            x[t] = c
            x[t, V // 2:] = 1.25 * c
    g = torch.Generator().manual_seed(5)
    for K in (1, 8, 40):
        ids = torch.stack([torch.randperm(V // 2 - 1, generator=g)[:K] for _ in range(T)])
        z = torch.log_softmax(torch.randn(T, K, generator=g), 1).sub(0.3).cuda()
        w = torch.ones(T).cuda()
        for tail in ((False, True) if tau == 1.0 else (False,)):
            loss, _ = sot.sot_distill_topk(x, ids.cuda(), z, weight=w, temperature=tau, tail=tail)
            rl, _, _ = R.distill(host(x), ids.numpy(), host(z), host(w), tau, tail)
            # the terms of a KL divergence are as large as the log-probabilities, at most 64 here
            alike(loss, rl, 4.0 * tau * tau * (ATOL + RTOL * 64.0))
    # entries on the lower half: as large a loss as their distance, to the rounding of its terms
    ids = torch.full((T, 2), V - 1)
    ids[:, 0] = 3
    z = torch.log(torch.tensor([[0.4, 0.3]] * T)).cuda()
    for tail in ((False, True) if tau == 1.0 else (False,)):
        loss, _ = sot.sot_distill_topk(x, ids.cuda(), z, weight=torch.ones(T).cuda(), temperature=tau, tail=tail)
        rl, _, _ = R.distill(host(x), ids.numpy(), host(z), np.ones(T), tau, tail)
        far = np.abs(np.where(np.isfinite(rl), rl, 0.0))
        alike(loss, np.where(far < 3e37, rl, np.nan_to_num(host(loss))) if (far >= 3e37).any() else rl,
              4.0 * tau * tau * (ATOL + RTOL * 64.0) + 8.0 * RTOL * far)


def test_distillation_with_the_rest_at_the_lowest_value(sot):
    """The rest of the vocabulary masked with the type's lowest value: its log-probability is that value."""
    low = torch.finfo(torch.float32).min
    for V in (60, 40000):
        x = torch.full((1, V), low).cuda()
        x[0, :2] = 1.0
        z = torch.log(torch.tensor([[0.5, 0.375]])).cuda()
        loss, _ = sot.sot_distill_topk(x, torch.tensor([[0, 1]]).cuda(), z, weight=torch.ones(1).cuda(), tail=True)
        want = 0.125 * -float(low)  # everything else is far below its rounding
        assert abs(loss.item() - want) <= 2.0 ** -20 * want


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,E", [(600, 64), (600, 61), (6000, 64)])
def test_z_gradient_of_rows_at_the_lowest_value(sot, T, E, dtype):
    """The coefficient times the log-sum-exp is out of range, the gradient 1 / (N E) of it is not."""
    x = rows(T, E, dtype, 0, seed=E)
    x[::2] = torch.finfo(x.dtype).min
    ids = x.float().topk(2, 1).indices.int().contiguous()
    counts, loss, grad = sot.sot_balance_loss(x, ids, balance_coef=1.0, z_coef=300.0)
    rc, rl, rg, size = R.balance(host(x), ids.cpu().numpy(), None, 1.0, 300.0)
    assert np.abs(rg).max() < 3e38
    alike(loss, [rl[0], INF], ATOL * np.abs(rl))
    close_grad(grad, rg, size, dtype)
