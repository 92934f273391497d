"""The language-model training losses' workloads: what a pass through each operator is, and its plain form.

Operators: ``distill`` (a teacher's top logits), ``policy`` (clipped policy loss with a KL term), ``preference``
(paired log ratios, from logits to the gradient with respect to them), ``logprob`` (a token's log-probability) and
``balance`` (a router's balance loss with per-expert counts).  With ``own`` false, ``run`` computes the plain form in
elementary torch operations in 32 bits; with ``own`` true it calls the package's operators.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
MOST = 1 << 29  # logits in the largest case
#: Loss scale of a half-precision step: without it most gradients would fall below the type's smallest value.
F16_SCALE = 256.0


def listed():
    return [
        # a distillation micro-step on one short answer: launch latency counts
        dict(name="distill_small", op="distill", T=16, V=32000, K=8, dtype="bf16", tau=1.0, tail=False, grad=True, skip=0.0, pad=0),
        # the ordinary distillation step: a batch of 4096 tokens over a 128 Ki vocabulary, teacher's 64 best kept
        dict(name="distill_large", op="distill", T=4096, V=131072, K=64, dtype="bf16", tau=2.0, tail=False, grad=True, skip=0.0, pad=0),
        # full-precision distillation with the teacher's remaining mass as one more outcome, odd vocabulary, prompts left out
        dict(name="distill_tail_odd", op="distill", T=1001, V=50021, K=100, dtype="f32", tau=1.0, tail=True, grad=True, skip=0.25, pad=0),
        # a policy update on a handful of tokens
        dict(name="policy_small", op="policy", T=8, V=65536, dtype="bf16", tau=1.0, grad=True, skip=0.0, ref=True, pad=0),
        # a policy update on packed rollouts: a third of the tokens are prompts and take no part
        dict(name="policy_large", op="policy", T=8192, V=65536, dtype="bf16", tau=1.0, grad=True, skip=0.34, ref=True, pad=0),
        # half precision, odd vocabulary, sampling temperature, no reference model
        dict(name="policy_odd", op="policy", T=3001, V=50021, dtype="f16", tau=0.7, grad=True, skip=0.1, ref=False, pad=0),
        # two short pairs
        dict(name="preference_small", op="preference", P=2, L=24, V=32000, dtype="bf16", pad=0),
        # a preference batch of 16 pairs of answers of up to 512 tokens
        dict(name="preference_large", op="preference", P=16, L=512, V=32768, dtype="bf16", pad=0),
        # scoring one drafted token per sequence of a small serving batch
        dict(name="logprob_token", op="logprob", T=4, V=131072, dtype="bf16", tau=1.0, skip=0.0, pad=0),
        # scoring whole rollouts under the old or the reference model
        dict(name="logprob_large", op="logprob", T=16384, V=32000, dtype="bf16", tau=1.0, skip=0.0, pad=0),
        # a router's balance loss on a decoding-sized batch
        dict(name="balance_small", op="balance", T=256, E=64, K=4, dtype="f32", skip=0.0),
        # a router's balance loss on a training batch with padding tokens
        dict(name="balance_large", op="balance", T=65536, E=256, K=8, dtype="bf16", skip=0.1),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["distill", "policy", "preference", "logprob", "balance"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "balance":
        E = _log_int(rng, 4, 512)
        return dict(op=op, T=_log_int(rng, 16, 65536), E=E, K=rng.randint(1, min(E, 12)), dtype=dtype,
                    skip=rng.choice([0.0, 0.1, 0.5]))
    V = _log_int(rng, 1000, 131072)
    if rng.random() < 0.5:
        V += 8 - V % 8
    most = min(16384, MOST // (2 * V))
    pad = rng.choice([0, 0, 0, 64])
    if op == "preference":
        P = _log_int(rng, 1, 32)
        return dict(op=op, P=P, L=_log_int(rng, 8, max(9, min(1024, most // (4 * P)))), V=V, dtype=dtype, pad=pad)
    case = dict(op=op, T=_log_int(rng, 1, most), V=V, dtype=dtype, pad=pad, tau=rng.choice([1.0, 1.0, 0.7, 2.0]),
                skip=rng.choice([0.0, 0.0, 0.1, 0.5]))
    if op != "logprob":
        case["grad"] = rng.random() < 0.75
    if op == "policy":
        case["ref"] = rng.random() < 0.7
    if op == "distill":
        case.update(K=_log_int(rng, 1, 256), tail=rng.random() < 0.5)
        if case["tail"]:
            case["tau"] = 1.0
    return case


# ---- inputs ---------------------------------------------------------------------------------------------------------
def _skipped(T, share, g, dev):
    """A truth value for each token: exactly int(T share) of them are left out."""
    out = torch.zeros(T, dtype=torch.bool, device=dev)
    out[torch.randperm(T, generator=g, device=dev)[:int(T * share)]] = True
    return out


def _lengths(case):
    """Lengths of the 2 P sequences, from a quarter of L to L tokens in no order."""
    least = max(1, case["L"] // 4)
    return [least + 7919 * (j + 1) % (case["L"] - least + 1) for j in range(2 * case["P"])]


def _logits(T, V, pad, dtype, g, dev):
    """Logits of a language model's spread; `pad` more columns in memory than the vocabulary has."""
    full = torch.empty(T, V + pad, dtype=TYPES[dtype], device=dev)
    step = max(1, (1 << 26) // (V + pad))
    for a in range(0, T, step):
        full[a:a + step] = torch.randn(min(step, T - a), V + pad, generator=g, device=dev).mul_(2.0).to(full.dtype)
    return full[:, :V]


def _reference_logp(logits, target, tau):
    out = torch.empty(logits.shape[0], device=logits.device)
    step = max(1, (1 << 26) // logits.shape[1])
    for a in range(0, logits.shape[0], step):
        y = logits[a:a + step].float() / tau
        out[a:a + step] = y.gather(1, target[a:a + step, None])[:, 0] - torch.logsumexp(y, 1)
    return out


def prepare(case, seed):
    dev = torch.device("cuda" if torch.cuda.is_available() else "cpu")
    g = torch.Generator(device=dev).manual_seed(int(seed))
    op = case["op"]
    s = dict(case)
    rand = lambda *n: torch.rand(*n, generator=g, device=dev)  # noqa: E731
    randn = lambda *n: torch.randn(*n, generator=g, device=dev)  # noqa: E731
    if op == "balance":
        T, E, K = case["T"], case["E"], case["K"]
        # a router that prefers some experts, its choices taken from its own scores
        logits = (randn(T, E) + 0.7 * randn(1, E)).to(TYPES[case["dtype"]])
        s["logits"] = logits
        s["ids"] = logits.float().topk(K, dim=1).indices.to(torch.int32).contiguous()
        s["mask"] = ~_skipped(T, case["skip"], g, dev)
        s["scale"] = F16_SCALE * T if case["dtype"] == "f16" else 1.0
        return s
    V = case["V"]
    if op == "preference":
        P = case["P"]
        lens = _lengths(case)
        T = sum(lens)
        offsets = torch.tensor([0] + lens, device=dev).cumsum(0)
        s["offsets"] = offsets
        s["scale"] = F16_SCALE if case["dtype"] == "f16" else 1.0 / P
    else:
        T = case["T"]
    logits = _logits(T, V, case["pad"], case["dtype"], g, dev)
    if op == "distill":
        K = min(case["K"], V)
        # distinct entries in random order, and a student that leans towards them
        ids = (torch.arange(K, device=dev) * (V // K) + (rand(T, K) * (V // K)).long()).gather(1, rand(T, K).argsort(1))
        z = 2.5 * randn(T, K) + 6.0
        logits.scatter_(1, ids, (z + 1.5 * randn(T, K)).to(logits.dtype))
        if case["tail"]:
            rest = torch.log(rand(T, 1) * 0.3 + 0.02)
            z = z - torch.logsumexp(z, 1, keepdim=True) + torch.log1p(-rest.exp())
        if K > 2:
            ids = torch.where(rand(T, K) < 0.02, torch.full_like(ids, -1), ids)  # entries the teacher left empty
        s.update(logits=logits, ids=ids.to(torch.int32).contiguous(), teacher=z.contiguous())
        weight = torch.full((T,), F16_SCALE if case["dtype"] == "f16" else 1.0 / T, device=dev)
        s["weight"] = weight.masked_fill(_skipped(T, case["skip"], g, dev), 0.0)
        return s
    target = torch.randint(0, V, (T,), generator=g, device=dev)
    logits.scatter_(1, target[:, None], (6.0 + 2.5 * randn(T, 1)).to(logits.dtype))
    s.update(logits=logits, target=target)
    if op == "logprob":
        s["target"] = torch.where(_skipped(T, case["skip"], g, dev), torch.full_like(target, -100), target)
        return s
    logp = _reference_logp(logits, target, case.get("tau", 1.0))
    if op == "preference":
        s["ref_logp"] = logp + 0.15 * randn(T)
        return s
    s["old_logp"] = logp + 0.1 * randn(T)
    s["ref_logp"] = logp + 0.2 * randn(T) if case["ref"] else None
    s["advantage"] = randn(T)
    weight = torch.full((T,), F16_SCALE if case["dtype"] == "f16" else 1.0 / T, device=dev)
    s["weight"] = weight.masked_fill(_skipped(T, case["skip"], g, dev), 0.0)
    return s


# ---- the plain forms: elementary operations in 32 bits, rounded once at the end -----------------------------------------
def _scores(logits, tau):
    """(log-probabilities, log-sum-exp) of each row."""
    y = logits.float()
    if tau != 1.0:
        y = y / tau
    m = y.amax(1, keepdim=True)
    lse = m + torch.exp(y - m).sum(1, keepdim=True).log()
    return y - lse, lse[:, 0]


def _from_logp(logp, target, dlogp, tau, dtype):
    """The gradient with respect to the logits of something whose gradient with respect to each token's logp is dlogp."""
    grad = torch.exp(logp) * (-dlogp / tau)[:, None]
    grad.scatter_add_(1, target[:, None], (dlogp / tau)[:, None])
    return grad.to(dtype)


def _plain_distill(s):
    x, ids, z, w, tau = s["logits"], s["ids"].long(), s["teacher"].float(), s["weight"], s["tau"]
    used = ids >= 0
    at = ids.clamp(min=0)
    logp, _ = _scores(x, tau)
    lp = logp.gather(1, at)
    zero = torch.zeros_like(z)
    keep = (w != 0)[:, None]
    if s["tail"]:
        q = torch.where(used, torch.exp(z), zero)
        qr = (1.0 - q.sum(1)).clamp(min=0.0)
        inside = torch.zeros_like(logp, dtype=torch.bool)
        inside.scatter_(1, at, used)
        # an unused entry points at column 0: set again what a used entry may say of it
        inside[:, 0] = (used & (ids == 0)).any(1)
        log_pr = torch.where(inside, torch.full_like(logp, -math.inf), logp)
        top = log_pr.amax(1, keepdim=True)
        log_pr = (top + torch.exp(log_pr - top).sum(1, keepdim=True).log())[:, 0]
        loss = torch.where(used, q * (z - lp), zero).sum(1) + torch.where(qr > 0, qr * (qr.log() - log_pr), torch.zeros_like(qr))
        total = q.sum(1) + qr
        if s["grad"]:
            outer = total - torch.where(qr > 0, qr / torch.exp(log_pr), torch.zeros_like(qr))
            grad = torch.exp(logp) * torch.where(inside, total[:, None], outer[:, None])
    else:
        y = torch.where(used, z / tau, torch.full_like(z, -math.inf))
        m = y.amax(1, keepdim=True)
        e = torch.exp(y - m)
        lq = y - m - e.sum(1, keepdim=True).log()
        q = torch.exp(lq)
        loss = torch.where(used, q * (lq - lp), zero).sum(1) * (tau * tau)
        if s["grad"]:
            grad = torch.exp(logp)
    loss = torch.where(keep[:, 0], loss * w, torch.zeros_like(loss))
    if not s["grad"]:
        return {"loss": loss}
    grad.scatter_add_(1, at, torch.where(used, -q, zero))
    grad = torch.where(keep, grad * (w * tau)[:, None], torch.zeros_like(grad))
    return {"loss": loss, "grad": grad.to(x.dtype)}


def _plain_policy(s):
    x, target, w, tau = s["logits"], s["target"], s["weight"], s["tau"]
    all_logp, _ = _scores(x, tau)
    logp = all_logp.gather(1, target[:, None])[:, 0]
    keep, zero = w != 0, torch.zeros_like(logp)
    r = torch.exp(logp - s["old_logp"])
    a = s["advantage"]
    free, held = r * a, r.clamp(0.8, 1.2) * a
    loss = -torch.minimum(free, held)
    d = torch.where(free <= held, -a * r, zero)
    kl = zero
    if s["ref"]:
        u = s["ref_logp"] - logp
        kl = torch.expm1(u) - u
        loss = loss + 0.04 * kl
        d = d - 0.04 * torch.expm1(u)
    out = {"loss": torch.where(keep, w * loss, zero), "logp": torch.where(keep, logp, zero), "kl": torch.where(keep, kl, zero)}
    if s["grad"]:
        out["grad"] = _from_logp(all_logp, target, torch.where(keep, w * d, zero), tau, x.dtype)
    return out


def _plain_preference(s):
    x, target, off, P = s["logits"], s["target"], s["offsets"], s["P"]
    all_logp, _ = _scores(x, 1.0)
    logp = all_logp.gather(1, target[:, None])[:, 0]
    which = torch.searchsorted(off, torch.arange(x.shape[0], device=x.device), right=True) - 1
    sums = torch.zeros(2 * P, device=x.device).index_add_(0, which, logp - s["ref_logp"])
    h = sums[0::2] - sums[1::2]
    loss = torch.log1p(torch.exp(-(0.1 * h).abs())) + (-0.1 * h).clamp(min=0.0)
    d = -0.1 / (1.0 + torch.exp(0.1 * h)) * s["scale"]
    sign = 1.0 - 2.0 * (which % 2).float()
    return {"loss": loss, "margin": h, "logp": logp, "grad": _from_logp(all_logp, target, d[which // 2] * sign, 1.0, x.dtype)}


def _plain_logprob(s):
    x, target = s["logits"], s["target"]
    keep = target >= 0
    logp, lse = _scores(x, s["tau"])
    logp = logp.gather(1, target.clamp(min=0)[:, None])[:, 0]
    zero = torch.zeros_like(lse)
    return {"logp": torch.where(keep, logp, zero), "lse": torch.where(keep, lse, zero)}


def _plain_balance(s):
    x, ids, mask, E, K = s["logits"], s["ids"].long(), s["mask"], s["E"], s["K"]
    cb, cz = 0.01 * s["scale"], 0.001 * s["scale"]
    one = mask[:, None].expand_as(ids).to(torch.int32)
    counts = torch.zeros(E, dtype=torch.int32, device=x.device).index_add_(0, ids.reshape(-1), one.reshape(-1))
    N = mask.sum().float()
    y = x.float()
    m = y.amax(1, keepdim=True)
    e = torch.exp(y - m)
    total = e.sum(1, keepdim=True)
    p = e / total
    lse = m + total.log()
    f = counts.float() * E / (K * N)
    inner = (p * f).sum(1, keepdim=True)
    keep = mask[:, None]
    zero = torch.zeros_like(inner)
    loss = torch.stack([cb * torch.where(keep, inner, zero).sum() / N,
                        cz * torch.where(keep, lse * lse, zero).sum() / N])
    grad = p * (cb * (f - inner) + 2.0 * cz * lse) / N
    return {"counts": counts, "loss": loss, "grad": torch.where(keep, grad, torch.zeros_like(grad)).to(x.dtype)}


# ---- a pass ----------------------------------------------------------------------------------------------------------
def _own(s):
    import sinkhorn_point_cloud_gb300 as sot
    op = s["op"]
    if op == "distill":
        loss, grad = sot.sot_distill_topk(s["logits"], s["ids"], s["teacher"], weight=s["weight"], temperature=s["tau"],
                                          tail=s["tail"], grad=s["grad"])
        return {"loss": loss, "grad": grad} if s["grad"] else {"loss": loss}
    if op == "policy":
        loss, logp, kl, grad = sot.sot_policy_loss(s["logits"], s["target"], s["old_logp"], s["advantage"],
                                                   ref_logp=s["ref_logp"], weight=s["weight"], temperature=s["tau"],
                                                   clip_low=0.2, clip_high=0.2, kl_coef=0.04, grad=s["grad"])
        out = {"loss": loss, "logp": logp, "kl": kl}
        if s["grad"]:
            out["grad"] = grad
        return out
    if op == "preference":
        logp, lse = sot.sot_token_logprob(s["logits"], s["target"])
        loss, margin, dlogp = sot.sot_preference_loss(logp, s["offsets"], ref_logp=s["ref_logp"], beta=0.1, scale=s["scale"])
        grad = sot.sot_token_logprob_grad(s["logits"], s["target"], lse, dlogp)
        return {"loss": loss, "margin": margin, "logp": logp, "grad": grad}
    if op == "logprob":
        logp, lse = sot.sot_token_logprob(s["logits"], s["target"], temperature=s["tau"])
        return {"logp": logp, "lse": lse}
    counts, loss, grad = sot.sot_balance_loss(s["logits"], s["ids"], mask=s["mask"], balance_coef=0.01 * s["scale"],
                                              z_coef=0.001 * s["scale"])
    return {"counts": counts, "loss": loss, "grad": grad}


_PLAIN = {"distill": _plain_distill, "policy": _plain_policy, "preference": _plain_preference, "logprob": _plain_logprob,
          "balance": _plain_balance}


def run(state):
    return _own(state) if own else _PLAIN[state["op"]](state)


def work(case):
    """Each input read once, each output written once; rows that take no part are not read."""
    op, size = case["op"], SIZE[case["dtype"]]
    if op == "balance":
        T, E, K = case["T"], case["E"], case["K"]
        n = T - int(T * case["skip"])
        return {"bytes": n * E * size + T * E * size + n * K * 4 + T + E * 4, "flops": 10 * n * E}
    V = case["V"]
    if op == "preference":
        T = sum(_lengths(case))
        return {"bytes": 2 * T * V * size + T * 20, "flops": 8 * T * V}
    T = case["T"]
    n = T - int(T * case["skip"])
    if op == "logprob":
        return {"bytes": n * V * size + T * 16, "flops": 4 * n * V}
    rows = T * 24 if op == "policy" else T * (8 * min(case["K"], V) + 8)
    return {"bytes": n * V * size + (T * V * size if case["grad"] else 0) + rows, "flops": (8 if case["grad"] else 4) * n * V}


# ---- 64 bits, from the definitions ------------------------------------------------------------------------------------
def _rows64(s, fn, keys):
    """fn on slices of rows in 64 bits, joined."""
    T, V = s["logits"].shape
    step = max(1, (1 << 25) // V)
    parts = [fn(slice(a, min(T, a + step))) for a in range(0, T, step)]
    return {k: torch.cat([p[k] for p in parts]) for k in keys}


def exact(case, seed):
    s = prepare(case, seed)
    op, d = case["op"], torch.float64
    if op == "balance":
        x, ids, mask, E, K = s["logits"].to(d), s["ids"].long(), s["mask"], s["E"], s["K"]
        cb, cz = 0.01 * s["scale"], 0.001 * s["scale"]
        N = int(mask.sum())
        chosen = torch.zeros(x.shape, dtype=d, device=x.device).scatter_(1, ids, 1.0) * mask[:, None]
        counts = chosen.sum(0)
        lse = torch.logsumexp(x, 1)
        p = torch.softmax(x, 1) * mask[:, None]
        f = counts * E / (K * N)
        dot = p @ f
        loss = torch.stack([cb * dot.sum() / N, cz * (lse ** 2 * mask).sum() / N])
        grad = (cb * (p * f - p * dot[:, None]) + 2.0 * cz * p * lse[:, None]) / N
        return {"counts": counts.to(torch.int32), "loss": loss, "grad": grad}
    tau = float(case.get("tau", 1.0))
    if op == "distill":
        def part(r):
            ls = torch.log_softmax(s["logits"][r].to(d) / tau, 1)
            ids, z, w = s["ids"][r].long(), s["teacher"][r].to(d), s["weight"][r].to(d)
            n, V = ls.shape
            wide = torch.zeros(n, V + 1, dtype=d, device=ls.device)  # the last column takes the unused entries
            at = torch.where(ids < 0, torch.full_like(ids, V), ids)
            if case["tail"]:
                q = z.exp()
            else:
                q = torch.softmax((z / tau).masked_fill(ids < 0, -math.inf), 1)
            q = wide.scatter(1, at, q)[:, :V]
            listed_ = wide.scatter(1, at, 1.0)[:, :V] > 0
            loss = torch.special.xlogy(q, q).sum(1) - (q * ls).sum(1)
            total = q.sum(1, keepdim=True)
            grad = ls.exp() * total - q
            if case["tail"]:
                qr = (1.0 - total).clamp(min=0.0)
                log_pr = torch.logsumexp(ls.masked_fill(listed_, -math.inf), 1, keepdim=True)
                loss = loss + (torch.special.xlogy(qr, qr) - torch.where(qr > 0, qr * log_pr, qr))[:, 0]
                share = torch.where(qr > 0, qr * (ls - log_pr).exp(), torch.zeros_like(ls))
                grad = grad + qr * ls.exp() - share.masked_fill(listed_, 0.0)
            out = {"loss": w * tau * tau * loss}
            if case["grad"]:
                out["grad"] = grad * (w * tau)[:, None]
            return out
        return _rows64(s, part, ["loss", "grad"] if case["grad"] else ["loss"])

    def logprob(r):
        y = s["logits"][r].to(d) / tau
        return {"lse": torch.logsumexp(y, 1), "logp": y.gather(1, s["target"][r].clamp(min=0)[:, None])[:, 0] - torch.logsumexp(y, 1)}
    got = _rows64(s, logprob, ["logp", "lse"])
    logp = got["logp"]
    if op == "logprob":
        keep = s["target"] >= 0
        return {"logp": logp * keep, "lse": got["lse"] * keep}

    def gradient(dlogp):
        def part(r):
            p = torch.softmax(s["logits"][r].to(d) / tau, 1)
            hot = torch.zeros_like(p).scatter_(1, s["target"][r][:, None], 1.0)
            return {"grad": (hot - p) * (dlogp[r] / tau)[:, None]}
        return _rows64(s, part, ["grad"])["grad"]
    if op == "preference":
        P, off = case["P"], s["offsets"].tolist()
        ratio = logp - s["ref_logp"].to(d)
        sums = torch.stack([ratio[a:b].sum() for a, b in zip(off[:-1], off[1:])])
        h = sums[0::2] - sums[1::2]
        per = -0.1 * torch.sigmoid(-0.1 * h) * s["scale"]
        dlogp = torch.cat([(per[j // 2] * (1 - 2 * (j % 2))).expand(off[j + 1] - off[j]) for j in range(2 * P)])
        return {"loss": -torch.nn.functional.logsigmoid(0.1 * h), "margin": h, "logp": logp, "grad": gradient(dlogp)}
    w, a = s["weight"].to(d), s["advantage"].to(d)
    keep = (w != 0).to(d)
    r = (logp - s["old_logp"].to(d)).exp()
    clipped = ((r > 1.2) & (a > 0)) | ((r < 0.8) & (a < 0))
    loss = torch.where(clipped, -r.clamp(0.8, 1.2) * a, -r * a)
    dlogp = torch.where(clipped, torch.zeros_like(r), -r * a)
    kl = torch.zeros_like(r)
    if case["ref"]:
        u = s["ref_logp"].to(d) - logp
        kl = torch.expm1(u) - u
        loss, dlogp = loss + 0.04 * kl, dlogp + 0.04 * (1 - u.exp())
    out = {"loss": w * loss, "logp": logp * keep, "kl": kl * keep}
    if case["grad"]:
        out["grad"] = gradient(w * dlogp)
    return out
