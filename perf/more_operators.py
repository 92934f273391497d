"""The language-model operators around the losses: what a pass through each is, and its plain form.

Operators: ``topk`` (log-probabilities of given tokens with entropies and the best alternatives), ``topk_grad`` (its
gradient), ``embed`` (embedding lookup with scaling), ``embed_grad`` (its gradient) and ``routed`` (a routed layer, from
the router to the joined experts, for a few tokens).  With ``own`` false, ``run`` computes the plain form in elementary
torch operations in 32 bits (the router's scores, which decide between neighbours, in 64); with ``own`` true it calls
the package's operators.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
MOST = 1 << 29  # logits in the largest case
ROWS = 1 << 29  # elements of the largest embedding table
WEIGHTS = 128 * 3 * 1408 * 4096  # experts' weights of the largest routed layer
#: Loss scale of a half-precision step: without it most gradients would fall below the type's smallest value.
F16_SCALE = 256.0


def listed():
    return [
        # one decoding step of four sequences: the sampled tokens' scores with their twenty best alternatives
        dict(name="topk_token", op="topk", T=4, V=131072, K=20, dtype="bf16", tau=1.0, skip=0.0, pad=0),
        # a teacher's 64 best entries over 4096 tokens of text, kept for a distillation
        dict(name="topk_teacher", op="topk", T=4096, V=131072, K=64, dtype="bf16", tau=1.0, skip=0.0, pad=0),
        # rollouts scored in half precision at a sampling temperature, odd vocabulary, a few alternatives, prompts left out
        dict(name="topk_odd", op="topk", T=3001, V=50021, K=5, dtype="f16", tau=0.7, skip=0.25, pad=64),
        # the gradient of scores, entropies and alternatives of a handful of tokens
        dict(name="topk_grad_small", op="topk_grad", T=8, V=65536, K=8, dtype="bf16", tau=1.0, skip=0.0, pad=0),
        # an entropy bonus beside a policy's log-probabilities on packed rollouts, a third of the tokens are prompts
        dict(name="topk_grad_large", op="topk_grad", T=8192, V=65536, K=0, dtype="bf16", tau=1.0, skip=0.34, pad=0),
        # the next tokens of four sequences
        dict(name="embed_token", op="embed", T=4, V=131072, D=4096, dtype="bf16", out="bf16", distinct=1.0, skip=0.0),
        # a packed training batch, full-precision table, activations in 16 bits, padding tokens left at zero
        dict(name="embed_large", op="embed", T=32768, V=131072, D=4096, dtype="f32", out="bf16", distinct=0.3, skip=0.05),
        # the whole table's gradient of a training batch with the frequent tokens of text
        dict(name="embed_grad_large", op="embed_grad", T=16384, V=131072, D=4096, dtype="bf16", out="bf16", distinct=0.3,
             skip=0.05),
        # a full-precision gradient of a long batch over a smaller table, odd sizes
        dict(name="embed_grad_odd", op="embed_grad", T=65001, V=32003, D=1001, dtype="f32", out="f32", distinct=0.15,
             skip=0.1),
        # one token of one sequence through a layer of 64 experts
        dict(name="routed_token", op="routed", T=1, H=2048, E=64, F=1024, K=8, dtype="bf16", renorm=True, bias=False),
        # a decoding batch that reaches nearly all of 128 experts
        dict(name="routed_batch", op="routed", T=64, H=4096, E=128, F=1408, K=8, dtype="bf16", renorm=True, bias=True),
        # few wide experts, sizes that end inside every tile, half precision
        dict(name="routed_odd", op="routed", T=37, H=1160, E=10, F=1736, K=2, dtype="f16", renorm=False, bias=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["topk", "topk_grad", "embed", "embed_grad", "routed"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "routed":
        case = dict(op=op, T=_log_int(rng, 1, 128), H=8 * _log_int(rng, 32, 512), F=8 * _log_int(rng, 16, 256),
                    E=_log_int(rng, 4, 256), dtype=rng.choice(["bf16", "bf16", "f16"]), renorm=rng.random() < 0.5,
                    bias=rng.random() < 0.5)
        case["E"] = min(case["E"], WEIGHTS // (3 * case["F"] * case["H"]))
        case["K"] = rng.randint(1, min(8, case["E"]))
        return case
    if op in ("embed", "embed_grad"):
        D = _log_int(rng, 64, 4096)
        if rng.random() < 0.7:
            D += 8 - D % 8
        D = min(D, 4096)
        most = min(131072, ROWS // D)
        case = dict(op=op, T=_log_int(rng, 1, min(32768, most)), V=_log_int(rng, 1000, most), D=D, dtype=dtype,
                    out=rng.choice([dtype, dtype, "f32"]), distinct=rng.choice([0.1, 0.3, 0.6, 1.0]),
                    skip=rng.choice([0.0, 0.0, 0.1]))
        if SIZE[case["out"]] == 4 or SIZE[dtype] == 4:  # no larger in bytes than in 16 bits
            case["V"], case["T"] = max(1000, case["V"] // 2), max(1, case["T"] // 2)
        return case
    V = _log_int(rng, 1000, 131072)
    if rng.random() < 0.5:
        V = min(131072, V + 8 - V % 8)
    most = min(16384, MOST // (2 * V))
    if op == "topk_grad":
        K = rng.choice([0, 0, _log_int(rng, 1, 64)])
    else:
        K = _log_int(rng, 1, 256)
    return dict(op=op, T=_log_int(rng, 1, most), V=V, K=K, dtype=dtype, tau=rng.choice([1.0, 1.0, 0.7, 2.0]),
                skip=rng.choice([0.0, 0.0, 0.1, 0.5]), pad=rng.choice([0, 0, 0, 64]))


# ---- inputs ---------------------------------------------------------------------------------------------------------
def _skipped(T, share, g, dev):
    """A truth value for each token: exactly int(T share) of them are left out."""
    out = torch.zeros(T, dtype=torch.bool, device=dev)
    out[torch.randperm(T, generator=g, device=dev)[:int(T * share)]] = True
    return out


def _normal(shape, scale, dtype, g, dev):
    """Normal numbers of a type, made a slice at a time."""
    full = torch.empty(shape, dtype=TYPES[dtype], device=dev)
    flat = full.view(-1)
    for a in range(0, flat.numel(), 1 << 26):
        n = min(1 << 26, flat.numel() - a)
        flat[a:a + n] = torch.randn(n, generator=g, device=dev).mul_(scale).to(full.dtype)
    return full


def _distinct(case):
    """Tokens in use and how many different rows they name."""
    n = case["T"] - int(case["T"] * case["skip"])
    return n, min(case["V"], max(1, int(n * case["distinct"])))


def _tokens(case, g, dev):
    """Token ids in no order: every one of the distinct rows at least once, the rest by a text's frequencies (the r-th
    most frequent token about as often as 1 / r); padding is negative."""
    n, k = _distinct(case)
    rows = torch.randperm(case["V"], generator=g, device=dev)[:k]
    rank = torch.exp(torch.rand(n, generator=g, device=dev) * math.log(k + 1.0)).long().clamp(1, k) - 1
    rank[:k] = torch.arange(k, device=dev)
    ids = torch.full((case["T"],), -1, dtype=torch.int64, device=dev)
    ids[~_skipped(case["T"], case["skip"], g, dev)] = rows[rank[torch.randperm(n, generator=g, device=dev)]]
    return ids


def prepare(case, seed):
    dev = torch.device("cuda" if torch.cuda.is_available() else "cpu")
    g = torch.Generator(device=dev).manual_seed(int(seed))
    op = case["op"]
    s = dict(case)
    if op == "routed":
        T, H, E, F, dtype = case["T"], case["H"], case["E"], case["F"], case["dtype"]
        s["x"] = _normal((T, H), 1.0, dtype, g, dev)
        s["router"] = _normal((E, H), H ** -0.5, dtype, g, dev)
        s["gate_up"] = _normal((E, 2 * F, H), H ** -0.5, dtype, g, dev)
        s["down"] = _normal((E, H, F), F ** -0.5, dtype, g, dev)
        s["lean"] = 0.3 * torch.randn(E, generator=g, device=dev) if case["bias"] else None
        return s
    if op in ("embed", "embed_grad"):
        s["ids"] = _tokens(case, g, dev)
        s["scale"] = math.sqrt(case["D"])
        if op == "embed":
            s["table"] = _normal((case["V"], case["D"]), case["D"] ** -0.5, case["dtype"], g, dev)
        else:
            size = F16_SCALE * 1e-3 if case["dtype"] == "f16" else 1e-3
            s["grad_out"] = _normal((case["T"], case["D"]), size, case["dtype"], g, dev)
        return s
    T, V, K, pad = case["T"], case["V"], min(case["K"], case["V"]), case["pad"]
    logits = _normal((T, V + pad), 2.0, case["dtype"], g, dev)[:, :V]
    target = torch.randint(0, V, (T,), generator=g, device=dev)
    logits.scatter_(1, target[:, None], (6.0 + 2.5 * torch.randn(T, 1, generator=g, device=dev)).to(logits.dtype))
    s.update(logits=logits, target=torch.where(_skipped(T, case["skip"], g, dev), torch.full_like(target, -100), target))
    if op == "topk":
        return s
    # a backward pass: what the forward one kept, and the gradients that come in
    _, lse, entropy, ids, _ = _plain_scores(logits, s["target"], K, case["tau"])
    scale = F16_SCALE if case["dtype"] == "f16" else 1.0 / T
    s.update(lse=lse, entropy=entropy, ids=ids, grad_logp=scale * torch.randn(T, generator=g, device=dev),
             grad_entropy=-0.1 * scale * torch.rand(T, generator=g, device=dev),
             grad_top=scale / max(K, 1) * torch.randn(T, K, generator=g, device=dev))
    return s


# ---- the plain forms: elementary operations in 32 bits, rounded once at the end -----------------------------------------
def _plain_scores(logits, target, K, tau):
    """(logp, lse, entropy, ids, top) a slice of rows at a time."""
    T, V = logits.shape
    step = max(1, (1 << 27) // V)
    parts = []
    for a in range(0, T, step):
        x, t = logits[a:a + step].float(), target[a:a + step]
        keep = t >= 0
        y = x / tau if tau != 1.0 else x
        m = y.amax(1, keepdim=True)
        e = torch.exp(y - m)
        total = e.sum(1, keepdim=True)
        lse = m + total.log()
        zero = torch.zeros_like(lse[:, 0])
        entropy = total.log()[:, 0] - (e * (y - m)).sum(1) / total[:, 0]
        logp = (y - lse).gather(1, t.clamp(min=0)[:, None])[:, 0]
        ids = torch.empty(x.shape[0], 0, dtype=torch.int32, device=x.device)
        top = torch.empty(x.shape[0], 0, device=x.device)
        if K:
            # larger values first, lower columns first among equal ones: one whole number says both
            bits = (x + 0.0).contiguous().view(torch.int32)
            order = (bits ^ ((bits >> 31) & 0x7fffffff)).long() * (1 << 32)
            order += V - 1 - torch.arange(V, device=x.device)
            best = order.topk(K, dim=1).values
            ids = (V - 1 - (best & 0xffffffff)).to(torch.int32)
            top = torch.where(keep[:, None], (y - lse).gather(1, ids.long()), torch.zeros_like(ids, dtype=torch.float32))
            ids = torch.where(keep[:, None], ids, torch.full_like(ids, -1))
        parts.append((torch.where(keep, logp, zero), torch.where(keep, lse[:, 0], zero), torch.where(keep, entropy, zero),
                      ids, top))
    return tuple(torch.cat(p) for p in zip(*parts))


def _plain_topk(s):
    logp, lse, entropy, ids, top = _plain_scores(s["logits"], s["target"], min(s["K"], s["V"]), s["tau"])
    return {"logp": logp, "lse": lse, "entropy": entropy, "ids": ids, "top": top}


def _plain_topk_grad(s):
    x, target, tau = s["logits"], s["target"], s["tau"]
    keep = target >= 0
    logp = x.float() / tau - s["lse"][:, None]
    p = torch.exp(logp)
    gl, gh = s["grad_logp"], s["grad_entropy"]
    total = gl + s["grad_top"].sum(1)
    grad = -p * (total[:, None] + gh[:, None] * (logp + s["entropy"][:, None]))
    grad.scatter_add_(1, target.clamp(min=0)[:, None], gl[:, None])
    grad.scatter_add_(1, s["ids"].long().clamp(min=0), s["grad_top"])
    return {"grad": torch.where(keep[:, None], grad / tau, torch.zeros_like(grad)).to(x.dtype)}


def _plain_embed(s):
    ids = s["ids"]
    rows = s["table"][ids.clamp(min=0)].float() * s["scale"]
    return {"out": torch.where((ids >= 0)[:, None], rows, torch.zeros_like(rows)).to(TYPES[s["out"]])}


def _plain_embed_grad(s):
    ids, g = s["ids"], s["grad_out"].float()
    g = torch.where((ids >= 0)[:, None], g, torch.zeros_like(g))
    grad = torch.zeros(s["V"], s["D"], device=g.device).index_add_(0, ids.clamp(min=0), g)
    return {"grad": grad.mul_(s["scale"]).to(TYPES[s["out"]])}


def _plain_routed(s):
    x, K = s["x"], s["K"]
    r = x.double() @ s["router"].double().T  # two experts' scores may lie closer than 32 bits tell them apart
    if s["lean"] is not None:
        r = r + s["lean"].double()
    r = r.float()
    bits = (r + 0.0).view(torch.int32)
    order = (bits ^ ((bits >> 31) & 0x7fffffff)).long() * (1 << 32) + (s["E"] - 1 - torch.arange(s["E"], device=x.device))
    ids = s["E"] - 1 - (order.topk(K, dim=1).values & 0xffffffff)
    e = torch.exp(r - r.amax(1, keepdim=True))
    w = e.gather(1, ids)
    w = w / (w if s["renorm"] else e).sum(1, keepdim=True)
    share = torch.zeros_like(r).scatter_(1, ids, w)
    out = torch.zeros(x.shape, device=x.device)
    for j in range(s["E"]):
        a = x.float() @ s["gate_up"][j].float().T
        gate, up = a[:, :s["F"]], a[:, s["F"]:]
        h = gate / (1.0 + torch.exp(-gate)) * up
        out += share[:, j:j + 1] * (h @ s["down"][j].float().T)
    return {"out": out.to(x.dtype), "logits": r, "ids": ids.to(torch.int32), "weights": w}


# ---- a pass ----------------------------------------------------------------------------------------------------------
def _own(s):
    import sinkhorn_point_cloud_gb300 as sot
    op = s["op"]
    if op == "topk":
        logp, lse, entropy, ids, top = sot.sot_token_topk(s["logits"], min(s["K"], s["V"]), target=s["target"],
                                                          temperature=s["tau"])
        return {"logp": logp, "lse": lse, "entropy": entropy, "ids": ids, "top": top}
    if op == "topk_grad":
        some = s["K"] > 0
        return {"grad": sot.sot_token_topk_grad(s["logits"], s["lse"], entropy=s["entropy"], target=s["target"],
                                                grad_logp=s["grad_logp"], grad_entropy=s["grad_entropy"],
                                                ids=s["ids"] if some else None, grad_top=s["grad_top"] if some else None,
                                                temperature=s["tau"])}
    if op == "embed":
        return {"out": sot.sot_embed(s["table"], s["ids"], scale=s["scale"], dtype=TYPES[s["out"]])}
    if op == "embed_grad":
        return {"grad": sot.sot_embed_grad(s["grad_out"], s["ids"], s["V"], scale=s["scale"], dtype=TYPES[s["out"]])}
    out, logits, ids, weights = sot.sot_routed_layer(s["x"], s["router"], s["gate_up"], s["down"], s["K"], bias=s["lean"],
                                                     renorm=s["renorm"])
    return {"out": out, "logits": logits, "ids": ids, "weights": weights}


_PLAIN = {"topk": _plain_topk, "topk_grad": _plain_topk_grad, "embed": _plain_embed, "embed_grad": _plain_embed_grad,
          "routed": _plain_routed}


def run(state):
    return _own(state) if own else _PLAIN[state["op"]](state)


def work(case):
    """Each input read once, each output written once; rows that take no part are not read, nor experts no token chose
    (for independent tokens, the expected number of those that are)."""
    op, size = case["op"], SIZE[case["dtype"]]
    T = case["T"]
    if op == "routed":
        H, E, F, K = case["H"], case["E"], case["F"], case["K"]
        chosen = E * (1.0 - (1.0 - K / E) ** T)
        return {"bytes": int(size * (chosen * 3 * F * H + E * H + 2 * T * H)) + 4 * T * E + 8 * T * K,
                "flops": 2 * T * (E * H + K * 3 * F * H)}
    if op in ("embed", "embed_grad"):
        n, k = _distinct(case)
        D, out = case["D"], SIZE[case["out"]]
        if op == "embed":
            return {"bytes": k * D * size + T * D * out + 8 * T, "flops": n * D}
        return {"bytes": n * D * size + case["V"] * D * out + 8 * T, "flops": n * D}
    V, K = case["V"], min(case["K"], case["V"])
    n = T - int(T * case["skip"])
    if op == "topk":
        return {"bytes": n * V * size + T * (20 + 8 * K), "flops": 6 * n * V}
    return {"bytes": n * V * size + T * V * size + T * (24 + 8 * K), "flops": 8 * n * V}


# ---- 64 bits, from the definitions ------------------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    op, d = case["op"], torch.float64
    if op == "embed":
        out = s["table"].to(d).index_select(0, s["ids"].clamp(min=0)) * s["scale"]
        return {"out": out * (s["ids"] >= 0)[:, None]}
    if op == "embed_grad":
        used = s["ids"] >= 0
        grad = torch.zeros(case["V"], case["D"], dtype=d, device=s["ids"].device)
        grad.index_put_((s["ids"][used],), s["grad_out"][used].to(d) * s["scale"], accumulate=True)
        return {"grad": grad}
    if op == "routed":
        x, E, K, F = s["x"].to(d), case["E"], case["K"], case["F"]
        r = torch.nn.functional.linear(x, s["router"].to(d), None if s["lean"] is None else s["lean"].to(d))
        ids = r.to(torch.float32).sort(dim=1, descending=True, stable=True).indices[:, :K]
        w = torch.softmax(r, 1).gather(1, ids)
        if case["renorm"]:
            w = w / w.sum(1, keepdim=True)
        out = torch.zeros_like(x)
        for e in range(E):
            t, k = (ids == e).nonzero(as_tuple=True)
            if len(t):
                gate, up = (x[t] @ s["gate_up"][e].to(d).T).split(F, 1)
                out.index_add_(0, t, w[t, k, None] * ((torch.nn.functional.silu(gate) * up) @ s["down"][e].to(d).T))
        return {"out": out, "logits": r, "ids": ids.to(torch.int32), "weights": w}
    T, V, tau, K = case["T"], case["V"], case["tau"], min(case["K"], case["V"])
    keep = s["target"] >= 0
    step = max(1, (1 << 25) // V)
    parts = []
    for a in range(0, T, step):
        x, t, use = s["logits"][a:a + step].to(d), s["target"][a:a + step].clamp(min=0), keep[a:a + step]
        ls = torch.log_softmax(x / tau, 1)
        entropy = -(ls.exp() * ls).sum(1)
        if op == "topk":
            ids = x.sort(dim=1, descending=True, stable=True).indices[:, :K]
            parts.append({"logp": ls.gather(1, t[:, None])[:, 0] * use, "lse": torch.logsumexp(x / tau, 1) * use,
                          "entropy": entropy * use, "ids": torch.where(use[:, None], ids, -1).to(torch.int32),
                          "top": ls.gather(1, ids) * use[:, None]})
        else:
            gl, gh = s["grad_logp"][a:a + step].to(d), s["grad_entropy"][a:a + step].to(d)
            into = torch.zeros_like(ls).scatter_(1, t[:, None], gl[:, None])  # with respect to the log-probabilities
            into.scatter_add_(1, s["ids"][a:a + step].long().clamp(min=0), s["grad_top"][a:a + step].to(d))
            grad = into - ls.exp() * into.sum(1, keepdim=True) - gh[:, None] * ls.exp() * (ls + entropy[:, None])
            parts.append({"grad": grad / tau * use[:, None]})
    return {k: torch.cat([p[k] for p in parts]) for k in parts[0]}
