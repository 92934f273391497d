"""Plain 64-bit forms of the language-model losses, row by row, for the tests.

Each returns its outputs and, for a gradient, the size of the terms that are
added up in each of its elements (rounding errors are relative to these)."""
from __future__ import annotations

import numpy as np


def log_softmax(x, tau):
    y = np.asarray(x, np.float64) / tau
    m = np.max(y, axis=-1, keepdims=True)
    with np.errstate(invalid="ignore", divide="ignore"):
        ls = np.log(np.sum(np.exp(y - m), axis=-1, keepdims=True))
        return (y - m) - ls, (m + ls)[..., 0]


def token_logprob(x, target, tau):
    T, V = x.shape
    logp, lse = np.zeros(T), np.zeros(T)
    for t in range(T):
        if 0 <= target[t] < V:
            lp, l = log_softmax(x[t], tau)
            logp[t], lse[t] = lp[target[t]], l
    return logp, lse


def token_grad(x, target, tau, g):
    T, V = x.shape
    grad, size = np.zeros((T, V)), np.zeros((T, V))
    for t in range(T):
        if 0 <= target[t] < V and g[t] != 0:
            lp, _ = log_softmax(x[t], tau)
            p = np.exp(lp)
            grad[t] = -p
            size[t] = p
            grad[t, target[t]] += 1
            size[t, target[t]] += 1
            grad[t] *= g[t] / tau
            size[t] *= abs(g[t]) / tau
    return grad, size


def policy(x, target, old, adv, ref, w, tau, lo, hi, kc):
    T, V = x.shape
    loss, logp, kl, d = (np.zeros(T) for _ in range(4))
    for t in range(T):
        if w[t] == 0 or not 0 <= target[t] < V:
            continue
        lp = log_softmax(x[t], tau)[0][target[t]]
        r = np.exp(lp - old[t])
        free, held = r * adv[t], min(max(r, 1 - lo), 1 + hi) * adv[t]
        loss[t] = -min(free, held)
        d[t] = -free if free <= held else 0.0
        if ref is not None:
            u = ref[t] - lp
            kl[t] = np.expm1(u) - u
            loss[t] += kc * kl[t]
            d[t] -= kc * np.expm1(u)
        logp[t] = lp
    return w * loss, logp, kl, w * d


def distill(x, ids, z, w, tau, tail):
    T, V = x.shape
    loss, grad, size = np.zeros(T), np.zeros((T, V)), np.zeros((T, V))
    for t in range(T):
        if w[t] == 0:
            continue
        lp, _ = log_softmax(x[t], tau)
        p = np.exp(lp)
        used = (ids[t] >= 0) & (ids[t] < V)
        at, zt = ids[t][used], np.asarray(z[t], np.float64)[used]
        q = np.zeros(0)
        if len(at):
            if tail:
                lq = zt
            else:
                lq = log_softmax(zt, tau)[0] if np.max(zt) > -np.inf else np.full(len(zt), -np.inf)
            q = np.exp(lq)
        pos = q > 0
        value = float(np.sum(q[pos] * (lq[pos] - lp[at][pos]))) if len(at) else 0.0
        Q = q.sum()
        outer = np.zeros(V)
        if tail:
            rest = np.ones(V, bool)
            rest[at] = False
            pr = p[rest].sum()
            qr = max(0.0, 1.0 - Q) if pr > 0 else 0.0
            if qr > 0:
                value += qr * (np.log(qr) - np.log(pr))
                outer[rest] = qr * p[rest] / pr
            Q += qr
        g = Q * p - outer
        s = Q * p + outer
        g[at] -= q
        s[at] += q
        loss[t] = w[t] * tau * tau * value
        grad[t], size[t] = w[t] * tau * g, abs(w[t]) * tau * s
    return loss, grad, size


def preference(logp, ref, target, off, beta, ls, average, scale):
    P = len(off) // 2
    loss, margin, grad = np.zeros(P), np.zeros(P), np.zeros(len(logp))
    r = np.asarray(logp, np.float64) - (0 if ref is None else np.asarray(ref, np.float64))
    use = np.ones(len(logp), bool) if target is None else target >= 0
    for p in range(P):
        part = [np.arange(off[2 * p + h], off[2 * p + h + 1]) for h in (0, 1)]
        part = [i[use[i]] for i in part]
        n = [max(len(i), 1) if average else 1 for i in part]
        margin[p] = r[part[0]].sum() / n[0] - r[part[1]].sum() / n[1]
        zed = beta * margin[p]
        loss[p] = (1 - ls) * np.logaddexp(0, -zed) + ls * np.logaddexp(0, zed)
        sn = np.exp(-np.logaddexp(0, zed))
        d = scale * beta * (ls * (1 - sn) - (1 - ls) * sn)
        grad[part[0]], grad[part[1]] = d / n[0], -d / n[1]
    return loss, margin, grad


def balance(x, ids, mask, cb, cz):
    T, E = x.shape
    K = ids.shape[1]
    keep = np.ones(T, bool) if mask is None else mask
    N = int(keep.sum())
    counts = np.zeros(E, np.int64)
    for t in range(T):
        if keep[t]:
            for e in ids[t]:
                if 0 <= e < E:
                    counts[e] += 1
    grad, size = np.zeros((T, E)), np.zeros((T, E))
    if N == 0:
        return counts, np.zeros(2), grad, size
    f = counts * (E / (K * N))
    lp, lse = log_softmax(x[keep], 1.0)
    p = np.exp(lp)
    dot = p @ f
    grad[keep] = p * (cb * (f - dot[:, None]) + 2 * cz * lse[:, None]) / N
    size[keep] = p * (abs(cb) * (f + dot[:, None]) + 2 * abs(cz) * np.abs(lse)[:, None]) / N
    return counts, np.array([cb * dot.sum() / N, cz * (lse ** 2).sum() / N]), grad, size
