"""Plain 64-bit forms of the language-model operators around the losses, for the tests.

Each returns its outputs and, where sums cancel, the size of the terms that are added up
(rounding errors are relative to these)."""
from __future__ import annotations

import numpy as np

import lm_ref as R


def token_topk(x, target, K, tau):
    """(logp, lse, entropy, ids, top); target None: every row takes part."""
    T, V = x.shape
    logp, lse, ent = np.zeros(T), np.zeros(T), np.zeros(T)
    ids, top = np.full((T, K), -1, np.int32), np.zeros((T, K))
    for t in range(T):
        if target is not None and not 0 <= target[t] < V:
            continue
        lp, lse[t] = R.log_softmax(x[t], tau)
        if target is not None:
            logp[t] = lp[target[t]]
        if not (np.isfinite(lse[t]) and not np.isnan(x[t]).any()):
            lse[t] = -np.inf if (x[t] == -np.inf).all() else np.nan
            logp[t] = np.nan if target is not None else 0.0
            ent[t] = np.nan
            top[t] = np.nan
            continue
        p = np.exp(lp)
        ent[t] = -np.sum(np.where(p > 0, p * np.where(p > 0, lp, 0.0), 0.0))
        order = np.argsort(-x[t], kind="stable")[:K]
        order = order[x[t][order] > -np.inf]
        ids[t, :len(order)] = order
        top[t] = -np.inf
        top[t, :len(order)] = lp[order]
    return logp, lse, ent, ids, top


def token_topk_grad(x, target, ids, tau, gl, gh, gt):
    """Gradient with respect to the logits; any of gl, gh, gt None."""
    T, V = x.shape
    grad, size = np.zeros((T, V)), np.zeros((T, V))
    for t in range(T):
        if target is not None and not 0 <= target[t] < V:
            continue
        into, mass = np.zeros(V), np.zeros(V)
        if gl is not None and target is not None:
            into[target[t]] += gl[t]
            mass[target[t]] += abs(gl[t])
        if gt is not None:
            for k, v in enumerate(ids[t]):
                if 0 <= v < V:
                    into[v] += gt[t, k]
                    mass[v] += abs(gt[t, k])
        h = 0.0 if gh is None else gh[t]
        if not mass.any() and h == 0:
            continue
        lp, _ = R.log_softmax(x[t], tau)
        p = np.exp(lp)
        l = np.where(p > 0, lp, 0.0)
        H = -np.sum(p * l)
        grad[t] = (into - p * into.sum() - h * p * (l + H)) / tau
        size[t] = (mass + p * mass.sum() + abs(h) * p * (np.abs(l) + H + 1 + np.log(V))) / tau
    return grad, size


def embed(table, ids, scale):
    out = np.zeros((len(ids), table.shape[1]))
    use = (ids >= 0) & (ids < table.shape[0])
    out[use] = scale * table[ids[use]]
    return out


def embed_grad(g, ids, V, scale):
    grad, size = np.zeros((V, g.shape[1])), np.zeros((V, g.shape[1]))
    use = (ids >= 0) & (ids < V)
    np.add.at(grad, ids[use], scale * g[use])
    np.add.at(size, ids[use], np.abs(scale * g[use]))
    return grad, size


def routed(x, router, gate_up, down, K, bias, renorm, scale):
    """(out, logits, ids, weights, size of out's terms)."""
    T, E, F = x.shape[0], router.shape[0], down.shape[2]
    r = x @ router.T + (0 if bias is None else bias)
    ids, w = np.full((T, K), -1, np.int32), np.zeros((T, K))
    out, size = np.zeros(x.shape), np.zeros(x.shape)
    for t in range(T):
        if np.isnan(r[t]).any() or (r[t] == np.inf).any():
            w[t] = out[t] = np.nan
            continue
        r32 = r[t].astype(np.float32)
        order = np.argsort(-r32, kind="stable")[:K]
        order = order[r32[order] > -np.inf]
        ids[t, :len(order)] = order
        if len(order) == 0:
            continue
        e = np.exp(r[t] - r[t].max())
        w[t, :len(order)] = scale * e[order] / (e[order].sum() if renorm else e.sum())
        for k, j in enumerate(order):
            g, u = gate_up[j, :F] @ x[t], gate_up[j, F:] @ x[t]
            h = g / (1 + np.exp(-g)) * u
            out[t] += w[t, k] * (down[j] @ h)
            size[t] += abs(w[t, k]) * (np.abs(down[j]) @ np.abs(h))
    return out, r, ids, w, size
