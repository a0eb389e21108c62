"""CPU oracle of the operators over rows of logits (test infrastructure, NumPy fp64).

Written from the definitions in ``include/eqat.h``; loops over rows, no sharing with the
CUDA path.
"""
import numpy as np


def _lse(z):
    m = z.max()
    if m == -np.inf:
        return -np.inf
    return m + np.log(np.exp(z - m).sum())


def _centred(z):
    """z less its maximum (a row of the type's lowest value is uniform: -3e38 plus the log
    of a sum would lose it even in fp64), and the log of the sum of its exponentials."""
    m = z.max()
    z = z - m if m > -np.inf else z
    return z, _lse(z)


def token_logprobs(x, targets, top_k=0, temperature=1.0):
    """(logprob, entropy, top_ids, top_logprobs) of rows x [T, V] as fp64."""
    x = np.asarray(x, np.float64)
    T, V = x.shape
    lp, ent = np.zeros(T), np.zeros(T)
    ids, top = np.full((T, top_k), -1, np.int64), np.full((T, top_k), -np.inf)
    for t in range(T):
        row, id_ = x[t], int(targets[t])
        if np.isnan(row).any() or (row == np.inf).any():
            lp[t], ent[t], top[t] = np.nan if id_ >= 0 else 0.0, np.nan, np.nan
            continue
        z, lse = _centred(row / temperature)
        if id_ >= V:
            lp[t] = np.nan
        elif id_ >= 0:
            lp[t] = -np.inf if lse == -np.inf else z[id_] - lse
        if lse == -np.inf:
            continue
        live = np.flatnonzero(row > -np.inf)
        logp = z[live] - lse
        ent[t] = -(np.exp(logp) * logp).sum()
        order = live[np.lexsort((live, -row[live]))][:top_k]
        ids[t, :len(order)] = order
        top[t, :len(order)] = z[order] - lse
    return lp, ent, ids, top


def distill_topk(x, ids, tlp, weight=None, temperature=1.0, tail=False):
    """(loss [T], gradient [T, V]) as fp64."""
    x, tlp = np.asarray(x, np.float64), np.asarray(tlp, np.float64)
    T, V = x.shape
    loss, grad = np.zeros(T), np.zeros((T, V))
    for t in range(T):
        w = 1.0 if weight is None else float(weight[t])
        if w == 0.0:
            continue
        use = ids[t] >= 0
        if (ids[t] >= V).any() or not (tlp[t][use] < np.inf).all() or not (x[t] < np.inf).all():
            loss[t], grad[t] = np.nan, np.nan
            continue
        z, lse = _centred(x[t] / temperature)
        slots, lq = ids[t][use], tlp[t][use]
        if lse == -np.inf or (not tail and not (lq > -np.inf).any()):
            continue
        if not tail:
            lq = lq - _lse(lq)
        q = np.exp(lq)
        logp = z - lse
        p = np.exp(logp)
        m = q > 0
        L = (q[m] * (lq[m] - logp[slots[m]])).sum()
        g = p.copy()
        if tail:
            outside = np.ones(V, bool)
            outside[slots] = False
            qr = max(0.0, 1.0 - q.sum())
            lpr = _lse(z[outside]) - lse if outside.any() else -np.inf
            if qr > 0 and lpr > -np.inf:
                L += qr * (np.log(qr) - lpr)
                g[outside] -= qr * np.exp(logp[outside] - lpr)
        np.subtract.at(g, slots, q)
        loss[t] = w * L
        grad[t] = g * (w / temperature)
    return loss, grad
