"""Plain 64-bit forms of a teacher's top logits and of the distillation loss (numpy), for the tests.  No code
of the library."""

import numpy as np


def topk(x, k, temperature, labels=None):
    """(ids, values, tail) of each row: by falling value (NaN first), then rising index; -inf is not listed."""
    T, V = x.shape
    ids, values, tail = np.full((T, k), -1, dtype=np.int64), np.full((T, k), -np.inf), np.full(T, -np.inf)
    for t in range(T):
        if labels is not None and labels[t] < 0:
            continue
        key = np.where(np.isnan(x[t]), np.inf, x[t] + 0.0)
        order = np.lexsort((np.arange(V), -key, ~np.isnan(x[t])))
        for j, v in enumerate(order[:k]):
            if x[t, v] != -np.inf:
                ids[t, j], values[t, j] = v, x[t, v]
        rest = x[t, order[k:]] / temperature
        if rest.size and not np.all(rest == -np.inf):
            top = np.max(rest[~np.isnan(rest)], initial=-np.inf)
            top = top if np.isfinite(top) else 0.0
            with np.errstate(over="ignore"):
                tail[t] = top + np.log(np.sum(np.exp(rest - top)))
    return ids, values, tail


def _xlogx(p, q):
    """p log(p / q), 0 where p is 0."""
    with np.errstate(divide="ignore", invalid="ignore"):
        return np.where(p > 0, p * (np.log(np.where(p > 0, p, 1.0)) - np.log(q)), 0.0)


def _row(x, ids, values, tail, label, kind, mix, tau, kd_weight, ce_weight):
    """(kd, ce, gradient, size) of a row that counts; size bounds what the gradient's parts add up to."""
    V = x.size
    none = np.all(x == -np.inf)
    here = [j for j in range(len(ids)) if ids[j] >= 0 and values[j] != -np.inf]
    ids = np.array([ids[j] for j in here], dtype=np.int64)
    w = np.array([values[j] for j in here] + [tail], dtype=np.float64)
    w[:-1] /= tau
    teacher = np.any(w != -np.inf)
    if none:
        return (np.inf if teacher else 0.0), (np.inf if ce_weight > 0 else 0.0), np.zeros(V), np.zeros(V)
    z = x / tau
    e = np.exp(z - np.max(z))
    q_all = e / e.sum()
    rest = np.ones(V, dtype=bool)
    rest[ids] = False
    qb = np.append(q_all[ids], e[rest].sum() / e.sum())
    kd, grad, size = 0.0, np.zeros(V), np.zeros(V)
    if teacher:
        p = np.exp(w - np.max(w))
        p /= p.sum()
        with np.errstate(divide="ignore", invalid="ignore"):
            if kind == "forward":
                kd = _xlogx(p, qb).sum()
                e_ = np.where(qb > 0, 1 - p / qb, 0.0)
                C = 0.0
                direct = qb - p
            elif kind == "reverse":
                kd = _xlogx(qb, p).sum()
                e_ = np.where(qb > 0, np.log(qb / p), 0.0)
                C = (qb * e_).sum()
                direct = None
            else:
                m = mix * p + (1 - mix) * qb
                kd = mix * _xlogx(p, m).sum() + (1 - mix) * _xlogx(qb, m).sum()
                e_ = np.where(qb > 0, (1 - mix) * np.log(qb / m), 0.0)
                C = (qb * e_).sum()
                direct = None
        if np.isfinite(C):
            grad = q_all * (e_[-1] - C)
            grad[ids] = direct[:-1] if direct is not None else qb[:-1] * (e_[:-1] - C)
            size = q_all * (abs(e_[-1]) + abs(C) + 1 + (p[-1] / qb[-1] if qb[-1] > 0 else 0))
            size[ids] = qb[:-1] * (np.abs(np.where(np.isfinite(e_[:-1]), e_[:-1], 0)) + abs(C) + 1) + p[:-1]
            grad, size = grad * kd_weight / tau, size * kd_weight / tau
    ce = 0.0
    if ce_weight > 0:
        e = np.exp(x - np.max(x))
        ce = -(x[label] - np.max(x) - np.log(e.sum()))
        soft = e / e.sum()
        grad, size = grad + ce_weight * soft, size + ce_weight * soft
        grad[label] -= ce_weight
        size[label] += ce_weight
    return kd, ce, grad, size


def distill(x, ids, values, tail=None, labels=None, weight=None, kind="forward", mix=0.5, temperature=1.0, kd_weight=1.0,
            ce_weight=0.0, grad_scale=1.0):
    """dict of loss, kd, ce [T], grad [T, V], size [T, V] and spread [T] (the largest logarithm of a row, which
    fp32 rounds)."""
    T, V = x.shape
    out = dict(loss=np.zeros(T), kd=np.zeros(T), ce=np.zeros(T), grad=np.zeros((T, V)), size=np.zeros((T, V)), spread=np.zeros(T))
    for t in range(T):
        on = [i for i, v in zip(ids[t], values[t]) if i >= 0 and v != -np.inf]
        if labels is not None and (labels[t] < 0 or labels[t] >= V) or any(i >= V for i in on) or len(set(on)) < len(on):
            continue
        w = 1.0 if weight is None else float(weight[t])
        label = -1 if labels is None else int(labels[t])
        kd, ce, grad, size = _row(x[t], ids[t], values[t], -np.inf if tail is None else tail[t], label, kind, mix, temperature,
                                  kd_weight, ce_weight)
        out["kd"][t], out["ce"][t] = kd, ce
        if w != 0:
            out["loss"][t] = w * ((kd_weight * kd if kd_weight > 0 else 0.0) + (ce_weight * ce if ce_weight > 0 else 0.0))
            out["grad"][t], out["size"][t] = grad_scale * w * grad, abs(grad_scale * w) * size
        seen = np.concatenate([[0.0 if tail is None or not np.isfinite(tail[t]) else tail[t]],
                               [v / temperature for v in values[t] if np.isfinite(v)],
                               (x[t] - np.max(x[t]))[np.array(on, dtype=int)] / temperature if np.isfinite(np.max(x[t])) else [0.0],
                               [x[t, label] - np.max(x[t])] if label >= 0 and np.isfinite(np.max(x[t])) else []])
        out["spread"][t] = np.max(np.abs(seen[np.isfinite(seen)]), initial=0.0)
    return out
