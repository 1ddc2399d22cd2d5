"""Plain 64-bit forms of the training operators (numpy), for the tests: the losses on logits with
their gradients, the e4m3 rounding of moments, and the AdamW step.  No code of the library."""

import numpy as np


def bf16_round(a):
    """Nearest bf16 value (ties to even) of doubles that are far from the format's limits."""
    a = np.asarray(a, dtype=np.float64)
    m, e = np.frexp(a)
    return np.ldexp(np.round(np.ldexp(m, 8)), e - 8)


# ------------------------------------------------------------- losses on logits --

def logprobs(x, labels):
    """(logp, lse) of each row; 0 where the label is negative or past the row."""
    T, V = x.shape
    logp, lse = np.zeros(T), np.zeros(T)
    for t in range(T):
        if labels[t] < 0 or labels[t] >= V:
            continue
        top = np.max(x[t])
        if np.isnan(x[t]).any():
            lse[t] = logp[t] = np.nan
        elif top == -np.inf:
            lse[t] = logp[t] = -np.inf
        elif top == np.inf:
            lse[t] = np.inf
            logp[t] = x[t, labels[t]] - np.inf
        else:
            lse[t] = top + np.log(np.sum(np.exp(x[t] - top)))
            logp[t] = x[t, labels[t]] - lse[t]
    return logp, lse


def softmax_grad(x, labels, lse, coef):
    """coef[t] * (1[v = label] - softmax) with zero rows where nothing counts."""
    g = np.zeros(x.shape)
    for t in range(x.shape[0]):
        if labels[t] < 0 or labels[t] >= x.shape[1] or lse[t] == -np.inf or coef[t] == 0:
            continue
        g[t] = -coef[t] * np.exp(x[t] - lse[t])
        g[t, labels[t]] += coef[t]
    return g


def _softplus(z):
    return max(z, 0.0) + np.log1p(np.exp(-abs(z)))


def _sigmoid(z):
    return 1 / (1 + np.exp(-z)) if z > 0 else np.exp(z) / (1 + np.exp(z))


def preference(x, labels, ref, indptr, kind, beta, smooth, margin, average, grad_scale):
    """(loss [P], seq_logp [2P], dlogits, coef) of the paired loss."""
    T, V = x.shape
    logp, lse = logprobs(x, labels)
    on = (labels >= 0) & (labels < V)
    n = len(indptr) // 2
    loss, seq, coef = np.zeros(n), np.zeros(2 * n), np.zeros(T)
    for p in range(n):
        r, share = [], []
        for s in (2 * p, 2 * p + 1):
            rows = [t for t in range(indptr[s], indptr[s + 1]) if on[t]]
            seq[s] = sum(logp[t] for t in rows)
            d = sum(logp[t] - (0.0 if ref is None else float(ref[t])) for t in rows)
            share.append(1.0 / len(rows) if average and rows else 1.0)
            r.append(d * share[-1])
        D = r[0] - r[1]
        z = beta * D - margin
        if kind == "sigmoid":
            loss[p] = (1 - smooth) * _softplus(-z) + smooth * _softplus(z)
            dD = beta * (smooth * _sigmoid(z) - (1 - smooth) * _sigmoid(-z))
        elif kind == "hinge":
            loss[p], dD = max(0.0, 1 - z), (-beta if z < 1 else 0.0)
        else:
            off = D - 0.5 / beta
            loss[p], dD = off * off, 2 * off
        for k, s in enumerate((2 * p, 2 * p + 1)):
            coef[indptr[s]: indptr[s + 1]] = (1 - 2 * k) * dD * share[k] * grad_scale
    coef = np.where(on, coef, 0.0)
    return loss, seq, softmax_grad(x, labels, lse, coef), coef


def policy(x, labels, old, adv, ref, weight, lo, hi, kl_coef, grad_scale):
    """(logp, loss, kl, dlogits, coef) of the clipped policy loss."""
    T, V = x.shape
    logp, lse = logprobs(x, labels)
    loss, kl, coef = np.zeros(T), np.zeros(T), np.zeros(T)
    for t in range(T):
        if labels[t] < 0 or labels[t] >= V:
            continue
        w = 1.0 if weight is None else float(weight[t])
        q = np.exp(logp[t] - float(old[t]))
        a = float(adv[t])
        first, second = q * a, min(max(q, 1 - lo), 1 + hi) * a
        g = 0.0
        if kl_coef > 0:
            d = float(ref[t]) - logp[t]
            kl[t] = np.expm1(d) - d
            g = np.expm1(d)
        if w != 0:
            loss[t] = w * (kl_coef * kl[t] - min(first, second))
            coef[t] = -grad_scale * w * (kl_coef * g + (first if first <= second else 0.0))
    return logp, loss, kl, softmax_grad(x, labels, lse, coef), coef


# ---------------------------------------------------------------- optimizer step --

def positions(pool, i):
    """Pool positions of adapter i's elements: A's, then B's."""
    P = pool.page_elems
    out = []
    for page0, d in ((int(pool.desc[i]["a_page0"]), pool.d_in), (int(pool.desc[i]["b_page0"]), pool.d_out)):
        e = np.arange(int(pool.ranks[i]) * d, dtype=np.int64)
        out.append(pool.page_list[page0 + e // P].astype(np.int64) * P + e % P)
    return out


def decode_e4m3(c):
    """Values of e4m3 codes (uint8)."""
    c = np.asarray(c, dtype=np.int64)
    s, e, m = c >> 7, (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(s == 1, -v, v)


def adamw(w, g, m, v, h, sumsq=None):
    """(w, m, v, c) after a step in 64 bits; h: dict of one adapter's settings."""
    gs = h["grad_scale"]
    c = 1.0
    if sumsq is not None and h["max_norm"] > 0:
        c = min(1.0, h["max_norm"] / (np.sqrt(sumsq) * abs(gs) + 1e-6))
    g = g * (gs * c)
    m = h["beta1"] * m + (1 - h["beta1"]) * g
    v = h["beta2"] * v + (1 - h["beta2"]) * g * g
    up = (m / (1 - h["beta1"] ** h["step"])) / (np.sqrt(v / (1 - h["beta2"] ** h["step"])) + h["eps"])
    return w * (1 - h["lr"] * h["weight_decay"]) - h["lr"] * up, m, v, c
