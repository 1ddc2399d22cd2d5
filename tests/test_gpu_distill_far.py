"""The distillation loss where logarithms are large: rows that lie far from zero as a whole, lists hidden by a finite
mask, warps of a list without entries; in each form of the kernel."""

import numpy as np
import pytest
import torch

import distill_ref as R
from gpu_util import cuda_or_skip
from test_gpu_distill import BF16, F32, batch, device, run_loss

pytestmark = pytest.mark.gpu

# rows, vocabulary and list by which a call takes its form: streamed by a CTA of 64, 128, 256, 512 and 1024 threads, and
# held by a cluster
FORMS = [(310, 700, 32), (310, 700, 33), (160, 9000, 33), (160, 9000, 200), (3, 3000, 256), (40, 40000, 40), (3, 300001, 40),
         (3, 40001, 100), (2, 128256, 256)]


def check_far(x, ids, values, tail, labels=None, dtype=F32, far=0.0, **kw):
    """Against the plain form.  A logarithm of p or q is off by three roundings of the largest logarithm of the row (the
    listed entries' and `far`, those of the rest) and of a sum's logarithm below 16, and by the sums' errors (2^-19): d
    in all.  kd = sum of p (log p - log q) - p + q moves by q - p with log q, at most 2 d together, and by
    p (log p - log q) with log p, where those of one sign add up to little more than kd itself: by d of kd; a term's own
    arithmetic is off by 2^-18 of it.  A gradient's parts move by d of themselves, four of them, and are rounded once."""
    loss, kd, ce, grad = run_loss(x, ids, values, tail, labels, dtype=dtype, **kw)
    x = device(x, dtype)[2]
    want = R.distill(x, ids, values.astype(np.float32).astype(np.float64), tail, labels, **kw)
    d = 3 * 2.0 ** -24 * (want["spread"] + far + 16) + 2.0 ** -19
    for name, got in (("kd", kd), ("ce", ce), ("loss", loss)):
        w = want[name]
        with np.errstate(invalid="ignore"):
            assert np.array_equal(got[~np.isfinite(w)], w[~np.isfinite(w)]), (name, got, w)
            scale = kw.get("kd_weight", 1.0) + kw.get("ce_weight", 0.0) if name == "loss" else 1.0
            tol = scale * 2 * d + (2.0 ** -18 + d) * np.abs(w) + 1e-37
            bad = np.isfinite(w) & ~(np.abs(got - w) <= tol)
        assert not bad.any(), (name, got[bad][:4], w[bad][:4], tol[bad][:4])
    tol = 4 * d[:, None] * want["size"] + np.abs(want["grad"]) * (torch.finfo(dtype).eps / 2) * 1.01 + 2.0 ** -126
    bad = ~(np.abs(grad - want["grad"]) <= tol)
    assert not bad.any(), (np.argwhere(bad)[:5], grad[bad][:4], want["grad"][bad][:4], tol[bad][:4])


def some(T, V, k):
    return batch(np.random.default_rng(T + V + k), T, V, k, absent=0.0)


@pytest.mark.parametrize("kind", ["forward", "reverse", "jsd"])
@pytest.mark.parametrize("T,V,k", FORMS)
def test_rows_far_from_zero(T, V, k, kind):
    """Only differences count: student's and teacher's rows moved by -90, -200, -1e4 and +1e4, also apart."""
    cuda_or_skip()
    x, ids, values, rest, labels = some(T, V, k)
    moves = [(-90, -90), (-200, -200), (-1e4, -1e4), (-95, 0), (0, -95), (1e4, 1e4), (-300, 50)]
    for temperature, ce in ((1.0, 0.0), (0.5, 0.5)):
        y, w, r = x.copy(), values.copy(), rest.copy()
        for t in range(T):
            a, b = moves[t % len(moves)] if T >= len(moves) else moves[(t + (3 if ce else 0)) % len(moves)]
            y[t] += a
            w[t] += b
            r[t] += np.float32(b / temperature)
        if temperature != 1.0:  # the rest in the measure of the temperature
            r = (r - rest + np.log(np.exp((values.astype(np.float64) - 20) / temperature).sum(1)) + 20 / temperature - 1).astype(np.float32)
        for dtype in ((F32, BF16) if T < 100 else (F32,)):
            check_far(y, ids, w, r, labels, dtype, kind=kind, mix=0.4, temperature=temperature, ce_weight=ce)


@pytest.mark.parametrize("kind", ["forward", "reverse", "jsd"])
@pytest.mark.parametrize("T,V,k", FORMS)
def test_lists_hidden_by_a_finite_mask(T, V, k, kind):
    """The student's whole list at a mask of -1e4 or -1e30: the row is the rest's."""
    cuda_or_skip()
    x, ids, values, rest, labels = some(T, V, k)
    for t in range(T):
        x[t, ids[t]] = (-1e4, -1e30, -3e38)[t % 3]
        x[t, ids[t, 0]] -= 1.0 if t % 3 == 0 else 0.0
        if labels[t] in ids[t]:
            labels[t] = next(v for v in range(V) if v not in set(ids[t]))
    check_far(x, ids, values, rest, labels, kind=kind, mix=0.4, ce_weight=0.25)
    check_far(x, ids, values, rest, labels, kind=kind, mix=0.4, ce_weight=0.25, temperature=2.0)


@pytest.mark.parametrize("kind", ["forward", "reverse", "jsd"])
@pytest.mark.parametrize("T,V,k", [f for f in FORMS if f[2] > 32])
def test_absent_parts_of_lists_far_from_zero(T, V, k, kind):
    """Whole warps' entries of a list absent, and whole lists with a tail far below zero."""
    cuda_or_skip()
    x, ids, values, rest, labels = some(T, V, k)
    x, values, rest = x - 150, values - 150, rest - 150
    for t in range(T):
        if t % 4 == 0:
            values[t, :32] = -np.inf
        elif t % 4 == 1:
            ids[t, 32:] = -1
        elif t % 4 == 2:
            values[t] = -np.inf
    check_far(x, ids, values.astype(np.float32), rest.astype(np.float32), labels, kind=kind, mix=0.4, ce_weight=0.25)


GAPS = (80, 92, 95, 104, 110, 150, 300, 700)


def gapped(T, V, k, temperature, gaps, seed):
    """Rows with one part far below the others, `gap` temperatures: of the student a listed entry, the rest, the whole
    list; of the teacher an entry, the rest, the whole list."""
    rng = np.random.default_rng(seed)
    n = 6 * len(gaps)
    x, ids, values, rest, labels = batch(rng, n, V, k, absent=0.0)
    x, values = x * min(1.0, temperature), values.astype(np.float64) * min(1.0, temperature)
    top = np.log(np.exp(values / temperature - values.max() / temperature).sum(1)) + values.max() / temperature
    rest = top - rng.uniform(0.2, 6, n)
    for t in range(n):
        gap, part = gaps[t // 6] * temperature, t % 6
        others = np.ones(V, dtype=bool)
        others[ids[t]] = False
        if part == 0:
            x[t, ids[t, 1]] = x[t].max() - gap
        elif part == 1:
            x[t, others] += x[t, ids[t]].max() - x[t, others].max() - gap
        elif part == 2:
            x[t, ids[t]] += x[t, others].max() - x[t, ids[t]].max() - gap
        elif part == 3:
            values[t, 1] = values[t].max() - gap
        elif part == 4:
            rest[t] = top[t] - gap / temperature
        else:
            values[t] -= gap + values[t].max() - rest[t] * temperature
    at = rng.permutation(n)[np.arange(T) % n] if T < n else np.arange(T) % n
    return x[at], ids[at], values[at].astype(np.float32), rest[at].astype(np.float32), labels[at]


@pytest.mark.parametrize("kind", ["forward", "reverse", "jsd"])
@pytest.mark.parametrize("temperature", [1.0, 0.1, 2.0])
@pytest.mark.parametrize("T,V,k", [(310, 700, 32), (310, 701, 33), (160, 9000, 33), (96, 3000, 256), (60, 9003, 200), (72, 40001, 40)])
def test_shares_that_vanish(T, V, k, temperature, kind):
    """A divergence and a gradient that are numbers stay so where a share is below what fp32 holds."""
    cuda_or_skip()
    rows = gapped(T, V, k, temperature, GAPS, T + V)
    far = max(GAPS) * max(1.0, temperature)
    check_far(*rows, dtype=F32, far=far, kind=kind, mix=0.4, temperature=temperature)
    check_far(*rows, dtype=F32, far=far, kind=kind, mix=0.4, temperature=temperature, ce_weight=0.3, kd_weight=0.7)
    if temperature >= 1.0:
        check_far(*rows, dtype=BF16, far=far, kind=kind, mix=0.4, temperature=temperature, kd_weight=temperature ** 2)


@pytest.mark.parametrize("kind", ["forward", "reverse", "jsd"])
@pytest.mark.parametrize("gap", [92, 110, 700])
@pytest.mark.parametrize("T,V,k", [(6, 300001, 40), (6, 40001, 100), (6, 128256, 256)])
def test_shares_that_vanish_in_long_rows(T, V, k, gap, kind):
    cuda_or_skip()
    rows = gapped(T, V, k, 1.0, (gap,), V + gap)
    for dtype in (F32, BF16):
        check_far(*rows, dtype=dtype, far=gap, kind=kind, mix=0.4, ce_weight=0.3)


@pytest.mark.parametrize("V", [600, 9000, 70000])
def test_shares_of_less_than_64_bits_hold_are_none(V):
    """A finite mask over what the teacher lists, or over the rest, or in the teacher's list hides like -inf."""
    cuda_or_skip()
    x, ids, values, rest, labels = some(6, V, 8)
    hidden = x.copy(), values.copy(), rest.copy()
    for low, (y, w, r) in ((-3000.0, (x, values, rest)), (-np.inf, hidden)):
        y[0, ids[0, 2]] = low
        y[1] = np.where(np.isin(np.arange(V), ids[1]), y[1], low)
        y[2, ids[2]] = low
        w[3, 5] = low
        r[4] = low
        w[5] = low
    for kind in ("forward", "reverse", "jsd"):
        for temperature in (1.0, 2.0):
            kw = dict(kind=kind, temperature=temperature, mix=0.4)
            a, b = run_loss(x, ids, values, rest, **kw), run_loss(hidden[0], ids, *hidden[1:], **kw)
            for t in range(6):
                # an entry that the teacher lists as -inf is of the rest, one at a mask is listed with nothing
                if t in (3, 5):
                    continue
                assert np.array_equal(a[0][t], b[0][t]) and np.array_equal(a[3][t], b[3][t]), (kind, t)
            want = R.distill(x, ids, values.astype(np.float64), rest, **kw)
            assert np.array_equal(np.isfinite(a[1]), np.isfinite(want["kd"])), kind
            assert (a[3][~np.isfinite(a[1]) & (kind == "reverse")] == 0).all()


@pytest.mark.parametrize("kind", ["forward", "reverse", "jsd"])
@pytest.mark.parametrize("T,V,k", [(310, 700, 32), (160, 9000, 200), (6, 40001, 100)])
def test_gradients_of_entries_with_subnormal_shares(T, V, k, kind):
    """One side's share of an entry below 2^-126, where fp32 has few bits, the other's not: the entry's gradient is the
    greater one's, to its last digits."""
    cuda_or_skip()
    x, ids, values, rest, labels = some(T, V, k)
    values = values.astype(np.float64)
    top = np.log(np.exp(values).sum(1) + np.exp(rest))
    for t in range(T):
        for j in range(min(k, 12)):
            values[t, j] = top[t] - (89, 95, 99, 102.5)[j % 4]
            x[t, ids[t, j]] = x[t, ids[t, 12:]].max() - (20, 40, 70)[j % 3]
        if t % 2:  # the other way round
            values[t, :12], x[t, ids[t, :12]] = top[t] - 30, x[t, ids[t, 12:]].max() - (89 + 3.5 * (np.arange(12) % 4))
    check_far(x, ids, values.astype(np.float32), rest, dtype=F32, far=110, kind=kind, mix=0.4)
