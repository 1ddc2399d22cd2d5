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
    listed entries' and `far`, those of the rest) and of a sum's logarithm below 16, and by the sums' errors (2^-19);
    kd's derivative with respect to one is p - q, a term's own arithmetic is off by 2^-18 of it; a gradient's parts move
    by as much of themselves, four of them, and are rounded once."""
    loss, kd, ce, grad = run_loss(x, ids, values, tail, labels, dtype=dtype, **kw)
    x = device(x, dtype)[2]
    want = R.distill(x, ids, values.astype(np.float32).astype(np.float64), tail, labels, **kw)
    d = 3 * 2.0 ** -24 * (want["spread"] + far + 16) + 2.0 ** -19
    for name, got in (("kd", kd), ("ce", ce), ("loss", loss)):
        w = want[name]
        with np.errstate(invalid="ignore"):
            assert np.array_equal(got[~np.isfinite(w)], w[~np.isfinite(w)]), (name, got, w)
            scale = kw.get("kd_weight", 1.0) + kw.get("ce_weight", 0.0) if name == "loss" else 1.0
            tol = scale * 2 * d + 2.0 ** -18 * np.abs(w) + 1e-37
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
