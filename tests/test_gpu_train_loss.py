"""Losses on logits on the GPU against the plain forms in 64 bits.

Tolerances, derived for |logits| <= 40 and rows of at most 2^18 entries.  A row is its maximum m and the sum
s of exp(x - m): s is positive terms, each with 2^-21 (the exponent's roundings and the exponential), added
at most about 100 deep (2^-24 each, in the worst case), so 1e-5 relative bounds s, and lse = m + log s below
64 adds half its spacing, 2e-6.  1e-5 holds both with the deep sums' usual error (ATOL).  A softmax entry
2^((x - m) log2 e - log2 s) carries the error of log s and the exponent's rounding (below 2^-17): 2e-5
relative (PTOL).  What follows from logp carries ATOL by its derivative, and a bf16 gradient adds half a
unit in its last place (2^-8 relative)."""

import numpy as np
import pytest
import torch

import train_ref as R
from gpu_util import cuda_or_skip, new_err
from segmented_gather_gemm_lora_gb300 import binding as B

pytestmark = pytest.mark.gpu

ATOL, PTOL = 1e-5, 2e-5
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
GUARD = 77.0


@pytest.fixture(autouse=True)
def _cuda():
    cuda_or_skip()


def make_logits(rng, T, V, ld, dtype, shift=0, masked=True):
    """(device [T, V] view inside guarded memory, its values in 64 bits): some entries and one row masked."""
    flat = torch.full((T * ld + shift + 16,), GUARD, dtype=DTYPES[dtype], device="cuda")
    x = flat[shift: shift + T * ld].view(T, ld)[:, :V]
    v = np.clip(rng.normal(size=(T, V)) * 4, -40, 40)
    if masked and V > 3:
        v[:, rng.integers(0, V, max(1, V // 50))] = -np.inf
        if T > 2:
            v[T // 2] = -np.inf  # a row whose mask leaves nothing
    x.copy_(torch.from_numpy(v).to(DTYPES[dtype]))
    return flat, x, x.double().cpu().numpy()


def make_labels(rng, x64, skip=0.2):
    """Labels on finite entries where the row has one, some rows not counted."""
    T, V = x64.shape
    lab = rng.integers(0, V, T)
    for t in range(T):
        fine = np.flatnonzero(np.isfinite(x64[t]))
        if fine.size:
            lab[t] = rng.choice(fine)
    lab[rng.random(T) < skip] = -1
    return lab.astype(np.int32)


def dev(a, dtype=np.float32):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=dtype)).cuda()


def close(got, want, tol, what):
    got = np.asarray(got, dtype=np.float64)
    assert np.array_equal(np.isnan(got), np.isnan(want)), what
    inf = np.isinf(want)
    assert np.array_equal(got[inf], want[inf]), what
    err = np.abs(got - want)[np.isfinite(want)]
    bound = np.broadcast_to(tol, np.shape(want))[np.isfinite(want)]
    worst = int(np.argmax(err - bound)) if err.size else 0
    assert (err <= bound).all(), "%s: |err| %.3g above %.3g" % (what, err[worst], bound[worst])


def grad_bound(x64, lse, labels, coef, dcoef, dtype):
    """Bound of |dlogits - exact| per entry: the coefficient's error dcoef [T], PTOL of the softmax."""
    with np.errstate(invalid="ignore", over="ignore"):
        p = np.nan_to_num(np.exp(x64 - lse[:, None]), nan=0.0, posinf=0.0)
    one = np.zeros_like(p)
    ok = (labels >= 0) & (labels < x64.shape[1])
    one[np.flatnonzero(ok), labels[ok]] = 1.0
    c, d = np.abs(coef)[:, None], np.asarray(dcoef)[:, None]
    exact = c * np.abs(one - p)
    # the coefficient's error times the entry, the softmax's and two fp32 roundings of at most c
    b = d * (np.abs(one - p) + PTOL) + c * (p * PTOL + (one + p) * 2.0 ** -22) + 1e-37
    return b + (2.0 ** -8 * (exact + b) if dtype == "bf16" else 0.0)


SIZES = [(1, 1, 1, 0), (3, 2, 2, 1), (5, 7, 9, 3), (4, 8, 8, 0), (6, 33, 40, 5), (2, 1000, 1003, 7), (3, 8192, 8192, 0),
         (1, 32000, 32000, 0), (2, 50257, 50257, 1), (400, 257, 257, 2), (1, 151936, 151936, 4), (700, 2049, 2056, 0)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,V,ld,shift", SIZES)
def test_logprobs(T, V, ld, shift, dtype):
    rng = np.random.default_rng(T * 1000 + V)
    flat, x, x64 = make_logits(rng, T, V, ld, dtype, shift)
    lab = make_labels(rng, x64)
    logp, lse = (torch.full((T,), GUARD, device="cuda") for _ in range(2))
    err = new_err()
    B.lora_token_logprobs(x, dev(lab, np.int32), logp, lse, err=err)
    want_p, want_l = R.logprobs(x64, lab)
    close(logp.cpu().numpy(), want_p, ATOL, "logp")
    close(lse.cpu().numpy(), want_l, ATOL, "lse")
    again = torch.empty_like(logp)
    B.lora_token_logprobs(x, dev(lab, np.int32), again, err=err)  # without lse
    assert torch.equal(logp.view(torch.int32), again.view(torch.int32))
    assert int(err) == 0


def test_logprobs_of_unusual_values():
    """NaN and +inf stay in their row; a bad label sets its bit; nothing visible gives -inf."""
    for V in (12, 5000):
        x64 = np.random.default_rng(0).normal(size=(8, V))
        x64[0, 3] = np.nan
        x64[1, 5] = np.inf
        x64[2] = -np.inf
        x64[3, 1:] = -np.inf
        x64[4] = -3.0e38
        x64[5] = 3.0e38
        x64[6] = -1.0e4
        lab = np.array([1, 2, 0, 0, 3, 4, 5, V], dtype=np.int32)
        x = torch.from_numpy(x64).float().cuda()
        logp, lse, err = torch.empty(8, device="cuda"), torch.empty(8, device="cuda"), new_err()
        B.lora_token_logprobs(x, dev(lab, np.int32), logp, lse, err=err)
        p, s = logp.cpu().numpy(), lse.cpu().numpy()
        assert np.isnan(p[0]) and np.isnan(s[0])
        assert p[1] == -np.inf and s[1] == np.inf
        assert p[2] == -np.inf and s[2] == -np.inf
        assert p[3] == 0 and abs(s[3] - x64[3, 0]) <= ATOL
        assert s[4] <= -2.9e38 and s[5] >= 2.9e38  # fp32 holds no finer difference there
        assert all(abs(p[t] + np.log(V)) <= ATOL for t in (4, 5, 6))
        assert p[7] == 0 and s[7] == 0
        assert int(err) == B.LORA_DERR_BAD_LABEL


def policy_case(seed, T, V, ld, dtype, shift=0):
    rng = np.random.default_rng(seed)
    flat, x, x64 = make_logits(rng, T, V, ld, dtype, shift)
    lab = make_labels(rng, x64)
    lp = np.where(np.isfinite(R.logprobs(x64, lab)[0]), R.logprobs(x64, lab)[0], 0)
    # ratios on both sides of both bounds and none near one (the loss has a corner there)
    old = (lp + rng.choice([-0.6, -0.1, 0.0, 0.1, 0.6], T)).astype(np.float32)
    ref = (lp + 0.3 * rng.normal(size=T)).astype(np.float32)
    adv = rng.normal(size=T).astype(np.float32)
    w = rng.uniform(0.1, 2, T).astype(np.float32)
    if T > 3:
        w[T // 3] = 0
    return rng, flat, x, x64, lab, old, ref, adv, w


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,V,ld,shift", SIZES)
@pytest.mark.parametrize("form", ["apart", "in place", "off the boundary", "no kl", "forward"])
def test_policy(T, V, ld, shift, dtype, form):
    rng, flat, x, x64, lab, old, ref, adv, w = policy_case(T + V, T, V, ld, dtype, shift)
    kl_coef = 0.0 if form == "no kl" else 0.07
    ldd = ld + 3
    out = torch.full((T * ldd + 16,), GUARD, dtype=DTYPES[dtype], device="cuda")
    first = {"off the boundary": (shift + 1) % 8}.get(form, shift)
    d = {"in place": x, "forward": None}.get(form, out[first: first + T * ldd].view(T, ldd)[:, :V])
    logp, loss, kl = (torch.full((T,), GUARD, device="cuda") for _ in range(3))
    err = new_err()
    B.lora_policy_loss(x, dev(lab, np.int32), dev(old), dev(adv), logp, loss, kl, d, ref_logp=None if kl_coef == 0 else dev(ref),
                       weight=dev(w), clip_low=0.2, clip_high=0.3, kl_coef=kl_coef, grad_scale=1.7, err=err)
    e_lp, e_loss, e_kl, e_g, coef = R.policy(x64, lab, old, adv, ref, w, 0.2, 0.3, kl_coef, 1.7)
    on = lab >= 0
    close(logp.cpu().numpy(), e_lp, ATOL, "logp")
    fine = np.isfinite(e_lp)  # rows with nothing visible: ratio 0, no gradient
    q = np.where(on & fine, np.exp(np.where(fine, e_lp, 0) - old.astype(np.float64)), 0)
    gd = np.where(on & fine, np.abs(np.exp(ref.astype(np.float64) - np.where(fine, e_lp, 0))), 0)
    dq = 2e-5 * q * np.abs(adv)  # ATOL by q, the rounding of the difference and of expf
    close(kl.cpu().numpy()[fine], e_kl[fine], ((gd + 1) * 2e-5 + 2.0 ** -22 * np.abs(e_kl) + 1e-7)[fine], "kl")
    close(loss.cpu().numpy()[fine], e_loss[fine], (w * (kl_coef * (gd + 1) * 2e-5 + dq) + 1e-6 * np.abs(e_loss) + 1e-7)[fine],
          "loss")
    if d is not None:
        dcoef = 1.7 * w * (kl_coef * (gd + 1) * 2e-5 + dq) + 1e-6 * np.abs(coef)
        lse = R.logprobs(x64, lab)[1]
        got = d.double().cpu().numpy()
        close(got, e_g, grad_bound(x64, lse, lab, np.where(fine, coef, 0), np.where(fine, dcoef, 0), dtype), "gradient")
        assert not got[~on].any() and (T < 4 or not got[T // 3].any())
        if form == "in place":  # nothing around the rows was written
            x.fill_(GUARD)
            assert bool((flat == GUARD).all())
        else:
            d.fill_(GUARD)
            assert bool((out == GUARD).all())
    assert int(err) == 0


def test_policy_forbidden_label_and_zero_weight():
    """A label whose entry is masked: logp -inf, ratio 0; weight 0 silences a row with an infinite ratio."""
    x = torch.zeros(4, 300, device="cuda")
    x[0, 7] = float("-inf")
    lab, adv = dev([7, 7, 7, 7], np.int32), dev([1.0, 1.0, -1.0, 2.0])
    old = dev([-3.0, -np.inf, -np.inf, -np.inf])
    logp, loss, d = torch.empty(4, device="cuda"), torch.empty(4, device="cuda"), torch.empty(4, 300, device="cuda")
    B.lora_policy_loss(x, lab, old, adv, logp, loss, None, d, weight=dev([1.0, 1.0, 1.0, 0.0]))
    lp, ls, g = logp.cpu().numpy(), loss.cpu().numpy(), d.cpu().numpy()
    assert lp[0] == -np.inf and ls[0] == 0 and not g[0].any()
    assert abs(ls[1] + 1.2) <= 1e-6 and not g[1].any()  # held at 1 + clip_high, outside it
    assert ls[2] == np.inf
    assert ls[3] == 0 and not g[3].any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("low", ["-1e30", "lowest", "-1e4"])
def test_rows_masked_with_large_finite_values(low, dtype):
    """A mask of a large finite value: beside visible entries it weighs nothing, alone it is uniform."""
    V = 4100
    low = torch.finfo(DTYPES[dtype]).min if low == "lowest" else float(low)
    x = torch.full((2, V), low, dtype=DTYPES[dtype], device="cuda")
    x[0, :100] = torch.arange(100, device="cuda").to(x.dtype) / 64
    lab = dev([5, 9], np.int32)
    logp, loss, d = torch.empty(2, device="cuda"), torch.empty(2, device="cuda"), torch.empty_like(x)
    B.lora_policy_loss(x, lab, logp.zero_().clone(), dev([1.0, 1.0]), logp, loss, None, d)
    x64 = x.double().cpu().numpy()
    want, lse = R.logprobs(x64, lab.cpu().numpy())
    close(logp.cpu().numpy()[:1], want[:1], ATOL, "logp")
    assert abs(float(logp[1]) + np.log(V)) <= ATOL
    p = np.zeros((2, V))
    p[0, :100] = np.exp(x64[0, :100] - lse[0])
    p[1] = 1 / V
    coef = -np.exp([want[0], -np.log(V)])
    g = -coef[:, None] * p
    g[[0, 1], [5, 9]] += coef
    tol = np.abs(coef)[:, None] * p * 2 * PTOL + 1e-9 + (2.0 ** -8 * np.abs(g) if dtype == "bf16" else 0)
    tol[[0, 1], [5, 9]] += np.abs(coef) * 2 * PTOL
    close(d.double().cpu().numpy(), g, tol, "gradient")


def sequences(rng, T, n):
    cuts = np.sort(rng.integers(0, T + 1, 2 * n + 1))  # empty sequences and rows of no sequence among them
    return cuts.astype(np.int32)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["sigmoid", "hinge", "ipo"])
@pytest.mark.parametrize("average", [False, True])
@pytest.mark.parametrize("T,V,ld,shift,n", [(1, 5, 5, 0, 1), (40, 33, 40, 1, 3), (300, 257, 257, 2, 40), (9, 50257, 50257, 3, 2),
                                            (600, 1000, 1000, 0, 1), (4, 32000, 32000, 0, 2)])
def test_preference(T, V, ld, shift, n, kind, average, dtype):
    rng = np.random.default_rng(T + V + n)
    flat, x, x64 = make_logits(rng, T, V, ld, dtype, shift, masked=False)
    x[:, 1::97] = float("-inf")
    x64 = x.double().cpu().numpy()
    lab = make_labels(rng, x64)
    ref = (R.logprobs(x64, lab)[0] + 0.2 * rng.normal(size=T)).astype(np.float32)
    indptr = sequences(rng, T, n)
    beta, smooth, margin, gs = 0.1, 0.15, 0.05, 0.5
    e_loss, e_seq, e_g, coef = R.preference(x64, lab, ref, indptr, kind, beta, smooth, margin, average, gs)
    loss, seq = torch.full((n,), GUARD, device="cuda"), torch.full((2 * n,), GUARD, device="cuda")
    ws, err = B.preference_workspace(T, n), new_err()
    out = torch.full((T, V), GUARD, dtype=DTYPES[dtype], device="cuda")
    kw = dict(ref_logp=dev(ref), kind=getattr(B, "LORA_PREF_" + kind.upper()), beta=beta, label_smoothing=smooth, margin=margin,
              average=average, grad_scale=gs, err=err)
    args = (x, dev(lab, np.int32), dev(indptr, np.int32), loss, seq)
    B.lora_preference_loss(*args, out, ws, **kw)
    counts = np.array([((lab >= 0)[a:b]).sum() for a, b in zip(indptr, indptr[1:])])
    close(seq.cpu().numpy(), e_seq, ATOL * np.maximum(counts, 1) + 2.0 ** -23 * np.abs(e_seq), "seq_logp")
    # a pair's difference: ATOL for each counted row (or their mean); its derivative bounds the loss and slope
    dD = np.array([ATOL * (2 if average else counts[2 * p] + counts[2 * p + 1]) for p in range(n)]) + 1e-6
    D = np.sqrt(np.maximum(e_loss, 0)) + 0.5 / beta if kind == "ipo" else None
    slope = 2 * np.sqrt(e_loss) if kind == "ipo" else np.full(n, beta)
    close(loss.cpu().numpy(), e_loss, slope * dD + dD * dD + 1e-6 * (1 + np.abs(e_loss)) + (1e-6 * slope * D if D is not None else 0),
          "loss")
    curve = 2.0 if kind == "ipo" else beta * beta / 4 if kind == "sigmoid" else 0.0
    dcoef, lse = np.zeros(T), R.logprobs(x64, lab)[1]
    for p in range(n):
        for s in (2 * p, 2 * p + 1):
            share = 1.0 / counts[s] if average and counts[s] else 1.0
            dcoef[indptr[s]: indptr[s + 1]] = gs * share * (curve * dD[p] + (1e-6 * 2 * D[p] if D is not None else 0))
    dcoef = dcoef + 1e-6 * np.abs(coef)
    bound = grad_bound(x64, lse, lab, coef, dcoef, dtype)
    close(out.double().cpu().numpy(), e_g, bound, "gradient")
    # the gradient in the logits' place, and the loss alone, give the same bits
    loss2 = torch.empty_like(loss)
    B.lora_preference_loss(x, args[1], args[2], loss2, None, None, ws, **kw)
    assert torch.equal(loss, loss2)
    B.lora_preference_loss(x, args[1], args[2], loss2, None, x, ws, **kw)
    assert torch.equal(loss, loss2) and torch.equal(x, out)
    x.fill_(GUARD)
    assert bool((flat == GUARD).all())
    assert int(err) == 0


@pytest.mark.parametrize("bad", [[0, 4, 2], [0, 4, 21], [-1, 4, 8], [5, 3, 2]])
def test_preference_bad_offsets(bad):
    x = torch.randn(20, 300, device="cuda")
    lab = torch.zeros(20, dtype=torch.int32, device="cuda")
    indptr = dev(bad, np.int32)
    loss, seq = torch.full((1,), GUARD, device="cuda"), torch.full((2,), GUARD, device="cuda")
    d, err = torch.full_like(x, GUARD), new_err()
    B.lora_preference_loss(x, lab, indptr, loss, seq, d, B.preference_workspace(20, 1), err=err)
    assert int(err) == B.LORA_DERR_BAD_SEQ
    assert not loss.any() and not seq.any() and not d.any()


def test_preference_extremes():
    """Infinite differences keep a finite gradient; a term of weight 0 does not turn them into NaN."""
    x = torch.zeros(4, 64, device="cuda")
    x[0, 5] = x[3, 5] = float("-inf")
    lab, indptr = dev([5, 5, 5, 5], np.int32), dev([0, 1, 2, 3, 4], np.int32)
    loss, d = torch.empty(2, device="cuda"), torch.empty_like(x)
    B.lora_preference_loss(x, lab, indptr, loss, None, d, B.preference_workspace(4, 2), beta=0.5)
    ls, g = loss.cpu().numpy(), d.cpu().numpy()
    assert ls[0] == np.inf and ls[1] == 0
    assert np.isfinite(g).all() and g[0, 5] == -0.5 and not g[2:].any()


def test_no_pairs_clears_the_gradient():
    x, d = torch.randn(5, 40, device="cuda"), torch.full((5, 40), GUARD, device="cuda")
    B.lora_preference_loss(x, torch.zeros(5, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda"),
                           torch.empty(0, device="cuda"), None, d, B.preference_workspace(5, 0))
    assert not d.any()


def test_gradient_against_differences_of_the_loss():
    """The kernel's own fp32 loss, moved along a direction by +-h: h^2 times a third derivative below 1 and
    fp32 noise of 4 * ATOL over 2 h, h = 0.05."""
    rng = np.random.default_rng(5)
    T, V, h = 24, 120, 0.05
    x = torch.from_numpy(rng.normal(size=(T, V))).float().cuda()
    lab = dev(rng.integers(0, V, T), np.int32)
    step = torch.from_numpy(rng.normal(size=(T, V)) / np.sqrt(T * V)).float().cuda()
    ws, loss, d = B.preference_workspace(T, 2), torch.empty(2, device="cuda"), torch.empty_like(x)
    indptr = dev([0, 6, 12, 18, 24], np.int32)

    def total(y, grad=None):
        B.lora_preference_loss(y, lab, indptr, loss, None, grad, ws, beta=0.5, label_smoothing=0.1)
        return float(loss.double().sum())

    total(x, d)
    slope = float((d.double() * step.double()).sum())
    num = (total(x + h * step) - total(x - h * step)) / (2 * h)
    assert abs(num - slope) <= h * h + 4 * ATOL / (2 * h)


def test_rows_past_32_bits():
    """Row offsets above 2^31 elements."""
    V, ld = 700, 1 << 30
    flat = torch.empty(2 * ld + 8192, dtype=torch.bfloat16, device="cuda")
    x = flat[: 2 * ld + V].as_strided((3, V), (ld, 1))
    x.copy_(torch.randn(3, V, device="cuda"))
    lab = dev([3, 699, 0], np.int32)
    args = [dev(np.zeros(3)), dev(np.ones(3))]
    logp, loss = torch.empty(3, device="cuda"), torch.empty(3, device="cuda")
    d = torch.empty(3, V, dtype=torch.bfloat16, device="cuda")
    c = torch.empty(3, 704, dtype=torch.bfloat16, device="cuda")[:, :V]  # rows aligned as those of x
    c.copy_(x)
    B.lora_policy_loss(x, lab, *args, logp, loss, None, d)
    logp2, loss2, d2 = torch.empty_like(logp), torch.empty_like(loss), torch.empty_like(d)
    B.lora_policy_loss(c, lab, *args, logp2, loss2, None, d2)
    assert torch.equal(d, d2) and torch.equal(logp, logp2) and torch.equal(loss, loss2)


def test_other_stream_and_graph():
    rng, flat, x, x64, lab, old, ref, adv, w = policy_case(9, 50, 3001, 3001, "bf16")
    labels, d_old, d_adv = dev(lab, np.int32), dev(old), dev(adv)
    logp, loss, d = torch.empty(50, device="cuda"), torch.empty(50, device="cuda"), torch.empty_like(x)
    B.lora_policy_loss(x, labels, d_old, d_adv, logp, loss, None, d)
    torch.cuda.synchronize()
    want = [t.clone() for t in (logp, loss, d)]
    s = torch.cuda.Stream()
    for t in (logp, loss, d):
        t.zero_()
    s.wait_stream(torch.cuda.current_stream())
    B.lora_policy_loss(x, labels, d_old, d_adv, logp, loss, None, d, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((logp, loss, d), want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.lora_policy_loss(x, labels, d_old, d_adv, logp, loss, None, d)
    for t in (logp, loss, d):
        t.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((logp, loss, d), want))


@pytest.mark.parametrize("dtype,V", [("bf16", 500009), ("f32", 262147), ("bf16", 303110), ("f32", 151940)])
def test_rows_longer_than_a_clusters_shared_memory(dtype, V):
    """The longest rows that are staged in shared memory, and rows that are not."""
    rng = np.random.default_rng(V)
    flat, x, x64 = make_logits(rng, 2, V, V + 3, dtype, 1, masked=False)
    lab = np.array([V - 1, 17], dtype=np.int32)
    want, lse = R.logprobs(x64, lab)
    logp, loss, d = torch.empty(2, device="cuda"), torch.empty(2, device="cuda"), torch.empty_like(x)
    old = dev(want)
    B.lora_policy_loss(x, dev(lab, np.int32), old, dev([1.0, -1.0]), logp, loss, None, d)
    close(logp.cpu().numpy(), want, 2 * ATOL, "logp")  # twice as many terms a thread
    coef = np.array([-1.0, 1.0])
    bound = grad_bound(x64, lse, lab, coef, np.full(2, 3e-5), dtype)
    close(d.double().cpu().numpy(), R.softmax_grad(x64, lab, lse, coef), bound, "gradient")
    B.lora_policy_loss(x, dev(lab, np.int32), old, dev([1.0, -1.0]), logp, loss, None, x)
    assert torch.equal(x, d)


def test_timeout_leaves_the_outputs():
    """With the timeout probe armed every row gives up after about a millisecond, sets its bit and writes
    nothing; the next calls are right."""
    x = torch.randn(6, 9000, device="cuda")
    lab = torch.zeros(6, dtype=torch.int32, device="cuda")
    f = torch.zeros(6, device="cuda")
    logp, loss, pair = (torch.full((6,), GUARD, device="cuda") for _ in range(3))
    d, ws, err = torch.full_like(x, GUARD), B.preference_workspace(6, 1), new_err()
    indptr = dev([0, 3, 6], np.int32)

    def calls():
        B.lora_token_logprobs(x, lab, logp, err=err)
        B.lora_policy_loss(x, lab, f, f, logp, loss, None, d, err=err)
        B.lora_preference_loss(x, lab, indptr, pair[:1], None, d, ws, err=err)

    try:
        B.debug_wait_probe(2_000_000)
        calls()
        torch.cuda.synchronize()
    finally:
        B.debug_wait_probe(0)
    assert int(err) == B.LORA_DERR_TIMEOUT
    assert bool((logp == GUARD).all()) and bool((loss == GUARD).all()) and bool((d == GUARD).all())
    assert float(pair[0]) == GUARD
    err.zero_()
    calls()
    assert int(err) == 0
    want = torch.log_softmax(x.double(), 1)[:, 0]
    assert float((logp.double() - want).abs().max()) <= ATOL


def policy64(x, lab, old, adv, ref, w, lo, hi, kl_coef, scale):
    """(logp, loss, kl, gradient, coefficient) of the policy loss in 64 bits on the GPU (rows with visible labels)."""
    x, on = x.double(), lab >= 0
    at = lab.long().clamp(min=0)[:, None]
    lse = torch.logsumexp(x, 1)
    lp = torch.where(on, x.gather(1, at)[:, 0] - lse, torch.zeros_like(lse))
    q, d, a = torch.exp(lp - old.double()), ref.double() - lp, adv.double()
    first, held = q * a, q.clamp(1 - lo, 1 + hi) * a
    kl = torch.expm1(d) - d
    loss = w.double() * (kl_coef * kl - torch.minimum(first, held))
    coef = -scale * w.double() * (kl_coef * torch.expm1(d) + torch.where(first <= held, first, torch.zeros_like(first)))
    coef = torch.where(on, coef, torch.zeros_like(coef))
    g = -coef[:, None] * torch.exp(x - lse[:, None])
    g.scatter_add_(1, at, coef[:, None])
    g = torch.where(on[:, None], g, torch.zeros_like(g))
    zero = torch.zeros_like(lp)
    return lp, torch.where(on, loss, zero), torch.where(on, kl, zero), g, coef, lse, q, torch.exp(d)


# row lengths and counts on both sides of every change of the kernels' form
FORMS = [(400, 1020), (400, 1030), (290, 3001), (400, 3001), (400, 4100), (400, 8001), (400, 8203), (400, 12003), (400, 16400),
         (60, 20000), (150, 20000), (330, 20000), (20, 50257), (400, 50257), (310, 128256), (320, 65600)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,V", FORMS)
@pytest.mark.parametrize("shift", [0, 3])
def test_policy_forms(T, V, shift, dtype):
    """Every form of the row kernels over many rows, aligned and not, apart and in place, with the same bits
    twice."""
    g = torch.Generator(device="cuda").manual_seed(T + V)
    ld = V + (-V % 8 if shift == 0 else 5)
    flat = torch.full((T * ld + 32,), GUARD, dtype=DTYPES[dtype], device="cuda")
    x = flat[shift: shift + T * ld].view(T, ld)[:, :V]
    x.copy_((torch.randn(T, V, generator=g, device="cuda") * 3).clamp(-30, 30))
    lab = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
    lab[torch.rand(T, generator=g, device="cuda") < 0.2] = -1
    lp = torch.log_softmax(x.float(), 1).gather(1, lab.long().clamp(min=0)[:, None])[:, 0]
    pick = torch.tensor([-0.6, -0.1, 0.0, 0.1, 0.6], device="cuda")[torch.randint(0, 5, (T,), generator=g, device="cuda")]
    old, ref = lp + pick, lp + 0.3 * torch.randn(T, generator=g, device="cuda")
    adv, w = torch.randn(T, generator=g, device="cuda"), 0.1 + torch.rand(T, generator=g, device="cuda")
    e_lp, e_loss, e_kl, e_g, coef, lse, q, ed = policy64(x, lab, old, adv, ref, w, 0.2, 0.3, 0.07, 1.3)
    logp, loss, kl = (torch.full((T,), GUARD, device="cuda") for _ in range(3))
    d, err = torch.full((T, V), GUARD, dtype=DTYPES[dtype], device="cuda"), new_err()
    kw = dict(ref_logp=ref, weight=w, clip_low=0.2, clip_high=0.3, kl_coef=0.07, grad_scale=1.3, err=err)
    B.lora_policy_loss(x, lab, old, adv, logp, loss, kl, d, **kw)
    assert float((logp - e_lp).abs().max()) <= ATOL
    dq = 2e-5 * q * adv.abs().double()
    dk = 0.07 * (ed + 1) * 2e-5
    on = lab >= 0
    assert bool(((loss - e_loss).abs() <= w * (dk + dq) + 1e-6 * e_loss.abs() + 1e-7)[on].all())
    assert bool(((kl - e_kl).abs() <= (ed + 1) * 2e-5 + 2.0 ** -22 * e_kl + 1e-7)[on].all())
    assert not loss[~on].any() and not kl[~on].any() and not logp[~on].any() and not d[~on].any()
    c = coef.abs()[:, None]
    p = torch.exp(x.double() - lse[:, None])
    dc = (1.3 * w.double() * (dk + dq) + 1e-6 * coef.abs())[:, None]
    one = torch.zeros_like(p).scatter_(1, lab.long().clamp(min=0)[:, None], 1.0)
    bound = dc * ((one - p).abs() + PTOL) + c * (p * PTOL + (one + p) * 2.0 ** -22) + 1e-37
    if dtype == "bf16":
        bound = bound + 2.0 ** -8 * (e_g.abs() + bound)
    assert bool(((d.double() - e_g).abs() <= bound)[on].all())
    again, logp2 = torch.empty_like(d), torch.empty_like(logp)
    B.lora_policy_loss(x, lab, old, adv, logp2, loss, kl, again, **kw)
    assert torch.equal(again, d) and torch.equal(logp2, logp)
    B.lora_policy_loss(x, lab, old, adv, logp2, loss, kl, x, **kw)
    if shift == 0:
        assert torch.equal(x, d)
    else:  # another store path, the same values
        assert torch.equal(x, d) and torch.equal(logp2, logp)
    x.fill_(GUARD)
    assert bool((flat == GUARD).all())
    assert int(err) == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,V,n", [(128, 9001, 3), (129, 9001, 3), (100, 9000, 64), (100, 9000, 65), (8, 40000, 4), (400, 50257, 6)])
def test_preference_forms(T, V, n, dtype):
    """Few and many rows, sequences without rows: loss, sums and gradient against 64 bits on the GPU."""
    g = torch.Generator(device="cuda").manual_seed(T + V + n)
    rng = np.random.default_rng(n)
    x = (torch.randn(T, V, generator=g, device="cuda") * 3).to(DTYPES[dtype])
    lab = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
    lab[torch.rand(T, generator=g, device="cuda") < 0.3] = -1
    indptr = sequences(rng, T, n)
    indptr[2] = indptr[0]  # the first pair has no rows
    indptr[1] = indptr[0]
    indptr[-1] = T
    x64 = x.double()
    lse = torch.logsumexp(x64, 1)
    at = lab.long().clamp(min=0)[:, None]
    on = lab >= 0
    lp = torch.where(on, x64.gather(1, at)[:, 0] - lse, torch.zeros_like(lse))
    ref = (lp + 0.2 * torch.randn(T, generator=g, device="cuda")).float()
    gap = torch.where(on, lp - ref.double(), torch.zeros_like(lp))
    loss, seq, err = torch.full((n,), GUARD, device="cuda"), torch.full((2 * n,), GUARD, device="cuda"), new_err()
    d = torch.full_like(x, GUARD)
    B.lora_preference_loss(x, lab, dev(indptr, np.int32), loss, seq, d, B.preference_workspace(T, n), ref_logp=ref, beta=0.1,
                           grad_scale=2.0, err=err)
    coef = torch.zeros_like(lp)
    for p in range(n):
        i0, i1, i2 = (int(v) for v in indptr[2 * p: 2 * p + 3])
        z = 0.1 * float(gap[i0:i1].sum() - gap[i1:i2].sum())
        counted = int(on[i0:i2].sum())
        assert abs(float(loss[p]) - np.log1p(np.exp(-z))) <= 0.1 * ATOL * counted + 1e-6 * (1 + abs(z))
        for s, (a, b) in enumerate(((i0, i1), (i1, i2))):
            assert abs(float(seq[2 * p + s]) - float(lp[a:b].sum())) <= ATOL * max(1, int(on[a:b].sum())) + 2.0 ** -23 * abs(float(lp[a:b].sum()))
        slope = -0.1 * 2.0 / (1 + np.exp(z))
        coef[i0:i1], coef[i1:i2] = slope, -slope
    coef = torch.where(on, coef, torch.zeros_like(coef))
    p = torch.exp(x64 - lse[:, None])
    e_g = -coef[:, None] * p
    e_g.scatter_add_(1, at, coef[:, None])
    one = torch.zeros_like(p).scatter_(1, at, 1.0)
    c = coef.abs()[:, None]
    bound = c * 1e-6 + 2.0 * 0.0025 * ATOL * T * (one + p) + c * (p * PTOL + (one + p) * 2.0 ** -22) + 1e-37
    if dtype == "bf16":
        bound = bound + 2.0 ** -8 * (e_g.abs() + bound)
    err_g = (d.double() - torch.where(on[:, None], e_g, torch.zeros_like(e_g))).abs()
    assert bool((err_g <= bound).all())
    assert int(err) == 0


def test_preference_bad_offsets_of_long_rows():
    x = torch.randn(20, 9000, device="cuda")
    lab = torch.zeros(20, dtype=torch.int32, device="cuda")
    loss, seq = torch.full((2,), GUARD, device="cuda"), torch.full((4,), GUARD, device="cuda")
    d, err = torch.full_like(x, GUARD), new_err()
    B.lora_preference_loss(x, lab, dev([0, 5, 10, 8, 20], np.int32), loss, seq, d, B.preference_workspace(20, 2), err=err)
    assert int(err) == B.LORA_DERR_BAD_SEQ
    assert not loss.any() and not seq.any() and not d.any()


@pytest.mark.parametrize("T,V", [(6, 100), (6, 3000), (400, 3000), (6, 40000), (400, 40000), (2, 600000)])
def test_nan_logits_show_in_their_row_alone(T, V):
    """A NaN among the logits makes its row's loss and gradient NaN (so the gradient norm skips the adapter)
    and leaves the other rows as they are; in a pair it reaches the pair's rows and no other's."""
    x = torch.randn(T, V, device="cuda")
    lab = torch.arange(T, dtype=torch.int32, device="cuda") % V
    old, adv = torch.full((T,), -8.0, device="cuda"), torch.ones(T, device="cuda")
    adv[T // 2:] = -1.0
    outs = []
    for bad in (False, True):
        if bad:
            x[1, V // 3] = float("nan")
        logp, loss, d = torch.empty(T, device="cuda"), torch.empty(T, device="cuda"), torch.empty_like(x)
        B.lora_policy_loss(x, lab, old, adv, logp, loss, None, d)
        outs.append((logp, loss, d))
    keep = torch.arange(T, device="cuda") != 1
    for good, bad in zip(*outs):
        assert torch.equal(good[keep], bad[keep])
        assert bool(torch.isnan(bad[1]).all())
    if T >= 4:
        n = 2
        indptr = dev([0, 1, T // 2, T // 2 + 1, T], np.int32)
        loss, d = torch.empty(n, device="cuda"), torch.empty_like(x)
        B.lora_preference_loss(x, lab, indptr, loss, None, d, B.preference_workspace(T, n), beta=0.01)
        assert np.isnan(float(loss[0])) and np.isfinite(float(loss[1]))
        assert bool(torch.isnan(d[: T // 2]).all()) and bool(torch.isfinite(d[T // 2:]).all())
