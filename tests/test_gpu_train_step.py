"""The optimizer step over paged adapters on the GPU against the plain form in 64 bits.

Tolerances, derived for fp32 arithmetic (unit e = 2^-24) on the same inputs:
* the clipped gradient: c from sumsq, whose sum is 32 squares a thread deep and a tree, 3e-6, so g carries
  GREL = 4e-6; without clipping its product's e (within GREL);
* m and v: two products and a sum, 3 e of each term, and GREL (twice for g^2) of the new term;
* the weights: |w| 2 e, and of the update 2e-6 (bias corrections, root, quotients) with m's and v's errors;
* a code: half the distance of e4m3 neighbours at the value (2^-4 relative, 2^-10 of the scale below the
  normal range; the whole 2^-9 for a root that is kept from 0), and a scale: half a bf16 unit (2^-8 relative
  to the value it rounds), each with the error of what is rounded;
* a bf16 weight: half a unit, 2^-8 relative."""

import numpy as np
import pytest
import torch

import train_ref as R
from gpu_util import cuda_or_skip, new_err
from segmented_gather_gemm_lora_gb300 import binding as B
from segmented_gather_gemm_lora_gb300 import workloads as W

pytestmark = pytest.mark.gpu

E, GREL = 2.0 ** -24, 4e-6


@pytest.fixture(autouse=True)
def _cuda():
    cuda_or_skip()


class Setup:
    """One projection's pool and state with NaN (or code 0x7f) everywhere that no adapter owns."""

    def __init__(self, seed, d_in, d_out, ranks, page, state="f32", master=False, max_rank=None):
        rng = np.random.default_rng(seed)
        self.pool = W.build_pool(rng, d_in, d_out, ranks, page_elems=page, max_rank=max_rank)
        self.view = B.PoolView.from_host(self.pool)
        n = self.pool.pool.size
        self.own = np.zeros(n, dtype=bool)
        for i, r in enumerate(ranks):
            if r > 0:
                for q in R.positions(self.pool, i):
                    self.own[q] = True
        nan = np.where(self.own, 0, np.nan).astype(np.float32)
        level = np.repeat(np.exp(rng.normal(size=n // 64)) * 1e-3, 64)
        f = lambda a: (a + nan).astype(np.float32)  # noqa: E731
        self.g = f(rng.normal(size=n) * level)
        self.m = f(rng.normal(size=n) * level * 0.3)
        self.v = f((rng.uniform(0.5, 1.5, n) * level) ** 2)
        self.w = W.bf16_bits_to_f32(self.pool.pool.reshape(-1)).astype(np.float32) + nan
        if master:
            self.w = f(self.w * (1 + 2.0 ** -10 * rng.uniform(-1, 1, n)))
        dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
        self.state, self.master = state, master
        if state == "f32":
            t = B.TrainProj(self.view, dev(self.g), dev(self.m), dev(self.v), master=dev(self.w) if master else None)
        else:
            self.mc, self.vc = (np.where(self.own, c, 0x7F).astype(np.uint8) for c in
                                (rng.integers(0, 0x7F, n) | (rng.integers(0, 2, n) << 7), rng.integers(1, 0x7F, n)))
            self.ms, self.vs = (R.bf16_round(np.exp(rng.normal(size=n // 64)) * s) for s in (1e-6, 1e-5))
            code = lambda a: dev(a).view(torch.float8_e4m3fn)  # noqa: E731
            bf = lambda a: dev(a.astype(np.float32)).bfloat16()  # noqa: E731
            t = B.TrainProj(self.view, dev(self.g), code(self.mc), code(self.vc), master=dev(self.w) if master else None,
                            m_scale=bf(self.ms), v_scale=bf(self.vs))
            self.m = np.where(self.own, R.decode_e4m3(self.mc) * np.repeat(self.ms, 64), np.nan)
            self.v = np.where(self.own, (R.decode_e4m3(self.vc) * np.repeat(self.vs, 64)) ** 2, np.nan)
        self.t = t

    def host(self):
        """Every array's bits as they are now."""
        t = self.t
        out = {"pool": self.view.pool.view(torch.int16), "grad": t.grad.view(torch.int32)}
        kind = torch.int32 if self.state == "f32" else torch.uint8
        out.update(m=t.m.view(kind), v=t.v.view(kind))
        if self.master:
            out["master"] = t.master.view(torch.int32)
        if self.state != "f32":
            out.update(m_scale=t.m_scale.view(torch.int16), v_scale=t.v_scale.view(torch.int16))
        return {k: x.flatten().cpu().numpy().copy() for k, x in out.items()}


def settings(n, seed, **kw):
    rng = np.random.default_rng(seed)
    h = dict(step=rng.integers(1, 3000, n), lr=rng.uniform(1e-5, 1e-3, n), beta1=rng.choice([0.0, 0.9, 0.95], n),
             beta2=rng.choice([0.99, 0.999], n), eps=np.full(n, 1e-8), weight_decay=rng.choice([0.0, 0.1], n),
             max_norm=np.zeros(n), grad_scale=rng.uniform(0.2, 2.0, n))
    h.update({k: np.broadcast_to(v, n) for k, v in kw.items()})
    return {k: v if k == "step" else v.astype(np.float32) for k, v in h.items()}


def one(h, i):
    return {k: float(v[i]) for k, v in h.items()}


def check_adapter(s, before, after, i, h, sumsq, zero):
    """Adapter i of a Setup against the 64-bit step; its positions."""
    P = R.positions(s.pool, i)
    gs = [s.g[q].astype(np.float64) for q in P]
    for q, g0 in zip(P, gs):
        w0, m0, v0 = (a[q].astype(np.float64) for a in (s.w, s.m, s.v))
        w, m, v, c = R.adamw(w0, g0, m0, v0, h, sumsq)
        g = np.abs(g0 * h["grad_scale"] * c)
        n1, n2 = 1 - h["beta1"], 1 - h["beta2"]
        em = 3 * E * (np.abs(h["beta1"] * m0) + n1 * g) + GREL * n1 * g + 1e-44
        ev = 3 * E * (v + n2 * g * g) + 2 * GREL * n2 * g * g + 1e-44
        c1, c2 = 1 - h["beta1"] ** h["step"], 1 - h["beta2"] ** h["step"]
        root = np.sqrt(v / c2) + h["eps"]
        up = h["lr"] / c1 * np.abs(m) / root
        ew = 2 * E * np.abs(w0) + up * (2e-6 + ev / np.maximum(v, 1e-300)) + h["lr"] / c1 * em / root
        got_w = after["pool"][q].view(np.uint16).astype(np.uint32) << 16
        err = np.abs(got_w.view(np.float32).astype(np.float64) - w)
        assert (err <= ew + 2.0 ** -8 * (np.abs(w) + ew)).all(), "pool: %.3g" % err.max()
        if s.master:
            err = np.abs(after["master"][q].view(np.float32).astype(np.float64) - w)
            assert (err <= ew).all(), "master: %.3g" % np.max(err / ew)
            assert np.array_equal(got_w, (W.f32_to_bf16_bits(after["master"][q].view(np.float32)).astype(np.uint32) << 16))
        if s.state == "f32":
            for k, want, tol in (("m", m, em), ("v", v, ev)):
                err = np.abs(after[k][q].view(np.float32).astype(np.float64) - want)
                assert (err <= tol).all(), "%s: %.3g of its bound" % (k, np.max(err / tol))
        else:
            er = np.where(v > 0, ev / np.maximum(2 * np.sqrt(v), 1e-300), 0) + E * np.sqrt(v)
            for k, want, tol in (("m", m, em), ("v", np.sqrt(v), er)):
                pad = -len(q) % 64
                blocks = lambda a: np.pad(a, (0, pad)).reshape(-1, 64)  # noqa: E731
                top = np.abs(blocks(want)).max(1)
                sc = (after[k + "_scale"][q[::64] // 64].view(np.uint16).astype(np.uint32) << 16).view(np.float32)
                small = top < 2.0 ** -100
                assert (np.abs(sc - top / 448)[~small] <= (top / 448 * (2.0 ** -8 + 1e-5) + blocks(tol).max(1) / 448)[~small]).all()
                assert not sc[small].any()
                each = np.repeat(sc.astype(np.float64), 64)[: len(q)]
                got = R.decode_e4m3(after[k][q]) * each
                half = np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10 * each)
                if k == "v":
                    assert ((got > 0) | (want < 2.0 ** -100)).all(), "a root was rounded to zero"
                    half = np.maximum(half, 2.0 ** -9 * each)
                # the largest of a block may round past 448 times a scale that was rounded down: 2^-8
                err = np.abs(got - want)
                assert (err <= half + 2.0 ** -8 * np.abs(want) * (np.abs(want) > 447 * each) + tol + 1e-44).all(), k
        assert np.array_equal(after["grad"][q], np.zeros_like(after["grad"][q]) if zero else before["grad"][q])
    return np.concatenate(P)


def untouched(s, before, after, positions):
    """Nothing outside the given pool positions changed, bit for bit."""
    moved = np.zeros(s.own.size, dtype=bool)
    if len(positions):
        moved[np.concatenate(positions)] = True
    blocks = moved.reshape(-1, 64).any(1)
    for k in before:
        keep = ~blocks if k.endswith("_scale") else ~moved
        assert np.array_equal(before[k][keep], after[k][keep]), k


def ids_of(ids):
    return torch.tensor(list(ids), dtype=torch.int32, device="cuda")


# widths that end a matrix inside a page, inside a block of 64 and on their boundaries
GEOMETRY = [(256, 256, [8, 8], 64), (1000, 2056, [1, 13, 0, 5], 64), (4096, 328, [64, 1, 16], 4096), (8, 8, [1, 3], 64),
            (4104, 1016, [7, 33], 512), (2048, 2048, [16], 1 << 20)]


@pytest.mark.parametrize("d_in,d_out,ranks,page", GEOMETRY)
@pytest.mark.parametrize("state", ["f32", "e4m3"])
@pytest.mark.parametrize("master", [False, True])
@pytest.mark.parametrize("clip,zero", [(False, False), (True, True)])
def test_step(d_in, d_out, ranks, page, state, master, clip, zero):
    s = Setup(d_in + d_out, d_in, d_out, ranks, page, state, master, max_rank=64)
    ts = B.TrainSet([s.t])
    n = len(ranks)
    h = settings(n, 3, max_norm=[1e-3, 1e3, 1e-2, 0.0][:n] if clip else 0.0)
    listed = [i for i in reversed(range(n)) if ranks[i] > 0 and (n < 3 or i != 1)]  # one adapter left out where there are several
    ids, err = ids_of(listed), new_err()
    sumsq = torch.full((n,), 7.0, device="cuda")
    before = s.host()
    if clip:
        B.lora_grad_sumsq(ts, ids, sumsq, ts.sumsq_workspace(len(listed)), err=err)
        got = sumsq.cpu().numpy()
        for i in range(n):
            if i in listed:
                want = sum(float((s.g[q].astype(np.float64) ** 2).sum()) for q in R.positions(s.pool, i))
                assert abs(got[i] - want) <= 3e-6 * want
            else:
                assert got[i] == 7.0
    B.lora_adamw_step(ts, ids, B.adamw_hyper(n, **h), sumsq=sumsq if clip else None, zero_grad=zero, err=err)
    after = s.host()
    assert int(err) == 0
    where = []
    for i in listed:
        total = sum(float((s.g[q].astype(np.float64) ** 2).sum()) for q in R.positions(s.pool, i)) if clip else None
        where.append(check_adapter(s, before, after, i, one(h, i), total, zero))
    untouched(s, before, after, where)


def test_many_projections_in_one_call_and_repeatability():
    """More projections than one launch takes; norms over all of them, accumulated or at once; the same
    bits from the same state."""
    shapes = [(64 * (1 + g % 3), 128, 64 << (g % 3)) for g in range(19)]
    runs = []
    for _ in range(2):
        sets = [Setup(g, a, b, [4, 0, 9], p, "e4m3" if g < 0 else "f32", True, max_rank=16) for g, (a, b, p) in enumerate(shapes)]
        ts, ids, err = B.TrainSet([s.t for s in sets]), ids_of([2, 0]), new_err()
        h = settings(3, 1, max_norm=1e-2)
        sumsq, other = torch.zeros(3, device="cuda"), torch.zeros(3, device="cuda")
        B.lora_grad_sumsq(ts, ids, sumsq, ts.sumsq_workspace(2), err=err)
        for k, part in enumerate((B.TrainSet([s.t for s in sets[:5]]), B.TrainSet([s.t for s in sets[5:]]))):
            B.lora_grad_sumsq(part, ids, other, part.sumsq_workspace(2), accumulate=k > 0, err=err)
        want = [sum(float((s.g[q].astype(np.float64) ** 2).sum()) for s in sets for q in R.positions(s.pool, i)) for i in (0, 2)]
        assert np.allclose(sumsq[[0, 2]].cpu().numpy(), want, rtol=3e-6) and np.allclose(other[[0, 2]].cpu().numpy(), want, rtol=3e-6)
        before = [s.host() for s in sets]
        B.lora_adamw_step(ts, ids, B.adamw_hyper(3, **h), sumsq=sumsq, zero_grad=True, err=err)
        assert int(err) == 0
        after = [s.host() for s in sets]
        for s, b, a in zip(sets, before, after):
            where = [check_adapter(s, b, a, i, one(h, i), t, True) for i, t in zip((0, 2), want)]
            untouched(s, b, a, where)
        runs.append((sumsq.cpu().numpy(), after))
    assert np.array_equal(runs[0][0], runs[1][0])
    for a, b in zip(runs[0][1], runs[1][1]):
        assert all(np.array_equal(a[k], b[k]) for k in a)


def test_pool_of_many_steps_keeps_8_bit_moments_near_fp32():
    """50 steps of 8-bit moments against the 64-bit step on the same gradients.  Each step rounds m by at most
    2^-4 relative of itself (and the root by 2^-4), so the update stays within (1 + 2^-4 / (1 - 0.9))-ish of
    it in the worst case; independent roundings leave far less.  The test's claim is coarse: the weights'
    total movement agrees to a tenth."""
    s = Setup(4, 256, 256, [8], 256, "e4m3", True)
    ts, ids, err = B.TrainSet([s.t]), ids_of([0]), new_err()
    B.lora_adamw_init(ts, ids, err=err)
    q = np.concatenate(R.positions(s.pool, 0))
    w = s.t.master.cpu().numpy().astype(np.float64)[q]
    w_start, m, v = w.copy(), np.zeros(len(q)), np.zeros(len(q))
    rng = np.random.default_rng(0)
    drift = rng.normal(size=len(q)) * 1e-3
    h = settings(1, 0, lr=1e-3, beta1=0.9, beta2=0.999, weight_decay=0.0, grad_scale=1.0)
    for step in range(1, 51):
        g = (drift + rng.normal(size=len(q)) * 1e-3).astype(np.float32)
        full = torch.zeros_like(s.t.grad)
        full[torch.from_numpy(q).cuda()] = torch.from_numpy(g).cuda()
        s.t.grad.copy_(full)
        h["step"] = np.array([step])
        B.lora_adamw_step(ts, ids, B.adamw_hyper(1, **h), zero_grad=True, err=err)
        w, m, v, _ = R.adamw(w, g.astype(np.float64), m, v, one(h, 0))
    got = s.t.master.cpu().numpy().astype(np.float64)[q]
    assert int(err) == 0
    assert np.linalg.norm((got - w_start) - (w - w_start)) <= 0.1 * np.linalg.norm(w - w_start)


@pytest.mark.parametrize("state", ["f32", "e4m3"])
def test_init(state):
    s = Setup(8, 1000, 264, [5, 3, 2], 128, state, True)
    before, err = s.host(), new_err()
    B.lora_adamw_init(B.TrainSet([s.t]), ids_of([2, 0]), err=err)
    after = s.host()
    where = [np.concatenate(R.positions(s.pool, i)) for i in (2, 0)]
    for q in where:
        assert not after["grad"][q].any() and not after["m"][q].any() and not after["v"][q].any()
        assert np.array_equal(after["master"][q].view(np.uint32), before["pool"][q].view(np.uint16).astype(np.uint32) << 16)
        if state == "e4m3":
            assert not after["m_scale"][q // 64].any() and not after["v_scale"][q // 64].any()
    assert np.array_equal(before["pool"], after["pool"])
    untouched(s, before, after, where)
    assert int(err) == 0


def test_zero_gradients_and_extreme_values():
    """All-zero blocks, gradients whose squares underflow, and large ones."""
    s = Setup(6, 512, 64, [2], 64, "e4m3", True)
    ts, ids, err = B.TrainSet([s.t]), ids_of([0]), new_err()
    B.lora_adamw_init(ts, ids, err=err)
    qa, qb = R.positions(s.pool, 0)
    g = np.zeros(s.own.size, dtype=np.float32)
    g[qa[64:128]] = 1e-25
    g[qa[128:192]] = 1e15 * np.linspace(-1, 1, 64)
    g[qa[192]] = 1.0
    g[qa[193:256]] = 1e-7  # 2^-23 of the block's largest: its root's code would be zero
    s.t.grad.copy_(torch.from_numpy(g))
    h = settings(1, 0, step=1, lr=1e-3, beta1=0.9, beta2=0.999, weight_decay=0.0, grad_scale=1.0)
    w0 = s.t.master.cpu().numpy().copy()
    B.lora_adamw_step(ts, ids, B.adamw_hyper(1, **h), err=err)
    after = s.host()
    w1 = after["master"].view(np.float32)
    assert np.isfinite(w1[qa]).all() and np.isfinite(w1[qb]).all()
    assert np.array_equal(w1[qb], w0[qb]) and np.array_equal(w1[qa[:64]], w0[qa[:64]])
    assert not after["m"][qb].any() and not after["v"][qb].any()
    assert (after["v"][qa[192:256]] > 0).all()
    # a second step without gradient: m decays, and no element moves by more than the bound of the first
    B.lora_adamw_step(ts, ids, B.adamw_hyper(1, **dict(h, step=np.array([2]))), zero_grad=True, err=err)
    w2 = s.t.master.cpu().numpy()
    assert np.isfinite(w2[qa]).all() and np.abs(w2[qa] - w0[qa]).max() <= 0.01
    assert int(err) == 0


def test_adapters_that_are_passed_over():
    """Bad and repeated ids, an adapter that is not resident, one that does not train, a page outside the pool
    and norms that are not finite: each leaves its bits and sets its bit, the others step."""
    ranks = [4, 0, 4, 4, 4]
    s = Setup(1, 128, 64, ranks, 64, "f32", True)
    h = settings(5, 2)
    h["step"] = np.array([5, 5, 0, 5, 5])
    hyper, ts = B.adamw_hyper(5, **h), B.TrainSet([s.t])
    before, err = s.host(), new_err()
    B.lora_adamw_step(ts, ids_of([0, 1, 2, 0, -1, 5, 1 << 30, -(1 << 31)]), hyper, err=err)
    after = s.host()
    assert int(err) == B.LORA_DERR_BAD_ADAPTER | B.LORA_DERR_BAD_RANK
    untouched(s, before, after, [check_adapter(s, before, after, 0, one(h, 0), None, False)])

    s = Setup(1, 128, 64, ranks, 64, "f32", True)
    ts, before, err = B.TrainSet([s.t]), s.host(), new_err()
    sumsq = torch.tensor([float("inf"), 0, 0, float("nan"), 1.0], device="cuda")
    B.lora_adamw_step(ts, ids_of([0, 3, 4]), hyper, sumsq=sumsq, zero_grad=True, err=err)
    after = s.host()
    assert int(err) == B.LORA_DERR_NONFINITE
    untouched(s, before, after, [check_adapter(s, before, after, 4, one(h, 4), 1.0, True)])

    for state in ("f32", "e4m3"):
        s = Setup(1, 128, 64, ranks, 64, state, True)
        slot = int(s.pool.desc[3]["a_page0"]) + 2
        s.view.page_list[slot] = s.pool.pool.shape[0]  # adapter 3's elements 128 .. 191 of A
        ts, before, err = B.TrainSet([s.t]), s.host(), new_err()
        total = torch.zeros(5, device="cuda")
        B.lora_grad_sumsq(ts, ids_of([3]), total, ts.sumsq_workspace(1), err=err)
        A, Bq = R.positions(s.pool, 3)
        good = np.concatenate([A[:128], A[192:], Bq])
        want = float((s.g[good].astype(np.float64) ** 2).sum())
        assert int(err) == B.LORA_DERR_BAD_PAGE and abs(float(total[3]) - want) <= 3e-6 * want
        B.lora_adamw_step(ts, ids_of([3, 4]), hyper, err=err)
        after = s.host()
        assert int(err) == B.LORA_DERR_BAD_PAGE
        moved = [good, check_adapter(s, before, after, 4, one(h, 4), None, False)]
        untouched(s, before, after, moved)
        assert not np.array_equal(before["master"][good], after["master"][good])


def test_a_gradient_that_is_not_finite_marks_its_norm_alone():
    s = Setup(2, 64, 64, [2, 2], 64)
    ts, err = B.TrainSet([s.t]), new_err()
    s.t.grad[int(R.positions(s.pool, 1)[0][5])] = float("nan")
    sumsq = torch.zeros(2, device="cuda")
    B.lora_grad_sumsq(ts, ids_of([0, 1]), sumsq, ts.sumsq_workspace(2), err=err)
    assert np.isfinite(float(sumsq[0])) and np.isnan(float(sumsq[1])) and int(err) == 0


def test_pages_past_32_bits():
    """Elements whose place in the pool is above 2^31, their byte offsets above 2^33."""
    page, n_pages = 1 << 20, 2050
    n = page * n_pages
    view = B.PoolView(torch.empty(n_pages, page, dtype=torch.bfloat16, device="cuda"),
                      torch.tensor([2049, 2048], dtype=torch.int32, device="cuda"),
                      torch.tensor([[8, 0, 0, 1]], dtype=torch.int32, device="cuda"), page, 8, 512, 256)
    t = B.TrainProj(view, *(torch.empty(n, device="cuda") for _ in range(3)))
    small = Setup(3, 512, 256, [8], page)
    A, Bq = R.positions(small.pool, 0)
    for q, at in ((A, 2049 * page), (Bq, 2048 * page)):
        to = torch.arange(len(q), device="cuda") + at
        qt = torch.from_numpy(q).cuda()
        for big, little in ((t.grad, small.t.grad), (t.m, small.t.m), (t.v, small.t.v), (view.pool.view(-1), small.view.pool.view(-1))):
            big[to] = little[qt]
    h, err = B.adamw_hyper(1, **settings(1, 0, max_norm=1e-3)), new_err()
    got = []
    for proj in (t, small.t):
        ts, sumsq = B.TrainSet([proj]), torch.zeros(1, device="cuda")
        B.lora_grad_sumsq(ts, ids_of([0]), sumsq, ts.sumsq_workspace(1), err=err)
        B.lora_adamw_step(ts, ids_of([0]), h, sumsq=sumsq, zero_grad=True, err=err)
        got.append(sumsq)
    assert int(err) == 0 and torch.equal(got[0], got[1])
    for q, at in ((A, 2049 * page), (Bq, 2048 * page)):
        qt = torch.from_numpy(q).cuda()
        for big, little in ((t.grad, small.t.grad), (t.m, small.t.m), (t.v, small.t.v), (view.pool.view(-1), small.view.pool.view(-1))):
            assert torch.equal(big[at: at + len(q)], little[qt])


def test_other_stream_and_graph():
    s = [Setup(9, 512, 256, [8, 4], 128, "e4m3") for _ in range(3)]
    h, err = B.adamw_hyper(2, **settings(2, 0, max_norm=1e-3)), new_err()
    side = torch.cuda.Stream()

    def go(x, **kw):
        B.lora_grad_sumsq(x.ts, x.ids, x.total, x.ws, err=err, **kw)
        B.lora_adamw_step(x.ts, x.ids, h, sumsq=x.total, zero_grad=True, err=err, **kw)

    for x in s:
        x.ts, x.ids, x.total = B.TrainSet([x.t]), ids_of([1, 0]), torch.zeros(2, device="cuda")
        x.ws = x.ts.sumsq_workspace(2)
    go(s[0])
    side.wait_stream(torch.cuda.current_stream())
    go(s[1], stream=side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go(s[2])
    graph.replay()
    torch.cuda.synchronize()
    want = s[0].host()
    for x in s[1:]:
        got = x.host()
        assert all(np.array_equal(want[k], got[k]) for k in want)


@pytest.mark.parametrize("state", ["f32", "e4m3"])
def test_hundreds_of_adapters(state):
    """More listed adapters than a CTA has threads, one listed twice far apart, each with its own settings; the
    chunks of long matrices (several spans) beside those of short ones."""
    n = 300
    ranks = [1 + (k * 7) % 3 for k in range(n)]
    s = Setup(11, 64, 72, ranks, 64, state, True)
    ts, err = B.TrainSet([s.t]), new_err()
    order = np.random.default_rng(0).permutation(n)
    listed = list(order) + [int(order[3])]
    h = settings(n, 5, max_norm=[0.002 if k % 2 else 0.0 for k in range(n)])
    sumsq = torch.zeros(n, device="cuda")
    before = s.host()
    B.lora_grad_sumsq(ts, ids_of(listed), sumsq, ts.sumsq_workspace(n + 1), err=err)
    assert int(err) == B.LORA_DERR_BAD_ADAPTER  # the repeated id
    err.zero_()
    B.lora_adamw_step(ts, ids_of(listed), B.adamw_hyper(n, **h), sumsq=sumsq, zero_grad=True, err=err)
    assert int(err) == B.LORA_DERR_BAD_ADAPTER
    after, got = s.host(), sumsq.cpu().numpy()
    where = []
    for i in range(n):
        total = sum(float((s.g[q].astype(np.float64) ** 2).sum()) for q in R.positions(s.pool, i))
        assert abs(got[i] - total) <= 3e-6 * total
        where.append(check_adapter(s, before, after, i, one(h, i), total, True))
    untouched(s, before, after, where)


@pytest.mark.parametrize("state", ["f32", "e4m3"])
@pytest.mark.parametrize("master", [False, True])
def test_chunks_of_several_spans(state, master):
    """A launch of so many places (by max_rank) that a chunk is several spans, of the step and of the norms:
    matrices that end inside a span, a block and a page."""
    ranks = [1 + (k * 3) % 5 for k in range(72)]
    s = Setup(12, 8200, 12008, ranks, 1024, state, master, max_rank=64)
    listed = [k for k in reversed(range(72)) if k != 4]
    ts, ids, err = B.TrainSet([s.t]), ids_of(listed), new_err()
    h = settings(72, 6, max_norm=0.01)
    sumsq, before = torch.zeros(72, device="cuda"), s.host()
    B.lora_grad_sumsq(ts, ids, sumsq, ts.sumsq_workspace(len(listed)), err=err)
    B.lora_adamw_step(ts, ids, B.adamw_hyper(72, **h), sumsq=sumsq, err=err)
    after, got, where = s.host(), sumsq.cpu().numpy(), []
    for i in listed:
        total = sum(float((s.g[q].astype(np.float64) ** 2).sum()) for q in R.positions(s.pool, i))
        assert abs(got[i] - total) <= 3e-6 * total
        where.append(check_adapter(s, before, after, i, one(h, i), total, False))
    untouched(s, before, after, where)
    assert int(err) == 0
