"""A teacher's top logits and the distillation loss on a GPU against their plain 64-bit forms."""

import numpy as np
import pytest
import torch

import distill_ref as R
from gpu_util import cuda_or_skip
from segmented_gather_gemm_lora_gb300 import binding as B

pytestmark = pytest.mark.gpu

KIND = {"forward": B.LORA_DISTILL_FORWARD, "reverse": B.LORA_DISTILL_REVERSE, "jsd": B.LORA_DISTILL_JSD}
BF16, F32 = torch.bfloat16, torch.float32


def room(T, V, dtype, pad=0, first=0, fill=3.0):
    """Rows of V elements, pad more between them, the first `first` elements into a buffer."""
    return torch.full((T * (V + pad) + first + 8,), fill, dtype=dtype, device="cuda")[first: first + T * (V + pad)].view(T, V + pad)


def device(x, dtype, pad=0, first=0):
    """(padded buffer, its view of the logits, their values in doubles)."""
    T, V = x.shape
    buf = room(T, V, dtype, pad, first)
    buf[:, :V] = torch.from_numpy(x).cuda().to(dtype)
    return buf, buf[:, :V], buf[:, :V].double().cpu().numpy()


# ----------------------------------------------------------------------- top k --

def check_topk(x, k, dtype, temperature=1.0, labels=None, pad=0, first=0):
    T, V = x.shape
    _, logits, x = device(x, dtype, pad, first)
    ids = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
    values, tail = torch.full((T, k), 7.0, device="cuda"), torch.full((T,), 7.0, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    lab = None if labels is None else torch.tensor(labels, dtype=torch.int32, device="cuda")
    B.lora_topk_logits(logits, ids, values, tail, temperature=temperature, labels=lab, err=err)
    torch.cuda.synchronize()
    want = R.topk(x, k, temperature, labels)
    assert int(err.item()) == 0
    assert np.array_equal(ids.cpu().numpy(), want[0])
    assert np.array_equal(values.cpu().numpy().astype(np.float64), want[1], equal_nan=True)
    got = tail.cpu().numpy().astype(np.float64)
    assert np.array_equal(np.isfinite(got), np.isfinite(want[2])) and np.array_equal(np.isnan(got), np.isnan(want[2]))
    on = np.isfinite(want[2])
    assert np.array_equal(got[~on & ~np.isnan(got)], want[2][~on & ~np.isnan(got)])
    # exponents of up to 40 rounded three times, the hardware's 2^x (2^-22), the sum's chains of additions: 2^-16
    # of a sum; the logarithm and its sum with the maximum: four roundings of the result
    assert (np.abs(got[on] - want[2][on]) <= 2.0 ** -16 + 4 * 2.0 ** -24 * (np.abs(want[2][on]) + 40)).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,V,k,pad,first", [(1, 1, 1, 0, 0), (3, 5, 5, 1, 0), (2, 33, 1, 0, 1), (7, 100, 17, 0, 0),
                                             (4, 256, 256, 0, 0), (9, 1000, 64, 3, 3), (3, 4096, 256, 0, 0), (5, 5003, 100, 0, 0),
                                             (2, 32000, 20, 0, 0), (6, 50257, 64, 0, 5), (2, 128256, 256, 8, 0),
                                             (400, 3001, 33, 0, 0), (700, 640, 8, 0, 0), (2, 300007, 64, 0, 0)])
def test_topk_matches_the_plain_form(T, V, k, pad, first, dtype):
    cuda_or_skip()
    rng = np.random.default_rng(T + V)
    check_topk(rng.normal(size=(T, V)) * 3, k, dtype, pad=pad, first=first)


@pytest.mark.parametrize("temperature", [0.5, 3.0])
@pytest.mark.parametrize("V", [700, 40000])
def test_topk_at_a_temperature(V, temperature):
    cuda_or_skip()
    check_topk(np.random.default_rng(V).normal(size=(5, V)) * 4 + 20, 50, F32, temperature=temperature)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("V", [300, 9000, 70000])
@pytest.mark.parametrize("k", [1, 64, 256])
def test_topk_of_rows_that_are_hard_to_filter(V, k, dtype):
    """Ties by the thousand, rising and falling rows, everything of one sign, all but a few hidden."""
    cuda_or_skip()
    rng = np.random.default_rng(V + k)
    few = np.full(V, -np.inf)
    few[rng.choice(V, 5, replace=False)] = rng.normal(size=5)
    rows = [np.zeros(V), np.arange(V) / 64.0, -np.arange(V) / 64.0, np.full(V, -3.0), rng.integers(0, 3, V) * 1.0,
            np.where(np.arange(V) % 2 == 0, 0.0, -0.0), few, np.full(V, -np.inf), np.where(np.arange(V) < V // 2, -1e30, 1e30),
            np.where(np.arange(V) >= V - 3, 5.0, 1.0), -np.abs(rng.normal(size=V)) - 1, rng.normal(size=V) * 1e-3 + 1e4,
            np.sort(rng.normal(size=V)), np.full(V, torch.finfo(torch.bfloat16).min)]
    x = np.stack(rows)
    x[4, V // 3] = np.inf
    check_topk(x, k, dtype)


def test_topk_lists_a_nan_first():
    cuda_or_skip()
    x = np.random.default_rng(3).normal(size=(4, 3000))
    x[1, [5, 2000]] = np.nan
    x[2, 7] = np.inf
    x[3, ::10] = np.nan
    check_topk(x, 20, F32)
    check_topk(x, 20, BF16)


def test_topk_passes_over_rows_that_do_not_count():
    cuda_or_skip()
    check_topk(np.random.default_rng(4).normal(size=(6, 900)), 12, BF16, labels=[3, -1, 900, 0, -100, 5])


def test_topk_without_tail_and_without_rows():
    cuda_or_skip()
    x = torch.randn(3, 500, device="cuda")
    ids, values = torch.empty(3, 9, dtype=torch.int32, device="cuda"), torch.empty(3, 9, device="cuda")
    B.lora_topk_logits(x, ids, values)
    assert torch.equal(values, torch.sort(x, dim=1, descending=True).values[:, :9])
    B.lora_topk_logits(x[:0], ids[:0], values[:0])
    torch.cuda.synchronize()


def test_topk_does_not_depend_on_timing():
    cuda_or_skip()
    x = torch.randn(700, 60000, device="cuda").to(BF16)
    out = []
    for _ in range(4):
        ids, values = torch.empty(700, 128, dtype=torch.int32, device="cuda"), torch.empty(700, 128, device="cuda")
        tail = torch.empty(700, device="cuda")
        B.lora_topk_logits(x, ids, values, tail, temperature=1.5)
        out.append((ids, values, tail))
    for o in out[1:]:
        assert all(torch.equal(a, b) for a, b in zip(o, out[0]))


# -------------------------------------------------------------------- the loss --

def batch(rng, T, V, k, tail=True, absent=0.1):
    """Logits, a teacher's lists (some entries absent, in any order) and labels, of which some are listed."""
    x = rng.normal(size=(T, V)) * 2
    ids = np.stack([rng.choice(V, k, replace=False) for _ in range(T)])
    values = 8 + 3 * rng.normal(size=(T, k))
    for t in range(T):
        x[t, ids[t]] = values[t] * 0.8 + rng.normal(size=k)
    labels = np.where(rng.random(T) < 0.5, ids[:, 0], rng.integers(0, V, T))
    ids = np.where(rng.random((T, k)) < absent / 2, -1, ids)
    values = np.where(rng.random((T, k)) < absent / 2, -np.inf, values).astype(np.float32)
    rest = (np.log(np.exp(values.astype(np.float64)).sum(1) + 1) - rng.uniform(0.2, 6, T)).astype(np.float32)
    return x, ids, values, rest if tail else None, labels


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(torch.int32).cuda()


def f32(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).float().cuda()


def run_loss(x, ids, values, tail=None, labels=None, weight=None, dtype=F32, pad=0, first=0, inplace=False, gpad=None, err_want=0,
             want_grad=True, **kw):
    T, V = x.shape
    buf, logits, _ = device(x, dtype, pad, first)
    gbuf = buf if inplace else room(T, V, dtype, pad if gpad is None else gpad, first)
    grad = gbuf[:, :V]
    loss, kd, ce = (torch.full((T,), 9.0, device="cuda") for _ in range(3))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    opts = dict(kw, kind=KIND[kw.get("kind", "forward")])
    B.lora_distill_loss(logits, i32(ids), f32(values), loss, kd, grad if want_grad else None, tail=f32(tail),
                        labels=None if labels is None else i32(labels), weight=f32(weight), ce=ce, err=err, **opts)
    torch.cuda.synchronize()
    assert int(err.item()) == err_want
    if want_grad and gbuf.shape[1] > V:
        assert (gbuf[:, V:] == 3.0).all()
    host = lambda t: t.double().cpu().numpy()  # noqa: E731
    return host(loss), host(kd), host(ce), host(grad) if want_grad else None


def check_loss(x, ids, values, tail=None, labels=None, weight=None, dtype=F32, pad=0, first=0, inplace=False, gpad=None, err_want=0,
               **kw):
    loss, kd, ce, grad = run_loss(x, ids, values, tail, labels, weight, dtype, pad, first, inplace, gpad, err_want, **kw)
    x = device(x, dtype)[2]
    values = values.astype(np.float32).astype(np.float64)
    want = R.distill(x, ids, values, tail, labels, weight, **kw)
    # A logarithm of p or q is off by its own rounding and those of what it is the difference of (three of the row's
    # spread and of a sum's logarithm, below 16) and by the sums' errors (2^-19: terms of 2^-22 each, of one sign, and
    # their chains of additions).  kd's derivative with respect to one is p - q, so kd moves by twice that; a term's
    # own arithmetic by 2^-19 of it.  A gradient's parts move by as much of themselves, four of them.
    d = 3 * 2.0 ** -24 * (want["spread"] + 16) + 2.0 ** -19
    for name, got in (("kd", kd), ("ce", ce), ("loss", loss)):
        w = want[name]
        with np.errstate(invalid="ignore"):
            assert np.array_equal(got[~np.isfinite(w)], w[~np.isfinite(w)]), name
            scale = np.ones_like(w)
            if name == "loss":
                scale = np.abs(np.ones_like(w) if weight is None else weight) * (kw.get("kd_weight", 1.0) + kw.get("ce_weight", 0.0))
            tol = scale * 2 * d + 2.0 ** -18 * np.abs(w) + 1e-37
            bad = np.isfinite(w) & ~(np.abs(got - w) <= tol)
        assert not bad.any(), (name, got[bad][:4], w[bad][:4], tol[bad][:4])
    if grad is None:
        return
    tol = 4 * d[:, None] * want["size"] + np.abs(want["grad"]) * (torch.finfo(dtype).eps / 2) * 1.01 + 2.0 ** -126
    bad = ~(np.abs(grad - want["grad"]) <= tol)
    assert not bad.any(), (np.argwhere(bad)[:5], grad[bad][:4], want["grad"][bad][:4], tol[bad][:4])


SHAPES = [(1, 1, 1, 0, 0), (3, 7, 7, 0, 0), (4, 40, 3, 1, 1), (9, 200, 20, 0, 0), (5, 1003, 64, 5, 3), (3, 4099, 256, 0, 0),
          (4, 20000, 100, 0, 0), (3, 50257, 50, 0, 0), (2, 128256, 64, 0, 0), (300, 1500, 10, 0, 0), (2, 160001, 256, 0, 1),
          (2, 300000, 33, 0, 0)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("kind,tail", [("forward", True), ("forward", False), ("reverse", True), ("jsd", True), ("jsd", False)])
@pytest.mark.parametrize("T,V,k,pad,first", SHAPES)
def test_loss_matches_the_plain_form(T, V, k, pad, first, kind, tail, dtype):
    cuda_or_skip()
    x, ids, values, rest, _ = batch(np.random.default_rng(V + k), T, V, k, tail)
    if V == k and tail:
        x[:, :] += 0.01  # nothing outside the list: the student gives the rest nothing
        rest[:] = -np.inf
    check_loss(x, ids, values, rest, dtype=dtype, pad=pad, first=first, kind=kind, mix=0.3)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("kind", ["forward", "reverse", "jsd"])
@pytest.mark.parametrize("temperature", [1.0, 2.0, 0.5])
@pytest.mark.parametrize("V", [300, 6000, 40000])
def test_loss_with_labels_weights_and_temperature(V, temperature, kind, dtype):
    cuda_or_skip()
    rng = np.random.default_rng(V)
    x, ids, values, rest, labels = batch(rng, 11, V, 30)
    labels[[2, 5]] = -1
    weight = rng.uniform(0.1, 2, 11).astype(np.float32)
    weight[7] = 0.0
    check_loss(x, ids, values, rest, labels, weight, dtype, kind=kind, mix=0.7, temperature=temperature, kd_weight=temperature ** 2,
               ce_weight=0.5, grad_scale=0.25)


@pytest.mark.parametrize("V", [50, 5000, 30000, 200000])
@pytest.mark.parametrize("kind", ["forward", "jsd"])
def test_gradient_in_the_logits_place(V, kind):
    cuda_or_skip()
    rng = np.random.default_rng(V)
    x, ids, values, rest, labels = batch(rng, 7, V, 20)
    labels[3] = -1
    weight = np.ones(7, dtype=np.float32)
    weight[5] = 0.0
    for dtype in (BF16, F32):
        check_loss(x, ids, values, rest, labels, weight, dtype, pad=3, inplace=True, kind=kind, mix=0.5, ce_weight=0.3)


def test_gradient_rows_of_another_alignment():
    cuda_or_skip()
    x, ids, values, rest, labels = batch(np.random.default_rng(8), 6, 5001, 40)
    for dtype in (BF16, F32):
        check_loss(x, ids, values, rest, labels, dtype=dtype, pad=0, gpad=7, ce_weight=1.0)


def test_loss_without_its_gradient():
    cuda_or_skip()
    x, ids, values, rest, labels = batch(np.random.default_rng(9), 6, 5001, 40)
    a = run_loss(x, ids, values, rest, labels, kind="reverse", ce_weight=1.0, want_grad=False)
    b = run_loss(x, ids, values, rest, labels, kind="reverse", ce_weight=1.0)
    for p, q in zip(a[:3], b[:3]):
        assert np.array_equal(p, q)


@pytest.mark.parametrize("kind", ["forward", "reverse", "jsd"])
def test_a_student_near_its_teacher(kind):
    """Divergences of 1e-8 to 1e-2 keep their digits: their terms are small, not differences of large sums."""
    cuda_or_skip()
    rng = np.random.default_rng(10)
    T, V, k = 8, 2000, 32
    x = (rng.normal(size=(T, V)) * 2).astype(np.float32).astype(np.float64)
    ids, _, _ = R.topk(x, k, 1.0)
    step = 10.0 ** -np.linspace(1, 4, T)[:, None]
    teacher = (x + step * rng.normal(size=(T, V))).astype(np.float32).astype(np.float64)
    values = np.take_along_axis(teacher, ids, 1).astype(np.float32)
    rest = np.exp(teacher)
    np.put_along_axis(rest, ids, 0.0, 1)
    rest = np.log(rest.sum(1)).astype(np.float32)
    kd = run_loss(x, ids, values, rest, kind=kind, mix=0.4)[1]
    want = R.distill(x, ids, values.astype(np.float64), rest, kind=kind, mix=0.4)["kd"]
    # logarithms are off by 2^-20 here (values below 16, sums of 2000); kd by twice the mean of |p - q| times that,
    # and |p - q| adds up to at most sqrt(2 kd)
    assert (np.abs(kd - want) <= 2 * 2.0 ** -19 * np.sqrt(2 * want) + 2.0 ** -38 + 1e-5 * want).all(), (kd, want)


def edge_rows(V=600, k=8):
    """(logits, ids, values, tail) of rows where something is missing, extreme or bad; the last bad ones from 10 on."""
    rng = np.random.default_rng(11)
    x, ids, values, rest, _ = batch(rng, 13, V, k, absent=0.0)
    x[0] = -np.inf                      # nothing visible
    x[1, :] = -np.inf                   # nothing but the list
    x[1, ids[1]] = rng.normal(size=k)
    x[2, ids[2]] = -np.inf              # nothing of the list
    x[3, ids[3, 0]] = -np.inf           # a listed entry hidden
    values[4], ids[5] = -np.inf, -1     # teachers without a list, with a rest
    values[6], rest[6] = -np.inf, -np.inf  # a teacher without anything
    rest[7] = -np.inf                   # a teacher that gives the rest nothing
    x[8] = np.where(np.arange(V) % 3 == 0, x[8], -1e30)
    x[9] = x[9] + 3e4                   # large logits
    ids[10, 3] = V                      # bad rows
    ids[11, 5] = ids[11, 2]
    ids[12, 1] = 2 ** 31 - 1
    return x, ids, values, rest


@pytest.mark.parametrize("V", [600, 9000, 70000])
@pytest.mark.parametrize("kind", ["forward", "reverse", "jsd"])
def test_missing_and_extreme_entries(kind, V):
    cuda_or_skip()
    x, ids, values, rest = edge_rows(V)
    check_loss(x, ids, values, rest, kind=kind, mix=0.5, err_want=B.LORA_DERR_BAD_LABEL)
    ok = slice(0, 10)
    labels = np.array([1, 2, 3, 4, 5, 6, 7, 8, 9, 0])
    labels[1], labels[3] = ids[1, 0], ids[3, 1]
    check_loss(x[ok], ids[ok], values[ok], rest[ok], labels, kind=kind, mix=0.5, ce_weight=0.5, temperature=2.0, inplace=True)


def test_bad_labels_do_not_count():
    cuda_or_skip()
    x, ids, values, rest, labels = batch(np.random.default_rng(12), 5, 700, 9)
    labels[2], labels[4] = 700, 2 ** 31 - 1
    check_loss(x, ids, values, rest, labels, ce_weight=1.0, err_want=B.LORA_DERR_BAD_LABEL)
    check_loss(x, ids, values, rest, labels, err_want=B.LORA_DERR_BAD_LABEL)


@pytest.mark.parametrize("V", [900, 60000])
def test_a_nan_stays_in_its_row(V):
    cuda_or_skip()
    x, ids, values, rest, labels = batch(np.random.default_rng(13), 6, V, 9, absent=0.0)
    x[1, (ids[1, 0] + 1) % V] = np.nan
    values[3, 2] = np.nan
    x[4, ids[4, 1]] = np.inf
    loss, kd, _, grad = run_loss(x, ids, values, rest, labels, ce_weight=0.5)
    for t in (1, 3, 4):
        assert np.isnan(loss[t]) and np.isnan(kd[t])
        assert np.isnan(grad[t]).any()
    keep = [0, 2, 5]
    again = run_loss(x[keep], ids[keep], values[keep], rest[keep], labels[keep], ce_weight=0.5)
    assert np.array_equal(loss[keep], again[0]) and np.array_equal(grad[keep], again[3])


def test_gradient_against_differences():
    """The loss's own differences, on the GPU: steps of 2^-7 in fp32."""
    cuda_or_skip()
    rng = np.random.default_rng(14)
    x, ids, values, rest, labels = batch(rng, 1, 60, 6, absent=0.0)
    x = (np.round(x * 64) / 64)
    kw = dict(tail=np.repeat(rest, 120), labels=np.repeat(labels, 120), temperature=1.5, ce_weight=0.4, mix=0.3)
    h = 2.0 ** -7
    step = np.concatenate([np.eye(60), -np.eye(60)]) * h
    for kind in ("forward", "reverse", "jsd"):
        grad = run_loss(x, ids, values, rest, labels, kind=kind, temperature=1.5, ce_weight=0.4, mix=0.3)[3][0]
        loss = run_loss(x + step, np.repeat(ids, 120, 0), np.repeat(values, 120, 0), kind=kind, **kw)[0]
        diff = (loss[:60] - loss[60:]) / (2 * h)
        # a loss near 1 is off by 2^-19 at most (two logarithms), its difference by that over h; and h^2 / 6 times a
        # third derivative, which for these is below 4
        assert (np.abs(diff - grad) <= 2.0 ** -19 / h + 4 * h * h / 6).all(), kind


def test_loss_does_not_depend_on_timing_and_replays():
    cuda_or_skip()
    x, ids, values, rest, labels = batch(np.random.default_rng(15), 40, 30000, 50)
    first = run_loss(x, ids, values, rest, labels, dtype=BF16, kind="jsd", ce_weight=0.5)
    for _ in range(3):
        again = run_loss(x, ids, values, rest, labels, dtype=BF16, kind="jsd", ce_weight=0.5)
        assert all(np.array_equal(a, b) for a, b in zip(first, again))
    _, logits, _ = device(x, BF16)
    out = [torch.zeros(40, device="cuda") for _ in range(3)]
    grad, args = torch.zeros(40, 30000, dtype=BF16, device="cuda"), (i32(ids), f32(values))
    more = dict(tail=f32(rest), labels=i32(labels), kind=B.LORA_DISTILL_JSD, ce_weight=0.5)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.lora_distill_loss(logits, *args, out[0], out[1], grad, ce=out[2], **more)
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(first, (*out, grad)):
        assert np.array_equal(a, b.double().cpu().numpy())


def test_a_teacher_that_is_the_student_has_no_divergence():
    """The lists of lora_topk_logits taken back by the same logits: the two calls agree on what is left."""
    cuda_or_skip()
    for dtype, V, tau in ((BF16, 50000, 1.0), (F32, 3000, 2.0)):
        x = (torch.randn(9, V, device="cuda") * 3).to(dtype)
        ids, values = torch.empty(9, 30, dtype=torch.int32, device="cuda"), torch.empty(9, 30, device="cuda")
        tail, loss = torch.empty(9, device="cuda"), torch.empty(9, device="cuda")
        grad, err = torch.empty_like(x), torch.zeros(1, dtype=torch.int32, device="cuda")
        B.lora_topk_logits(x, ids, values, tail, temperature=tau, err=err)
        for kind in KIND.values():
            B.lora_distill_loss(x, ids, values, loss, None, grad, tail=tail, kind=kind, temperature=tau, err=err)
            # logarithms off by 2^-18 at most: kd is of the order of their square
            assert float(loss.abs().max()) <= 2.0 ** -30 and float(grad.abs().max()) <= 2.0 ** -17
        assert int(err.item()) == 0


def test_no_rows():
    cuda_or_skip()
    e = torch.empty(0, device="cuda")
    B.lora_distill_loss(torch.empty(0, 50, device="cuda"), torch.empty(0, 4, dtype=torch.int32, device="cuda"),
                        torch.empty(0, 4, device="cuda"), e, e, None)
    torch.cuda.synchronize()
