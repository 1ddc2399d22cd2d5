"""The distillation loss and the top logits over many rows: each form of the kernels at its borders (rows by a CTA of
128 to 1024 threads, rows held by clusters), with rows in turn on a CTA and rows that do not count between them."""

import numpy as np
import pytest
import torch

from gpu_util import cuda_or_skip
from segmented_gather_gemm_lora_gb300 import binding as B
from test_gpu_distill import BF16, F32, batch, check_loss, check_topk, f32, i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,V,k", [(700, 1000, 32), (700, 999, 33), (640, 10000, 20), (640, 20001, 50), (700, 2000, 96),
                                   (700, 2001, 97), (640, 4099, 60), (400, 16500, 224), (400, 16500, 225),
                                   (330, 33001, 224), (330, 33000, 256), (320, 70003, 40), (200, 180000, 256)])
def test_rows_in_turn(T, V, k, dtype):
    cuda_or_skip()
    rng = np.random.default_rng(T + V + k)
    x, ids, values, rest, labels = batch(rng, T, V, k)
    labels = np.where(rng.random(T) < 0.25, -1, labels)
    weight = np.where(rng.random(T) < 0.1, 0.0, rng.uniform(0.1, 2, T)).astype(np.float32)
    check_loss(x, ids, values, rest, labels, weight, dtype, inplace=True, temperature=2.0, kd_weight=4.0)
    check_loss(x[:160], ids[:160], values[:160], rest[:160], labels[:160], dtype=dtype, kind="jsd", mix=0.4, ce_weight=0.5,
               temperature=1.5)


@pytest.mark.parametrize("kind", ["forward", "reverse"])
@pytest.mark.parametrize("T,V", [(38, 60000), (76, 60000), (150, 60000), (152, 33000), (160, 65000)])
def test_rows_of_clusters(T, V, kind):
    cuda_or_skip()
    rng = np.random.default_rng(T + V)
    x, ids, values, rest, labels = batch(rng, T, V, 256 if T < 100 else 70)
    labels[rng.random(T) < 0.25] = -1
    for dtype in (BF16, F32):
        check_loss(x, ids, values, rest, labels, None, dtype, inplace=True, kind=kind, ce_weight=0.25, temperature=2.0)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,V,k", [(1000, 5000, 64), (600, 20000, 256), (520, 40001, 20), (70, 30000, 100), (150, 9000, 256)])
def test_topk_of_rows_in_turn(T, V, k, dtype):
    cuda_or_skip()
    rng = np.random.default_rng(T + V + k)
    x = rng.normal(size=(T, V)) * 3
    x[::7] = np.round(x[::7])        # ties
    x[3::11, 100:] = -np.inf         # little to list
    check_topk(x, k, dtype, temperature=1.5, labels=np.where(rng.random(T) < 0.2, -1, 0), pad=3)


def test_two_streams_at_once():
    """Calls that overlap share nothing."""
    cuda_or_skip()
    rng = np.random.default_rng(5)
    x, ids, values, rest, _ = batch(rng, 300, 20000, 50)
    logits, args, tail = torch.from_numpy(x).cuda().to(BF16), (i32(ids), f32(values)), f32(rest)

    def run(stream):
        out = [torch.empty(300, 64, dtype=torch.int32, device="cuda"), torch.empty(300, 64, device="cuda")]
        out += [torch.empty(300, device="cuda") for _ in range(3)] + [torch.empty_like(logits)]
        torch.cuda.synchronize()
        for _ in range(4):
            B.lora_topk_logits(logits, out[0], out[1], out[2], stream=stream)
            B.lora_distill_loss(logits, *args, out[3], out[4], out[5], tail=tail, kind=B.LORA_DISTILL_JSD, stream=stream)
        return out

    want = run(None)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    got = []
    for s in streams:
        with torch.cuda.stream(s):
            got.append(run(s))
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(g, want))


def test_the_longest_rows():
    """Up to the documented length a row is right; above it the call is refused and nothing is written."""
    cuda_or_skip()
    for dtype, V in ((BF16, 1_400_000), (F32, 1_200_000)):
        x, ids, values, rest, labels = batch(np.random.default_rng(6), 2, V, 40)
        check_loss(x, ids, values, rest, labels, None, dtype, ce_weight=1.0)
        logits = torch.zeros(1, 1_500_000, dtype=dtype, device="cuda")
        loss, grad = torch.full((1,), 9.0, device="cuda"), torch.full_like(logits, 9.0)
        with pytest.raises(B.LoraError):
            B.lora_distill_loss(logits, i32(ids[:1]), f32(values[:1]), loss, None, grad)
        torch.cuda.synchronize()
        assert float(loss) == 9.0 and bool((grad == 9.0).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,V,k", [(2000, 250, 20), (1100, 700, 8), (1000, 9000, 32), (1000, 9000, 33), (1000, 1000, 60),
                                   (1000, 2500, 120), (500, 5000, 250), (20, 1000, 60), (300, 200, 100)])
def test_topk_of_many_short_rows(T, V, k, dtype):
    cuda_or_skip()
    check_topk(np.random.default_rng(T + V + k).normal(size=(T, V)) * 3, k, dtype, temperature=0.7, first=3)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,V,k", [(1120, 3000, 30), (1120, 3000, 60), (560, 15000, 30), (980, 20000, 64), (504, 20000, 100),
                                   (490, 33000, 128), (462, 20000, 256), (14, 128000, 64), (14, 128000, 256)])
def test_topk_of_rows_that_are_hard_to_filter_in_each_form(T, V, k, dtype):
    """Ties by the thousand, rising and falling rows, crowds in few places, all but a few hidden, NaNs, each between
    ordinary rows."""
    cuda_or_skip()
    rng = np.random.default_rng(T + V + k)
    few, crowd, nans = np.full(V, -np.inf), rng.normal(size=V), rng.normal(size=V)
    few[rng.choice(V, 5, replace=False)] = rng.normal(size=5)
    crowd[V // 2: V // 2 + 600] += 50
    nans[::50] = np.nan
    at = np.arange(V)
    rows = [np.zeros(V), at / 64.0, -at / 64.0, rng.integers(0, 3, V) * 1.0, np.where(at % 2 == 0, 0.0, -0.0), few,
            np.full(V, -np.inf), np.where(at < V // 2, -1e30, 1e30), np.where(at >= V - 3, 5.0, 1.0), crowd, nans,
            rng.normal(size=V) * 1e-3 + 1e4, np.where(at % 32 == 0, 9.0, rng.normal(size=V)),
            np.full(V, torch.finfo(torch.bfloat16).min)]
    x = rng.normal(size=(T, V)) if T > 14 else np.zeros((T, V))
    for i, r in enumerate(rows):
        x[i * (T // 14)] = r
    check_topk(x, k, dtype)


@pytest.mark.parametrize("T,V,k", [(2000, 500, 20), (1000, 3000, 60), (600, 30000, 100), (500, 20000, 200), (16, 100000, 256)])
def test_topk_in_each_form_does_not_depend_on_timing(T, V, k):
    cuda_or_skip()
    x = (torch.randn(T, V, device="cuda") * 3).to(BF16)
    x[::5] = torch.round(x[::5])
    want = None
    for _ in range(6):
        out = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda"), torch.empty(T, device="cuda")
        B.lora_topk_logits(x, *out, temperature=1.5)
        want = want or out
        assert all(torch.equal(a, b) for a, b in zip(out, want))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,V,k", [(14, 40003, 64), (14, 130001, 256), (1400, 2005, 32), (700, 20003, 60), (700, 20003, 128)])
def test_topk_of_rows_whose_ties_fill_the_list(T, V, k, dtype):
    """The k-th largest is one of thousands that tie: some above it or none, few or many below, odd fractions, both
    infinities, at any alignment; the first by index are listed and the tail has the others."""
    cuda_or_skip()
    rng = np.random.default_rng(T + V + k)
    tie = lambda v, other: np.where(rng.random(V) < 0.7, v, other)  # noqa: E731
    rows = [tie(0.1, rng.normal(size=V) - 9), tie(-0.3, -np.inf), tie(1e-40, -1.0), tie(np.inf, 0.0), tie(-1e30, -2e30),
            tie(3.3, 3.2), np.full(V, -7.7), np.full(V, torch.finfo(torch.bfloat16).min)]
    for n in (1, 5, k - 1, k, k + 3):
        r = np.full(V, -1e30)
        r[rng.choice(V, n, replace=False)] = rng.normal(size=n)
        rows.append(r)
    r = tie(0.1, -5.0)
    r[V - 1], r[0], r[1] = 2.0, 1.0, 0.1
    rows.append(r)
    x = np.zeros((T, V))
    for i in range(T):
        x[i] = rows[i % len(rows)]
    check_topk(x, k, dtype, pad=3, first=1)


@pytest.mark.parametrize("T,V", [(3, 10), (3, 70000), (700, 300)])
def test_lists_longer_than_the_row_and_absent_entries(T, V):
    """An absent entry's id says nothing: not twice listed, not out of range."""
    cuda_or_skip()
    rng = np.random.default_rng(T + V)
    x, ids, values, rest, labels = batch(rng, T, V, 6, absent=0.0)
    k = 50
    more_ids, more = np.full((T, k), -1), np.full((T, k), -np.inf, dtype=np.float32)
    at = rng.choice(k, 6, replace=False)
    more_ids[:, at], more[:, at] = ids, values
    free = [j for j in range(k) if j not in at]
    more_ids[:, free[0]], more_ids[:, free[1]], more_ids[:, free[2]] = ids[:, 0], V + 5, 2 ** 31 - 1  # value -inf
    more_ids[:, free[3]], more[:, free[3]] = -7, 3.0                                              # a negative id
    for kind in ("forward", "reverse", "jsd"):
        check_loss(x, more_ids, more, rest, labels, kind=kind, ce_weight=0.3)
