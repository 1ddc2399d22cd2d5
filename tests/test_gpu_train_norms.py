"""Gradient norms: one workspace for lists of every length, sums that do not depend on the list, and 8-bit
moments over more projections than one launch takes."""

import numpy as np
import pytest
import torch

import train_ref as R
from gpu_util import cuda_or_skip, new_err
from segmented_gather_gemm_lora_gb300 import binding as B
from test_gpu_train_step import Setup, check_adapter, ids_of, one, settings, untouched

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _cuda():
    cuda_or_skip()


def test_one_workspace_and_the_same_sums_for_every_list():
    """Lists on both sides of the count from which a chunk is longer, in the workspace of the longest (which
    holds NaN): each adapter's sum has the same bits in all of them."""
    n = 72
    ranks = [1 + (k * 3) % 5 for k in range(n)]
    s = Setup(31, 8200, 12008, ranks, 1024, max_rank=64)
    ts, err = B.TrainSet([s.t]), new_err()
    ws = ts.sumsq_workspace(n)
    whole = torch.zeros(n, device="cuda")
    B.lora_grad_sumsq(ts, ids_of(range(n)), whole, ws, err=err)
    for i in range(0, n, 7):
        want = sum(float((s.g[q].astype(np.float64) ** 2).sum()) for q in R.positions(s.pool, i))
        assert abs(float(whole[i]) - want) <= 3e-6 * want
    for count in (1, 2, 15, 40, 61, 62, 71):
        ws.view(torch.float32).fill_(float("nan"))
        listed = list(np.random.default_rng(count).permutation(n)[:count])
        some = torch.full((n,), 7.0, device="cuda")
        B.lora_grad_sumsq(ts, ids_of(listed), some, ws, err=err)
        ix = torch.tensor(listed, device="cuda")
        assert torch.equal(some[ix].view(torch.int32), whole[ix].view(torch.int32)), count
        some[ix] = 7.0
        assert bool((some == 7.0).all())
    assert int(err) == 0


@pytest.mark.parametrize("master", [False, True])
def test_8_bit_moments_over_more_projections_than_a_launch_takes(master):
    """Nineteen projections in one call: every one steps as the 64-bit form does, by the norm over all of them,
    nothing else moves, and a second run gives the same bits."""
    shapes = [(64 * (1 + g % 3), 128, 64 << (g % 3)) for g in range(19)]
    runs = []
    for _ in range(2):
        sets = [Setup(g, a, b, [4, 0, 9], p, "e4m3", master, max_rank=16) for g, (a, b, p) in enumerate(shapes)]
        ts, ids, err = B.TrainSet([s.t for s in sets]), ids_of([2, 0]), new_err()
        h = settings(3, 1, max_norm=1e-2)
        sumsq = torch.zeros(3, device="cuda")
        B.lora_grad_sumsq(ts, ids, sumsq, ts.sumsq_workspace(2), err=err)
        want = [sum(float((s.g[q].astype(np.float64) ** 2).sum()) for s in sets for q in R.positions(s.pool, i)) for i in (0, 2)]
        assert np.allclose(sumsq[[0, 2]].cpu().numpy(), want, rtol=3e-6)
        before = [s.host() for s in sets]
        B.lora_adamw_step(ts, ids, B.adamw_hyper(3, **h), sumsq=sumsq, zero_grad=True, err=err)
        assert int(err) == 0
        after = [s.host() for s in sets]
        for s, b, a in zip(sets, before, after):
            untouched(s, b, a, [check_adapter(s, b, a, i, one(h, i), t, True) for i, t in zip((0, 2), want)])
        runs.append(after)
    for a, b in zip(*runs):
        assert all(np.array_equal(a[k], b[k]) for k in a)
