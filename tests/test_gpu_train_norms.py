"""Gradient norms: one workspace for lists of every length, sums that do not depend on the list, and 8-bit
moments over more projections than one launch takes."""

import numpy as np
import pytest
import torch

import train_ref as R
from gpu_util import cuda_or_skip, new_err
from segmented_gather_gemm_lora_gb300 import binding as B
from test_gpu_train_step import Setup, ids_of

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
