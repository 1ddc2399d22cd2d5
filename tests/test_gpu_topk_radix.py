"""Top logits of rows that the radix selection lists, whose first and last elements (the row's edges, outside its whole
16-byte vectors) are among the listed: the same list at each call, and the plain form's."""

import numpy as np
import pytest
import torch

import distill_ref as R
from gpu_util import cuda_or_skip
from segmented_gather_gemm_lora_gb300 import binding as B
from test_gpu_distill import BF16, F32, device

pytestmark = pytest.mark.gpu


def crowded(T, V, per, rng):
    """Rows whose large values sit in r of every 32 vectors (of `per` elements): a thread's vectors are a multiple of 32
    apart, so they crowd in few threads' slots, more than a list of slots' largest entries can hold."""
    x = rng.normal(size=(T, V)) * 0.5 - 30
    vector = np.arange(V) // per % 32
    for t in range(T):
        r = (3, 7, 15, 31)[t % 4]
        x[t] = np.where(vector < r, x[t] + 40, x[t])
    return x


def check(x, k, dtype, first, pad, calls=6):
    T, V = x.shape
    # the edges' values are the row's largest, no two alike as bf16
    x[:, 0], x[:, V - 1], x[:, 1] = 100.0, 101.0, 102.0
    _, logits, x = device(x, dtype, pad, first)
    want = R.topk(x, k, 1.5)
    ids, values, tail = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda"), torch.empty(T, device="cuda")
    tails = None
    for _ in range(calls):
        ids.fill_(-7)
        B.lora_topk_logits(logits, ids, values, tail, temperature=1.5)
        assert np.array_equal(ids.cpu().numpy(), want[0])
        assert np.array_equal(values.double().cpu().numpy(), want[1])
        tails = tail.clone() if tails is None else tails
        assert torch.equal(tail, tails)
    # as for every list: the sum's terms and chains of additions 2^-16, four roundings of the result
    got = tails.double().cpu().numpy()
    assert (np.abs(got - want[2]) <= 2.0 ** -16 + 4 * 2.0 ** -24 * (np.abs(want[2]) + 40)).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("k", [64, 128, 256])
@pytest.mark.parametrize("T,V", [(1300, 4003), (700, 9001), (12, 9001), (8, 70001)])
def test_listed_edges_of_crowded_rows(T, V, k, dtype):
    cuda_or_skip()
    rng = np.random.default_rng(T + V + k)
    check(crowded(T, V, 8 if dtype is BF16 else 4, rng), k, dtype, first=3, pad=2)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,V,k", [(1200, 5001, 250), (1200, 1001, 120), (1200, 301, 64), (5, 2003, 256)])
def test_listed_edges_of_lists_long_for_their_row(T, V, k, dtype):
    cuda_or_skip()
    check(np.random.default_rng(V + k).normal(size=(T, V)) * 3, k, dtype, first=5, pad=0)


def test_the_longest_rows():
    """As many entries as 32-bit steps allow: planted ones at both ends and between, and a row of ties."""
    cuda_or_skip()
    V, k = 0x7fff0000, 70
    x = torch.zeros(1, V, dtype=BF16, device="cuda")
    at = torch.cat([torch.arange(30), V - 1 - torch.arange(30), torch.tensor([V // 2, V // 3, V // 5])]).cuda()
    ids, values, tail = torch.empty(1, k, dtype=torch.int32, device="cuda"), torch.empty(1, k, device="cuda"), torch.empty(1, device="cuda")
    B.lora_topk_logits(x, ids, values, tail)
    assert torch.equal(ids[0].cpu(), torch.arange(k, dtype=torch.int32)) and bool((values == 0).all())
    # sums of ones are exact up to 2^24, and their joins round 512 threads' parts: 2^-20; the logarithm 2^-19
    assert abs(float(tail) - np.log(V - k)) <= 2.0 ** -18
    x[0, at] = torch.arange(at.numel(), 0, -1, device="cuda").to(BF16)
    B.lora_topk_logits(x, ids, values, tail)
    rest = torch.arange(30, 30 + k - at.numel())
    assert torch.equal(ids[0].cpu().long(), torch.cat([at.cpu(), rest]))
    assert abs(float(tail) - np.log(V - k)) <= 2.0 ** -18
