"""Logits and gradient whose rows take turns in one buffer."""

import pytest
import torch

from gpu_util import cuda_or_skip, new_err
from segmented_gather_gemm_lora_gb300 import binding as B

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _cuda():
    cuda_or_skip()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,V", [(5, 33), (40, 5003), (400, 9000), (9, 128256), (2, 600000)])
def test_halves_of_one_buffer(T, V, dtype):
    """The gradient is written between the logits' rows, element beside element, and nothing else is: the
    same bits as apart from them, and the logits stay."""
    both = torch.randn(T, 2 * V, device="cuda").to(dtype)
    x, d = both[:, :V], both[:, V:]
    keep = x.clone()
    lab = torch.randint(0, V, (T,), device="cuda", dtype=torch.int32)
    old, adv = torch.full((T,), -9.0, device="cuda"), torch.randn(T, device="cuda")
    logp, loss = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    err = new_err()
    apart = torch.empty_like(both)[:, :V]  # rows aligned as the logits' are
    B.lora_policy_loss(x, lab, old, adv, logp, loss, None, apart, err=err)
    B.lora_policy_loss(x, lab, old, adv, logp, loss, None, d, err=err)
    assert torch.equal(d, apart) and torch.equal(x, keep)
    if T > 2:
        indptr = torch.tensor([0, T // 2, T], dtype=torch.int32, device="cuda")
        ws = B.preference_workspace(T, 1)
        B.lora_preference_loss(x, lab, indptr, loss[:1], None, apart, ws, err=err)
        B.lora_preference_loss(x, lab, indptr, loss[:1], None, d, ws, err=err)
        assert torch.equal(d, apart) and torch.equal(x, keep)
    assert int(err) == 0
