"""One row has one log-probability, whichever call gives it."""

import pytest
import torch

from gpu_util import cuda_or_skip, new_err
from segmented_gather_gemm_lora_gb300 import binding as B

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _cuda():
    cuda_or_skip()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,V", [(1, 1), (7, 33), (500, 500), (500, 1021), (500, 2000), (64, 300)])
def test_a_policy_that_has_not_moved_has_ratio_one(T, V, dtype):
    """Rows that a warp holds in both calls: the log-probabilities are the same bits, so the ratio to them is
    1, the loss minus the advantage and the KL term 0, exactly."""
    g = torch.Generator(device="cuda").manual_seed(T + V)
    x = (torch.randn(T, V, generator=g, device="cuda") * 3).to(dtype)
    lab = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
    adv = torch.randn(T, generator=g, device="cuda")
    old, logp, loss, kl = (torch.empty(T, device="cuda") for _ in range(4))
    err = new_err()
    B.lora_token_logprobs(x, lab, old, err=err)
    B.lora_policy_loss(x, lab, old, adv, logp, loss, kl, None, ref_logp=old, kl_coef=0.1, err=err)
    assert torch.equal(logp.view(torch.int32), old.view(torch.int32))
    assert torch.equal(loss, -adv) and not kl.any()
    assert int(err) == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,V", [(40, 5003), (400, 9000), (64, 32000), (9, 128256), (2, 600000)])
def test_longer_rows_differ_by_the_order_of_their_sums_alone(T, V, dtype):
    """Both calls take x - m and log s with the same functions; s is added in another order where a row is
    held by one call and streamed by the other.  Two such sums of positive terms are within 2e-5 of each
    other (each within 1e-5 of the exact one), so log s moves by that and half a unit of each rounding."""
    g = torch.Generator(device="cuda").manual_seed(T + V)
    x = (torch.randn(T, V, generator=g, device="cuda") * 3).to(dtype)
    lab = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
    old, logp, loss = (torch.empty(T, device="cuda") for _ in range(3))
    B.lora_token_logprobs(x, lab, old)
    B.lora_policy_loss(x, lab, old, torch.ones(T, device="cuda"), logp, loss, None, None)
    assert float((logp - old).abs().max()) <= 2e-5 + 4 * 2.0 ** -20
