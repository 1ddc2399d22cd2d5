"""The bounded waits of the 8-bit products, the top logits and the distillation loss, exercised without any fault:
with the test-only timeout probe armed a CTA waits (about a millisecond at most) on a barrier that nothing arrives on,
gives up, sets LORA_DERR_TIMEOUT and writes nothing; with the probe disarmed the same call is right again."""

import pytest
import torch

from gpu_util import cuda_or_skip, new_err
from segmented_gather_gemm_lora_gb300 import binding as B

pytestmark = pytest.mark.gpu

PROBE_CYCLES = 2_000_000  # about a millisecond at the GB300's clocks


@pytest.fixture(autouse=True)
def _cuda():
    cuda_or_skip()
    yield
    B.debug_wait_probe(0)  # never leave the probe armed for later tests


def times_out_and_recovers(call, outs):
    """call(err) writes outs."""
    err = new_err()
    call(err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    want = [o.clone() for o in outs]
    for o in outs:
        o.fill_(3)
    kept = [o.clone() for o in outs]
    B.debug_wait_probe(PROBE_CYCLES)
    call(err)
    torch.cuda.synchronize()
    assert int(err.item()) == B.LORA_DERR_TIMEOUT
    assert all(torch.equal(a, b) for a, b in zip(outs, kept)), "a CTA that gave up wrote output"
    B.debug_wait_probe(0)
    err.zero_()
    call(err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    assert all(torch.equal(a, b) for a, b in zip(outs, want))


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("T", [1, 30, 64, 130, 1500])  # split (16, 32 and 64 tokens across), mid, wide
def test_products(T, back):
    x, w = B.F8Matrix.empty(T, 1024), B.F8Matrix.empty(1024, 1024, block_rows=128)
    B.lora_f8_quantize(torch.randn(T, 1024, device="cuda"), x)
    B.lora_f8_quantize(torch.randn(1024, 1024, device="cuda"), w)
    y = torch.empty(T, 1024, dtype=torch.bfloat16, device="cuda")
    times_out_and_recovers(lambda err: (B.lora_base_f8_backward if back else B.lora_base_f8)(x, w, y, err=err), [y])


@pytest.mark.parametrize("T", [2, 400])  # a cluster a row, a CTA a row
def test_top_logits(T):
    x = torch.randn(T, 30000, device="cuda")
    ids = torch.empty(T, 40, dtype=torch.int32, device="cuda")
    values, tail = torch.empty(T, 40, device="cuda"), torch.empty(T, device="cuda")
    times_out_and_recovers(lambda err: B.lora_topk_logits(x, ids, values, tail, err=err), [ids, values, tail])


@pytest.mark.parametrize("T", [2, 400])  # held by a cluster, streamed
def test_distillation_loss(T):
    x = torch.randn(T, 60000, device="cuda")
    ids = torch.empty(T, 40, dtype=torch.int32, device="cuda")
    values, tail = torch.empty(T, 40, device="cuda"), torch.empty(T, device="cuda")
    B.lora_topk_logits(torch.randn(T, 60000, device="cuda"), ids, values, tail)
    loss, kd, grad = torch.empty(T, device="cuda"), torch.empty(T, device="cuda"), torch.empty_like(x)
    times_out_and_recovers(lambda err: B.lora_distill_loss(x, ids, values, loss, kd, grad, tail=tail, err=err), [loss, kd, grad])
