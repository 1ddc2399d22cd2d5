"""A gradient in the logits' place, of rows held by clusters: a CTA writes its share of a row while the others are still
at the row, so every logit that a CTA reads (the listed, the label's) is read before."""

import numpy as np
import pytest
import torch

from gpu_util import cuda_or_skip
from segmented_gather_gemm_lora_gb300 import binding as B
from test_gpu_distill import BF16, F32, batch, f32, i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,V", [(16, 128256), (38, 60000), (76, 60001), (4, 260000)])
def test_held_rows_in_place_are_those_of_another_place(T, V, dtype):
    cuda_or_skip()
    x, ids, values, rest, labels = batch(np.random.default_rng(T + V), T, V, 100)
    labels[::3] = V - 1 - np.arange(T)[::3]  # the last CTA's share, not listed but by chance
    labels[1] = -1
    logits = torch.from_numpy(x).cuda().to(dtype)
    lists = i32(ids), f32(values)
    for kind in (B.LORA_DISTILL_FORWARD, B.LORA_DISTILL_JSD):
        kw = dict(tail=f32(rest), labels=i32(labels), kind=kind, ce_weight=0.5, temperature=2.0)
        loss, ce, grad = torch.empty(T, device="cuda"), torch.empty(T, device="cuda"), torch.empty_like(logits)
        B.lora_distill_loss(logits, *lists, loss, None, grad, ce=ce, **kw)
        for _ in range(12):
            own, loss2, ce2 = logits.clone(), torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
            B.lora_distill_loss(own, *lists, loss2, None, own, ce=ce2, **kw)
            assert torch.equal(loss2, loss) and torch.equal(ce2, ce) and torch.equal(own, grad)
