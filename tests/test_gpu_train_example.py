"""The training calls together, as examples/train_adapters.py runs them: several tenants learn at once, a
step in a CUDA graph gives the same weights, and a tenant's gradient agrees with differences of its loss."""

import os
import sys

import pytest
import torch

from gpu_util import cuda_or_skip
from segmented_gather_gemm_lora_gb300 import binding as B

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _cuda():
    cuda_or_skip()


def trainer(*args):
    from train_adapters import Trainer

    return Trainer(*args)


@pytest.mark.parametrize("state", ["f32", "e4m3"])
def test_preference_training_separates_the_pairs(state):
    """At the start every ratio is 0 (B = 0), so each loss is log 2 to the error of bf16 logits; training
    on the same pairs lowers every tenant's."""
    t = trainer("preference", state)
    first = None
    for _ in range(30):
        t.step()
        first = t.loss.clone() if first is None else first
    assert int(t.err) == 0
    assert float((first - 0.6931).abs().max()) <= 1e-3
    assert bool((t.loss < first - 0.05).all())


def test_policy_training_raises_the_reward():
    t = trainer("policy", "f32")
    first = float(t.step())
    for _ in range(29):
        last = float(t.step())
    assert int(t.err) == 0 and last < first


def test_a_captured_step_gives_the_same_weights():
    a, b = trainer(), trainer()
    a.step()
    b.step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.step()
    for _ in range(3):
        a.step()
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(a.view.pool.view(torch.int16), b.view.pool.view(torch.int16))
    assert int(a.err) == 0 and int(b.err) == 0


def test_gradient_of_the_whole_step_against_differences():
    """dA and dB of one tenant against differences of its loss: fp32 weights change by +-h along the gradient
    (normed), the pool takes their bf16.  The loss moves by 2 h |g| to a tenth: bf16 logits and gradients carry
    2^-8 each, and so does the rounding of the changed weights."""
    t = trainer()
    for _ in range(10):
        t.step()
    logits = t.logits(t.ids)
    B.lora_preference_loss(logits, t.labels, t.indptr, t.loss, None, logits, t.pref_space, ref_logp=t.ref, beta=0.1,
                           grad_scale=1.0, err=t.err)
    t.grad.zero_()
    B.lora_sgmv_backward(t.x, logits @ t.head, None, t.grad, t.hu, t.seg, t.view, err=t.err)
    B.lora_grad_sumsq(t.train, t.tenants, t.sumsq, t.space, err=t.err)
    tenant, keep = 1, t.view.pool.clone()
    owned = torch.zeros_like(t.grad, dtype=torch.bool)
    desc = t.view.adapters.view(torch.int32).view(-1, 4)[tenant].tolist()
    P = t.view.c.page_elems
    for slot, d in ((desc[2], t.view.d_in), (desc[3], t.view.d_out)):
        e = torch.arange(desc[0] * d, device="cuda")
        owned[t.view.page_list.long()[slot + e // P] * P + e % P] = True
    norm = float(t.sumsq[tenant]) ** 0.5
    assert abs(norm - float(t.grad[owned].double().norm())) <= 1e-5 * norm
    h, moved = 0.05, []
    for side in (1, -1):
        t.view.pool.copy_((keep.float().flatten() + side * h * torch.where(owned, t.grad, torch.zeros_like(t.grad)) / norm)
                          .bfloat16().view_as(keep))
        t.view.pool.copy_(torch.where(owned.view_as(keep), t.view.pool, keep))
        B.lora_preference_loss(t.logits(t.ids), t.labels, t.indptr, t.loss, None, None, t.pref_space, ref_logp=t.ref, beta=0.1,
                               err=t.err)
        moved.append(float(t.loss[tenant]))
    assert abs((moved[0] - moved[1]) / (2 * h) - norm) <= 0.1 * norm
    assert int(t.err) == 0
