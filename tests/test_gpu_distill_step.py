"""A training step on an 8-bit base after a teacher, its calls together as examples/train_adapters.py runs them: a
captured step gives the same weights, the gradients are those of the formulas, and a tenant's agrees with
differences of its loss."""

import os
import sys

import numpy as np
import pytest
import torch

import distill_ref as R
from gpu_util import cuda_or_skip
from segmented_gather_gemm_lora_gb300 import binding as B
from segmented_gather_gemm_lora_gb300 import workloads as W

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _cuda():
    cuda_or_skip()


def trainer(*args):
    from train_adapters import Trainer

    return Trainer(*args)


@pytest.mark.parametrize("state", ["f32", "e4m3"])
def test_a_step_runs_and_a_captured_one_gives_the_same_weights(state):
    a, b = trainer("distill", state), trainer("distill", state)
    before = a.view.pool.clone()
    a.step()
    b.step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        loss = b.step()
    for _ in range(3):
        last = a.step()
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(a.view.pool.view(torch.int16), b.view.pool.view(torch.int16))
    assert not torch.equal(a.view.pool.view(torch.int16), before.view(torch.int16))
    assert torch.equal(last, loss) and bool(torch.isfinite(last))
    assert int(a.err) == 0 and int(b.err) == 0


def wide(m):
    """An 8-bit matrix's values, in doubles."""
    rows, cols = m.codes.shape
    s = m.scales.double().repeat_interleave(m.block_rows, 0)[:rows].repeat_interleave(128, 1)[:, :cols]
    return m.codes.float().double() * s


def adapters(view, pool_values, n):
    """[(scale, A [r, d_in], B [r, d_out])] of a pool-shaped array, in doubles."""
    out, P = [], view.c.page_elems
    desc = view.adapters.view(torch.int32).view(-1, 4)
    flat = pool_values.flatten().double()
    for i in range(n):
        d = desc[i].tolist()
        parts = []
        for slot, width in ((d[2], view.d_in), (d[3], view.d_out)):
            e = torch.arange(d[0] * width, device="cuda")
            parts.append(flat[view.page_list.long()[slot + e // P] * P + e % P].view(d[0], width))
        scale = desc[i, 1:2].view(torch.float32).item()
        out.append((scale, *parts))
    return out


def test_the_step_is_its_formulas():
    """Forward and backward through an 8-bit projection with adapters and an 8-bit one behind it, with a pad row, an
    unlisted adapter and rows without one, in doubles from the codes that the calls chose."""
    rng = np.random.default_rng(1)
    T, d0, d1, d2, V, k = 150, 384, 520, 264, 700, 24
    pool = W.build_pool(rng, d0, d1, (8, 16, 4))
    view = B.PoolView.from_host(pool)
    g = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ids = torch.from_numpy(rng.integers(-1, 3, T).astype(np.int32)).cuda()
    labels = torch.from_numpy(rng.integers(0, V, T).astype(np.int32)).cuda()
    labels[::9] = -1
    x, head = rnd(T, d0).bfloat16(), rnd(V, d2) / d2 ** 0.5
    q0, q1 = B.F8Matrix.empty(d1, d0, block_rows=128), B.F8Matrix.empty(d2, d1, block_rows=128)
    qx, qy, qdz = B.F8Matrix.empty(T, d0), B.F8Matrix.empty(T, d1), B.F8Matrix.empty(T, d2, type=B.LORA_F8_E5M2)
    for v, q in ((rnd(d1, d0) / d0 ** 0.5, q0), ((rnd(d2, d1) / d1 ** 0.5).bfloat16(), q1), (x, qx)):
        B.lora_f8_quantize(v, q, err=err)
    top, values = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    tail, loss, kd, ce = (torch.empty(T, device="cuda") for _ in range(4))
    B.lora_topk_logits(rnd(T, V) * 2, top, values, tail, temperature=2.0, labels=labels, err=err)

    seg, n = B.Segments(T), 3
    y, z = torch.empty(T, d1, dtype=torch.bfloat16, device="cuda"), torch.empty(T, d2, device="cuda")
    B.lora_segments_build(ids, n, seg, err=err)
    B.lora_base_f8(qx, q0, y, err=err)
    B.lora_apply(x, y, seg, view, err=err)
    B.lora_f8_quantize(y, qy, err=err)
    B.lora_base_f8(qy, q1, z, err=err)
    logits = z @ head.t()
    dlogits = torch.empty_like(logits)
    opts = dict(kind="jsd", mix=0.4, temperature=2.0, kd_weight=4.0, ce_weight=0.5, grad_scale=1.0 / T)
    B.lora_distill_loss(logits, top, values, loss, kd, dlogits, tail=tail, labels=labels, ce=ce, err=err,
                        **dict(opts, kind=B.LORA_DISTILL_JSD))
    dz = dlogits @ head
    B.lora_f8_quantize(dz, qdz, err=err)
    dy, dx = torch.empty(T, d1, dtype=torch.bfloat16, device="cuda"), torch.zeros(T, d0, dtype=torch.bfloat16, device="cuda")
    B.lora_base_f8_backward(qdz, q1, dy, err=err)
    qdy = B.F8Matrix.empty(T, d1)
    B.lora_f8_quantize(dy, qdy, err=err)
    B.lora_base_f8_backward(qdy, q0, dx, err=err)
    grad = torch.zeros_like(view.pool, dtype=torch.float32).flatten()
    B.lora_sgmv_backward(x, dy, dx, grad, torch.empty(2 * T, B.LORA_MAX_RANK, device="cuda"), seg, view, err=err)
    torch.cuda.synchronize()
    assert int(err) == 0

    def near(got, want, tol):
        assert float((got.double() - want).norm()) <= tol * float(want.norm())

    # y: rounded to bf16 by the base and by the adapters' term, whose intermediate is bf16 too: 2^-8 each
    xd, ad = x.double(), adapters(view, view.pool, n)
    want_y = wide(qx) @ wide(q0).t()
    for i, (s, A, C) in enumerate(ad):
        want_y[ids == i] += s * (xd[ids == i] @ A.t()) @ C
    near(y, want_y, 3 * 2.0 ** -8)
    near(wide(qy), y.double(), 2.0 ** -4)  # e4m3 at half a step; below the normal codes an absolute half step, far less
    # z: fp32 sums of d1 products over groups, in any order within one: d1 roundings at most, of their sizes
    zb = wide(qy).abs() @ wide(q1).abs().t() * d1 * 2.0 ** -24
    assert bool(((z.double() - wide(qy) @ wide(q1).t()).abs() <= zb).all())
    want = R.distill(logits.double().cpu().numpy(), top.cpu().numpy(), values.double().cpu().numpy(), tail.double().cpu().numpy(),
                     labels.cpu().numpy(), **opts)
    # as the loss alone is tested: logarithms off by 2^-17 at these spreads, four parts of the gradient
    assert float((dlogits.double().cpu() - torch.from_numpy(want["grad"])).abs().max()) <= 4 * 2.0 ** -17 * float(want["size"].max())
    assert float((loss.double().cpu() - torch.from_numpy(want["loss"])).abs().max()) <= 2.0 ** -14
    assert not bool(dlogits[labels < 0].any()) and not bool(wide(qdz)[labels < 0].any())
    near(wide(qdz), dz.double(), 2.0 ** -3)  # e5m2
    near(dy, wide(qdz) @ wide(q1), 2.0 ** -8)
    dyd, want_dx, gd = dy.double(), wide(qdy) @ wide(q0), adapters(view, grad, n)
    # dx: bf16 by the base and with the adapters' part, intermediates too; dA and dB: fp32 sums of bf16 products
    # with one bf16 intermediate each
    for i, (s, A, C) in enumerate(ad):
        on = ids == i
        u, v = xd[on] @ A.t(), dyd[on] @ C.t()
        want_dx[on] += s * v @ A
        near(gd[i][1], s * v.t() @ xd[on], 2 * 2.0 ** -8)
        near(gd[i][2], s * u.t() @ dyd[on], 2 * 2.0 ** -8)
    near(dx, want_dx, 3 * 2.0 ** -8)
    assert not bool(dy[labels < 0].any())


def test_the_gradient_of_a_tenant_against_differences():
    """dA and dB of one tenant, the adapters on an 8-bit base before the head, against differences of its loss: fp32
    weights change by +-h along the gradient (normed), the pool takes their bf16.  The loss moves by 2 h |g| to a
    tenth: bf16 outputs and gradients carry 2^-8 each, and so does the rounding of the changed weights."""
    t = trainer("distill")
    for _ in range(10):
        t.step()
    w = dict(tail=t.tail, labels=t.labels, temperature=2.0, kd_weight=4.0, err=t.err)
    head, rows = t.head.float(), t.loss.numel() // t.tenants.numel()

    def logits():
        B.lora_base_f8(t.qx, t.q0, t.y, err=t.err)
        B.lora_apply(t.x, t.y, t.seg, t.view, err=t.err)
        return t.y.float() @ head.t()

    x = logits()
    B.lora_distill_loss(x, t.top, t.top_values, t.loss, None, x, **w)
    t.grad.zero_()
    B.lora_sgmv_backward(t.x, (x @ head).bfloat16(), None, t.grad, t.hu, t.seg, t.view, err=t.err)
    B.lora_grad_sumsq(t.train, t.tenants, t.sumsq, t.space, err=t.err)
    tenant, keep = 1, t.view.pool.clone()
    owned = torch.zeros_like(t.grad, dtype=torch.bool)
    desc = t.view.adapters.view(torch.int32).view(-1, 4)[tenant].tolist()
    P = t.view.c.page_elems
    for slot, d in ((desc[2], t.view.d_in), (desc[3], t.view.d_out)):
        e = torch.arange(desc[0] * d, device="cuda")
        owned[t.view.page_list.long()[slot + e // P] * P + e % P] = True
    norm = float(t.sumsq[tenant]) ** 0.5
    h, moved = 0.05, []
    for side in (1, -1):
        t.view.pool.copy_((keep.float().flatten() + side * h * torch.where(owned, t.grad, torch.zeros_like(t.grad)) / norm)
                          .bfloat16().view_as(keep))
        t.view.pool.copy_(torch.where(owned.view_as(keep), t.view.pool, keep))
        B.lora_distill_loss(logits(), t.top, t.top_values, t.loss, None, None, **w)
        moved.append(float(t.loss[tenant * rows: (tenant + 1) * rows].double().sum()))
    assert abs((moved[0] - moved[1]) / (2 * h) - norm) <= 0.1 * norm
    assert int(t.err) == 0
