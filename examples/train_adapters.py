"""Train several tenants' adapters at once on preference pairs, on sampled answers or after a teacher.

One frozen projection with a LoRA adapter per tenant and a frozen head stand for a model:

    y = x W0^T + s_i (x A_i^T) B_i,     logits = y H^T

A step runs, on one stream and without reading anything back:

    lora_base_apply       y, every row with its tenant's adapter
    lora_preference_loss  (or lora_policy_loss) the loss and dL/dlogits, in the logits' place
    lora_sgmv_backward    dA_i, dB_i, added into an array laid out like the pool
    lora_grad_sumsq       each tenant's gradient norm
    lora_adamw_step       new weights in the pool's pages, the gradients cleared

The reference model's log-probabilities come from lora_token_logprobs with every row on adapter -1.

With --loss distill the tenants learn from a teacher's top logits (lora_topk_logits, listed once) on a base in 8-bit
floating point, of two frozen projections with the adapters on the first:

    lora_base_f8, lora_apply           y = x W0^T, each tenant's term added
    lora_f8_quantize, lora_base_f8     z = y W1^T,  logits = z H^T
    lora_distill_loss                  the loss and dL/dlogits, in the logits' place
    lora_f8_quantize, lora_base_f8_backward    dy = dz W1
    lora_sgmv_backward ...             as above

    python examples/train_adapters.py [--loss policy|distill] [--state e4m3] [--steps 30]
"""

import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from segmented_gather_gemm_lora_gb300 import binding as B  # noqa: E402
from segmented_gather_gemm_lora_gb300 import workloads as W  # noqa: E402

RANKS = (8, 16, 4, 32)  # one tenant each
D, V = 512, 1000
ROWS = 24               # rows of an answer
TOP = 32                # a teacher's listed logits


class Trainer:
    def __init__(self, loss="preference", state="f32", seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
        n = len(RANKS)
        pool = W.build_pool(np.random.default_rng(seed), D, D, RANKS, zero_B=True)  # B = 0: adapters start as the base model
        self.kind, self.view = loss, B.PoolView.from_host(pool)
        self.train = B.TrainSet([B.TrainProj.zeros(self.view, state=B.LORA_STATE_E4M3 if state == "e4m3" else B.LORA_STATE_F32,
                                                   master=True)])
        self.grad = self.train.projs[0].grad
        self.tenants = torch.arange(n, dtype=torch.int32, device="cuda")
        self.hyper = B.adamw_hyper(n, step=0, lr=[2e-3, 1e-3, 2e-3, 1e-3], max_norm=1.0, weight_decay=0.01)
        self.sumsq, self.space = torch.zeros(n, device="cuda"), self.train.sumsq_workspace(n)
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        B.lora_adamw_init(self.train, self.tenants, err=self.err)

        # each tenant has one chosen and one rejected answer; the first rows of an answer are its prompt
        T = 2 * n * ROWS
        self.ids = torch.arange(n, dtype=torch.int32, device="cuda").repeat_interleave(2 * ROWS)
        self.labels = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
        self.labels.view(2 * n, ROWS)[:, : ROWS // 4] = -1
        self.indptr = torch.arange(0, T + 1, ROWS, dtype=torch.int32, device="cuda")
        self.x, self.y = rnd(T, D).bfloat16(), torch.empty(T, D, dtype=torch.bfloat16, device="cuda")
        self.w0, self.head = (rnd(D, D) / D ** 0.5).bfloat16(), (rnd(V, D) / D ** 0.5).bfloat16()
        self.seg, none = B.Segments(T), torch.full_like(self.ids, -1)
        self.hu = torch.empty(2 * T, B.LORA_MAX_RANK, device="cuda")
        if loss == "distill":
            B.lora_segments_build(self.ids, n, self.seg, err=self.err)
            self.distill_from((rnd(D, D) / D ** 0.5).bfloat16(), (self.w0 + 0.3 * rnd(D, D) / D ** 0.5).bfloat16())
            return

        # the reference model: no adapter on any row
        self.ref, self.logp = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
        B.lora_segments_build(none, n, self.seg, err=self.err)
        B.lora_token_logprobs(self.logits(none), self.labels, self.ref, err=self.err)
        B.lora_segments_build(self.ids, n, self.seg, err=self.err)
        if loss == "preference":
            self.loss, self.seq_logp = torch.empty(n, device="cuda"), torch.empty(2 * n, device="cuda")
            self.pref_space = B.preference_workspace(T, n)
        else:
            self.loss, self.kl = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
            # answers sampled by the reference model: rewarded where chosen, else punished
            side = torch.tensor([1.0, -1.0], device="cuda").repeat(n).repeat_interleave(ROWS)
            self.advantage, self.weight = side.contiguous(), torch.full((T,), 1.0 / T, device="cuda")

    def distill_from(self, w1, teacher):
        """The teacher, the base with `teacher` in W0's place, says its part; the base itself goes into 8 bits."""
        T = self.x.shape[0]
        self.top, self.top_values = torch.empty(T, TOP, dtype=torch.int32, device="cuda"), torch.empty(T, TOP, device="cuda")
        self.tail, self.loss = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
        B.lora_topk_logits(self.x @ teacher.t() @ w1.t() @ self.head.t(), self.top, self.top_values, self.tail,
                           temperature=2.0, labels=self.labels, err=self.err)
        self.q0, self.q1 = B.F8Matrix.empty(D, D, block_rows=128), B.F8Matrix.empty(D, D, block_rows=128)
        self.qx, self.qy = B.F8Matrix.empty(T, D), B.F8Matrix.empty(T, D)
        self.qdz = B.F8Matrix.empty(T, D, type=B.LORA_F8_E5M2)
        for x, q in ((self.w0, self.q0), (w1, self.q1), (self.x, self.qx)):
            B.lora_f8_quantize(x, q, err=self.err)
        self.z, self.dy = torch.empty_like(self.x), torch.empty_like(self.x)

    def logits(self, ids):
        if self.kind == "distill":
            B.lora_base_f8(self.qx, self.q0, self.y, err=self.err)
            B.lora_apply(self.x, self.y, self.seg, self.view, err=self.err)
            B.lora_f8_quantize(self.y, self.qy, err=self.err)
            B.lora_base_f8(self.qy, self.q1, self.z, err=self.err)
            return self.z @ self.head.t()
        B.lora_base_apply(self.x, self.w0, self.y, ids, self.seg, self.view, err=self.err)
        return self.y @ self.head.t()

    def step(self):
        """One step of every tenant; the mean loss, still on the device."""
        logits = self.logits(self.ids)
        if self.kind == "distill":
            B.lora_distill_loss(logits, self.top, self.top_values, self.loss, None, logits, tail=self.tail, labels=self.labels,
                                temperature=2.0, kd_weight=4.0, grad_scale=1.0 / self.loss.numel(), err=self.err)
        elif self.kind == "preference":
            B.lora_preference_loss(logits, self.labels, self.indptr, self.loss, self.seq_logp, logits, self.pref_space,
                                   ref_logp=self.ref, beta=0.1, grad_scale=1.0 / self.loss.numel(), err=self.err)
        else:
            B.lora_policy_loss(logits, self.labels, self.ref, self.advantage, self.logp, self.loss, self.kl, logits,
                               ref_logp=self.ref, weight=self.weight, kl_coef=0.02, err=self.err)
        dy = logits @ self.head  # the logits hold their gradient now
        if self.kind == "distill":
            B.lora_f8_quantize(dy, self.qdz, err=self.err)
            B.lora_base_f8_backward(self.qdz, self.q1, self.dy, err=self.err)
            dy = self.dy
        B.lora_sgmv_backward(self.x, dy, None, self.grad, self.hu, self.seg, self.view, err=self.err)
        self.hyper.view(torch.int32)[:, 0].add_(1)
        B.lora_grad_sumsq(self.train, self.tenants, self.sumsq, self.space, err=self.err)
        B.lora_adamw_step(self.train, self.tenants, self.hyper, sumsq=self.sumsq, zero_grad=True, err=self.err)
        return self.loss.sum() if self.kind == "policy" else self.loss.mean()


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--loss", choices=("preference", "policy", "distill"), default="preference")
    ap.add_argument("--state", choices=("f32", "e4m3"), default="f32")
    ap.add_argument("--steps", type=int, default=30)
    a = ap.parse_args()
    t = Trainer(a.loss, a.state)
    for k in range(a.steps):
        loss = t.step()
        if k % 5 == 0 or k == a.steps - 1:
            print("step %3d  loss %.4f  gradient norms %s" % (k, float(loss), [round(v ** 0.5, 3) for v in t.sumsq.tolist()]))
    if int(t.err):
        sys.exit("device error bits %d" % int(t.err))


if __name__ == "__main__":
    main()
