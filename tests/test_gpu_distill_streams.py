"""Top logits and distillation losses in flight on several streams together, and in graphs replayed so: calls share
nothing, whatever their forms."""

import numpy as np
import pytest
import torch

from gpu_util import cuda_or_skip
from segmented_gather_gemm_lora_gb300 import binding as B
from test_gpu_distill import BF16, F32, batch, f32, i32

pytestmark = pytest.mark.gpu

# rows, vocabulary and list of a set of calls: short rows, streamed rows, rows held by clusters, few long ones
SETS = [(600, 1000, 20, BF16), (300, 20000, 50, BF16), (40, 60000, 100, F32), (16, 128256, 64, BF16), (2, 300001, 40, F32)]


def operands(T, V, k, dtype, seed):
    x, ids, values, rest, labels = batch(np.random.default_rng(seed), T, V, k)
    logits = torch.from_numpy(x).cuda().to(dtype)
    lists = dict(ids=torch.zeros(T, k, dtype=torch.int32, device="cuda"), values=torch.zeros(T, k, device="cuda"),
                 tail=torch.zeros(T, device="cuda"))
    out = dict(loss=torch.zeros(T, device="cuda"), kd=torch.zeros(T, device="cuda"), ce=torch.zeros(T, device="cuda"),
               grad=torch.zeros_like(logits), err=torch.zeros(1, dtype=torch.int32, device="cuda"))
    return logits, (i32(ids), f32(values)), f32(rest), i32(labels), lists, out


def calls(o, kind, stream=None):
    logits, teacher, rest, labels, lists, out = o
    B.lora_topk_logits(logits, lists["ids"], lists["values"], lists["tail"], err=out["err"], stream=stream)
    B.lora_distill_loss(logits, *teacher, out["loss"], out["kd"], out["grad"], tail=rest, labels=labels, ce=out["ce"], kind=kind,
                        ce_weight=0.5, temperature=2.0, err=out["err"], stream=stream)


def results(o):
    return [*o[4].values(), *o[5].values()]


def clear(sets):
    for o in sets:
        for t in results(o):
            t.zero_()
    torch.cuda.synchronize()


def same(sets, want):
    torch.cuda.synchronize()
    for o, w in zip(sets, want):
        assert all(torch.equal(a, b) for a, b in zip(results(o), w))


@pytest.mark.parametrize("which", [(0, 1, 2, 3, 4), (3, 3, 3, 3), (1, 1, 2, 2), (0, 0, 4, 4)])
def test_calls_in_flight_together(which):
    cuda_or_skip()
    sets = [operands(*SETS[w], seed) for seed, w in enumerate(which)]
    kinds = [(B.LORA_DISTILL_FORWARD, B.LORA_DISTILL_REVERSE, B.LORA_DISTILL_JSD)[i % 3] for i in range(len(sets))]
    want = []
    for o, kind in zip(sets, kinds):
        calls(o, kind)
        torch.cuda.synchronize()
        want.append([t.clone() for t in results(o)])
    streams = [torch.cuda.Stream() for _ in sets]
    clear(sets)
    for _ in range(6):  # no wait between: a stream's calls run while the others' do
        for o, kind, s in zip(sets, kinds, streams):
            calls(o, kind, s)
    same(sets, want)
    graphs = []
    for o, kind in zip(sets, kinds):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            calls(o, kind)
        graphs.append(g)
    clear(sets)
    for _ in range(4):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    same(sets, want)
