"""The 8-bit calls on several streams at once and in graphs: they share nothing, so results are those of one call."""

import pytest
import torch

from gpu_util import cuda_or_skip
from segmented_gather_gemm_lora_gb300 import binding as B

pytestmark = pytest.mark.gpu


def operands(T, n, k, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(T, k, generator=g, device="cuda").bfloat16()
    w = torch.randn(n, k, generator=g, device="cuda")
    return x, w, B.F8Matrix.empty(T, k), B.F8Matrix.empty(n, k, block_rows=128), torch.empty(T, n, device="cuda")


def calls(o, stream=None):
    x, w, qx, qw, y = o
    B.lora_f8_quantize(x, qx, stream=stream)
    B.lora_f8_quantize(w, qw, stream=stream)
    B.lora_base_f8(qx, qw, y, stream=stream)


@pytest.mark.parametrize("T", [5, 50, 200, 1500])  # shared sums of few tokens, of tiles, wide tiles
def test_streams_at_once_and_graphs(T):
    cuda_or_skip()
    sets = [operands(T, 1100, 1300, s) for s in range(3)]
    want = []
    for o in sets:
        calls(o)
        want.append(o[4].clone())
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for o in sets:
        o[4].zero_()
    torch.cuda.synchronize()
    for _ in range(5):
        for o, s in zip(sets, streams):
            calls(o, s)
    torch.cuda.synchronize()
    assert all(torch.equal(o[4], w) for o, w in zip(sets, want))
    graphs = []
    for o in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            calls(o)
        graphs.append(g)
        o[4].zero_()
    torch.cuda.synchronize()
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o[4], w) for o, w in zip(sets, want))
    sets[0][0].copy_(sets[1][0])  # a replay reads its inputs anew
    sets[0][1].copy_(sets[1][1])
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(sets[0][4], want[1])
