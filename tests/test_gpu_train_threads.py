"""The losses called from two threads of one program, each on its own stream."""

import os
import subprocess
import sys

import pytest

from gpu_util import cuda_or_skip

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
import threading
import torch
from segmented_gather_gemm_lora_gb300 import binding as B

def case(V):
    g = torch.Generator(device="cuda").manual_seed(V)
    T = 400
    x = torch.randn(T, V, generator=g, device="cuda").bfloat16()
    lab = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
    return x, lab, torch.full((T,), -9.0, device="cuda"), torch.ones(T, device="cuda")

def call(c, s):
    x, lab, old, adv = c
    logp, loss, d = torch.empty_like(old), torch.empty_like(old), torch.empty_like(x)
    B.lora_policy_loss(x, lab, old, adv, logp, loss, None, d, stream=s)
    return logp, loss, d

cases = [case(V) for V in (20000, 32000)]
torch.cuda.synchronize()
B.lib()
gate, out = threading.Barrier(2), [None, None]

def work(k):
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        gate.wait(20)
        for _ in range(20):
            out[k] = call(cases[k], s)
        s.synchronize()

threads = [threading.Thread(target=work, args=(k,)) for k in range(2)]
[t.start() for t in threads]
[t.join() for t in threads]
torch.cuda.synchronize()
for k in range(2):  # and again, each alone
    assert out[k] is not None
    assert all(torch.equal(a, b) for a, b in zip(out[k], call(cases[k], None)))
print("same")
"""


def test_two_threads_first_calls_of_one_kernel():
    """Different row lengths that one kernel holds, so with different shared memory, in a program whose first
    calls these are: every call succeeds and gives what it gives alone."""
    cuda_or_skip()
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]
