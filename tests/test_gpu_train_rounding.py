"""Roundings of the optimizer step that its definition fixes to the last bit.

With beta1 = beta2 = 0 and no clipping the first moment is the gradient itself and the second its square, so
every result below follows from the gradient alone: fp32 products by 1 and sums with 0 are exact, and the
correctly rounded root of a correctly rounded square is the number again (its squares stay in the normal
range here).  Equality is asked for, no tolerance."""

import numpy as np
import pytest
import torch

import train_ref as R
from gpu_util import cuda_or_skip, new_err
from segmented_gather_gemm_lora_gb300 import binding as B
from test_gpu_train_step import Setup, ids_of

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _cuda():
    cuda_or_skip()


def nearest_e4m3(y):
    """The value e4m3 keeps of y: to nearest, ties to the even code, at most 448."""
    a = np.abs(y)
    unit = np.exp2(np.maximum(np.frexp(a)[1] - 1, -6) - 3.0)
    return np.sign(y) * np.minimum(np.round(a / unit) * unit, 448.0)


def tie_blocks(rng, n):
    """[n, 64] fp32 blocks: the largest on, one unit above and one below the middle of two bf16 scales, or
    anywhere; the others on, above and below the middles of two codes, or anywhere."""
    k = rng.integers(128, 256, n) + 0.5
    top = (448 * k * np.exp2(rng.integers(-50, 30, n) - 7.0)).astype(np.float32)
    side = rng.integers(0, 4, n)
    top = np.where(side == 1, np.nextafter(top, np.float32(np.inf)), np.where(side == 2, np.nextafter(top, np.float32(0)), top))
    top = np.where(rng.random(n) < 0.2, (top * rng.uniform(0.6, 1, n)).astype(np.float32), top)
    scale = R.bf16_round(top.astype(np.float64) / 448)
    e = rng.integers(-8, 8, (n, 64))  # below the normal range the codes are 2^-9 apart
    code = np.where(e < -6, (rng.integers(0, 8, (n, 64)) + 0.5) * 2.0 ** -9, (rng.integers(8, 16, (n, 64)) + 0.5) * np.exp2(e - 3.0))
    x = (code * scale[:, None]).astype(np.float32)  # 5 bits by 8: exact
    side = rng.integers(0, 4, (n, 64))
    x = np.where(side == 1, np.nextafter(x, np.float32(np.inf)), np.where(side == 2, np.nextafter(x, np.float32(0)), x))
    x = np.where(rng.random((n, 64)) < 0.2, (x * rng.uniform(0.5, 2, (n, 64))).astype(np.float32), x)
    x = np.minimum(x, top[:, None])
    x[np.arange(n), rng.integers(0, 64, n)] = top
    x *= rng.choice([-1, 1], (n, 64)).astype(np.float32)
    return x.astype(np.float32)


@pytest.mark.parametrize("master", [False, True])
def test_codes_and_scales_are_those_of_the_definition(master):
    """Scales bf16(largest / 448) and codes to nearest, for the first moments and for the roots."""
    s = Setup(21, 4096, 4096, [16], 4096, "e4m3", master)
    ts, ids, err = B.TrainSet([s.t]), ids_of([0]), new_err()
    B.lora_adamw_init(ts, ids, err=err)
    q = np.concatenate(R.positions(s.pool, 0))
    x = tie_blocks(np.random.default_rng(0), len(q) // 64).reshape(-1)
    g = np.zeros(s.own.size, dtype=np.float32)
    g[q] = x
    s.t.grad.copy_(torch.from_numpy(g))
    B.lora_adamw_step(ts, ids, B.adamw_hyper(1, lr=1e-3, beta1=0.0, beta2=0.0), err=err)
    after = s.host()
    assert int(err) == 0
    x64 = x.astype(np.float64).reshape(-1, 64)
    scale = R.bf16_round(np.abs(x64).max(1) / 448)
    for k, y in (("m", x64), ("v", np.abs(x64))):
        sc = (after[k + "_scale"][q[::64] // 64].view(np.uint16).astype(np.uint32) << 16).view(np.float32)
        assert np.array_equal(sc, scale), "%s: %d of %d scales" % (k, (sc != scale).sum(), scale.size)
        want = nearest_e4m3(y / scale[:, None])
        if k == "v":
            want = np.where((want == 0) & (y > 0), 2.0 ** -9, want)
        got = R.decode_e4m3(after[k][q]).reshape(-1, 64)
        assert np.array_equal(got, want), "%s: %d of %d codes" % (k, (got != want).sum(), want.size)


def test_a_square_past_fp32_leaves_its_weight_and_a_tiny_one_counts_as_zero():
    """v = inf from a finite gradient divides its update to zero; v below 2^-126 is zero (the update is then
    m / eps); neither reaches another block."""
    s = Setup(23, 512, 64, [2], 64, "e4m3", True)
    ts, ids, err = B.TrainSet([s.t]), ids_of([0]), new_err()
    B.lora_adamw_init(ts, ids, err=err)
    q = R.positions(s.pool, 0)[0]
    g = np.zeros(s.own.size, dtype=np.float32)
    g[q[5]], g[q[64 + 7]], g[q[128]] = 1e25, 2.0 ** -64, 1.0
    s.t.grad.copy_(torch.from_numpy(g))
    w0 = s.t.master.cpu().numpy().copy()
    B.lora_adamw_step(ts, ids, B.adamw_hyper(1, lr=0.5, beta1=0.0, beta2=0.0, eps=2.0 ** -60), err=err)
    assert int(err) == 0
    after = s.host()
    w1 = after["master"].view(np.float32)
    assert w1[q[5]] == w0[q[5]]
    assert abs(float(w1[q[71]]) - (float(w0[q[71]]) - 0.5 * 2.0 ** -4)) <= 2.0 ** -20  # m / eps = 2^-4
    assert not after["v"][q[64:128]].any() and not after["v_scale"][q[64] // 64]
    assert abs(float(w1[q[128]]) - (float(w0[q[128]]) - 0.5)) <= 2.0 ** -20
    rest = np.setdiff1d(q[64:], [q[71], q[128]])
    assert np.array_equal(w1[rest], w0[rest])


def test_fp32_update_of_a_first_gradient_is_its_sign():
    """fp32 moments: m / (sqrt(v) + 0) is +-1 to the last bit, so weights of 0 move by the rate itself."""
    s = Setup(22, 4096, 4096, [16], 4096, "f32", True)
    ts, ids, err = B.TrainSet([s.t]), ids_of([0]), new_err()
    B.lora_adamw_init(ts, ids, err=err)
    q = np.concatenate(R.positions(s.pool, 0))
    rng = np.random.default_rng(1)
    g = np.zeros(s.own.size, dtype=np.float32)
    g[q] = (np.exp(rng.uniform(np.log(1e-15), np.log(1e15), len(q))) * rng.choice([-1, 1], len(q))).astype(np.float32)
    s.t.grad.copy_(torch.from_numpy(g))
    s.t.master.zero_()
    B.lora_adamw_step(ts, ids, B.adamw_hyper(1, lr=0.37, beta1=0.0, beta2=0.0, eps=0.0), err=err)
    assert int(err) == 0
    w = s.t.master.cpu().numpy()[q]
    want = -np.sign(g[q]) * np.float32(0.37)
    assert np.array_equal(w, want), "%d of %d" % ((w != want).sum(), len(q))
