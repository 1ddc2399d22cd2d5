"""The 8-bit base on a GPU against its plain 64-bit form: quantising, the product and its input's gradient."""

import numpy as np
import pytest
import torch

import f8_ref as R
from gpu_util import cuda_or_skip
from segmented_gather_gemm_lora_gb300 import binding as B

pytestmark = pytest.mark.gpu

TORCH = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
CODE = {"e4m3": B.LORA_F8_E4M3, "e5m2": B.LORA_F8_E5M2}


def values_of(codes, type):
    """The values of device codes, by the table of the format."""
    return R.table(type)[codes.contiguous().view(torch.uint8).cpu().numpy()]


def data(rng, rows, cols, dtype):
    """fp32 values of a type, of many sizes, with zeros, a silent group and entries on the ties of codes."""
    x = rng.normal(size=(rows, cols)) * np.exp(2 * rng.normal(size=(rows, 1)))
    x[rng.random((rows, cols)) < 0.05] = 0.0
    x[:, ::7] = np.round(x[:, ::7] * 16) / 16
    x[rows // 2, :128] = 0.0
    t = torch.from_numpy(x.astype(np.float32))
    return t.to(torch.bfloat16).float().numpy() if dtype is torch.bfloat16 else t.numpy()


def whole_rows(q):
    """The bytes of a matrix's rows with their padding."""
    return q.codes.as_strided((q.c.rows, q.c.ld), (q.c.ld, 1)).view(torch.uint8)


def quantized(x, dtype, block, type, pow2, ld=None):
    """(matrix, device error bits) of values x, quantised on the GPU; rows of x are ld apart."""
    rows, cols = x.shape
    room = torch.full((rows, ld or cols), float("nan"), dtype=dtype, device="cuda")
    room[:, :cols] = torch.from_numpy(x).cuda().to(dtype)
    q = B.F8Matrix.empty(rows, cols, block_rows=block, type=CODE[type])
    whole_rows(q).fill_(0xAA)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    B.lora_f8_quantize(room[:, :cols], q, pow2=pow2, err=err)
    torch.cuda.synchronize()
    return q, int(err.item())


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("type", ["e4m3", "e5m2"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols,block,ld", [(1, 1, 1, None), (1, 4096, 1, None), (3, 128, 1, 131), (17, 1000, 1, None),
                                                (9, 257, 1, 264), (130, 333, 1, None), (1, 128, 128, None), (128, 128, 128, None),
                                                (300, 515, 128, None), (129, 1000, 128, 1003), (5, 7, 128, 8),
                                                (700, 96, 1, 96), (2, 20000, 1, None)])
def test_quantize_matches_the_plain_form(rows, cols, block, ld, dtype, type, pow2):
    cuda_or_skip()
    rng = np.random.default_rng(rows * 31 + cols)
    x = data(rng, rows, cols, dtype)
    q, err = quantized(x, dtype, block, type, pow2, ld)
    want, scales = R.quantize(x, block, type, pow2)
    # fp32 quotients are rounded alike on both sides: codes and scales are equal, not near
    assert np.array_equal(q.scales.cpu().numpy(), scales)
    assert np.array_equal(values_of(q.codes, type), want)
    assert err == 0
    assert (whole_rows(q)[:, cols:] == 0xAA).all()


@pytest.mark.parametrize("type", ["e4m3", "e5m2"])
def test_quantize_at_the_ends_of_the_range(type):
    cuda_or_skip()
    rows = [np.full(128, 2.0 ** -65), np.full(128, 2.0 ** -64), np.full(128, 3e38), np.full(128, np.finfo(np.float32).max),
            np.where(np.arange(128) == 5, 1.0, 2.0 ** -130), np.where(np.arange(128) % 2, 1e-30, -1e-25),
            np.linspace(-448, 448, 128), np.linspace(-57344, 57344, 128), np.float32(1.75) * 2.0 ** np.arange(-60, 68)]
    x = np.stack(rows).astype(np.float32)
    for pow2 in (False, True):
        q, err = quantized(x, torch.float32, 1, type, pow2)
        want, scales = R.quantize(x, 1, type, pow2)
        assert np.array_equal(q.scales.cpu().numpy(), scales) and np.array_equal(values_of(q.codes, type), want) and err == 0


def test_quantize_reports_and_keeps_what_is_not_finite():
    cuda_or_skip()
    x = np.ones((4, 300), dtype=np.float32)
    x[1, 130], x[2, 299] = np.inf, np.nan
    q, err = quantized(x, torch.float32, 1, "e4m3", False)
    v, s = values_of(q.codes, "e4m3"), q.scales.cpu().numpy()
    assert err == B.LORA_DERR_NONFINITE
    assert np.isinf(s[1, 1]) and np.isnan(s[2, 2]) and np.isnan(v[2, 256:]).all() and np.isnan(v[1, 130])
    ok = np.ones((4, 3), dtype=bool)
    ok[1, 1] = ok[2, 2] = False
    assert (s[ok] == np.float32(1) / np.float32(448)).all()
    # whatever is computed from such a group is NaN, and nothing else is
    w, _ = quantized(np.ones((5, 300), dtype=np.float32), torch.float32, 128, "e4m3", False)
    y = torch.zeros(4, 5, device="cuda")
    B.lora_base_f8(q, w, y)
    y = y.cpu().numpy()
    assert np.isnan(y[1:3]).all() and np.isfinite(y[[0, 3]]).all()


def matrix(rng, rows, cols, block, type, scale_layout="own"):
    """(F8Matrix of random codes and scales, its values in doubles)."""
    t = R.table(type)
    codes = rng.integers(0, 256, (rows, cols)).astype(np.uint8)
    codes[~np.isfinite(t[codes])] = 0
    if type == "e5m2":  # within e4m3's range: sums of 57344 squared hide everything else
        codes[np.abs(t[codes]) > 448] = 0x2C
    q = B.F8Matrix.empty(rows, cols, block_rows=block, type=CODE[type])
    q.codes.view(torch.uint8).copy_(torch.from_numpy(codes).cuda())
    blocks, groups = -(-rows // block), -(-cols // 128)
    s = np.exp(rng.normal(size=(blocks, groups))).astype(np.float32) * 2.0 ** -8
    if scale_layout == "own":
        q.scales.copy_(torch.from_numpy(s).cuda())
    else:
        if scale_layout == "rows":  # the groups of a row side by side
            st = torch.from_numpy(s).cuda()
        elif scale_layout == "wide":  # places between the scales
            st = torch.zeros(blocks, groups, 3, device="cuda")
            st[:, :, 1] = torch.from_numpy(s).cuda()
            st = st[:, :, 1]
        else:  # one scale for all
            s[:] = s[0, 0]
            st = torch.full((1, 1), float(s[0, 0]), device="cuda").expand(blocks, groups)
        q = B.F8Matrix(q.codes, st, block)
    return q, R.widen(t[codes], s, block)


def check_product(rng, T, N, K, back, out, xtype="e4m3", wtype="e4m3", pad=0, layout="own"):
    inner, outer = (N, K) if back else (K, N)
    xq, x = matrix(rng, T, inner, 1, xtype, layout)
    wq, w = matrix(rng, N, K, 128, wtype, layout)
    w = w if back else w.T
    room = torch.full((T + 1, outer + pad), 7.0, dtype=out, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    call = B.lora_base_f8_backward if back else B.lora_base_f8
    call(xq, wq, room[:T, :outer], err=err)
    torch.cuda.synchronize()
    y = room.float().cpu().numpy().astype(np.float64)
    assert int(err.item()) == 0
    assert (y[T] == 7.0).all() and (y[:, outer:] == 7.0).all()
    want, size = x @ w, np.abs(x) @ np.abs(w)
    # a group's 128 products in the tensor cores' fp32 (a bit lost at each addition at most), two roundings a
    # group for its scales and one for the sum over groups, seven more additions where the sum is split
    bound = (128 + 3 + -(-inner // 128) + 7) * 2.0 ** -23 * size
    bound += np.abs(want) * (torch.finfo(out).eps / 2) * 1.01
    bad = np.abs(y[:T, :outer] - want) > bound
    assert not bad.any(), (np.argwhere(bad)[:5], np.max(np.abs(y[:T, :outer] - want) / np.maximum(bound, 1e-300)))


SIZES = [(1, 1, 1), (1, 128, 128), (1, 4096, 4096), (3, 130, 257), (8, 200, 1000), (15, 2050, 333), (16, 128, 2056),
         (17, 96, 5000), (31, 1000, 1000), (33, 500, 640), (64, 1024, 1024), (65, 129, 4096), (127, 333, 128), (128, 256, 256),
         (129, 257, 384), (200, 2048, 300), (333, 1000, 2050), (513, 700, 1100), (1025, 640, 200)]


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,N,K", SIZES)
def test_product_matches_the_plain_form(T, N, K, out, back):
    cuda_or_skip()
    check_product(np.random.default_rng(T * 7 + N + K), T, N, K, back, out)


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("xtype,wtype", [("e5m2", "e4m3"), ("e4m3", "e5m2"), ("e5m2", "e5m2")])
@pytest.mark.parametrize("T,N,K", [(5, 300, 260), (40, 257, 513), (300, 520, 392)])
def test_product_of_each_pair_of_types(T, N, K, xtype, wtype, back):
    cuda_or_skip()
    check_product(np.random.default_rng(T), T, N, K, back, torch.float32, xtype, wtype)


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("layout", ["rows", "wide", "one"])
@pytest.mark.parametrize("T", [4, 300])
def test_product_with_scales_of_any_strides(T, layout, back):
    cuda_or_skip()
    check_product(np.random.default_rng(T), T, 400, 900, back, torch.float32, layout=layout)


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,pad", [(3, 1), (3, 8), (140, 3), (140, 4), (700, 1), (700, 8)])
def test_product_into_rows_of_any_stride(T, pad, out, back):
    cuda_or_skip()
    check_product(np.random.default_rng(T + pad), T, 391, 517, back, out, pad=pad)


def test_product_of_many_tiles():
    """More tiles than the GPU holds at once, ends of every dimension inside a tile."""
    cuda_or_skip()
    for back in (False, True):
        check_product(np.random.default_rng(9), 4000, 3001, 391, back, torch.bfloat16)


def test_no_rows():
    cuda_or_skip()
    w, _ = matrix(np.random.default_rng(0), 40, 50, 128, "e4m3")
    B.lora_base_f8(B.F8Matrix.empty(0, 50), w, torch.empty(0, 40, device="cuda"))
    B.lora_base_f8_backward(B.F8Matrix.empty(0, 40), w, torch.empty(0, 50, device="cuda"))
    B.lora_f8_quantize(torch.empty(0, 50, device="cuda"), B.F8Matrix.empty(0, 50))
    torch.cuda.synchronize()


def test_rounding_of_one_product_is_one_rounding():
    """A single product of two codes and two scales: exact in doubles but for the scales' product."""
    cuda_or_skip()
    x, xv = matrix(np.random.default_rng(1), 64, 1, 1, "e4m3")
    w, wv = matrix(np.random.default_rng(2), 300, 1, 128, "e4m3")
    y = torch.empty(64, 300, device="cuda")
    B.lora_base_f8(x, w, y)
    want = xv @ wv.T
    # the product of the scales and its product with the sum: two roundings of 2^-24 (and their product)
    assert (np.abs(y.cpu().numpy() - want) <= 2.01 * 2.0 ** -24 * np.abs(want)).all()


@pytest.mark.parametrize("T", [1, 24, 200, 600])
def test_same_inputs_give_the_same_bits_and_graphs_replay(T):
    cuda_or_skip()
    rng = np.random.default_rng(T)
    x = torch.from_numpy(data(rng, T, 1500, torch.float32)).cuda()
    wq, _ = matrix(rng, 1200, 1500, 128, "e4m3")
    xq = B.F8Matrix.empty(T, 1500)
    y, first = (torch.zeros(T, 1200, device="cuda") for _ in range(2))
    B.lora_f8_quantize(x, xq)
    B.lora_base_f8(xq, wq, first)
    for _ in range(3):
        y.zero_()
        B.lora_base_f8(xq, wq, y)
        assert torch.equal(y, first)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        B.lora_f8_quantize(x, xq)
        B.lora_base_f8(xq, wq, y)
    x.mul_(2.0)  # scales double, codes stay: so does the product
    for _ in range(2):
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, 2 * first)


def test_two_streams_at_once():
    cuda_or_skip()
    rng = np.random.default_rng(5)
    jobs = []
    for T in (12, 300, 64):
        xq, _ = matrix(rng, T, 2000, 1, "e4m3")
        wq, _ = matrix(rng, 900, 2000, 128, "e4m3")
        y = torch.zeros(T, 900, device="cuda")
        B.lora_base_f8(xq, wq, y)
        jobs.append((xq, wq, y, torch.zeros_like(y), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(5):
        for xq, wq, _, again, s in jobs:
            B.lora_base_f8(xq, wq, again, stream=s)
    torch.cuda.synchronize()
    for _, _, y, again, _ in jobs:
        assert torch.equal(y, again)
