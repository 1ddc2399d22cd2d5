"""The 8-bit base without a GPU: the plain form's rounding, the layout of its structure, and the refusals that
happen on the host before anything is launched."""

import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

import f8_ref as R
from segmented_gather_gemm_lora_gb300 import binding as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("type,dtype", [("e4m3", torch.float8_e4m3fn), ("e5m2", torch.float8_e5m2)])
def test_the_plain_form_rounds_as_the_format(type, dtype):
    codes = torch.arange(256, dtype=torch.uint8).view(dtype).float().double().numpy()
    assert np.array_equal(R.table(type), codes, equal_nan=True)
    x = np.random.default_rng(0).normal(size=20000) * np.exp(np.random.default_rng(1).normal(size=20000) * 3)
    x = np.concatenate([x, np.arange(-1024, 1025) / 64]).astype(np.float32)
    x = x[np.abs(x) <= R.LARGEST[type]]
    assert np.array_equal(R.nearest(x.astype(np.float64), type), torch.from_numpy(x).to(dtype).float().double().numpy())


def test_a_power_of_two_scale_is_the_least_that_reaches():
    for a in (1.0, 448.0, 448.1, 1.75, 1.7500001, 3.5, 57344.0, 2.0 ** -64):
        for type in ("e4m3", "e5m2"):
            _, s = R.quantize(np.full((1, 3), a, dtype=np.float32), 1, type, True)
            s = float(s[0, 0])
            a32 = float(np.float32(a))
            assert np.frexp(s)[0] == 0.5 and R.LARGEST[type] * s >= a32 > R.LARGEST[type] * s / 2


def test_struct_layout_matches_the_header(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    names = {"lora_f8_matrix_t": B.lora_f8_matrix_t, "lora_distill_opts_t": B.lora_distill_opts_t}
    lines = ["#include <stddef.h>", "#include <stdio.h>", '#include "lora_f8.h"', "int main(void) {"]
    for n, c in names.items():
        lines.append('  printf("%%zu\\n", sizeof(%s));' % n)
        lines += ['  printf("%%zu %%zu\\n", offsetof(%s, %s), sizeof(((%s*)0)->%s));' % (n, f, n, f) for f, _ in c._fields_]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines + ["  return 0;", "}"]))
    subprocess.run([cc, "-std=c99", "-Wall", "-Wextra", "-Werror", "-pedantic", "-I", os.path.join(ROOT, "include"), str(src),
                    "-o", str(exe)], check=True)
    out = iter(subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split())
    for c in names.values():
        assert ctypes.sizeof(c) == int(next(out))
        for f, _ in c._fields_:
            d = getattr(c, f)
            assert (d.offset, d.size) == (int(next(out)), int(next(out))), f


# Addresses that no call gets as far as using: every case below is refused on the host.
FAKE = 1 << 20


def f8(rows=4, cols=256, block=1, at=0, **kw):
    m = B.lora_f8_matrix_t(FAKE + (at << 30), -(-cols // 16) * 16, FAKE + (at << 30) + (1 << 28), 1 if block == 1 else -(-cols // 128),
                           rows if block == 1 else 1, rows, cols, block, 0)
    for k, v in kw.items():
        setattr(m, k, v)
    return m


BAD_MATRIX = [dict(rows=-1), dict(cols=0), dict(type=2), dict(type=-1), dict(block_rows=2), dict(block_rows=0), dict(ld=255),
              dict(ld=264), dict(ld=240), dict(scale_row=-1), dict(scale_col=-1), dict(codes=None), dict(codes=FAKE + 8),
              dict(scales=None), dict(scales=FAKE + 2), dict(ld=1 << 41), dict(scale_row=1 << 41), dict(scale_col=1 << 41)]


def quantize(q, x=FAKE + (5 << 30), ldx=256, dtype=0, flags=0):
    return B.lib().lora_f8_quantize(x, ldx, dtype, ctypes.byref(q) if q is not None else None, flags, None, None)


@pytest.mark.parametrize("kw", BAD_MATRIX)
def test_quantize_refuses_bad_matrices(kw):
    assert quantize(f8(**kw)) == B.LORA_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(x=None), dict(x=FAKE + 1), dict(ldx=255), dict(dtype=2), dict(dtype=-1), dict(flags=2),
                                dict(ldx=1 << 41), dict(dtype=1, x=FAKE + 2), dict(x=FAKE), dict(x=FAKE + (1 << 28))])
def test_quantize_refuses_bad_arguments(kw):
    assert quantize(f8(), **kw) == B.LORA_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(scale_row=0), dict(scale_col=0), dict(scale_row=1, scale_col=3), dict(scale_row=1, scale_col=1),
                                dict(scale_row=2, scale_col=4)])
def test_quantize_refuses_scales_that_share_places(kw):
    # rows 0..3 and groups 0..2: with strides 2 and 4 the third row's first scale is the first row's second
    assert quantize(f8(cols=384, **kw), ldx=384) == B.LORA_ERR_INVALID_ARG


def test_quantize_refuses_no_matrix_and_codes_over_scales():
    assert quantize(None) == B.LORA_ERR_INVALID_ARG
    assert quantize(f8(scales=FAKE + 512)) == B.LORA_ERR_INVALID_ARG


def product(x, w, y=FAKE + (9 << 30), ldy=None, dtype=1, back=False):
    call = B.lib().lora_base_f8_backward if back else B.lib().lora_base_f8
    outer = w.cols if back else w.rows
    return call(ctypes.byref(x), ctypes.byref(w), y, outer if ldy is None else ldy, dtype, None, None)


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("kw", BAD_MATRIX)
def test_product_refuses_bad_matrices(kw, back):
    for which in (0, 1):
        m = [f8(256, 256, 1), f8(256, 256, 128, 1)]
        for k, v in kw.items():
            setattr(m[which], k, v)
        assert product(*m, ldy=256, back=back) == B.LORA_ERR_INVALID_ARG


@pytest.mark.parametrize("back", [False, True])
def test_product_refuses_bad_arguments(back):
    x, w = f8(cols=300 if back else 256), f8(300, 256, 128, 1)
    bad = B.LORA_ERR_INVALID_ARG
    assert product(f8(cols=257), w, back=back) == bad  # widths that do not meet
    assert product(f8(cols=300 if back else 256, block=128), w, back=back) == bad
    assert product(x, f8(300, 256, 1, 1), back=back) == bad
    assert product(x, f8(0, 256, 128, 1), back=back) == bad
    assert product(x, w, y=None, back=back) == bad
    assert product(x, w, y=FAKE + (9 << 30) + 2, back=back) == bad
    assert product(x, w, y=FAKE + (9 << 30) + 1, dtype=0, back=back) == bad
    assert product(x, w, ldy=255, back=back) == bad
    assert product(x, w, ldy=1 << 41, back=back) == bad
    assert product(x, w, dtype=2, back=back) == bad
    for m in (x, w):
        assert product(x, w, y=m.codes, back=back) == bad
        assert product(x, w, y=m.scales, back=back) == bad


def test_more_rows_or_columns_than_tiles_can_count_are_refused():
    many = 0x7fff0001
    assert quantize(f8(rows=many, ld=16, cols=16), ldx=16) == B.LORA_ERR_UNSUPPORTED
    assert quantize(f8(rows=4, cols=many), ldx=many) == B.LORA_ERR_UNSUPPORTED
    assert product(f8(rows=many, cols=16, ld=16), f8(300, 16, 128, 1)) == B.LORA_ERR_UNSUPPORTED
    assert product(f8(cols=16), f8(many, 16, 128, 1)) == B.LORA_ERR_UNSUPPORTED


def test_no_rows_is_nothing_to_do():
    assert quantize(f8(rows=0, codes=None, scales=None), x=None) == B.LORA_OK
    assert product(f8(rows=0, codes=None, scales=None), f8(300, 256, 128, 1), y=None) == B.LORA_OK


# ------------------------------------------------------------------ the binding --

def codes(rows, cols, dtype=torch.float8_e4m3fn):
    return torch.zeros(rows, -(-cols // 16) * 16, dtype=torch.uint8).view(dtype)[:, :cols]


def test_binding_refuses_what_is_no_matrix():
    s = torch.zeros(3, 2)
    for c, scales, block in [(torch.zeros(3, 256), s, 1), (torch.zeros(3, 256, dtype=torch.uint8), s, 1),
                             (codes(3, 256)[:, 1:], s, 1), (codes(3, 256)[:, ::2], torch.zeros(3, 1), 1),
                             (torch.zeros(3, 250, dtype=torch.uint8).view(torch.float8_e4m3fn), s, 1),
                             (codes(3, 256).t(), torch.zeros(256, 1), 1), (codes(3, 256), s, 64), (codes(3, 256), s.double(), 1),
                             (codes(3, 256), torch.zeros(2, 3), 1), (codes(3, 256), torch.zeros(3, 3), 1), (codes(3, 256), s, 128),
                             (codes(3, 256)[0], s, 1), (codes(3, 0), torch.zeros(3, 0), 1),
                             (codes(1, 256).expand(3, 256), s, 1)]:
        with pytest.raises(ValueError):
            B.F8Matrix(c, scales, block)


def test_binding_takes_scales_of_any_strides():
    m = B.F8Matrix(codes(3, 200), torch.zeros(2, 3).t())
    assert (m.c.scale_row, m.c.scale_col, m.c.ld) == (1, 3, 208)
    m = B.F8Matrix(codes(3, 200, torch.float8_e5m2), torch.zeros(1, 1).expand(1, 2), 128)
    assert (m.c.scale_row, m.c.scale_col, m.c.type, m.c.block_rows) == (0 if m.c.scale_row == 0 else 1, 0, 1, 128)
    m = B.F8Matrix.empty(5, 300, device="cpu")
    assert (m.c.scale_row, m.c.scale_col, m.c.rows, m.c.cols, m.c.ld) == (1, 5, 5, 300, 304)
    m = B.F8Matrix.empty(300, 300, block_rows=128, device="cpu")
    assert tuple(m.scales.shape) == (3, 3) and m.c.scale_col == 1


def test_binding_refuses_tensors_off_the_device():
    x, w = B.F8Matrix.empty(4, 256, device="cpu"), B.F8Matrix.empty(300, 256, block_rows=128, device="cpu")
    for stream in (None, 0):
        with pytest.raises(ValueError):
            B.lora_f8_quantize(torch.zeros(4, 256), x, stream=stream)
        with pytest.raises(ValueError):
            B.lora_base_f8(x, w, torch.zeros(4, 300), stream=stream)
        with pytest.raises(ValueError):
            B.lora_base_f8_backward(B.F8Matrix.empty(4, 300, device="cpu"), w, torch.zeros(4, 256), stream=stream)


def test_binding_refuses_outputs_of_another_shape_or_type(monkeypatch):
    monkeypatch.setattr(B, "_one_device", lambda *a: None)
    x, w = B.F8Matrix.empty(4, 256, device="cpu"), B.F8Matrix.empty(300, 256, block_rows=128, device="cpu")
    for y in (torch.zeros(4, 299), torch.zeros(5, 300), torch.zeros(4, 300, dtype=torch.float16), torch.zeros(300, 4).t(),
              torch.zeros(1, 300).expand(4, 300), torch.zeros(1200)):
        with pytest.raises(ValueError):
            B.lora_base_f8(x, w, y, stream=0)
    for v in (torch.zeros(4, 255), torch.zeros(4, 256, dtype=torch.float16), torch.zeros(256, 4).t()):
        with pytest.raises(ValueError):
            B.lora_f8_quantize(v, x, stream=0)
    with pytest.raises(ValueError):
        B.lora_f8_quantize(torch.zeros(4, 256), x, err=torch.zeros(1), stream=0)
