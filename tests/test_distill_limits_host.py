"""Sizes and settings at the ends of what a teacher's top logits and the distillation loss take: refused on the host
before anything is launched."""

import pytest

from segmented_gather_gemm_lora_gb300 import binding as B
from test_distill_host import loss, topk


@pytest.mark.parametrize("dtype", [B.LORA_LOGITS_BF16, B.LORA_LOGITS_F32])
@pytest.mark.parametrize("V", [0x7fff0001, 0x7fffffff])
def test_topk_refuses_rows_that_its_steps_would_pass(V, dtype):
    """A pass over a row by single elements goes up to a CTA's threads past its end, in 32 bits."""
    assert topk(ld=V, V=V, T=1, dtype=dtype) == B.LORA_ERR_UNSUPPORTED
    assert topk(ld=V, V=V, T=0, dtype=dtype) == B.LORA_ERR_UNSUPPORTED


SMALLEST = 2.0 ** -126


@pytest.mark.parametrize("temperature", [2.0 ** -149, 2.0 ** -140, 2.0 ** -128])
def test_temperatures_without_an_inverse_are_refused(temperature):
    assert topk(temperature=temperature) == B.LORA_ERR_INVALID_ARG
    assert loss(temperature=temperature) == B.LORA_ERR_INVALID_ARG


def test_the_smallest_and_largest_temperatures_are_taken():
    for temperature in (SMALLEST, 3.4e38):
        assert topk(temperature=temperature, T=0) == B.LORA_OK
        assert loss(temperature=temperature, T=0) == B.LORA_OK
