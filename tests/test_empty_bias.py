"""A layer without outputs has an empty bias, whose address may be null: no call
refuses it, and with outputs a bias and its dtype still come together."""
import ctypes

import pytest

import lora_bypass_linear_amd as L

BF16 = L.BF16


def _calls(N, bias):
    """(name, status) of each forward that takes a bias, over M = 0 rows."""
    lib, n = L.lib(), None
    yield "linear", lib.lyc_linear_fwd(n, BF16, n, BF16, bias, BF16, n, BF16, 0, N, 64, n, 0, n)
    yield "lora", lib.lyc_lora_linear_fwd(n, BF16, n, BF16, bias, BF16, n, BF16, n, BF16, 0, 1.0, n, BF16, 0, N, 64, n, 0, n)
    yield "gated", lib.lyc_lora_gated_fwd(n, BF16, n, n, BF16, bias, bias, BF16, n, n, BF16, n, n, BF16, 0, 1.0, 0, n, BF16,
                                          n, n, n, 0, N, 64, n, 0, n)
    yield "fp8", lib.lyc_fp8_linear_fwd(n, n, n, n, bias, BF16, n, BF16, 0, N, 64, n, 0, n)
    yield "int8", lib.lyc_int8_linear_fwd(n, n, n, n, bias, BF16, n, BF16, 0, N, 64, n, 0, n)
    yield "int8 gated", lib.lyc_int8_gated_fwd(n, n, n, n, n, n, bias, bias, BF16, 0, n, BF16, 0, N, 64, n, 0, n)


@pytest.mark.parametrize("N", [0, 48])
def test_empty_bias(N):
    for name, status in _calls(N, None):
        assert status == (L.OK if N == 0 else L.ERR_INVALID_ARG), name
    for name, status in _calls(N, ctypes.c_void_p(4096)):
        assert status == L.OK, name
