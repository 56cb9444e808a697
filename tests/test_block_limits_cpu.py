"""Limits of the C entry points at sizes and strides whose products do not fit 64 or 32 bits (CPU only:
every call here is refused before a launch)."""
from __future__ import annotations

import ctypes

import pytest

import fp8_quantization_grouped_amd as fq

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
P = ctypes.c_void_p(4096)  # aligned, never dereferenced


def refuse(name, good, changes):
    f = getattr(fq.lib(), name)
    for change, status in changes:
        args = list(good)
        for at, value in change.items():
            args[at] = value
        assert f(*args) == status, (name, change, status)


@pytest.mark.parametrize("power", [31, 48, 55, 56, 57, 60, 62])
def test_product_strides_of_any_size_are_refused(power):
    big = 1 << power
    M, N, K = 1, 1, 256
    #       0  1  2  3  4  5  6  7  8  9  10 11 12    13 14 15 16 17 18 19 20    21 22
    good = [0, P, K, P, M, P, K, 0, P, 2, 1, 2, None, 1, M, N, K, P, N, 0, None, 0, None]
    refuse("fp8_block_grouped_gemm", good, [
        ({2: big}, UNSUPPORTED), ({6: big}, UNSUPPORTED), ({18: big}, UNSUPPORTED), ({18: big, 19: 1}, UNSUPPORTED),
        ({9: big}, UNSUPPORTED), ({9: big, 15: 256, 18: 256}, UNSUPPORTED)])
    good = [1, P, 128, P, K, P, 128, 0, P, 1, N, 0, None, 1, 128, N, K, P, N, 0, None, 0, None]
    refuse("fp8_block_grouped_gemm", good, [({2: big}, UNSUPPORTED), ({6: big}, UNSUPPORTED), ({18: big}, UNSUPPORTED)])
    #       0  1  2  3  4  5  6  7  8  9  10 11 12 13 14 15 16 17 18   19
    good = [0, 1, P, K, P, P, K, 0, P, P, 1, M, N, K, P, N, 0, P, 256, None]
    refuse("fp8_grouped_gemm", good, [({3: big}, UNSUPPORTED), ({6: big}, UNSUPPORTED)])


@pytest.mark.parametrize("power", [30, 48, 57, 60, 62])
def test_layer_strides_of_any_size_are_refused(power):
    big = 1 << power
    T, H, I, E, k = 4, 256, 128, 8, 2
    size = fq.lib().fp8_moe_few_tokens_workspace_size(T, H, I, k)
    good = [P, T, H, H, P, P, k, P, H, 2 * I * H, P, 2, 1, 4, P, I, H * I, P, 1, 1, 2, E, I, P, H, P, size, None]
    refuse("fp8_moe_few_tokens", good, [({3: big}, UNSUPPORTED), ({8: big}, UNSUPPORTED), ({15: big}, UNSUPPORTED), ({1: 128, 3: big}, UNSUPPORTED)])


@pytest.mark.parametrize("rows,cols", [(1 << 31, 1), (1, 1 << 31), (1 << 24, 129 * 128), (1 << 62, 1), ((1 << 63) - 1, 1), (1 << 40, 1 << 40)])
def test_quantizers_of_more_tiles_than_a_launch_takes(rows, cols):
    big = (1 << 63) - 1
    refuse("fp8_block_quant_rowwise", [P, rows, cols, big, P, big, P, big, None], [({}, UNSUPPORTED)])
    refuse("fp8_block_quant_dual", [P, rows, cols, big, P, big, P, big, P, big, P, big, None], [({}, UNSUPPORTED)])
    refuse("fp8_block_quant_weights", [P, 1, rows, cols, big, P, big, P, big, P, None], [({}, UNSUPPORTED)])
