"""The few-token layer on every path that its launches take, against 64 bits with the bounds that it
promises: 16 significant bits between the products, sums in 32 bits, one rounding to bf16."""
from __future__ import annotations

import pytest
import torch

from tests import block_cases, moelib, planlib

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def fq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import fp8_quantization_grouped_amd as m
    m.lib()
    return m


def weights(g, E, n, k):
    """Random finite codes and factors that make rows of about unit size."""
    w = torch.randint(0, 256, (E, n, k), dtype=torch.uint8, device=DEV, generator=g)
    w[(w & 0x7F) == 0x7F] = 0x38
    up = lambda v: -(-v // 128)
    return w, (0.5 + torch.rand(E, up(n), up(k), device=DEV, generator=g)) / (120 * k ** 0.5)


@pytest.mark.parametrize("name", list(block_cases.LAYERS))
def test_layer(fq, name):
    (T, k, E, H, I, few), gate_up, down = block_cases.LAYERS[name]
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    assert planlib.stream(False, T, k, E, H, I, cus) == gate_up and planlib.stream(True, T, k, E, H, I, cus) == down
    g = torch.Generator(device=DEV).manual_seed(T + H)
    w13, s13 = weights(g, E, 2 * I, H)
    w2, s2 = weights(g, E, H, I)
    x = torch.randn(T, H, device=DEV, generator=g).to(torch.bfloat16)
    # the experts in use are the last ones; most tokens share one, and one choice is of an expert elsewhere
    ids = torch.randint(E - few, E, (T, k), device=DEV, generator=g).to(torch.int32)
    ids[: T * 3 // 4, 0] = E - 1
    if k > 1:
        ids[T // 2, 1] = -1
    share = torch.rand(T, k, device=DEV, generator=g) + 0.25
    y = fq.fp8_moe_few_tokens(x, ids, share, w13, s13, w2, s2)
    n1, n2 = moelib.additions(-(-H // 128), gate_up[2]), moelib.additions(-(-I // 128), down[2], 2)
    moelib.check(y, *moelib.formula(x, ids, share, w13, s13, w2, s2, n1, n2))
    assert torch.equal(y, fq.fp8_moe_few_tokens(x, ids, share, w13, s13, w2, s2))
