"""Every output tile of the block-scaled products against 64-bit arithmetic, bf16 and float32 outputs:
groups that end inside a tile, empty groups, wide and unaligned stores, stores past the cache."""
from __future__ import annotations

import pytest
import torch

from tests import block_cases, planlib
from tests import test_gpu_block as block

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import fp8_quantization_grouped_amd as m
    m.lib()
    return m


def cases(table):
    return [pytest.param(tile, *case, id="-".join(map(str, (tile, *case)))) for tile, cs in table.items() for case in cs]


def cus():
    return torch.cuda.get_device_properties(0).multi_processor_count


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("tile,M,N,K,G,kind", cases(block_cases.FORWARD))
def test_forward(fq, tile, M, N, K, G, kind, out):
    assert planlib.tile(True, M, N, K, G, cus()) == tile
    block.test_forward(fq, M, N, K, G, kind, out)


@pytest.mark.parametrize("tile,M,N,K,G,kind", cases(block_cases.DATA_GRADIENT))
def test_data_gradient(fq, tile, M, N, K, G, kind):
    assert planlib.tile(True, M, K, N, G, cus()) == tile
    block.test_data_gradient(fq, M, N, K, G, kind)


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("tile,M,N,K,G,kind", cases(block_cases.WEIGHT_GRADIENT))
def test_weight_gradient(fq, tile, M, N, K, G, kind, out):
    assert planlib.tile(False, M, N, K, G, cus()) == tile
    block.test_weight_gradient(fq, M, N, K, G, kind, out)
