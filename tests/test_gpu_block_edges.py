"""Edges of the block-scaled products: contractions of length zero, refusals of overlapping rows."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def fq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import fp8_quantization_grouped_amd as m
    m.lib()
    return m


def offsets(*ends):
    return torch.tensor(ends, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("ends,status", [((3, 8), (0, -1)), ((3, 7), (1, 1)), ((9, 8), (1, 0)), ((-1, 8), (1, 0))])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_nothing_to_sum(fq, ends, status, out):
    """K == 0: the forward's output is zeros, and the offsets check is reported as at any other K."""
    ws = torch.full((256,), 0x55, dtype=torch.uint8, device=DEV)
    e = lambda *s, dtype=torch.uint8: torch.empty(*s, dtype=dtype, device=DEV)
    y = fq.fp8_block_grouped_gemm(fq.GEMM_FWD_MGROUPED, e(8, 0), e(0, 8, dtype=torch.float32), e(2, 5, 0), e(2, 1, 0, dtype=torch.float32),
                                  offsets(*ends), out_dtype=out, workspace=ws)
    assert y.shape == (8, 5) and not bool(y.any())
    assert fq.gemm_offsets_status(ws) == status


def test_overlapping_rows_are_refused(fq):
    M, N, K, G = 64, 32, 512, 2
    z = lambda *s, dtype=torch.uint8: torch.zeros(*s, dtype=dtype, device=DEV)
    f = torch.float32
    off, F, W = offsets(32, 64), fq.GEMM_FWD_MGROUPED, fq.GEMM_WGRAD_KGROUPED
    x = z(M, 256, dtype=torch.bfloat16)
    for bad in (lambda: fq.fp8_block_grouped_gemm(F, z(M, K), z(1, M, dtype=f).expand(4, M), z(G, N, K), z(G, 1, 4, dtype=f), off),
                lambda: fq.fp8_block_grouped_gemm(W, z(N, K), z(1, N, dtype=f).expand(4, N), z(N, K), z(4, N, dtype=f), offsets(100, 512)),
                lambda: fq.fp8_block_grouped_gemm(W, z(N, K), z(4, N, dtype=f), z(N, K), z(1, N, dtype=f).expand(4, N), offsets(100, 512)),
                lambda: fq.fp8_block_quant_dual(x, s_rows=z(1, M, dtype=f).expand(2, M)),
                lambda: fq.fp8_block_quant_dual(x, q_t=z(1, M).expand(256, M)),
                lambda: fq.fp8_block_quant_weights(x, 2, q_t=z(1, M).expand(256, M))):
        with pytest.raises(RuntimeError, match="invalid"):
            bad()
    # rows of one factor each for all of the contraction, as rows of their own, are what was meant
    y = fq.fp8_block_grouped_gemm(F, z(M, K) + 0x38, (z(1, M, dtype=f) + 0.5).expand(4, M).contiguous(), z(G, N, K) + 0x38, z(G, 1, 4, dtype=f) + 1, off)
    assert bool((y == 256.0).all())
