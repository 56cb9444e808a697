"""What lies between the few-token layer's two products: its range and its 16 significant bits."""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"

ONE, TWO, HALF, MINUS = 0x38, 0x40, 0x30, 0xB8  # e4m3fn bytes of 1, 2, 0.5 and -1


@pytest.fixture(scope="module")
def fq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import fp8_quantization_grouped_amd as m
    m.lib()
    return m


def experts(E, H, I, s13=1.0, s2=1.0):
    """Zero weights [E, 2I, H] and [E, H, I] on the host, and factors."""
    up = lambda n: -(-n // 128)
    return (torch.zeros(E, 2 * I, H, dtype=torch.uint8), torch.full((E, up(2 * I), up(H)), s13, device=DEV),
            torch.zeros(E, H, I, dtype=torch.uint8), torch.full((E, up(H), up(I)), s2, device=DEV))


@pytest.mark.parametrize("T", [1, 20, 40])
@pytest.mark.parametrize("sign", [1, -1])
def test_a_value_past_the_largest_bf16(fq, T, sign):
    """h = 1023 * 2^118 is finite in 32 bits and rounds to infinity in bf16."""
    H, I = 16, 16
    w13, s13, w2, s2 = experts(1, H, I)
    w13[0, :I, 0] = ONE       # gate: x0 = 31 * 2^40, so silu(gate) = gate
    w13[0, I:, 1] = ONE       # up: x1 = 33 * 2^78
    w2[0, :, 0] = HALF
    x = torch.zeros(T, H, dtype=torch.bfloat16, device=DEV)
    x[:, 0], x[:, 1] = 31.0 * 2.0 ** 40, sign * 33.0 * 2.0 ** 78
    ids = torch.zeros(T, 1, dtype=torch.int32, device=DEV)
    y = fq.fp8_moe_few_tokens(x, ids, torch.full((T, 1), 2.0 ** -100, device=DEV), w13.to(DEV), s13, w2.to(DEV), s2)
    want = torch.tensor(sign * 1023.0 * 2.0 ** 17).to(torch.bfloat16)
    assert bool((y.cpu() == want).all())


@pytest.mark.parametrize("T", [1, 16, 20, 40, 70, 128])
def test_the_second_plane_reaches_the_result(fq, T):
    """Two choices that share what one bf16 plane holds, with weights 1 and -1: what is left of them is the
    rest that the second plane holds, and every operation on it is exact."""
    H = I = 256
    g = torch.Generator().manual_seed(T)
    # values 1 .. 15 and 0.25 .. 240, of 4 significant bits
    codes = lambda lo, hi: torch.randint(lo, hi, (I,), generator=g, dtype=torch.uint8)
    a, b = codes(0x38, 0x58), codes(0x28, 0x78)
    w13, s13, w2, s2 = experts(2, H, I)
    for e in range(2):
        w13[e, :I, 0] = ONE
        w13[e, I:, 1] = a
        w2[e, range(H), range(I)] = ONE
    w13[0, I:, 200] = b
    x = torch.zeros(T, H, dtype=torch.bfloat16, device=DEV)
    x[:, 0], x[:, 1], x[:, 200] = 64.0, 1.0, 2.0 ** -12  # silu(64) = 64; h = 64 (a + b 2^-12) and 64 a
    ids = torch.tensor([[0, 1]] * T, dtype=torch.int32, device=DEV)
    share = torch.tensor([[1.0, -1.0]] * T, device=DEV)
    y = fq.fp8_moe_few_tokens(x, ids, share, w13.to(DEV), s13, w2.to(DEV), s2)
    want = b.view(torch.float8_e4m3fn).double() * 2.0 ** -6
    assert torch.equal(y.cpu().double(), want.expand(T, H))
