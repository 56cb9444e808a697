"""moe_balance and moe_route_backward at the ends of what they take."""
from __future__ import annotations

import pytest
import torch

from tests.test_gpu_route_grad import fq  # noqa: F401

pytestmark = pytest.mark.gpu
I32 = torch.int32


@pytest.mark.parametrize("S", [1, 64, 65, 1000])
@pytest.mark.parametrize("E", [8, 300])
def test_no_tokens_in_any_number_of_sequences(fq, S, E):  # noqa: F811
    l, ids = torch.empty(0, E, device="cuda"), torch.empty(0, 2, dtype=I32, device="cuda")
    loss, counts = torch.full((S,), 7.0, device="cuda"), torch.full((S, E), 7, dtype=I32, device="cuda")
    seq = torch.zeros(S, dtype=I32, device="cuda")
    fq.moe_balance(l, ids, sequences=seq, loss=loss, counts=counts)
    assert bool((loss == 0).all()) and bool((counts == 0).all())
    assert fq.moe_route_backward(l, ids, None, dloss=torch.ones(S, device="cuda"), counts=counts, sequences=seq).shape == (0, E)
