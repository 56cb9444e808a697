"""Launches of the norm's and the router's calls at the ends of what they take (tests/launchlib.py), without a GPU."""
from __future__ import annotations

import pytest

import fp8_quantization_grouped_amd as fq
from tests.launchlib import launches

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
P = 4096


def balance(T, E, S, workspace, size):
    return "moe_balance", (P, 1, T, E, E, 0, P, 2, P, S, P, P, workspace, size)


@pytest.mark.parametrize("E", [8, 300])
def test_balance_of_no_tokens_takes_no_workspace(E):
    """A null workspace where the size asked for is 0, with any number of sequences; the join alone leaves the zeros."""
    S = [1, 3, 64, 65, 1000, (1 << 22) - 1]
    assert [fq.moe_balance_workspace_size(0, E, s) for s in S] == [0] * len(S)
    for s, (status, made) in zip(S, launches(*(balance(0, E, s, None, 0) for s in S))):
        assert status == OK and len(made) == 1 and "balance_join" in made[0].kernel and made[0].grid == [s, 1, 1]
