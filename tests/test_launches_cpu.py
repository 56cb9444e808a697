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


def test_gradient_without_a_loss_hands_no_sequences_on():
    """Without dloss the kernel has no ends to read, whatever stands in the arguments: of the losses' part nothing but
    nulls and zeros reaches it, and the launch is the one of a call that was given nothing."""
    T, E = 100, 8

    def back(counts, sequences, S):
        return "moe_route_backward", (P, 1, T, E, E, 0, P, 2, P, 1, 1.0, None, counts, sequences, S, 2 * P, E)

    (status, bare), *others = launches(back(None, None, 0), back(3 * P, 5 * P, 50), back(None, 5 * P, -7), back(3 * P, None, 1 << 30))
    assert status == OK and len(bare) == 1 and "route_back" in bare[0].kernel
    size = 15 * 8 + 3 * 4  # the argument's pointers and sizes, the last of them the number of sequences
    assert bare[0].arg[size - 4:size] == bytes(4)
    for status, made in others:
        assert status == OK and made[0]._replace(arg=b"") == bare[0]._replace(arg=b"")
        assert made[0].arg[:size] == bare[0].arg[:size]


@pytest.mark.parametrize("rows,cols", [(1, (1 << 27) - 33), (1, (1 << 27) - 32), (3, (1 << 27) - 31), (0, (1 << 27) - 32), (0, (1 << 27) - 31),
                                       (1, (1 << 27) - 1), (5, 1 << 27)])
def test_norm_backward_starts_nothing_that_it_cannot_finish(rows, cols):
    """A launch takes fewer than 2^32 threads, the join of dw too: columns past that are refused before the first."""
    need = fq.fp8_rms_norm_backward_workspace_size(rows, cols)
    (status, made), = launches(("fp8_rms_norm_backward", (P, cols, None, 0, 0, P, rows, cols, cols, P, P, 0, P, cols, P, P, need)))
    if cols > (1 << 27) - 32:
        assert status == UNSUPPORTED and not made
    else:
        assert status == OK and len(made) == (2 if rows else 1)
        assert all(l.grid[0] * l.block[0] < 1 << 32 and l.grid[1:] == l.block[1:] == [1, 1] for l in made)
