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


def test_a_workspace_serves_fewer_rows_too():
    """A program that holds one workspace for its largest batch: no smaller one is refused."""
    rows = sorted({r + d for r in (1, 16, 255, 256, 257, 512, 4095, 4096, 4097, 8192, 65536, 131072, 1 << 20) for d in (-1, 0, 1)} | set(range(0, 1100)))
    for cols in (7, 64, 512, 513, 1024, 7168, 8192, 8193, 16384, 20000):
        sizes = [fq.fp8_rms_norm_backward_workspace_size(r, cols) for r in rows if r]
        assert sizes == sorted(sizes) and sizes[-1] <= 256 * cols * 4
    for E in (1, 8, 16, 17, 64, 65, 256, 300, 1024):
        last = None
        for S in (1, 2, 5, 9, 16, 64, 65, 1000):
            sizes = [fq.moe_balance_workspace_size(r, E, S) for r in rows]
            assert sizes == sorted(sizes)
            assert last is None or all(a <= b for a, b in zip(last, sizes))
            last = sizes


def test_the_launches_stay_inside_the_workspace():
    """What the kernels take of it, by the launches' own numbers: blocks of sums in the norm's backward, places in the
    balance's (the argument's pointers to the masses, the counts and the groups' parts, and the rows of a chunk)."""
    sizes = [(T, E, S) for T in (513, 4096, 4097, 5000, 65536, 300000) for E in (8, 64, 300, 1024) for S in (1, 3, 9, 70)]
    calls = [balance(T, E, S, P, fq.moe_balance_workspace_size(T, E, S)) for T, E, S in sizes]
    word = lambda l, at: int.from_bytes(l.arg[at:at + 8], "little")
    for (T, E, S), (status, made) in zip(sizes, launches(*calls)):
        need = fq.moe_balance_workspace_size(T, E, S)
        assert status == OK
        sums, join = made[0], made[1] if len(made) > 1 else None
        if join is None:
            assert need == 0
            continue
        mass, part, groups, rows = (word(join, 88 + 8 * i) for i in range(4))
        places = -(-T // rows) + S
        assert sums.grid[0] == places - S and mass == P and part == P + 4 * places * E and part + 4 * places * E <= P + need
        if groups:
            assert groups == P + 8 * places * E and groups + 4 * S * join.grid[1] <= P + need
        else:
            assert join.grid == [S, 1, 1]
    for rows, cols in ((1, 64), (257, 64), (300, 7168), (257, 7168), (5000, 16384), (1000, 20000)):
        need = fq.fp8_rms_norm_backward_workspace_size(rows, cols)
        (status, made), = launches(("fp8_rms_norm_backward", (P, cols, None, 0, 0, P, rows, cols, cols, P, P, 0, P, cols, P, P, need)))
        assert status == OK and made[0].grid[0] * cols * 4 <= need
