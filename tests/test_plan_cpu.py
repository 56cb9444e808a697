"""The launch rules of the block-scaled kernels, without a GPU."""
from __future__ import annotations

import random

import pytest

from tests import block_cases, planlib


def test_the_rules_count_the_chips_compute_units():
    """The same products on chips of other sizes: a 256-tile for every compute unit there is."""
    for cus in (64, 128, 256, 304):
        assert planlib.tile(True, 16 * 256, cus // 16 * 256, 512, 1, cus) == "256x256"  # one each
        assert planlib.tile(True, 15 * 256, cus // 16 * 256, 512, 1, cus) == "128x128"
        assert planlib.tile(False, 4096, cus // 16 * 256, 512, 8, cus) == "256x256"     # 8 x 2 row tiles
        assert planlib.tile(False, 4096, cus // 16 * 256 - 256, 512, 8, cus) == "128x128"
        # the layer: 33 tokens take passes of 64 where the waves fill half of the chip, else of 32
        assert planlib.stream(False, 33, 1, 1, 512, 16 * 8 * cus, cus)[:2] == (4, 64)
        assert planlib.stream(False, 33, 1, 1, 512, 16 * (8 * cus - 1), cus)[:2] == (2, 32)


@pytest.mark.parametrize("fwd", [True, False])
def test_small_products_take_small_tiles(fwd):
    assert planlib.tile(fwd, 1, 1, 16, 1) == "64x64"
    assert planlib.tile(fwd, 1 << 20, 1 << 14, 1 << 14, 2048) == "256x256"


def test_a_plans_parts_fit_the_staging_buffer():
    rng = random.Random(1)
    for _ in range(20000):
        T, E, k = rng.randint(1, 128), rng.randint(1, 1024), rng.randint(1, 32)
        H, I = 16 * int(2 ** rng.uniform(0, 12)), 16 * int(2 ** rng.uniform(0, 12))
        for down in (False, True):
            mt, tokens, parts = planlib.stream(down, T, k, E, H, I)
            assert mt in (1, 2, 4) and parts in (1, 2, 4) and tokens & (tokens - 1) == 0
            assert tokens <= 16 * mt and (tokens >= T or tokens == 16 * mt)
            assert parts * (2 if down else 1) * tokens * 256 <= 8192 * (4 if mt == 1 else 8) // 2
            assert parts <= (4 if mt == 1 else (2 if down else 4) if mt == 2 else 1)  # what is compiled
            assert parts <= max(1, -(-(I if down else H) // 128))


def _cases(table):
    return [(tile, case) for tile, cases in table.items() for case in cases]


@pytest.mark.parametrize("tile,case", _cases(block_cases.FORWARD))
def test_forward_cases_take_their_tile(tile, case):
    M, N, K, G, _ = case
    assert planlib.tile(True, M, N, K, G) == tile


@pytest.mark.parametrize("tile,case", _cases(block_cases.DATA_GRADIENT))
def test_data_gradient_cases_take_their_tile(tile, case):
    M, N, K, G, _ = case
    assert planlib.tile(True, M, K, N, G) == tile  # the same product with N and K exchanged


@pytest.mark.parametrize("tile,case", _cases(block_cases.WEIGHT_GRADIENT))
def test_weight_gradient_cases_take_their_tile(tile, case):
    M, N, K, G, _ = case
    assert planlib.tile(False, M, N, K, G) == tile


def test_every_tile_has_cases():
    """Several groups, empty ones, columns that allow wide stores and columns that do not."""
    for table, tiles in ((block_cases.FORWARD, planlib.TILES), (block_cases.WEIGHT_GRADIENT, ["64x64", "128x128", "256x256"])):
        assert sorted(table) == sorted(tiles)
        for tile in tiles:
            assert any(c[3] > 1 for c in table[tile])
            assert any(c[1] % 8 == 0 for c in table[tile]) and any(c[1] % 8 for c in table[tile])
        assert {c[4] for c in table["256x256"]} >= {"cuts", "empties"}


@pytest.mark.parametrize("name", list(block_cases.LAYERS))
def test_layer_cases_take_their_plans(name):
    (T, k, E, H, I, _), gate_up, down = block_cases.LAYERS[name]
    assert planlib.stream(False, T, k, E, H, I) == gate_up
    assert planlib.stream(True, T, k, E, H, I) == down


def test_the_layers_paths_have_cases():
    """Each size of a pass with more blocks of the contraction than are staged at once, and more blocks of a
    part than a wave holds factors of (64), in both products."""
    seen = set()
    for (T, k, E, H, I, _), *plans in block_cases.LAYERS.values():
        for down, (mt, tokens, parts) in enumerate(plans):
            blocks = -(-(-(-(I if down else H) // 128)) // parts)
            rows = parts * (2 if down else 1) * tokens * 256  # bytes that one block of every part takes
            chunk = 1
            while 2 * chunk * rows <= 8192 * (4 if mt == 1 else 8) // 2 and chunk < blocks:
                chunk *= 2
            seen.add((down, mt, "turns") if blocks > 2 * chunk else None)
            seen.add((down, "factors") if blocks > 64 else None)
            seen.add((down, mt, "passes") if T > tokens else None)
    assert seen >= {(d, mt, "turns") for d in (0, 1) for mt in (1, 2, 4)} | {(0, "factors"), (1, "factors"), (0, 4, "passes"), (0, 2, "passes")}
