"""Inline assembly in the device code (CPU only): a memory instruction there has the wait states before
it that gfx9 needs and that the compiler inserts only around its own instructions."""
from __future__ import annotations

import os

import pytest

from fp8_quantization_grouped_amd import _build

BLOCK = "\t;;#ASMSTART\n{}\t;;#ASMEND\n"


def block(*lines):
    return BLOCK.format("".join(f"\t{line}\n" for line in lines))


LOAD = "buffer_load_dwordx4 v40, s[40:43], s2 offen lds"


def test_loads_without_waits_are_found():
    assert _build.unguarded_asm(block("s_mov_b32 m0, s76", LOAD)) == [LOAD]
    assert _build.unguarded_asm(block("s_nop 7", "s_mov_b32 m0, s76", LOAD)) == [LOAD]      # M0 alone
    assert _build.unguarded_asm(block("s_mov_b32 m0, s76", "s_nop 2", LOAD)) == [LOAD]      # a descriptor's registers
    assert _build.unguarded_asm(block(LOAD.replace(" lds", ""))) == [LOAD.replace(" lds", "")]
    assert _build.unguarded_asm(block("s_nop 0") + "\ts_nop 7\n" + block("s_mov_b32 m0, s1", LOAD)) == [LOAD]


def test_loads_with_waits_pass():
    assert _build.unguarded_asm(block("s_mov_b32 m0, s76", "s_nop 3", LOAD)) == []
    assert _build.unguarded_asm(block("s_nop 3", "s_mov_b32 m0, s76", "s_nop 0", LOAD)) == []
    assert _build.unguarded_asm(block("s_nop 4", LOAD.replace(" lds", ""))) == []
    assert _build.unguarded_asm("\ts_mov_b32 m0, s1\n\t" + LOAD + "\n" + block("s_waitcnt vmcnt(0)")) == []  # the compiler's own


def test_every_kernel_has_them():
    srcs = sorted(f[:-4] for f in os.listdir(_build.CSRC) if f.endswith(".hip"))
    missing = [n for n in srcs if not os.path.exists(_build.device_asm(n))]
    if missing:
        pytest.skip(f"device assembly not kept for {missing} (run __graft_entry__.build())")
    blocks = 0
    for n in srcs:
        text = open(_build.device_asm(n)).read()
        blocks += sum("lds" in b for b in _build.ASM_BLOCK.findall(text))
        assert not _build.unguarded_asm(text), (n, _build.unguarded_asm(text)[:4])
    assert blocks > 0  # the loads to LDS are written that way
