"""The build's check of the wait states before direct loads into LDS: on listings
made here, and on the built library (disassembled; no GPU needed)."""
import os

import pytest

from precision_moe_numerics_quant_amd import wait_states
from test_capi_exports import LIB


def listing(*code):
    """A disassembly of one function of four-byte instructions, labels as 'L:' and branches to them by name."""
    at, lines = {}, []
    for c in code:
        if c.endswith(":"):
            at[c[:-1]] = len(lines)
        else:
            lines.append(c)
    out = ["0000000000001000 <f>:"]
    for i, c in enumerate(lines):
        op, _, to = c.partition(" ")
        if to in at:
            c = f"{op} {(at[to] - i - 1) % 65536}"
        out.append(f"\t{c:<60}// {0x1000 + 4 * i:012X}: BF800000")
    return "\n".join(out)


LOAD = ("s_mov_b32 m0, s9", "s_nop 0", "buffer_load_dwordx4 v5, s[40:43], s11 offen lds")


@pytest.mark.parametrize("write,bad", [
    ("v_readlane_b32 s41, v255, 3", True), ("v_readfirstlane_b32 s11, v2", True), ("v_cmp_lt_u32_e64 s[42:43], v1, v2", True),
    ("v_add_co_u32_e64 v1, s[40:41], v2, v3", True),
    ("v_readlane_b32 s44, v255, 3", False), ("v_readlane_b32 s4, v255, 3", False), ("v_add_u32_e32 v1, s41, v2", False),
    ("s_mov_b32 s41, s2", False), ("s_add_u32 s11, s2, s3", False), ("v_readfirstlane_b32 m0, v2", False)])
def test_writes_before_a_load(write, bad):
    """Two wait states behind a vector write of what the load reads (m0 is written anew in between)."""
    n, found = wait_states.violations(listing(write, *LOAD, "s_endpgm"))
    assert n == 1 and len(found) == bad


@pytest.mark.parametrize("between,bad", [([], True), (["s_nop 0"], True), (["v_mov_b32_e32 v1, v2"] * 2, True), (["v_mov_b32_e32 v1, v2"] * 3, False),
                                         (["s_nop 2"], False), (["s_nop 1"], True), (["s_nop 0", "s_add_u32 s2, s2, 4", "s_nop 0"], False)])
def test_distance(between, bad):
    n, found = wait_states.violations(listing("v_readlane_b32 s41, v255, 3", *between, *LOAD, "s_endpgm"))
    assert n == 1 and bool(found) == bad


def test_along_every_path():
    """A write at the end of a loop before a load at its start; one on the branch that skips the wait; one that no path leads from."""
    wait = "s_nop 7"
    back = listing(wait, "L:", *LOAD, wait, "v_readlane_b32 s40, v1, 0", "s_cbranch_scc1 L", "s_endpgm")
    assert len(wait_states.violations(back)[1]) == 1
    skip = listing("v_readlane_b32 s40, v1, 0", "s_cbranch_scc1 L", wait, "L:", *LOAD, "s_endpgm")
    assert len(wait_states.violations(skip)[1]) == 1
    dead = listing("s_branch L", "v_readlane_b32 s40, v1, 0", "s_branch M", "L:", *LOAD, "M:", "s_endpgm")
    assert wait_states.violations(dead) == (1, [])


def test_the_library():
    if not os.path.exists(LIB):
        pytest.skip("libmoe4.so not built (run __graft_entry__.build())")
    if not os.path.exists(wait_states.OBJDUMP):
        pytest.skip("no llvm-objdump")
    assert wait_states.check(LIB) > 0
