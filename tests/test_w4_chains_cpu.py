"""The compiled 4-bit kernels keep 32 cycles between matrix steps of different
opcodes that share an accumulator (see tests/mfma_chain_check.py), checked on the
device assembly the build writes; the check itself is pinned on hand-written
snippets."""
import os

import pytest

from invariant_matmul_amd import build
from tests.mfma_chain_check import chain_hazards, file_chain_hazards

START = "v_mfma_f32_16x16x32_bf16 v[0:3], v[8:11], v[12:15], 0"
STEP = "v_mfma_f32_16x16x32_f16 v[0:3], v[8:11], v[12:15], v[0:3]"
OTHER = "v_mfma_f32_16x16x32_f16 v[20:23], v[8:11], v[12:15], 0"


@pytest.mark.parametrize("kernel,least", [("w4_rows_kernel", 48), ("w4_tile_kernel", 12)])
def test_steps_of_different_opcodes_keep_their_distance(kernel, least):
    if not os.path.exists(build.W4_ASM):
        pytest.skip("device assembly not built (run invariant_matmul_amd.build)")
    with open(build.W4_ASM) as f:
        hazards, n, mixed = file_chain_hazards(f.read(), kernel)
    # (the fp16 half of the kernels starts on another opcode, the bf16 half on its own)
    assert n >= least and 2 * mixed == n, (n, mixed)
    assert not hazards, {k[:90]: list(v.items())[:3] for k, v in list(hazards.items())[:5]}


def check(*lines):
    return list(chain_hazards([*lines, "s_endpgm"])[0].values())


def test_the_check_itself():
    assert check(START, STEP) == [0]
    assert check(START, "s_nop 7", "v_mov_b32_e32 v30, 0", "s_mov_b32 s0, 0", STEP) == [12]
    assert check(START, OTHER, STEP) == [16]
    assert check(START, OTHER, OTHER, STEP) == []
    assert check(START, "s_nop 15", "s_nop 15", STEP) == []
    assert check(START, STEP.replace("_f16", "_bf16")) == []                      # the same opcode
    assert check(START, STEP.replace("v[0:3]", "v[20:23]")) == []                 # another accumulator
    assert check(START, STEP.replace("v[0:3]", "v[2:5]")) == [0]                  # a part of it
    assert check(START, STEP.replace("bf16", "f16").replace("v[0:3]", "v[0:3]", 1)
                 .replace(", v[0:3]", ", 0"), STEP) == []                         # written anew in between
    # the short way round a branch, and a start at the end of a loop
    assert check(START, "s_cbranch_scc1 .LBB0_1", OTHER, OTHER, ".LBB0_1:", STEP) == [0]
    assert check("s_nop 0", ".LBB0_1:", STEP, "s_nop 15", "s_nop 15", START, "s_cbranch_scc1 .LBB0_1") == [0]
