"""Wait states behind vector instructions whose results other lanes read.

Some maxima and minima are inline assembly, which the compiler's own check of
these waits need not see through: a DPP or lane-swap instruction reads a vector
register two states after a vector instruction wrote it at the earliest, a lane
read one state after, and one state lies between a transcendental
instruction and a plain one that takes its result.  The listing of the built
library is checked on the straight line in front of each such reader."""

import os
import re
import subprocess
import tempfile

import pytest

from moe_expert_layer_r3_amd import ops
from test_dma_waits import OBJDUMP, code_objects

pytestmark = pytest.mark.skipif(not (os.path.exists(ops.LIB_PATH) and os.path.exists(OBJDUMP)),
                                reason="library not built, or no objdump")
TRANS = ("v_exp_", "v_rcp_", "v_sqrt_", "v_rsq_", "v_log_", "v_sin_", "v_cos_")
REGISTERS = re.compile(r"\bv(?:\[(\d+):(\d+)\]|(\d+)\b)")


def vectors(text):
    """Numbers of the vector registers in an operand list."""
    out = set()
    for a, b, one in REGISTERS.findall(text):
        out |= {int(one)} if one else set(range(int(a), int(b) + 1))
    return out


def missing_waits(lines):
    """(readers, complaints) of a disassembly."""
    readers, bad, line, fn = 0, [], [], ""
    for text in lines:
        if not text.startswith("\t"):
            if text.endswith(">:"):
                fn, line = text, []
            continue
        op, _, args = text.split("//")[0].strip().partition(" ")
        if not op.startswith("v_"):
            line.append((op, args))
            continue
        target, _, sources = args.partition(",")
        swap = op.startswith("v_permlane")
        if swap or op.endswith("_dpp") or "quad_perm" in args or " row_" in args:
            need, by = 2, "v_"
        elif op.startswith(("v_readlane", "v_readfirstlane")):
            need, by = 1, "v_"
        else:
            need, by = 0 if op.startswith(TRANS) else 1, TRANS
        if need:
            readers += by == "v_"
            reads, states = None, 0
            for prev, pargs in reversed(line[-3:]):
                if states >= need:
                    break
                if prev.startswith(by):
                    reads = vectors(args if swap else sources) if reads is None else reads
                    wrote = pargs if prev.startswith("v_permlane") else pargs.partition(",")[0]
                    if vectors(wrote) & reads:
                        bad.append(f"{fn} {prev} {pargs} {states} states before: {text.strip()}")
                states += int(pargs, 0) + 1 if prev == "s_nop" else 1
        line.append((op, args))
    return readers, bad


def test_scan_sees_missing_waits():
    """The scan itself, on lines made up for it."""
    f = "0000 <f>:"
    made = "\tv_max_f64 v[2:3], v[4:5], v[6:7]"
    dpp, swap = "\tv_mov_b32_dpp v8, v3 quad_perm:[1,0,3,2] row_mask:0xf bank_mask:0xf", "\tv_permlane16_swap_b32_e32 v9, v2"
    exp, use = "\tv_exp_f32_e32 v1, v0", "\tv_max_f32_e32 v4, v1, v2"
    for lines, n in (([f, made, dpp], 1), ([f, made, "\ts_nop 0", dpp], 1), ([f, made, "\ts_nop 1", dpp], 0),
                     ([f, made, swap], 1), ([f, made, "\tv_mov_b32_e32 v20, v21", "\ts_nop 0", swap], 0),
                     ([f, made, "\tv_readlane_b32 s0, v2, 3"], 1), ([f, made, "\ts_nop 0", "\tv_readlane_b32 s0, v2, 3"], 0),
                     ([f, exp, use], 1), ([f, exp, "\ts_nop 0", use], 0), ([f, exp, "\tv_exp_f32_e32 v4, v1"], 0)):
        assert len(missing_waits(lines)[1]) == n, lines


def test_results_have_their_waits():
    readers, bad = 0, []
    for elf in code_objects(ops.LIB_PATH):
        with tempfile.NamedTemporaryFile(suffix=".elf") as f:
            f.write(elf)
            f.flush()
            text = subprocess.run([OBJDUMP, "-d", "--mcpu=gfx950", f.name], capture_output=True, text=True, check=True).stdout
        n, b = missing_waits(text.splitlines())
        readers, bad = readers + n, bad + b
    assert readers > 10000
    assert not bad, f"{len(bad)} of {readers} readers: " + "; ".join(bad[:4])
