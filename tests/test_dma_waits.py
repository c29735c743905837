"""Wait states in front of the library's loads into LDS.

The loads are inline assembly, so the compiler does not see that a memory
instruction follows and inserts none of the waits one needs: one state between
a scalar instruction's write of M0 and a load that takes its LDS address from
it, five between a vector instruction's write of a scalar register and a load
that reads it.  The listing of the built library has them on every path if
they lie on the straight line in front of each load."""

import os
import re
import struct
import subprocess
import tempfile

import pytest

from moe_expert_layer_r3_amd import ops

OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"
pytestmark = pytest.mark.skipif(not (os.path.exists(ops.LIB_PATH) and os.path.exists(OBJDUMP)),
                                reason="library not built, or no objdump")
MAGIC = b"__CLANG_OFFLOAD_BUNDLE__"
M0_STATES, SGPR_STATES = 1, 5


def code_objects(path):
    """The gfx950 ELF images inside the library."""
    with open(path, "rb") as f:
        data = f.read()
    at = data.find(MAGIC)
    while at >= 0:
        n, p = struct.unpack_from("<Q", data, at + 24)[0], at + 32
        for _ in range(n):
            off, size, idlen = struct.unpack_from("<QQQ", data, p)
            name = data[p + 24:p + 24 + idlen]
            p += 24 + idlen
            if size and b"gfx950" in name:
                yield data[at + off:at + off + size]
        at = data.find(MAGIC, at + 1)


def scalars(text):
    """Numbers of the scalar registers in an operand list."""
    out = set()
    for a, b in re.findall(r"\bs\[(\d+):(\d+)\]", text):
        out |= set(range(int(a), int(b) + 1))
    return out | {int(a) for a in re.findall(r"\bs(\d+)\b", text)}


def missing_waits(lines):
    """(loads, complaints) of a disassembly."""
    loads, bad, line, fn = 0, [], [], ""
    for text in lines:
        if re.match(r"^[0-9a-f]+ <.*>:$", text):
            fn, line = text, []
            continue
        if not text.startswith("\t"):
            continue
        text = text.split("//")[0].strip()
        op, _, args = text.partition(" ")
        if op.startswith("global_load_lds") or (op.startswith("buffer_load") and args.endswith(" lds")):
            loads += 1
            reads, states = scalars(args), 0
            for prev, pargs in reversed(line):
                if states >= SGPR_STATES:
                    break
                written = pargs.split(",")[0]
                if states < M0_STATES and prev.startswith("s_") and re.search(r"\bm0\b", written):
                    bad.append(f"{fn} M0 {states} states before: {text}")
                if prev.startswith("v_") and scalars(written) & reads:
                    bad.append(f"{fn} {prev} {pargs} {states} states before: {text}")
                if states < M0_STATES and (prev.startswith("s_cbranch") or prev == "s_branch"):
                    bad.append(f"{fn} a branch inside the waits of: {text}")
                states += int(pargs, 0) + 1 if prev == "s_nop" else 1
        line.append((op, args))
        del line[:-16]
    return loads, bad


def test_scan_sees_missing_waits():
    """The scan itself, on lines made up for it."""
    f = "0000 <f>:"
    load, pair = "\tglobal_load_lds_dwordx4 v1, s[4:5]", "\tbuffer_load_dwordx4 v1, s[8:11], 0 offen lds"
    for lines, n in (([f, "\ts_mov_b32 m0, s3", load], 1), ([f, "\ts_mov_b32 m0, s3", "\ts_nop 0", load], 0),
                     ([f, "\tv_readfirstlane_b32 s5, v0", "\ts_nop 3", load], 1),
                     ([f, "\tv_readfirstlane_b32 s5, v0", "\ts_nop 4", load], 0),
                     ([f, "\tv_readfirstlane_b32 s9, v0", "\ts_add_u32 m0, m0, 0x400", "\ts_nop 0", pair], 1),
                     ([f, "\tv_readfirstlane_b32 s7, v0", pair], 0)):
        assert missing_waits(lines)[0] == 1 and len(missing_waits(lines)[1]) == n, lines


def test_loads_into_lds_have_their_waits():
    loads, bad = 0, []
    for elf in code_objects(ops.LIB_PATH):
        with tempfile.NamedTemporaryFile(suffix=".elf") as f:
            f.write(elf)
            f.flush()
            text = subprocess.run([OBJDUMP, "-d", "--mcpu=gfx950", f.name], capture_output=True, text=True, check=True).stdout
        n, b = missing_waits(text.splitlines())
        loads, bad = loads + n, bad + b
    assert loads > 1000
    assert not bad, f"{len(bad)} of {loads} loads: " + "; ".join(bad[:4])
