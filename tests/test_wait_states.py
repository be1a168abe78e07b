"""Wait states in the built library's gfx950 code, read on the host (no GPU).

The hardware does not wait by itself where a vector instruction writes a scalar
register (v_readlane and the like) and a memory instruction reads it within the
next five, or where m0 is written right before a load to LDS.  The compiler puts
instructions between them, but not around memory instructions in inline
assembly, which have to bring their own.
"""
import os
import re
import shutil
import subprocess
import tempfile

import pytest

from exact_row_top_amd import LIB_PATH
from test_codeobj import _code_objects

OBJDUMP = next((p for p in ("/opt/rocm/llvm/bin/llvm-objdump", shutil.which("llvm-objdump"))
                if p and os.path.exists(p)), None)
MEMORY = re.compile(r"(global|buffer|flat|scratch)_")


def _scalars(operand):
    m = re.match(r"s\[(\d+):(\d+)\]$", operand)
    if m:
        return range(int(m[1]), int(m[2]) + 1)
    m = re.match(r"s(\d+)$", operand)
    return [int(m[1])] if m else ["m0"] if operand == "m0" else []


def _short_waits(lines):
    """(kernel, instruction, wait states) of what follows too closely, in straight lines."""
    kernel, at, written, m0, bad = "", 0, {}, None, []
    for line in lines:
        label = re.match(r"[0-9a-f]+ <(.+)>:", line)
        if label:
            kernel, written, m0 = label[1], {}, None
            continue
        text = line.split("//")[0].strip()
        if not text:
            continue
        op, _, rest = text.partition(" ")
        args = [a.strip().split(" ")[0] for a in rest.split(",")]
        if MEMORY.match(op):
            reads = [r for a in args for r in _scalars(a)] + (["m0"] if "_lds_" in op else [])
            bad += [(kernel, text, at - written[r] - 1) for r in reads if r in written and at - written[r] - 1 < 5]
            if "_lds_" in op and m0 is not None and at - m0 - 1 < 1:
                bad.append((kernel, text, at - m0 - 1))
        outs = args[:2] if "_co_" in op or op.startswith("v_div_scale") or op.startswith("v_mad_u64") else args[:1]
        for r in (r for a in outs for r in _scalars(a)):
            if op.startswith("v_"):
                written[r] = at
            elif op.startswith("s_"):
                written.pop(r, None)
                m0 = at if r == "m0" else m0
        at += int(rest, 0) + 1 if op == "s_nop" else 1
        if op in ("s_branch", "s_endpgm", "s_setpc_b64"):
            written, m0 = {}, None
    return bad


def test_the_reading_finds_what_is_too_close():
    close = ["0 <k>:", "v_readlane_b32 s2, v4, 0", "v_readlane_b32 s3, v5, 0", "s_mov_b32 m0, s4", "s_nop 0",
             "global_load_lds_dwordx4 v7, s[2:3]"]
    assert [b[2] for b in _short_waits(close)] == [3, 2]
    apart = close[:4] + ["s_nop 3"] + close[5:]
    assert _short_waits(apart) == []
    assert len(_short_waits(["0 <k>:", "s_mov_b32 m0, s4", "global_load_lds_dwordx4 v[2:3], off"])) == 1
    assert len(_short_waits(["0 <k>:", "v_readfirstlane_b32 m0, v1", "s_nop 3", "global_load_lds_dwordx4 v[2:3], off"])) == 1


@pytest.mark.skipif(not os.path.exists(LIB_PATH) or OBJDUMP is None, reason="needs the built library and llvm-objdump")
def test_memory_instructions_come_late_enough():
    loads = 0
    for _, co in _code_objects(LIB_PATH):
        with tempfile.NamedTemporaryFile(suffix=".co", delete=False) as f:
            f.write(co)
        try:
            lines = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", f.name], capture_output=True, text=True,
                                   check=True).stdout.splitlines()
        finally:
            os.unlink(f.name)
        loads += sum("global_load_lds" in line for line in lines)
        bad = _short_waits(lines)
        assert not bad, (len(bad), bad[:3])
    assert loads
