"""The machine code of the transfers into LDS, which are inline assembly: the compiler
keeps no wait states around an instruction it does not see. On gfx950 such a load needs
one wait state behind a scalar write of M0 (the LDS address it reads), and five behind a
vector instruction's write of a scalar register it reads (its buffer resource or offset,
restored from a spill, say). Disassembles the built library; needs no GPU."""
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "combine_top_router_amd", "libmoe.so")
OBJDUMP = shutil.which("llvm-objdump") or "/opt/rocm/llvm/bin/llvm-objdump"
M0_WAIT, SGPR_WAIT = 1, 5

pytestmark = pytest.mark.skipif(not (os.path.exists(LIB) and os.path.exists(OBJDUMP)),
                                reason="needs the built library and llvm-objdump")


def scalars(operands):
    """Numbers of the scalar registers that an operand text names; M0 is "m0"."""
    out = set()
    for lo, hi, one, m0 in re.findall(r"\bs\[(\d+):(\d+)\]|\bs(\d+)\b|\b(m0)\b", operands):
        out |= {"m0"} if m0 else {int(one)} if one else set(range(int(lo), int(hi) + 1))
    return out


def hazards(listing):
    """(transfers into LDS, [function, writer, transfer] of those that come too early)."""
    count, bad, func, before = 0, [], "", []
    for line in listing:
        head = re.match(r"[0-9a-f]+ <(.*)>:", line)
        if head:
            func, before = head[1], []
            continue
        text = line.split("//")[0].strip()
        if not text or not line[0].isspace():
            continue
        op, _, rest = text.partition(" ")
        if op.startswith("buffer_load") and rest.split()[-1] == "lds":
            count += 1
            reads, waited = scalars(rest) | {"m0"}, 0
            for kind, writes, states, what in reversed(before):
                if waited >= SGPR_WAIT:
                    break
                if writes & reads and (kind == "v" or waited < M0_WAIT and "m0" in writes):
                    bad.append((func, what, text))
                    break
                waited += states
        # what it writes: its first operand, and a carry or scale flag in the second
        n = 0 if op[:2] not in ("s_", "v_") else 2 if "_co_" in op or "div_scale" in op else 1
        writes = scalars(" ".join(rest.split(", ")[:n])) if ", " in rest else set()
        states = int(rest, 0) + 1 if op == "s_nop" else 1
        before = before[-7:] + [(op[0], writes, states, text)]
    return count, bad


def test_the_check_sees_what_it_should():
    def listing(*lines):
        return ["0000 <f>:"] + ["\t" + l + "   // 0000" for l in lines]

    load = "buffer_load_dwordx4 v1, s[4:7], s9 offen lds"
    for writer, states, early in (("s_mov_b32 m0, s3", 0, True), ("s_mov_b32 m0, s3", 1, False),
                                  ("v_readlane_b32 s6, v3, 1", 4, True),
                                  ("v_readlane_b32 s6, v3, 1", 5, False),
                                  ("v_readfirstlane_b32 s9, v3", 0, True),
                                  ("v_readfirstlane_b32 m0, v3", 4, True),
                                  ("v_cmp_lt_u32_e64 s[6:7], v2, v3", 0, True),
                                  ("v_add_co_u32_e64 v2, s[4:5], v2, v3", 4, True),
                                  ("v_readlane_b32 s8, v3, 1", 0, False),
                                  ("s_add_i32 s4, s3, 1", 0, False)):
        for between in (["s_nop %d" % (states - 1)] if states else [], ["v_mov_b32 v9, v8"] * states):
            n, bad = hazards(listing(writer, *between, load))
            assert n == 1 and bool(bad) == early, (writer, between)
    assert hazards(listing("s_mov_b32 m0, s3", "buffer_load_dwordx4 v[1:4], v5, s[4:7], 0 offen")) == (0, [])


def test_transfers_into_lds_keep_their_wait_states(tmp_path):
    lib = shutil.copy(LIB, tmp_path)
    subprocess.run([OBJDUMP, "--offloading", lib], cwd=tmp_path, check=True, capture_output=True)
    objects = [str(f) for f in tmp_path.iterdir() if "gfx950" in f.name]
    assert objects
    count = 0
    for obj in objects:
        text = subprocess.run([OBJDUMP, "-d", obj], check=True, capture_output=True, text=True).stdout
        n, bad = hazards(text.splitlines())
        assert not bad, (len(bad), bad[:3])
        count += n
    assert count > 1000  # the matrix products' tiles all come this way
