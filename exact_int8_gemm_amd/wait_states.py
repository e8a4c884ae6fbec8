"""Wait states in front of the copies from buffers into LDS, in the machine code of the built library.

The copies are written as inline assembly (csrc/lds_copy.h), where the compiler adds no wait states of its own.  The
instruction set asks for two (its table of wait states that a program has to insert):
  * five between a vector instruction that writes a scalar register (a lane read, also one that brings back a spilled
    register) and a memory instruction that reads it, as a copy reads its buffer's descriptor;
  * one between a scalar write of M0 and a copy into LDS, which takes its address from there.
A copy that comes too early reads the register's old value: another buffer's rows, or an address outside of any.
An instruction is one wait state, s_nop N is N + 1.

Where descriptors come from is the register allocator's choice, so the build looks at what it made: a library with a copy
that comes too early is not put in place.
"""
from __future__ import annotations

import collections
import os
import re
import shutil
import subprocess
import tempfile

LINE = re.compile(r"^\s+([a-z]\w+)\s*(.*?)\s*//\s*([0-9A-F]{8,}):(.*)$")
FUNCTION = re.compile(r"^[0-9a-f]+ <(.+)>:$")
SGPR_STATES, M0_STATES = 5, 1

Instruction = collections.namedtuple("Instruction", "at name operands target")


def _operands(text):
    return [t.strip() for t in re.split(r",(?![^\[]*\])", text)]


def _scalars(operand):
    """Numbers of the scalar registers that an operand names (-2, -1: vcc)."""
    first = operand.split(" ")[0] if operand else ""
    m = re.fullmatch(r"s(?:(\d+)|\[(\d+):(\d+)\])", first)
    if m:
        return {int(m[1])} if m[1] else set(range(int(m[2]), int(m[3]) + 1))
    return {"vcc": {-2, -1}, "vcc_lo": {-2}, "vcc_hi": {-1}}.get(first, set())


def parse(text):
    """{function: [Instruction]} of llvm-objdump's listing; target is a branch's offset in its function."""
    out, code = {}, None
    for line in text.splitlines():
        m = FUNCTION.match(line)
        if m:
            code = out.setdefault(m[1], [])
            continue
        m = LINE.match(line)
        if m and code is not None:
            target = None
            if m[1].startswith(("s_branch", "s_cbranch")):
                t = re.search(r"<[^<>+]+(?:\+0x([0-9a-f]+))?>\s*$", m[4])
                target = int(t[1] or "0", 16)
            code.append(Instruction(int(m[3], 16), m[1], _operands(m[2]), target))
    return out


def is_copy(i):
    return i.name.startswith(("buffer_load", "global_load", "scratch_load")) and (
        "_lds_" in i.name or "lds" in i.operands[-1].split(" "))


def _vector_writes(i):
    if not i.name.startswith("v_"):
        return set()
    carry = re.match(r"v_((add|sub|subrev)_co|(addc|subb|subbrev)_co|div_scale|mad_(u64_u32|i64_i32))", i.name)
    return _scalars(i.operands[0]) | (_scalars(i.operands[1]) if carry else set())


def _writes_m0(i):
    return i.name.startswith("s_") and i.operands[0] == "m0"


def _states(i):
    return int(i.operands[0], 0) + 1 if i.name == "s_nop" else 1


def too_early(code):
    """A function's instructions -> (copies, [(copy, writer, wait states between)]) over all paths to each copy."""
    place = {i.at: n for n, i in enumerate(code)}
    before = collections.defaultdict(list)
    for n, i in enumerate(code):
        if i.name not in ("s_branch", "s_endpgm", "s_setpc_b64") and n + 1 < len(code):
            before[n + 1].append(n)
        if i.target is not None:
            before[place[code[0].at + i.target]].append(n)
    copies, found = 0, []
    for n, copy in enumerate(code):
        if not is_copy(copy):
            continue
        copies += 1
        read = set().union(*map(_scalars, copy.operands))
        nearest, todo = {}, [(n, 0)]
        while todo:
            at, passed = todo.pop()
            for p in before[at]:
                if read & _vector_writes(code[p]) or (passed < M0_STATES and _writes_m0(code[p])):
                    found.append((copy, code[p], passed))
                upto = passed + _states(code[p])
                if upto < SGPR_STATES and nearest.get(p, SGPR_STATES) > upto:
                    nearest[p] = upto
                    todo.append((p, upto))
    return copies, found


def check(library, objdump, arch):
    """(copies, [(function, address, copy, writer, wait states between)]) of all of `library`'s code for `arch`."""
    copies, found = 0, []
    with tempfile.TemporaryDirectory() as folder:
        shutil.copy(library, os.path.join(folder, "lib.so"))
        subprocess.run([objdump, "--offloading", "lib.so"], cwd=folder, check=True, capture_output=True)
        for f in sorted(os.listdir(folder)):
            if not f.endswith("--" + arch):
                continue
            text = subprocess.run([objdump, "-d", "--no-show-raw-insn", f], cwd=folder, check=True, capture_output=True,
                                  text=True).stdout
            for name, code in parse(text).items():
                n, wrong = too_early(code)
                copies += n
                found += [(name, "%x" % c.at, c.name, w.name, states) for c, w, states in wrong]
    return copies, found
