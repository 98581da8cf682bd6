"""Distances around the matrix instructions that newton_schulz.hip writes as
inline assembly (CPU only, on the disassembly of the built library).

The compiler does not take those for matrix instructions, so it neither counts
nor fills the wait states that they need.  What has to hold, on every path
through the code:
- a result of a matrix instruction is touched by anything but a matrix
  instruction 19 or more wait states later (18 is the most that the hardware
  asks for, after the longest of them);
- a register that a matrix instruction reads was written by a vector
  instruction 5 or more wait states before (2 is what the hardware asks for).
An instruction counts as one wait state, `s_nop n` as n + 1.  A wave has lanes
at work until an instruction masks them: before, a branch on whether it has any
goes one way.
"""

import os
import re
import shutil
import subprocess

import numpy as np
import pytest

import sharded_bucket_plan_amd as sbp

OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"
AFTER, BEFORE = 19, 5  # wait states
ACC = 512  # where the accumulation registers begin in a set of both kinds

_REG = re.compile(r"\b([va])(?:\[(\d+):(\d+)\]|(\d+)\b)")


def _registers(text):
    out = []
    for kind, lo, hi, one in _REG.findall(text):
        lo, hi = (int(lo), int(hi)) if lo else (int(one), int(one))
        out += [r + (ACC if kind == "a" else 0) for r in range(lo, hi + 1)]
    return np.array(out, int)


class _Instruction:
    def __init__(self, line):
        code, _, at = line.partition("//")
        op, _, operands = code.strip().partition(" ")
        self.text, self.op = code.strip(), op
        self.at = int(at.split(":")[0], 16)
        self.target = None
        m = re.search(r"<([^>+]+)(?:\+0x([0-9a-f]+))?>", at)
        if op.startswith(("s_branch", "s_cbranch")):
            self.target = int(m.group(2) or "0", 16)
        first, _, rest = operands.partition(",")
        self.mfma = op.startswith("v_mfma")
        self.waits = int(operands) + 1 if op == "s_nop" else 1
        vector = op.startswith("v_")
        self.writes = _registers(first) if vector else np.array([], int)
        self.reads = _registers(rest)
        self.touches = _registers(operands)
        self.vector = vector and not self.mfma
        self.masks = first.strip().startswith("exec") or "saveexec" in op or op.startswith("v_cmpx")


def _kernels(lines):
    """Name and instructions of every function of a disassembly."""
    name, body = None, []
    for line in lines:
        m = re.match(r"[0-9a-f]+ <(.*)>:", line)
        if m:
            if name:
                yield name, body
            name, body = m.group(1), []
        elif name and "//" in line:
            body.append(_Instruction(line))
    if name:
        yield name, body


def hazards(body):
    """Instructions that come too soon, in words, over all paths."""
    start = body[0].at
    index = {i.at - start: k for k, i in enumerate(body)}
    heads = {0}
    for k, i in enumerate(body):
        if i.target is not None:
            heads |= {index[i.target], k + 1}
    heads = sorted(h for h in heads if h < len(body))
    end_of = dict(zip(heads, heads[1:] + [len(body)]))
    far = np.full((2, 2 * ACC), 1000)  # since written by a matrix, a vector instruction
    entry = {0: (far, True)}  # and whether some lane is surely at work
    todo, found = [0], set()
    while todo:
        head = todo.pop()
        since, lanes = entry[head][0].copy(), entry[head][1]
        for k in range(head, end_of[head]):
            i = body[k]
            if i.mfma:
                near = i.reads[since[1][i.reads] < BEFORE]
                if near.size:
                    found.add(f"{i.at:x}: {i.text}: reads what a vector instruction just wrote")
            else:
                near = i.touches[since[0][i.touches] < AFTER]
                if near.size:
                    found.add(f"{i.at:x}: {i.text}: touches what a matrix instruction just wrote")
            since += i.waits
            if i.mfma:
                since[0][i.writes] = 0
                since[1][i.writes] = 1000
            elif i.vector:
                since[1][i.writes] = 0
            if i.masks:
                lanes = i.op == "s_or_b64"  # the end of a masked part
        last = body[end_of[head] - 1]
        nexts = [] if last.op in ("s_endpgm", "s_branch") else [end_of[head]]
        if last.target is not None:
            nexts.append(index[last.target])
        if lanes and last.op in ("s_cbranch_execnz", "s_cbranch_execz"):
            nexts = nexts[1:] if last.op == "s_cbranch_execnz" else nexts[:1]
        for n in nexts:
            if n >= len(body):
                continue
            was = entry.get(n, (far, True))
            now = np.minimum(was[0], since), was[1] and lanes
            if n not in entry or (now[0] < was[0]).any() or now[1] != was[1]:
                entry[n] = now
                todo.append(n)
    return sorted(found)


def _body(text):
    return [_Instruction(f"{t} // {4 * k:012X}: 0 {to}") for k, (t, to) in enumerate(text)]


def test_hazards_are_found():
    """Planted in a few lines of assembly: too near in line, round a loop, and
    over a branch; and nothing where the distances hold."""
    mfma = ("v_mfma_f32_16x16x32_f16 a[0:3], v[0:3], v[4:7], a[0:3]", "")
    read, end = ("v_accvgpr_read_b32 v9, a2", ""), ("s_endpgm", "")
    wait = ("s_nop 15", "")
    assert len(hazards(_body([mfma, read, end]))) == 1
    assert hazards(_body([mfma, wait, wait, read, end])) == []
    assert len(hazards(_body([mfma, wait, read, end]))) == 1
    write = ("v_mov_b32_e32 v5, 0", "")
    assert len(hazards(_body([write, mfma, end]))) == 1
    assert hazards(_body([write, ("s_nop 4", ""), mfma, end])) == []
    # the loop's last vector write is near its first matrix instruction
    back = ("s_cbranch_scc1 1", "<f+0x0>")
    assert len(hazards(_body([mfma, ("s_nop 4", ""), write, back, end]))) == 1
    # skipping the waits
    skip = ("s_cbranch_scc1 1", "<f+0x10>")
    assert len(hazards(_body([mfma, skip, wait, wait, read, end]))) == 1
    assert len(hazards(_body([mfma, ("ds_write_b32 v1, a0", ""), end]))) == 1


@pytest.mark.skipif(shutil.which(OBJDUMP) is None, reason="needs llvm-objdump")
def test_large_tile_keeps_its_distances(tmp_path):
    """The accumulators that are held in place by hand, in the library as built."""
    sbp.lib()
    library = shutil.copy(sbp.LIB_PATH, tmp_path)
    subprocess.run([OBJDUMP, "--offloading", library], cwd=tmp_path, check=True,
                   capture_output=True)
    checked = {}
    for part in sorted(os.listdir(tmp_path)):
        if not part.endswith("gfx950"):
            continue
        r = subprocess.run([OBJDUMP, "-d", part], cwd=tmp_path, check=True, capture_output=True,
                           text=True)
        lines = r.stdout.splitlines()
        for name, body in _kernels(lines):
            if "ns_product_kernel" in name and "TileILi256" in name:
                checked[name] = len([i for i in body if i.mfma])
                found = hazards(body)
                assert not found, f"{name}: {len(found)}, of them {found[:5]}"
    # gram, poly and the three forms of apply; 64 products a slice
    assert len(checked) == 5 and all(n >= 64 * 8 for n in checked.values()), checked
