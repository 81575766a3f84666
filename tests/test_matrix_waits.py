"""Results of matrix instructions that hand-written LDS writes read (CPU: the generated code of the sources is read).

The compiler puts the wait states between a matrix instruction and an instruction of its own that reads the result; of
an instruction in inline assembly it does not know the operands' hazards.  The states it takes on gfx950 before an LDS
write: 8 behind an instruction of 4 passes, 12 behind one of 8, 20 behind one of 16.
"""
import os
import re
import shutil
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest

from combine_route_histogram_amd.build import HIPCC_FLAGS, INC, PKG, hipcc

STATES = {"v_mfma_i32_16x16x64_i8": 8, "v_mfma_i32_32x32x32_i8": 12}   # any other: 20
MOST = 20


def registers(operand):
    m = re.fullmatch(r"([va])\[(\d+):(\d+)\]", operand)
    if m:
        return {(m[1], i) for i in range(int(m[2]), int(m[3]) + 1)}
    m = re.fullmatch(r"([va])(\d+)", operand)
    return {(m[1], int(m[2]))} if m else set()


class Op:
    def __init__(self, text, inline):
        name, _, rest = text.partition(" ")
        self.name, self.inline, self.text = name.strip(), inline, text
        self.args = [a.strip() for a in rest.split(",")] if rest else []
        self.states = int(self.args[0], 0) + 1 if name == "s_nop" else 1
        writes = self.args and (name.startswith("v_") or re.match(r"(ds_read|global_load|buffer_load|scratch_load|flat_load)", name))
        self.writes = registers(self.args[0]) if writes else set()

    @property
    def matrix(self):
        return self.name.startswith(("v_mfma", "v_smfmac"))


def blocks(lines):
    """Functions of an assembly listing as {function: (ops, predecessors of each op)}."""
    out, name, ops, labels, jumps, inline = {}, None, [], {}, [], False

    def close():
        if name is None:
            return
        before = [[] for _ in ops]
        for i, op in enumerate(ops):
            if i + 1 < len(ops) and op.name not in ("s_branch", "s_endpgm", "s_setpc_b64"):
                before[i + 1].append(i)
        for i, label in jumps:
            if labels[label] < len(ops):
                before[labels[label]].append(i)
        out[name] = (ops, before)

    for line in lines:
        text = line.split("; ")[0].strip() if not line.strip().startswith(";") else line.strip()
        if text == ";;#ASMSTART":
            inline = True
        elif text == ";;#ASMEND":
            inline = False
        elif re.fullmatch(r"_Z\w+:", text):
            close()
            name, ops, labels, jumps = text[:-1], [], {}, []
        elif re.fullmatch(r"\.L\w+:", text):
            labels[text[:-1]] = len(ops)
        elif text.startswith(".section") and ops:
            close()
            name = None
        elif name is not None and re.match(r"[a-z]\w+( |\t|$)", text) and not text.startswith("."):
            op = Op(re.sub(r"\s+", " ", text), inline)
            if op.name.startswith(("s_cbranch", "s_branch")):
                jumps.append((len(ops), op.args[0]))
            ops.append(op)
    close()
    return out


def short_waits(ops, before):
    """(write, matrix instruction, states between) of inline LDS writes that come too soon, over every path."""
    found = []
    for i, op in enumerate(ops):
        if not (op.inline and op.name.startswith("ds_")):
            continue
        reads = set().union(*(registers(a.split(" ")[0]) for a in op.args))
        todo, seen = [(p, 0, frozenset(reads)) for p in before[i]], {}
        while todo:
            p, states, live = todo.pop()
            if states >= MOST or not live or seen.get((p, live), MOST) <= states:
                continue
            seen[(p, live)] = states
            q = ops[p]
            if q.matrix and q.writes & live and states < STATES.get(q.name, MOST):
                found.append((op.text, q.text, states))
            live = live - q.writes
            todo += [(r, states + q.states, live) for r in before[p]]
    return found


def listing(name, out):
    subprocess.run([hipcc(), *HIPCC_FLAGS, "-w", "-I", INC, "--cuda-device-only", "-S", os.path.join(PKG, "csrc", f"mdc_{name}.hip"),
                    "-o", out], check=True, capture_output=True, timeout=600)
    with open(out) as f:
        return f.read().splitlines()


def test_the_reader_sees_a_short_wait():
    """Of a listing made by hand: over the loop's back edge, past a copy, and far enough."""
    text = """
_Zk:
.LBB0_1:
\tds_read_b128 v[20:23], v9
\tv_mfma_i32_16x16x64_i8 v[0:3], v[4:7], v[8:11], v[0:3]
\ts_cbranch_scc1 .LBB0_1
\tv_mov_b32_e32 v3, v2
\t;;#ASMSTART
\tds_write_b128 v12, v[0:3]
\t;;#ASMEND
\ts_nop 3
\t;;#ASMSTART
\tds_write_b32 v12, v1
\t;;#ASMEND
\tv_mov_b32_e32 v1, v2
\t;;#ASMSTART
\tds_write_b32 v12, v1
\t;;#ASMEND
\ts_endpgm
""".splitlines()
    ops, before = blocks(text)["_Zk"]
    assert [(w, s) for w, _, s in short_waits(ops, before)] == [("ds_write_b128 v12, v[0:3]", 2), ("ds_write_b32 v12, v1", 7)]


@pytest.mark.skipif(shutil.which(hipcc()) is None, reason="needs hipcc")
def test_waits_before_hand_written_lds_writes(tmp_path):
    names = ("gmm", "gmm8", "moe")   # the sources with such writes
    with ThreadPoolExecutor(len(names)) as pool:
        lists = list(pool.map(lambda n: listing(n, str(tmp_path / f"{n}.s")), names))
    writes, bad = 0, []
    for name, lines in zip(names, lists):
        functions = blocks(lines)
        assert functions, name
        for f, (ops, before) in functions.items():
            writes += sum(op.inline and op.name.startswith("ds_write") for op in ops)
            bad += [(name, f, *b) for b in short_waits(ops, before)]
    assert writes > 100
    assert not bad, "\n".join(map(str, bad))
