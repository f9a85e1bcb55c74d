"""Waits that the hardware leaves to the program, looked for in the built library's gfx950 code (no GPU).

The kernels copy global memory to LDS by inline assembly, which the compiler's own count of wait states does not
look into, so the disassembly is read back and every path through it is followed:

 * a copy to LDS takes its address from M0, and one wait state has to lie between a write of M0 and the copy;
 * M0 is not the kernels' to keep: each copy's block saves it and puts it back;
 * a matrix instruction's result is not there for other units until 8 wait states (16 x 16 x 32 in bf16, four passes)
   or 10 (16 x 16 x 4 in fp32, eight passes) have gone by, on whatever path the reader is reached;
 * the walk back of the gated delta rule waits for a stage's copies by their place in line: at most 5 later memory
   operations may be outstanding, so at least 5 have to lie behind the last copy, on every path.
"""
import os
import re
import shutil
import subprocess

import pytest

from mamba_ssd_sequence_chunked_amd import _build

LLVM = "/opt/rocm/llvm/bin"
OBJDUMP = os.path.join(LLVM, "llvm-objdump")

pytestmark = pytest.mark.skipif(not os.path.exists(OBJDUMP), reason="needs the ROCm disassembler")


def registers(token):
    """The registers of an operand, as (class, number)."""
    token = token.strip().lstrip("-").strip("|")
    m = re.match(r"^([vas])(\d+)$", token)
    if m:
        return [(m[1], int(m[2]))]
    m = re.match(r"^([vas])\[(\d+):(\d+)\]$", token)
    if m:
        return [(m[1], i) for i in range(int(m[2]), int(m[3]) + 1)]
    return [("m0", 0)] if token == "m0" else []


class Ins:
    __slots__ = ("op", "args", "at", "target", "states", "succ")

    def __init__(self, op, args, at, target):
        self.op, self.args, self.at, self.target = op, [a.split()[0] if a.split() else "" for a in args.split(",")], at, target
        self.states = int(self.args[0], 0) + 1 if op == "s_nop" else 1      # wait states that pass with it
        self.succ = ()

    @property
    def is_copy(self):
        return "lds_dword" in self.op

    @property
    def is_memory(self):
        return self.op.startswith(("global_", "buffer_", "flat_", "scratch_"))


def functions(path):
    """{name: [Ins]} of a code object, with every instruction's possible successors."""
    text = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", path], capture_output=True, text=True, check=True).stdout
    out, body = {}, None
    for line in text.splitlines():
        m = re.match(r"^[0-9a-f]+ <(.+)>:$", line)
        if m:
            body = out.setdefault(m[1], [])
            continue
        m = re.match(r"^\t(\S+)\s*(.*?)\s*// ([0-9A-F]+):(.*)$", line)
        if m and body is not None:
            to = re.search(r"<.+?(?:\+0x([0-9a-f]+))?>", m[4]) if m[1].startswith(("s_cbranch", "s_branch")) else None
            body.append(Ins(m[1], m[2], int(m[3], 16), int(to[1] or "0", 16) if to else None))
    for body in out.values():
        where = {i.at - body[0].at: n for n, i in enumerate(body)}
        for n, i in enumerate(body):
            nxt = [n + 1] if n + 1 < len(body) and i.op not in ("s_branch", "s_endpgm", "s_setpc_b64") else []
            i.succ = tuple(nxt + ([where[i.target]] if i.target in where else []))
    return out


@pytest.fixture(scope="module")
def code(tmp_path_factory):
    """All kernels of the library."""
    if not os.path.exists(_build.LIB_PATH):
        _build.build()
    d = tmp_path_factory.mktemp("code")
    lib = shutil.copy(_build.LIB_PATH, d)
    subprocess.run([OBJDUMP, "--offloading", lib], cwd=d, capture_output=True, check=True)
    out = {}
    for f in sorted(os.listdir(d)):
        if f.endswith("gfx950"):
            out.update(functions(os.path.join(d, f)))
    assert any("delta_chain" in n for n in out) and any("chunk_scan" in n for n in out)
    return out


def test_copies_to_lds_wait_for_their_address(code):
    seen = 0
    for name, body in code.items():
        for n, i in enumerate(body):
            if not (i.op.startswith("s_") and i.args[0] == "m0"):
                continue
            # no copy right behind a write of M0, on any path
            for k in i.succ:
                assert not body[k].is_copy, (name, hex(body[k].at))
        seen += sum(i.is_copy for i in body)
    assert seen > 1000


def test_copies_to_lds_restore_m0(code):
    for name, body in code.items():
        for n, i in enumerate(body):
            if not i.is_copy:
                continue
            back = body[n + 1]
            assert (back.op, back.args[0]) == ("s_mov_b32", "m0"), (name, hex(i.at))
            save = [(j.op, j.args) for j in body[n - 3:n]]
            assert save[0] == ("s_mov_b32", [back.args[1], "m0"]) and save[2][0] == "s_nop", (name, hex(i.at))


# wait states behind a matrix instruction before another unit may touch its result
PASSES = {"v_mfma_f32_16x16x32_bf16": 8, "v_mfma_f32_16x16x4_f32": 10}


def _touched(i):
    """(registers read or written by another unit than the matrix cores, registers written)."""
    every = [registers(a) for a in i.args]
    if i.op.startswith("v_mfma"):
        return every[1] + every[2], every[0]             # (an accumulator passed on is the matrix cores' own affair)
    if i.op.startswith(("v_", "ds_")) or i.is_memory:
        out = every[0] if i.op.startswith("v_") or "load" in i.op or "read" in i.op else []
        return sum(every, []), out
    return [], []


def _waits(body, start, end, pending, passes, seen=None):
    """Follows a block from {register: wait states still to pass}; returns what is pending behind it."""
    now, due = 0, {r: n for r, n in pending.items()}
    for i in body[start:end]:
        touched, written = _touched(i)
        if seen is not None:
            for r in touched:
                if r[0] in "va" and due.get(r, 0) > now:
                    seen.append((i, r, due[r] - now))
        for r in written:
            due.pop(r, None)
        now += i.states
        if i.op.startswith("v_mfma"):
            need = passes.get(i.op, passes.get(i.op.rsplit("_e64", 1)[0], 18))
            for r in written:
                due[r] = now + need
    return {r: t - now for r, t in due.items() if t > now}


def early_uses(body, passes):
    """[(instruction, register, wait states missing)] over every path."""
    heads = sorted({0} | {k for n, i in enumerate(body) if i.target is not None for k in (*i.succ, n + 1)} - {len(body)})
    end = dict(zip(heads, heads[1:] + [len(body)]))
    entry, todo = {0: {}}, [0]
    while todo:
        h = todo.pop()
        out = _waits(body, h, end[h], entry[h], passes)
        for k in body[end[h] - 1].succ:
            old = entry.get(k)
            new = dict(old or {})
            for r, n in out.items():
                new[r] = max(new.get(r, 0), n)
            if new != old:
                entry[k] = new
                todo.append(k)
    early = []
    for h in heads:
        if h in entry:
            _waits(body, h, end[h], entry[h], passes, early)
    return early


def test_matrix_results_are_waited_for(code):
    kernels = 0
    for name, body in code.items():
        if not any(i.op.startswith("v_mfma") for i in body):
            continue
        kernels += 1
        early = early_uses(body, PASSES)
        assert not early, (name, [(i.op, hex(i.at), r, n) for i, r, n in early[:3]])
    assert kernels > 100


def test_group_products_wait_before_the_branch(code):
    """The products of a group's keys and queries are read behind a loop whose length is not known and a branch: the
    longest wait, 16 states, is spent before it, whatever the compiler counts."""
    kernels = 0
    for name, body in code.items():
        if "delta_prep" in name:
            kernels += 1
            early = [e for e in early_uses(body, {op: 16 for op in PASSES}) if e[0].op.startswith("ds_write")]
            assert not early, (name, [(i.op, hex(i.at), r, n) for i, r, n in early[:3]])
    assert kernels == 4


def test_walk_back_counts_its_stores(code):
    kernels = 0
    for name, body in code.items():
        if "delta_rev" not in name:
            continue
        before = {}
        for n, i in enumerate(body):
            for k in i.succ:
                before.setdefault(k, []).append(n)
        if not any(i.op == "s_barrier" for i in body):
            continue                     # one wavefront: nothing tells this wait from the compiler's own
        waits = []
        for n, i in enumerate(body):
            if i.op == "s_waitcnt" and "vmcnt(5)" in i.args[0]:
                k = n + 1
                while body[k].op.startswith(("s_", "v_")) and body[k].op != "s_barrier" and body[k].target is None:
                    k += 1
                if body[k].op == "s_barrier":            # (the compiler's own waits stand before an operand's use)
                    waits.append(n)
        assert waits, name
        kernels += 1
        # the copies of the loop (the one block copied before it is waited for with everything else)
        inside, todo = set(waits), list(waits)
        while todo:
            new = [k for k in body[todo.pop()].succ if k not in inside]
            inside.update(new)
            todo += new
        for w in waits:
            fewest, todo, ends = {w: 0}, [w], []
            while todo:
                n = todo.pop()
                for p in before.get(n, []):
                    if p not in inside:
                        continue
                    if body[p].is_copy:
                        ends.append(fewest[n])
                        continue
                    c = fewest[n] + body[p].is_memory
                    if c < fewest.get(p, 99):
                        fewest[p] = c
                        todo.append(p)
            assert ends and min(ends) >= 5, (name, hex(body[w].at), ends)
    assert kernels >= 12
