"""The counted waits of linear attention's walks, looked for in the built library's gfx950 code (no GPU).

A walk copies chunks into a ring of LDS stages by inline assembly and waits for a chunk's copies by their place in line: the
memory operations issued behind them may be outstanding, so at least as many as the wait lets pass have to lie behind
them.  Those are the stores of a chunk's outputs (two for each tile of columns) or, where only states are wanted and the
ring has three stages, the next chunk's copies.  A store that the compiler merged with another, split or moved to the other
side of the wait or of the copies would break the count, so the disassembly is read back:

 * a wait before a chunk's barrier counts what the kernel's shape says;
 * every straight piece of code that stores a chunk's outputs holds all of its stores;
 * a chunk's order is wait, barrier, copies, stores: no copy can be reached from a store without a barrier between, and on
   every way back from a counted wait that meets a chunk's stores before its copies there are enough of them;
 * where copies are counted, a chunk has as many.

A segment of a chain hands its state on: all of it has left the wavefront (a wait for everything) and a barrier has
been passed before the word that says so is written.
"""
import os
import re
import subprocess

import pytest

from test_compiled_waits import OBJDUMP, code, pytestmark          # noqa: F401  (the fixture that reads the library)

WALK = re.compile(r"linear_walk_kernelI(DF16b|f)Li(\d+)ELi(\d+)ELi(\d+)ELi(\d+)ELb(\d)ELb(\d)E")
TWIN = re.compile(r"linear_twin_kernelI(DF16b|f)Li(\d+)ELi(\d+)ELi(\d+)ELb(\d)E")


class Shape:
    """What LinearShape says of a walk: stages of its ring, the copies a wavefront issues for a chunk at least, its
    stores for a chunk, and how many chunks ago the copies that a wait is for were issued."""

    def __init__(self, elem, KB, NW, JT, budget, out, dg):
        chunk_k, chunk_v = KB * 32 * elem // 16, NW * JT * 16 * elem // 16
        k, v = 32 * chunk_k * 16, 32 * chunk_v * 16
        has_x = out and dg and not (elem == 4 and KB == 8)
        stage = (2 if out else 1) * k + (2 if has_x else 1) * v
        scores = 3 * 64 * 4 * elem if out else 0
        self.stages = min(max((budget - 2 * scores) // stage, 2), 3)
        self.copies = (2 if out else 1) * (chunk_k // 2 // NW) + (2 if has_x else 1) * (chunk_v // 2 // NW)
        self.stores = 2 * JT if out else 0
        self.ago = self.stages - (2 if out and self.stages > 2 else 1)
        self.lets_pass = (self.ago - 1) * self.copies + self.ago * self.stores


def shapes(name):
    m = WALK.search(name)
    if m:
        KB, NW, JT, budget, out, dg = (int(x) for x in m.groups()[1:])
        return [Shape(2 if m[1] == "DF16b" else 4, KB, NW, JT, budget, out, dg)]
    m = TWIN.search(name)
    if not m:
        return []
    elem = 2 if m[1] == "DF16b" else 4
    KB, KB2, budget, out = (int(x) for x in m.groups()[1:])
    tiles = lambda other: 2 if elem == 2 and other > 2 else 1                       # noqa: E731
    return [Shape(elem, KB, 4, tiles(KB2), budget, out, 0), Shape(elem, KB2, 4, tiles(KB), budget, out, 0)]


def is_store(i):
    return i.op.startswith("buffer_store")


def reach(body, start, stop, back=None):
    """Instructions reached from `start` (successors, or predecessors by `back`), not going on from those where stop(i)."""
    seen, todo = set(), list(start)
    while todo:
        n = todo.pop()
        if n in seen:
            continue
        seen.add(n)
        if not stop(body[n]):
            todo += back.get(n, []) if back is not None else body[n].succ
    return seen


def counted_waits(body):
    """{wait: (what it lets pass, its barrier)} for the waits in a loop that a barrier follows with nothing but arithmetic
    between."""
    out = {}
    for n, i in enumerate(body):
        m = re.search(r"vmcnt\((\d+)\)", " ".join(i.args)) if i.op == "s_waitcnt" else None
        if not m or m[1] == "0":
            continue
        todo, seen, barriers, other = list(i.succ), set(), set(), False
        while todo:
            k = todo.pop()
            if k in seen:
                continue
            seen.add(k)
            if body[k].op == "s_barrier":
                barriers.add(k)
            elif body[k].op.startswith("ds_") or body[k].is_memory:
                other = True                              # (the compiler's own waits stand before an operand's use)
            else:
                todo += body[k].succ
        if barriers and not other and n in reach(body, i.succ, lambda j: False):
            assert len(barriers) == 1
            out[n] = (int(m[1]), barriers.pop())
    return out


def predecessors(body):
    before = {}
    for n, i in enumerate(body):
        for k in i.succ:
            before.setdefault(k, []).append(n)
    return before


def loop_of(body, wait, before):
    """What lies on a way from the wait back to it."""
    return reach(body, body[wait].succ, lambda i: False) & reach(body, [wait], lambda i: False, before)


def straight_stores(body, inside):
    """Sizes of the groups of output stores that no branch, label or copy divides."""
    targets = {k for i in body if i.target is not None for k in i.succ}
    sizes, run = [], 0
    for n, i in enumerate(body):
        if run and (n in targets or i.target is not None or i.is_copy or i.op == "s_barrier"):
            sizes.append(run)
            run = 0
        if n in inside and is_store(i):
            run += 1
    return sizes + ([run] if run else [])


def fewest_to_copies(body, wait, inside, before, chunks):
    """The fewest memory operations between a chunk's copies and the wait behind it, over the ways that meet a store."""
    # (the outputs are stored in one type or the other, by a flag that the graph does not know: a way without any is none)
    best, todo, ends = {(wait, False): 0}, [(wait, False)], []
    while todo:
        at = todo.pop()
        for p in before.get(at[0], []):
            if p not in inside or p in chunks:                      # (`chunks`: the barriers that chunks begin with)
                continue
            if body[p].is_copy:
                if at[1]:
                    ends.append(best[at])
                continue
            key, count = (p, at[1] or is_store(body[p])), best[at] + body[p].is_memory
            if count < best.get(key, 1 << 30):
                best[key] = count
                todo.append(key)
    return ends


def test_walks_wait_for_what_their_shape_says(code):                # noqa: F811
    walks = 0
    for name, body in code.items():
        kinds = shapes(name)
        if not kinds:
            continue
        walks += 1
        allowed = {s.lets_pass for s in kinds} | {(s.ago - 1) * s.copies for s in kinds}
        waits = counted_waits(body)
        assert waits and {n for n, _ in waits.values()} == allowed - {0}, (name, waits, allowed)
    assert walks >= 80


def test_outputs_are_stored_whole_and_behind_the_copies(code):      # noqa: F811
    walks = 0
    for name, body in code.items():
        kinds = shapes(name)
        if not kinds or not kinds[0].stores:
            continue
        walks += 1
        waits, before = counted_waits(body), predecessors(body)
        inside = reach(body, waits, lambda i: False)                # the loop: what a chunk's wait leads to
        sizes = straight_stores(body, inside)
        assert sizes and set(sizes) <= {s.stores for s in kinds}, (name, sizes)
        chunks = {barrier for _, barrier in waits.values()}
        for w, (passes, _) in waits.items():
            loop = loop_of(body, w, before)
            for n in loop:
                if is_store(body[n]):
                    behind = loop & reach(body, body[n].succ, lambda j: j.op == "s_barrier")
                    assert not any(body[k].is_copy for k in behind), (name, hex(body[n].at))
            ends = fewest_to_copies(body, w, loop, before, chunks)
            assert ends and min(ends) >= passes, (name, hex(body[w].at), passes, ends)
    assert walks >= 40


def test_states_only_walks_issue_the_copies_that_are_counted(code):  # noqa: F811
    walks = 0
    for name, body in code.items():
        kinds = shapes(name)
        if not kinds or kinds[0].stores:
            continue
        walks += 1
        waits, before = counted_waits(body), predecessors(body)
        for w, (passes, _) in waits.items():
            assert all(s.ago == 2 for s in kinds)
            # (a copy stands there twice: for whole chunks, and with its lanes masked for narrow rows and a row's last chunk)
            copies = sum(body[n].is_copy for n in loop_of(body, w, before))
            assert copies >= 2 * passes, (name, hex(body[w].at), passes, copies)
    assert walks >= 20


@pytest.fixture(scope="module")
def modifiers(code, tmp_path_factory):                              # noqa: F811
    """{kernel: {address: the instruction's text}} of the walks."""
    import shutil
    from mamba_ssd_sequence_chunked_amd import _build
    d = tmp_path_factory.mktemp("text")
    lib = shutil.copy(_build.LIB_PATH, d)
    subprocess.run([OBJDUMP, "--offloading", lib], cwd=d, capture_output=True, check=True)
    out, now = {}, None
    for f in sorted(os.listdir(d)):
        if f.endswith("gfx950"):
            text = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", os.path.join(d, f)], capture_output=True, text=True,
                                  check=True).stdout
            for line in text.splitlines():
                m = re.match(r"^[0-9a-f]+ <(.+)>:$", line)
                if m:
                    now = out.setdefault(m[1], {}) if shapes(m[1]) else None
                    continue
                m = re.match(r"^\t(.*?)\s*// ([0-9A-F]+):", line) if now is not None else None
                if m:
                    now[int(m[2], 16)] = m[1]
    return out


def test_states_have_arrived_before_they_are_announced(code, modifiers):         # noqa: F811
    kernels = 0
    for name, body in code.items():
        if not shapes(name) or not shapes(name)[0].stores:
            continue
        text, before = modifiers[name], predecessors(body)
        words = [n for n, i in enumerate(body) if i.op == "global_store_dword" and " sc1" in text[i.at]]
        parts = [n for n, i in enumerate(body) if i.op == "global_store_dwordx2" and " sc1" in text[i.at]]
        assert words and parts, name
        kernels += 1
        drained = lambda i: i.op == "s_waitcnt" and "vmcnt(0)" in i.args[0]          # noqa: E731
        for n in words:
            # back to the barrier, from there back to a wait for everything: no part of a state on either way
            near = reach(body, before[n], lambda i: i.op == "s_barrier", before)
            gates = [k for k in near if body[k].op == "s_barrier"]
            assert gates and not near & set(parts), (name, hex(body[n].at))
            for g in gates:
                assert not reach(body, before[g], drained, before) & set(parts), (name, hex(body[g].at))
    assert kernels >= 40
