"""CPU checks of the hand-counted memory-counter waits of the int8 tile kernel against the compiled gfx950
code.

A tile's K steps are brought by DMA into two LDS stages, 8 instructions of a wave a step.  The next tile's
first two steps are issued between the stores of the last tile's results, and two waits count what is behind
them: the one at the tile's end leaves in flight what was issued after the first step's last DMA, the one in
the next tile's first step what was issued after the second step's.  Both are right if at least that many
operations really follow in the compiled code on every path; operations that the compiler adds (reloads of
spilled registers, waits of its own) make them wait for more, never for less.  The K loop's own wait is for
everything.

The compiled kernel's branches are followed from each barrier on (memory operations retire in issue order)."""
import os
import re

import pytest

from test_waits_isa_cpu import CSRC, HIPCC, _asm, _functions

STEP = 8  # DMAs of a wave for a K step


@pytest.fixture(scope="module")
def asm():
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not available")
    return _asm(os.path.join(CSRC, "gemm_i8.hip"))


def flow(body):
    """[(event or None, next instructions)] of a kernel: 'D' a DMA, 'S' a store of results, 'B' a barrier, a
    number a wait that leaves so many operations in flight."""
    code, labels = [], {}
    for l in body:
        t = l.strip()
        m = re.match(r"(\.LBB\d+_\d+):", t)
        if m:
            labels[m.group(1)] = len(code)
        elif re.match(r"[a-z]", t):
            code.append(t)
    out = []
    for i, t in enumerate(code):
        ev = None
        if t.startswith("buffer_load_dwordx4") and " lds" in t:
            ev = "D"
        elif t.startswith("buffer_store"):
            ev = "S"
        elif t.startswith("s_barrier"):
            ev = "B"
        elif t.startswith("s_waitcnt") and "vmcnt(" in t:
            ev = int(re.search(r"vmcnt\((\d+)\)", t).group(1))
        if t.startswith("s_branch"):
            nxt = [labels[t.split()[1]]]
        elif t.startswith("s_cbranch"):
            nxt = [i + 1, labels[t.split()[1]]]
        else:
            nxt = [] if t.startswith("s_endpgm") else [i + 1]
        out.append((ev, nxt))
    return out


def paths(code, start):
    """What the paths from instruction `start` on do up to the next barrier or to a wait that leaves a step's
    DMAs or more in flight, as a set of (events, end): 'B', the wait's number, or 'end'.  A path that comes back
    to where it was without either is not followed again."""
    memo, on = {}, set()

    def walk(i):
        if i in memo:
            return memo[i]
        if i in on:
            return set()
        ev, nxt = code[i]
        if ev == "B" or isinstance(ev, int) and ev >= STEP:
            got = {("", ev)}
        elif not nxt:
            got = {("", "end")}
        else:
            on.add(i)
            own = "" if ev is None else "0" if ev == 0 else "w" if isinstance(ev, int) else ev
            got = {(own + s, e) for n in nxt for s, e in walk(n)}
            on.discard(i)
        memo[i] = got
        return got

    import sys
    old = sys.getrecursionlimit()
    sys.setrecursionlimit(100000)
    try:
        return set().union(*(walk(n) for n in code[start][1]))
    finally:
        sys.setrecursionlimit(old)


def tile_kernel(asm, gate_up):
    f = _functions(asm, r"tile_i8_kernelILb%dE" % gate_up)
    assert len(f) == 1
    return flow(next(iter(f.values())))


# (operations behind the first step's last DMA, behind the second's) of the prologue and of a tile's end with
# no, two and four blocks of rows: two stores leave for a block of gate and up, four for two of the down
# product's blocks of columns.
ENDS = {True: {(8, 0), (12, 2), (14, 2)}, False: {(8, 0), (16, 4), (24, 12)}}


@pytest.mark.parametrize("gate_up", [True, False])
def test_waits_at_a_tiles_end_leave_what_follows_the_steps(asm, gate_up):
    code = tile_kernel(asm, gate_up)
    ends = set()
    for i, (ev, _) in enumerate(code):
        if ev != "B":
            continue
        for s, end in paths(code, i):
            if end == "B" or "D" not in s:  # not the way through a tile's end
                continue
            assert s.count("D") == 2 * STEP, (s, end)
            ops = s.replace("0", "").replace("w", "")
            at = [j for j, c in enumerate(ops) if c == "D"]
            behind = len(ops) - 1 - at[STEP - 1], len(ops) - 1 - at[2 * STEP - 1]
            assert end == behind[0], (ops, end)  # the first step has landed, and nothing more is waited for
            ends.add(behind)
    assert ends == ENDS[gate_up]


@pytest.mark.parametrize("gate_up", [True, False])
def test_waits_of_the_steps_cover_them(asm, gate_up):
    """Between two barriers of the K loop, and from its last one to the barrier before the results, every DMA
    is followed by a wait for everything."""
    code = tile_kernel(asm, gate_up)
    steps = set()
    for i, (ev, _) in enumerate(code):
        if ev != "B":
            continue
        for s, end in paths(code, i):
            if end == "B" and "D" in s and "S" not in s:
                assert "0" in s[s.rindex("D"):], s
                steps.add(s.count("D"))
    assert STEP in steps and steps <= {3, STEP}  # a whole step, or the three (dropped) ones of the last


@pytest.mark.parametrize("gate_up", [True, False])
def test_the_second_steps_wait_has_the_counts_of_the_tiles_ends(asm, gate_up):
    """The waits of a tile's first step: for everything, or for all but the operations behind the second step
    in one of the forms of a tile's end."""
    code = tile_kernel(asm, gate_up)
    counts = {ev for ev, _ in code if isinstance(ev, int)}
    first = {a for a, _ in ENDS[gate_up]}
    second = {b for _, b in ENDS[gate_up]}
    # 3, 2 and 1: the offsets' loads, one after another, when the tiles are counted; the down
    # product's code keeps the pair's count (2), which it never reaches
    assert counts <= first | second | {0, 1, 2, 3}, counts
    assert first <= counts and second <= counts
