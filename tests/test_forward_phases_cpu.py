"""The two-tile forwards wait on mbarriers by the parity of a phase, so a warp may be at most one
phase behind the barrier it waits on: two behind, the phase looks as if it were still to come. A model
of the roles over items without a tile B (runs of sequences of at most 128 rows), explored over every
order of their steps, shows that O_FINAL of tile B needs a wait for that tile's warps (O_EMPTY) in
items where no product waits for them, with two Q buffers as with one; and the kernels have it."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "causal_flash_attention_attn_b200", "csrc")


def roles(passes, buffers, empty_wait):
    """Each role's steps: ("wait", barrier, phase), ("arrive", barrier) or ("meet",), tile B's group barrier."""
    load, mma, tile_a, first, other = [], [], [], [], []
    for p in range(passes):
        if p >= buffers:
            load.append(("wait", f"q_empty{p % buffers}", p // buffers - 1))
        load += [("arrive", f"q_full{p % buffers}"), ("arrive", f"item{p + 1}")]
        if p:
            mma.append(("wait", f"item{p}", 0))
        mma.append(("wait", f"q_full{p % buffers}", p // buffers))
        if p:
            mma.append(("wait", "o_empty_a", p - 1))  # the first PV of tile A
            if empty_wait:
                mma.append(("wait", "o_empty_b", p - 1))
        mma += [("arrive", "o_final_a"), ("arrive", "o_final_b")]
        tile_a += [("wait", f"item{p + 1}", 0), ("wait", "o_final_a", p), ("arrive", "o_empty_a"),
                   ("arrive", f"q_empty{p % buffers}")]
        for warp in (first, other):
            warp += [("wait", f"item{p + 1}", 0), ("wait", "o_final_b", p), ("arrive", "o_empty_b"), ("meet",)]
        first.append(("arrive", f"q_empty{p % buffers}"))
    return load, mma, tile_a, first, other


def lost_phase(passes, buffers, empty_wait):
    """A wait that some order of the steps leaves two phases behind its barrier, or None."""
    steps = roles(passes, buffers, empty_wait)
    needs = {"o_empty_b": 2, "q_empty0": 2, "q_empty1": 2}  # arrivals of a phase, 1 elsewhere
    seen, todo = {(0,) * 5}, [(0,) * 5]
    while todo:
        at = todo.pop()
        arrived = {}
        for role, n in zip(steps, at):
            for s in role[:n]:
                if s[0] == "arrive":
                    arrived[s[1]] = arrived.get(s[1], 0) + 1
        now = [role[n] if n < len(role) else None for role, n in zip(steps, at)]
        moves = []
        for i, s in enumerate(now):
            if s is None or s[0] == "meet":
                continue
            if s[0] == "wait":
                done = arrived.get(s[1], 0) // needs.get(s[1], 1)
                if not s[2] <= done <= s[2] + 1:
                    return s, done
                if done == s[2]:
                    continue
            moves.append(tuple(n + (j == i) for j, n in enumerate(at)))
        if now[3] == now[4] == ("meet",):
            moves.append(at[:3] + (at[3] + 1, at[4] + 1))
        if not moves:
            assert all(s is None for s in now), ("stuck", now)
        for m in moves:
            if m not in seen:
                seen.add(m)
                todo.append(m)
    return None


@pytest.mark.parametrize("buffers", [1, 2])
def test_no_warp_falls_two_phases_behind(buffers):
    assert lost_phase(5, buffers, True) is None


def test_the_model_finds_the_lost_phase_without_the_wait():
    s, done = lost_phase(5, 2, False)
    assert s[1] == "o_final_b" and done == s[2] + 2


@pytest.mark.parametrize("name", ["varlen_fwd.cuh", "fwd2_tc.cuh"])
def test_the_kernels_wait_before_the_last_commit(name):
    text = re.sub(r"//.*", "", open(os.path.join(CSRC, name)).read())
    assert "hi1 = I.hasB ? I.tB : -1;" in text
    issuer = text[text.index("warp == C::W_MMA) {\n" if name == "varlen_fwd.cuh" else "issue_pv"):]
    assert re.search(r"if \((?:!I\.hasB|hi1 < 0) && pass > 0 &&\s*!\(ok = mbar_wait(_warp)?\(bar\(C::B_O_EMPTY \+ 1\), "
                     r"\(uint32_t\)\(\(pass - 1\) & 1\), abort_flag\)\)\)\s*break;\s*"
                     r"(if \(lead\) \{\s*)?tc_commit\(bar\(C::B_O_FINAL \+ 0\)\);", issuer)
