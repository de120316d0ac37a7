"""CTA barriers (bar.sync) have no timeout, so no warp of a group may meet one that another warp of
the group can fail to reach. A bounded wait on an mbarrier can run out for one warp and be met for
another (a phase that completes after the abort flag is raised, between their looks at it). The
kernels therefore leave a group of warps only through named_barrier_all, to which each member brings
its answer. Read from the source, since a GPU must not be hung to see it: between a bounded wait and
the next plain group barrier there is a named_barrier_all, and its answer is acted upon."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "causal_flash_attention_attn_b200", "csrc")
EVENT = re.compile(r"\b(mbar_wait|mbar_wait_warp|item_of|item_of_warp|named_barrier_all|named_barrier_sync)\(")
FILES = [f for f in sorted(glob.glob(os.path.join(CSRC, "*.cuh"))) if "named_barrier" in open(f).read() and
         not f.endswith("sm100.cuh")]


def code(path):
    return re.sub(r"//.*|/\*.*?\*/", "", open(path).read())


def test_the_files_with_group_barriers_are_found():
    assert {os.path.basename(f) for f in FILES} >= {"bwd_tc.cuh", "fwd2_tc.cuh", "fwd_tc.cuh", "varlen_fwd.cuh"}


@pytest.mark.parametrize("path", FILES, ids=os.path.basename)
def test_a_group_agrees_between_a_bounded_wait_and_its_next_barrier(path):
    text, last = code(path), None
    for m in EVENT.finditer(text):
        if m[1] == "named_barrier_sync":
            line = text[:m.start()].count("\n") + 1
            assert last == "named_barrier_all", f"{os.path.basename(path)}:{line}: a plain group barrier behind {last}"
        else:
            last = m[1]


@pytest.mark.parametrize("path", FILES, ids=os.path.basename)
def test_the_groups_answer_is_acted_upon(path):
    text = code(path)
    calls = len(re.findall(r"\bnamed_barrier_all\(", text))
    used = (len(re.findall(r"if \(!(?:\(ok = )?named_barrier_all\([^;]*?\)\)?\) break;", text)) +
            len(re.findall(r"\bok = named_barrier_all\([^;]*\);\s*(?:l \+=[^;]*;\s*)?if \(ok\)", text)) +
            # (a warp whose own wait ran out)
            len(re.findall(r"\bok = (?:u \+ 1 < n && |j < hix && )?named_barrier_all\([^;]*, false\);\s*break;", text)) +
            # (the pair's answer, carried to the tile's barrier)
            len(re.findall(r"ok = named_barrier_all\(pair_bar, 64, ok\);(?:(?!named_barrier|mbar_wait).)*"
                           r"if \(!named_barrier_all\(tile_bar, 256, ok\)\) break;", text, flags=re.S)))
    assert calls > 0 and used == calls, (calls, used)
