"""Every wait between the warps of the ragged-attention kernels is bounded: shown by
reading their sources, since a wait that is not would hang the GPU."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_decode_15_gb300", "csrc")


def source(name):
    """A source file without its comments."""
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def roles():
    """The prompt kernel between the barrier that ends its set-up and the one of its
    tear-down, which every warp reaches: there warps give up one by one."""
    kernel = source("attend_prompt.cuh").split("attend_prompt_kernel(", 1)[1]
    return kernel.split("const uint32_t tmem = *tslot;", 1)[1].rsplit("__syncthreads();", 1)[0]


def test_no_barrier_of_several_warps_among_the_roles():
    """A warp may give up (pt_wait) while its siblings go on: a hardware barrier of
    several warps would then wait for it for ever."""
    body = roles()
    for barrier in ("bar.sync", "bar.red", "barrier.", "__syncthreads", "bar.arrive"):
        assert barrier not in body, barrier


def test_waits_on_memory_barriers_are_bounded():
    body = roles()
    assert "pt_wait(" in body and "mbar_try_wait(" not in body and "mbar_test_wait(" not in body
    wait = source("attend_prompt.cuh").split("bool pt_wait(", 1)[1].split("\n}", 1)[0]
    assert "kErrTimeout" in wait and "__all_sync" in wait and "break" in wait


def test_lanes_of_a_step_warp_give_up_together():
    """mbar_wait answers per lane: a warp whose lanes part there would meet the shuffles
    and products of the whole warp with some of them gone."""
    loop = source("attend_step.cuh").split("for (int k = 0; k < my_n; ++k) {", 1)[1]
    waits = re.findall(r"if \(([^{]*mbar_wait\([^{]*)\{", loop.split("if (timed_out)", 1)[0])
    assert len(waits) == 1 and waits[0].startswith("!__all_sync(kFull, mbar_wait(")


def test_the_loading_warp_always_waits_for_its_copies():
    """The last copies are waited for by the warp that issued them on every way out of its
    role, not only where it gave up itself: the warps that read them may have."""
    role = roles().split("if (warp == 8) {", 1)[1].split("} else if (warp == 9) {", 1)[0]
    depth, found = 0, 0
    for line in role.splitlines():
        if "mbar_wait(bar(S::B_UF" in line or "mbar_wait(bar(S::B_QF" in line:
            assert depth == 0, f"under a condition: {line.strip()}"
            found += 1
        depth += line.count("{") - line.count("}")
    assert found == 2 and "return" not in role.rsplit("mbar_wait(bar(S::B_UF", 1)[0].rsplit("for (int r = 0; ok; ++r)", 1)[1]
