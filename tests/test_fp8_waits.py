"""How the fp8 kernels wait, read from their sources: a wait that gives up, or lanes that leave a wait at
different times, cannot be provoked on a GPU in a test."""
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
KERNELS = ["fp8_decode.cu", "fp8_mid.cu", "fp8_pair.cu"]


def source(name: str) -> str:
    with open(os.path.join(ROOT, "int4_routed_expert_gemv_b200", "csrc", name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


@pytest.mark.parametrize("name", KERNELS)
def test_tensor_memory_loads_follow_a_whole_warps_wait(name):
    # every lane polls for itself: only the vote in warp_wait brings the warp together before tcgen05.ld.sync.aligned
    calls = re.findall(r"\b(mbar_wait|lane_wait|warp_wait|tmem_ld\d+)\(", source(name))
    loads = [i for i, c in enumerate(calls) if c.startswith("tmem_ld")]
    assert loads
    for i in loads:
        waits = [c for c in calls[:i] if not c.startswith("tmem_ld")]
        assert waits[-1] == "warp_wait"
    assert "!mbar_wait" not in source(name), "one lane's answer would be its own"


def test_the_vote_is_the_whole_warps():
    body = re.search(r"void warp_wait\([^)]*\)\s*\{(.*?)\n\}", source("fp8_tiles.cuh"), re.S).group(1)
    assert re.search(r"dead = !__all_sync\(0xffffffffu, ok\);\s*$", body)


def test_a_warp_that_gave_up_goes_through_every_item():
    # the other warps wait for it at named barriers, which have no limit: no loop over items may end on `dead`
    for name in KERNELS:
        assert not re.search(r"dead \|\||\|\| dead|!dead &&[^;]*(next|more)|if \(dead\) (break|return)", source(name)), name
    look_up = re.search(r"auto look_up = .*?return true;\s*\};", source("fp8_pair.cu"), re.S).group(0)
    assert re.search(r"if \(dead\) \{[^}]*again\.init\([^}]*return again\.at\(\(int\)briefs - 1, w\.it\);\s*\}", look_up)
    # and briefs are not overwritten under a warp that still reads them
    assert "if (lane == 0 && !dead)" in source("fp8_pair.cu")


@pytest.mark.parametrize("name", KERNELS)
def test_copies_asked_for_are_waited_for(name):
    # by their own count: after a wait that gave up the step counter runs on
    s = source(name)
    assert re.search(r"if \(dead\) continue;\s*sent = n \+ 1;", s)
    assert re.search(r"drain\(sm\.full, kStages, sent, p\.status", s)


def test_no_wait_of_the_pairs_lasts_a_whole_launch():
    # rank 1 issues no MMAs: it may wait for the last commits only when its own sums are formed
    s = source("fp8_pair.cu")
    at = s.index("if (rank == 1 && tid < 2) mbar_wait(&sm.mma_done[tid]")
    assert s.index("warp_wait(dead, &sm.acc_full") < s.rindex("__syncthreads();") < at < s.rindex("cluster_sync();")
    assert len(re.findall(r"wait\([^;]*mma_done", s)) == 2
