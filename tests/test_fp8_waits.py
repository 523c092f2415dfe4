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


@pytest.mark.parametrize("name", KERNELS + ["gemm.cu"])
def test_tensor_memory_loads_follow_a_whole_warps_wait(name):
    # every lane polls for itself: only the vote in warp_wait brings the warp together before tcgen05.ld.sync.aligned
    calls = re.findall(r"\b(mbar_wait|lane_wait|warp_wait|tmem_ld\d+)\(", source(name))
    loads = [i for i, c in enumerate(calls) if c.startswith("tmem_ld")]
    assert loads
    for i in loads:
        waits = [c for c in calls[:i] if not c.startswith("tmem_ld")]
        assert waits[-1] == "warp_wait"
    assert name == "gemm.cu" or "!mbar_wait" not in source(name), "one lane's answer would be its own"


def test_the_vote_is_the_whole_warps():
    body = re.search(r"void warp_wait\([^)]*\)\s*\{(.*?)\n\}", source("tcgen05.cuh"), re.S).group(1)
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


def issued_too_early(stages: int, order, steps: int = 13) -> bool:
    """Every order of events in the pair kernel's ring of `stages` tiles and two accumulator buffers, with two
    issuers that take the steps in turn: can an MMA be issued before its tiles have landed?  Barriers are what the
    hardware has, a count of phases of which a wait sees the parity."""
    # state: steps sent, landed steps (bits), per issuer (its step, waits done), MMAs done (bits), steps added up
    start = (0, 0, (0, 0), (1, 0), 0, 0)
    seen, todo = {start}, [start]
    while todo:
        sent, landed, a, b, done, added = todo.pop()
        new = []
        if sent < steps and (sent < stages or done >> (sent - stages) & 1):
            new.append((sent + 1, landed, a, b, done, added))
        for p in range(max(0, sent - stages), sent):
            if not landed >> p & 1:
                new.append((sent, landed | 1 << p, a, b, done, added))
        for i, (n, waits) in enumerate((a, b)):
            if n >= steps:
                continue
            if waits < 2:
                if order[waits] == "full":
                    phases = sum(landed >> p & 1 for p in range(n % stages, steps, stages))
                    ok = phases % 2 != n // stages % 2
                else:
                    phases = sum(1 for p in range(n % 2, added, 2))
                    ok = phases % 2 != (n // 2 % 2) ^ 1
                to = (n, waits + 1) if ok else None
            elif not landed >> n & 1:
                return True
            else:      # issued; it ends at some later time
                to = (n + 2, 0)
            if to:
                new.append((sent, landed) + ((to, b) if i == 0 else (a, to)) + (done, added))
        for n in range(steps):
            if not done >> n & 1 and n < (a, b)[n % 2][0] and (n < 2 or done >> (n - 2) & 1):
                new.append((sent, landed, a, b, done | 1 << n, added))
        if added < steps and done >> added & 1:
            new.append((sent, landed, a, b, done, added + 1))
        for s in new:
            if s not in seen:
                seen.add(s)
                todo.append(s)
    assert any(s[5] == steps for s in seen)
    return False


def test_the_pairs_mmas_wait_for_their_tiles():
    s = source("fp8_pair.cu")
    order = re.findall(r"lane_wait\(dead, &sm\.(full|acc_empty)\[", s)
    stages = [int(v) for v in re.search(r"kStages = MODE == FP8_GATE_UP \? (\d+) : (\d+);", s).groups()]
    assert len(order) == 2 and re.search(r"kBufs = 2;", s)
    for n in stages:
        assert not issued_too_early(n, order), (n, order)
    assert issued_too_early(3, ["full", "acc_empty"]), "the model knows the other order's fault"


@pytest.mark.parametrize("name", KERNELS + ["fp8_product.cu"])
def test_only_weights_go_through_the_read_only_path(name):
    # the kernel before may still write everything else when these begin
    for arg in re.findall(r"__ldg\(((?:[^()]|\([^()]*\))*)\)", source(name)):
        assert re.match(r"(reinterpret_cast<const float4\*>\()?w[sab01] \+ k", arg), arg


@pytest.mark.parametrize("name", KERNELS + ["gemm.cu"])
def test_waits_for_tensor_memory_name_what_was_loaded(name):
    # the registers of a load are valid after the wait only, which the compiler learns from the operands alone
    waits = re.findall(r"tmem_wait_ld\(([^)]*)\)", source(name))
    assert waits and all(waits)
