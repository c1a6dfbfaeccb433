"""Rules of the linear kernels that no run can show to be kept: breaking them
is undefined behaviour that may work by chance. Read off the source (these run
without a GPU)."""
import os
import re

import pytest

from conftest import ROOT

CSRC = os.path.join(ROOT, "combine_top_group_b200", "csrc")


def code(name: str) -> str:
    from combine_top_group_b200 import metrics
    with open(os.path.join(CSRC, name), encoding="utf-8") as f:
        return metrics.code_of(f.read())


def kernels() -> dict:
    """Name and code of each kernel of linear_kernels.cuh."""
    parts = re.split(r"__global__ void ", code("linear_kernels.cuh"))[1:]
    return {re.search(r"(\w+)\s*\(\s*const __grid_constant__", p)[1]: p for p in parts}


def test_kernels_are_found():
    assert set(kernels()) == {"linear_kernel", "linear_pair_kernel"}


@pytest.mark.parametrize("name", ["linear_kernel", "linear_pair_kernel"])
def test_one_register_instruction_per_warpgroup(name):
    """All warps of a warpgroup have to execute the same setmaxnreg, so a
    kernel names it once for the epilogue's warpgroups and once for the other,
    before that one's warps part. (One in each warp's branch is undefined; the
    epilogue's request may then wait for registers that nobody gives back.)"""
    k = kernels()[name]
    assert len(re.findall(r"more_registers<", k)) == 1
    assert len(re.findall(r"fewer_registers<", k)) == 1
    assert re.search(r"if \(warp >= kEpiWarps\) \{ tc::fewer_registers<", k)
    roles = [m.start() for m in re.finditer(r"if \(warp == kEpiWarps( \+ \d)?\) \{", k)]
    assert roles and all(k.index("fewer_registers<") < at for at in roles)


def test_inboxes_are_handed_over_at_the_clusters_scope():
    """The CTAs of a cluster write each other's inboxes in shared memory. The
    order of those writes and of the reads before and after them rests on the
    inboxes' barriers, so each arrival and wait on these names the cluster's
    scope; the default is the CTA's."""
    k = kernels()["linear_kernel"]
    for bar in ("inbox_free", "inbox_full"):
        waits = re.findall(r"bar_wait(<[\w:]+>)?\(" + bar, k)
        assert waits and set(waits) == {"<tc::kCluster>"}, (bar, waits)
    arrivals = re.findall(r"bar_arrive\w*(<[\w:]+>)?\([^;]*inbox_free", k)
    assert arrivals == ["<tc::kCluster>"]
    ptx = code("tcgen05.cuh")
    assert "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64" in ptx
    assert "mbarrier.arrive.release.cluster.shared::cluster.b64" in ptx


@pytest.mark.parametrize("name", ["linear_kernel", "linear_pair_kernel"])
def test_a_stopped_cta_drains_whatever_stopped_it(name):
    """A wait that gives up may be any warp's. So what is in flight is drained
    after the barrier of the whole CTA, where the stop flag is final, and not
    by the one warp that saw its own wait fail."""
    k = kernels()[name]
    assert k.count("all_done();") == 2  # the epilogue's and the other warps' arrival at one barrier
    end = k.index("all_done();")
    assert "bar_drain" not in k[:end]
    after = k[end:]
    assert re.match(r"all_done\(\); if \(\*stop( && rank == 0)?\) \{", after)
    assert re.search(r"bar_drain\(full\(", after) and re.search(r"commit\(drained\); tc::bar_drain\(drained", after)
    assert after.rindex("bar_drain") < after.rindex("all_done();") < after.rindex("cluster_sync") < after.index("tmem_free")
    assert re.search(r'all_done\(\) \{ asm volatile\("bar.sync 6, %0;" ::"n"\(kThreads\)', code("linear.cuh"))


def test_an_unfilled_inbox_is_not_armed_again():
    """Arming an mbarrier whose phase is incomplete is undefined: the epilogue
    leaves its loop as soon as an inbox wait has given up."""
    k = kernels()["linear_kernel"]
    wait = k.index("bar_wait<tc::kCluster>(inbox_full")
    assert re.match(r"[^;]*; ok = epi_sync_and\(ok\); if \(!ok\) break;", k[wait:])
    assert k.count("bar_expect(inbox_full") == 1
