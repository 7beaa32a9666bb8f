"""The scopes of what CTAs of a pair tell one another, from the sources (no GPU needed): an arrival on another CTA's
barrier and the waits for it name the cluster's scope. A narrower one works on today's hardware and is not promised by the
memory model, so no run shows the difference."""
import glob
import os
import re

import pytest

from newton_schulz_quintic_gb300 import build

FILES = sorted(glob.glob(os.path.join(build.CSRC, "*.cu")) + glob.glob(os.path.join(build.CSRC, "*.cuh")))


def code(path):
    with open(path) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_arrivals_on_other_ctas_barriers_have_cluster_scope():
    found = 0
    for path in FILES:
        for op in re.findall(r"mbarrier\.arrive[\w.:]*", code(path)):
            if "shared::cluster" in op:
                found += 1
                assert ".cluster.shared::cluster" in op, (os.path.basename(path), op)
    assert found >= 2


@pytest.mark.parametrize("name", ["ns_tc.cu", "ns_wgrad.cu", "ns_blocks_mm.cu"])
def test_waits_for_other_ctas_acquire_at_cluster_scope(name):
    text = code(os.path.join(build.CSRC, name))
    # barriers of the pair: those arrived on by address in the cluster, and those that a commit signals in both CTAs
    shared = set(re.findall(r"mapa_shared\(smem_u32\(&bar->(\w+)\[", text))
    shared |= set(re.findall(r"umma_commit_pair_multicast\(&bar->(\w+)\[", text))
    shared |= set(re.findall(r"uint64_t \*const (\w+) = &bar->\w+\[stage\]", text))
    assert {"empty", "tfull", "tempty"} <= shared
    waits = re.findall(r"(mbar_wait|mbar_try_wait|mbar_try_wait_cluster)(<\w+>)?\(&bar->(\w+)\[", text)
    assert waits
    for how, scope, bar in waits:
        if bar in shared:
            assert scope == "<true>" or how == "mbar_try_wait_cluster", (bar, how, scope)
