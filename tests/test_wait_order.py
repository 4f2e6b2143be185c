"""One lane of a warp waits on an mbarrier and a shuffle gives the others its outcome.  A shuffle orders no memory, so a
barrier of the warp has to follow it before the others touch what was waited for; and what another block of the cluster
stored is waited for at the cluster's scope.  Both are properties of the source: a chip may well keep an order that it
does not promise."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "broadcast_implicit_gemm_gb300", "csrc")


def sources():
    return {os.path.basename(p): open(p).read() for ext in ("cu", "cuh") for p in glob.glob(os.path.join(CSRC, "*." + ext))}


def test_a_warp_barrier_follows_each_outcome_that_is_passed_on():
    found = 0
    for name, text in sources().items():
        for m in re.finditer(r"__shfl_sync\(0xffffffffu, ok\w*, 0\)([^;]*;)\s*(.*)", text):
            found += 1
            assert m.group(1) == ";" and m.group(2).startswith("__syncwarp();"), f"{name}: {m.group(0)}"
    assert found >= 3


def test_a_wait_for_a_peers_stores_is_at_the_clusters_scope():
    text = sources()
    assert "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64" in text["ptx.cuh"]
    waits = re.findall(r"(mbar_wait\w*(?:<\w+>)?)\(&sent", text["norm_back.cuh"])
    assert waits and set(waits) == {"mbar_wait_warp<true>"}
