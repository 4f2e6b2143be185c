"""What a launch remembers between calls is shared by threads: the layer calls let go of Python's lock."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "broadcast_implicit_gemm_gb300", "csrc")


def test_what_is_kept_between_calls_is_atomic():
    kept = []
    for path in glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh")):
        text = open(path).read()
        kept += re.findall(r"static ([\w:<> ]+?) attr_set", text)
    assert len(kept) >= 8 and set(kept) == {"std::atomic<unsigned long long>"}
