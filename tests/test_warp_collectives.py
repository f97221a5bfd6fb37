"""Instructions that need a whole warp together, checked in the sources (CPU): a kernel that
reaches one with lanes missing can wait for ever, so none is left to a GPU run to show."""
import glob
import os
import re

import pytest

from compressed_kv_cache_gva_b200 import _build

SOURCES = sorted(glob.glob(os.path.join(_build.CSRC, "*.cu*")))


def text(path):
    return re.sub(r"//[^\n]*", "", open(path).read())


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_cluster_barriers_bring_the_warp_together(path):
    """`barrier.cluster.*.aligned` stands in helpers only, each behind a __syncwarp."""
    src = text(path)
    bodies = re.findall(r"void \w+\(\) \{([^}]*barrier\.cluster\.\w+[^}]*)\}", src)
    assert sum(b.count("barrier.cluster") for b in bodies) == src.count("barrier.cluster")
    for b in bodies:
        assert b.index("__syncwarp()") < b.index("asm")


# plain waits per file: of one thread, or of a draining loop
SINGLE = {"paged_tc.cu": 6, "prefill_tc.cu": 6, "decode_tc.cu": 3, "decode_mma.cuh": 4, "paged_mma.cu": 1}


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_bounded_waits_of_warps_have_one_answer(path):
    """Waits of whole warps go through mbar_wait_warp.  The plain wait is left to single
    threads (producers, the MMA thread) and to draining loops that ignore its result; the
    number of those places is pinned, so that a new one is looked at."""
    name = os.path.basename(path)
    plain = len(re.findall(r"\bmbar_wait\(", text(path)))
    if name == "common.cuh":
        assert plain == 2          # its definition, and its use by the warp's
    else:
        assert plain == SINGLE.get(name, 0)
