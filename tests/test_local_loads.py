"""The library is one file that the ranks of a head-sharded run load as well, and its tensor maps are over whatever memory a
caller passes. A bulk copy that multicasts over a cluster is for one GPU and its own memory only, so no source has one."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "up_proj_gemm_gb300", "csrc")
SOURCES = sorted(f for e in ("cu", "cuh", "h", "cpp") for f in glob.glob(os.path.join(CSRC, "*." + e)))
MULTICAST_COPY = re.compile(r"cp\.async\.bulk[^;]*?\.multicast")


def test_the_pattern():
    assert MULTICAST_COPY.search('"cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.multicast::cluster"')
    assert MULTICAST_COPY.search('"cp.async.bulk.shared::cluster.global"\n  ".mbarrier::complete_tx::bytes.multicast::cluster [%0]"')
    assert not MULTICAST_COPY.search('"cp.async.bulk.tensor.2d [%0];" "tcgen05.commit.multicast::cluster.b64 [%0], %1;"')


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_no_multicast_copies(path):
    code = re.sub(r"//[^\n]*|/\*.*?\*/", "", open(path, encoding="utf-8").read(), flags=re.S)
    assert not MULTICAST_COPY.findall(code)
