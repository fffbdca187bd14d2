"""A cluster's barrier wants whole warps at one instruction: each use of it is behind a __syncwarp, so
that lanes which come from loops of their own meet first.  (A source check: a barrier that part of a
warp passes is not provoked.)"""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "grouped_expert_gemm_gb300", "csrc")


def bare(text):
    """Cluster barriers whose statement does not follow a __syncwarp."""
    text = re.sub(r"//[^\n]*", "", text)
    return [m.group(0) for m in re.finditer(r"([^;{}]*;)?\s*asm volatile\(\s*\"barrier\.cluster\.arrive", text)
            if not re.match(r"\s*__syncwarp\(\);", m.group(1) or "")]


def test_whole_warps_come_to_a_clusters_barrier():
    assert bare('f() { asm volatile("barrier.cluster.arrive.release.aligned;"); }')
    assert bare('f() { __syncwarp(); g(); asm volatile("barrier.cluster.arrive;"); }')
    assert not bare('f() {\n  __syncwarp();  // meet\n  asm volatile("barrier.cluster.arrive;"); }')
    files = glob.glob(os.path.join(CSRC, "*.cu*"))
    seen = 0
    for name in files:
        with open(name) as f:
            text = f.read()
        seen += text.count('"barrier.cluster.arrive')
        assert bare(text) == [], os.path.basename(name)
    assert seen > 0
