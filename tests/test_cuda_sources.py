"""Rules of the CUDA sources that no run shows (CPU only)."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "fp8_quantization_moe_gb300", "csrc")


def statements(path):
    """The file's statements without comments, each on a line."""
    with open(path) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    return [re.sub(r"\s+", " ", s).strip() for s in re.split(r"[;{}]", text) if s.strip()]


def test_cluster_barriers_are_reached_by_whole_warps():
    """barrier.cluster.*.aligned is executed by all lanes of a warp together;
    only __syncwarp() right before it makes sure of that behind divergent code."""
    found = 0
    for path in glob.glob(os.path.join(CSRC, "*.cu*")):
        lines = statements(path)
        for i, line in enumerate(lines):
            if "barrier.cluster." in line:
                found += 1
                assert ".aligned" in line and lines[i - 1] == "__syncwarp()", (os.path.basename(path), line)
    assert found == 2  # one place each for the arrival and the wait
