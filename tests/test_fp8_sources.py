"""What the 8-bit float kernels' sources may not hold.  CPU only."""
import glob
import os
import re

import pytest

import gemm_collective_tiles_gb300 as gct

SOURCES = sorted(glob.glob(os.path.join(os.path.dirname(gct.__file__), "csrc_fp8", "*.cu*")))


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_no_read_only_path(path):
    """These kernels start while the one before them still writes what they
    will read.  Loads by the read-only path are for data that nobody writes
    during the kernel, and a compiler may move them over the wait."""
    with open(path) as f:
        code = re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)
    assert not re.search(r"__ldg\b|\b__restrict(__)?\b|\bld\.global\S*\.nc\b", code)


def test_there_are_sources():
    assert len(SOURCES) >= 5
