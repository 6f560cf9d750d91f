"""What the compiler finds in the sources by itself, without building them."""
import os
import subprocess

import pytest

from greedy_iou_nms_amd import build

pytestmark = pytest.mark.skipif(not os.path.exists(build.HIPCC), reason="no hipcc")


@pytest.mark.parametrize("source", build.SOURCES)
def test_no_constant_index_past_an_array(source):
    """Of the last array of a struct too, which is no flexible one here."""
    flags = [f for f in build.FLAGS if f not in ("-O3", "-Wall")]
    r = subprocess.run([build.HIPCC, *flags, "-O0", "-fsyntax-only", "--offload-device-only",
                        "-fstrict-flex-arrays=3", "-Werror=array-bounds",
                        os.path.join(build.CSRC, source)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
