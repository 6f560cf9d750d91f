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


def test_kernels_that_must_not_spill_are_watched():
    fine = {"VGPRs": 75, "ScratchSize [bytes/lane]": 0, "VGPRs Spill": 0}
    for kernel in ("quick", "exact", "back", "adjust", "slice", "whole", "join"):
        name = "_ZN4gnms12_GLOBAL__N_1%d%s_kernelEv" % (len(kernel) + 7, kernel)
        assert build.check_resources({name: fine}) == []
        for field, value in (("VGPRs", 256), ("ScratchSize [bytes/lane]", 16), ("VGPRs Spill", 1)):
            assert len(build.check_resources({name: {**fine, field: value}})) == 1
