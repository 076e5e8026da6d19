"""The HIP sources through the compiler's front end (no code is generated):
what it warns of and the build does not show."""

import glob
import os
import subprocess

import pytest

from mxfp4_moe_expert_route_amd import build

SOURCES = sorted(glob.glob(os.path.join(build.CSRC, "*.hip")))


@pytest.mark.parametrize("path", SOURCES, ids=[os.path.basename(p) for p in SOURCES])
def test_packed_fields_are_packed(path):
    """A field that `packed` leaves aligned makes a load or store claim an
    alignment that its address does not have."""
    cmd = [build.HIPCC] + build.FLAGS + ["-Werror=packed-non-pod", "--cuda-device-only", "-emit-llvm",
                                         "-Xclang", "-disable-llvm-passes", "-S", "-o", os.devnull, path]
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    assert r.returncode == 0, r.stdout
