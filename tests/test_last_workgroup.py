"""No workgroup of the few-token path waits for or counts another one of its launch (CPU
only: the compiled instructions are looked at, nothing runs).

A workgroup that counts itself as arrived would need its results in memory first, and a
barrier on this GPU waits for no store, so a fence behind the barrier in one thread leaves
the other waves' stores on their way.  The path has no such count: results of a launch
are read by the next one."""
import os
import subprocess

import pytest

from mixture_experts_layer_sort_amd import build as B


@pytest.fixture(scope="module")
def listing(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("asm") / "decode.s")
    subprocess.run([B.hipcc(), f"--offload-arch={B.ARCH}", "-O3", "-std=c++17", "-Xclang", "-target-feature", "-Xclang",
                    "-packed-fp32-ops", f"-I{B.INCLUDE}", f"-I{B.CSRC}", "-x", "hip", "-S", "--cuda-device-only", "-o",
                    out, os.path.join(B.CSRC, "decode.hip")], check=True, stdout=subprocess.PIPE,
                   stderr=subprocess.STDOUT)
    with open(out) as f:
        return f.read().splitlines()


def test_no_workgroup_counts_others(listing):
    assert any("v_mfma" in line for line in listing)
    assert not [line for line in listing if "global_atomic" in line or "flat_atomic" in line]
