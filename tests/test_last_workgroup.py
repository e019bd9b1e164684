"""A workgroup that counts itself as arrived has its results in memory (CPU only: the
compiled instructions are looked at, nothing runs).

A barrier on this GPU waits for no store, so each wave waits for its own stores before
the barrier that stands between them and the count."""
import os
import re
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


def test_every_wave_waits_for_its_stores_before_the_count(listing):
    counts = [i for i, line in enumerate(listing) if "global_atomic_add" in line]
    assert counts
    for at in counts:
        barrier = max(i for i in range(at) if re.match(r"\s*s_barrier", listing[i]))
        store = max(i for i in range(barrier) if "global_store" in listing[i])
        assert any(re.search(r"s_waitcnt .*vmcnt\(0\)", line) for line in listing[store:barrier]), at
