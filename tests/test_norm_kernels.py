"""The norm's kernels are built for the rows that its entry points take, and no others (CPU
only: the names in the library built here are looked at)."""
import os
import re

import pytest

from mixture_experts_layer_sort_amd import _lib as L
from mixture_experts_layer_sort_amd import build as B


@pytest.fixture(scope="module")
def built():
    if not os.path.exists(L.LIB_PATH):
        B.build()
    # the device code is a part of the library, its kernels named in a string table
    with open(L.LIB_PATH, "rb") as f:
        return f.read()


@pytest.mark.parametrize("kernel", ["k_norm", "k_norm_bwd"])
def test_every_norm_kernel_has_rows(built, kernel):
    names = set(re.findall(rb"_ZN12_GLOBAL__N_1%d%sI([tf])Li(\d+)ELi(\d+)ELb[01]E" % (len(kernel), kernel.encode()), built))
    assert names
    for t, threads, per in names:
        vec = 8 if t == b"t" else 4
        assert int(threads) * int(per) * vec <= L.MOE_NORM_MAX_H, (t, threads, per)
    # the longest rows of both types have one
    assert {(t, int(n) * int(v)) for t, n, v in names} >= {(b"t", L.MOE_NORM_MAX_H // 8), (b"f", L.MOE_NORM_MAX_H // 4)}
