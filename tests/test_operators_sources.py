"""What the library must not contain, checked on its sources and symbols without a GPU."""
import glob
import os
import shutil
import subprocess

import pytest

import dtensor_reshard_gb300 as rs

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _sources():
    names = glob.glob(os.path.join(ROOT, "dtensor_reshard_gb300", "csrc", "*"))
    names += glob.glob(os.path.join(ROOT, "include", "*"))
    assert len(names) > 15
    return {n: open(n, encoding="utf-8").read() for n in names}


def test_no_multicast_over_a_cluster():
    """The library is loaded by every rank of a run on several GPUs, and an operand may be
    memory of another GPU: every CTA loads its own tiles."""
    for name, text in _sources().items():
        assert ".multicast" not in text, name


@pytest.mark.skipif(shutil.which("nm") is None, reason="nm lists the library's symbols")
def test_resident_clusters_are_on_record_for_each_kernel():
    """The product's choice of kernel asks how many clusters fit on the GPU; an answer kept for
    one kernel must not serve another (all have the same C++ type)."""
    names = subprocess.run(["nm", "-C", rs.LIB_PATH], capture_output=True, text=True, check=True).stdout
    records = {line.split(" ", 2)[2] for line in names.splitlines()
               if "resident_clusters" in line and line.endswith("::known") and "guard" not in line}
    kernels = {(k, y) for k in ("narrow_kernel<16", "narrow_kernel<32", "narrow_kernel<64", "wide_kernel<")
               for y in ("float", "__half", "__nv_bfloat16")}
    assert len(records) == len(kernels), records
