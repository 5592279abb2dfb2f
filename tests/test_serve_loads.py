"""The serving kernels' blocks may be resident while the kernel before them writes what they read: their sources use no
load that is defined only for data nothing writes meanwhile, and no pointer qualified so that the compiler would choose one."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sparse_selected_cell_gb300", "csrc")
OVERLAPPED = sorted(f for f in os.listdir(CSRC) if f.endswith(".cu")
                    and "launch_overlapped(" in open(os.path.join(CSRC, f), encoding="utf-8").read())


def code(name):
    return re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name), encoding="utf-8").read())


def test_the_files_are_found():
    assert {"paged_attn.cu", "cache_rows.cu", "extend_tables.cu"} <= set(OVERLAPPED)


@pytest.mark.parametrize("name", OVERLAPPED + ["serve.cuh"])
def test_ordinary_loads_only(name):
    assert not re.findall(r"__ldg\s*\(|\.nc\.|\bld\.global\.nc\b|__restrict__", code(name))


@pytest.mark.parametrize("name", OVERLAPPED)
def test_every_overlapped_kernel_waits(name):
    text = code(name)
    kernels = re.split(r"__global__", text)[1:]
    assert kernels and all("wait_for_stream();" in k for k in kernels)
