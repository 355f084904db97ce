"""Kernels that start while the one before them runs (launch_overlapped) may not read through the
non-coherent path: what that kernel writes is not read-only for their lifetime."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "indexer_topk_long_gb300", "csrc")


def _code(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


OVERLAPPED = sorted(n for n in os.listdir(CSRC) if "launch_overlapped(" in _code(n))


def test_overlapped_kernels_are_found():
    assert {"k_kv_append.cu", "k_kv_list.cu", "k_kv_rows.cu", "k_kv_tile.cu"} <= set(OVERLAPPED)


@pytest.mark.parametrize("name", sorted(set(OVERLAPPED) | {"kv_internal.cuh", "kv_tensor.cuh"}))
def test_no_non_coherent_loads(name):
    found = re.findall(r"__ldg\s*\(|ld\.global(?:\.\w+)*\.nc\b|__restrict__", _code(name))
    assert not found, found


@pytest.mark.parametrize("name", [n for n in OVERLAPPED if n.endswith(".cu")])
def test_every_kernel_waits_for_the_one_before(name):
    code = _code(name)
    kernels = re.findall(r"__global__ void", code)
    assert len(kernels) == len(re.findall(r"\bbegin_after_previous\(\);", code)) > 0
