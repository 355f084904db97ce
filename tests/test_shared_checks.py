"""Refusals of the entry points for continuations (shared attention, reading back) without a handle, and how the
sampler's kernel begins and loads, as its source has it."""
import ctypes
import os
import re

import pytest

from indexer_topk_long_gb300 import ltk


def test_null_arguments(ltk_lib):
    b, size = ltk.KvBatch(), ctypes.c_ulonglong(7)
    for batch in (ctypes.byref(b), None):
        assert ltk_lib.ltk_kv_attention_shared(None, batch, None, 0, 0, None, 0, 8, 1, 1.0, None, None, None, 0, None) == 1
        assert ltk_lib.ltk_kv_read(None, batch, 0, None, None, 0, 0, 0, None, None, None) == 1
    assert ltk_lib.ltk_kv_shared_bytes(None, 1, 1, 1, ctypes.byref(size)) == 1
    assert size.value == 7


@pytest.mark.parametrize("name,uses", [("k_sampling.cu", "cudaLaunchKernelEx("), ("k_kv_share.cu", "launch_overlapped("), ("k_kv_read.cu", "launch_overlapped(")])
def test_overlapped_kernels_wait_and_load_coherently(name, uses):
    csrc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "indexer_topk_long_gb300", "csrc")
    with open(os.path.join(csrc, name)) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    assert uses in code
    assert len(re.findall(r"__global__ void", code)) == len(re.findall(r"\bbegin_after_previous\(\);", code)) > 0
    assert not re.findall(r"__ldg\s*\(|ld\.global(?:\.\w+)*\.nc\b|__restrict__", code)
