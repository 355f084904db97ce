"""Refusals of the paged cache's calls, without a GPU: the C entry points check
their arguments on the host before any CUDA work, the binding its tensors."""
import ctypes

import pytest
import torch

from indexer_topk_long_gb300 import kv, ltk

CPU = torch.device("cpu")


def _config(**kw):
    cfg = ltk.KvConfig(4, 2, 128, 64, 0, 1 << 12, 1 << 13, 1 << 14, 1 << 15)
    for k, v in kw.items():
        setattr(cfg, k, v)
    return cfg


@pytest.mark.parametrize("field,value,status", [
    ("num_pages", 0, 1), ("num_pages", 1 << 31, 1), ("heads", 0, 1), ("heads", 1 << 17, 1), ("page", 8, 6),
    ("page", 48, 6), ("page", 256, 6), ("dim", 96, 6), ("dim", 0, 6), ("engine", -1, 1), ("engine", 3, 1), ("k_codes", None, 1), ("v_codes", 8, 1),
    ("k_scale", None, 1), ("v_scale", 4, 1)])
def test_create_refuses(ltk_lib, field, value, status):
    h = ctypes.c_void_p()
    assert ltk_lib.ltk_kv_create(ctypes.byref(_config(**{field: value})), ctypes.byref(h)) == status
    assert not h.value


def test_null_arguments(ltk_lib):
    h = ctypes.c_void_p()
    b = ltk.KvBatch()
    assert ltk_lib.ltk_kv_create(None, ctypes.byref(h)) == 1
    assert ltk_lib.ltk_kv_create(ctypes.byref(_config()), None) == 1
    assert ltk_lib.ltk_kv_append(None, ctypes.byref(b), 0, None, 0, None, 0, None, None, 0, 0, 0, None, 0, 0, None,
                                 None) == 1
    assert ltk_lib.ltk_kv_attention(None, ctypes.byref(b), 0, None, 0, 8, 1, 1.0, 0, 0, None, None, None) == 1
    assert ltk_lib.ltk_kv_attention_selected(None, ctypes.byref(b), 0, None, 0, 8, None, 4, 1.0, None, None,
                                             None) == 1
    assert ltk_lib.ltk_kv_attention_selected(None, None, 0, None, 0, 8, None, 0, 1.0, None, None, None) == 1
    v = ctypes.c_int(0)
    assert ltk_lib.ltk_kv_status(None, ctypes.byref(v), None) == 1
    ltk_lib.ltk_kv_destroy(None)


def _batch(B=3, W=5):
    return (torch.zeros((B, W), dtype=torch.int32), torch.zeros(B, dtype=torch.int32),
            torch.zeros(B + 1, dtype=torch.int32))


def test_batch_accepted():
    b = kv.check_batch(*_batch(), 7, CPU)
    assert (b.B, b.table_width, b.N) == (3, 5, 7)


@pytest.mark.parametrize("at,bad,msg", [
    (0, torch.zeros((3, 5), dtype=torch.int64), "int32"),
    (0, torch.zeros((3, 10), dtype=torch.int32)[:, ::2], "contiguous"),
    (0, torch.zeros(15, dtype=torch.int32), "2-D"),
    (1, torch.zeros(4, dtype=torch.int32), "shape"),
    (1, torch.zeros(3), "int32"),
    (2, torch.zeros(3, dtype=torch.int32), "shape"),
])
def test_batch_refused(at, bad, msg):
    t = list(_batch())
    t[at] = bad
    with pytest.raises(ValueError, match=msg):
        kv.check_batch(*t, 7, CPU)


def test_batch_on_another_device():
    with pytest.raises(ValueError, match="expected a tensor on"):
        kv.check_batch(*_batch(), 7, torch.device("cuda", 0))


def test_rows_accepted():
    x = torch.zeros((6, 10, 128), dtype=torch.bfloat16)
    assert kv._rows(x, "q", 6, 128, CPU) == (10, 1280)
    assert kv._rows(x[:, 2:6], "q", 6, 128, CPU) == (4, 1280)
    assert kv._rows(x[:1, 2:6], "q", 1, 128, CPU)[0] == 4
    assert kv._rows(x[:0], "q", 0, 128, CPU)[0] == 10


@pytest.mark.parametrize("bad,msg", [
    (torch.zeros((6, 4, 64), dtype=torch.bfloat16), "shape"),
    (torch.zeros((5, 4, 128), dtype=torch.bfloat16), "shape"),
    (torch.zeros((6, 512), dtype=torch.bfloat16), "shape"),
    (torch.zeros((6, 4, 128)), "bfloat16 or float16"),
    (torch.zeros((6, 4, 128), dtype=torch.float16), "like the others"),
    (torch.zeros((6, 128, 4), dtype=torch.bfloat16).transpose(1, 2), "contiguous"),
    (torch.zeros((6, 8, 128), dtype=torch.bfloat16)[:, ::2], "contiguous"),
    (torch.zeros((6 * 513 + 8,), dtype=torch.bfloat16).as_strided((6, 4, 128), (513, 128, 1)), "16-byte"),
    (torch.zeros((6 * 512 + 8,), dtype=torch.bfloat16)[4:].as_strided((6, 4, 128), (512, 128, 1), 4), "16-byte"),
    (torch.zeros((1, 4, 128), dtype=torch.bfloat16).expand(6, 4, 128), "not overlap"),
    (torch.zeros((6, 0, 128), dtype=torch.bfloat16), "heads"),
])
def test_rows_refused(bad, msg):
    with pytest.raises(ValueError, match=msg):
        kv._rows(bad, "q", 6, 128, CPU, torch.bfloat16)
