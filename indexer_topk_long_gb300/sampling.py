"""A token for each row of logits from given random numbers: binding over
``ltk_sample_tokens`` (argument checks and marshalling only).

    token, logp = sample(logits, u, temperature=0.8, top_k=50, top_p=0.95)

Filters apply in the order min-p, top-k, top-p, each to what the one before left;
``include/ltk.h`` has the definition.
"""
from __future__ import annotations

import ctypes
import math
import struct

from . import ltk
from .ltk import LTK_BF16, LTK_F16, LTK_F32, Sampling

# A Sampling as bytes: see kv.py
_PACK = struct.Struct("@PPPPfiff").pack
assert struct.calcsize("@PPPPfiff") == ctypes.sizeof(Sampling)


_ready = None                              # (torch, codes of the types, the entry point), once a call has been made


def _load():
    global _ready
    import torch
    _ready = (torch, {torch.bfloat16: LTK_BF16, torch.float16: LTK_F16, torch.float32: LTK_F32},
              ltk.load_library().ltk_sample_tokens)
    return _ready


def _fail(name: str, what: str):
    raise ValueError(f"{name}: {what}")


def _per_row(t, name: str, rows: int, dtype, device) -> int:
    """Address of a contiguous [rows] tensor of ``dtype`` on ``device``."""
    if t.dtype is dtype and t.shape == (rows,) and t.is_contiguous() and t.device == device:
        return t.data_ptr()
    if t.dtype is not dtype:
        _fail(name, f"expected {dtype} elements, got {t.dtype}")
    if tuple(t.shape) != (rows,):
        _fail(name, f"expected shape {(rows,)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        _fail(name, "must be contiguous")
    _fail(name, f"expected a tensor on {device}, got one on {t.device}")


def _setting(x, name: str, rows: int, dtype, device, kind, lo, hi):
    """(address or 0, value): a tensor of one value for each row, or one for all."""
    if isinstance(x, kind):
        return _per_row(x, name, rows, dtype, device), 0
    if not lo <= x <= hi:
        _fail(name, f"expected a value from {lo} to {hi}, got {x}")
    return 0, x


def sample(logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, token=None, logp=None, stream=None):
    """Draws from logits [B, V] (bfloat16, float16 or float32; rows may be strided) with the random numbers u [B]
    (float32 in [0, 1)).  Each setting is a number or a tensor [B] (float32; ``top_k`` int32).  Returns
    (token [B] int32, logp [B] float32); a row that nothing can be drawn from gives -1."""
    torch, codes, entry = _ready or _load()
    shape = logits.shape
    if len(shape) != 2:
        _fail("logits", f"expected a 2-D [rows, vocabulary] tensor, got shape {tuple(shape)}")
    B, V = shape
    code = codes.get(logits.dtype)
    if code is None:
        _fail("logits", f"expected bfloat16, float16 or float32 elements, got {logits.dtype}")
    device = logits.device
    if device.type != "cuda":
        _fail("logits", f"expected a CUDA tensor, got one on {device}")
    index = torch.cuda.current_device()
    if device.index != index:
        _fail("logits", f"is on {device}, the current device is cuda:{index}")
    if V < 1:
        _fail("logits", "has no tokens")
    between, within = logits.stride()
    stride = between if B > 1 else V
    if (within != 1 and V > 1) or stride < V:
        _fail("logits", "each row must be contiguous, and rows must not overlap")
    f32, i32, kind, empty = torch.float32, torch.int32, torch.Tensor, torch.empty
    up = _per_row(u, "u", B, f32, device)
    tp, t = _setting(temperature, "temperature", B, f32, device, kind, 0.0, 3.4e38)
    kp, k = _setting(top_k, "top_k", B, i32, device, kind, -2**31, 2**31 - 1)
    pp, p = _setting(top_p, "top_p", B, f32, device, kind, 0.0, math.inf)
    mp, m = _setting(min_p, "min_p", B, f32, device, kind, 0.0, 1.0)
    if token is not None:
        _per_row(token, "token", B, i32, device)
    if logp is not None:
        _per_row(logp, "logp", B, f32, device)
    whole = int(k)
    if whole != k:
        _fail("top_k", f"expected a whole number, got {k}")
    settings = _PACK(tp, kp, pp, mp, t, whole, min(p, 1.0), m)
    current = torch._C._cuda_getCurrentRawStream(index)
    if stream is None or stream.cuda_stream == current:
        st = current
        token = empty(B, dtype=i32, device=device) if token is None else token
        logp = empty(B, dtype=f32, device=device) if logp is None else logp
    else:
        st = stream.cuda_stream
        for x in (logits, u, temperature, top_k, top_p, min_p, token, logp):
            if isinstance(x, kind):
                x.record_stream(stream)
        with torch.cuda.stream(stream):
            token = empty(B, dtype=i32, device=device) if token is None else token
            logp = empty(B, dtype=f32, device=device) if logp is None else logp
    failed = entry(logits.data_ptr(), code, stride, B, V, settings, up, token.data_ptr(), logp.data_ptr(), st)
    if failed:
        ltk._check(failed, "ltk_sample_tokens")
    return token, logp
