"""Paged key/value cache held in 8 bits and the attention that reads it: binding
over the ``ltk_kv_*`` entry points (argument checks and marshalling only).

    cache = PagedKVCache(num_pages, heads, dim, page=64)
    q = cache.append(k, v, page_table, seq_lens, cu_q, cos, sin, q=q)      # rotate, quantise, store
    out, lse = cache.attention(q, page_table, seq_lens, cu_q)              # causal, optional window
    out, lse = cache.attention_selected(q, idx, page_table, seq_lens, cu_q)  # the indexer's keys

The batch is three int32 CUDA tensors: ``page_table`` [B, width], ``seq_lens``
[B] (cached tokens, this step's among them) and ``cu_q`` [B + 1] (first new
token of each sequence).  Nothing is copied to the host.  Calls on one cache
share its workspace: issue them on one stream, or synchronise between streams.
"""
from __future__ import annotations

import ctypes
import math
import struct

from . import ltk
from .ltk import KvBatch, KvConfig, LTK_BF16, LTK_F16

DTYPES = {"torch.bfloat16": LTK_BF16, "torch.float16": LTK_F16}
# A KvBatch as bytes: a decode step is host-bound, and packing takes a third of a ctypes structure's time.
_PACK = struct.Struct("@PiPPii").pack
assert struct.calcsize("@PiPPii") == ctypes.sizeof(KvBatch)


def _fail(name: str, what: str):
    raise ValueError(f"{name}: {what}")


def _int32s(**values) -> None:
    """ctypes cuts whole numbers to 32 bits without a word."""
    for name, x in values.items():
        if not -2**31 <= x < 2**31:
            _fail(name, f"expected a 32-bit whole number, got {x}")


def _device_ok(t, name: str, device) -> None:
    if t.device != device:
        _fail(name, f"expected a tensor on {device}, got one on {t.device}")


def _ints(t, name: str, shape, device) -> None:
    import torch
    if t.dtype != torch.int32:
        _fail(name, f"expected int32 elements, got {t.dtype}")
    if tuple(t.shape) != shape:
        _fail(name, f"expected shape {shape}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        _fail(name, "must be contiguous")
    _device_ok(t, name, device)


def _rows(t, name: str, n: int, dim: int, device, dtype=None) -> tuple[int, int]:
    """[n, heads, dim] of 16-bit elements, each token's heads contiguous and tokens
    a multiple of 8 elements apart; returns (heads, token stride)."""
    shape = t.shape
    if len(shape) != 3 or shape[0] != n or shape[2] != dim:
        _fail(name, f"expected shape ({n}, heads, {dim}), got {tuple(shape)}")
    if dtype is None:
        if str(t.dtype) not in DTYPES:
            _fail(name, f"expected bfloat16 or float16 elements, got {t.dtype}")
    elif t.dtype is not dtype:
        _fail(name, f"expected {dtype} elements like the others, got {t.dtype}" if str(t.dtype) in DTYPES
              else f"expected bfloat16 or float16 elements, got {t.dtype}")
    _device_ok(t, name, device)
    heads = shape[1]
    if heads < 1:
        _fail(name, "has no heads")
    s0, s1, s2 = t.stride()
    width = heads * dim
    stride = s0 if n > 1 else width
    if s2 != 1 or (s1 != dim and heads > 1):
        _fail(name, "each token's heads must be contiguous")
    if stride & 7 or stride < width or t.data_ptr() & 15:
        _fail(name, "tokens must start on 16-byte boundaries and not overlap")
    return heads, stride


def check_batch(page_table, seq_lens, cu_q, n: int, device) -> KvBatch:
    shape = page_table.shape
    if len(shape) != 2:
        _fail("page_table", f"expected a 2-D tensor, got shape {tuple(shape)}")
    b, width = shape
    kind = page_table.dtype
    # one look when all is well (this is on the path of every decode step), else say what is not
    if not (kind is seq_lens.dtype and kind is cu_q.dtype and str(kind) == "torch.int32"
            and seq_lens.shape == (b,) and cu_q.shape == (b + 1,)
            and page_table.is_contiguous() and seq_lens.is_contiguous() and cu_q.is_contiguous()
            and page_table.device == device and seq_lens.device == device and cu_q.device == device):
        _ints(page_table, "page_table", (b, width), device)
        _ints(seq_lens, "seq_lens", (b,), device)
        _ints(cu_q, "cu_q", (b + 1,), device)
    return KvBatch(page_table.data_ptr(), width, seq_lens.data_ptr(), cu_q.data_ptr(), b, n)


def _batch(page_table, seq_lens, cu_q, n: int, device, int32):
    """check_batch's checks, and the batch packed; (how many sequences, packed)."""
    shape = page_table.shape
    if (len(shape) == 2 and page_table.dtype is int32 and seq_lens.dtype is int32 and cu_q.dtype is int32
            and seq_lens.shape == ((b := shape[0]),) and cu_q.shape == (b + 1,)
            and page_table.is_contiguous() and seq_lens.is_contiguous() and cu_q.is_contiguous()
            and page_table.device == device and seq_lens.device == device and cu_q.device == device):
        return b, _PACK(page_table.data_ptr(), shape[1], seq_lens.data_ptr(), cu_q.data_ptr(), b, n)
    check_batch(page_table, seq_lens, cu_q, n, device)   # says what is wrong
    raise AssertionError("unreachable")


class PagedKVCache:
    """One layer's cache and its ``ltk_kv`` handle on the current device.

    Without the four buffers the cache is allocated, zeroed.  ``k_codes`` and
    ``v_codes`` are uint8 (or float8_e4m3fn) [num_pages, heads, page, dim],
    ``k_scale`` and ``v_scale`` fp32 [num_pages, heads] (0: a block of zeros; append
    writes powers of two).  ``engine`` 0 lets measured costs
    choose the attention kernel, 1 takes the one for few rows, 2 the tensor-core tiles."""

    def __init__(self, num_pages: int, heads: int, dim: int, page: int = 64, k_codes=None, v_codes=None,
                 k_scale=None, v_scale=None, engine: int = 0):
        import torch
        self.h = None
        self.lib = ltk.load_library()
        self.num_pages, self.heads, self.dim, self.page = int(num_pages), int(heads), int(dim), int(page)
        _int32s(heads=self.heads, dim=self.dim, page=self.page, engine=int(engine))
        given = [t is not None for t in (k_codes, v_codes, k_scale, v_scale)]
        if any(given) and not all(given):
            raise ValueError("k_codes, v_codes, k_scale, v_scale: give all four or none")
        self.device = torch.device("cuda", torch.cuda.current_device())
        self._torch, self._index, self._raw_stream = torch, self.device.index, torch._C._cuda_getCurrentRawStream
        self._int32, self._float32 = torch.int32, torch.float32
        self._default_scale = 1.0 / math.sqrt(self.dim)
        self._codes = {torch.bfloat16: LTK_BF16, torch.float16: LTK_F16}
        self._append, self._attend = self.lib.ltk_kv_append, self.lib.ltk_kv_attention
        self._attend_selected = self.lib.ltk_kv_attention_selected
        codes, scales = (self.num_pages, self.heads, self.page, self.dim), (self.num_pages, self.heads)
        if not all(given):
            k_codes, v_codes = (torch.zeros(codes, dtype=torch.uint8, device=self.device) for _ in range(2))
            k_scale, v_scale = (torch.zeros(scales, dtype=torch.float32, device=self.device) for _ in range(2))
        for t, name, shape, size in ((k_codes, "k_codes", codes, 1), (v_codes, "v_codes", codes, 1),
                                     (k_scale, "k_scale", scales, 4), (v_scale, "v_scale", scales, 4)):
            if tuple(t.shape) != shape:
                _fail(name, f"expected shape {shape}, got {tuple(t.shape)}")
            if size == 4 and t.dtype != torch.float32:
                _fail(name, f"expected float32 elements, got {t.dtype}")
            if size == 1 and t.dtype not in (torch.uint8, torch.float8_e4m3fn):
                _fail(name, f"expected uint8 or float8_e4m3fn elements, got {t.dtype}")
            if not t.is_contiguous():
                _fail(name, "must be contiguous")
            _device_ok(t, name, self.device)
        self.k_codes, self.v_codes, self.k_scale, self.v_scale = k_codes, v_codes, k_scale, v_scale
        cfg = KvConfig(self.num_pages, self.heads, self.dim, self.page, int(engine), k_codes.data_ptr(), v_codes.data_ptr(),
                       k_scale.data_ptr(), v_scale.data_ptr())
        # the handle's workspace must not be set up before the buffers' own stream has made them
        torch.cuda.current_stream().synchronize()
        h = ctypes.c_void_p()
        ltk._check(self.lib.ltk_kv_create(ctypes.byref(cfg), ctypes.byref(h)), "ltk_kv_create")
        self.h = h

    # -- helpers ---------------------------------------------------------------
    def _begin(self, stream, *tensors) -> int:
        """The stream to launch on (its handle).  Tensors of the caller's that another
        stream than the current one reads or writes are kept from reuse until it has."""
        if self.h is None:
            raise ValueError("the cache is closed")
        if stream is None:
            return self._raw_stream(self._index)
        if stream.cuda_stream != self._raw_stream(self._index):
            for t in (*tensors, self.k_codes, self.v_codes, self.k_scale, self.v_scale):
                if t is not None:
                    t.record_stream(stream)
        return stream.cuda_stream

    def _queries(self, q, n: int, kind=None) -> tuple[int, int]:
        """_rows' checks of q (elements of ``kind``, or any the library takes); the usual case
        in one look, since a decode step is bound by what the host does."""
        shape = q.shape
        if len(shape) == 3 and shape[0] == n and shape[2] == self.dim and (
                q.dtype in self._codes if kind is None else q.dtype is kind) and q.device == self.device:
            s0, s1, s2 = q.stride()
            if s1 == self.dim and s2 == 1 and s0 >= shape[1] * s1 > 0 and s0 & 7 == 0 and q.data_ptr() & 15 == 0:
                return shape[1], s0
        return _rows(q, "q", n, self.dim, self.device, kind)

    def _new(self, stream, shape, dtype):
        """An output that belongs to the stream the call runs on."""
        if stream is None:
            return self._torch.empty(shape, dtype=dtype, device=self.device)
        with self._torch.cuda.stream(stream):
            return self._torch.empty(shape, dtype=dtype, device=self.device)

    def _outputs(self, stream, q, n, heads, out, lse):
        f32 = self._float32
        if out is None and lse is None and stream is None:
            empty, device = self._torch.empty, self.device
            return empty((n, heads, self.dim), dtype=q.dtype, device=device), empty((n, heads), dtype=f32, device=device)
        shape = (n, heads, self.dim)
        if out is None:
            out = self._new(stream, shape, q.dtype)
        elif tuple(out.shape) != shape or out.dtype != q.dtype or not out.is_contiguous() or out.device != q.device:
            _fail("out", f"expected a contiguous {q.dtype} tensor of shape {shape} on {q.device}")
        if lse is None:
            lse = self._new(stream, (n, heads), f32)
        elif tuple(lse.shape) != (n, heads) or lse.dtype != f32 or not lse.is_contiguous() or lse.device != q.device:
            _fail("lse", f"expected a contiguous float32 tensor of shape {(n, heads)} on {q.device}")
        return out, lse

    # -- API -------------------------------------------------------------------
    def append(self, k, v, page_table, seq_lens, cu_q, cos=None, sin=None, interleaved: bool = False, q=None,
               q_out=None, stream=None):
        """Stores the new tokens' k, v [N, heads, dim]; keys and q are rotated by the rows
        of cos, sin [positions, rot / 2] when given.  Returns the rotated q (None without q)."""
        dim, device = self.dim, self.device
        shape, kind = k.shape, k.dtype
        n = shape[0]
        B, batch = _batch(page_table, seq_lens, cu_q, n, device, self._int32)
        kp, vp = k.data_ptr(), v.data_ptr()
        if (kind in self._codes and shape == (n, self.heads, dim) and v.shape == shape and v.dtype is kind
                and k.device == device and v.device == device and (kp | vp) & 15 == 0
                and k.stride()[1:] == (dim, 1) and v.stride()[1:] == (dim, 1)
                and (ks := k.stride(0)) & 7 == 0 and (vs := v.stride(0)) & 7 == 0 and ks >= self.heads * dim <= vs):
            pass                               # the usual case in one look; else what is wrong
        else:
            kh, ks = _rows(k, "k", n, dim, device)
            vh, vs = _rows(v, "v", n, dim, device, kind)
            if kh != self.heads or vh != self.heads:
                _fail("k" if kh != self.heads else "v", f"expected {self.heads} heads")
        rot = rows = 0
        if (cos is None) != (sin is None):
            raise ValueError("cos, sin: give both or neither")
        if cos is not None:
            table, f32 = cos.shape, self._float32
            if len(table) != 2 or sin.shape != table or cos.dtype is not f32 or sin.dtype is not f32 \
                    or not (cos.is_contiguous() and sin.is_contiguous()):
                raise ValueError("cos, sin: expected contiguous float32 tables of equal shape [positions, rot / 2]")
            if cos.device != device or sin.device != device:
                _device_ok(cos, "cos", device)
                _device_ok(sin, "sin", device)
            rows, rot = table[0], 2 * table[1]
        qh = qs = 0
        if q is not None:
            qh, qs = self._queries(q, n, kind)
        if q_out is not None:
            if q is None:
                raise ValueError("q_out: given without q")
            if tuple(q_out.shape) != (n, qh, self.dim) or q_out.dtype != q.dtype or not q_out.is_contiguous() \
                    or q_out.device != q.device:
                _fail("q_out", f"expected a contiguous {q.dtype} tensor of shape {(n, qh, self.dim)}")
        if stream is None and self.h is not None:
            st = self._raw_stream(self._index)
        else:
            st = self._begin(stream, k, v, page_table, seq_lens, cu_q, cos, sin, q, q_out)
        if q is not None and q_out is None:
            q_out = self._new(stream, (n, qh, dim), kind)
        failed = self._append(
            self.h, batch, self._codes[kind], kp, ks, vp, vs,
            None if cos is None else cos.data_ptr(), None if sin is None else sin.data_ptr(), rows, rot,
            1 if interleaved else 0, None if q is None else q.data_ptr(), qs, qh,
            None if q_out is None else q_out.data_ptr(), st)
        if failed:
            ltk._check(failed, "ltk_kv_append")
        return q_out

    def attention(self, q, page_table, seq_lens, cu_q, max_q: int | None = None, scale: float | None = None,
                  window: int = 0, sinks: int = 0, out=None, lse=None, stream=None):
        """Causal attention of q [N, q_heads, dim] over the cached tokens; with ``window`` > 0 a
        query at p sees keys j > p - window and the first ``sinks`` keys.  ``max_q`` (the most
        queries of one sequence) only helps choose a kernel; left out, the batch's mean stands in,
        which can choose a slower one where lengths differ much.  Returns (out, lse)."""
        n = q.shape[0]
        B, batch = _batch(page_table, seq_lens, cu_q, n, self.device, self._int32)
        heads, qs = self._queries(q, n)
        if max_q is None:
            max_q = -(-n // max(B, 1))
        if (window | sinks | max_q) >> 31:
            _int32s(window=window, sinks=sinks, max_q=max_q)
        if stream is None and self.h is not None:
            st = self._raw_stream(self._index)
        else:
            st = self._begin(stream, q, page_table, seq_lens, cu_q, out, lse)
        out, lse = self._outputs(stream, q, n, heads, out, lse)
        failed = self._attend(
            self.h, batch, self._codes[q.dtype], q.data_ptr(), qs, heads, max_q,
            self._default_scale if scale is None else float(scale), window, sinks, out.data_ptr(), lse.data_ptr(), st)
        if failed:
            ltk._check(failed, "ltk_kv_attention")
        return out, lse

    def attention_selected(self, q, idx, page_table, seq_lens, cu_q, scale: float | None = None, out=None,
                           lse=None, stream=None):
        """Attention of each query over its own key positions idx [N, k] (int32, -1 = empty
        slot), e.g. the indices IndexerTopK returns.  Returns (out, lse)."""
        n = q.shape[0]
        B, batch = _batch(page_table, seq_lens, cu_q, n, self.device, self._int32)
        heads, qs = self._queries(q, n)
        listed = idx.shape
        if len(listed) != 2:
            _fail("idx", f"expected a 2-D [queries, k] tensor, got shape {tuple(listed)}")
        if listed[0] != n or idx.dtype is not self._int32 or not idx.is_contiguous() or idx.device != self.device:
            _ints(idx, "idx", (n, listed[1]), self.device)
        if stream is None and self.h is not None:
            st = self._raw_stream(self._index)
        else:
            st = self._begin(stream, q, idx, page_table, seq_lens, cu_q, out, lse)
        out, lse = self._outputs(stream, q, n, heads, out, lse)
        failed = self._attend_selected(
            self.h, batch, self._codes[q.dtype], q.data_ptr(), qs, heads, idx.data_ptr(), listed[1],
            self._default_scale if scale is None else float(scale), out.data_ptr(), lse.data_ptr(), st)
        if failed:
            ltk._check(failed, "ltk_kv_attention_selected")
        return out, lse

    def status(self, stream=None) -> int:
        """First error the device raised since the last call (0: none); synchronises the stream."""
        st = self._begin(stream)
        value = ctypes.c_int(0)
        ltk._check(self.lib.ltk_kv_status(self.h, ctypes.byref(value), st), "ltk_kv_status")
        return value.value

    def close(self) -> None:
        if getattr(self, "h", None):
            self.lib.ltk_kv_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
