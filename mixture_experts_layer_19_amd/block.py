"""The operators next to the MoE layer in its decoder block: RMS norm with the
residual's addition and an 8-bit output, the paged KV cache, and attention of
new tokens over that cache.

Plumbing only, as in :mod:`.layer`: torch holds device memory and streams, the
HIP library (through :mod:`.binding`) does the arithmetic.  Calls run on the
current stream (or ``stream=``), do not synchronise, and take nothing from one
call to the next, so they can be captured into a graph; lengths and page tables
are read on the device when the kernels run.

    cache = PagedKVCache(kv_heads=8, head_dim=128, num_pages=4096, page_size=64, dtype="mxfp8")
    batch = KVBatch(page_table, row_offsets, kv_len, rows=q.shape[0], max_rows=1)
    cache.write(batch, k, v)
    o = cache.attention(batch, q, window=4096, sinks=16)
    norm = RMSNorm(weight, quant="mxfp8")
    residual, y, q8, scale = norm(x, residual)

What cannot be seen from the host (the contents of the page table, offsets and
lengths) is not checked: whatever it is, no access leaves the tensors.
Arguments of the wrong type, shape or device raise ValueError; what the library
refuses raises :class:`.binding.MoeError`.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

import torch

from . import binding as B

_ACT = {torch.float32: B.MOE_F32, torch.bfloat16: B.MOE_BF16}
_CACHE = {"bf16": (B.MOE_BF16, torch.bfloat16, torch.bfloat16),
          "f32": (B.MOE_F32, torch.float32, torch.float32),
          # OCP MX-fp8: E4M3 codes and one E8M0 scale byte per 32 elements of head_dim
          "mxfp8": (B.MOE_MXFP8, torch.uint8, torch.bfloat16)}
_INT32 = 0x7FFFFFFF   # the library counts rows, pages and positions in 32 bits; ctypes would cut a larger one
_QUANT = {"none": B.MOE_NO_QUANT, "mxfp8": B.MOE_MXFP8, "fp8": B.MOE_FP8}
# Small calls are bound by the host: the checks build no message unless they
# fail, the library's functions are called with plain integers, and the stream
# and device are asked for without torch's wrappers.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _require(ok, what):
    if not ok:
        raise ValueError(what)


class _Bound:
    """Attributes (`_bound`) that the C structs copy or that lengths follow from: a
    tensor's contents may change in place, another value needs another object."""
    _bound = frozenset()

    def __setattr__(self, name, value):
        if name in self._bound and value is not self.__dict__.get(name, value):
            raise AttributeError("%s is not replaced; its contents may change in place, another one needs "
                                 "another %s" % (name, type(self).__name__))
        object.__setattr__(self, name, value)


def _elsewhere(index, stream):
    """A context in which the current device and stream are the call's, or None
    if they are already."""
    if stream is not None:
        _require(stream.device_index == index, "the stream is of another device than the tensors")
        return torch.cuda.stream(stream)
    return None if _current_device() == index else torch.cuda.device(index)


def _device(t: torch.Tensor) -> torch.device:
    _require(t.device.type == "cuda", "tensors must be on a GPU, got %s" % t.device)
    return t.device


class NormResult(NamedTuple):
    residual: Optional[torch.Tensor]   # x + residual (None without a residual)
    y: Optional[torch.Tensor]          # the normed rows
    q: Optional[torch.Tensor]          # E4M3 codes, uint8 (None without quantisation)
    scale: Optional[torch.Tensor]      # E8M0 bytes [rows, hidden / 32] (mxfp8 only)


class RMSNorm(_Bound):
    """y = (x + residual) / sqrt(mean((x + residual)^2) + eps) * weight.

    quant: "none"; "mxfp8", E4M3 codes with an E8M0 scale byte per 32 elements;
    "fp8", E4M3 codes of y / fp8_scale.  The sum is held in fp32, the
    statistics, y and y / fp8_scale in 64 bits; every output is rounded once from them."""

    _bound = frozenset(("weight", "quant", "hidden", "dtype", "device"))

    def __init__(self, weight: torch.Tensor, eps: float = 1e-5, quant: str = "none",
                 fp8_scale: float = 0.0):
        _require(weight.dim() == 1 and weight.is_contiguous() and 0 < weight.numel() <= _INT32,
                 "weight must be a contiguous vector of fewer than 2^31 elements")
        _require(weight.dtype in _ACT, "weight must be float32 or bfloat16, got %s" % weight.dtype)
        _require(quant in _QUANT, "quant must be one of %s, got %r" % (sorted(_QUANT), quant))
        _require(quant != "mxfp8" or weight.numel() % 32 == 0, "mxfp8 needs a hidden size in multiples of 32")
        _require(quant != "fp8" or 0.0 < fp8_scale < 3.0e38, "fp8 needs a positive fp8_scale")
        _require(eps >= 0.0, "eps must not be negative")
        self.weight = weight
        self.eps, self.quant, self.fp8_scale = float(eps), quant, float(fp8_scale)
        self.hidden, self.dtype = weight.numel(), weight.dtype
        self.device = _device(weight)
        self._q, self._dtype = _QUANT[quant], _ACT[weight.dtype]
        self._call = B.lib().moe_rms_norm

    def __call__(self, x: torch.Tensor, residual: Optional[torch.Tensor] = None, *, want_y: bool = True,
                 stream=None) -> NormResult:
        """x, residual: [rows, hidden], rows contiguous inside.  want_y False
        leaves y out where there is an 8-bit output."""
        hidden, dev = self.hidden, self.device
        shape = x.shape
        for t in (x,) if residual is None else (x, residual):
            if t.dim() != 2 or t.shape != shape or shape[1] != hidden or t.dtype != self.dtype or t.device != dev:
                raise ValueError("expected [rows, %d] of %s on %s, got %s of %s on %s"
                                 % (hidden, self.dtype, dev, list(t.shape), t.dtype, t.device))
            if t.stride(1) != 1 and hidden != 1:
                raise ValueError("rows must be contiguous")
        if shape[0] > _INT32:
            raise ValueError("%d rows are more than 2^31 - 1" % shape[0])
        if not want_y and self._q == B.MOE_NO_QUANT:
            raise ValueError("without y there is no output")
        other = _elsewhere(dev.index, stream)
        if other is not None:
            with other:
                return self(x, residual, want_y=want_y)
        # (empty_like of overlapping rows need not be contiguous)
        new, r, y, q, scale = torch.empty_strided, None, None, None, None
        rp = rs = ro = yp = qp = sp = 0
        row = (hidden, 1)
        if residual is not None:
            r = new(shape, row, dtype=self.dtype, device=dev)
            rp, rs, ro = residual.data_ptr(), residual.stride(0), r.data_ptr()
        if want_y:
            y = new(shape, row, dtype=self.dtype, device=dev)
            yp = y.data_ptr()
        if self._q != B.MOE_NO_QUANT:
            q = new(shape, row, dtype=torch.uint8, device=dev)
            qp = q.data_ptr()
            if self._q == B.MOE_MXFP8:
                n = hidden // 32
                scale = new((shape[0], n), (n, 1), dtype=torch.uint8, device=dev)
                sp = scale.data_ptr()
        rc = self._call(x.data_ptr(), x.stride(0), rp, rs, self.weight.data_ptr(), self._dtype, shape[0], hidden,
                        self.eps, ro, yp, self._q, self.fp8_scale, qp, sp, _raw_stream(dev.index))
        if rc:
            B._check(rc)
        return NormResult(r, y, q, scale)


class KVBatch(_Bound):
    """New tokens of a batch of sequences and where their tokens lie.

    page_table [seqs, max_pages] int32 (entries that are no page hold nothing),
    row_offsets [seqs + 1] int32 ascending, kv_len [seqs] int32: the length of
    each sequence with its new tokens.  rows: new tokens of all sequences;
    max_rows: at least the most of one sequence (rows if not given).  The
    tensors may be changed in place between calls; other counts need another
    batch."""

    _bound = frozenset(("page_table", "row_offsets", "kv_len", "seqs", "rows", "max_rows", "device", "c"))

    def __init__(self, page_table: torch.Tensor, row_offsets: torch.Tensor, kv_len: torch.Tensor, rows: int,
                 max_rows: Optional[int] = None):
        _require(page_table.dim() == 2, "page_table must be [seqs, max_pages]")
        seqs = page_table.shape[0]
        _require(row_offsets.shape == (seqs + 1,) and kv_len.shape == (seqs,),
                 "expected row_offsets [%d] and kv_len [%d], got %s and %s"
                 % (seqs + 1, seqs, list(row_offsets.shape), list(kv_len.shape)))
        self.device = _device(page_table)
        for t in (page_table, row_offsets, kv_len):
            _require(t.dtype == torch.int32 and t.is_contiguous() and t.device == self.device,
                     "page_table, row_offsets and kv_len must be contiguous int32 on one device")
        max_rows = rows if max_rows is None else max_rows
        _require(max(rows, seqs, page_table.shape[1]) <= _INT32, "rows, sequences and pages of one must be below 2^31")
        _require(rows >= 0 and 0 <= max_rows <= rows and (rows == 0 or max_rows > 0),
                 "rows %d and max_rows %d do not fit together" % (rows, max_rows))
        self.page_table, self.row_offsets, self.kv_len = page_table, row_offsets, kv_len
        self.seqs, self.rows, self.max_rows = seqs, rows, max_rows
        self.c = B.MoeKvBatch(page_table.data_ptr(), row_offsets.data_ptr(), kv_len.data_ptr(), seqs,
                              page_table.shape[1], rows, max_rows)
        self._ref = ctypes.byref(self.c)


class PagedKVCache(_Bound):
    """Pools of pages [num_pages, kv_heads, page_size, head_dim] of keys and
    values: dtype "bf16", "f32" or "mxfp8" (uint8 E4M3 codes, and E8M0 scale
    bytes [num_pages, kv_heads, page_size, head_dim / 32]).  Activations are
    bf16, for an "f32" cache fp32.

    storage: (k, v, k_scale, v_scale) to use instead of new, zeroed pools."""

    _bound = frozenset(("k", "v", "k_scale", "v_scale", "kv_heads", "head_dim", "num_pages", "page_size", "dtype",
                        "act_dtype", "device", "c"))

    def __init__(self, kv_heads: int, head_dim: int, num_pages: int, page_size: int, dtype: str = "bf16",
                 device="cuda", storage=None):
        _require(dtype in _CACHE, "dtype must be one of %s, got %r" % (sorted(_CACHE), dtype))
        _require(kv_heads > 0 and num_pages > 0 and page_size > 0, "a cache needs heads, pages and slots")
        _require(max(kv_heads, num_pages) <= _INT32, "heads and pages must be below 2^31")
        _require(page_size & (page_size - 1) == 0 and page_size <= 65536,
                 "page_size must be a power of two up to 65536, got %d" % page_size)
        _require(head_dim in (64, 128, 256), "head_dim must be 64, 128 or 256, got %d" % head_dim)
        code, store, self.act_dtype = _CACHE[dtype]
        shape = (num_pages, kv_heads, page_size, head_dim)
        scale_shape = shape[:3] + (head_dim // 32,)
        mx = dtype == "mxfp8"
        if storage is None:
            k, v = (torch.zeros(shape, dtype=store, device=device) for _ in "kv")
            ks, vs = ((torch.zeros(scale_shape, dtype=torch.uint8, device=device) for _ in "kv")
                      if mx else (None, None))
        else:
            k, v, ks, vs = storage
            _require((ks is not None) == mx and (vs is not None) == mx, "scales go with an mxfp8 cache only")
            for t, want, kind in ((k, shape, store), (v, shape, store), (ks, scale_shape, torch.uint8),
                                  (vs, scale_shape, torch.uint8)):
                _require(t is None or (tuple(t.shape) == want and t.dtype == kind and t.is_contiguous()
                                       and t.device == k.device),
                         "storage must be contiguous %s of %s on one device" % (list(want), kind))
        self.k, self.v, self.k_scale, self.v_scale = k, v, ks, vs
        self.kv_heads, self.head_dim, self.num_pages, self.page_size = kv_heads, head_dim, num_pages, page_size
        self.dtype, self.device = dtype, _device(k)
        self.c = B.MoeKvCache(k.data_ptr(), v.data_ptr(), ks.data_ptr() if mx else None,
                              vs.data_ptr() if mx else None, num_pages, page_size, kv_heads, head_dim, code)
        lib = B.lib()
        self._ref = ctypes.byref(self.c)
        self._write, self._read = lib.moe_kv_write, lib.moe_kv_read
        self._attend, self._attend_ws = lib.moe_attention, lib.moe_attention_workspace_bytes

    def _check(self, batch, t, heads, what):
        if t.shape != (batch.rows, heads, self.head_dim) or t.dtype != self.act_dtype or t.device != self.device:
            raise ValueError("%s must be [%d, %d, %d] of %s on %s, got %s of %s on %s"
                             % (what, batch.rows, heads, self.head_dim, self.act_dtype, self.device, list(t.shape),
                                t.dtype, t.device))
        if t.stride(2) != 1:
            raise ValueError("%s must be contiguous along head_dim" % what)
        if batch.device != self.device:
            raise ValueError("the batch is on %s, the cache on %s" % (batch.device, self.device))

    def write(self, batch: KVBatch, k: torch.Tensor, v: torch.Tensor, *, stream=None) -> None:
        """Put the new tokens' k and v [rows, kv_heads, head_dim] (row and head
        strides in whole 16-byte pieces) into their pages."""
        self._check(batch, k, self.kv_heads, "k")
        self._check(batch, v, self.kv_heads, "v")
        other = _elsewhere(self.device.index, stream)
        if other is not None:
            with other:
                return self.write(batch, k, v)
        rc = self._write(self._ref, batch._ref, k.data_ptr(), k.stride(0), k.stride(1), v.data_ptr(), v.stride(0),
                         v.stride(1), _raw_stream(self.device.index))
        if rc:
            B._check(rc)

    def read(self, batch: KVBatch, *, stream=None):
        """The batch's tokens' (k, v) [rows, kv_heads, head_dim], dequantised."""
        _require(batch.device == self.device, "the batch and the cache are on different devices")
        other = _elsewhere(self.device.index, stream)
        if other is not None:
            with other:
                return self.read(batch)
        heads, dim = self.kv_heads, self.head_dim
        k = torch.empty_strided((batch.rows, heads, dim), (heads * dim, dim, 1), dtype=self.act_dtype,
                                device=self.device)
        v = torch.empty_like(k)
        rc = self._read(self._ref, batch._ref, k.data_ptr(), v.data_ptr(), _raw_stream(self.device.index))
        if rc:
            B._check(rc)
        return k, v

    def attention(self, batch: KVBatch, q: torch.Tensor, scale: Optional[float] = None, window: int = 0,
                  sinks: int = 0, *, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """Attention of q [rows, heads, head_dim] over each row's sequence up to
        its own position; with window > 0 over the last `window` positions and
        the first `sinks`.  heads is a multiple of kv_heads.  scale:
        head_dim ** -0.5 if not given.  A row that sees nothing gives zeros."""
        if q.dim() != 3:
            raise ValueError("q must be [rows, heads, head_dim]")
        heads = q.shape[1]
        self._check(batch, q, heads, "q")
        if heads == 0 or heads % self.kv_heads:
            raise ValueError("%d heads do not share %d KV heads" % (heads, self.kv_heads))
        if window < 0 or sinks < 0:
            raise ValueError("window and sinks must not be negative")
        if out is not None:
            self._check(batch, out, heads, "out")
            _require(out.is_contiguous(), "out must be contiguous")
        # the library counts positions in 32 bits: a larger window hides nothing either
        window, sinks = min(window, _INT32), min(sinks, _INT32)
        other = _elsewhere(self.device.index, stream)
        if other is not None:
            with other:
                return self.attention(batch, q, scale, window, sinks, out=out)
        if out is None:
            out = torch.empty_like(q, memory_format=torch.contiguous_format)
        n, ws, wp = self._attend_ws(self._ref, batch._ref, heads, window, sinks), None, 0
        if n:
            ws = torch.empty_strided((n,), (1,), dtype=torch.uint8, device=self.device)
            wp = ws.data_ptr()
        rc = self._attend(self._ref, batch._ref, q.data_ptr(), q.stride(0), q.stride(1), heads,
                          self.head_dim ** -0.5 if scale is None else scale, window, sinks, out.data_ptr(), wp, n,
                          _raw_stream(self.device.index))
        if rc:
            B._check(rc)
        return out
