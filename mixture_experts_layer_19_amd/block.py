"""The operators next to the MoE layer in its decoder block: RMS norm with the
residual's addition and an 8-bit output, the matrix product in 8 bits with a
scale per block of 128, the norms of queries and keys with their rotation, the
paged KV cache, attention of new tokens over that cache, and the log
probabilities of tokens behind the last block.

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

    qkv = BlockLinear(w_qkv)(y).unflatten(1, (-1, 128))
    q, k, v = qkv.split((heads, kv_heads, kv_heads), 1)
    q = HeadNormRope(q_weight, k_weight, base=1e4).write(cache, batch, q, k, v)
    logprob, entropy, _, _ = token_logprobs(BlockLinear(w_head, out_dtype=torch.float32)(y), tokens)

What cannot be seen from the host (the contents of the page table, offsets and
lengths) is not checked: whatever it is, no access leaves the tensors.
Arguments of the wrong type, shape or device raise ValueError; what the library
refuses raises :class:`.binding.MoeError`.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional, Tuple

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


class HeadNormRope(_Bound):
    """RMS norm of each head of the queries and keys and their rotation by position,
    in one pass.

    q_weight, k_weight [head_dim] (float32 or bfloat16, the type of q, k and v;
    head_dim 64, 128 or 256).  Pairs of elements (i, i + rotary_dim / 2), or with
    interleaved (2i, 2i + 1), turn by position * inv_freq[i]; inv_freq:
    [rotary_dim / 2], base ** (-2i / rotary_dim) if not given; rotary_dim: head_dim
    if not given (a multiple of 16, with interleaved of 2), the elements behind it are
    normed only.  norm_after: the weights multiply what is turned already."""

    _bound = frozenset(("q_weight", "k_weight", "inv_freq", "head_dim", "rotary_dim", "interleaved", "norm_after",
                        "eps", "dtype", "device", "c"))

    def __init__(self, q_weight: torch.Tensor, k_weight: torch.Tensor, base: float = 10000.0,
                 rotary_dim: Optional[int] = None, inv_freq: Optional[torch.Tensor] = None, eps: float = 1e-5,
                 interleaved: bool = False, norm_after: bool = False):
        for w in (q_weight, k_weight):
            _require(w.dim() == 1 and w.is_contiguous() and w.shape == q_weight.shape and w.dtype == q_weight.dtype
                     and w.device == q_weight.device, "weights must be contiguous vectors of one size, type and device")
        _require(q_weight.dtype in _ACT, "weights must be float32 or bfloat16, got %s" % q_weight.dtype)
        head_dim = q_weight.numel()
        _require(head_dim in (64, 128, 256), "head_dim must be 64, 128 or 256, got %d" % head_dim)
        self.device = _device(q_weight)
        if inv_freq is not None:
            _require(inv_freq.dim() == 1 and inv_freq.device == self.device
                     and inv_freq.dtype in (torch.float32, torch.float64),
                     "inv_freq must be a float32 or float64 vector on %s" % self.device)
            _require(rotary_dim is None or rotary_dim == 2 * inv_freq.numel(),
                     "inv_freq must have rotary_dim / 2 elements")
            rotary_dim = 2 * inv_freq.numel()
        rotary_dim = head_dim if rotary_dim is None else rotary_dim
        _require(0 < rotary_dim <= head_dim and rotary_dim % (2 if interleaved else 16) == 0,
                 "rotary_dim must be a multiple of %d up to %d, got %d" % (2 if interleaved else 16, head_dim, rotary_dim))
        _require(eps >= 0.0, "eps must not be negative")
        if inv_freq is None:
            _require(base > 0.0, "base must be positive")
            at = torch.arange(0, rotary_dim, 2, dtype=torch.float64)
            inv_freq = (float(base) ** (at / -rotary_dim)).to(self.device)
        self.q_weight, self.k_weight = q_weight, k_weight
        self.inv_freq = inv_freq.to(torch.float64).contiguous()
        self.head_dim, self.rotary_dim, self.eps = head_dim, rotary_dim, float(eps)
        self.interleaved, self.norm_after, self.dtype = bool(interleaved), bool(norm_after), q_weight.dtype
        self.c = B.MoeHeadNorm(q_weight.data_ptr(), k_weight.data_ptr(), self.inv_freq.data_ptr(), head_dim,
                               rotary_dim, int(interleaved), int(norm_after), _ACT[q_weight.dtype], self.eps)
        self._ref = ctypes.byref(self.c)
        lib = B.lib()
        self._turn, self._write = lib.moe_head_norm_rope, lib.moe_head_norm_rope_write

    def _check(self, t, rows, what):
        if t.dim() != 3 or t.shape[0] != rows or t.shape[1] == 0 or t.shape[2] != self.head_dim \
                or t.dtype != self.dtype or t.device != self.device:
            raise ValueError("%s must be [%d, heads, %d] of %s on %s, got %s of %s on %s"
                             % (what, rows, self.head_dim, self.dtype, self.device, list(t.shape), t.dtype, t.device))
        if t.stride(2) != 1:
            raise ValueError("%s must be contiguous along head_dim" % what)

    def __call__(self, q: torch.Tensor, k: torch.Tensor, positions: torch.Tensor, *, stream=None):
        """(q, k) [rows, heads, head_dim] and [rows, kv_heads, head_dim] (row and head
        strides in whole 16-byte pieces), normed and turned to positions [rows] int32."""
        rows = q.shape[0] if q.dim() else 0
        self._check(q, rows, "q")
        self._check(k, rows, "k")
        if positions.shape != (rows,) or positions.dtype != torch.int32 or not positions.is_contiguous() \
                or positions.device != self.device:
            raise ValueError("positions must be contiguous int32 [%d] on %s" % (rows, self.device))
        _require(rows <= _INT32, "rows must be below 2^31")
        other = _elsewhere(self.device.index, stream)
        if other is not None:
            with other:
                return self(q, k, positions)
        h, g, d = q.shape[1], k.shape[1], self.head_dim
        q_out = torch.empty_strided((rows, h, d), (h * d, d, 1), dtype=self.dtype, device=self.device)
        k_out = torch.empty_strided((rows, g, d), (g * d, d, 1), dtype=self.dtype, device=self.device)
        rc = self._turn(self._ref, q.data_ptr(), q.stride(0), q.stride(1), h, k.data_ptr(), k.stride(0), k.stride(1),
                        g, positions.data_ptr(), rows, q_out.data_ptr(), k_out.data_ptr(),
                        _raw_stream(self.device.index))
        if rc:
            B._check(rc)
        return q_out, k_out

    def write(self, cache: PagedKVCache, batch: KVBatch, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, *,
              stream=None) -> torch.Tensor:
        """q [rows, heads, head_dim] at the batch's positions; its keys, normed and
        turned, and the values v go into the cache in the same pass."""
        self._check(q, batch.rows, "q")
        _require(self.head_dim == cache.head_dim, "the norm's head_dim is %d, the cache's %d"
                 % (self.head_dim, cache.head_dim))
        cache._check(batch, k, cache.kv_heads, "k")
        cache._check(batch, v, cache.kv_heads, "v")
        _require(self.dtype == cache.act_dtype and self.device == cache.device,
                 "the norm and the cache's activations differ in type or device")
        other = _elsewhere(self.device.index, stream)
        if other is not None:
            with other:
                return self.write(cache, batch, q, k, v)
        rows, h, d = q.shape
        out = torch.empty_strided((rows, h, d), (h * d, d, 1), dtype=self.dtype, device=self.device)
        rc = self._write(self._ref, cache._ref, batch._ref, q.data_ptr(), q.stride(0), q.stride(1), h, k.data_ptr(),
                         k.stride(0), k.stride(1), v.data_ptr(), v.stride(0), v.stride(1), out.data_ptr(),
                         _raw_stream(self.device.index))
        if rc:
            B._check(rc)
        return out


class BlockCodes(NamedTuple):
    q: torch.Tensor        # packed E4M3 codes, uint8
    scale: torch.Tensor    # float32 [in_features / 128, rows up to a multiple of 16]
    rows: int
    shape: Tuple[int, int] # (rows, in_features) of what they are the codes of


class BlockLinear(_Bound):
    """y = x W^T in E4M3 with one fp32 scale per 128 x 128 of the weights and one per
    row and 128 columns of x, accumulated in fp32.

    weight [out_features, in_features]: float32 or bfloat16, quantised here (a block's
    scale is max * (1 / 448), both fp32, as x's is: what ``max / 448`` gives on the GPU, which may
    differ by a step from the quotient); or E4M3 codes (uint8 or float8_e4m3fn) with their scale
    [out_features / 128, in_features / 128] float32, rounded up.  Either is packed
    once; codes of quantised weights are not kept otherwise.  dtype: x's, float32 or bfloat16; out_dtype:
    y's, dtype if not given.  Any sizes."""

    _bound = frozenset(("q", "scale", "out_features", "in_features", "dtype", "out_dtype", "device"))

    def __init__(self, weight: torch.Tensor, scale: Optional[torch.Tensor] = None, dtype=torch.bfloat16,
                 out_dtype=None):
        out_dtype = dtype if out_dtype is None else out_dtype
        _require(dtype in _ACT and out_dtype in _ACT, "dtype and out_dtype must be float32 or bfloat16")
        _require(weight.dim() == 2 and weight.numel() > 0, "weight must be [out_features, in_features]")
        n, k = weight.shape
        _require(max(n, k) <= 1 << 30, "features must not be above 2^30")
        self.device = _device(weight)
        codes = weight.dtype in (torch.uint8, torch.float8_e4m3fn)
        _require(codes or weight.dtype in _ACT, "weight must be float32, bfloat16 or E4M3 codes, got %s" % weight.dtype)
        _require(codes == (scale is not None), "a scale goes with E4M3 codes only, and they with a scale")
        shape = (-(-n // 128), -(-k // 128))
        if codes:
            _require(tuple(scale.shape) == shape and scale.dtype == torch.float32 and scale.is_contiguous()
                     and scale.device == self.device, "scale must be contiguous float32 %s on %s"
                     % (list(shape), self.device))
        if weight.stride(1) != 1 and k != 1:
            weight = weight.contiguous()
        self.out_features, self.in_features, self.dtype, self.out_dtype = n, k, dtype, out_dtype
        lib = B.lib()
        with torch.cuda.device(self.device):
            self.scale = scale if codes else torch.empty(shape, dtype=torch.float32, device=self.device)
            self.q = torch.empty(lib.moe_block_packed_bytes(n, k), dtype=torch.uint8, device=self.device)
            B.moe_block_pack(weight, B.MOE_FP8 if codes else _ACT[weight.dtype], weight.stride(0), n, k, self.q,
                             self.scale, _raw_stream(self.device.index))
        self._in, self._out = _ACT[dtype], _ACT[out_dtype]
        self._w, self._ws = self.q.data_ptr(), self.scale.data_ptr()
        self._call, self._quantize = lib.moe_block_linear, lib.moe_block_quantize
        self._bytes = lib.moe_block_linear_workspace_bytes

    def _check(self, x):
        if x.dim() != 2 or x.shape[1] != self.in_features or x.dtype != self.dtype or x.device != self.device:
            raise ValueError("expected [rows, %d] of %s on %s, got %s of %s on %s"
                             % (self.in_features, self.dtype, self.device, list(x.shape), x.dtype, x.device))
        if x.stride(1) != 1 and self.in_features != 1:
            raise ValueError("rows must be contiguous")
        if x.shape[0] > 1 << 30:
            raise ValueError("%d rows are more than 2^30" % x.shape[0])

    def quantize(self, x: torch.Tensor, *, stream=None) -> BlockCodes:
        """x's codes, for products that share it (weights of the same in_features)."""
        self._check(x)
        other = _elsewhere(self.device.index, stream)
        if other is not None:
            with other:
                return self.quantize(x)
        rows, k = x.shape
        q = torch.empty(B.lib().moe_block_packed_bytes(rows, k), dtype=torch.uint8, device=self.device)
        scale = torch.empty((-(-k // 128), -(-rows // 16) * 16), dtype=torch.float32, device=self.device)
        B.moe_block_quantize(x, self._in, x.stride(0), rows, k, q, scale, _raw_stream(self.device.index))
        return BlockCodes(q, scale, rows, (rows, k))

    def __call__(self, x: Optional[torch.Tensor] = None, *, codes: Optional[BlockCodes] = None,
                 stream=None) -> torch.Tensor:
        """x [rows, in_features], or its codes of :meth:`quantize`, -> [rows, out_features]."""
        k, dev = self.in_features, self.device
        if codes is None:
            if x is None:
                raise ValueError("x or its codes are needed")
            self._check(x)
            rows = x.shape[0]
        else:
            if x is not None:
                raise ValueError("x and its codes exclude each other")
            rows = codes.rows
            # (the tensors, filled up to whole blocks, do not tell one width from another)
            if tuple(codes.shape) != (rows, k):
                raise ValueError("codes of %s are not those of [%d, %d]" % (list(codes.shape), rows, k))
            want = (-(-k // 128), -(-rows // 16) * 16)
            for t, shape, kind in ((codes.q, (want[0] * want[1] * 128,), torch.uint8),
                                   (codes.scale, want, torch.float32)):
                if tuple(t.shape) != shape or t.dtype != kind or not t.is_contiguous() or t.device != dev:
                    raise ValueError("codes must be those of [rows, %d] on %s" % (k, dev))
        other = _elsewhere(dev.index, stream)
        if other is not None:
            with other:
                return self(x, codes=codes)
        n = self.out_features
        out = torch.empty_strided((rows, n), (n, 1), dtype=self.out_dtype, device=dev)
        xp = xs = qp = sp = wp = 0
        if codes is not None:
            qp, sp = codes.q.data_ptr(), codes.scale.data_ptr()
        else:
            xp, xs = x.data_ptr(), x.stride(0)
        size, ws = self._bytes(rows, n, k, codes is not None), None
        if size:
            ws = torch.empty_strided((size,), (1,), dtype=torch.uint8, device=dev)
            wp = ws.data_ptr()
        rc = self._call(self._w, self._ws, n, k, xp, self._in, xs, qp, sp, rows, out.data_ptr(), self._out, wp, size,
                        _raw_stream(dev.index))
        if rc:
            B._check(rc)
        return out


class TokenLogprobs(NamedTuple):
    logprob: torch.Tensor                  # [rows] float32
    entropy: torch.Tensor                  # [rows] float32
    top_logprob: Optional[torch.Tensor]    # [rows, top] float32, best first (None without alternatives)
    top_token: Optional[torch.Tensor]      # [rows, top] int32


def token_logprobs(logits: torch.Tensor, tokens: torch.Tensor, top: int = 0, *, stream=None) -> TokenLogprobs:
    """Log probabilities of tokens [rows] (int32 or int64) under logits [rows, vocab]
    (float32 or bfloat16, rows contiguous inside), the entropy of each row, and the
    `top` (up to 64) best tokens, equal logits by their index.

    Masked logits are -inf: no part of the distribution, log probability -inf, as a
    token outside the vocabulary; a row of nothing else has the entropy 0.  A row with a
    NaN or +inf gives NaN."""
    if logits.dim() != 2 or logits.dtype not in _ACT:
        raise ValueError("logits must be [rows, vocab] of float32 or bfloat16, got %s of %s"
                         % (list(logits.shape), logits.dtype))
    rows, vocab = logits.shape
    dev = _device(logits)
    if vocab == 0 or max(rows, vocab) > _INT32:
        raise ValueError("rows must be below 2^31, the vocabulary from 1 to 2^31 - 1")
    if logits.stride(1) != 1 and vocab != 1:
        raise ValueError("rows must be contiguous")
    if tokens.shape != (rows,) or tokens.dtype not in (torch.int32, torch.int64) or not tokens.is_contiguous() \
            or tokens.device != dev:
        raise ValueError("tokens must be contiguous int32 or int64 [%d] on %s, got %s of %s on %s"
                         % (rows, dev, list(tokens.shape), tokens.dtype, tokens.device))
    if not 0 <= top <= min(vocab, 64):
        raise ValueError("top must be from 0 to %d, got %d" % (min(vocab, 64), top))
    other = _elsewhere(dev.index, stream)
    if other is not None:
        with other:
            return token_logprobs(logits, tokens, top)
    new = torch.empty_strided
    logprob, entropy = new((2, rows), (rows, 1), dtype=torch.float32, device=dev).unbind()
    values = ids = None
    vp = ip = 0
    if top:
        values = new((rows, top), (top, 1), dtype=torch.float32, device=dev)
        ids = new((rows, top), (top, 1), dtype=torch.int32, device=dev)
        vp, ip = values.data_ptr(), ids.data_ptr()
    rc = B.lib().moe_token_logprobs(logits.data_ptr(), _ACT[logits.dtype], logits.stride(0), tokens.data_ptr(),
                                    tokens.element_size(), rows, vocab, top, logprob.data_ptr(), entropy.data_ptr(),
                                    vp, ip, _raw_stream(dev.index))
    if rc:
        B._check(rc)
    return TokenLogprobs(logprob, entropy, values, ids)
