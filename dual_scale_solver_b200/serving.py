"""Binding of the serving operators (``include/dq_serving.h``): the residual +
root-mean-square norm that feeds an activation quantizer, the paged 4-bit
key/value cache, and attention over it.

Argument marshalling only, as in the rest of the package: every step runs in
the CUDA kernels of ``libdq.so``, tensors supply device memory, calls are
ordered on ``stream`` (default: the current stream of the tensors' device).
A cache is the tuple (k_codes, k_scales, v_codes, v_scales); a batch is
(starts, kv_lens, block_table), int32 device tensors: sequence s owns the
token rows starts[s] .. starts[s+1] - 1, its last new ones, at the end of
kv_lens[s] positions, position p of it in page block_table[s, p // page_size].
"""
from __future__ import annotations

import ctypes
import math
from ctypes import c_float, c_int32, c_int64, c_size_t, c_void_p

import torch

__all__ = ["add_rmsnorm_quant", "kv_cache", "kv_append", "kv_read", "kv_attention",
           "kv_attention_workspace", "SERVING_EXPORTS"]

SERVING_EXPORTS = ("dq_add_rmsnorm_quant", "dq_kv_append", "dq_kv_read", "dq_kv_attention",
                   "dq_kv_attention_workspace")


class dq_kv_cache(ctypes.Structure):
    _fields_ = [("k_codes", c_void_p), ("k_scales", c_void_p), ("v_codes", c_void_p),
                ("v_scales", c_void_p), ("pages", c_int64), ("page_size", c_int32),
                ("heads", c_int32), ("head_dim", c_int32)]


class dq_kv_batch(ctypes.Structure):
    _fields_ = [("starts", c_void_p), ("kv_lens", c_void_p), ("block_table", c_void_p),
                ("seqs", c_int32), ("max_pages", c_int32), ("table_stride", c_int64)]


_fns = None


def _lib():
    global _fns
    if _fns is None:
        from . import lib
        L = lib()
        P, i32, i64 = c_void_p, c_int32, c_int64
        sig = {
            "dq_add_rmsnorm_quant": [P, i64, P, i64, P, i32, P, c_float, i64, i64, P, P, i64, P, P, P],
            "dq_kv_append": [P, i64, i64, P, i64, i64, i64, P, P, P, P],
            "dq_kv_read": [P, i64, i64, P, i64, i64, i64, P, P, P, P],
            "dq_kv_attention_workspace": [i64, i32, i32, i32, i32, P],
            "dq_kv_attention": [P, i64, i64, P, i64, i64, i64, i32, c_float, i32, P, P, P, P, c_size_t, P],
        }
        for name, args in sig.items():
            f = getattr(L, name)
            f.restype, f.argtypes = c_int32, args
        _fns = L
    return _fns


class _On:
    """Device and stream of a call: the tensors' device is made current for
    the launch, and the stream defaults to that device's current one."""

    def __init__(self, device, stream):
        self.index = device.index
        self.stream = stream
        self.back = None

    def __enter__(self):
        if self.index != torch.cuda.current_device():
            self.back = torch.cuda.current_device()
            torch.cuda.set_device(self.index)
        s = self.stream
        return (torch.cuda.current_stream() if s is None else s).cuda_stream

    def __exit__(self, *exc):
        if self.back is not None:
            torch.cuda.set_device(self.back)


def _check(status, where):
    if status != 0:
        from . import DqError
        raise DqError(status, where)


def _device(first, *others):
    """The one CUDA device of the tensors (None skipped)."""
    if not first.is_cuda:
        raise ValueError("tensors must be CUDA tensors")
    d = first.device
    for t in others:
        if t is not None and t.device != d:
            raise ValueError("tensors must be on one CUDA device")
    return d


def _bf16(t, name, dims):
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} is bfloat16")
    if t.dim() != dims or (t.shape[-1] > 1 and t.stride(-1) != 1):
        raise ValueError(f"{name}: {dims} dimensions, the last one contiguous")
    return t


def _strides(t):
    """Element strides of the leading dimensions; a dimension of one element
    takes the stride of a contiguous tensor (torch leaves it arbitrary)."""
    out = []
    inner = t.shape[-1]
    for i in range(t.dim() - 2, -1, -1):
        out.append(inner if t.shape[i] <= 1 else t.stride(i))
        inner *= max(t.shape[i], 1)
    return out[::-1]


def add_rmsnorm_quant(x, weight, fmt, residual=None, b=None, eps=1e-5, codes=None, gscales=None,
                      residual_out=None, stream=None):
    """Q(((x + residual) / rms) * weight * b) per row: returns (codes [tokens,
    K*bits/8] uint8, group scales [tokens, K/G], residual_out bf16 [tokens, K]
    or None).

    x, residual: bf16 [tokens, K], rows may be strided.  The sum x + residual
    is written to ``residual_out`` (allocated when a residual is given and
    none is passed; pass ``residual`` itself to update it in place) rounded
    to bf16; the norm uses the unrounded float32 sum.  weight: [K] float32 or
    bf16; b: [K] float32 (the solver's inverse column scales) or None."""
    from . import _dtype_code, _outputs
    dev = _device(x, weight, residual, b, codes, gscales, residual_out)
    _bf16(x, "x", 2)
    tokens, K = x.shape
    if weight.shape != (K,) or not weight.is_contiguous():
        raise ValueError("weight: [K], contiguous")
    if b is not None and (b.dtype != torch.float32 or b.shape != (K,) or not b.is_contiguous()):
        raise ValueError("b: float32 [K], contiguous")
    if residual is not None and _bf16(residual, "residual", 2).shape != x.shape:
        raise ValueError("residual: the shape of x")
    if residual is not None and residual_out is None:
        residual_out = torch.empty(tokens, K, dtype=torch.bfloat16, device=dev)
    if residual_out is not None and _bf16(residual_out, "residual_out", 2).shape != x.shape:
        raise ValueError("residual_out: the shape of x")
    if codes is None or gscales is None:
        codes, gscales = _outputs(tokens, K, fmt, dev, codes, gscales)
    for t, name in ((codes, "codes"), (gscales, "gscales")):
        if not t.is_contiguous():
            raise ValueError(f"{name}: contiguous")
    res, ro = residual, residual_out
    with _On(dev, stream) as st:
        _check(_lib().dq_add_rmsnorm_quant(
            x.data_ptr(), _strides(x)[0], None if res is None else res.data_ptr(),
            0 if res is None else _strides(res)[0], weight.data_ptr(), _dtype_code(weight),
            None if b is None else b.data_ptr(), eps, tokens, K, ctypes.byref(fmt),
            None if ro is None else ro.data_ptr(), 0 if ro is None else _strides(ro)[0],
            codes.data_ptr(), gscales.data_ptr(), st), "dq_add_rmsnorm_quant")
    return codes, gscales, residual_out


def kv_cache(pages, page_size, heads, head_dim, fmt, device="cuda"):
    """An empty cache: (k_codes, k_scales, v_codes, v_scales), zeroed."""
    from . import gscale_dtype
    one = lambda n, dt: torch.zeros(pages, heads, page_size, n, dtype=dt, device=device)  # noqa: E731
    c, s = head_dim // 2, head_dim // fmt.group
    return (one(c, torch.uint8), one(s, gscale_dtype(fmt)), one(c, torch.uint8),
            one(s, gscale_dtype(fmt)))


def _cache(cache, fmt):
    kc, ks, vc, vs = cache
    pages, heads, page_size, half = kc.shape
    if vc.shape != kc.shape or kc.dtype != torch.uint8 or vc.dtype != torch.uint8:
        raise ValueError("cache codes: uint8 [pages, heads, page_size, head_dim / 2]")
    want = (pages, heads, page_size, 2 * half // max(fmt.group, 1))
    bits = 2 if fmt.group_scale == 0 else 1
    for s in (ks, vs):
        if tuple(s.shape) != want or s.element_size() != bits:
            raise ValueError(f"cache scales: {list(want)} of {8 * bits} bits")
    for t in cache:
        if not t.is_contiguous():
            raise ValueError("cache tensors: contiguous")
    return dq_kv_cache(kc.data_ptr(), ks.data_ptr(), vc.data_ptr(), vs.data_ptr(), pages, page_size,
                       heads, 2 * half)


def _batch(starts, kv_lens, block_table):
    seqs = kv_lens.shape[0]
    if starts.dim() != 1 or starts.shape[0] != seqs + 1 or kv_lens.dim() != 1 or \
            block_table.dim() != 2 or block_table.shape[0] != seqs:
        raise ValueError("starts [seqs + 1], kv_lens [seqs], block_table [seqs, pages]")
    for t in (starts, kv_lens, block_table):
        if t.dtype != torch.int32:
            raise TypeError("starts, kv_lens and block_table are int32")
    if not starts.is_contiguous() or not kv_lens.is_contiguous() or \
            (block_table.shape[1] > 1 and block_table.stride(1) != 1):
        raise ValueError("starts, kv_lens and the rows of block_table: contiguous")
    cols = block_table.shape[1]
    return dq_kv_batch(starts.data_ptr(), kv_lens.data_ptr(), block_table.data_ptr(), seqs, cols,
                       cols if seqs <= 1 else block_table.stride(0))


def _copy(fn, name, k, v, cache, starts, kv_lens, block_table, fmt, stream):
    c, b = _cache(cache, fmt), _batch(starts, kv_lens, block_table)
    for t, what in ((k, "k"), (v, "v")):
        if _bf16(t, what, 3).shape[1:] != (c.heads, c.head_dim) or t.shape[0] != k.shape[0]:
            raise ValueError(f"{what}: [tokens, heads, head_dim] of the cache")
    dev = _device(k, v, *cache, starts, kv_lens, block_table)
    kt, kh = _strides(k)
    vt, vh = _strides(v)
    with _On(dev, stream) as st:
        _check(fn(k.data_ptr(), kt, kh, v.data_ptr(), vt, vh, k.shape[0], ctypes.addressof(c),
                  ctypes.addressof(b), ctypes.byref(fmt), st), name)


def kv_append(k, v, cache, starts, kv_lens, block_table, fmt, stream=None):
    """Quantize the new keys and values (bf16 [tokens, heads, head_dim], may be
    strided) and write them to their places in the cache."""
    _copy(_lib().dq_kv_append, "dq_kv_append", k, v, cache, starts, kv_lens, block_table, fmt, stream)


def kv_read(cache, starts, kv_lens, block_table, fmt, tokens, k=None, v=None, stream=None):
    """The values the cache holds for the batch's new tokens: (k, v) bf16
    [tokens, heads, head_dim].  Rows that belong to no sequence are left as
    they are (undefined in tensors allocated here)."""
    pages, heads, page_size, half = cache[0].shape
    dev = cache[0].device
    if k is None:
        k = torch.empty(tokens, heads, 2 * half, dtype=torch.bfloat16, device=dev)
    if v is None:
        v = torch.empty(tokens, heads, 2 * half, dtype=torch.bfloat16, device=dev)
    if k.shape[0] != tokens:
        raise ValueError("k: [tokens, heads, head_dim]")
    _copy(_lib().dq_kv_read, "dq_kv_read", k, v, cache, starts, kv_lens, block_table, fmt, stream)
    return k, v


def kv_attention_workspace(tokens, q_heads, heads, head_dim, seqs) -> int:
    """Bytes of workspace ``kv_attention`` needs."""
    out = c_size_t(0)
    _check(_lib().dq_kv_attention_workspace(tokens, q_heads, heads, head_dim, seqs,
                                            ctypes.addressof(out)), "dq_kv_attention_workspace")
    return out.value


def kv_attention(q, cache, starts, kv_lens, block_table, fmt, scale=None, causal=True, out=None,
                 ws=None, stream=None):
    """softmax(scale q k^T) v of the new tokens' queries q (bf16 [tokens,
    q_heads, head_dim], may be strided) over the cache, which already holds
    their keys and values; returns bf16 [tokens, q_heads, head_dim].

    scale: 1 / sqrt(head_dim) when None.  causal: a token sees the positions
    up to its own; otherwise all of its sequence's.  Rows that see nothing
    are zeros; rows that belong to no sequence are left as they are (undefined
    in a tensor allocated here).  ws: a uint8 tensor of
    ``kv_attention_workspace`` bytes (allocated when None); calls that may
    overlap on the device need one each."""
    c, b = _cache(cache, fmt), _batch(starts, kv_lens, block_table)
    if _bf16(q, "q", 3).shape[2] != c.head_dim:
        raise ValueError("q: [tokens, q_heads, head_dim] of the cache")
    dev = _device(q, *cache, starts, kv_lens, block_table, out, ws)
    tokens, q_heads, dim = q.shape
    with _On(dev, stream) as st:
        if out is None:
            out = torch.empty(tokens, q_heads, dim, dtype=torch.bfloat16, device=dev)
        elif _bf16(out, "out", 3).shape != q.shape:
            raise ValueError("out: the shape of q")
        if ws is None:
            ws = torch.empty(kv_attention_workspace(tokens, q_heads, c.heads, dim, b.seqs),
                             dtype=torch.uint8, device=dev)
            if stream is not None:
                ws.record_stream(stream)
        qt, qh = _strides(q)
        ot, oh = _strides(out)
        _check(_lib().dq_kv_attention(
            q.data_ptr(), qt, qh, out.data_ptr(), ot, oh, tokens, q_heads,
            1.0 / math.sqrt(dim) if scale is None else scale, 1 if causal else 0,
            ctypes.addressof(c), ctypes.addressof(b), ctypes.byref(fmt), ws.data_ptr(), ws.numel(),
            st), "dq_kv_attention")
    return out
