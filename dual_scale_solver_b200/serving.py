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

What a call allocates belongs to the stream that it runs on (memory that an
earlier call on another stream still uses is not handed to it), and results
may also be used and dropped on the stream that is current at the call.  With
an explicit ``stream`` the caller orders that stream behind the work that
makes the inputs, and its reads of the results behind that stream.
"""
from __future__ import annotations

import ctypes
import functools
import math
import struct
from ctypes import byref, c_float, c_int32, c_int64, c_size_t, c_void_p

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


# The same two structures as bytes: packing them takes a third of the time of
# filling a ctypes.Structure, and a call's Python side is what a small call
# costs (a single token's kernels run for 2 to 10 us).
_pack_cache = struct.Struct("PPPPqiii4x").pack
_pack_batch = struct.Struct("PPPiiq").pack
assert struct.calcsize("PPPPqiii4x") == ctypes.sizeof(dq_kv_cache)
assert struct.calcsize("PPPiiq") == ctypes.sizeof(dq_kv_batch)

_bf16 = torch.bfloat16
_new = torch.empty_strided            # (half the time of torch.empty)
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


def _check(status, where):
    from . import DqError
    raise DqError(status, where)


def _device(tensors):
    """Index of the one CUDA device of the tensors (None skipped)."""
    d = tensors[0].get_device()
    if d < 0:
        raise ValueError("tensors must be CUDA tensors")
    for t in tensors:
        if t is not None and t.get_device() != d:
            raise ValueError("tensors must be on one CUDA device")
    return d


def _fresh(shape, strides, dtype, device, stream):
    """A tensor for a call on ``stream``, from that stream's pool: the current
    stream's may hand out memory that its pending kernels still use, which
    ``stream`` does not wait for."""
    current = None if stream is None else torch.cuda.current_stream(device)
    if stream == current:
        return _new(shape, strides, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = _new(shape, strides, dtype=dtype, device=device)
    t.record_stream(current)
    return t


def _call(device, stream, fn, *args):
    """fn(*args, stream) with the tensors' device current; the stream defaults
    to that device's current one."""
    back = torch._C._cuda_getDevice()
    if back == device:
        return fn(*args, torch._C._cuda_getCurrentRawStream(device) if stream is None
                  else stream.cuda_stream)
    with torch.cuda.device(device):
        return fn(*args, torch._C._cuda_getCurrentRawStream(device) if stream is None
                  else stream.cuda_stream)


def _rows(t, name):
    """(shape, element strides of the leading dimensions) of a bf16 array
    whose last dimension is contiguous; a dimension of one element takes the
    stride of a contiguous tensor (torch leaves it arbitrary)."""
    if t.dtype is not _bf16:
        raise TypeError(f"{name} is bfloat16")
    shape, st = t.shape, t.stride()
    if len(shape) == 2:
        if st[1] == 1 or shape[1] <= 1:
            return shape, (st[0] if shape[0] > 1 else shape[1],)
    elif len(shape) == 3 and (st[2] == 1 or shape[2] <= 1):
        head = st[1] if shape[1] > 1 else shape[2]
        return shape, (st[0] if shape[0] > 1 else max(head * shape[1], shape[2]), head)
    raise ValueError(f"{name}: the last dimension is contiguous")


def add_rmsnorm_quant(x, weight, fmt, residual=None, b=None, eps=1e-5, codes=None, gscales=None,
                      residual_out=None, stream=None):
    """Q(((x + residual) / rms) * weight * b) per row: returns (codes [tokens,
    K*bits/8] uint8, group scales [tokens, K/G], residual_out bf16 [tokens, K]
    or None).

    x, residual: bf16 [tokens, K], rows may be strided.  The sum x + residual
    is written to ``residual_out`` (allocated when a residual is given and
    none is passed; pass ``residual`` itself to update it in place) rounded
    to bf16; the norm uses the unrounded float32 sum.  weight: [K] float32 or
    bf16; b: [K] float32 (the solver's inverse column scales) or None.  codes,
    gscales: buffers of exactly those sizes to write, or None."""
    dev = _device((x, weight, residual, b, codes, gscales, residual_out))
    (tokens, K), (xs,) = _rows(x, "x")
    if weight.shape != (K,) or not weight.is_contiguous():
        raise ValueError("weight: [K], contiguous")
    wd = weight.dtype
    if wd is not _bf16 and wd is not torch.float32:
        raise TypeError("weight is float32 or bfloat16")
    if b is not None and (b.dtype is not torch.float32 or b.shape != (K,) or not b.is_contiguous()):
        raise ValueError("b: float32 [K], contiguous")
    rp = op = None
    rs = os = 0
    if residual is not None:
        shape, (rs,) = _rows(residual, "residual")
        if shape != (tokens, K):
            raise ValueError("residual: the shape of x")
        rp = residual.data_ptr()
        if residual_out is None:
            residual_out = _fresh((tokens, K), (K, 1), _bf16, x.device, stream)
    if residual_out is not None:
        shape, (os,) = _rows(residual_out, "residual_out")
        if shape != (tokens, K):
            raise ValueError("residual_out: the shape of x")
        op = residual_out.data_ptr()
    codes, gscales = _outputs(tokens, K, fmt, x.device, codes, gscales, stream)
    status = _call(dev, stream, _lib().dq_add_rmsnorm_quant, x.data_ptr(), xs, rp, rs,
                   weight.data_ptr(), 1 if wd is _bf16 else 0, None if b is None else b.data_ptr(), eps,
                   tokens, K, byref(fmt), op, os, codes.data_ptr(), gscales.data_ptr())
    if status:
        _check(status, "dq_add_rmsnorm_quant")
    return codes, gscales, residual_out


_BITS = (4, 4, 8, 8, 8, 6, 6)           # of a code, by DQ_CODES_*


def _outputs(tokens, K, fmt, device, codes, gscales, stream):
    """codes and gscales, allocated where not given, of exactly the format's
    size where given (the library sees addresses only)."""
    if not 0 <= fmt.codes < 7 or fmt.group <= 0 or K % fmt.group:
        from . import DqError
        raise DqError(-2 if 0 <= fmt.codes < 7 and fmt.group > 0 else -3, "dq_add_rmsnorm_quant")
    n, size = K * _BITS[fmt.codes] // 8, 2 if fmt.group_scale == 0 else 1
    if codes is None:
        codes = _fresh((tokens, n), (n, 1), torch.uint8, device, stream)
    elif codes.nbytes != tokens * n or not codes.is_contiguous():
        raise ValueError(f"codes: {tokens} x {n} bytes, contiguous")
    n = K // fmt.group
    if gscales is None:
        gscales = _fresh((tokens, n), (n, 1), torch.int16 if size == 2 else torch.uint8, device, stream)
    elif gscales.numel() != tokens * n or gscales.element_size() != size or not gscales.is_contiguous():
        raise ValueError(f"gscales: {tokens} x {n} of {8 * size} bits, contiguous")
    return codes, gscales


def kv_cache(pages, page_size, heads, head_dim, fmt, device="cuda"):
    """An empty cache: (k_codes, k_scales, v_codes, v_scales), zeroed."""
    from . import gscale_dtype
    one = lambda n, dt: torch.zeros(pages, heads, page_size, n, dtype=dt, device=device)  # noqa: E731
    c, s = head_dim // 2, head_dim // fmt.group
    return (one(c, torch.uint8), one(s, gscale_dtype(fmt)), one(c, torch.uint8),
            one(s, gscale_dtype(fmt)))


def _cache(cache, fmt):
    """(packed structure, heads, head_dim) of a cache."""
    kc, ks, vc, vs = cache
    shape = kc.shape
    pages, heads, page_size, half = shape
    if vc.shape != shape or kc.dtype is not torch.uint8 or vc.dtype is not torch.uint8:
        raise ValueError("cache codes: uint8 [pages, heads, page_size, head_dim / 2]")
    want = (pages, heads, page_size, 2 * half // max(fmt.group, 1))
    size = 2 if fmt.group_scale == 0 else 1
    if ks.shape != want or vs.shape != want or ks.element_size() != size or vs.element_size() != size:
        raise ValueError(f"cache scales: {list(want)} of {8 * size} bits")
    if not (kc.is_contiguous() and ks.is_contiguous() and vc.is_contiguous() and vs.is_contiguous()):
        raise ValueError("cache tensors: contiguous")
    return (_pack_cache(kc.data_ptr(), ks.data_ptr(), vc.data_ptr(), vs.data_ptr(), pages, page_size,
                        heads, 2 * half), heads, 2 * half)


_i32 = torch.int32


def _batch(starts, kv_lens, block_table):
    """(packed structure, sequences) of a batch."""
    ns, nl, nt = starts.shape, kv_lens.shape, block_table.shape
    if len(nl) != 1 or len(ns) != 1 or len(nt) != 2 or ns[0] != nl[0] + 1 or nt[0] != nl[0]:
        raise ValueError("starts [seqs + 1], kv_lens [seqs], block_table [seqs, pages]")
    if starts.dtype is not _i32 or kv_lens.dtype is not _i32 or block_table.dtype is not _i32:
        raise TypeError("starts, kv_lens and block_table are int32")
    seqs, cols = nt
    st = block_table.stride()
    if not (starts.is_contiguous() and kv_lens.is_contiguous()) or (cols > 1 and st[1] != 1):
        raise ValueError("starts, kv_lens and the rows of block_table: contiguous")
    return (_pack_batch(starts.data_ptr(), kv_lens.data_ptr(), block_table.data_ptr(), seqs, cols,
                        cols if seqs <= 1 else st[0]), seqs)


def _copy(fn, name, k, v, cache, starts, kv_lens, block_table, fmt, stream):
    c, heads, dim = _cache(cache, fmt)
    b, _ = _batch(starts, kv_lens, block_table)
    ks, (kt, kh) = _rows(k, "k")
    vs, (vt, vh) = _rows(v, "v")
    if len(ks) != 3 or vs != ks or ks[1] != heads or ks[2] != dim:
        raise ValueError("k and v: [tokens, heads, head_dim] of the cache")
    dev = _device((k, v, *cache, starts, kv_lens, block_table))
    status = _call(dev, stream, fn, k.data_ptr(), kt, kh, v.data_ptr(), vt, vh, ks[0], c, b, byref(fmt))
    if status:
        _check(status, name)


def kv_append(k, v, cache, starts, kv_lens, block_table, fmt, stream=None):
    """Quantize the new keys and values (bf16 [tokens, heads, head_dim], may be
    strided) and write them to their places in the cache."""
    _copy(_lib().dq_kv_append, "dq_kv_append", k, v, cache, starts, kv_lens, block_table, fmt, stream)


def kv_read(cache, starts, kv_lens, block_table, fmt, tokens, k=None, v=None, stream=None):
    """The values the cache holds for the batch's new tokens: (k, v) bf16
    [tokens, heads, head_dim].  Rows that belong to no sequence are left as
    they are (undefined in tensors allocated here)."""
    _, heads, _, half = cache[0].shape
    if k is None:
        k = _fresh((tokens, heads, 2 * half), (2 * heads * half, 2 * half, 1), _bf16, cache[0].device,
                   stream)
    if v is None:
        v = _fresh((tokens, heads, 2 * half), (2 * heads * half, 2 * half, 1), _bf16, cache[0].device,
                   stream)
    if k.shape[0] != tokens:
        raise ValueError("k: [tokens, heads, head_dim]")
    _copy(_lib().dq_kv_read, "dq_kv_read", k, v, cache, starts, kv_lens, block_table, fmt, stream)
    return k, v


@functools.lru_cache(maxsize=1024)
def kv_attention_workspace(tokens, q_heads, heads, head_dim, seqs) -> int:
    """Bytes of workspace ``kv_attention`` needs."""
    out = c_size_t(0)
    status = _lib().dq_kv_attention_workspace(tokens, q_heads, heads, head_dim, seqs, byref(out))
    if status:
        _check(status, "dq_kv_attention_workspace")
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
    c, heads, dim = _cache(cache, fmt)
    b, seqs = _batch(starts, kv_lens, block_table)
    shape, (qt, qh) = _rows(q, "q")
    if len(shape) != 3 or shape[2] != dim:
        raise ValueError("q: [tokens, q_heads, head_dim] of the cache")
    dev = _device((q, *cache, starts, kv_lens, block_table, out, ws))
    tokens, q_heads, _ = shape
    if out is None:
        ot, oh = q_heads * dim, dim
        out = _fresh(shape, (ot, oh, 1), _bf16, q.device, stream)
    else:
        so, (ot, oh) = _rows(out, "out")
        if so != shape:
            raise ValueError("out: the shape of q")
    if ws is None:
        ws = _fresh((kv_attention_workspace(tokens, q_heads, heads, dim, seqs),), (1,), torch.uint8, q.device,
                    stream)
    status = _call(dev, stream, _lib().dq_kv_attention, q.data_ptr(), qt, qh, out.data_ptr(), ot, oh,
                   tokens, q_heads, 1.0 / math.sqrt(dim) if scale is None else scale, 1 if causal else 0,
                   c, b, byref(fmt), ws.data_ptr(), ws.nbytes)
    if status:
        _check(status, "dq_kv_attention")
    return out
