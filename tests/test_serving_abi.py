"""The serving operators' C ABI (include/dq_serving.h): exports, and arguments
refused on the host before anything is launched (no GPU)."""
import ctypes
import os
import re

import pytest
import torch

import dual_scale_solver_b200 as dq
from dual_scale_solver_b200 import serving

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = ctypes.c_void_p(4096)                   # aligned, never dereferenced
ODD = ctypes.c_void_p(4096 + 8)


@pytest.fixture(scope="module", autouse=True)
def built():
    from dual_scale_solver_b200 import build
    build.build()


def test_exports_match_header():
    src = open(os.path.join(ROOT, "include", "dq_serving.h")).read()
    names = sorted(set(re.findall(r"^DQ_API\s+[^(]*?\b(dq_\w+)\s*\(", src, flags=re.M)))
    assert names == sorted(dq.SERVING_EXPORTS)
    for n in names:
        assert hasattr(dq.lib(), n), n
    for n in serving.__all__:
        assert hasattr(dq, n), n
    assert dq.lib().dq_strerror(-12).decode().startswith("a sequence start")


def _norm(fmt="mxfp8_e4m3", G=0, x=P, xs=64, res=None, rs=64, w=P, wd=1, b=None, eps=1e-5, tokens=4,
          K=64, ro=None, ros=64, codes=P, gs=P):
    f = dq.format_preset(fmt, G) if isinstance(fmt, str) else fmt
    return serving._lib().dq_add_rmsnorm_quant(x, xs, res, rs, w, wd, b, eps, tokens, K, ctypes.byref(f),
                                               ro, ros, codes, gs, None)


def test_norm_refusals():
    assert _norm(tokens=0) == 0 and _norm(K=0, xs=0) == 0          # empty
    assert _norm(fmt=dq.dq_format(2, 32, 0, 0, 0)) == -3
    assert _norm(K=48) == -2 and _norm(K=-32) == -2 and _norm(tokens=-1) == -2
    assert _norm(tokens=1 << 31) == -2
    assert _norm(K=1 << 29) == -2
    assert _norm(x=None) == -1 and _norm(w=None) == -1 and _norm(codes=None) == -1 and _norm(gs=None) == -1
    assert _norm(wd=2) == -1
    for eps in (0.0, -1.0, float("nan"), float("inf")):
        assert _norm(eps=eps) == -1
    assert _norm(xs=56) == -2 and _norm(xs=68) == -2               # below K; not a multiple of 8
    assert _norm(res=P, rs=32) == -2 and _norm(ro=P, ros=65) == -2
    assert _norm(res=P, rs=64, ro=P, ros=72) == -2                 # in place with another stride
    assert _norm(ro=P, ros=72) == -2
    for kw in ("x", "res", "w", "b", "ro", "codes", "gs"):
        assert _norm(**{kw: ODD}) == -9, kw


def _cache(**kw):
    a = dict(k_codes=4096, k_scales=4096, v_codes=4096, v_scales=4096, pages=8, page_size=16, heads=2,
             head_dim=128)
    a.update(kw)
    return serving.dq_kv_cache(**a)


def _batch(**kw):
    a = dict(starts=4096, kv_lens=4096, block_table=4096, seqs=2, max_pages=4, table_stride=4)
    a.update(kw)
    return serving.dq_kv_batch(**a)


def _copy(which, fmt="mxfp4", G=0, k=P, kt=256, kh=128, v=P, vt=256, vh=128, tokens=3, cache=None,
          batch=None):
    f = dq.format_preset(fmt, G)
    c, b = cache or _cache(), batch or _batch()
    return getattr(serving._lib(), which)(k, kt, kh, v, vt, vh, tokens, ctypes.addressof(c),
                                          ctypes.addressof(b), ctypes.byref(f), None)


BAD_PLACES = [
    (dict(cache=_cache(head_dim=96)), -2), (dict(cache=_cache(head_dim=256)), -2),
    (dict(cache=_cache(page_size=24)), -2), (dict(cache=_cache(page_size=0)), -2),
    (dict(cache=_cache(heads=0)), -2), (dict(cache=_cache(pages=-1)), -2),
    (dict(cache=_cache(pages=1 << 31)), -2), (dict(cache=_cache(v_scales=None)), -1),
    (dict(cache=_cache(k_codes=4104)), -9), (dict(cache=_cache(k_scales=4100)), -9),
    (dict(batch=_batch(seqs=-1)), -2), (dict(batch=_batch(max_pages=-1)), -2),
    (dict(batch=_batch(table_stride=3)), -2), (dict(batch=_batch(starts=None)), -1),
    (dict(batch=_batch(kv_lens=None)), -1), (dict(batch=_batch(block_table=None)), -1),
    (dict(batch=_batch(starts=4098)), -9),
    (dict(batch=_batch(max_pages=1 << 28, table_stride=1 << 28)), -2),   # positions past 32 bits
    (dict(batch=_batch(max_pages=(1 << 27) - 255, table_stride=1 << 28)), -2),
]


@pytest.mark.parametrize("which", ["dq_kv_append", "dq_kv_read"])
def test_cache_copy_refusals(which):
    assert _copy(which, tokens=0) == 0 and _copy(which, batch=_batch(seqs=0)) == 0
    assert _copy(which, fmt="mxint8") == -3 and _copy(which, fmt="mxfp6_e2m3") == -3
    assert _copy(which, tokens=-1) == -2
    assert _copy(which, k=None) == -1 and _copy(which, v=None) == -1
    assert _copy(which, k=ODD) == -9 and _copy(which, v=ODD) == -9
    assert _copy(which, kt=-256) == -2 and _copy(which, vh=132) == -2
    for kw, status in BAD_PLACES:
        assert _copy(which, **kw) == status, kw
    # rows that are written may not overlap; rows that are read may
    if which == "dq_kv_read":
        assert _copy(which) == -1                                  # both over each other
        assert _copy(which, kt=128) == -2 and _copy(which, kh=64) == -2 and _copy(which, vt=0) == -2


def _attend(fmt="mxfp4", G=0, q=P, qt=512, qh=128, out=P, ot=512, oh=128, tokens=3, q_heads=4, scale=0.1,
            causal=1, cache=None, batch=None, ws=P, bytes_=1 << 30):
    f = dq.format_preset(fmt, G)
    c, b = cache or _cache(), batch or _batch()
    return serving._lib().dq_kv_attention(q, qt, qh, out, ot, oh, tokens, q_heads, scale, causal,
                                          ctypes.addressof(c), ctypes.addressof(b), ctypes.byref(f), ws,
                                          bytes_, None)


def test_attention_refusals():
    assert _attend(tokens=0) == 0 and _attend(batch=_batch(seqs=0)) == 0
    assert _attend(fmt="mxfp8_e4m3") == -3
    assert _attend(q_heads=3) == -2 and _attend(q_heads=0) == -2   # not a multiple of the cache's heads
    for s in (0.0, -1.0, float("nan"), float("inf")):
        assert _attend(scale=s) == -1
    assert _attend(causal=2) == -1
    assert _attend(q=None) == -1 and _attend(out=None) == -1
    assert _attend(q=ODD) == -9 and _attend(out=ODD) == -9
    assert _attend() == -1                                         # out over q
    assert _attend(ot=256) == -2 and _attend(oh=0) == -2 and _attend(qh=12) == -2
    assert _attend(ws=None) == -7 and _attend(bytes_=1024) == -7
    assert _attend(ws=ctypes.c_void_p(4096 + 16)) == -9
    assert _attend(tokens=1 << 30, q_heads=128, ot=1 << 14) == -2  # rows past 32 bits
    for kw, status in BAD_PLACES:
        assert _attend(**kw) == status, kw
    most = _batch(max_pages=(1 << 27) - 256, table_stride=1 << 28)  # 2^31 - 4096 positions
    assert _attend(batch=most, ws=None) == -7


def test_attention_workspace():
    n = dq.kv_attention_workspace(64, 32, 8, 128, 64)
    assert 0 < n < 64 << 20
    for bad in ((-1, 32, 8, 128, 4), (4, 30, 8, 128, 4), (4, 32, 0, 128, 4), (4, 32, 8, 80, 4),
                (4, 32, 8, 128, -1)):
        with pytest.raises(dq.DqError) as e:
            dq.kv_attention_workspace(*bad)
        assert e.value.status == -2
    assert serving._lib().dq_kv_attention_workspace(4, 8, 8, 64, 1, None) == -1


def test_binding_checks_tensors():
    f = dq.format_preset("mxfp4")
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):                                # not on a GPU: no fallback
        dq.add_rmsnorm_quant(x, torch.ones(64, dtype=torch.bfloat16), f)
    cache = dq.kv_cache(2, 16, 2, 64, f, device="cpu")
    assert [tuple(t.shape) for t in cache] == [(2, 2, 16, 32), (2, 2, 16, 2)] * 2
    i = lambda *v: torch.tensor(v, dtype=torch.int32)              # noqa: E731
    k = torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    table = torch.zeros(1, 2, dtype=torch.int32)
    for call in (lambda **a: dq.kv_append(a.get("k", k), k, a.get("cache", cache), a.get("starts", i(0, 1)),
                                          i(1), a.get("table", table), f),
                 lambda **a: dq.kv_attention(a.get("k", k), a.get("cache", cache), a.get("starts", i(0, 1)),
                                             i(1), a.get("table", table), f)):
        with pytest.raises(ValueError):                            # CPU tensors
            call()
        with pytest.raises(ValueError):
            call(starts=i(0, 1, 2))
        with pytest.raises(TypeError):
            call(table=table.long())
        with pytest.raises(TypeError):
            call(k=k.float())
        with pytest.raises(ValueError):
            call(k=k[..., ::2])
        with pytest.raises(ValueError):                            # scales of another format
            call(cache=(cache[0], cache[1][..., :1], cache[2], cache[3]))
