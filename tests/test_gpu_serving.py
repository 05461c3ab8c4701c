"""The serving operators on the GPU against their plain 64-bit forms."""
import math

import numpy as np
import pytest
import torch

import oracle as O
from _helpers import MX_MORE, PRESET_COMBOS, gpu_scales_np, lib_format
from _serving import KV_FORMATS, Batch, attend64, bf16_from, decoded

pytestmark = pytest.mark.gpu

dq = pytest.importorskip("dual_scale_solver_b200")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from dual_scale_solver_b200 import build
    build.build()


# --------------------------------------------------------------------------- #
# residual + norm + quantization
# --------------------------------------------------------------------------- #

def _check_norm(x, w, name, G, residual=None, b=None, eps=1e-5, **kw):
    """Every code and scale must be Q of some y within the float32 error of
    the exact one.  y = h inv w b: h has one rounding (2^-24), the products
    three more, division and square root one each; the mean's sum is a chain
    of at most 64 additions per thread and 10 over lanes and warps, each off
    by 2^-24 of a sum of squares at most, halved by the square root: (4 + 2 +
    74 / 2) 2^-24 < 2^-18."""
    f, fo = lib_format(name, G), PRESET_COMBOS[name](G)
    codes, gs, ro = dq.add_rmsnorm_quant(x, w, f, residual=residual, b=b, eps=eps, **kw)
    torch.cuda.synchronize()
    h = x.cpu().double().numpy()
    if residual is not None:
        assert torch.equal(ro, (x.float() + residual.float()).to(torch.bfloat16))
        h = h + residual.cpu().double().numpy()
    y = h / np.sqrt((h * h).mean(1, keepdims=True) + eps) * w.cpu().double().numpy()
    if b is not None:
        y = y * b.cpu().double().numpy()
    c, s = decoded(codes, gs, fo)
    d = 2.0 ** -18
    yg = y.reshape(*s.shape, fo.group)
    m = np.abs(yg).max(-1)
    pos = m > 0
    lo, hi = (np.where(pos, O.project_group_scale(np.where(pos, m * e / fo.qmax, 1.0), fo), 1.0)
              for e in (1 - d, 1 + d))
    assert np.all((s >= lo) & (s <= hi))
    q = yg / s[..., None]
    ends = [O.round_codes(q * e, fo) for e in (1 - d, 1 + d)]
    cg = c.reshape(yg.shape)
    assert np.all((cg >= np.minimum(*ends)) & (cg <= np.maximum(*ends)))
    # and the slack is rarely used
    exact = np.all(lo == hi) and np.mean(ends[0] != ends[1]) < 1e-2
    assert exact or yg.size < 10000 or np.mean(lo != hi) < 1e-2
    return codes, gs, ro


@pytest.mark.parametrize("name,G", [("int4_bf16", 64), ("mxint4", 32), ("mxfp4", 32), ("nvfp4", 16)] +
                         [(n, 32) for n in MX_MORE] + [("mxfp8_e4m3", 16), ("mxint8", 64), ("nvfp4_ts1", 64)])
@pytest.mark.parametrize("tokens,K", [(1, 64), (7, 576), (3, 4160)])
def test_norm_formats(name, G, tokens, K):
    rng = np.random.default_rng([1, tokens, K])
    x, r = bf16_from(rng, (tokens, K)), bf16_from(rng, (tokens, K), 3.0)
    w = bf16_from(rng, K)
    _check_norm(x.cuda(), w.cuda(), name, G, residual=r.cuda())


@pytest.mark.parametrize("tokens,K", [(1, 32), (2, 8192), (600, 96), (700, 8192), (601, 8224), (2, 32768),
                                      (2, 32800), (3, 40000)])
@pytest.mark.parametrize("residual", [False, True])
def test_norm_shapes(tokens, K, residual):
    """Row lengths on both sides of each kernel's limits (one chunk per
    thread, four, rows read twice)."""
    rng = np.random.default_rng([2, tokens, K])
    x = bf16_from(rng, (tokens, K), 0.1)
    r = bf16_from(rng, (tokens, K)) if residual else None
    w = torch.from_numpy(rng.standard_normal(K).astype(np.float32))
    b = torch.from_numpy(np.exp2(rng.integers(-3, 3, K)).astype(np.float32))
    _check_norm(x.cuda(), w.cuda(), "mxfp8_e4m3", 32, residual=r.cuda() if residual else None, b=b.cuda())


def test_norm_strided_in_place_and_special_rows():
    rng = np.random.default_rng(3)
    K = 256
    big = bf16_from(rng, (9, 2 * K)).cuda()
    x, r = big[:, :K], big[:, K:]                        # rows of a wider matrix
    w = bf16_from(rng, K).cuda()
    r[4] = -x[4]                                         # a sum of exact zeros
    x[5] *= 1e-18                                        # eps rules
    r[5] *= 1e-18
    x[6, 3] = 3e4                                        # one value rules
    before = r.clone()
    fresh = _check_norm(x, w, "mxfp4", 32, residual=r)
    assert torch.equal(r, before)
    codes, gs, ro = dq.add_rmsnorm_quant(x, w, dq.format_preset("mxfp4"), residual=r, residual_out=r)
    torch.cuda.synchronize()
    assert ro is r and torch.equal(r, fresh[2]) and torch.equal(codes, fresh[0]) and torch.equal(gs, fresh[1])
    assert torch.equal(x, big[:, :K])
    # the same in place on rows that are read twice
    K = 33024
    x, r, w = bf16_from(rng, (2, K)).cuda(), bf16_from(rng, (2, K)).cuda(), bf16_from(rng, K).cuda()
    fresh = _check_norm(x, w, "mxfp8_e4m3", 32, residual=r)
    codes, gs, _ = dq.add_rmsnorm_quant(x, w, dq.format_preset("mxfp8_e4m3"), residual=r, residual_out=x)
    torch.cuda.synchronize()
    assert torch.equal(x, fresh[2]) and torch.equal(codes, fresh[0]) and torch.equal(gs, fresh[1])


def test_norm_empty_and_nonfinite():
    f = dq.format_preset("mxfp8_e4m3")
    w = torch.ones(64, device="cuda")
    codes, gs, ro = dq.add_rmsnorm_quant(torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), w, f)
    assert codes.numel() == 0 and gs.shape == (0, 2) and ro is None
    assert dq.last_device_status() == 0
    for bad in (float("nan"), float("inf"), 3e38):       # the last: finite, its square is not
        x = torch.ones(3, 64, dtype=torch.bfloat16, device="cuda")
        x[1, 5] = bad
        good = dq.add_rmsnorm_quant(torch.ones_like(x), w, f)
        got = dq.add_rmsnorm_quant(x, w, f)
        assert dq.last_device_status() == -4
        for i in (0, 2):                                 # its neighbours are not touched
            assert torch.equal(got[0][i], good[0][i]) and torch.equal(got[1][i], good[1][i])


# --------------------------------------------------------------------------- #
# the cache
# --------------------------------------------------------------------------- #

@pytest.mark.parametrize("name,G", [("int4_bf16", 64), ("int4_bf16", 16), ("mxint4", 32), ("mxfp4", 32),
                                    ("mxfp4", 64), ("nvfp4_ts1", 16), ("nvfp4", 32)])
@pytest.mark.parametrize("heads,dim,page", [(3, 64, 16), (2, 128, 48), (8, 128, 64)])
def test_append_and_read(name, G, heads, dim, page):
    seqs = [(1, 1), (5, 37), (0, 9), (20, 20), (1, 130)]
    B = Batch(seqs, page, heads, dim, name, G, pad=2)
    rng = np.random.default_rng([4, heads, dim, G])
    # one fused array of keys and values: strided rows
    kv = bf16_from(rng, (B.tokens, 2, heads, dim))
    kv[1] = 0.0                                          # all-zero groups
    kv = kv.cuda()
    k, v = kv[:, 0], kv[:, 1]
    cache, _ = B.fill()
    before = [t.clone() for t in cache]
    meta = B.device()
    dq.kv_append(k, v, cache, *meta, B.fmt)
    kk = torch.full((heads, B.tokens, dim), 7.0, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    vv = torch.full((B.tokens, heads, dim), 7.0, dtype=torch.bfloat16, device="cuda")
    dq.kv_read(cache, *meta, B.fmt, B.tokens, k=kk, v=vv)
    assert dq.last_device_status() == 0
    n = int(B.starts[-1])
    touched = np.zeros(B.pages * heads * page, dtype=bool)
    for x, codes, gs, got in ((k, cache[0], cache[1], kk), (v, cache[2], cache[3], vv)):
        cc = codes.cpu().numpy().reshape(-1, dim // 2)
        ss = gpu_scales_np(gs).reshape(-1, dim // G)
        for s, (new, m) in enumerate(seqs):
            for h in range(heads):
                rows = B.rows(s, h)[m - new:]
                t0 = B.starts[s]
                c, sc = O.quantize(x[t0:t0 + new, h].cpu().double().numpy(), B.fo, 1.0)
                assert np.array_equal(cc[rows], O.encode_codes(c, B.fo))
                assert np.array_equal(ss[rows], O.encode_scales(sc, B.fo))
                val = torch.from_numpy(O.dequantize(c, sc, B.fo)).to(torch.bfloat16)
                assert torch.equal(got[t0:t0 + new, h].cpu(), val)
                touched[rows] = True
        assert bool((got[n:] == 7.0).all())              # padding rows left as they were
    for t, o in zip(cache, before):                      # and every other slot
        a, b = t.reshape(touched.size, -1).cpu(), o.reshape(touched.size, -1).cpu()
        keep = torch.from_numpy(~touched)
        assert torch.equal(a[keep], b[keep])


def test_append_many_tokens_and_sequences():
    """More tokens than one pass of the grid, more sequences than one look of
    a warp, some of them without new tokens."""
    rng = np.random.default_rng(5)
    seqs = [(int(n), int(n + m)) for n, m in zip(rng.integers(0, 60, 700), rng.integers(0, 40, 700))]
    B = Batch(seqs, 16, 1, 64, "mxfp4", 32)
    k, v = (bf16_from(rng, (B.tokens, 1, 64)).cuda() for _ in range(2))
    cache = dq.kv_cache(B.pages, 16, 1, 64, B.fmt)
    meta = B.device()
    dq.kv_append(k, v, cache, *meta, B.fmt)
    kk, vv = dq.kv_read(cache, *meta, B.fmt, B.tokens)
    assert dq.last_device_status() == 0
    for x, got in ((k, kk), (v, vv)):
        c, s = O.quantize(x.cpu().double().numpy().reshape(-1, 64), B.fo, 1.0)
        assert np.array_equal(got.cpu().double().numpy().reshape(-1, 64), O.dequantize(c, s, B.fo))


def test_append_nonfinite_flag():
    B = Batch([(2, 2)], 16, 1, 64, "mxint4", 32)
    k = torch.ones(2, 1, 64, dtype=torch.bfloat16, device="cuda")
    v = k.clone()
    v[1, 0, 3] = float("inf")
    cache = dq.kv_cache(B.pages, 16, 1, 64, B.fmt)
    dq.kv_append(k, v, cache, *B.device(), B.fmt)
    assert dq.last_device_status() == -4


# --------------------------------------------------------------------------- #
# attention
# --------------------------------------------------------------------------- #

def _check_attention(B, q, cache, values, scale=None, causal=True, out=None, **kw):
    """|out - exact| <= 2^-8 |exact| (the output's rounding) + e W, W = sum_p
    w_p |v_p|.  e: half a step of the probabilities' type (2^-11 fp16, 2^-8
    bf16 where prompts take that) and of the values' (2^-8: code * BF16 scale
    in bf16), on both the numerator's terms; and the scores' error: a sum of
    D products of queries and codes (bf16 each for prompts: 2^-8 of |k|
    where the scale has 8 bits) off by at most (2^-8 x [BF16 scales] + D
    2^-23) A scale, A = the row's largest sum |q k|, which moves every weight
    by that twice (its own and the sum's).  Last, fp16's absolute step, half
    of it 2^-25 below 2^-14.  With 2^E <= S, S the largest value scale: for
    few rows the operand is p s 2^(13 - E) against a sum of at least one 2^(13
    - E), times a code of at most 8: 2^-35 S for each position (and p itself,
    2^(7 .. 9) times a scale of at most 2^7: 2^-28 S); for prompts
    it is p 2^(E + 7 .. 15) against a sum that holds the row's largest of
    them, 2^7, times 2^-E, multiplied by code x scale / 2^E of at most 16:
    2^-28 S."""
    D = q.shape[2]
    sc = 1 / math.sqrt(D) if scale is None else scale
    got = dq.kv_attention(q, cache, *B.device(), B.fmt, scale=scale, causal=causal, out=out, **kw)
    assert dq.last_device_status() == 0
    exact, mag, size = attend64(q, B, values, sc, causal)
    bf = B.fo.gscale == "bf16"
    e = 2.0 ** -8 + 2.0 ** -8 * bf + 2 * size * sc * (D * 2.0 ** -23 + (2.0 ** -8 if bf else 0)) + 2.0 ** -18
    n = int(B.starts[-1])
    d = np.abs(got.cpu().double().numpy() - exact)[:n]
    bound = (2.0 ** -8 * np.abs(exact) + e * mag + (mag > 0) * max(B.lens) * 2.0 ** -28 * B.top_scale)[:n]
    worst = float(np.max(d - bound, initial=-1.0))
    assert worst <= 0, (worst, np.argwhere(d > bound)[:5])
    # and far closer in the mean: independent roundings, the output's own first
    if d.size >= 1000:
        assert np.sqrt((d ** 2).mean()) <= 4 * 2.0 ** -9 * np.sqrt((exact[:n] ** 2).mean())
    return got


COMBOS = [(n, g) for n in KV_FORMATS for g in (16, 32, 64)]


@pytest.mark.parametrize("name,G", COMBOS)
@pytest.mark.parametrize("dim", [64, 128])
def test_attention_single_tokens(name, G, dim):
    seqs = [(1, 1), (1, 2), (1, 31), (1, 32), (1, 33), (1, 255), (1, 257), (1, 700)]
    B = Batch(seqs, 48, 2, dim, name, G)
    cache, values = B.fill()
    q = bf16_from(B.rng, (B.tokens, 8, dim)).cuda()
    _check_attention(B, q, cache, values)


@pytest.mark.parametrize("name,G", [("int4_bf16", 64), ("mxint4", 16), ("mxfp4", 32), ("nvfp4_ts1", 16)])
@pytest.mark.parametrize("group", [1, 3, 7, 16])
def test_attention_groups_and_drafts(name, G, group):
    """Row tiles that end inside a token's heads, drafts of several tokens,
    sequences without new tokens, more new tokens than positions."""
    seqs = [(5, 300), (0, 40), (1, 17), (3, 3), (2, 64), (7, 4), (1, 0), (12, 90)]
    B = Batch(seqs, 16, 3, 64, name, G, pad=3)
    cache, values = B.fill()
    q = bf16_from(B.rng, (B.tokens, 3 * group, 64)).cuda()
    out = torch.full_like(q, 5.0)
    for causal in (True, False):
        _check_attention(B, q, cache, values, causal=causal, out=out)
        assert bool((out[int(B.starts[-1]):] == 5.0).all())          # padding rows
        t = int(B.starts[6])                                         # an empty sequence: zeros
        assert bool((out[t] == 0).all())
        if causal:
            assert bool((out[int(B.starts[5]):int(B.starts[5]) + 3] == 0).all())


@pytest.mark.parametrize("name,G", [("int4_bf16", 64), ("mxint4", 32), ("mxfp4", 32), ("nvfp4_ts1", 16)])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("seqs", [[(129, 129)], [(64, 300), (1, 5), (200, 200)], [(33, 1000), (0, 0), (127, 128)]])
def test_attention_prompts(name, G, dim, seqs):
    B = Batch(seqs, 16, 2, dim, name, G, pad=1)
    cache, values = B.fill()
    q = bf16_from(B.rng, (B.tokens, 8, dim)).cuda()
    for causal in (True, False):
        _check_attention(B, q, cache, values, causal=causal)


@pytest.mark.parametrize("name,G", [("int4_bf16", 64), ("mxint4", 32), ("mxfp4", 32), ("nvfp4_ts1", 16)])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("seqs,group", [([(40, 6000)], 4), ([(300, 2500), (0, 700), (3, 0), (70, 50)], 2),
                                        ([(700, 700), (300, 100), (260, 1500)], 2)])
def test_attention_prompts_cut_and_joined(name, G, dim, seqs, group):
    """Few row tiles over many positions: shares of the grid begin and end
    inside them.  Row tiles that do not fill the 256 rows, rows that see
    nothing, more CTAs than positions; the same bits again."""
    B = Batch(seqs, 16, 1, dim, name, G, pad=2)
    cache, values = B.fill()
    q = bf16_from(B.rng, (B.tokens, group, dim)).cuda()
    out = torch.full_like(q, 5.0)
    for causal in (True, False):
        a = _check_attention(B, q, cache, values, causal=causal, out=out).clone()
        assert bool((a[int(B.starts[-1]):] == 5.0).all())
        b = dq.kv_attention(q, cache, *B.device(), B.fmt, causal=causal)
        n = int(B.starts[-1])
        assert torch.equal(a[:n], b[:n])


def test_attention_prompts_many_sequences():
    """More row tiles than CTAs, sequences of every length; and more sequences
    than shares are planned for."""
    rng = np.random.default_rng(11)
    for count, longest in ((200, 60), (1100, 12)):
        seqs = [(int(n), int(n + m)) for n, m in zip(rng.integers(0, longest, count), rng.integers(0, 50, count))]
        seqs[count // 2] = (longest, 900)
        B = Batch(seqs, 16, 2, 64, "mxfp4", 32)
        cache, values = B.fill()
        q = bf16_from(B.rng, (B.tokens, 8, 64)).cuda()
        _check_attention(B, q, cache, values)


@pytest.mark.parametrize("name,G", [("int4_bf16", 64), ("mxfp4", 32)])
@pytest.mark.parametrize("seqs,group", [([(1, 300)] * 40 + [(100, 500), (32, 700)], 2),      # 7 rows in the mean
                                        ([(1, 900), (600, 1300), (4, 50), (0, 9), (9, 40), (8, 3)], 4),
                                        ([(1, 600), (1, 5), (3, 3)], 48)])
def test_attention_mixed_batches(name, G, seqs, group):
    """Single tokens, drafts and prompts in one call: sequences of up to 32
    rows and longer ones."""
    B = Batch(seqs, 16, 2, 64, name, G, pad=2)
    cache, values = B.fill()
    q = bf16_from(B.rng, (B.tokens, 2 * group, 64)).cuda()
    out = torch.full_like(q, 5.0)
    for causal in (True, False):
        a = _check_attention(B, q, cache, values, causal=causal, out=out).clone()
        assert bool((a[int(B.starts[-1]):] == 5.0).all())


@pytest.mark.parametrize("length", [-1, 65, 0x7FFFFFFF])
def test_bad_length_of_a_lone_prompt(length):
    cache = dq.kv_cache(5, 16, 1, 64, dq.format_preset("mxfp4"))
    q = torch.ones(40, 4, 64, dtype=torch.bfloat16, device="cuda")
    i = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    out = torch.full_like(q, 5.0)
    table = i(0, 1, 2, 3).view(1, 4)
    dq.kv_attention(q, cache, i(0, 40), i(length), table, dq.format_preset("mxfp4"), out=out)
    assert dq.last_device_status() == -12 and bool((out == 5.0).all())


@pytest.mark.parametrize("name,G", [("int4_bf16", 64), ("nvfp4_ts1", 16)])
@pytest.mark.parametrize("seqs", [[(1, 300), (1, 2000)], [(20, 300), (30, 2000)]])
def test_attention_nonfinite_queries_stay_in_their_rows(name, G, seqs):
    B = Batch(seqs, 16, 2, 64, name, G)
    cache, values = B.fill()
    q = bf16_from(B.rng, (B.tokens, 8, 64)).cuda()
    want = _check_attention(B, q, cache, values)
    bad = q.clone()
    bad[0, 1, 5], bad[B.tokens - 1, 6, 63] = float("nan"), float("nan")
    got = dq.kv_attention(bad, cache, *B.device(), B.fmt)
    assert bool(got[0, 1].isnan().all()) and bool(got[B.tokens - 1, 6].isnan().all())
    got[0, 1], got[B.tokens - 1, 6] = want[0, 1], want[B.tokens - 1, 6]
    assert torch.equal(got, want)


@pytest.mark.parametrize("new", [1, 20])
def test_bad_places_are_flagged_and_touch_nothing_else(new):
    """Pages out of range, lengths beyond the table, starts that decrease or
    pass the last row: flagged, and the other sequences' results are those of
    the clean batch."""
    B = Batch([(new, 200)] * 4, 16, 2, 64, "mxfp4", 32, spare=0)
    cache, values = B.fill()
    q = bf16_from(B.rng, (B.tokens, 8, 64)).cuda()
    k, v = (bf16_from(B.rng, (B.tokens, 2, 64)).cuda() for _ in range(2))
    starts, lens, table = B.device()
    want = _check_attention(B, q, cache, values)
    whole = [t.clone() for t in cache]
    dq.kv_append(k, v, cache, starts, lens, table, B.fmt)
    after = [t.clone() for t in cache]
    kk, vv = dq.kv_read(cache, starts, lens, table, B.fmt, B.tokens)
    assert dq.last_device_status() == 0
    last = table[2, 12].item()

    def put(t, at, value):
        t = t.clone()
        t[at] = value
        return t

    bad = [(starts, lens, put(table, (2, 12), x)) for x in (-1, B.pages, 1 << 30)]
    bad += [(starts, put(lens, 2, x), table) for x in (-1, 16 * table.shape[1] + 1, 0x7FFFFFFF)]
    rows = slice(2 * new, 3 * new)
    for meta in bad:
        for t, w in zip(cache, whole):
            t.copy_(w)
        out = torch.full_like(q, 5.0)
        dq.kv_attention(q, cache, *meta, B.fmt, out=out)
        assert dq.last_device_status() == -12
        out[rows] = want[rows]
        assert torch.equal(out, want)
        dq.kv_append(k, v, cache, *meta, B.fmt)
        assert dq.last_device_status() == -12
        for t, w, a in zip(cache, whole, after):
            same = torch.arange(B.pages, device="cuda") != last           # (its new tokens' last page)
            assert torch.equal(t[last], w[last])
            if meta[1] is lens and new == 1:
                assert torch.equal(t[same], a[same])
        for t, a in zip(cache, after):
            t.copy_(a)
        k2, v2 = dq.kv_read(cache, *meta, B.fmt, B.tokens)
        assert dq.last_device_status() == -12
        for x, y in ((k2, kk), (v2, vv)):
            x[rows] = y[rows]
            assert torch.equal(x, y)
    for t, w in zip(cache, whole):
        t.copy_(w)
    # starts: sequence 1 beyond the rows or behind its own start: 0 is still answered
    for x in (B.tokens + 1, -1):
        out = dq.kv_attention(q, cache, put(starts, 2, x), lens, table, B.fmt)
        assert dq.last_device_status() == -12
        assert torch.equal(out[:new], want[:new])
        dq.kv_append(k, v, cache, put(starts, 2, x), lens, table, B.fmt)
        assert dq.last_device_status() == -12
        for t, w in zip(cache, whole):
            t.copy_(w)


def test_places_past_32_bits():
    """Pages whose codes lie more than 2^32 bytes into the cache, the same
    bits as in a small one."""
    B = Batch([(1, 700), (2, 90)], 64, 8, 128, "mxfp4", 32)
    P = Batch([(60, 700), (30, 90)], 64, 8, 128, "mxfp4", 32)
    for b in (B, P):
        small, _ = b.fill()
        shift = (1 << 32) // (8 * 64 * 64) + 7
        big = tuple(torch.empty((b.pages + shift,) + t.shape[1:], dtype=t.dtype, device="cuda") for t in small)
        for t, s in zip(big, small):
            t[shift:] = s
        starts, lens, table = b.device()
        far = torch.where(table < b.pages, table + shift, table)
        q = bf16_from(b.rng, (b.tokens, 16 if b is P else 8, 128)).cuda()
        k, v = (bf16_from(b.rng, (b.tokens, 8, 128)).cuda() for _ in range(2))
        got = []
        for cache, tab in ((small, table), (big, far)):
            dq.kv_append(k, v, cache, starts, lens, tab, b.fmt)
            got.append((dq.kv_attention(q, cache, starts, lens, tab, b.fmt),
                        *dq.kv_read(cache, starts, lens, tab, b.fmt, b.tokens)))
        assert dq.last_device_status() == 0
        for x, y in zip(*got):
            assert torch.equal(x, y)
        for t, s in zip(big, small):
            assert torch.equal(t[shift:], s)
        del big


def test_attention_strides_scale_and_repeatability():
    B = Batch([(1, 500), (3, 77), (1, 2000)], 32, 2, 128, "mxfp4", 32)
    cache, values = B.fill()
    qkv = bf16_from(B.rng, (B.tokens, 12, 128)).cuda()
    q = qkv[:, 2:10]                                                 # heads of a fused projection
    out = torch.zeros(8, B.tokens, 128, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    a = _check_attention(B, q, cache, values, scale=0.3, out=out).clone()
    b = _check_attention(B, q, cache, values, scale=0.3)
    assert torch.equal(a, b)


@pytest.mark.parametrize("k_scale,v_scale,q_scale", [(1e-4, 1e4, 1e3), (200.0, 1e-20, 2e-2), (1e18, 1e25, 1e-18),
                                                     (1.0, 1.0, 0.0)])
@pytest.mark.parametrize("name,G", [("mxfp4", 32), ("int4_bf16", 64)])
def test_attention_far_magnitudes(name, G, k_scale, v_scale, q_scale):
    """Magnitudes far from one in keys, values and queries (fp16 operands are
    scaled by powers of two), sharp and flat softmaxes."""
    for seqs in ([(1, 300), (2, 40)], [(130, 300)]):
        B = Batch(seqs, 16, 1, 64, name, G)
        cache, values = B.fill(k_scale, v_scale)
        q = bf16_from(B.rng, (B.tokens, 4, 64), q_scale).cuda()
        _check_attention(B, q, cache, values, scale=0.02)


def test_attention_one_large_value_does_not_hide_the_rest():
    """A position with hardly any weight and values 2^20 times the others'."""
    B = Batch([(1, 64)], 16, 1, 64, "mxfp4", 32)
    cache, values = B.fill(k_scale=0.01)
    rows = B.rows(0, 0)
    k, v = bf16_from(B.rng, (64, 64), 0.02).double().numpy(), bf16_from(B.rng, (64, 64)).double().numpy()
    k[10], v[10] = -4.0, v[10] * 2.0 ** 20
    q = torch.full((1, 4, 64), 4.0, dtype=torch.bfloat16, device="cuda")
    for i, x in ((0, k), (2, v)):
        c, s = O.quantize(x, B.fo, 1.0)
        values[i // 2][rows] = O.dequantize(c, s, B.fo)
        cache[i].view(-1, 32)[torch.from_numpy(rows).cuda()] = torch.from_numpy(O.encode_codes(c, B.fo)).cuda()
        cache[i + 1].view(-1, 2)[torch.from_numpy(rows).cuda()] = torch.from_numpy(O.encode_scales(s, B.fo)).cuda()
    B.top_scale = 2.0 ** 20
    got = _check_attention(B, q, cache, values)
    assert float(got.abs().max()) < 100.0


def test_attention_many_sequences():
    """More sequences than a CTA's scan takes at once, most of them short."""
    rng = np.random.default_rng(7)
    seqs = [(1, int(m)) for m in rng.integers(1, 40, 600)]
    seqs[299], seqs[511] = (1, 3000), (0, 900)
    B = Batch(seqs, 16, 1, 64, "mxint4", 32)
    cache, values = B.fill()
    q = bf16_from(B.rng, (B.tokens, 2, 64)).cuda()
    _check_attention(B, q, cache, values)


def test_attention_long_context_is_cut_and_joined():
    B = Batch([(1, 40000)], 64, 1, 128, "mxfp4", 32)
    cache, values = B.fill()
    q = bf16_from(B.rng, (1, 8, 128)).cuda()
    _check_attention(B, q, cache, values)


def test_empty_calls():
    f = dq.format_preset("mxfp4")
    cache = dq.kv_cache(2, 16, 2, 64, f)
    z = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    e = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    dq.kv_append(e, e, cache, z(2), z(1), z(1, 1), f)
    assert dq.kv_attention(e, cache, z(2), z(1), z(1, 1), f).shape == (0, 2, 64)
    one = torch.ones(1, 2, 64, dtype=torch.bfloat16, device="cuda")
    out = torch.full_like(one, 3.0)
    dq.kv_attention(one, cache, z(1), z(0), z(0, 1), f, out=out)      # no sequences: nothing is written
    torch.cuda.synchronize()
    assert bool((out == 3.0).all()) and dq.last_device_status() == 0


def test_a_step_in_a_graph_on_another_stream():
    """Norm, append and attention captured together on a side stream and
    replayed on new inputs: the results of direct calls, and two graphs with
    their own workspaces side by side."""
    B = Batch([(1, 200), (1, 33), (1, 1)], 16, 2, 128, "mxfp4", 32)
    cache, _ = B.fill()
    meta = B.device()
    f8 = dq.format_preset("mxfp8_e4m3")
    rng = np.random.default_rng(8)
    w = bf16_from(rng, 1024).cuda()
    x, r, k, v = (torch.zeros(3, 1024, dtype=torch.bfloat16, device="cuda") for _ in range(4))

    def step():
        codes, gs, h = dq.add_rmsnorm_quant(x, w, f8, residual=r)
        dq.kv_append(k.view(3, 8, 128)[:, :2], v.view(3, 8, 128)[:, :2], cache, *meta, B.fmt)
        o = dq.kv_attention(h.view(3, 8, 128), cache, *meta, B.fmt)
        return codes, gs, h, o

    step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            outs = step()
        graphs.append((g, outs))
    for i in range(3):
        for t in (x, r, k, v):
            t.copy_(bf16_from(rng, (3, 1024)))
        want = [t.clone() for t in step()]
        for g, outs in graphs:
            for t in outs:
                t.zero_()
            g.replay()
        torch.cuda.synchronize()
        for g, outs in graphs:
            for a, b in zip(outs, want):
                assert torch.equal(a, b)
    assert dq.last_device_status() == 0


def test_explicit_stream():
    B = Batch([(1, 3000), (4, 700)], 16, 2, 64, "nvfp4_ts1", 16)
    cache, values = B.fill()
    q = bf16_from(B.rng, (B.tokens, 4, 64)).cuda()
    want = _check_attention(B, q, cache, values)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a = dq.kv_attention(q, cache, *B.device(), B.fmt, stream=side)
    side.synchronize()
    assert torch.equal(a, want)


def test_two_streams_at_once():
    """Calls that overlap, each with its own workspace."""
    B = Batch([(1, 3000), (1, 700)], 16, 2, 64, "mxfp4", 32)
    P = Batch([(90, 1500)], 16, 2, 64, "mxfp4", 32)
    work = []
    for b in (B, P):
        cache, values = b.fill()
        q = bf16_from(b.rng, (b.tokens, 8, 64)).cuda()
        work.append((b, cache, q, b.device(), _check_attention(b, q, cache, values)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    outs = []
    for i in range(20):
        for j, s in enumerate(streams):
            b, cache, q, meta, want = work[(i + j) % 2]
            with torch.cuda.stream(s):
                outs.append((dq.kv_attention(q, cache, *meta, b.fmt), want))
    torch.cuda.synchronize()
    for got, want in outs:
        assert torch.equal(got, want)
    assert dq.last_device_status() == 0


def test_a_layer_with_quantized_products():
    """The pieces as they are used: norm and quantization, the W4A4 product
    that gives queries, keys and values, the cache, attention, and the next
    norm, against the same chain in float64 on the values that each step
    handed on."""
    fm, fo = dq.format_preset("mxfp4"), O.preset("mxfp4")
    rng = np.random.default_rng(9)
    T, K, heads, dim = 128, 512, 2, 64
    x, w = bf16_from(rng, (T, K)).cuda(), bf16_from(rng, K).cuda()
    W = bf16_from(rng, (768, K), 0.05).cuda()                        # 8 query heads, 2 + 2 of the cache
    sol = dq.solve_dual_scale(W, fm, 3)
    codes, gs, _ = _check_norm(x, w, "mxfp4", 32, b=sol["b"])
    qkv = dq.w4a4_gemm(codes, gs, sol["codes"], sol["gscales"], sol["a"]).to(torch.bfloat16)
    ref = O.w4a4_gemm(O.decode_codes(codes.cpu().numpy(), fo), O.decode_scales(gs.cpu().numpy(), fo),
                      O.decode_codes(sol["codes"].cpu().numpy(), fo),
                      O.decode_scales(sol["gscales"].cpu().numpy(), fo), sol["a"].cpu().double().numpy(), fo)
    assert np.max(np.abs(qkv.double().cpu().numpy() - ref)) <= (2.0 ** -8 + 1e-5) * np.max(np.abs(ref))
    qkv = qkv.view(T, 12, dim)
    B = Batch([(100, 100), (28, 28)], 16, heads, dim, "mxfp4", 32)
    cache = dq.kv_cache(B.pages, 16, heads, dim, fm)
    B.top_scale = 1.0
    dq.kv_append(qkv[:, 8:10], qkv[:, 10:], cache, *B.device(), fm)
    values = [O.dequantize(O.decode_codes(cache[i].cpu().numpy().reshape(-1, dim // 2), fo),
                           O.decode_scales(cache[i + 1].cpu().numpy().reshape(-1, dim // 32), fo), fo)
              for i in (0, 2)]
    o = _check_attention(B, qkv[:, :8], cache, values)
    o2, x2 = o.reshape(T, K), x.clone()
    _check_norm(o2, w, "mxfp4", 32, residual=x2)
    assert dq.last_device_status() == 0
