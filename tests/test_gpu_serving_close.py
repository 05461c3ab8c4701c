"""How close the serving operators come to their definitions in 64 bits, by
the roundings that their kernels make."""
import math

import numpy as np
import pytest
import torch

import oracle as O
from _helpers import PRESET_COMBOS, lib_format
from _serving import KV_FORMATS, Batch, bf16_from, decoded

pytestmark = pytest.mark.gpu

dq = pytest.importorskip("dual_scale_solver_b200")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from dual_scale_solver_b200 import build
    build.build()


# --------------------------------------------------------------------------- #
# norm
# --------------------------------------------------------------------------- #

@pytest.mark.parametrize("K", [1 << 24, (1 << 24) + 4064])
@pytest.mark.parametrize("off", [-1.0, 1.0])
def test_norm_of_a_very_long_row(K, off):
    """All of x is 1 + 2^-7, so y is the weight (eps moves it by 2^-39 of
    itself at most).  Its square is 1 + 2^-6 + 2^-14; the last term is lost to
    every addition of a float32 sum above 2^12, which a thread's 2^14 squares
    pass: 6e-5 of the sum, 3e-5 of y.  Weights 1e-5 off the middle of two codes
    fall on the exact side only if the sum is better than that."""
    x = torch.full((1, K), 1.0078125, dtype=torch.bfloat16, device="cuda")
    w = torch.full((K,), 1.0625 * (1.0 + off * 1e-5), device="cuda")
    w[::32] = 440.0                                       # every group's scale is 1
    codes, gs, _ = dq.add_rmsnorm_quant(x, w, dq.format_preset("mxfp8_e4m3"), eps=1e-12)
    assert dq.last_device_status() == 0
    assert bool((gs == 127).all())
    y = codes.view(torch.float8_e4m3fn).float().view(-1, 32)
    assert bool((y[:, 0] == 448.0).all())                 # (440 lies between 416 and 448)
    assert bool((y[:, 1:] == (1.0 if off < 0 else 1.125)).all())


@pytest.mark.parametrize("tokens,K", [(64, 8192), (600, 8192), (13, 40000)])
@pytest.mark.parametrize("name,G", [("mxfp8_e4m3", 32), ("mxfp4", 32), ("nvfp4_ts1", 16)])
def test_norm_codes_are_those_of_the_exact_y(tokens, K, name, G):
    """Both numbers of elements a thread, and rows read twice.  y = h inv w b:
    h has one rounding (2^-24); the sum at most 32 additions in a thread and 5
    over lanes, halved by the root; the root 1.1; the three products one each:
    below 25 x 2^-24.  Codes that differ from the exact y's lie within that of
    a border, and as the roundings are independent, the mean error is far
    below the greatest: not a quarter of the codes that near a border differ."""
    rng = np.random.default_rng([22, tokens, K])
    f, fo = lib_format(name, G), PRESET_COMBOS[name](G)
    x, r, w = bf16_from(rng, (tokens, K)), bf16_from(rng, (tokens, K), 2.0), bf16_from(rng, K)
    b = torch.from_numpy(rng.uniform(0.5, 2.0, K).astype(np.float32))
    codes, gs, _ = dq.add_rmsnorm_quant(x.cuda(), w.cuda(), f, residual=r.cuda(), b=b.cuda())
    assert dq.last_device_status() == 0
    h = x.double().numpy() + r.double().numpy()
    y = h / np.sqrt((h * h).mean(1, keepdims=True) + 1e-5) * w.double().numpy() * b.double().numpy()
    c, s = decoded(codes, gs, fo)
    d = 25 * 2.0 ** -24
    yg = y.reshape(*s.shape, G)
    m = np.abs(yg).max(-1)
    lo, mid, hi = (O.project_group_scale(m * e / fo.qmax, fo) for e in (1 - d, 1.0, 1 + d))
    assert np.all((s >= lo) & (s <= hi))
    assert (s != mid).sum() <= (lo != hi).sum() / 4 + 8
    q, cg = yg / s[..., None], c.reshape(yg.shape)
    lo, mid, hi = (O.round_codes(q * e, fo) for e in (1 - d, 1.0, 1 + d))
    assert np.all((cg >= np.minimum(lo, hi)) & (cg <= np.maximum(lo, hi)))
    assert (cg != mid).sum() <= (lo != hi).sum() / 4 + 8


# --------------------------------------------------------------------------- #
# attention
# --------------------------------------------------------------------------- #

def _exact(q, B, values, scale, causal):
    """softmax(scale q k^T) v in float64: (out, sum w |v|, sqrt(sum w^2 v^2),
    largest sum |q k| of the row)."""
    T, Hq, D = q.shape
    g, q = Hq // B.heads, q.double()
    K, V = (torch.from_numpy(x).cuda() for x in values)
    out, mag, sq = (torch.zeros(T, Hq, D, dtype=torch.float64, device="cuda") for _ in range(3))
    size = torch.zeros(T, Hq, 1, dtype=torch.float64, device="cuda")
    for i, (n, m) in enumerate(B.seqs):
        t0 = int(B.starts[i])
        if n == 0 or m == 0:
            continue
        limit = torch.arange(n, device="cuda") + m - n + 1 if causal else torch.full((n,), m, device="cuda")
        hidden = torch.arange(m, device="cuda")[None, :] >= limit[:, None]
        for h in range(B.heads):
            rows = torch.from_numpy(B.rows(i, h)).cuda()
            k, v = K[rows], V[rows]
            for j in range(h * g, (h + 1) * g):
                x = q[t0:t0 + n, j]
                w = torch.softmax((scale * x @ k.T).masked_fill(hidden, -math.inf), 1).nan_to_num(0.0)
                out[t0:t0 + n, j], mag[t0:t0 + n, j] = w @ v, w @ v.abs()
                sq[t0:t0 + n, j] = ((w * w) @ (v * v)).sqrt()
                size[t0:t0 + n, j] = (x.abs() @ k.abs().T).amax(1, keepdim=True)
    return out, mag, sq, size


def _check_close(B, q, cache, values, scale, causal=True):
    """Operands are exact in fp16, but for the probabilities (half a step,
    2^-11) and, for few rows, their products with value scales (2^-11 again).
    Sums are float32 with an error of 2^-23 of the sum of magnitudes for each
    product: D in a score, which moves a weight twice (its own, and the sum of
    all), as many as there are positions in an output.  The exponent and its
    function: 2^-16.  fp16's least step: 2^-28 of the largest value scale for
    each position.  The output is rounded to bf16 (2^-8).
    In the mean square: the output's own rounding, and for each position one
    (prompts) or two independent roundings to fp16 of w v, at most 2^-11 / sqrt(3)
    each, here with sqrt(3 / 2) for what else is rounded."""
    D, n = q.shape[2], int(B.starts[-1])
    sc = 1 / math.sqrt(D) if scale is None else scale
    got = dq.kv_attention(q, cache, *B.device(), B.fmt, scale=scale, causal=causal)[:n].double()
    assert dq.last_device_status() == 0
    exact, mag, sq, size = (t[:n] for t in _exact(q, B, values, sc, causal))
    longest = int(max(B.lens))
    e = 2.0 ** -10 + 2 * size * sc * D * 2.0 ** -23 + longest * 2.0 ** -23 + 2.0 ** -16
    bound = 2.0 ** -8 * exact.abs() + 1.01 * e * mag + (mag > 0) * longest * 2.0 ** -28 * B.top_scale
    d = got - exact
    assert bool((d.abs() <= bound).all()), float((d.abs() - bound).max())
    assert d.numel() >= 4000
    own = exact.to(torch.bfloat16).double() - exact
    ms = lambda t: float(t.square().mean())                        # noqa: E731
    assert ms(d) <= ms(own) + (2 * 2.0 ** -11) ** 2 * ms(sq), (ms(d) / ms(own), ms(own) / ms(sq))


COMBOS = [(n, g) for n in KV_FORMATS for g in (16, 32, 64)]


@pytest.mark.parametrize("name,G", COMBOS)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("seqs", [[(1, 700), (4, 257), (1, 33), (8, 90)], [(150, 400), (200, 200), (40, 333)],
                                  [(1, 500), (90, 300), (3, 70), (0, 20)]])
def test_attention_close_at_every_group(name, G, dim, seqs):
    """Few rows, prompts and both, in each format with each group."""
    B = Batch(seqs, 16, 2, dim, name, G, pad=1)
    cache, values = B.fill()
    q = bf16_from(B.rng, (B.tokens, 8, dim)).cuda()
    for scale, causal in ((0.02, True), (0.02, False), (None, True)):
        _check_close(B, q, cache, values, scale, causal)


@pytest.mark.parametrize("name,G", [("int4_bf16", 64), ("mxfp4", 32), ("nvfp4_ts1", 16)])
def test_attention_close_when_cut(name, G):
    B = Batch([(40, 3000), (1, 3000)], 16, 1, 64, name, G)
    cache, values = B.fill()
    q = bf16_from(B.rng, (B.tokens, 4, 64)).cuda()
    for scale in (0.02, None):
        _check_close(B, q, cache, values, scale)


def test_outputs_between_the_rows_of_inputs():
    """Interleaved slices of one array share no element: they are answered,
    and the input's rows stay as they were."""
    B = Batch([(1, 700), (4, 257), (40, 300)], 16, 2, 64, "mxfp4", 32)
    cache, _ = B.fill()
    both = bf16_from(B.rng, (B.tokens, 16, 64)).cuda()
    q, out, before = both[:, :8], both[:, 8:], both[:, :8].clone()
    want = dq.kv_attention(before, cache, *B.device(), B.fmt)
    dq.kv_attention(q, cache, *B.device(), B.fmt, out=out)
    assert torch.equal(out, want) and torch.equal(q, before)
    both = torch.zeros(B.tokens, 2, 2, 64, dtype=torch.bfloat16, device="cuda")
    kv = dq.kv_read(cache, *B.device(), B.fmt, B.tokens)
    dq.kv_read(cache, *B.device(), B.fmt, B.tokens, k=both[:, 0], v=both[:, 1])
    assert torch.equal(both[:, 0], kv[0]) and torch.equal(both[:, 1], kv[1])
    rows = bf16_from(B.rng, (5, 3 * 256)).cuda()
    x, r, s = rows[:, :256], rows[:, 256:512], rows[:, 512:]
    w, f, keep = torch.ones(256, device="cuda"), dq.format_preset("mxfp4"), rows.clone()
    want = dq.add_rmsnorm_quant(x, w, f, residual=r)
    got = dq.add_rmsnorm_quant(x, w, f, residual=r, residual_out=s)
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(rows[:, :512], keep[:, :512])
    with pytest.raises(dq.DqError):
        dq.add_rmsnorm_quant(x, w, f, residual=r, residual_out=rows[:, 8:264])
    fused = torch.zeros(B.tokens, 9, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(dq.DqError):                  # one head's rows in common
        dq.kv_attention(fused[:, :8], cache, *B.device(), B.fmt, out=fused[:, 1:])
    assert dq.last_device_status() == 0
