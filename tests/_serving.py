"""Plain 64-bit forms of the serving operators, and the inputs of their tests."""
import numpy as np
import torch

import oracle as O
from _helpers import PRESET_COMBOS, gpu_scales_np, lib_format

KV_FORMATS = ["int4_bf16", "mxint4", "mxfp4", "nvfp4_ts1"]


def bf16_from(rng, shape, scale=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).to(torch.bfloat16)


class Batch:
    """Sequences of (new tokens, length) on a cache of shuffled pages."""

    def __init__(self, seqs, page, heads, dim, name, G, seed=0, pad=0, spare=3):
        self.seqs, self.page, self.heads, self.dim, self.pad = seqs, page, heads, dim, pad
        self.fmt, self.fo = lib_format(name, G), PRESET_COMBOS[name](G)
        self.rng = np.random.default_rng([seed, page, heads, dim, G, len(seqs)])
        need = [-(-m // page) for _, m in seqs]
        self.pages = sum(need) + spare
        order = self.rng.permutation(self.pages)
        cols = max(max(need, default=0), 1)
        # entries behind a sequence's pages are never read: out of range on purpose
        self.table = np.full((len(seqs), cols + 1), 1 << 30, dtype=np.int32)
        at = 0
        for i, n in enumerate(need):
            self.table[i, :n] = order[at:at + n]
            at += n
        self.starts = np.concatenate([[0], np.cumsum([n for n, _ in seqs])]).astype(np.int32)
        self.lens = np.array([m for _, m in seqs], dtype=np.int32)
        self.tokens = int(self.starts[-1]) + pad

    def device(self):
        return [torch.from_numpy(x).cuda() for x in (self.starts, self.lens, self.table)]

    def rows(self, s, head):
        """Row numbers in a [pages * heads * page, ...] view of a sequence's positions."""
        p = np.arange(self.lens[s])
        return (self.table[s, p // self.page].astype(np.int64) * self.heads + head) * self.page + p % self.page

    def fill(self, k_scale=1.0, v_scale=1.0, garbage=True):
        """A cache whose sequences hold quantized normal values (float64
        values returned too) and whose other slots hold anything at all."""
        import dual_scale_solver_b200 as dq
        rng, fo, D = self.rng, self.fo, self.dim
        G = fo.group
        n = self.pages * self.heads * self.page
        cache, values = [], []
        for scale in (k_scale, v_scale):
            y = bf16_from(rng, (n, D), scale).double().numpy()
            y *= np.exp2(rng.integers(-3, 4, (n, 1)))            # token magnitudes differ
            y = torch.from_numpy(y).to(torch.bfloat16).double().numpy()
            c, s = O.quantize(y, fo, 1.0)
            codes, scales = O.encode_codes(c, fo), O.encode_scales(s, fo)
            used = np.zeros(n, dtype=bool)
            for b in range(len(self.seqs)):
                for h in range(self.heads):
                    used[self.rows(b, h)] = True
            if garbage:
                codes[~used] = rng.integers(0, 256, codes[~used].shape)
                scales[~used] = (0x7FC0 if fo.gscale == "bf16" else 0xFF if fo.gscale == "e8m0" else 0x7F)
            cache += [torch.from_numpy(codes.reshape(self.pages, self.heads, self.page, D // 2).copy()),
                      torch.from_numpy(scales.reshape(self.pages, self.heads, self.page, D // G).copy())]
            values.append(O.dequantize(c, s, fo))
            self.top_scale = float(s[used].max()) if used.any() else 1.0     # (of the values, last)
        cache = [t.view(torch.int16) if t.dtype == torch.uint16 else t for t in cache]
        assert cache[1].dtype == dq.gscale_dtype(self.fmt)
        return tuple(t.cuda() for t in cache), values


def attend64(q, batch, values, scale, causal):
    """softmax(scale q k^T) v per sequence and head in float64.  Returns (out,
    sum_p w_p |v_p|, largest sum_d |q_d k_pd| of the row) [tokens, heads, ...]."""
    q = q.double().cpu().numpy()
    T, Hq, D = q.shape
    g = Hq // batch.heads
    out, mag, size = np.zeros((T, Hq, D)), np.zeros((T, Hq, D)), np.zeros((T, Hq, 1))
    for b, (n, m) in enumerate(batch.seqs):
        if m == 0:
            continue
        for h in range(batch.heads):
            rows = batch.rows(b, h)
            K, V = values[0][rows], values[1][rows]
            for i in range(n):
                seen = min(m - n + i + 1, m) if causal else m
                if seen <= 0:
                    continue
                t = batch.starts[b] + i
                Q = q[t, h * g:(h + 1) * g]
                z = scale * Q @ K[:seen].T
                w = np.exp(z - z.max(1, keepdims=True))
                w /= w.sum(1, keepdims=True)
                out[t, h * g:(h + 1) * g] = w @ V[:seen]
                mag[t, h * g:(h + 1) * g] = w @ np.abs(V[:seen])
                size[t, h * g:(h + 1) * g, 0] = (np.abs(Q) @ np.abs(K[:seen]).T).max(1)
    return out, mag, size


def decoded(codes, gs, fo):
    return (O.decode_codes(codes.cpu().numpy(), fo),
            O.decode_scales(gpu_scales_np(gs), fo))
