"""Plain 64-bit references of the ragged paged-attention operators and of the
rotary cache append, and the error bounds their tests use.

Everything is computed token by token from the definition (numpy, fp64, on the
CPU), without the library.
"""
from __future__ import annotations

import numpy as np
import torch

# a rounding to the type is off by at most half a step: eps / 2 relative
HALF_STEP = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": 2.0 ** -24, "fp8": 2.0 ** -4}
TORCH = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp8": torch.float8_e4m3fn}


def values(t: torch.Tensor) -> np.ndarray:
    """A CPU tensor's values in fp64."""
    return t.float().double().numpy()


def token_interval(i, n, L, *, causal, window=0, prefix=0, doc=0):
    """Keys [lo, hi) that query token i of n sees in a request of L keys."""
    pos = L - n + i
    hi = min(max(pos + 1, prefix), L) if causal else L
    lo = max(0, pos - (window - 1) if window > 0 else 0, doc)
    return (lo, hi) if lo < hi else (0, 0)


def paged_rows(cache, table_row, keys, page_size, num_pages):
    """K, V rows [n, Hkv, D] of the given keys of one request, and which of them
    lie on a page of the pool."""
    D = cache.shape[-1] // 2
    pages = table_row[keys // page_size] if len(keys) else np.zeros(0, int)
    ok = (pages >= 0) & (pages < num_pages)
    rows = cache[np.where(ok, pages, 0), :, keys % page_size]
    return rows[..., :D], rows[..., D:], ok


def attention(q, cache, table, lens, starts, scale, *, causal=True, window=0, softcap=0.0, slopes=None,
              prefix_lens=None, doc_start=None, q_scale=1.0, k_scale=1.0, v_scale=1.0):
    """out [T, Hq, D], lse [T, Hq] in fp64, and per output the two scales its
    error bound needs: A = sum_t w_t |v_t| [T, Hq, D] and S = max_t scale sum_d
    |q_d k_d| [T, Hq].  Tokens of no request come back as NaN."""
    T, Hq, D = q.shape
    num_pages, Hkv, P, _ = cache.shape
    G = Hq // Hkv
    out, mag = np.full((T, Hq, D), np.nan), np.zeros((T, Hq, D))
    lse, smax = np.full((T, Hq), np.nan), np.zeros((T, Hq))
    s0 = scale * q_scale * k_scale
    for b in range(len(lens)):
        n, L = int(starts[b + 1] - starts[b]), int(lens[b])
        for i in range(n):
            t = int(starts[b]) + i
            lo, hi = token_interval(i, n, L, causal=causal, window=window,
                                    prefix=int(prefix_lens[b]) if prefix_lens is not None else 0,
                                    doc=int(doc_start[t]) if doc_start is not None else 0)
            keys = np.arange(lo, hi)
            k, v, ok = paged_rows(cache, table[b], keys, P, num_pages)
            k, v, keys = k[ok], v[ok] * v_scale, keys[ok]
            if not len(keys):
                out[t], lse[t] = 0.0, -np.inf
                continue
            for h in range(Hq):
                s = (k[:, h // G] @ q[t, h]) * s0
                smax[t, h] = (np.abs(k[:, h // G]) @ np.abs(q[t, h])).max() * abs(s0)
                if softcap:
                    s = softcap * np.tanh(s / softcap)
                if slopes is not None:
                    s = s - slopes[h] * np.abs(L - n + i - keys)
                    smax[t, h] += slopes[h] * np.abs(L - n + i - keys).max()
                m = s.max()
                w = np.exp(s - m)
                lse[t, h] = m + np.log(w.sum())
                w /= w.sum()
                out[t, h] = w @ v[:, h // G]
                mag[t, h] = w @ np.abs(v[:, h // G])
    return out, lse, mag, smax


def check(got, got_lse, ref, dtype, out_dtype=None, what=""):
    """got, got_lse (CPU tensors) against attention()'s result.

    A score is a sum of D fp32 products scaled in fp32: off by ds = 1e-5 (1 + S)
    at most (S: the scale times the sum of the absolute products), so a weight is
    off by e^{2 ds} - 1 relative, and by half a step of the operand type where it
    is rounded for the product (fp16 for e4m3 caches); the output is rounded once
    more.  The LSE is off by ds and the fp32 rounding of its own size.
    """
    out, lse, mag, smax = ref
    real = ~np.isnan(lse)
    g, gl = values(got), values(got_lse)
    ds = 1e-5 * (1 + smax)
    operand = HALF_STEP["fp16" if dtype == "fp8" else dtype]
    final = HALF_STEP[out_dtype or ("bf16" if dtype == "fp8" else dtype)]
    tol = (operand + 2 * ds + 1e-5)[..., None] * mag * (1 + final) + final * np.abs(out) + 1e-7
    nans = int(np.isnan(g[real]).sum()), int(np.isnan(gl[real]).sum())
    assert nans == (0, 0), f"{what}: NaN in {nans} values of out, lse"
    share = float((np.abs(g - out)[real] > tol[real]).mean()) if real.any() else 0.0
    assert share == 0.0, f"{what}: out off by {np.abs(g - out)[real].max():.3g}, {share:.2%} outside the bound"
    empty = np.isneginf(lse)
    differ = int((np.isneginf(gl) != empty)[real].sum()), int((g[real & empty] != 0).sum())
    assert differ == (0, 0), f"{what}: rows without keys differ: {differ}"
    fin = real & ~empty
    off = np.abs(gl - np.where(fin, lse, 0.0))[fin]
    lim = (ds + 1e-6 * np.abs(np.where(fin, lse, 0.0)) + 1e-6)[fin]
    over = int((off > lim).sum())
    assert over == 0, f"{what}: lse off by {off.max():.3g}, {over} values"


class Paged:
    """A seeded paged problem on the CPU: q, cache, table, lengths, starts.

    Slots past a request's length, unused pages and (with `hole`) keys that no
    token sees hold NaN, so that a read of them shows.
    """

    def __init__(self, *, lens, news, Hq, Hkv, D, P=16, dtype="bf16", seed=0, extra_tokens=0, spread=2.0, width=None):
        rng = np.random.default_rng(seed)
        self.lens, self.news = np.asarray(lens, np.int32), np.asarray(news, np.int32)
        self.starts = np.concatenate([[0], np.cumsum(self.news)]).astype(np.int32)
        self.T, self.dtype, self.P, self.D, self.Hq, self.Hkv = int(self.starts[-1]) + extra_tokens, dtype, P, D, Hq, Hkv
        counts = [-(-int(n) // P) for n in self.lens]
        self.num_pages = sum(counts) + 3
        order = rng.permutation(self.num_pages)
        width = width or max(max(counts, default=1), 1)
        self.table = np.full((len(counts), width), order[-1], np.int32)
        used = np.zeros((self.num_pages, P), bool)
        at = 0
        for b, n in enumerate(counts):
            self.table[b, :n] = order[at:at + n]
            at += n
            t = np.arange(int(self.lens[b]))
            used[self.table[b, t // P], t % P] = True
        kv = rng.standard_normal((self.num_pages, Hkv, P, 2 * D)).astype(np.float32)
        q = spread * rng.standard_normal((self.T, Hq, D)).astype(np.float32)
        self.q_scale = self.k_scale = self.v_scale = 1.0
        if dtype == "fp8":
            self.q_scale, self.k_scale, self.v_scale = (float(np.float32(x)) for x in (8.5 / 448, 5.3 / 448, 4.7 / 448))
            q /= self.q_scale
            kv[..., :D] /= self.k_scale
            kv[..., D:] /= self.v_scale
            q, kv = np.clip(q, -448, 448), np.clip(kv, -448, 448)
        kv[~used.repeat(Hkv, 0).reshape(self.num_pages, Hkv, P)] = np.nan
        self.q, self.cache = (torch.from_numpy(x).to(TORCH[dtype]) for x in (q, kv))
        self.scale = D ** -0.5

    def scales(self):
        return dict(q_scale=self.q_scale, k_scale=self.k_scale, v_scale=self.v_scale)

    def reference(self, **kw):
        return attention(values(self.q), np.nan_to_num(values(self.cache)), self.table, self.lens, self.starts,
                         self.scale, **self.scales(), **kw)
