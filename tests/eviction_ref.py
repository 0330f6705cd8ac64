"""Plain 64-bit references of the operators that bound a paged cache (weights that keys
receive, choice of the keys that stay, compaction) and the error bound of the first.

Computed key by key from the definitions (numpy, fp64, on the CPU), without the library.
"""
from __future__ import annotations

import numpy as np

from tests.ragged_ref import paged_rows, token_interval


def key_weights(q, cache, table, lens, starts, lse, scale, *, prior=None, decay=1.0, causal=True, window=0, softcap=0.0,
                last=0, q_scale=1.0, k_scale=1.0):
    """weights [B, Hkv, keys of the table] (NaN behind a request's keys) and the bound of their error.

    The kernels sum D exact products in fp32, each addition off by a step (2^-23) of the
    sum of their magnitudes at most; the logit's scaling, the LSE's and their difference by
    four half steps of |s| + |lse|; the capped score by 2^-21 of the cap; the exponential by
    2^-22 of itself.  So a probability is off by a factor exp(e), and the sum of the rows by
    a half step of itself for each.  (Every term is below 1: e is taken to the first order.)
    """
    T, Hq, D = q.shape
    num_pages, Hkv, P, _ = cache.shape
    G, s0 = Hq // Hkv, scale * q_scale * k_scale
    out = np.full((len(lens), Hkv, table.shape[1] * P), np.nan)
    err = np.zeros_like(out)
    for b in range(len(lens)):
        n, L = int(starts[b + 1] - starts[b]), int(lens[b])
        out[b, :, :L] = 0.0
        if prior is not None:
            old = max(0, L - n)
            out[b, :, :old] = decay * prior[b, :, :old]
            err[b, :, :old] = 2.0 ** -23 * np.abs(out[b, :, :old])
        m = min(n, last) if last else n
        for i in range(n - m, n):
            t = int(starts[b]) + i
            lo, hi = token_interval(i, n, L, causal=causal, window=window)
            keys = np.arange(lo, hi)
            k, _, ok = paged_rows(cache, table[b], keys, P, num_pages)
            k, keys = k[ok], keys[ok]
            for h in range(Hq):
                if lse[t, h] == -np.inf or not len(keys):
                    continue
                s = (k[:, h // G] @ q[t, h]) * s0
                size = (np.abs(k[:, h // G]) @ np.abs(q[t, h])) * abs(s0)
                if softcap:
                    s = softcap * np.tanh(s / softcap)
                w = np.exp(s - lse[t, h])
                e = D * 2.0 ** -23 * size + 2.0 ** -22 * (np.abs(s) + abs(lse[t, h])) + 2.0 ** -22 + 2.0 ** -21 * softcap
                out[b, h // G, keys] += w
                err[b, h // G, keys] += w * (e + (m * G + 3) * 2.0 ** -24)
    return out, err


def evict_select(weights, lens, budget, *, sinks=0, recent=0, pool=1, positions=None, context=None):
    B, H, S = weights.shape
    kept, kept_lens = np.full((B, H, budget), -1, np.int32), np.zeros(B, np.int32)
    for b in range(B):
        L = min(max(int(lens[b]), 0), S)
        n = kept_lens[b] = min(L, budget)
        for h in range(H):
            seen = L if positions is None else int(context[b])
            rank = []
            free = {}
            for t in range(L):
                at = t if positions is None else int(positions[b, h, t])
                if sinks <= at < seen - recent:
                    x = float(weights[b, h, t])
                    free[t] = -np.inf if np.isnan(x) else x
            for t in range(L):
                if t not in free:
                    rank.append((0, 0.0, t))
                else:
                    near = [free[s] for s in range(t - pool // 2, t + pool // 2 + 1) if s in free]
                    rank.append((1, -max(near), t))
            kept[b, h, :n] = sorted(t for _, _, t in sorted(rank)[:n])
    return kept, kept_lens


def cache_compact(cache, table, kept, kept_lens, arrays=()):
    """In place, on arrays of any kind; pages outside the pool do not move."""
    num_pages, H, P = cache.shape[:3]
    for b in range(len(kept_lens)):
        n = int(kept_lens[b])
        for h in range(H):
            stay = kept[b, h, :n]
            source, target = [s for s in stay if s >= n], sorted(set(range(n)) - set(int(s) for s in stay))
            for s, t in zip(source, target):
                a, z = table[b, s // P], table[b, t // P]
                if not (0 <= a < num_pages and 0 <= z < num_pages):
                    continue
                cache[z, h, t % P] = cache[a, h, s % P]
                for x in arrays:
                    x[b, h, t] = x[b, h, s]
