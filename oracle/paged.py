"""The paged bf16 cache in float64, token by token: what fa_cache_append, fa_select_blocks, fa_decode_blocks and
fa_decode_shared compute, from the definitions in include/fa.h.  Shares no code with the GPU path.

A cache is a dict: k, v float64 [num_pages, Hkv, page, d] (bf16 values) and, with bounds, b float64 [num_pages, Hkv,
page / block, 2, d].
"""
import numpy as np


def append(cache, table, lens, k, v, new_lens=None):
    """Writes k, v [B,Hkv,N,d] (float64 of bf16 values) behind lens[b] tokens, in place; the bounds too, if there."""
    B, Hkv, N, _ = k.shape
    page = cache["k"].shape[2]
    bounds = cache.get("b")
    block = page // bounds.shape[2] if bounds is not None else 0
    for b in range(B):
        n = N if new_lens is None else int(new_lens[b])
        for i in range(min(n, table.shape[1] * page - int(lens[b]))):
            t = int(lens[b]) + i
            pg, at = int(table[b, t // page]), t % page
            cache["k"][pg, :, at] = k[b, :, i]
            cache["v"][pg, :, at] = v[b, :, i]
            if bounds is None:
                continue
            x = bounds[pg, :, at // block]
            if t % block == 0:
                x[:, 0], x[:, 1] = k[b, :, i], k[b, :, i]
            else:
                x[:, 0] = np.minimum(x[:, 0], k[b, :, i])  # NaN stays
                x[:, 1] = np.maximum(x[:, 1], k[b, :, i])


def scores(q, bounds, table, n, b, h):
    """Scores of the first n blocks of sequence b and kv head h: the largest bound over the group's rows."""
    Hkv, per = bounds.shape[1], bounds.shape[2]
    G = q.shape[1] // Hkv
    rows = q[b, h * G:(h + 1) * G].reshape(-1, q.shape[-1])
    out = np.empty(n)
    for j in range(n):
        lo, hi = bounds[int(table[b, j // per]), h, j % per]
        with np.errstate(invalid="ignore"):
            u = [(np.maximum(r, 0.0) * hi + np.minimum(r, 0.0) * lo).sum() for r in rows]
        out[j] = np.nan if np.isnan(u).any() else max(u)
    return out


def select(q, bounds, table, lens, block, keep, first, recent):
    """int32 [B, Hkv, keep]."""
    B, Hkv = table.shape[0], bounds.shape[1]
    out = np.full((B, Hkv, keep), -1, dtype=np.int32)
    for b in range(B):
        n = -(-int(lens[b]) // block)
        for h in range(Hkv):
            if n <= keep:
                out[b, h, :n] = np.arange(n)
                continue
            s = scores(q, bounds, table, n, b, h)
            mid = sorted(range(first, n - recent), key=lambda j: (not np.isnan(s[j]), 0 if np.isnan(s[j]) else -s[j], j))
            out[b, h] = sorted(list(range(first)) + mid[:keep - first - recent] + list(range(n - recent, n)))
    return out


def attend(q, cache, table, lens, scale, tokens=None):
    """O, LSE of q [B,Hq,Nq,d], the last Nq tokens, over tokens(b, h) (ascending or not; None: all).

    Also returns, per row, what an error bound needs: A = the largest sum |q_i k_i| scale over its keys, PV = sum p |v|.
    """
    q = np.asarray(q, dtype=np.float64)
    B, Hq, Nq, d = q.shape
    Hkv, page = cache["k"].shape[1:3]
    G = Hq // Hkv
    o, lse = np.zeros_like(q), np.full((B, Hq, Nq), -np.inf)
    A, PV = np.zeros((B, Hq, Nq)), np.zeros_like(q)
    for b in range(B):
        n = int(lens[b])
        for h in range(Hkv):
            j = np.arange(n) if tokens is None else np.asarray(tokens(b, h), dtype=np.int64)
            j = j[j < n]
            pg, at = np.asarray(table[b], dtype=np.int64)[j // page], j % page
            K, V = cache["k"][pg, h, at], cache["v"][pg, h, at]
            for r in range(G * Nq):
                hq, t = h * G + r // Nq, r % Nq
                see = j <= n - Nq + t
                if not see.any():
                    continue
                x = K[see] @ q[b, hq, t] * scale
                z = x.max() + np.log(np.exp(x - x.max()).sum())
                p = np.exp(x - z)
                o[b, hq, t], lse[b, hq, t] = p @ V[see], z
                A[b, hq, t] = (np.abs(K[see]) @ np.abs(q[b, hq, t])).max() * scale
                PV[b, hq, t] = p @ np.abs(V[see])
    return o, lse, A, PV


def tokens_of(blocks, block):
    """tokens(b, h) of a list of blocks [B, Hkv, keep]; negative ones are skipped."""
    def f(b, h):
        mine = blocks[b, h][blocks[b, h] >= 0]
        return (mine[:, None] * block + np.arange(block)).ravel()
    return f
