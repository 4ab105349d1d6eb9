"""Rotary positions and the paged 8-bit cache in float64, token by token: what
fa_rope, fa_cache_append_fp8, fa_decode_paged_fp8 and fa_cache_evict_fp8 compute,
from the definitions in include/fa.h.  Shares no code with the GPU path.

A cache is a dict: k, v uint8 [num_pages, Hkv, page, d] (e4m3 bytes), ks, vs
float64 [num_pages, Hkv, page / sb].
"""
import math

import numpy as np

from .naive import _E4M3



def rope(x, positions, inv_freq, interleaved=False, magnitude=1.0, inverse=False):
    """x [B,H,N,d] turned by positions [B,N]: pair i by positions * inv_freq[i] radians."""
    x = np.asarray(x, dtype=np.float64)
    y = x.copy()
    half = len(inv_freq)
    for i in range(half):
        a = np.asarray(positions, dtype=np.float64)[:, None, :] * float(inv_freq[i])
        if inverse:
            a = -a
        p, q = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        c, s = magnitude * np.cos(a), magnitude * np.sin(a)
        y[..., p] = x[..., p] * c - x[..., q] * s
        y[..., q] = x[..., q] * c + x[..., p] * s
    return y


def to_e4m3(x):
    """e4m3 bytes of a float64 array: nearest value, ties to the even mantissa, saturated; NaN -> 0x7F."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(np.where(np.isnan(x), 0.0, x)), 448.0)
    pos = _E4M3[:127]                                                   # 0 .. 448 ascending: bytes 0 .. 126
    hi = np.minimum(np.searchsorted(pos, a), 126)
    lo = np.maximum(hi - 1, 0)
    up = pos[hi] - a
    down = a - pos[lo]
    byte = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    byte = np.where(pos[hi] == a, hi, byte)
    byte = np.where(np.signbit(x), byte | 0x80, byte)
    return np.where(np.isnan(x), 0x7F, byte).astype(np.uint8)


def scale_for(amax):
    """Smallest power of two s >= 2^-126 with amax <= 448 s."""
    s = 2.0 ** -126
    if amax > 0:
        s = max(s, 2.0 ** (math.floor(math.log2(amax / 448.0)) - 1))
    while amax > 448.0 * s:
        s *= 2.0
    return s


def append(cache, table, lens, k, v, new_lens=None):
    """Writes k, v [B,Hkv,N,d] (float64 of bf16 values) behind lens[b] tokens, in place."""
    B, Hkv, N, _ = k.shape
    page = cache["k"].shape[2]
    sb = page // cache["ks"].shape[2]
    for b in range(B):
        n = N if new_lens is None else int(new_lens[b])
        n = min(n, table.shape[1] * page - int(lens[b]))
        t = int(lens[b])
        end = t + n
        while t < end:
            first = t // sb * sb
            stop = min(first + sb, end)
            pg, at = int(table[b, t // page]), t % page
            f = first % page
            for key, sk, x in (("k", "ks", k), ("v", "vs", v)):
                for h in range(Hkv):
                    new = x[b, h, t - int(lens[b]):stop - int(lens[b])]
                    fin = np.abs(new[np.isfinite(new)])
                    s = scale_for(fin.max() if fin.size else 0.0)
                    if t > first:
                        old = cache[sk][pg, h, f // sb]
                        s = max(s, old)
                        if s != old:
                            cache[key][pg, h, f:at] = to_e4m3(_E4M3[cache[key][pg, h, f:at]] * old / s)
                    cache[key][pg, h, at:at + stop - t] = to_e4m3(new / s)
                    cache[sk][pg, h, f // sb] = s
            t = stop


def tokens(cache, table_row, length, h):
    """K and V [length, d] of one sequence and kv head."""
    page = cache["k"].shape[2]
    sb = page // cache["ks"].shape[2]
    j = np.arange(length)
    pg, at = np.asarray(table_row)[j // page], j % page
    return tuple(_E4M3[cache[n][pg, h, at]] * cache[n + "s"][pg, h, at // sb][:, None] for n in ("k", "v"))


def decode(q, cache, table, lens, scale, weights=None):
    """O, LSE of q [B,Hq,Nq,d], the last Nq tokens; adds to weights [B,Hkv,tokens] in place.

    Also returns, per row, what an error bound needs: A = the largest sum |q_i k_i| scale over its keys,
    PV = sum p |v|, and T = max_j (p_j vs_j) * sum_j |v8_j| (a value product with weights relative to the largest).
    """
    q = np.asarray(q, dtype=np.float64)
    B, Hq, Nq, d = q.shape
    Hkv = cache["k"].shape[1]
    page = cache["k"].shape[2]
    sb = page // cache["ks"].shape[2]
    G = Hq // Hkv
    o, lse = np.zeros_like(q), np.full((B, Hq, Nq), -np.inf)
    A, PV, T = np.zeros((B, Hq, Nq)), np.zeros_like(q), np.zeros_like(q)
    for b in range(B):
        n = int(lens[b])
        for h in range(Hkv):
            K, V = tokens(cache, table[b], n, h)
            j = np.arange(n)
            vs = cache["vs"][np.asarray(table[b])[j // page], h, j % page // sb]
            for r in range(G * Nq):
                hq, t = h * G + r // Nq, r % Nq
                m = n - Nq + t + 1
                if m <= 0:
                    continue
                x = K[:m] @ q[b, hq, t] * scale
                z = x.max() + np.log(np.exp(x - x.max()).sum())
                p = np.exp(x - z)
                o[b, hq, t], lse[b, hq, t] = p @ V[:m], z
                A[b, hq, t] = (np.abs(K[:m]) @ np.abs(q[b, hq, t])).max() * scale
                PV[b, hq, t] = p @ np.abs(V[:m])
                T[b, hq, t] = (p * vs[:m]).max() * (np.abs(V[:m]) / vs[:m, None]).sum(0)
                if weights is not None:
                    weights[b, h, :m] += p
    return o, lse, A, PV, T


def evict(cache, table, lens, weights, new_table, keep, recent):
    """Copies the kept tokens into new_table's pages, in place; (new_lens, new_weights, kept)."""
    B, Hkv = weights.shape[:2]
    page = cache["k"].shape[2]
    sb = page // cache["ks"].shape[2]
    C = new_table.shape[1] * page
    new_w, kept = np.zeros((B, Hkv, C), dtype=weights.dtype), np.full((B, Hkv, C), -1, dtype=np.int32)
    new_lens = np.minimum(lens, keep).astype(np.int32)
    src = {n: cache[n].copy() for n in ("k", "v", "ks", "vs")}
    for b in range(B):
        n = int(lens[b])
        for h in range(Hkv):
            if n <= keep:
                idx = list(range(n))
            else:
                w = weights[b, h, :n - recent]
                rank = sorted(range(n - recent), key=lambda j: (not np.isnan(w[j]), -w[j] if not np.isnan(w[j]) else 0, j))
                idx = sorted(rank[:keep - recent] + list(range(n - recent, n)))
            kept[b, h, :len(idx)] = idx
            new_w[b, h, :len(idx)] = weights[b, h, idx]
            for f in range(0, len(idx), sb):
                part = idx[f:f + sb]
                pg, at = int(new_table[b, f // page]), f % page
                for key in ("k", "v"):
                    sc = [src[key + "s"][int(table[b, j // page]), h, j % page // sb] for j in part]
                    top = max(sc)
                    for i, j in enumerate(part):
                        byte = src[key][int(table[b, j // page]), h, j % page]
                        cache[key][pg, h, at + i] = byte if sc[i] == top else to_e4m3(_E4M3[byte] * sc[i] / top)
                    cache[key + "s"][pg, h, at // sb] = top
    return new_lens, new_w, kept
