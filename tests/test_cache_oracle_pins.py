"""Pins of the 8-bit cache's fp64 oracle: closed forms, invariants, torch's own
e4m3 conversion, and the plain attention oracle."""
import math

import numpy as np
import pytest
import torch

from oracle import cache as oc
from oracle import naive


def test_e4m3_rounding_is_torchs():
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.standard_normal(20000) * 10.0 ** rng.uniform(-4, 3, 20000), oc._E4M3[~np.isnan(oc._E4M3)],
                        (oc._E4M3[:126] + oc._E4M3[1:127]) / 2]).astype(np.float32)  # values, and every tie
    x = np.clip(x, -448, 448)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(oc.to_e4m3(x.astype(np.float64)), want)
    assert list(oc.to_e4m3(np.array([np.inf, -np.inf, np.nan, 1e9]))) == [0x7E, 0xFE, 0x7F, 0x7E]


def test_scale_is_the_smallest_power_of_two():
    assert oc.scale_for(0.0) == 2.0 ** -126
    for m, s in ((448.0, 1.0), (449.0, 2.0), (1.0, 2.0 ** -8), (1.75, 2.0 ** -8), (1.7578125, 2.0 ** -7),
                 (3.3895e38, 2.0 ** 120)):
        assert oc.scale_for(m) == s, m


def test_rope_rotates():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((2, 3, 5, 64))
    f = 10000.0 ** (-2.0 * np.arange(16) / 32)
    pos = rng.integers(0, 100000, (2, 5))
    for inter in (False, True):
        y = oc.rope(x, pos, f, inter)
        assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1))                      # a rotation
        assert np.array_equal(y[..., 32:], x[..., 32:])
        assert np.allclose(oc.rope(y, pos, f, inter, inverse=True), x)              # undone
        # products depend on the distance only
        a, b = x[:, :, :1], x[:, :, 1:2]
        dot = lambda p, q: (oc.rope(a, p, f, inter) * oc.rope(b, q, f, inter)).sum(-1)
        p = np.array([[7], [11]])
        assert np.allclose(dot(p, p + 5), dot(p + 1000, p + 1005))
    z = oc.rope(np.array([[[[1.0, 0.0]]]]), np.array([[3]]), [math.pi / 6])
    assert np.allclose(z, [[[[0.0, 1.0]]]])
    z = oc.rope(np.array([[[[1.0, 2.0, 3.0, 4.0]]]]), np.array([[1]]), [math.pi / 2, math.pi], True, 2.0)
    assert np.allclose(z, [[[[-4.0, 2.0, -6.0, -8.0]]]])


def _cache(seed, pages, Hkv, page, sb, d):
    rng = np.random.default_rng(seed)
    c = {n: oc.to_e4m3(rng.standard_normal((pages, Hkv, page, d)) * 100) for n in ("k", "v")}
    for n in ("ks", "vs"):
        c[n] = 2.0 ** rng.integers(-9, -5, (pages, Hkv, page // sb)).astype(np.float64)
    return c


def test_append_stores_values_within_half_a_step_whatever_the_order():
    rng = np.random.default_rng(2)
    x = np.sign(rng.standard_normal((1, 2, 37, 64))) * rng.uniform(0.5, 200, (1, 2, 37, 64))
    x = torch.from_numpy(x).to(torch.bfloat16).double().numpy()
    table = np.array([[2, 0, 1]])
    once, one = _cache(3, 3, 2, 16, 8, 64), _cache(3, 3, 2, 16, 8, 64)
    oc.append(once, table, [0], x, x)
    for t in range(37):
        oc.append(one, table, [t], x[:, :, t:t + 1], x[:, :, t:t + 1])
    for h in range(2):
        K, V = oc.tokens(once, table[0], 37, h)
        assert (np.abs(K - x[0, h]) <= 2.0 ** -4 * np.abs(x[0, h])).all() and np.array_equal(K, V)
        K1, _ = oc.tokens(one, table[0], 37, h)
        assert np.array_equal(K, K1)   # powers of two: rescaling moved exponents only
    for n in ("k", "v", "ks", "vs"):
        assert np.array_equal(once[n], one[n])


def test_decode_is_the_plain_attention():
    c = _cache(4, 7, 2, 16, 4, 64)
    table = np.random.default_rng(5).permutation(7)[:6].reshape(2, 3)
    lens = [41, 20]
    q = np.random.default_rng(6).standard_normal((2, 6, 3, 64))
    w = np.zeros((2, 2, 48))
    o, lse, A, PV, T = oc.decode(q, c, table, lens, 0.125, w)
    for b in range(2):
        for h in range(6):
            K, V = oc.tokens(c, table[b], lens[b], h // 3)
            ro, rl = naive.forward(q[b, h], K, V, 0.125, causal=True)
            assert np.allclose(o[b, h], ro) and np.allclose(lse[b, h], rl)
        assert np.allclose(w[b].sum(-1), 9.0)          # three heads times three tokens, each summing to one
        assert (w[b, :, lens[b]:] == 0).all()
    o, lse, *_ = oc.decode(q, c, table, [0, 2], 0.125)
    assert (o[0] == 0).all() and np.isneginf(lse[0]).all()
    assert np.isneginf(lse[1, :, 0]).all() and np.isfinite(lse[1, :, 1:]).all()


def test_evict_keeps_the_heavy_and_the_recent():
    c = _cache(7, 8, 1, 4, 2, 64)
    table, new = np.array([[5, 1, 6, 2]]), np.array([[0, 7]])
    w = np.array([[[3, 9, 1, 9, -0.0, 0.0, 2, 9, np.nan, 4, 0, 0, 5, 8, 8, 8]]], dtype=np.float32)
    before = [oc.tokens(c, table[0], 13, 0)]
    lens, nw, kept = oc.evict(c, table, np.array([13]), w, new, 6, 2)
    assert list(kept[0, 0]) == [1, 3, 7, 8, 11, 12, -1, -1] and lens[0] == 6   # nan, three nines, the last two
    K, V = oc.tokens(c, new[0], 6, 0)
    idx = kept[0, 0, :6]
    assert (np.abs(K - before[0][0][idx]) <= 2.0 ** -4 * np.abs(before[0][0][idx]) + 2.0 ** -18).all()
    assert list(nw[0, 0, 4:]) == [0, 5, 0, 0]
    c2 = _cache(7, 8, 1, 4, 2, 64)
    _, _, kept = oc.evict(c2, table, np.array([13]), w * 0, new, 6, 0)
    assert list(kept[0, 0, :6]) == [0, 1, 2, 3, 4, 8]  # 0 * nan = nan first, then ties by index
    _, _, kept = oc.evict(c2, table, np.array([3]), w, new, 6, 2)
    assert list(kept[0, 0]) == [0, 1, 2] + [-1] * 5
