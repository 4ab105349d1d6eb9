"""The float64 oracle of the paged bf16 cache against independent statements of what it computes."""
import numpy as np

from oracle import naive
from oracle import paged as op


def _cache(rng, lens, Hkv, page, d, block=0):
    B, maxp = len(lens), -(-max(lens) // page)
    c = {n: np.zeros((B * maxp, Hkv, page, d)) for n in ("k", "v")}
    if block:
        c["b"] = np.zeros((B * maxp, Hkv, page // block, 2, d))
    table = rng.permutation(B * maxp).reshape(B, maxp)
    k, v = rng.standard_normal((2, B, Hkv, max(lens), d))
    op.append(c, table, [0] * B, k, v, lens)
    return c, table, k, v


def test_attention_over_everything_is_plain_attention():
    rng = np.random.default_rng(0)
    lens, Hkv, G, Nq, d = [33, 7], 2, 3, 4, 16
    c, table, k, v = _cache(rng, lens, Hkv, 8, d)
    q = rng.standard_normal((2, Hkv * G, Nq, d))
    o, lse = op.attend(q, c, table, lens, 0.3)[:2]
    for b, n in enumerate(lens):
        rep = lambda x: np.repeat(x[b:b + 1, :, :n], G, 1)
        want, wlse = naive.forward(q[b:b + 1], rep(k), rep(v), 0.3, True)
        assert np.allclose(o[b], want[0], atol=1e-12) and np.allclose(lse[b], wlse[0], atol=1e-12)


def test_blocks_in_any_order_and_bounds():
    rng = np.random.default_rng(1)
    lens, Hkv, d, page, block = [45, 20], 2, 8, 12, 4
    c, table, k, v = _cache(rng, lens, Hkv, page, d, block)
    q = rng.standard_normal((2, Hkv * 2, 1, d))
    lists = np.stack([np.stack([rng.permutation(12) for _ in range(Hkv)]) for _ in range(2)])
    some = op.attend(q, c, table, lens, 1.0, op.tokens_of(lists, block))
    assert np.allclose(some[0], op.attend(q, c, table, lens, 1.0)[0], atol=1e-12)
    for b, n in enumerate(lens):
        for h in range(Hkv):
            s = op.scores(q, c["b"], table, -(-n // block), b, h)
            for j in range(len(s)):
                keys = k[b, h, j * block:min(n, (j + 1) * block)]
                at = c["b"][table[b][j * block // page], h, j * block % page // block]
                assert np.array_equal(at[0], keys.min(0)) and np.array_equal(at[1], keys.max(0))
                assert s[j] >= (keys @ q[b, 2 * h:2 * h + 2, 0].T).max() - 1e-12


def test_selection():
    rng = np.random.default_rng(2)
    bounds = rng.standard_normal((10, 1, 2, 2, 4))
    bounds.sort(3)
    table = np.arange(10)[None]
    q = rng.standard_normal((1, 1, 1, 4))
    s = op.scores(q, bounds, table, 20, 0, 0)
    got = op.select(q, bounds, table, [20 * 4 - 1], 4, 7, 2, 3)[0, 0]
    mid = np.argsort(-s[2:17], kind="stable")[:2] + 2
    assert list(got) == sorted([0, 1, 17, 18, 19] + list(mid))
    assert list(op.select(q, bounds, table, [17], 4, 7, 2, 3)[0, 0]) == [0, 1, 2, 3, 4, -1, -1]
