"""What the GPU tests of rotary positions and the 8-bit cache share: inputs, and bounds from the arithmetic."""
import numpy as np
import torch

from oracle import cache as oc

DEV = torch.device("cuda", 0)


def bf16(rng, shape, spread=1.0):
    x = rng.standard_normal(shape) * np.exp(spread * rng.standard_normal(shape[:-1] + (1,)))
    return torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16)


def f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def random_cache(seed, pages, Hkv, page, sb, d):
    """A full cache whose blocks differ in size by powers of two (oracle's dict)."""
    rng = np.random.default_rng(seed)
    c = {n: oc.to_e4m3(rng.standard_normal((pages, Hkv, page, d)) * 130.0) for n in ("k", "v")}
    for n in ("ks", "vs"):
        c[n] = 2.0 ** rng.integers(-9, -4, (pages, Hkv, page // sb)).astype(np.float64)
    return c


def table_of(seed, B, maxp, pages):
    return np.random.default_rng(seed).permutation(pages)[:B * maxp].reshape(B, maxp).astype(np.int32)


def to_gpu(c):
    return {n: torch.from_numpy(c[n] if n in ("k", "v") else c[n].astype(np.float32)).to(DEV) for n in c}


def args(g):
    return g["k"], g["v"], g["ks"], g["vs"]


def ints(v):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(v, dtype=np.int32))).to(DEV)


def copy(c):
    return {n: c[n].copy() for n in c}


def assert_same_cache(g, c, what=""):
    """Bytes and scales equal; NaN bytes (0x7F / 0xFF) are the same value."""
    for n in ("k", "v"):
        a, b = g[n].cpu().numpy(), c[n]
        nan = ((a & 0x7F) == 0x7F) & ((b & 0x7F) == 0x7F)
        bad = np.argwhere((a != b) & ~nan)
        assert bad.size == 0, "%s %s: %d bytes differ, first at %s" % (what, n, len(bad), bad[0])
    for n in ("ks", "vs"):
        a = g[n].cpu().numpy().astype(np.float64)
        assert np.array_equal(a, c[n]), "%s %s: scales differ at %s" % (what, n, np.argwhere(a != c[n])[:3])


def check_decode(o, lse, ref, w=None, w_ref=None, what=""):
    """ref: oracle.cache.decode's answer.

    Scores: q is exact in fp16 after its power of two (|q| within 2^28 of the row's largest), K exact, so a score's
    error is the fp32 summation's: 8 steps of 16 products, each step off by at most 2^-22 of the largest partial sum,
    and three roundings of 2^-24, all of at most A = max_j sum_i |q_i k_ij| scale: eps = 2^-18.9 A, below 2^-18 A.
    A weight p is off by a factor exp(2 eps) (score and LSE) and the hardware 2^x (2^-22): rel = 2^-17 A + 2^-21.
    O: p's rounding to fp16 (2^-11 relative, or 2^-25 of the row's largest p vs below fp16's normal range: T 2^-25),
    rel, and the result's own bf16 rounding (2^-8 |O|), with fp32 sums (2^-18 of sum p |v|).
    """
    o_ref, lse_ref, A, PV, T = ref
    o, lse = f64(o).reshape(o_ref.shape), f64(lse).reshape(lse_ref.shape)
    none = np.isneginf(lse_ref)
    assert np.array_equal(np.isneginf(lse), none), "%s: rows without keys" % what
    assert (o[none] == 0).all(), what
    rel = 2.0 ** -17 * A + 2.0 ** -21
    bound = 2.0 ** -8 * np.abs(o_ref) + (2.0 ** -11 + rel[..., None] + 2.0 ** -18) * PV + 2.0 ** -25 * T
    over = np.abs(o - o_ref) - bound
    assert over.max() <= 0, "%s: O exceeds its bound by %g at %s" % (what, over.max(), np.unravel_index(over.argmax(), over.shape))
    fin = ~none
    err = np.abs(np.where(none, 0, lse) - np.where(none, 0, lse_ref))[fin] - (rel + 2.0 ** -22 * np.abs(np.where(none, 0, lse_ref)))[fin]
    assert not err.size or err.max() <= 0, "%s: LSE exceeds its bound by %g" % (what, err.max())
    if w is not None:
        r = rel.max() if rel.size else 0.0
        over = np.abs(f64(w) - w_ref) - ((r + 2.0 ** -20) * np.abs(w_ref) + 1e-30)
        assert over.max() <= 0, "%s: weights exceed their bound by %g" % (what, over.max())
