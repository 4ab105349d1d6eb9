"""What the tests of the paged bf16 cache share: inputs, and bounds from the arithmetic."""
import numpy as np
import torch

from tests.cache_fp8_common import DEV, bf16, f64, ints, table_of  # noqa: F401


def ok(fa):
    st, detail = fa.fa_get_last_device_error()
    assert st == 0, detail


def random_pages(seed, pages, Hkv, page, d, block=0):
    """A full cache as the oracle's dict: every value a bf16 one."""
    rng = np.random.default_rng(seed)
    c = {n: f64(bf16(rng, (pages, Hkv, page, d), 0.3)) for n in ("k", "v")}
    if block:
        x = c["k"].reshape(pages, Hkv, page // block, block, d)
        c["b"] = np.stack([x.min(3), x.max(3)], 3)
    return c


def to_gpu(c):
    return {n: torch.from_numpy(c[n]).to(torch.bfloat16).to(DEV) for n in c}


def copy(c):
    return {n: c[n].copy() for n in c}


def assert_same(g, c):
    """Values equal; NaN is NaN."""
    for n in c:
        a, b = f64(g[n]), c[n]
        bad = np.argwhere((a != b) & ~(np.isnan(a) & np.isnan(b)))
        assert bad.size == 0, "%s: %d values differ, first at %s" % (n, len(bad), bad[0])


def check_rows(o, lse, ref, weight, what=""):
    """ref: oracle.paged.attend's answer; weight: the relative error of a softmax weight in the value product (2^-16 as a
    pair of bf16, whose second one leaves 2^-8 2^-8 at most; 2^-8 as one).

    Scores: the products of bf16 numbers are exact, so a score's error is the fp32 summation's: 8 steps of 16 products,
    each off by at most 2^-22 of the largest partial sum, and three roundings of 2^-24, all of at most A = max_j sum_i
    |q_i k_ij| scale: below 2^-18 A.  A weight p is off by a factor exp(2 eps) (score and LSE) and the hardware 2^x (2^-22):
    rel = 2^-17 A + 2^-21.  O: the weight's rounding and rel, fp32 sums and the merge of parts (2^-17 of sum p |v| in
    all), and the result's own bf16 rounding (2^-8 |O|).
    """
    o_ref, lse_ref, A, PV = ref
    o, lse = f64(o).reshape(o_ref.shape), f64(lse).reshape(lse_ref.shape)
    none = np.isneginf(lse_ref)
    assert np.array_equal(np.isneginf(lse), none), "%s: rows without keys" % what
    assert (o[none] == 0).all(), what
    rel = 2.0 ** -17 * A + 2.0 ** -21
    bound = 2.0 ** -8 * np.abs(o_ref) + (weight + rel[..., None] + 2.0 ** -17) * PV
    over = np.abs(o - o_ref) - bound
    assert over.max() <= 0, "%s: O exceeds its bound by %g at %s" % (what, over.max(),
                                                                     np.unravel_index(over.argmax(), over.shape))
    fin = ~none
    zero = lambda x: np.where(none, 0, x)
    err = np.abs(zero(lse) - zero(lse_ref))[fin] - (rel + 2.0 ** -21 * np.abs(zero(lse_ref)))[fin]
    assert not err.size or err.max() <= 0, "%s: LSE exceeds its bound by %g" % (what, err.max())
