"""The rotation's angles: the table's entries against integer arithmetic, the kernel's cosines and sines to their last
bits, and the gradient as the transpose."""
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

import exact_tiled_attention_21_gb300 as fa
from tests.cache_fp8_common import bf16, f64, ints

PI = Fraction("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")
FREQS = [1.0, 0.75, 10000.0 ** -0.5, 10000.0 ** (-126.0 / 128), 1e-9, 3.0, 7.5, 123456.789, 2.0 ** -40]


def test_table_is_the_quotient_in_double_precision():
    """turns = inv_freq / (2 pi) as a double has it (the division's half step, 2^-53, and 2 pi's own: 2^-52 of the
    quotient), rounded to 2^-65; negative frequencies turn the other way by exactly as much."""
    got = fa.fa_rope_table(FREQS)
    for t, x in zip(got, FREQS):
        exact = Fraction(x) / (2 * PI)
        off = Fraction(t, 1 << 64) - (exact - math.floor(exact))
        off = min(abs(off), 1 - abs(off))
        assert off <= exact / (1 << 52) + Fraction(1, 1 << 65), x
    back = fa.fa_rope_table([-x for x in FREQS])
    assert [(a + b) % (1 << 64) for a, b in zip(got, back)] == [0] * len(FREQS)


def _turned(p, freq):
    """cos and sin of p * freq, reduced exactly."""
    a = Fraction(int(p)) * Fraction(float(freq))
    r = float(a - round(a / (2 * PI)) * 2 * PI)
    return math.cos(r), math.sin(r)


@pytest.mark.gpu
@pytest.mark.parametrize("far", [0, 131072, 2 ** 26])
@pytest.mark.parametrize("inter", [False, True])
def test_cosines_and_sines_to_their_last_bits(cuda_lib, inter, far):
    """x1 cos - x2 sin for bf16 x1, x2 whose ratio is nearest the tangent: the terms cancel to about 2^-15, so the
    result's bf16 rounding is as small as an error of 2^-23 in cos or sin.  cos and sin are within 2^-23.9; the product
    and the sum round by 2^-24 of the product and of the result; the table's part is 2^-52 of the angle and 2^-33
    (2^-65 turn at these positions)."""
    d, N = 64, 96
    rng = np.random.default_rng(far + inter)
    freq = 10000.0 ** (-2.0 * np.arange(32) / 64)
    pos = (rng.integers(-far, far + 1, N) if far else np.arange(N)).astype(np.int32)
    cs = np.array([[_turned(p, f) for f in freq] for p in pos])             # [N, 32, 2]
    c, s = cs[..., 0], cs[..., 1]
    m = np.arange(128, 256)
    x1, x2 = np.zeros((N, 32)), np.zeros((N, 32))
    for n in range(N):
        for i in range(32):
            big, small = max(abs(c[n, i]), abs(s[n, i])), min(abs(c[n, i]), abs(s[n, i]))
            want = m * max(small, 2.0 ** -20) / big                          # the other one's size for each mantissa
            e = np.floor(np.log2(want)) - 7
            near = np.rint(want / 2.0 ** e) * 2.0 ** e
            at = np.argmin(np.abs(near * big - m * small) / m)
            pair = (near[at], m[at]) if abs(c[n, i]) >= abs(s[n, i]) else (m[at], near[at])
            x1[n, i], x2[n, i] = pair[0], pair[1] * (1 if c[n, i] * s[n, i] >= 0 else -1)
    x = np.zeros((1, 2, N, d))                                               # head 1: y2 cancels instead
    lo, hi = (slice(0, d, 2), slice(1, d, 2)) if inter else (slice(0, 32), slice(32, d))
    x[0, 0, :, lo], x[0, 0, :, hi] = x1, x2
    x[0, 1, :, lo], x[0, 1, :, hi] = -x2, x1
    xb = torch.from_numpy(x).to(torch.bfloat16)
    assert np.array_equal(f64(xb), x)                                        # the pairs are bf16
    y = f64(cuda_lib.rope(xb.cuda(), cuda_lib.rope_table(freq), ints(pos[None]), inter))
    angle = np.abs(pos[:, None] * freq) * 2.0 ** -52 + 2.0 ** -33
    for head, part, want in ((0, lo, x1 * c - x2 * s), (1, hi, x1 * c - x2 * s)):
        size = np.abs(x1) + np.abs(x2)
        bound = size * (2.0 ** -23.9 + angle) + 2.0 ** -24 * np.maximum(np.abs(x1), np.abs(x2)) + 2.0 ** -8 * np.abs(want)
        assert np.median(np.abs(want) / size) < 2.0 ** -14                   # they do cancel
        err = np.abs(y[0, head][:, part] - want) / bound
        assert err.max() <= 1, "%g times the bound" % err.max()


def _adjoint(g, jv, dx, v):
    """<g, J v> = <J^T g, v>, J v and dx = J^T g each rounded to bf16 (half a step: 2^-8 of the element)."""
    lhs, rhs = (g * jv).sum(), (dx * v).sum()
    return abs(lhs - rhs) <= 2.0 ** -8 * ((np.abs(g) * np.abs(jv)).sum() + (np.abs(dx) * np.abs(v)).sum())


@pytest.mark.gpu
@pytest.mark.parametrize("inter", [False, True])
def test_gradient_is_the_transpose(cuda_lib, inter):
    """With v = J^T g both sides are |J^T g|^2, far above what the roundings allow: no gradient, another sign of the
    angle and a missing magnitude fail."""
    rng = np.random.default_rng(8)
    table = cuda_lib.rope_table(10000.0 ** (-2.0 * np.arange(32) / 64))
    g = bf16(rng, (2, 3, 40, 64), 0.0).cuda()
    pos = ints(rng.integers(0, 9000, (2, 40)))
    dx = cuda_lib.rope(g, table, pos, inter, 1.5, inverse=True)
    jv = cuda_lib.rope(dx, table, pos, inter, 1.5)
    assert _adjoint(f64(g), f64(jv), f64(dx), f64(dx))
    wrong = {"zero": dx * 0, "negative": -dx, "other sign": cuda_lib.rope(g, table, pos, inter, 1.5),
             "no magnitude": cuda_lib.rope(g, table, pos, inter, 1.0, inverse=True)}
    for what, bad in wrong.items():
        assert not _adjoint(f64(g), f64(jv), f64(bad), f64(dx)), what
    # and against differences: J v from two rotations of points that bf16 holds, each rounded by 2^-8 of itself
    x = torch.zeros_like(dx)
    x[...] = dx * 0.5
    step = (x + dx)
    v = f64(step) - f64(x)
    a, b = f64(cuda_lib.rope(step, table, pos, inter, 1.5)), f64(cuda_lib.rope(x, table, pos, inter, 1.5))
    slack = 2.0 ** -8 * ((np.abs(f64(g)) * (np.abs(a) + np.abs(b))).sum() + (np.abs(f64(dx)) * np.abs(v)).sum())
    lhs, rhs = (f64(g) * (a - b)).sum(), (f64(dx) * v).sum()
    assert abs(lhs - rhs) <= slack and slack < 0.1 * abs(rhs)
