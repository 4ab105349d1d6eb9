"""fa_cache_append: every element and bound of the cache."""
import numpy as np
import pytest
import torch

from oracle import paged as op
from tests.paged_common import DEV, assert_same, bf16, copy, f64, ints, ok, random_pages, table_of, to_gpu

pytestmark = pytest.mark.gpu

# (Hkv, N, d, page, block (0: no bounds), lens, new)
CASES = [
    (1, 1, 64, 16, 16, [0], [1]),
    (2, 1, 128, 16, 16, [0, 15, 16, 17, 31], None),
    (2, 1, 128, 16, 0, [0, 15, 16, 17, 31], None),
    (2, 5, 128, 16, 8, [0, 7, 8, 30], [5, 5, 0, 2]),
    (3, 37, 64, 20, 4, [0, 3, 19], [37, 1, 36]),
    (3, 37, 64, 20, 0, [0, 3, 19], [37, 1, 36]),
    (1, 100, 128, 64, 32, [0, 31, 33, 64], [100, 99, 0, 50]),
    (2, 129, 64, 128, 128, [0, 127, 200], None),
    (9, 129, 128, 128, 128, [0, 127, 200], None),
    (2, 64, 128, 128, 64, [1, 64], None),
    (1, 300, 128, 256, 128, [0, 5], [300, 77]),
    (2, 50, 64, 48, 24, [23, 24, 25], None),
    (1, 9, 128, 1, 1, [0, 4], None),
    (1, 40, 64, 33, 11, [10, 11], None),
    (1, 3, 64, 96, 96, [95, 90], None),
    (2, 150, 128, 12, 3, [0, 1, 2, 3, 100], None),
    (1, 200, 64, 4, 2, [0, 7], [200, 0]),
    (2, 90, 128, 4, 1, [5, 0], [90, 13]),
    (16, 70, 64, 40, 8, [7, 33, 39], [1, 70, 64]),
    (11, 500, 128, 64, 0, [7, 33], [500, 499]),
]


def _layout(k, v, layout):
    if layout == "bnhd":
        return tuple(t.transpose(1, 2).contiguous().transpose(1, 2) for t in (k, v))
    if layout == "packed":
        kv = torch.stack([k.transpose(1, 2), v.transpose(1, 2)], 2).contiguous()   # [B, N, 2, Hkv, d]
        return kv[:, :, 0].transpose(1, 2), kv[:, :, 1].transpose(1, 2)
    return k, v


@pytest.mark.parametrize("Hkv,N,d,page,block,lens,new", CASES)
@pytest.mark.parametrize("layout", ["bhnd", "bnhd", "packed"])
@pytest.mark.parametrize("turned", [None, (False, 1.0), (True, 1.25)])
def test_append(cuda_lib, Hkv, N, d, page, block, lens, new, layout, turned):
    """Slots that are not written keep their values, padding rows of the new tokens may hold anything; with rotation the
    result is that of fa_rope followed by the append without."""
    fa, B = cuda_lib, len(lens)
    rng = np.random.default_rng(N * 7 + block + d)
    maxp = -(-(max(lens) + N) // page)
    pages = B * maxp + 2
    c = random_pages(N + page, pages, Hkv, page, d, block)
    table = table_of(block, B, maxp, pages)
    k, v = bf16(rng, (B, Hkv, N, d)), bf16(rng, (B, Hkv, N, d), 2.0)
    if new is not None:
        for b in range(B):
            k[b, :, new[b]:] = float("nan")
            v[b, :, new[b]:] = float("inf")
    g = to_gpu(c)
    kd, vd = _layout(k.to(DEV), v.to(DEV), layout)
    extra, want = {}, k
    if turned:
        rot = d if layout == "bhnd" else 32
        turns = fa.rope_table(fa.rope_frequencies(rot)[0])
        pos = None if layout == "bnhd" else ints(rng.integers(0, 1 << 20, (B, N)))
        extra = dict(turns=turns, positions=pos, interleaved=turned[0], magnitude=turned[1])
        at = pos if pos is not None else (ints(lens)[:, None] + torch.arange(N, device=DEV)).int().contiguous()
        want = fa.rope(kd, turns, at, interleaved=turned[0], magnitude=turned[1]).cpu()
    fa.cache_append(kd, vd, g["k"], g["v"], ints(table), ints(lens), None if new is None else ints(new),
                    bounds=g.get("b"), **extra)
    ok(fa)
    op.append(c, table, lens, f64(want), f64(v), new)
    assert_same(g, c)


def test_step_after_step_keeps_the_bounds(cuda_lib):
    """Tokens one by one and in odd chunks end at the same cache as all at once, bounds of untouched blocks included."""
    fa, B, Hkv, d, page, block = cuda_lib, 3, 4, 128, 48, 24
    rng = np.random.default_rng(5)
    lens, N, maxp = [0, 13, 47], 90, 4
    c = random_pages(6, B * maxp, Hkv, page, d, block)
    table = table_of(1, B, maxp, B * maxp)
    k, v = bf16(rng, (B, Hkv, N, d)).to(DEV), bf16(rng, (B, Hkv, N, d)).to(DEV)
    a, b = to_gpu(c), to_gpu(c)
    fa.cache_append(k, v, a["k"], a["v"], ints(table), ints(lens), bounds=a["b"])
    at = 0
    for n in (1, 1, 7, 24, 1, 30, 26):
        fa.cache_append(k[:, :, at:at + n], v[:, :, at:at + n], b["k"], b["v"], ints(table), ints(np.array(lens) + at),
                        bounds=b["b"])
        at += n
    assert at == N
    ok(fa)
    assert all(torch.equal(a[n], b[n]) for n in a)


def test_bounds_of_infinite_and_nan_keys(cuda_lib):
    fa, Hkv, d, page = cuda_lib, 1, 64, 16
    rng = np.random.default_rng(2)
    c = random_pages(3, 2, Hkv, page, d, 8)
    k, v = bf16(rng, (1, Hkv, 16, d)), bf16(rng, (1, Hkv, 16, d))
    k[0, 0, 3, 5], k[0, 0, 9, 7], k[0, 0, 10, 7], k[0, 0, 12, 8] = float("nan"), float("inf"), -float("inf"), -float("nan")
    g = to_gpu(c)
    fa.cache_append(k.to(DEV), v.to(DEV), g["k"], g["v"], ints([[1, 0]]), ints([0]), bounds=g["b"])
    ok(fa)
    op.append(c, np.array([[1, 0]]), [0], f64(k), f64(v))
    assert_same(g, c)
    # a NaN stays while its block grows
    k2 = bf16(rng, (1, Hkv, 1, d))
    g2 = to_gpu(c)
    fa.cache_append(k2.to(DEV), k2.to(DEV), g2["k"], g2["v"], ints([[1, 0]]), ints([5]), bounds=g2["b"])
    ok(fa)
    op.append(c, np.array([[1, 0]]), [5], f64(k2), f64(k2))
    assert_same(g2, c)


def test_bad_lengths_and_pages(cuda_lib):
    """Tokens that do not fit are left out, pages that are not there are not written: both recorded, the rest written."""
    fa, Hkv, d, page, block = cuda_lib, 2, 128, 16, 8
    rng = np.random.default_rng(9)
    c = random_pages(4, 6, Hkv, page, d, block)
    k, v = bf16(rng, (3, Hkv, 20, d)), bf16(rng, (3, Hkv, 20, d))
    for table, lens, new, fits in (([[0, 1], [2, 3], [4, 5]], [20, -3, 40], [20, 5, 4], [12, 5, 0]),
                                   ([[0, 1], [2, 3], [4, 5]], [0, 0, 0], [-1, 21, 3], [0, 20, 3])):
        g = to_gpu(c)
        fa.cache_append(k.to(DEV), v.to(DEV), g["k"], g["v"], ints(table), ints(lens), ints(new), bounds=g["b"])
        assert fa.fa_get_last_device_error()[0] == fa.FA_ERR_INVALID_ARG
        ref = copy(c)
        op.append(ref, np.array(table), np.clip(lens, 0, 32), f64(k), f64(v), fits)
        assert_same(g, ref)
    for bad in (-1, 6, 2 ** 31 - 1):
        g = to_gpu(c)
        fa.cache_append(k.to(DEV), v.to(DEV), g["k"], g["v"], ints([[0, bad], [bad, 3], [4, 5]]), ints([4, 0, 0]),
                        ints([20, 20, 20]), bounds=g["b"])
        assert fa.fa_get_last_device_error()[0] == fa.FA_ERR_INVALID_ARG
        ref = copy(c)
        grown = {n: np.concatenate([ref[n], ref[n][:1]]) for n in ref}      # page 6 takes what is left out
        op.append(grown, np.array([[0, 6], [6, 3], [4, 5]]), [4, 0, 0], f64(k), f64(v), [20, 20, 20])
        assert_same(g, {n: grown[n][:6] for n in grown})


def test_empty_sequences_are_left_alone(cuda_lib):
    fa, Hkv, d, page = cuda_lib, 2, 64, 16
    rng = np.random.default_rng(1)
    c = random_pages(2, 6, Hkv, page, d, 8)
    table = np.array([[0, 3], [1, -1], [-1, -1]], dtype=np.int32)
    k = bf16(rng, (3, Hkv, 4, d))
    for lens, new in (([5, 3, 20], [4, 0, 0]), ([8, 11, 0], [0, 0, 0])):
        g = to_gpu(c)
        fa.cache_append(k.to(DEV), k.to(DEV), g["k"], g["v"], ints(table), ints(lens), ints(new), bounds=g["b"])
        ok(fa)
        ref = copy(c)
        op.append(ref, table, lens, f64(k), f64(k), new)
        assert_same(g, ref)


def test_far_offsets(cuda_lib):
    """Pages whose elements lie beyond 2^32 bytes and 2^31 elements."""
    fa, Hkv, d, page, block = cuda_lib, 8, 128, 256, 32
    pages = (1 << 31) // (Hkv * d * page) + 3
    kp = torch.zeros((pages, Hkv, page, d), dtype=torch.bfloat16, device=DEV)
    vp, bounds = torch.zeros_like(kp), torch.zeros((pages, Hkv, page // block, 2, d), dtype=torch.bfloat16, device=DEV)
    rng = np.random.default_rng(4)
    k, v = (bf16(rng, (1, Hkv, 40, d)).to(DEV) for _ in "kv")
    fa.cache_append(k, v, kp, vp, ints([[pages - 1]]), ints([100]), bounds=bounds)
    ok(fa)
    assert torch.equal(kp[pages - 1, :, 100:140], k[0]) and torch.equal(vp[pages - 1, :, 100:140], v[0])
    assert torch.equal(bounds[pages - 1, :, 4, 0], k[0, :, 28:].amin(1)) and not bounds[:pages - 1].any()
    assert int(kp.count_nonzero()) == int(k.count_nonzero())
