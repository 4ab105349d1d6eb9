"""fa_select_blocks against float64: the very same blocks."""
import numpy as np
import pytest
import torch

from oracle import paged as op
from tests.paged_common import DEV, bf16, f64, ints, ok, table_of

pytestmark = pytest.mark.gpu


def _bounds(rng, pages, Hkv, per, d):
    mean = rng.standard_normal((pages, Hkv, per, 1, d))
    x = np.concatenate([mean - rng.random((pages, Hkv, per, 1, d)), mean + rng.random((pages, Hkv, per, 1, d))], 3)
    return f64(torch.from_numpy(x).to(torch.bfloat16))


def _run(fa, q, bounds, table, lens, block, keep, first, recent):
    out = fa.select_blocks(q.to(DEV), torch.from_numpy(np.ascontiguousarray(bounds)).to(torch.bfloat16).to(DEV), ints(table),
                           ints(lens), block=block,
                           keep=keep, first=first, recent=recent)
    return out.cpu().numpy()


# (lens, Hkv, G, Nq, d, block, blocks per page, keep, first, recent)
CASES = [
    ([1], 1, 1, 1, 64, 16, 1, 1, 0, 0),
    ([0, 5, 16, 17, 100], 2, 4, 1, 128, 16, 1, 3, 0, 1),
    ([1000, 999, 0, 3], 2, 1, 1, 128, 8, 4, 20, 1, 2),
    ([1000, 500], 1, 8, 4, 64, 4, 5, 33, 2, 3),
    ([700, 701], 3, 5, 3, 128, 1, 7, 100, 0, 0),
    ([4096], 1, 4, 1, 128, 8, 8, 512, 0, 1),           # all stay
    ([4097], 1, 4, 1, 128, 8, 8, 512, 0, 1),           # all but one stay
    ([9000], 2, 3, 1, 64, 4, 16, 1, 0, 0),             # one stays
    ([9000], 2, 2, 2, 128, 4, 16, 7, 3, 4),            # none but the fixed ones
    ([40000, 17], 1, 16, 3, 64, 4, 8, 1000, 1, 2),     # 10000 blocks; 48 rows
    ([5000, 4999], 2, 4, 16, 128, 128, 2, 9, 1, 1),
]


@pytest.mark.parametrize("lens,Hkv,G,Nq,d,block,per,keep,first,recent", CASES)
def test_select(cuda_lib, lens, Hkv, G, Nq, d, block, per, keep, first, recent):
    B = len(lens)
    rng = np.random.default_rng(sum(lens) + d + keep)
    maxp = -(-max(lens) // (block * per))
    pages = B * maxp + 2
    bounds, table = _bounds(rng, pages, Hkv, per, d), table_of(d, B, maxp, pages)
    q = bf16(rng, (B, Hkv * G, Nq, d))
    got = _run(cuda_lib, q, bounds, table, lens, block, keep, first, recent)
    ok(cuda_lib)
    assert np.array_equal(got, op.select(f64(q), bounds, table, lens, block, keep, first, recent))


def test_three_dimensional_queries(cuda_lib):
    rng = np.random.default_rng(1)
    bounds, q = _bounds(rng, 40, 2, 2, 64), bf16(rng, (3, 4, 64))
    table, lens = table_of(2, 3, 10, 40), [300, 280, 160]
    got = _run(cuda_lib, q, bounds, table, lens, 16, 5, 1, 1)
    ok(cuda_lib)
    assert np.array_equal(got, op.select(f64(q)[:, :, None], bounds, table, lens, 16, 5, 1, 1))


@pytest.mark.parametrize("n,keep", [(300, 20), (3000, 700)])
@pytest.mark.parametrize("rows", [1, 6])
def test_equal_scores_go_by_index(cuda_lib, n, keep, rows):
    """Whole numbers, so that every score is exact and many are equal; blocks that are copies of one another."""
    rng = np.random.default_rng(n + rows)
    d, per = 128, 4
    bounds = rng.integers(-2, 3, (n // per, 1, per, 2, d)).astype(np.float64)
    bounds[..., 4:] = 0
    table = np.arange(n // per, dtype=np.int32)[None]
    q = torch.from_numpy(rng.integers(-1, 2, (1, rows, 1, d)).astype(np.float32)).to(torch.bfloat16)
    got = _run(cuda_lib, q, bounds, table, [n * 8], 8, keep, 0, 1)
    ok(cuda_lib)
    assert np.array_equal(got, op.select(f64(q), bounds, table, [n * 8], 8, keep, 0, 1))
    got = _run(cuda_lib, q, np.zeros_like(bounds), table, [n * 8], 8, keep, 2, 3)
    want = list(range(keep - 3)) + [n - 3, n - 2, n - 1]
    assert np.array_equal(got[0, 0], want)


@pytest.mark.parametrize("d", [64, 128])
def test_scores_closer_than_fp32_tells_apart(cuda_lib, d):
    """Scores that differ by less than the rounding of an fp32 sum, in an order that such sums do not keep: large terms
    that cancel in every block, and small ones that decide."""
    rng = np.random.default_rng(d)
    n, per = 256, 4
    x = np.zeros((n, 2, d))
    big = rng.integers(1, 128, (n, d // 4)) * 2.0 ** 10
    x[:, :, 0:d // 4] = big[:, None]
    x[:, :, d // 2:d // 2 + d // 4] = -big[:, None]
    x[:, :, d // 4:d // 2] = rng.integers(-127, 128, (n, 1, d // 4)) * 2.0 ** -18
    perm = rng.permutation(d)                                # the same shuffle in every block
    bounds = x[:, :, perm].reshape(n // per, 1, per, 2, d)
    assert np.array_equal(bounds, f64(torch.from_numpy(bounds).to(torch.bfloat16)))
    q = torch.ones((1, 1, 1, d), dtype=torch.bfloat16)
    table = rng.permutation(n // per).astype(np.int32)[None]
    want = op.select(f64(q), bounds, table, [n * 16], 16, 40, 0, 0)
    got = _run(cuda_lib, q, bounds, table, [n * 16], 16, 40, 0, 0)
    ok(cuda_lib)
    assert np.array_equal(got, want)


def test_infinite_and_nan_bounds(cuda_lib):
    """A NaN, or an infinity that meets a zero, counts as largest; scores beyond fp32 keep their order."""
    rng = np.random.default_rng(8)
    d, n, per = 128, 200, 4
    base = _bounds(rng, n // per, 1, per, d)
    q = bf16(rng, (1, 2, 1, d))
    q[0, 0, 0, 7] = 0.0
    table = rng.permutation(n // per).astype(np.int32)[None]
    for at, value in (((3, 0, 1, 0, 5), np.nan), ((9, 0, 2, 1, 7), np.inf), ((4, 0, 0, 0, 9), -np.inf)):
        b = base.copy()
        b[at] = value
        got = _run(cuda_lib, q, b, table, [n * 4], 4, 12, 1, 1)
        ok(cuda_lib)
        assert np.array_equal(got, op.select(f64(q), b, table, [n * 4], 4, 12, 1, 1)), value
    huge = f64(torch.from_numpy(base * 2.0 ** 120).to(torch.bfloat16))
    big_q = (q.float() * 2.0 ** 30).to(torch.bfloat16)
    got = _run(cuda_lib, big_q, huge, table, [n * 4], 4, 12, 0, 1)
    assert np.array_equal(got, op.select(f64(big_q), huge, table, [n * 4], 4, 12, 0, 1))
    tiny = f64(torch.from_numpy(base * 2.0 ** -100).to(torch.bfloat16))
    small_q = (q.float() * 2.0 ** -40).to(torch.bfloat16)
    got = _run(cuda_lib, small_q, tiny, table, [n * 4], 4, 12, 0, 1)
    assert np.array_equal(got, op.select(f64(small_q), tiny, table, [n * 4], 4, 12, 0, 1))


def test_bad_lengths_and_pages(cuda_lib):
    """Clamped, read as zeros, and recorded."""
    fa = cuda_lib
    rng = np.random.default_rng(3)
    bounds, q = _bounds(rng, 50, 1, 2, 64), bf16(rng, (2, 2, 1, 64))
    table = table_of(2, 2, 20, 50)
    got = _run(fa, q, bounds, table, [-4, 700], 16, 6, 1, 1)
    assert fa.fa_get_last_device_error()[0] == fa.FA_ERR_INVALID_ARG
    assert np.array_equal(got, op.select(f64(q), bounds, table, [0, 640], 16, 6, 1, 1))
    for bad in (-1, 50, 2 ** 31 - 1):
        t = table.copy()
        t[0, 3] = bad
        got = _run(fa, q, bounds, t, [600, 640], 16, 6, 1, 1)
        assert fa.fa_get_last_device_error()[0] == fa.FA_ERR_INVALID_ARG
        t[0, 3] = 50
        grown = np.concatenate([bounds, np.zeros_like(bounds[:1])])
        assert np.array_equal(got, op.select(f64(q), grown, t, [600, 640], 16, 6, 1, 1))


# (lens, Hkv, G, d, blocks per page, pages of the table, keep): scores in shared memory and in the workspace, CTAs with an SM to
# themselves and two to an SM, one batch of blocks per warp and many, tables far wider than the lengths
WIDE = [
    ([1 << 15] + [40] * 39, 4, 4, 128, 8, 1024, 300),       # 160 pairs, 8192 blocks of 4
    ([4 * 12000] + [40, 0, 9000] * 13, 4, 9, 64, 8, 1500, 900),  # 12000 blocks, 9 rows
    ([4 * 13000 - 1] + [70] * 79, 2, 8, 128, 8, 2500, 64),  # 20000 blocks in the table
    ([4 * 60000], 1, 2, 64, 16, 3750, 2000),                # 60000 blocks
    ([4 * 60000, 333], 1, 1, 128, 16, 3760, 1),
    ([2000] * 40, 8, 1, 64, 4, 125, 17),                    # 320 pairs
    ([3000, 1500], 2, 80, 64, 8, 100, 50),                  # 80 rows: two tiles of them
    ([900, 1500, 0, 30] * 10, 8, 70, 128, 8, 50, 50),
]


@pytest.mark.parametrize("lens,Hkv,G,d,per,maxp,keep", WIDE)
def test_wide_tables_and_many_sequences(cuda_lib, lens, Hkv, G, d, per, maxp, keep):
    """Pages that many sequences share, so that scores repeat within a sequence too."""
    rng = np.random.default_rng(maxp + keep)
    pages = 700
    bounds, B = _bounds(rng, pages, Hkv, per, d), len(lens)
    table = rng.integers(0, pages, (B, maxp)).astype(np.int32)
    q = bf16(rng, (B, Hkv * G, 1, d))
    got = _run(cuda_lib, q, bounds, table, lens, 4, keep, 0, 1)
    ok(cuda_lib)
    assert np.array_equal(got, op.select(f64(q), bounds, table, lens, 4, keep, 0, 1))
