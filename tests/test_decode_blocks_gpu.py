"""fa_decode_blocks against float64."""
import math

import numpy as np
import pytest
import torch

from oracle import paged as op
from tests.paged_common import DEV, bf16, check_rows, copy, f64, ints, ok, random_pages, table_of, to_gpu

pytestmark = pytest.mark.gpu
PAIR = 2.0 ** -16


def _lists(rng, lens, Hkv, block, keep, order="any"):
    """Distinct blocks of each sequence, any order, some places skipped; the block that holds the last token among them."""
    out = np.full((len(lens), Hkv, keep), -1, dtype=np.int32)
    for b, n in enumerate(lens):
        many = -(-n // block)
        for h in range(Hkv):
            look = min(keep, many)                       # the entries that are looked at
            take = look if order == "all" else rng.integers(min(1, look), look + 1)
            if take == 0:
                continue
            mine = rng.permutation(many)[:take]
            if many - 1 not in mine:
                mine[0] = many - 1
            at = np.sort(rng.permutation(look)[:take])
            out[b, h, at] = rng.permutation(mine)
    return out


# (lens, Hkv, G, Nq, d, page, block, keep)
CASES = [
    ([1], 1, 1, 1, 64, 16, 16, 1),
    ([0, 5, 16, 17, 100], 2, 4, 1, 128, 16, 16, 3),
    ([777, 3, 0, 400], 2, 4, 1, 128, 32, 8, 40),
    ([777, 300], 1, 8, 1, 64, 48, 24, 20),
    ([500, 123, 1], 3, 3, 1, 128, 20, 4, 60),
    ([900], 1, 16, 1, 128, 64, 64, 9),
    ([900, 88], 2, 5, 5, 64, 16, 16, 30),
    ([1000, 31, 7], 1, 2, 16, 128, 128, 32, 12),
    ([2000, 1999], 2, 8, 4, 128, 128, 128, 8),
    ([600], 1, 40, 2, 64, 40, 20, 11),                  # 80 rows: tiles of 32, 32, 16
    ([70, 64, 65, 63], 1, 1, 3, 128, 1, 1, 50),
    ([5000], 8, 4, 1, 128, 64, 32, 100),
    ([11000] + [20] * 40, 2, 4, 1, 64, 256, 128, 60),
]


@pytest.mark.parametrize("lens,Hkv,G,Nq,d,page,block,keep", CASES)
def test_decode_blocks(cuda_lib, lens, Hkv, G, Nq, d, page, block, keep):
    """What lies behind a sequence's last token, and in blocks that are not listed, may hold anything."""
    B, scale = len(lens), 1.0 / math.sqrt(d)
    rng = np.random.default_rng(sum(lens) + d + keep)
    maxp = max(1, -(-max(lens) // page))
    pages = B * maxp + 2
    c, table = random_pages(d + page, pages, Hkv, page, d), table_of(page, B, maxp, pages)
    lists = _lists(rng, lens, Hkv, block, keep)
    tokens = op.tokens_of(lists, block)
    q = bf16(rng, (B, Hkv * G, Nq, d), 0.3)
    ref = op.attend(f64(q), c, table, lens, scale, tokens)
    wild = {n: np.full_like(c[n], np.nan) for n in c}
    for b, n in enumerate(lens):
        for h in range(Hkv):
            j = tokens(b, h)
            j = j[j < n]
            for m in wild:
                wild[m][table[b][j // page], h, j % page] = c[m][table[b][j // page], h, j % page]
    g = to_gpu(wild)
    o, lse = cuda_lib.decode_blocks(q.to(DEV), g["k"], g["v"], ints(table), ints(lens), ints(lists), block=block)
    ok(cuda_lib)
    check_rows(o, lse, ref, PAIR)
    again = cuda_lib.decode_blocks(q.to(DEV), g["k"], g["v"], ints(table), ints(lens), ints(lists), block=block)
    assert torch.equal(again[0], o) and torch.equal(again[1], lse)


@pytest.mark.parametrize("d,G,Nq", [(128, 4, 1), (64, 2, 3)])
def test_every_block_listed_is_the_whole_attention(cuda_lib, d, G, Nq):
    rng = np.random.default_rng(d)
    lens, Hkv, page, block = [600, 0, 77, 333], 2, 32, 16
    maxp = 19
    c, table = random_pages(1, 4 * maxp, Hkv, page, d), table_of(2, 4, maxp, 4 * maxp)
    g, q = to_gpu(c), bf16(rng, (4, Hkv * G, Nq, d), 0.3)
    lists = _lists(rng, lens, Hkv, block, 38, "all")
    o, lse = cuda_lib.decode_blocks(q.to(DEV), g["k"], g["v"], ints(table), ints(lens), ints(lists), block=block, scale=0.1)
    ok(cuda_lib)
    check_rows(o, lse, op.attend(f64(q), c, table, lens, 0.1), PAIR)
    if Nq == 1:
        o3, lse3 = cuda_lib.decode_blocks(q[:, :, 0].contiguous().to(DEV), g["k"], g["v"], ints(table), ints(lens),
                                          ints(lists), block=block, scale=0.1)
        assert o3.shape == (4, Hkv * G, d) and torch.equal(o3, o[:, :, 0]) and torch.equal(lse3, lse[:, :, 0])


def test_rows_without_keys(cuda_lib):
    """Lists without entries, and lists whose tokens only the last drafted query sees."""
    rng = np.random.default_rng(7)
    Hkv, G, Nq, d, page, block = 1, 2, 4, 128, 16, 8
    lens = [33, 64, 2, 0]
    c, table = random_pages(2, 20, Hkv, page, d), table_of(3, 4, 4, 20)
    lists = np.array([[[4, -1, -1]], [[-1, -1, -1]], [[0, -1, -1]], [[-1, -1, -1]]], dtype=np.int32)  # 4: token 32 alone
    g, q = to_gpu(c), bf16(rng, (4, Hkv * G, Nq, d), 0.3)
    o, lse = cuda_lib.decode_blocks(q.to(DEV), g["k"], g["v"], ints(table), ints(lens), ints(lists), block=block)
    ok(cuda_lib)
    ref = op.attend(f64(q), c, table, lens, 1 / math.sqrt(d), op.tokens_of(lists, block))
    assert np.isneginf(ref[1][0, :, :3]).all() and np.isneginf(ref[1][2, :, :2]).all()
    check_rows(o, lse, ref, PAIR)


@pytest.mark.parametrize("G,Nq,d", [(1, 4, 128), (4, 4, 64), (8, 4, 128), (5, 16, 64)])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_wild_values_of_drafted_tokens_stay_with_the_queries_that_see_them(cuda_lib, G, Nq, d, value):
    rng = np.random.default_rng(G + d)
    Hkv, page, block, lens = 2, 16, 8, [40, 100, 9 if Nq < 9 else 25]
    c, table = random_pages(3, 30, Hkv, page, d), table_of(4, 3, 7, 30)
    lists = _lists(rng, lens, Hkv, block, 13, "all")
    for b, n in enumerate(lens):
        for i, col in ((1, 3), (2, 17)):                 # the last token and the one before
            t = n - i
            c["v"][table[b][t // page], b % Hkv, t % page, col] = value
    g, q = to_gpu(c), bf16(rng, (3, Hkv * G, Nq, d), 0.3)
    o, lse = cuda_lib.decode_blocks(q.to(DEV), g["k"], g["v"], ints(table), ints(lens), ints(lists), block=block)
    ok(cuda_lib)
    clean = copy(c)
    clean["v"][~np.isfinite(clean["v"])] = 0.0
    ref = op.attend(f64(q), clean, table, lens, 1 / math.sqrt(d))
    got, want = f64(o), np.zeros_like(ref[0], dtype=bool)
    for b in range(3):
        heads = slice(b % Hkv * G, (b % Hkv + 1) * G)
        want[b, heads, Nq - 1, 3] = True                 # the last token is seen by the last query alone
        want[b, heads, max(0, Nq - 2):, 17] = True
    assert np.array_equal(~np.isfinite(got), want)
    if not math.isnan(value):
        assert (got[want] == value).all()
    check_rows(torch.from_numpy(np.where(want, ref[0], got)), lse, ref, PAIR)


def test_large_scores_and_flat_tails(cuda_lib):
    """One token far above a long flat tail, in the first and in the last block; scores around +-2000."""
    rng = np.random.default_rng(11)
    Hkv, G, d, page, block, n = 1, 4, 128, 64, 32, 4096
    for hot in (0, n - 1):
        c, table = random_pages(5, 64, Hkv, page, d), table_of(5, 1, 64, 64)
        q = bf16(rng, (1, G, 1, d), 0.3)
        c["k"] = f64(torch.from_numpy(c["k"] * 0.05).to(torch.bfloat16))
        c["k"][table[0][hot // page], 0, hot % page] = f64(torch.from_numpy(f64(q)[0, 0, 0] * 1.1).to(torch.bfloat16))
        lists = np.arange(128, dtype=np.int32)[None, None]
        for scale in (1 / math.sqrt(d), 15.0):
            g = to_gpu(c)
            o, lse = cuda_lib.decode_blocks(q.to(DEV), g["k"], g["v"], ints(table), ints([n]), ints(lists), block=block, scale=scale)
            ok(cuda_lib)
            check_rows(o, lse, op.attend(f64(q), c, table, [n], scale), PAIR, "hot %d scale %g" % (hot, scale))


def test_bad_entries_pages_and_lengths(cuda_lib):
    """Blocks past the sequence are skipped, pages that are not there read as zeros, lengths clamped: all recorded."""
    fa, Hkv, G, d, page, block = cuda_lib, 1, 4, 64, 16, 8
    rng = np.random.default_rng(6)
    c, table = random_pages(6, 12, Hkv, page, d), table_of(7, 2, 5, 12)
    q, lens, g = bf16(rng, (2, G, 1, d), 0.3), [75, 40], to_gpu(c)
    good = np.array([[[0, 3, 9]], [[4, 2, -1]]], dtype=np.int32)
    for entry in (10, 2 ** 31 - 1):
        lists = good.copy()
        lists[0, 0, 1] = entry
        o, lse = fa.decode_blocks(q.to(DEV), g["k"], g["v"], ints(table), ints(lens), ints(lists), block=block)
        assert fa.fa_get_last_device_error()[0] == fa.FA_ERR_INVALID_ARG
        lists[0, 0, 1] = -1
        check_rows(o, lse, op.attend(f64(q), c, table, lens, 0.125, op.tokens_of(lists, block)), PAIR)
    for bad in (-1, 12, 2 ** 31 - 1):
        t = table.copy()
        t[0, 1] = bad
        o, lse = fa.decode_blocks(q.to(DEV), g["k"], g["v"], ints(t), ints(lens), ints(good), block=block)
        assert fa.fa_get_last_device_error()[0] == fa.FA_ERR_INVALID_ARG
        t[0, 1] = 12
        grown = {n: np.concatenate([c[n], np.zeros_like(c[n][:1])]) for n in c}
        check_rows(o, lse, op.attend(f64(q), grown, t, lens, 0.125, op.tokens_of(good, block)), PAIR)
    o, lse = fa.decode_blocks(q.to(DEV), g["k"], g["v"], ints(table), ints([-7, 1000]), ints(good), block=block)
    assert fa.fa_get_last_device_error()[0] == fa.FA_ERR_INVALID_ARG
    check_rows(o, lse, op.attend(f64(q), c, table, [0, 80], 0.125, op.tokens_of(good, block)), PAIR)


@pytest.mark.parametrize("G,Nq,d", [(4, 1, 128), (4, 3, 64), (3, 8, 128)])
def test_many_sequences(cuda_lib, G, Nq, d):
    """More (sequence, kv head) pairs than CTAs run at once, of very different lengths, some of them empty."""
    rng = np.random.default_rng(G + Nq)
    B, Hkv, page, block, keep, scale = 80, 5, 32, 16, 12, 1.0 / math.sqrt(d)
    lens = [int(n) for n in rng.integers(0, 400, B)]
    lens[:4] = [0, 1, 0, 399]
    c, table = random_pages(5, B * 13, Hkv, page, d), table_of(6, B, 13, B * 13)
    lists = _lists(rng, lens, Hkv, block, keep)
    g, q = to_gpu(c), bf16(rng, (B, Hkv * G, Nq, d), 0.3)
    o, lse = cuda_lib.decode_blocks(q.to(DEV), g["k"], g["v"], ints(table), ints(lens), ints(lists), block=block)
    ok(cuda_lib)
    check_rows(o, lse, op.attend(f64(q), c, table, lens, scale, op.tokens_of(lists, block)), PAIR)


def test_entries_behind_a_sequence_s_number_of_blocks_are_not_looked_at(cuda_lib):
    """Of a list the first min(keep, n_b) entries count: what lies behind them, good or bad, is neither used nor recorded."""
    rng = np.random.default_rng(8)
    Hkv, G, d, page, block, lens = 2, 4, 128, 16, 8, [33, 3, 0]          # 5, 1 and no blocks
    c, table = random_pages(5, 12, Hkv, page, d), table_of(3, 3, 3, 12)
    lists = np.tile(np.array([[4, -1, 0, 2, -1, 1, 3], [0, 0, 5, 7, 9, 1, 2 ** 31 - 1], [0, 1, 2, 3, 4, 5, 6]], dtype=np.int32)[:, None],
                    (1, Hkv, 1))
    counted = lists.copy()
    for b, n in enumerate(lens):
        counted[b, :, -(-n // block):] = -1
    q, g = bf16(rng, (3, Hkv * G, 1, d), 0.3), to_gpu(c)
    o, lse = cuda_lib.decode_blocks(q.to(DEV), g["k"], g["v"], ints(table), ints(lens), ints(lists), block=block)
    ok(cuda_lib)
    check_rows(o, lse, op.attend(f64(q), c, table, lens, 1 / math.sqrt(d), op.tokens_of(counted, block)), PAIR)
