"""fa_decode_shared against float64."""
import math

import numpy as np
import pytest
import torch

from oracle import paged as op
from tests.paged_common import DEV, bf16, check_rows, f64, ints, ok, random_pages, table_of, to_gpu

pytestmark = pytest.mark.gpu
ONE, PAIR = 2.0 ** -8, 2.0 ** -16


def _case(seed, lens, shared, Hkv, page, d):
    """Pages and a table whose rows begin with the same pages; the page that the prefix ends in is each one's own copy."""
    B, full = len(lens), shared // page
    own = max(1, -(-max(max(lens), shared) // page) - full)
    c = random_pages(seed, full + B * own + 2, Hkv, page, d)
    p = np.random.default_rng(seed).permutation(full + B * own + 2).astype(np.int32)
    table = np.concatenate([np.tile(p[:full], (B, 1)), p[full:full + B * own].reshape(B, own)], 1)
    if shared % page:
        for n in c:
            c[n][table[:, full], :, :shared % page] = c[n][table[0, full], :, :shared % page]
    return c, np.ascontiguousarray(table)


# (own tokens, shared, Hkv, G, Nq, d, page); None: an empty slot
CASES = [
    ([1], 1, 1, 1, 1, 64, 8),
    ([1, 2], 128, 1, 1, 1, 128, 16),
    ([5, None, 17, 100], 129, 2, 4, 1, 128, 16),
    ([1] * 32, 777, 2, 4, 1, 128, 16),                  # 128 rows
    ([3] * 33, 1000, 1, 4, 1, 64, 48),                  # 132 rows
    ([1, 300, None, 64] * 9, 1024, 2, 8, 1, 128, 64),   # 288 rows: a second tile of 32
    ([9, 40, None, 8] * 4, 2000, 1, 5, 5, 64, 40),      # 400 rows, pages of 40
    ([16, 20], 300, 3, 1, 16, 128, 8),
    ([4, 1], 5000, 1, 16, 1, 128, 256),
    ([10] * 140, 130, 1, 8, 1, 64, 32),                 # 1120 rows
    ([2, 1, 700], 64, 4, 2, 1, 128, 128),
    ([600, 5], 0, 2, 4, 1, 128, 16),                    # nothing shared
]


@pytest.mark.parametrize("own,shared,Hkv,G,Nq,d,page", CASES)
def test_decode_shared(cuda_lib, own, shared, Hkv, G, Nq, d, page):
    """What lies behind a sequence's last token may hold anything, and the entries of whole shared pages are looked at in
    one row only."""
    lens = [0 if n is None else shared + n for n in own]
    B, scale = len(lens), 1.0 / math.sqrt(d)
    rng = np.random.default_rng(sum(lens) + d)
    c, table = _case(d + page, lens, shared, Hkv, page, d)
    q = bf16(rng, (B, Hkv * G, Nq, d), 0.3)
    ref = op.attend(f64(q), c, table, lens, scale)
    used = {n: np.full_like(c[n], np.nan) for n in c}
    for b, n in enumerate(lens):
        j = np.arange(n)
        for m in c:
            used[m][table[b][j // page], :, j % page] = c[m][table[b][j // page], :, j % page]
    seen = table.copy()
    seen[1:, :shared // page] = -1
    g = to_gpu(used)
    for t in (table, seen):
        o, lse = cuda_lib.decode_shared(q.to(DEV), g["k"], g["v"], ints(t), ints(lens), ints([shared]))
        ok(cuda_lib)
        check_rows(o, lse, ref, ONE)
    again = cuda_lib.decode_shared(q.to(DEV), g["k"], g["v"], ints(table), ints(lens), ints([shared]))
    assert torch.equal(again[0], o) and torch.equal(again[1], lse)


@pytest.mark.parametrize("d", [64, 128])
def test_sequences_that_do_not_see_all_of_the_prefix(cuda_lib, d):
    """Empty, shorter, and drafted queries of which the first does not see the prefix's end: they read their own rows, from
    pages of their own; also where the first sequences of the batch are such ones, or all."""
    rng = np.random.default_rng(d)
    Hkv, G, Nq, page, shared = 2, 2, 4, 16, 100
    for lens in ([0, 30, 103, 104, 150, 2], [3, 0, 99, 100, 101, 0], [0] * 6):
        c = random_pages(d, 80, Hkv, page, d)
        table = table_of(9, 6, 10, 80)
        share = [b for b in range(6) if lens[b] - Nq >= shared]
        for b in share[1:]:                              # of those that take part, the first one's pages
            table[b, :shared // page] = table[share[0], :shared // page]
            for n in c:
                c[n][table[b, 6], :, :4] = c[n][table[share[0], 6], :, :4]
        q, g = bf16(rng, (6, Hkv * G, Nq, d), 0.3), to_gpu(c)
        o, lse = cuda_lib.decode_shared(q.to(DEV), g["k"], g["v"], ints(table), ints(lens), ints([shared]))
        ok(cuda_lib)
        check_rows(o, lse, op.attend(f64(q), c, table, lens, 1 / math.sqrt(d)), ONE)


def test_nothing_shared_is_paged_decode(cuda_lib):
    rng = np.random.default_rng(3)
    lens, Hkv, G, d, page = [300, 1, 77], 2, 4, 128, 16
    c, table = _case(4, lens, 0, Hkv, page, d)
    q, g = bf16(rng, (3, Hkv * G, d), 0.3), to_gpu(c)
    o, lse = cuda_lib.decode_shared(q.to(DEV), g["k"], g["v"], ints(table), ints(lens), ints([0]))
    ok(cuda_lib)
    check_rows(o, lse, op.attend(f64(q)[:, :, None], c, table, lens, 1 / math.sqrt(d)), PAIR)
    o2, lse2 = cuda_lib.decode_paged(q.to(DEV), g["k"], g["v"], ints(table), ints(lens))
    check_rows(o2, lse2, op.attend(f64(q)[:, :, None], c, table, lens, 1 / math.sqrt(d)), ONE)


def test_large_scores(cuda_lib):
    """A dominant token at the start or end of the prefix, or among the own ones; scores around +-2000."""
    rng = np.random.default_rng(11)
    Hkv, G, d, page, shared, lens = 1, 4, 128, 64, 3000, [3100, 3001, 3050]
    for hot in (0, 2999, 3000):
        c, table = _case(5, lens, shared, Hkv, page, d)
        q = bf16(rng, (3, G, 1, d), 0.3)
        for n in c:
            c[n] = f64(torch.from_numpy(c[n] * (0.05 if n == "k" else 1.0)).to(torch.bfloat16))
        for b in range(3):
            c["k"][table[b][hot // page], 0, hot % page] = f64(torch.from_numpy(f64(q)[0, 0, 0] * 1.1).to(torch.bfloat16))
        for scale in (1 / math.sqrt(d), 15.0):
            g = to_gpu(c)
            o, lse = cuda_lib.decode_shared(q.to(DEV), g["k"], g["v"], ints(table), ints(lens), ints([shared]), scale=scale)
            ok(cuda_lib)
            check_rows(o, lse, op.attend(f64(q), c, table, lens, scale), ONE, "hot %d scale %g" % (hot, scale))


def test_bad_pages_and_lengths(cuda_lib):
    fa, Hkv, G, d, page, shared = cuda_lib, 1, 4, 64, 16, 64
    rng = np.random.default_rng(6)
    lens = [75, 70]
    c, table = _case(6, lens, shared, Hkv, page, d)
    q, g, pages = bf16(rng, (2, G, 1, d), 0.3), to_gpu(c), c["k"].shape[0]
    for bad in (-1, pages, 2 ** 31 - 1):
        for at in ((0, 1), (1, 4)):                      # a shared page, an own one
            t = table.copy()
            t[at] = bad
            o, lse = fa.decode_shared(q.to(DEV), g["k"], g["v"], ints(t), ints(lens), ints([shared]))
            assert fa.fa_get_last_device_error()[0] == fa.FA_ERR_INVALID_ARG
            t[at] = pages
            if at[0] == 0:
                t[:, 1] = pages
            grown = {n: np.concatenate([c[n], np.zeros_like(c[n][:1])]) for n in c}
            check_rows(o, lse, op.attend(f64(q), grown, t, lens, 0.125), ONE)
    for length in (-5, 1000):
        o, lse = fa.decode_shared(q.to(DEV), g["k"], g["v"], ints(table), ints(lens), ints([length]))
        assert fa.fa_get_last_device_error()[0] == fa.FA_ERR_INVALID_ARG
        check_rows(o, lse, op.attend(f64(q), c, table, lens, 0.125), ONE)
    o, lse = fa.decode_shared(q.to(DEV), g["k"], g["v"], ints(table), ints([-1, 70]), ints([shared]))
    assert fa.fa_get_last_device_error()[0] == fa.FA_ERR_INVALID_ARG
    check_rows(o, lse, op.attend(f64(q), c, table, [0, 70], 0.125), ONE)


@pytest.mark.parametrize("B,G,Nq,d", [(3, 2, 3, 128), (3, 8, 4, 64), (20, 4, 4, 128)])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_wild_values_of_drafted_tokens_stay_with_the_queries_that_see_them(cuda_lib, B, G, Nq, d, value):
    """Own tokens that some of the drafted queries see and others do not, beside a shared prefix; 20 sequences of 16 rows go
    through the prefix's matrix kernel."""
    rng = np.random.default_rng(G + d)
    Hkv, page, shared = 2, 16, 150
    lens = shared + rng.integers(Nq, 70, B)
    c, table = _case(7, lens, shared, Hkv, page, d)
    for b, n in enumerate(lens):
        for i, col in ((1, 3), (2, 17)):                 # the last token and the one before
            c["v"][table[b][(n - i) // page], b % Hkv, (n - i) % page, col] = value
    g, q = to_gpu(c), bf16(rng, (B, Hkv * G, Nq, d), 0.3)
    o, lse = cuda_lib.decode_shared(q.to(DEV), g["k"], g["v"], ints(table), ints(lens), ints([shared]))
    ok(cuda_lib)
    c["v"][~np.isfinite(c["v"])] = 0.0
    ref = op.attend(f64(q), c, table, lens, 1 / math.sqrt(d))
    got, want = f64(o), np.zeros_like(ref[0], dtype=bool)
    for b in range(B):
        heads = slice(b % Hkv * G, (b % Hkv + 1) * G)
        want[b, heads, Nq - 1, 3] = True                 # the last token is seen by the last query alone
        want[b, heads, Nq - 2:, 17] = True
    assert np.array_equal(~np.isfinite(got), want)
    if not math.isnan(value):
        assert (got[want] == value).all()
    check_rows(torch.from_numpy(np.where(want, ref[0], got)), lse, ref, ONE)


def test_wild_values_of_the_prefix_and_of_its_page(cuda_lib):
    """A NaN in a shared value reaches every sequence that takes part, one behind the prefix in its last page none."""
    rng = np.random.default_rng(1)
    Hkv, G, d, page, shared = 1, 4, 128, 16, 150
    for B in (3, 40):
        lens = np.full(B, shared + 2)
        lens[1] = 0
        c, table = _case(8, lens, shared, Hkv, page, d)
        last = table[:, shared // page]
        c["k"][last, :, shared % page + 2:] = np.nan
        c["v"][last, :, shared % page + 2:] = np.inf
        q = bf16(rng, (B, G, 1, d), 0.3)
        g = to_gpu(c)
        o, lse = cuda_lib.decode_shared(q.to(DEV), g["k"], g["v"], ints(table), ints(lens), ints([shared]))
        ok(cuda_lib)
        check_rows(o, lse, op.attend(f64(q), c, table, lens, 1 / math.sqrt(d)), ONE)
        c["v"][table[0, 3], 0, 5, 40] = np.nan
        g = to_gpu(c)
        o, lse = cuda_lib.decode_shared(q.to(DEV), g["k"], g["v"], ints(table), ints(lens), ints([shared]))
        ok(cuda_lib)
        there = np.isnan(f64(o))
        assert there[lens > 0, :, :, 40].all() and there.sum() == (B - 1) * G


@pytest.mark.parametrize("B,Hkv,G,Nq,d,shared", [
    (33, 2, 4, 1, 128, 700),      # 132 rows, one step of a second tile's
    (40, 8, 1, 8, 64, 1500),      # drafts
    (18, 1, 4, 2, 128, 2500),     # 144 rows of one kv head, the CTAs many to an item
    (18, 1, 4, 2, 128, 0),
    (160, 32, 8, 1, 64, 140),     # more (kv head, 256 rows) than CTAs
    (130, 16, 2, 1, 128, 129),
    (20, 2, 4, 4, 128, 600),      # 16 rows of a sequence, two passes over its own tokens
    (33, 3, 1, 9, 64, 1000),      # 9
    (9, 3, 5, 5, 128, 300),       # 25
    (7, 2, 8, 4, 64, 1500),       # 32
    (44, 3, 6, 4, 128, 260),      # 24 of more than 128 pairs: kernels of their own
])
def test_prefix_and_own_tokens_in_one_kernel(cuda_lib, B, Hkv, G, Nq, d, shared):
    """More than 128 query rows of all sequences: own tokens from few to more than the prefix, sequences that do not take part,
    and batches in which none does."""
    rng = np.random.default_rng(B + d)
    page, scale = 32, 1.0 / math.sqrt(d)
    lens = shared + rng.integers(Nq, 60, B)
    lens[1], lens[2], lens[3] = 0, shared // 2, shared + 900
    q = bf16(rng, (B, Hkv * G, Nq, d), 0.3)
    c, table = _case(8, lens, shared, Hkv, page, d)
    g = to_gpu(c)
    o, lse = cuda_lib.decode_shared(q.to(DEV), g["k"], g["v"], ints(table), ints(lens), ints([shared]))
    ok(cuda_lib)
    check_rows(o, lse, op.attend(f64(q), c, table, lens, scale), ONE)
    again = cuda_lib.decode_shared(q.to(DEV), g["k"], g["v"], ints(table), ints(lens), ints([shared]))
    assert torch.equal(again[0], o) and torch.equal(again[1], lse)
    for short in (np.minimum(lens, shared), np.zeros_like(lens)):  # nobody has all of the prefix and new tokens
        o, lse = cuda_lib.decode_shared(q.to(DEV), g["k"], g["v"], ints(table), ints(short), ints([shared]))
        ok(cuda_lib)
        check_rows(o, lse, op.attend(f64(q), c, table, short, scale), ONE)


@pytest.mark.parametrize("B", [4, 40])
def test_bad_lengths_are_noted_whichever_kernel_takes_them(cuda_lib, B):
    """A length out of range, the prefix's too, is clamped and recorded."""
    rng = np.random.default_rng(B)
    Hkv, G, d, page, shared = 2, 4, 128, 16, 100
    for where in ("negative", "long", "prefix"):
        lens = np.full(B, shared + 7)
        c, table = _case(3, lens, shared, Hkv, page, d)
        cap, given = table.shape[1] * page, shared
        if where == "prefix":
            given = cap + 5                              # nobody takes part
        else:
            lens[B - 1] = -3 if where == "negative" else cap + 9
        q, g = bf16(rng, (B, Hkv * G, 1, d), 0.3), to_gpu(c)
        o, lse = cuda_lib.decode_shared(q.to(DEV), g["k"], g["v"], ints(table), ints(lens), ints([given]))
        assert cuda_lib.fa_get_last_device_error()[0] == cuda_lib.FA_ERR_INVALID_ARG, where
        check_rows(o, lse, op.attend(f64(q), c, table, np.clip(lens, 0, cap), 1 / math.sqrt(d)), ONE)


def test_one_kernel_replayed_with_other_lengths_and_on_two_streams(cuda_lib):
    """The division of CTAs follows the lengths on the device: a captured call replayed with other lengths and another prefix
    gives what a fresh call does; two calls at once on streams of their own give what they do one after the other."""
    rng = np.random.default_rng(12)
    B, Hkv, G, d, page, scale = 40, 4, 4, 128, 32, 1.0 / math.sqrt(128)
    cases = []
    for shared, most in ((600, 40), (64, 500), (0, 30), (600, 0)):
        lens = shared + rng.integers(1, most + 2, B) if most else np.zeros(B, dtype=np.int64)
        cases.append((shared, lens))
    c, table = _case(4, np.full(B, 1200), 600, Hkv, page, d)
    table[:, :600 // page] = table[0, :600 // page]
    q, g, tab = bf16(rng, (B, Hkv * G, 1, d), 0.3).to(DEV), to_gpu(c), ints(table)
    lens, shared = ints(cases[0][1]), ints([cases[0][0]])
    cuda_lib.decode_shared(q, g["k"], g["v"], tab, lens, shared)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = cuda_lib.decode_shared(q, g["k"], g["v"], tab, lens, shared)
    fresh = []
    for n, (s, l) in enumerate(cases * 2):
        lens.copy_(ints(l))
        shared.copy_(ints([s]))
        graph.replay()
        want = cuda_lib.decode_shared(q, g["k"], g["v"], tab, ints(l), ints([s]))
        ok(cuda_lib)
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1]), n
        fresh.append(want)
        if n < 2:
            check_rows(o, lse, op.attend(f64(q.cpu()), c, table, l, scale), ONE)
    streams = [torch.cuda.Stream() for _ in range(2)]
    args = [(ints(l), ints([s])) for s, l in cases]
    torch.cuda.synchronize()
    for _ in range(10):
        got = [cuda_lib.decode_shared(q, g["k"], g["v"], tab, *args[i], stream=streams[i % 2]) for i in range(4)]
        torch.cuda.synchronize()
        for a, b in zip(got, fresh):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    ok(cuda_lib)
