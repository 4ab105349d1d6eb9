"""fa_cache_evict_fp8 against the oracle, byte for byte, and a serving run of all four operators."""
import math

import numpy as np
import pytest
import torch

import exact_tiled_attention_21_gb300 as fa_mod
from oracle import cache as oc
from tests.cache_fp8_common import (DEV, args, assert_same_cache, bf16, check_decode, copy, f64, ints, random_cache,
                                    table_of, to_gpu)

pytestmark = pytest.mark.gpu


def _ok(fa):
    st, detail = fa.fa_get_last_device_error()
    assert st == 0, detail


def _run(fa, c, table, lens, w, new, keep, recent):
    g = to_gpu(c)
    got = fa.cache_evict_fp8(*args(g), ints(table), ints(lens), torch.from_numpy(w).to(DEV), ints(new), keep, recent)
    return g, [t.cpu().numpy() for t in got]


def _weights(rng, shape, kind):
    if kind == "heavy":
        return np.exp(3 * rng.standard_normal(shape)).astype(np.float32)
    if kind == "ties":
        return rng.integers(0, 4, shape).astype(np.float32)
    if kind == "equal":
        return np.full(shape, 0.25, dtype=np.float32)
    w = rng.standard_normal(shape).astype(np.float32)   # signs, zeros of both signs, infinities, NaN, subnormals
    for x in (0.0, -0.0, np.inf, -np.inf, np.nan, 1e-40, -1e-40):
        w[rng.random(shape) < 0.06] = x
    return w


# (Hkv, page, sb, lens, keep, recent, d)
CASES = [
    (1, 16, 16, [40], 10, 4, 64),
    (2, 16, 8, [100, 17, 16, 0], 16, 5, 128),
    (2, 64, 64, [1000, 200], 129, 128, 64),
    (1, 20, 4, [333], 100, 0, 128),
    (3, 32, 32, [500, 64], 64, 64, 64),              # only the most recent
    (1, 1, 1, [30], 7, 2, 64),
    (1, 128, 128, [3001], 1500, 100, 128),
    (2, 48, 24, [2500, 2049], 1, 0, 64),
    (1, 33, 11, [1025], 1024, 1, 64),                # one token goes
    (2, 256, 64, [5000], 700, 77, 128),
    # several small blocks per turn
    (2, 12, 3, [400, 77], 150, 11, 128),
    (1, 4, 1, [200, 99], 90, 7, 128),
    (2, 40, 8, [900, 20], 333, 20, 64),
    (3, 6, 2, [700], 613, 100, 64),
    (8, 64, 32, [5000, 4000, 1, 3000, 80, 0, 64, 2500, 5000, 700], 70, 10, 64),  # one CTA per kv head, many tokens each
    (1, 256, 128, [140000], 90, 5, 64),              # more tokens than a cluster's registers hold
    (2, 128, 128, [40000, 39999], 300, 300, 64),     # a cluster of eight, recent ones only
]


@pytest.mark.parametrize("kind", ["heavy", "ties", "equal", "special"])
@pytest.mark.parametrize("Hkv,page,sb,lens,keep,recent,d", CASES)
def test_evict_bytes(cuda_lib, Hkv, page, sb, lens, keep, recent, d, kind):
    B = len(lens)
    rng = np.random.default_rng(keep + page)
    maxp, newp = -(-max(lens) // page) + 1, -(-keep // page) + 1
    c = random_cache(keep, B * (maxp + newp), Hkv, page, sb, d)
    both = table_of(page, B, maxp + newp, B * (maxp + newp))
    table, new = both[:, :maxp], both[:, maxp:]
    w = _weights(rng, (B, Hkv, maxp * page), kind)
    g, (new_lens, new_w, kept) = _run(cuda_lib, c, table, lens, w, new, keep, recent)
    _ok(cuda_lib)
    want_lens, want_w, want_kept = oc.evict(c, table, np.array(lens), w, new, keep, recent)
    assert np.array_equal(kept, want_kept) and np.array_equal(new_lens, want_lens)
    assert np.array_equal(new_w, want_w, equal_nan=True)
    assert_same_cache(g, c)   # the kept tokens, and every other byte as it was


def test_evict_many_long_heads(cuda_lib):
    """More clusters than run at once, over a cache whose logical pages share four physical ones."""
    Hkv, page, sb, d, n, keep = 90, 64, 64, 64, 20000, 100
    c = random_cache(2, 6, Hkv, page, sb, d)
    table = (np.arange(-(-n // page)) % 4).astype(np.int32)[None]
    new = np.array([[5, 4]], dtype=np.int32)
    w = _weights(np.random.default_rng(6), (1, Hkv, table.shape[1] * page), "ties")
    g, got = _run(cuda_lib, c, table, [n], w, new, keep, 30)
    _ok(cuda_lib)
    want = oc.evict(c, table, np.array([n]), w, new, keep, 30)
    assert all(np.array_equal(a, b) for a, b in zip(got, want))
    assert_same_cache(g, c)


def test_evict_bad_lengths_and_pages(cuda_lib):
    page, sb, d, Hkv = 16, 16, 64, 2
    c = random_cache(1, 20, Hkv, page, sb, d)
    both = table_of(2, 3, 5, 20)
    table, new = both[:, :3], both[:, 3:]
    w = np.random.default_rng(3).random((3, Hkv, 48)).astype(np.float32)
    g, got = _run(cuda_lib, c, table, [-1, 49, 40], w, new, 20, 4)
    assert cuda_lib.fa_get_last_device_error()[0] == fa_mod.FA_ERR_INVALID_ARG
    ref = copy(c)
    want = oc.evict(ref, table, np.array([0, 48, 40]), w, new, 20, 4)
    assert all(np.array_equal(a, b) for a, b in zip(got, want))
    assert_same_cache(g, ref)
    bad_new = new.copy()
    bad_new[1, 1], bad_new[2, 0] = 20, -1          # not written, recorded; the others are
    g, got = _run(cuda_lib, c, table, [48, 48, 40], w, bad_new, 20, 4)
    assert cuda_lib.fa_get_last_device_error()[0] == fa_mod.FA_ERR_INVALID_ARG
    ref = copy(c)
    want = oc.evict(ref, table, np.array([48, 48, 40]), w, new, 20, 4)
    for n in c:
        ref[n][new[1, 1]], ref[n][new[2, 0]] = c[n][new[1, 1]], c[n][new[2, 0]]
    assert all(np.array_equal(a, b) for a, b in zip(got, want))
    assert_same_cache(g, ref)
    bad = table.copy()
    bad[0, 1] = 1 << 30                            # its tokens read as zeros
    g, got = _run(cuda_lib, c, bad, [48, 10, 40], w, new, 20, 4)
    assert cuda_lib.fa_get_last_device_error()[0] == fa_mod.FA_ERR_INVALID_ARG
    lost = np.argwhere((got[2][0, 0] // page == 1) & (got[2][0, 0] >= 0))[:, 0]
    assert len(lost)
    for s in lost:
        assert (g["k"][new[0, s // page], 0, s % page].cpu().numpy() == 0).all()


def test_evict_bad_page_among_small_blocks(cuda_lib):
    """Blocks of 4 tokens whose new page does not exist are left out, the others of the same turn written."""
    page, sb, d, Hkv = 8, 4, 128, 2
    c = random_cache(5, 30, Hkv, page, sb, d)
    both = table_of(3, 1, 30, 30)
    table, new = both[:, :20], both[:, 20:28]
    w = np.random.default_rng(4).random((1, Hkv, 160)).astype(np.float32)
    bad = new.copy()
    bad[0, 0], bad[0, 3] = 30, -7
    g, got = _run(cuda_lib, c, table, [155], w, bad, 61, 9)
    assert cuda_lib.fa_get_last_device_error()[0] == fa_mod.FA_ERR_INVALID_ARG
    ref = copy(c)
    want = oc.evict(ref, table, np.array([155]), w, new, 61, 9)
    for n in c:
        for j in (0, 3):
            ref[n][new[0, j]] = c[n][new[0, j]]
    assert all(np.array_equal(a, b) for a, b in zip(got, want))
    assert_same_cache(g, ref)


def test_evict_far_pages(cuda_lib):
    Hkv, d, page = 8, 128, 64
    pages = 2 ** 32 // (Hkv * d * page) + 9
    c = random_cache(4, 6, Hkv, page, 32, d)
    far = {n: torch.zeros((pages,) + x.shape[1:], dtype=torch.uint8 if n in "kv" else torch.float32, device=DEV)
           for n, x in c.items()}
    for n, x in to_gpu(c).items():
        far[n][-6:] = x
    table, new = np.array([[0, 3, 1, 5]]), np.array([[4, 2]])
    w = np.random.default_rng(5).random((1, Hkv, 256)).astype(np.float32)
    off = pages - 6
    got = cuda_lib.cache_evict_fp8(*args(far), ints(table + off), ints([250]), torch.from_numpy(w).to(DEV),
                                   ints(new + off), 100, 10)
    _ok(cuda_lib)
    want = oc.evict(c, table, np.array([250]), w, new, 100, 10)
    assert all(np.array_equal(a.cpu().numpy(), b) for a, b in zip(got, want))
    assert_same_cache({n: far[n][-6:] for n in far}, c)
    assert int(far["k"][:-6].view(torch.int64).count_nonzero()) == 0


def test_evict_graph_and_stream(cuda_lib):
    c = random_cache(6, 12, 2, 16, 16, 64)
    both = table_of(7, 2, 6, 12)
    table, new = both[:, :4], both[:, 4:]
    rng = np.random.default_rng(8)
    w = torch.zeros((2, 2, 64), device=DEV)
    g, lens, s = to_gpu(c), ints([64, 50]), torch.cuda.Stream()
    tab, nt = ints(table), ints(new)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = cuda_lib.cache_evict_fp8(*args(g), tab, lens, w, nt, 30, 6)
    for kind, n in (("heavy", [64, 50]), ("ties", [33, 5])):
        x = _weights(rng, (2, 2, 64), kind)
        w.copy_(torch.from_numpy(x))
        lens.copy_(ints(n))
        graph.replay()
        torch.cuda.synchronize()
        want = oc.evict(c, table, np.array(n), x, new, 30, 6)
        assert all(np.array_equal(a.cpu().numpy(), b) for a, b in zip(out, want))
        assert_same_cache(g, c)
        s.wait_stream(torch.cuda.current_stream())
        again = cuda_lib.cache_evict_fp8(*args(g), tab, lens, w, nt, 30, 6, stream=s)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, again))
    _ok(cuda_lib)


def test_evict_refusals(cuda_lib):
    g = to_gpu(random_cache(1, 6, 2, 16, 8, 64))
    tab, new, lens, w = ints([[0, 1]]), ints([[2]]), ints([20]), torch.zeros((1, 2, 32), device=DEV)
    for bad in (dict(w=w[..., :31].contiguous()), dict(new=ints([[2], [3]])), dict(new=new.float()), dict(lens=lens.long())):
        a = dict(w=w, new=new, lens=lens) | bad
        with pytest.raises(ValueError):
            cuda_lib.cache_evict_fp8(*args(g), tab, a["lens"], a["w"], a["new"], 10)
    for keep, recent in ((0, 0), (17, 0), (8, 9), (8, -1)):
        with pytest.raises(fa_mod.FAError) as e:
            cuda_lib.cache_evict_fp8(*args(g), tab, lens, w, new, keep, recent)
        assert e.value.status == fa_mod.FA_ERR_INVALID_ARG


@pytest.mark.parametrize("d,page,sb,inter", [(64, 16, 16, True), (128, 32, 16, False)])
def test_serving_run(cuda_lib, d, page, sb, inter):
    """Prompt, decode steps with accumulating weights, eviction, more steps at the positions that go on counting, a
    drafted step: every state against the oracle fed with the rotated keys and queries."""
    fa = cuda_lib
    B, Hq, Hkv, rot, scale = 3, 8, 2, d // 2, 1 / math.sqrt(d)
    rng = np.random.default_rng(d)
    freq, mag = fa.rope_frequencies(rot, scaling="yarn", factor=4.0, original_context=64)
    turns = fa.rope_table(freq)
    prompt = np.array([50, 1, 33], dtype=np.int32)
    maxp, newp = -(-80 // page), -(-64 // page)
    c = random_cache(1, B * (maxp + newp), Hkv, page, sb, d)
    both = table_of(2, B, maxp + newp, B * (maxp + newp))
    table, new = both[:, :maxp].copy(), both[:, maxp:].copy()
    g, tab = to_gpu(c), ints(table)
    w, w_ref = torch.zeros((B, Hkv, maxp * page), device=DEV), np.zeros((B, Hkv, maxp * page))

    # the prompt: keys rotated once for the prompt's own attention and appended as they are
    k, v = bf16(rng, (B, Hkv, 50, d), 0.3).to(DEV), bf16(rng, (B, Hkv, 50, d), 0.3).to(DEV)
    kr = fa.rope(k, turns, interleaved=inter, magnitude=mag)
    fa.cache_append_fp8(kr, v, *args(g), tab, ints([0] * B), ints(prompt))
    oc.append(c, table, [0] * B, f64(kr), f64(v), prompt)
    assert_same_cache(g, c, "prompt")
    lens, pos = prompt.copy(), prompt.copy()   # tokens in the cache, and the next token's position

    def step(n):
        nonlocal lens, pos
        q = bf16(rng, (B, Hq, n, d), 0.3).to(DEV)
        k, v = (bf16(rng, (B, Hkv, n, d), 0.3).to(DEV) for _ in range(2))
        p = ints(pos[:, None] + np.arange(n))
        qr = fa.rope(q, turns, p, inter, mag)
        kr = fa.rope(k, turns, p, inter, mag)
        fa.cache_append_fp8(k, v, *args(g), tab, ints(lens), turns=turns, positions=p, interleaved=inter, magnitude=mag)
        oc.append(c, table, lens, f64(kr), f64(v))
        lens, pos = lens + n, pos + n
        o, lse = fa.decode_paged_fp8(qr, *args(g), tab, ints(lens), weights=w)
        ref = oc.decode(f64(qr), c, table, lens, scale, w_ref)
        assert_same_cache(g, c, "step")
        check_decode(o, lse, ref, w, w_ref, "step")

    for _ in range(8):
        step(1)
    x = w.cpu().numpy()
    new_lens, nw, kept = fa.cache_evict_fp8(*args(g), tab, ints(lens), w, ints(new), 30, 8)
    ref_lens, ref_w, ref_kept = oc.evict(c, table, lens, x, new, 30, 8)
    assert np.array_equal(kept.cpu().numpy(), ref_kept) and np.array_equal(nw.cpu().numpy(), ref_w)
    assert_same_cache(g, c, "evict")
    table, tab, w, w_ref, lens = new, ints(new), nw, ref_w.astype(np.float64), ref_lens
    assert np.array_equal(new_lens.cpu().numpy(), lens)
    for n in (1, 4, 1, 3):
        step(n)
    _ok(fa)


def _shifted(x):
    """The same values 4 bytes behind an aligned address."""
    y = torch.empty(x.numel() + 1, dtype=x.dtype, device=x.device)[1:].view(x.shape)
    return y.copy_(x)


@pytest.mark.parametrize("rows", [(4, 1), (7, 5)])
def test_four_byte_alignment_and_shared_pages(cuda_lib, rows):
    """Scales, tables, lengths, positions and weights on 4-byte addresses, and a prefix of pages that sequences share
    while they are read: the results of aligned tensors, bit for bit, and of a cache of their own."""
    G, Nq = rows
    Hkv, page, sb, d, B = 2, 16, 4, 64, 3
    c = random_cache(8, 24, Hkv, page, sb, d)
    own = table_of(5, B, 6, 24)
    shared = own.copy()
    shared[:, :2] = own[0, :2]
    for b in range(1, B):                       # the same tokens in pages of their own
        for n in c:
            c[n][own[b, :2]] = c[n][own[0, :2]]
    rng = np.random.default_rng(11)
    k, v = bf16(rng, (B, Hkv, 5, d)).to(DEV), bf16(rng, (B, Hkv, 5, d)).to(DEV)
    q = bf16(rng, (B, Hkv * G, Nq, d)).to(DEV)
    turns = cuda_lib.rope_table(10000.0 ** (-2.0 * np.arange(16) / 32))
    pos, lens, new = ints(rng.integers(0, 999, (B, 5))), ints([40, 33, 70]), ints([5, 0, 3])
    after = ints([45, 33, 73])
    out = []
    for table, move in ((own, lambda x: x), (own, _shifted), (shared, _shifted)):
        g = to_gpu(c)
        for n in ("ks", "vs"):
            g[n] = move(g[n])
        tab, w = move(ints(table)), move(torch.zeros((B, Hkv, 96), device=DEV))
        cuda_lib.cache_append_fp8(k, v, *args(g), tab, move(lens), move(new), turns, move(pos))
        got = list(cuda_lib.decode_paged_fp8(q, *args(g), tab, move(after), weights=w)) + [w]
        fresh = np.setdiff1d(np.arange(24), own)[:6].reshape(B, 2)
        got += list(cuda_lib.cache_evict_fp8(*args(g), tab, move(after), w, move(ints(fresh)), 30, 4))
        got += [g[n][torch.from_numpy(fresh.reshape(-1)).long()] for n in g]
        out.append(got)
    _ok(cuda_lib)
    for other in out[1:]:
        assert all(torch.equal(a, b) for a, b in zip(out[0], other))
