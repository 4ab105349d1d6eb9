"""fa_decode_paged_fp8 against the fp64 attention of the values that the cache stands for."""
import math

import numpy as np
import pytest
import torch

import exact_tiled_attention_21_gb300 as fa_mod
from oracle import cache as oc
from tests.cache_fp8_common import (DEV, args, bf16, check_decode, copy, f64, ints, random_cache, table_of, to_gpu)

pytestmark = pytest.mark.gpu


def _ok(fa):
    st, detail = fa.fa_get_last_device_error()
    assert st == 0, detail


def _case(seed, B, Hq, Hkv, Nq, page, sb, lens, d):
    maxp = max(1, -(-max(lens) // page))
    c = random_cache(seed, B * maxp + 2, Hkv, page, sb, d)
    return bf16(np.random.default_rng(seed + 1), (B, Hq, Nq, d), 0.3), c, table_of(seed + 2, B, maxp, B * maxp + 2)


# (Hq, Hkv, Nq, page, sb, lens, d)
CASES = [
    (1, 1, 1, 16, 16, [1], 64),
    (8, 2, 1, 16, 16, [1, 37, 200], 128),
    (8, 2, 1, 16, 16, [0, 33, 0, 128, 129], 128),      # sequences without tokens
    (8, 2, 1, 16, 16, [0, 0], 64),                     # none at all
    (6, 2, 1, 64, 32, [64, 1000], 64),
    (16, 2, 1, 32, 8, [1500, 513], 128),
    (32, 2, 1, 16, 4, [300, 17], 128),                 # 16 heads a group: two column tiles
    (40, 2, 1, 16, 16, [300, 17], 64),                 # 20: a tile of 32 rows, partly empty
    (5, 1, 1, 1, 1, [77], 128),                        # single-token pages and scales
    (4, 4, 1, 20, 20, [129, 1], 64),
    (4, 2, 1, 33, 11, [500, 64], 128),
    (7, 1, 1, 128, 128, [2000], 64),
    (3, 3, 1, 256, 64, [1000, 255], 128),
    (8, 2, 4, 16, 16, [4, 3, 1, 0, 500], 128),         # drafted tokens: rows that see no key
    (2, 2, 16, 48, 24, [16, 100, 31], 64),
    (16, 1, 5, 64, 64, [300, 5], 128),                 # 80 rows: three row tiles
    (21, 3, 5, 32, 32, [300, 70], 128),                # 35 rows: an odd number in the last tile, an odd kv head
    (21, 3, 5, 32, 32, [301, 71], 64),
    (9, 3, 3, 16, 16, [130, 20], 128),                 # 9 rows
    (6, 2, 2, 32, 16, [33, 64, 95], 64),
    (8, 8, 1, 64, 64, [9000], 128),                    # long: segments of many steps
    (8, 8, 1, 64, 64, [9000], 64),
    (4, 1, 1, 64, 64, [70000], 128),                   # one kv head over every SM: hundreds of segments to merge
    (1, 1, 1, 16, 16, list(range(0, 200, 3)) * 2, 64),  # more sequences than one scan step, some empty
    (2, 1, 2, 16, 16, [130] * 300, 128),               # more items than CTAs: shares that cross several
    (16, 1, 5, 16, 16, [0, 20, 3, 300, 1, 129] * 10, 128),   # 4800 rows: finished by runs
    (16, 1, 5, 16, 16, [7, 0, 140, 16] * 60, 64),            # 19200
    (9, 1, 1, 64, 64, [2000, 700] * 140, 128),               # 2520, of one tile each
]


@pytest.mark.parametrize("weights", [False, True])
@pytest.mark.parametrize("Hq,Hkv,Nq,page,sb,lens,d", CASES)
def test_decode_parity(cuda_lib, Hq, Hkv, Nq, page, sb, lens, d, weights):
    B = len(lens)
    q, c, table = _case(page * 3 + Hq + d, B, Hq, Hkv, Nq, page, sb, lens, d)
    g = to_gpu(c)
    cap = table.shape[1] * page
    w0 = np.random.default_rng(1).uniform(0, 2, (B, Hkv, cap)).astype(np.float32)
    w = torch.from_numpy(w0).to(DEV) if weights else None
    o, lse = cuda_lib.decode_paged_fp8(q.to(DEV), *args(g), ints(table), ints(lens), weights=w)
    _ok(cuda_lib)
    w_ref = w0.astype(np.float64)
    ref = oc.decode(f64(q), c, table, lens, 1 / math.sqrt(d), w_ref)
    check_decode(o, lse, ref, w, w_ref)
    if weights:
        for b in range(B):
            assert np.array_equal(w[b, :, lens[b]:].cpu().numpy(), w0[b, :, lens[b]:])   # behind the sequence
    if Nq == 1:
        o3, l3 = cuda_lib.decode_paged_fp8(q[:, :, 0].to(DEV), *args(g), ints(table), ints(lens))
        assert torch.equal(o3, o[:, :, 0]) and torch.equal(l3, lse[:, :, 0])


def test_decode_matches_the_bf16_decode(cuda_lib):
    """The cache's values are exact in bf16 (e4m3 times a power of two), so the framework's bf16 paged decode computes
    the same; its own weights are rounded to bf16 (2^-8), the 8-bit path's bounds aside."""
    B, Hq, Hkv, page, d, lens = 3, 8, 2, 64, 128, [700, 64, 1]
    q, c, table = _case(11, B, Hq, Hkv, 1, page, 32, lens, d)
    g = to_gpu(c)
    o, lse = cuda_lib.decode_paged_fp8(q[:, :, 0].to(DEV), *args(g), ints(table), ints(lens))
    val = {n: (torch.from_numpy(oc._E4M3[c[n]]) * torch.from_numpy(c[n + "s"]).repeat_interleave(32, 2)[..., None])
           .to(torch.bfloat16).to(DEV) for n in ("k", "v")}
    o2, lse2 = cuda_lib.decode_paged(q[:, :, 0].contiguous().to(DEV), val["k"], val["v"], ints(table), ints(lens))
    _ok(cuda_lib)
    ref = oc.decode(f64(q), c, table, lens, 1 / math.sqrt(d))
    assert np.abs(f64(o) - f64(o2)).max() <= 2.0 ** -6 * ref[3].max()
    assert np.abs(f64(lse) - f64(lse2)).max() <= 1e-3


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Nq", [1, 3])
def test_decode_ignores_what_is_behind_the_sequence(cuda_lib, d, Nq):
    """NaN bytes and scales behind seq_lens, in unused blocks and in pages that no table names change nothing, nor do
    table entries behind the last page in use."""
    page, sb, lens = 48, 16, [100, 3, 48]
    q, c, table = _case(21, 3, 8, 2, Nq, page, sb, lens, d)
    table = np.concatenate([table, np.full((3, 1), 1 << 30, dtype=np.int32)], 1)
    used = np.zeros((c["k"].shape[0], page), dtype=bool)
    for b, n in enumerate(lens):
        for j in range(n):
            used[table[b, j // page], j % page] = True
    bad = copy(c)
    for n in ("k", "v"):
        bad[n][np.broadcast_to(~used[:, None], bad[n].shape[:3])] = 0x7F
        dead = ~used.reshape(-1, page // sb, sb).any(-1)
        bad[n + "s"][np.broadcast_to(dead[:, None], bad[n + "s"].shape)] = np.nan
    out = []
    for x in (c, bad):
        w = torch.zeros((3, 2, table.shape[1] * page), device=DEV)
        out.append(cuda_lib.decode_paged_fp8(q.to(DEV), *args(to_gpu(x)), ints(table), ints(lens), weights=w) + (w,))
    _ok(cuda_lib)
    for a, b in zip(*out):
        assert torch.equal(a, b) and a.isfinite().all()
    check_decode(out[0][0], out[0][1], oc.decode(f64(q), c, table, lens, 1 / math.sqrt(d)))


def test_decode_scale_ranges(cuda_lib):
    """Block scales from 2^-126 to 2^100 within one sequence, queries from 2^-100 to 2^30, rows of zeros: the result
    keeps its relative precision."""
    B, Hq, Hkv, page, sb, d, n = 2, 4, 2, 32, 8, 128, 150
    q, c, table = _case(31, B, Hq, Hkv, 1, page, sb, [n, n], d)
    rng = np.random.default_rng(5)
    c["vs"] = 2.0 ** rng.integers(-126, 100, c["vs"].shape).astype(np.float64)
    c["ks"] = 2.0 ** rng.integers(-16, -6, c["ks"].shape).astype(np.float64)
    q[0, 0] *= 2.0 ** -100
    q[0, 1] = 0
    q[1, 2, 0, :5] *= 2.0 ** -30
    g = to_gpu(c)
    o, lse = cuda_lib.decode_paged_fp8(q.to(DEV), *args(g), ints(table), ints([n, n]))
    check_decode(o, lse, oc.decode(f64(q), c, table, [n, n], 1 / math.sqrt(d)))
    big = q.clone()
    big[1] *= 2.0 ** 30
    c["ks"] *= 2.0 ** -30
    o, lse = cuda_lib.decode_paged_fp8(big.to(DEV), *args(to_gpu(c)), ints(table), ints([n, n]))
    check_decode(o[1:], lse[1:], tuple(x[1:] for x in oc.decode(f64(big), c, table, [n, n], 1 / math.sqrt(d))))
    c["vs"][:] = 0.0   # values of zero
    o, lse = cuda_lib.decode_paged_fp8(q.to(DEV), *args(to_gpu(c)), ints(table), ints([n, n]))
    assert (o == 0).all() and lse.isfinite().all()
    _ok(cuda_lib)


def test_decode_wide_table(cuda_lib):
    """A block table of far more pages than any sequence uses: the work goes by the lengths, and the result is that of
    a narrow one, bit for bit."""
    lens = [300, 0, 129]
    q, c, table = _case(35, 3, 8, 2, 1, 16, 8, lens, 128)
    g = to_gpu(c)
    wide = np.full((3, 5000), -7, dtype=np.int32)
    wide[:, :table.shape[1]] = table
    a = cuda_lib.decode_paged_fp8(q.to(DEV), *args(g), ints(table), ints(lens))
    b = cuda_lib.decode_paged_fp8(q.to(DEV), *args(g), ints(wide), ints(lens))
    _ok(cuda_lib)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_decode_nan_shows(cuda_lib):
    """A NaN in a visible key or value, or in q, reaches its row's output."""
    q, c, table = _case(41, 1, 4, 2, 1, 16, 16, [50], 64)
    c["k"][table[0, 1], 0, 3, 5] = 0x7F
    c["v"][table[0, 2], 1, 7, 9] = 0xFF
    o, lse = cuda_lib.decode_paged_fp8(q.to(DEV), *args(to_gpu(c)), ints(table), ints([50]))
    assert o[0, :2].isnan().all() and lse[0, :2].isnan().all()
    assert o[0, 2:, 0, 9].isnan().all() and int(o[0, 2:].isnan().sum()) == 2 and lse[0, 2:].isfinite().all()


def test_decode_sharp_softmax(cuda_lib):
    """Scores spread over hundreds: one key takes all the weight, whatever the order of the running maximum."""
    q, c, table = _case(51, 2, 8, 2, 2, 32, 32, [400, 399], 128)
    q = q * 30
    w_ref = np.zeros((2, 2, table.shape[1] * 32))
    w = torch.zeros(w_ref.shape, device=DEV)
    o, lse = cuda_lib.decode_paged_fp8(q.to(DEV), *args(to_gpu(c)), ints(table), ints([400, 399]), weights=w)
    ref = oc.decode(f64(q), c, table, [400, 399], 1 / math.sqrt(128), w_ref)
    check_decode(o, lse, ref, w, w_ref)


def test_decode_bad_lengths_and_pages(cuda_lib):
    """Lengths are clamped and missing pages read as zeros (K and V), recorded in the error word."""
    page, d = 16, 64
    q, c, table = _case(61, 2, 4, 2, 1, page, 16, [40, 48], d)
    run = lambda tab, lens: cuda_lib.decode_paged_fp8(q.to(DEV), *args(to_gpu(c)), ints(tab), ints(lens))
    o, lse = run(table, [-3, 49])
    assert cuda_lib.fa_get_last_device_error()[0] == fa_mod.FA_ERR_INVALID_ARG
    check_decode(o, lse, oc.decode(f64(q), c, table, [0, 48], 0.125))
    for wrong in (c["k"].shape[0], -1, 1 << 30, -(1 << 31)):
        tab = table.copy()
        tab[0, 1] = wrong
        o, lse = run(tab, [40, 48])
        assert cuda_lib.fa_get_last_device_error()[0] == fa_mod.FA_ERR_INVALID_ARG
        z = {n: np.concatenate([c[n], np.zeros_like(c[n][:1])]) for n in c}
        z["vs"][-1] = 1.0
        tab[0, 1] = c["k"].shape[0]
        check_decode(o, lse, oc.decode(f64(q), z, tab, [40, 48], 0.125))
    run(table, [40, 48])
    _ok(cuda_lib)


def test_decode_far_pages(cuda_lib):
    """A pool of more than 2^32 bytes gives the bits that a small one gives."""
    Hkv, d, page, n = 8, 128, 64, 200
    q, c, table = _case(71, 1, 16, Hkv, 1, page, 32, [n], d)
    small = to_gpu(c)
    pages = 2 ** 32 // (Hkv * d * page) + 9
    far = {k: torch.zeros((pages,) + tuple(small[k].shape[1:]), dtype=small[k].dtype, device=DEV) for k in small}
    P = small["k"].shape[0]
    for k in small:
        far[k][-P:] = small[k]
    a = cuda_lib.decode_paged_fp8(q.to(DEV), *args(small), ints(table), ints([n]))
    b = cuda_lib.decode_paged_fp8(q.to(DEV), *args(far), ints(table + pages - P), ints([n]))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    _ok(cuda_lib)


def test_decode_repeats_streams_and_graphs(cuda_lib):
    """The same bits every time; on several streams at once; in two graphs replayed in turn, with lengths that grow."""
    q, c, table = _case(81, 4, 16, 4, 2, 16, 16, [1000, 900, 1, 500], 128)
    g, qd, tab = to_gpu(c), q.to(DEV), ints(table)
    lens = ints([1000, 900, 1, 500])
    W = torch.zeros((4, 4, table.shape[1] * 16), device=DEV)
    want = cuda_lib.decode_paged_fp8(qd, *args(g), tab, lens, weights=W)
    for _ in range(20):
        w = torch.zeros_like(W)
        got = cuda_lib.decode_paged_fp8(qd, *args(g), tab, lens, weights=w)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.equal(w, W)
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for i in range(9):
        outs.append(cuda_lib.decode_paged_fp8(qd, *args(g), tab, lens, stream=streams[i % 3]))
    torch.cuda.synchronize()
    assert all(torch.equal(o[0], want[0]) and torch.equal(o[1], want[1]) for o in outs)
    graphs = []
    for _ in range(2):
        gr, w = torch.cuda.CUDAGraph(), torch.zeros_like(W)
        with torch.cuda.graph(gr):
            out = cuda_lib.decode_paged_fp8(qd, *args(g), tab, lens, weights=w)
        graphs.append((gr, out, w))
    for n in ([0, 16, 77, 512], [1008, 2, 1, 300]):
        lens.copy_(ints(n))
        w_ref = np.zeros(W.shape)
        ref = oc.decode(f64(q), c, table, n, 1 / math.sqrt(128), w_ref)
        for gr, out, w in graphs:
            w.zero_()
            gr.replay()
            torch.cuda.synchronize()
            check_decode(out[0], out[1], ref, w, w_ref)
    _ok(cuda_lib)


def test_decode_own_workspace_and_refusals(cuda_lib):
    q, c, table = _case(91, 2, 8, 2, 1, 16, 16, [100, 50], 64)
    g, qd, tab, lens = to_gpu(c), q.to(DEV), ints(table), ints([100, 50])
    n = cuda_lib.fa_decode_paged_fp8_workspace_bytes(2, 8, 2, 1, 64, table.shape[1] * 16, True)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV)   # its contents (NaN here) do not matter
    w = torch.zeros((2, 2, table.shape[1] * 16), device=DEV)
    o, lse = cuda_lib.decode_paged_fp8(qd, *args(g), tab, lens, weights=w, workspace=ws)
    w_ref = np.zeros(w.shape)
    check_decode(o, lse, oc.decode(f64(q), c, table, [100, 50], 0.125, w_ref), w, w_ref)
    with pytest.raises(fa_mod.FAError) as e:
        cuda_lib.decode_paged_fp8(qd, *args(g), tab, lens, weights=w, workspace=ws[:n - 256])
    assert e.value.status == fa_mod.FA_ERR_WORKSPACE
    for bad in (dict(q=qd.float()), dict(q=qd[:1]), dict(q=qd[..., :32]), dict(w=w[:, :1].contiguous()), dict(w=w.double()),
                dict(lens=lens.long()), dict(tab=tab.t())):
        a = dict(q=qd, w=w, lens=lens, tab=tab) | bad
        with pytest.raises(ValueError):
            cuda_lib.decode_paged_fp8(a["q"], *args(g), a["tab"], a["lens"], weights=a["w"])
    with pytest.raises(fa_mod.FAError):
        cuda_lib.decode_paged_fp8(qd[:, :7].contiguous(), *args(g), tab, lens)
    _ok(cuda_lib)
