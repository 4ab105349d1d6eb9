"""fa_cache_append_fp8 against float64, byte for byte."""
import numpy as np
import pytest
import torch

import exact_tiled_attention_21_gb300 as fa_mod
from oracle import cache as oc
from tests.cache_fp8_common import (DEV, args, assert_same_cache, bf16, copy, f64, ints, random_cache, table_of, to_gpu)

pytestmark = pytest.mark.gpu


def _ok(fa):
    st, detail = fa.fa_get_last_device_error()
    assert st == 0, detail


# (Hkv, N, d, page, sb, lens, new)
CASES = [
    (1, 1, 64, 16, 16, [0], [1]),
    (2, 1, 128, 16, 16, [0, 15, 16, 17, 31], None),
    (2, 5, 128, 16, 8, [0, 7, 8, 30], [5, 5, 0, 2]),
    (3, 37, 64, 20, 4, [0, 3, 19], [37, 1, 36]),
    (1, 100, 128, 64, 32, [0, 31, 33, 64], [100, 99, 0, 50]),
    (2, 129, 64, 128, 128, [0, 127, 200], None),
    (2, 64, 128, 128, 64, [1, 64], None),
    (1, 300, 128, 256, 128, [0, 5], [300, 77]),
    (2, 50, 64, 48, 24, [23, 24, 25], None),
    (1, 9, 128, 1, 1, [0, 4], None),
    (1, 40, 64, 33, 11, [10, 11], None),
    (1, 3, 64, 96, 96, [95, 90], None),
    # several small blocks per CTA: of odd sizes, over ends of pages, behind a partly filled block
    (2, 150, 128, 12, 3, [0, 1, 2, 3, 100], None),
    (1, 200, 64, 4, 2, [0, 7], [200, 0]),
    (2, 90, 128, 4, 1, [5, 0], [90, 13]),
    (3, 100, 64, 40, 8, [7, 33, 39], [1, 100, 64]),
    (1, 61, 128, 8, 8, [4], None),
]


@pytest.mark.parametrize("Hkv,N,d,page,sb,lens,new", CASES)
@pytest.mark.parametrize("layout", ["bhnd", "bnhd", "packed"])
def test_append_bytes(cuda_lib, Hkv, N, d, page, sb, lens, new, layout):
    """Without rotation every byte and scale is the oracle's: rows that are not written keep theirs, padding rows
    of the new tokens may hold anything."""
    B = len(lens)
    rng = np.random.default_rng(N * 7 + sb + d)
    maxp = -(-(max(lens) + N) // page)
    pages = B * maxp + 2
    c = random_cache(N + page, pages, Hkv, page, sb, d)
    table = table_of(sb, B, maxp, pages)
    k, v = bf16(rng, (B, Hkv, N, d)), bf16(rng, (B, Hkv, N, d), 2.0)
    k[:, :, 0, 1] = 0.0
    if new is not None:
        for b in range(B):
            k[b, :, new[b]:] = float("nan")
            v[b, :, new[b]:] = float("inf")
    g = to_gpu(c)
    kd, vd = k.to(DEV), v.to(DEV)
    if layout == "bnhd":
        kd, vd = (t.transpose(1, 2).contiguous().transpose(1, 2) for t in (kd, vd))
    elif layout == "packed":
        kv = torch.stack([kd.transpose(1, 2), vd.transpose(1, 2)], 2).contiguous()   # [B, N, 2, Hkv, d]
        kd, vd = kv[:, :, 0].transpose(1, 2), kv[:, :, 1].transpose(1, 2)
    cuda_lib.cache_append_fp8(kd, vd, *args(g), ints(table), ints(lens), None if new is None else ints(new))
    _ok(cuda_lib)
    oc.append(c, table, lens, f64(k), f64(v), new)
    assert_same_cache(g, c)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("N,d,rot,page,sb,lens", [(1, 128, 128, 16, 16, [5, 16, 900]), (70, 64, 32, 32, 32, [0, 17]),
                                                  (33, 128, 48, 64, 64, [3]), (75, 128, 128, 20, 4, [3, 0]),
                                                  (41, 64, 16, 2, 1, [6])])
def test_append_rotates_as_rope_does(cuda_lib, N, d, rot, page, sb, lens, given, inter):
    """Rotation on the way: bit for bit fa_rope followed by the append; V is never rotated."""
    B, Hkv = len(lens), 2
    rng = np.random.default_rng(N + d)
    maxp = -(-(max(lens) + N) // page)
    c = random_cache(3, B * maxp, Hkv, page, sb, d)
    table = ints(table_of(4, B, maxp, B * maxp))
    k, v = bf16(rng, (B, Hkv, N, d)).to(DEV), bf16(rng, (B, Hkv, N, d)).to(DEV)
    turns = cuda_lib.rope_table(10000.0 ** (-2.0 * np.arange(rot // 2) / rot))
    at = torch.from_numpy(np.array(lens)[:, None] + np.arange(N)).to(DEV, torch.int32)
    pos = at * 3 + 100000 if given else at
    one, two = to_gpu(c), to_gpu(c)
    cuda_lib.cache_append_fp8(k, v, *args(one), table, ints(lens), turns=turns, positions=pos if given else None,
                              interleaved=inter, magnitude=1.25)
    turned = cuda_lib.rope(k, turns, pos.contiguous(), inter, 1.25)
    cuda_lib.cache_append_fp8(turned, v, *args(two), table, ints(lens))
    _ok(cuda_lib)
    for n in one:
        assert torch.equal(one[n], two[n]), n
    oc.append(c, table.cpu().numpy(), lens, f64(turned), f64(v))
    assert_same_cache(one, c)


@pytest.mark.parametrize("sb,page", [(16, 16), (24, 48), (128, 128), (4, 20), (1, 8)])
def test_append_token_by_token(cuda_lib, sb, page):
    """A sequence written one token at a time holds what one call writes (no element becomes subnormal here), and
    tokens of growing size rescale the block's earlier ones."""
    rng = np.random.default_rng(sb)
    N, Hkv, d = 150, 2, 64
    x = np.sign(rng.standard_normal((1, Hkv, N, d))) * rng.uniform(0.5, 1.0, (1, Hkv, N, d)) * 2.0 ** (np.arange(N) % 7)[:, None]
    k = torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16).to(DEV)
    maxp = -(-N // page)
    c = random_cache(9, maxp + 1, Hkv, page, sb, d)
    table = table_of(2, 1, maxp, maxp + 1)
    one, two = to_gpu(c), to_gpu(c)
    cuda_lib.cache_append_fp8(k, k, *args(one), ints(table), ints([0]))
    for t in range(N):
        cuda_lib.cache_append_fp8(k[:, :, t:t + 1], k[:, :, t:t + 1], *args(two), ints(table), ints([t]))
    _ok(cuda_lib)
    oc.append(c, table, [0], f64(k), f64(k))
    assert_same_cache(one, c)
    used = table[0]
    for n in one:
        assert torch.equal(one[n][used], two[n][used]), n


def test_append_rescales_subnormals_and_foreign_scales(cuda_lib):
    """A huge token after small ones pushes them to subnormals or zero; scales that are no powers of two (another
    writer's) are divided by as they are."""
    Hkv, d, page, sb = 2, 64, 32, 32
    rng = np.random.default_rng(0)
    c = random_cache(5, 2, Hkv, page, sb, d)
    c["ks"] = np.full_like(c["ks"], np.float32(0.0123)).astype(np.float32).astype(np.float64)
    c["vs"] = np.full_like(c["vs"], np.float32(3.3e-5)).astype(np.float32).astype(np.float64)
    k, v = bf16(rng, (1, Hkv, 3, d)) * 100, bf16(rng, (1, Hkv, 3, d)) * 1e-3
    k[0, 0] *= 1e-4   # smaller than the block's scale asks: stays with 0.0123
    g = to_gpu(c)
    table = np.array([[1]], dtype=np.int32)
    cuda_lib.cache_append_fp8(k.to(DEV), v.to(DEV), *args(g), ints(table), ints([20]))
    _ok(cuda_lib)
    got = {n: g[n].cpu().numpy() for n in g}
    for n, s, x in (("k", "ks", k), ("v", "vs", v)):
        for h in range(Hkv):
            # fp32 steps of the kernel: value * old / new, rounded twice before e4m3
            old = np.float32(c[s][1, h, 0])
            amax = float(x[0, h].float().abs().max())
            to = max(old, np.float32(oc.scale_for(amax)))
            assert got[s][1, h, 0] == to
            want = (oc._E4M3[c[n][1, h, :20]].astype(np.float32) * old) / to
            assert np.array_equal(got[n][1, h, :20], oc.to_e4m3(want.astype(np.float64)))
            new = x[0, h].float().numpy() / to
            assert np.array_equal(got[n][1, h, 20:23], oc.to_e4m3(new.astype(np.float64)))
            assert np.array_equal(got[n][1, h, 23:], c[n][1, h, 23:])


def test_append_special_values(cuda_lib):
    """Infinities saturate, NaN stays, neither moves the scale; zeros and bf16 subnormals take the smallest scale."""
    Hkv, d, page, sb = 1, 64, 16, 4
    c = random_cache(6, 1, Hkv, page, sb, d)
    k = torch.zeros((1, 1, 16, d), dtype=torch.bfloat16)
    k[0, 0, 4:8] = 3.0
    k[0, 0, 5, 7], k[0, 0, 6, 8], k[0, 0, 7, 9] = float("inf"), float("-inf"), float("nan")
    k[0, 0, 8, :5] = torch.tensor([1e-39, -1e-40, 2e-38, 0.0, -0.0])
    k[0, 0, 12, :4] = torch.tensor([3.3895e38, -3.3895e38, 1.0, 2.9e38])
    g = to_gpu(c)
    table = np.zeros((1, 1), dtype=np.int32)
    cuda_lib.cache_append_fp8(k.to(DEV), k.to(DEV), *args(g), ints(table), ints([0]))
    _ok(cuda_lib)
    oc.append(c, table, [0], f64(k), f64(k))
    assert_same_cache(g, c)
    assert g["ks"][0, 0, 0] == 2.0 ** -126 and g["ks"][0, 0, 3] == 2.0 ** 120


def test_append_overflow_and_bad_tables(cuda_lib):
    """Tokens behind the last page, lengths out of range and pages that do not exist are left out and recorded."""
    Hkv, d, page, sb, N = 2, 64, 16, 16, 8
    rng = np.random.default_rng(1)
    k, v = bf16(rng, (3, Hkv, N, d)), bf16(rng, (3, Hkv, N, d))
    base = random_cache(7, 9, Hkv, page, sb, d)
    table = table_of(8, 3, 2, 9)

    def run(lens, new=None, tab=table):
        c, g = copy(base), to_gpu(base)
        cuda_lib.cache_append_fp8(k.to(DEV), v.to(DEV), *args(g), ints(tab), ints(lens), None if new is None else ints(new))
        st, _ = cuda_lib.fa_get_last_device_error()
        return c, g, st

    c, g, st = run([28, 0, 32])       # four of eight fit; all; none
    assert st == fa_mod.FA_ERR_INVALID_ARG
    oc.append(c, table, [28, 0, 32], f64(k), f64(v))
    assert_same_cache(g, c)
    c, g, st = run([0, 0, 0], [9, -1, 3])
    assert st == fa_mod.FA_ERR_INVALID_ARG
    oc.append(c, table, [0, 0, 0], f64(k), f64(v), [8, 0, 3])
    assert_same_cache(g, c)
    c, g, st = run([-5, 0, 40], [2, 2, 2])
    assert st == fa_mod.FA_ERR_INVALID_ARG
    oc.append(c, table, [0, 0, 32], f64(k), f64(v), [2, 2, 0])
    assert_same_cache(g, c)
    bad = table.copy()
    bad[0, 0], bad[1, 0], bad[2, 1] = 9, -1, 1 << 30   # the last one is not reached
    c, g, st = run([0, 0, 0], None, bad)
    assert st == fa_mod.FA_ERR_INVALID_ARG
    oc.append(c, table[2:], [0], f64(k)[2:], f64(v)[2:])
    assert_same_cache(g, c)
    assert run([0, 16, 24])[2] == 0


def test_append_bad_page_among_small_blocks(cuda_lib):
    """A CTA's blocks of 4 tokens lie in several pages: those of one that does not exist are left out, the others
    written."""
    Hkv, d, page, sb, N = 2, 128, 8, 4, 60
    rng = np.random.default_rng(2)
    k, v = bf16(rng, (1, Hkv, N, d)), bf16(rng, (1, Hkv, N, d))
    c = random_cache(3, 10, Hkv, page, sb, d)
    table = table_of(9, 1, 8, 10)
    g, bad = to_gpu(c), table.copy()
    bad[0, 1], bad[0, 4] = -1, 10
    cuda_lib.cache_append_fp8(k.to(DEV), v.to(DEV), *args(g), ints(bad), ints([2]))
    assert cuda_lib.fa_get_last_device_error()[0] == fa_mod.FA_ERR_INVALID_ARG
    ref = copy(c)
    oc.append(ref, table, [2], f64(k), f64(v))
    for n in c:
        for j in (1, 4):
            ref[n][table[0, j]] = c[n][table[0, j]]
    assert_same_cache(g, ref)


def test_append_far_pages(cuda_lib):
    """A pool of more than 2^32 bytes: the last page is written, and nothing else."""
    Hkv, d, page = 8, 128, 64
    pages = 2 ** 32 // (Hkv * d * page) + 3
    k = bf16(np.random.default_rng(2), (1, Hkv, 5, d)).to(DEV)
    g = {n: torch.zeros((pages, Hkv, page, d), dtype=torch.uint8, device=DEV) for n in ("k", "v")}
    g |= {n: torch.zeros((pages, Hkv, 1), device=DEV) for n in ("ks", "vs")}
    cuda_lib.cache_append_fp8(k, k, *args(g), ints([[pages - 1]]), ints([59]))
    _ok(cuda_lib)
    small = {n: np.zeros((1, Hkv, page, d), dtype=np.uint8) for n in ("k", "v")}
    small |= {n: np.zeros((1, Hkv, 1)) for n in ("ks", "vs")}
    oc.append(small, np.zeros((1, 1), dtype=np.int64), [59], f64(k), f64(k))
    assert_same_cache({n: g[n][-1:] for n in g}, small)
    assert int(g["k"][:-1].view(torch.int64).count_nonzero()) == 0 and int(g["ks"][:-1].count_nonzero()) == 0


def test_append_streams_and_graph(cuda_lib):
    """Two sequences' appends on two streams, and a captured append replayed with other inputs."""
    Hkv, d, page, sb = 2, 128, 32, 32
    rng = np.random.default_rng(3)
    k = bf16(rng, (1, Hkv, 40, d)).to(DEV)
    c = random_cache(1, 4, Hkv, page, sb, d)
    g = to_gpu(c)
    t = [np.array([[0, 2]]), np.array([[3, 1]])]
    ts, zero = [ints(x) for x in t], ints([0])
    streams = [torch.cuda.Stream() for _ in t]
    for s, tab in zip(streams, ts):
        s.wait_stream(torch.cuda.current_stream())
        cuda_lib.cache_append_fp8(k, k, *args(g), tab, zero, stream=s)
    torch.cuda.synchronize()
    for x in t:
        oc.append(c, x, [0], f64(k), f64(k))
    assert_same_cache(g, c)
    lens, x = ints([40]), k[:, :, :1].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cuda_lib.cache_append_fp8(x, x, *args(g), ts[0], lens)
        lens += 1
    for i in range(3):
        x.copy_(k[:, :, i + 5:i + 6] * (4.0 ** i))
        xi = f64(x)
        graph.replay()
        oc.append(c, t[0], [40 + i], xi, xi)
    torch.cuda.synchronize()
    assert_same_cache(g, c)
    _ok(cuda_lib)


def test_append_shape_refusals(cuda_lib):
    g = to_gpu(random_cache(1, 4, 2, 16, 8, 64))
    k = torch.zeros((1, 2, 3, 64), dtype=torch.bfloat16, device=DEV)
    tab, lens = ints([[0, 1]]), ints([0])
    for bad in (dict(k=k[:, :1]), dict(k=k.half()), dict(lens=ints([0, 0])), dict(tab=tab.long()), dict(ks=g["ks"][:3]),
                dict(ks=g["ks"].double()), dict(new=ints([1, 1]))):
        a = dict(k=k, lens=lens, tab=tab, ks=g["ks"], new=None) | bad
        with pytest.raises(ValueError):
            cuda_lib.cache_append_fp8(a["k"], k, g["k"], g["v"], a["ks"], g["vs"], a["tab"], a["lens"], a["new"])
    with pytest.raises(ValueError):
        cuda_lib.cache_append_fp8(k, k, g["k"], g["v"], g["ks"], g["vs"], tab, lens, turns=torch.zeros(32, device=DEV))
