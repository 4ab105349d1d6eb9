"""Rotary positions and the 8-bit cache: what the host checks, before any CUDA call."""
import ctypes
import math

import pytest
import torch

import exact_tiled_attention_21_gb300 as fa

vp = ctypes.c_void_p
NAN = float("nan")


@pytest.fixture(scope="module")
def lib():
    fa.build()
    return fa.load()


def _rope(lib, x=16, y=32, xs=(0, 0, 64), ys=(0, 0, 64), pos=0, turns=16, B=1, H=1, N=8, d=64, rot=64, inter=0,
          mag=1.0, inv=0):
    return lib.fa_rope(vp(x), vp(y), *xs, *ys, vp(pos), vp(turns), B, H, N, d, rot, inter, mag, inv, None)


@pytest.mark.parametrize("bad,status", [
    (dict(x=0), fa.FA_ERR_INVALID_ARG), (dict(y=0), fa.FA_ERR_INVALID_ARG), (dict(turns=0), fa.FA_ERR_INVALID_ARG),
    (dict(B=0), fa.FA_ERR_INVALID_ARG), (dict(H=-1), fa.FA_ERR_INVALID_ARG), (dict(N=0), fa.FA_ERR_INVALID_ARG),
    (dict(d=96), fa.FA_ERR_UNSUPPORTED), (dict(rot=0), fa.FA_ERR_INVALID_ARG), (dict(rot=80), fa.FA_ERR_INVALID_ARG),
    (dict(rot=24), fa.FA_ERR_UNSUPPORTED), (dict(inter=2), fa.FA_ERR_INVALID_ARG), (dict(inv=-1), fa.FA_ERR_INVALID_ARG),
    (dict(mag=NAN), fa.FA_ERR_INVALID_ARG), (dict(mag=math.inf), fa.FA_ERR_INVALID_ARG),
    (dict(x=24), fa.FA_ERR_ALIGNMENT), (dict(y=40), fa.FA_ERR_ALIGNMENT), (dict(turns=8), fa.FA_ERR_ALIGNMENT),
    (dict(pos=2), fa.FA_ERR_ALIGNMENT), (dict(xs=(0, 0, 68)), fa.FA_ERR_ALIGNMENT),
    (dict(ys=(0, 0, 60)), fa.FA_ERR_ALIGNMENT), (dict(xs=(0, 0, -64)), fa.FA_ERR_INVALID_ARG),
    (dict(ys=(0, 0, 0)), fa.FA_ERR_INVALID_ARG), (dict(ys=(0, 0, 56)), fa.FA_ERR_INVALID_ARG),      # rows overlap
    (dict(H=2, ys=(0, 256, 64)), fa.FA_ERR_INVALID_ARG),                                            # heads overlap
    (dict(B=2, H=2, ys=(64, 64, 128)), fa.FA_ERR_INVALID_ARG),
    (dict(y=16, ys=(0, 0, 128)), fa.FA_ERR_INVALID_ARG),                                            # in place, other strides
    (dict(B=1 << 16, N=1 << 16, xs=(64, 0, 64), ys=(64 << 16, 0, 64)), fa.FA_ERR_UNSUPPORTED),
])
def test_rope_refusals(lib, bad, status):
    assert _rope(lib, **bad) == status


def test_rope_table():
    f = [1.0, 10000.0 ** -0.5, -0.25, 0.0, 2 * math.pi, 7.5]
    got = fa.fa_rope_table(f)
    for t, x in zip(got, f):
        want = x / (2 * math.pi)
        want -= math.floor(want)
        d = abs(t / 2.0 ** 64 - want)
        assert min(d, 1 - d) <= 2.0 ** -52, x
    assert got[3] == 0 and got[4] == 0
    for bad in ([], [NAN], [math.inf]):
        with pytest.raises(fa.FAError):
            fa.fa_rope_table(bad)
    t = fa.rope_table(f, device="cpu")
    assert t.dtype == torch.int64 and [int(v) % (1 << 64) for v in t] == got


def test_rope_frequencies():
    f, m = fa.rope_frequencies(8)
    assert m == 1.0 and f == [1.0, 0.1, 0.01, 0.001] or all(abs(a - b) < 1e-15 for a, b in zip(f, [1, .1, .01, .001]))
    lin, m = fa.rope_frequencies(8, scaling="linear", factor=4.0)
    assert m == 1.0 and all(abs(a * 4 - b) < 1e-15 for a, b in zip(lin, f))
    ntk, m = fa.rope_frequencies(8, scaling="ntk", factor=4.0)
    assert ntk[0] == 1.0 and abs(ntk[-1] * 4 - f[-1]) < 1e-12
    yarn, m = fa.rope_frequencies(8, scaling="yarn", factor=4.0, original_context=1000)
    assert abs(m - (0.1 * math.log(4.0) + 1)) < 1e-15
    assert yarn[0] == f[0] and abs(yarn[-1] * 4 - f[-1]) < 1e-15     # 159 turns kept, 0.16 turns stretched
    turns = 1000 * f[1] / (2 * math.pi)                              # 15.9: between 1 and 32
    keep = (turns - 1) / 31
    assert abs(yarn[1] - f[1] * (keep + (1 - keep) / 4)) < 1e-15
    for bad in (dict(rot=7), dict(rot=8, scaling="other"), dict(rot=8, scaling="yarn"), dict(rot=8, factor=0.5),
                dict(rot=8, base=0.0)):
        with pytest.raises(ValueError):
            fa.rope_frequencies(**bad)


CACHE_BAD = [  # B, Hkv, page, sb, max_pages, num_pages, d
    (dict(B=0), fa.FA_ERR_INVALID_ARG), (dict(Hkv=0), fa.FA_ERR_INVALID_ARG), (dict(page=0), fa.FA_ERR_INVALID_ARG),
    (dict(sb=0), fa.FA_ERR_INVALID_ARG), (dict(sb=3), fa.FA_ERR_INVALID_ARG), (dict(mp=0), fa.FA_ERR_INVALID_ARG),
    (dict(np=0), fa.FA_ERR_INVALID_ARG), (dict(d=80), fa.FA_ERR_UNSUPPORTED),
    (dict(page=256, sb=256), fa.FA_ERR_UNSUPPORTED), (dict(mp=1 << 27), fa.FA_ERR_UNSUPPORTED),
    (dict(np=1 << 30), fa.FA_ERR_UNSUPPORTED), (dict(B=1 << 24), fa.FA_ERR_UNSUPPORTED),
]


def _append(lib, p=(16,) * 8, extra=(0, 0, 0), ks=(0, 0, 64), vs=(0, 0, 64), B=1, Hkv=2, N=4, d=64, rot=64, inter=0,
            mag=1.0, page=16, sb=8, mp=4, np=9):
    k, v, kp, vpg, sk, sv, table, lens = map(vp, p)
    new, pos, turns = map(vp, extra)
    return lib.fa_cache_append_fp8(k, v, *ks, *vs, kp, vpg, sk, sv, table, lens, new, pos, turns, B, Hkv, N, d, rot,
                                   inter, mag, page, sb, mp, np, None)


@pytest.mark.parametrize("bad,status", CACHE_BAD + [
    (dict(N=0), fa.FA_ERR_INVALID_ARG), (dict(N=(1 << 30) + 1), fa.FA_ERR_UNSUPPORTED),
    (dict(N=1 << 30), fa.FA_ERR_UNSUPPORTED), (dict(N=(1 << 29) + 8, Hkv=1), fa.FA_ERR_UNSUPPORTED),
    (dict(ks=(0, 0, 4)), fa.FA_ERR_ALIGNMENT), (dict(vs=(0, -8, 64)), fa.FA_ERR_INVALID_ARG),
    (dict(extra=(0, 0, 16), rot=20), fa.FA_ERR_UNSUPPORTED), (dict(extra=(0, 0, 16), rot=80), fa.FA_ERR_INVALID_ARG),
    (dict(extra=(0, 0, 16), mag=NAN), fa.FA_ERR_INVALID_ARG), (dict(extra=(0, 0, 8)), fa.FA_ERR_ALIGNMENT),
    (dict(extra=(2, 0, 0)), fa.FA_ERR_ALIGNMENT), (dict(extra=(0, 6, 0)), fa.FA_ERR_ALIGNMENT),
])
def test_append_refusals(lib, bad, status):
    assert _append(lib, **bad) == status


def test_append_pointer_checks(lib):
    for i in range(8):
        p = [16] * 8
        p[i] = 0
        assert _append(lib, p=p) == fa.FA_ERR_INVALID_ARG, i
        p[i] = 18
        assert _append(lib, p=p) == fa.FA_ERR_ALIGNMENT, i


def _decode(lib, p=(16,) * 7 + (32,), lse=16, w=0, B=1, Hq=4, Hkv=2, Nq=1, page=16, sb=8, mp=4, np=9, d=64, scale=0.125,
            ws=16, nbytes=1 << 30):
    return lib.fa_decode_paged_fp8(*map(vp, p), vp(lse), vp(w), B, Hq, Hkv, Nq, page, sb, mp, np, d, scale,
                                   vp(ws), nbytes, None)


@pytest.mark.parametrize("bad,status", CACHE_BAD + [
    (dict(Hq=3), fa.FA_ERR_INVALID_ARG), (dict(Hq=0), fa.FA_ERR_INVALID_ARG), (dict(Nq=0), fa.FA_ERR_INVALID_ARG),
    (dict(Nq=17), fa.FA_ERR_UNSUPPORTED), (dict(B=1 << 10, Hkv=4, mp=1 << 26), fa.FA_ERR_UNSUPPORTED),
    (dict(B=1 << 7, Hkv=2, mp=1 << 26), fa.FA_ERR_UNSUPPORTED), (dict(p=(16,) * 8), fa.FA_ERR_INVALID_ARG),
    (dict(scale=0.0), fa.FA_ERR_INVALID_ARG), (dict(scale=NAN), fa.FA_ERR_INVALID_ARG),
    (dict(lse=6), fa.FA_ERR_ALIGNMENT), (dict(w=2), fa.FA_ERR_ALIGNMENT),
])
def test_decode_refusals(lib, bad, status):
    assert _decode(lib, **bad) == status


def test_decode_pointer_checks(lib):
    for i in range(8):
        p = [16] * 8
        p[i] = 0
        assert _decode(lib, p=p) == fa.FA_ERR_INVALID_ARG, i
        p[i] = 18
        assert _decode(lib, p=p) == fa.FA_ERR_ALIGNMENT, i


def test_decode_workspace_query():
    q = fa.fa_decode_paged_fp8_workspace_bytes
    # a slot (rows of a tile by d + 1 floats) for each of 1024 CTAs and for each item
    assert q(2, 8, 2, 1, 128, 4096, False) >= (1024 + 4) * 8 * 129 * 4 + 3 * 8
    assert q(2, 40, 2, 4, 64, 4096, False) >= (1024 + 2 * 2 * 3) * 32 * 65 * 4
    # and the scores, rows padded to a multiple of four
    assert q(2, 10, 2, 3, 128, 4097, True) - q(2, 10, 2, 3, 128, 4097, False) >= 2 * 2 * 16 * 4097 * 4
    assert q(1, 8, 8, 1, 128, 1, False) == q(1, 8, 8, 1, 128, 1 << 30, False) > 0
    for bad in ((0, 8, 2, 1, 128, 64, 0), (1, 7, 2, 1, 128, 64, 0), (1, 8, 0, 1, 128, 64, 0),
                (1, 8, 2, 17, 128, 64, 0), (1, 8, 2, 1, 96, 64, 0), (1, 8, 2, 1, 64, 0, 0)):
        assert q(*bad) == 0, bad


def _evict(lib, p=(16,) * 8 + (32,) * 3, B=1, Hkv=2, page=16, sb=8, mp=4, nmp=2, np=9, d=64, keep=20, recent=4):
    return lib.fa_cache_evict_fp8(*map(vp, p), B, Hkv, page, sb, mp, nmp, np, d, keep, recent, None)


@pytest.mark.parametrize("bad,status", CACHE_BAD + [
    (dict(keep=0), fa.FA_ERR_INVALID_ARG), (dict(keep=33), fa.FA_ERR_INVALID_ARG), (dict(recent=-1), fa.FA_ERR_INVALID_ARG),
    (dict(recent=21), fa.FA_ERR_INVALID_ARG), (dict(nmp=0), fa.FA_ERR_INVALID_ARG),
    (dict(nmp=1 << 27), fa.FA_ERR_UNSUPPORTED),
    (dict(p=(16,) * 9 + (32,) * 2), fa.FA_ERR_INVALID_ARG), (dict(p=(16,) * 8 + (32,) + (16,) + (32,)), fa.FA_ERR_INVALID_ARG),
])
def test_evict_refusals(lib, bad, status):
    assert _evict(lib, **bad) == status


def test_evict_pointer_checks(lib):
    for i in range(11):
        p = [16] * 11
        p[i] = 0
        assert _evict(lib, p=p) == fa.FA_ERR_INVALID_ARG, i
        p[i] = 18
        assert _evict(lib, p=p) == fa.FA_ERR_ALIGNMENT, i


def test_conveniences_refuse_other_tensors():
    """CPU tensors, other types and shapes raise ValueError before anything is called."""
    bf, i32 = torch.bfloat16, torch.int32
    x = torch.zeros(1, 2, 4, 64, dtype=bf)
    with pytest.raises(ValueError):
        fa.rope(x, torch.zeros(32, dtype=torch.int64))
    kp, ks = torch.zeros(3, 2, 16, 64, dtype=torch.uint8), torch.zeros(3, 2, 2)
    table, lens = torch.zeros(1, 2, dtype=i32), torch.zeros(1, dtype=i32)
    for call in (lambda: fa.cache_append_fp8(x, x, kp, kp, ks, ks, table, lens),
                 lambda: fa.decode_paged_fp8(torch.zeros(1, 2, 64, dtype=bf), kp, kp, ks, ks, table, lens),
                 lambda: fa.cache_evict_fp8(kp, kp, ks, ks, table, lens, torch.zeros(1, 2, 32), table, 8)):
        with pytest.raises(ValueError):
            call()
