"""The long-context operators of the bf16 cache: what the host checks, before any CUDA call, and their workspaces."""
import ctypes
import math

import pytest
import torch

import exact_tiled_attention_21_gb300 as fa

vp = ctypes.c_void_p
NAN = float("nan")
BAD, UNS, ALI, WSP = fa.FA_ERR_INVALID_ARG, fa.FA_ERR_UNSUPPORTED, fa.FA_ERR_ALIGNMENT, fa.FA_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    fa.build()
    return fa.load()


def _append(lib, k=16, v=16, ks=(0, 0, 64), vs=(0, 0, 64), kp=16, vpg=16, bounds=16, table=16, lens=16, new=0, pos=0,
            turns=16, B=1, Hkv=1, N=4, d=64, rot=64, inter=0, mag=1.0, page=16, block=16, maxp=4, pages=4):
    return lib.fa_cache_append(vp(k), vp(v), *ks, *vs, vp(kp), vp(vpg), vp(bounds), vp(table), vp(lens), vp(new), vp(pos),
                               vp(turns), B, Hkv, N, d, rot, inter, mag, page, block, maxp, pages, None)


@pytest.mark.parametrize("bad,status", [
    (dict(k=0), BAD), (dict(v=0), BAD), (dict(kp=0), BAD), (dict(vpg=0), BAD), (dict(table=0), BAD), (dict(lens=0), BAD),
    (dict(B=0), BAD), (dict(Hkv=0), BAD), (dict(N=0), BAD), (dict(page=0), BAD), (dict(maxp=0), BAD), (dict(pages=0), BAD),
    (dict(block=0), BAD), (dict(block=3), BAD), (dict(block=32), BAD), (dict(page=256, block=256), UNS), (dict(d=96), UNS),
    (dict(rot=24), UNS), (dict(rot=128), BAD), (dict(inter=2), BAD), (dict(mag=NAN), BAD), (dict(mag=math.inf), BAD),
    (dict(k=24), ALI), (dict(v=8), ALI), (dict(kp=8), ALI), (dict(vpg=8), ALI), (dict(bounds=8), ALI), (dict(turns=8), ALI),
    (dict(table=2), ALI), (dict(lens=2), ALI), (dict(new=2), ALI), (dict(pos=2), ALI), (dict(ks=(0, 0, 60)), ALI),
    (dict(vs=(0, 0, -64)), BAD), (dict(N=1 << 30), UNS), (dict(B=1 << 12, Hkv=1 << 13), UNS),
    (dict(maxp=1 << 20, page=2048), UNS), (dict(pages=1 << 28, page=16), UNS),
    (dict(B=1 << 10, Hkv=1 << 10, N=1 << 12, ks=(64, 64, 64), vs=(64, 64, 64)), UNS),
])
def test_append_refusals(lib, bad, status):
    assert _append(lib, **bad) == status


def test_append_ignores_what_it_does_not_use(lib):
    """Without bounds the block, without turns the rotation's arguments: an alignment error behind them shows that they pass."""
    assert _append(lib, bounds=0, block=7, table=2) == ALI
    assert _append(lib, turns=0, rot=3, inter=9, mag=NAN, table=2) == ALI


def _select(lib, q=16, bounds=16, table=16, lens=16, out=16, B=1, Hq=4, Hkv=2, Nq=1, block=16, per=4, maxp=4, pages=8, d=64,
            keep=4, first=1, recent=1, ws=16, nbytes=1 << 30):
    return lib.fa_select_blocks(vp(q), vp(bounds), vp(table), vp(lens), vp(out), B, Hq, Hkv, Nq, block, per, maxp, pages, d,
                                keep, first, recent, vp(ws), nbytes, None)


@pytest.mark.parametrize("bad,status", [
    (dict(q=0), BAD), (dict(bounds=0), BAD), (dict(table=0), BAD), (dict(lens=0), BAD), (dict(out=0), BAD), (dict(B=0), BAD),
    (dict(Hq=0), BAD), (dict(Hq=3), BAD), (dict(Hkv=0), BAD), (dict(Nq=0), BAD), (dict(Nq=17), UNS), (dict(block=0), BAD),
    (dict(block=129), UNS), (dict(per=0), BAD), (dict(per=1 << 28), UNS), (dict(maxp=0), BAD), (dict(pages=0), BAD),
    (dict(d=32), UNS), (dict(keep=0, first=0, recent=0), BAD), (dict(first=-1), BAD), (dict(recent=-1), BAD),
    (dict(first=3, recent=2), BAD), (dict(first=2 ** 31 - 1, recent=2 ** 31 - 1), BAD), (dict(q=8), ALI), (dict(bounds=8), ALI),
    (dict(table=2), ALI), (dict(lens=2), ALI), (dict(out=2), ALI), (dict(maxp=1 << 26), UNS), (dict(B=1 << 23), UNS),
])
def test_select_refusals(lib, bad, status):
    assert _select(lib, **bad) == status


def _blocks(lib, q=16, kp=16, vpg=16, table=16, lens=16, blocks=16, o=32, lse=0, B=1, Hq=4, Hkv=2, Nq=1, page=32, block=16,
            keep=4, maxp=4, pages=8, d=64, scale=0.1, ws=16, nbytes=1 << 40):
    return lib.fa_decode_blocks(vp(q), vp(kp), vp(vpg), vp(table), vp(lens), vp(blocks), vp(o), vp(lse), B, Hq, Hkv, Nq, page,
                                block, keep, maxp, pages, d, scale, vp(ws), nbytes, None)


def _shared(lib, q=16, kp=16, vpg=16, table=16, lens=16, shared=16, o=32, lse=0, B=1, Hq=4, Hkv=2, Nq=1, page=32, maxp=4,
            pages=8, d=64, scale=0.1, ws=16, nbytes=1 << 40):
    return lib.fa_decode_shared(vp(q), vp(kp), vp(vpg), vp(table), vp(lens), vp(shared), vp(o), vp(lse), B, Hq, Hkv, Nq, page,
                                maxp, pages, d, scale, vp(ws), nbytes, None)


COMMON = [
    (dict(q=0), BAD), (dict(kp=0), BAD), (dict(vpg=0), BAD), (dict(table=0), BAD), (dict(lens=0), BAD), (dict(o=0), BAD),
    (dict(B=0), BAD), (dict(Hq=0), BAD), (dict(Hq=5), BAD), (dict(Hkv=0), BAD), (dict(Nq=0), BAD), (dict(Nq=17), UNS),
    (dict(page=0), BAD), (dict(maxp=0), BAD), (dict(pages=0), BAD), (dict(d=256), UNS), (dict(scale=0.0), BAD),
    (dict(scale=NAN), BAD), (dict(scale=math.inf), BAD), (dict(scale=-1.0), BAD), (dict(q=8), ALI), (dict(kp=8), ALI),
    (dict(vpg=8), ALI), (dict(o=40), ALI), (dict(table=2), ALI), (dict(lens=2), ALI), (dict(lse=2), ALI), (dict(o=16), BAD),
    (dict(maxp=1 << 26), UNS), (dict(B=1 << 23), UNS), (dict(pages=1 << 27, page=32), UNS),
    (dict(B=1 << 12, maxp=1 << 20, pages=64), UNS),
]


@pytest.mark.parametrize("bad,status", COMMON + [
    (dict(blocks=0), BAD), (dict(keep=0), BAD), (dict(block=0), BAD), (dict(block=12), BAD), (dict(page=256, block=256), UNS)])
def test_blocks_refusals(lib, bad, status):
    assert _blocks(lib, **bad) == status


@pytest.mark.parametrize("bad,status", COMMON + [(dict(shared=0), BAD), (dict(page=20), UNS), (dict(page=4), UNS),
                                                  (dict(shared=18), ALI)])
def test_shared_refusals(lib, bad, status):
    assert _shared(lib, **bad) == status


@pytest.mark.parametrize("call,G,Nq,Hkv,few,tile", [
    (_blocks, 4, 2, 64, 0, 8), (_blocks, 4, 4, 64, 0, 16), (_blocks, 17, 1, 64, 0, 32), (_blocks, 8, 16, 16, 0, 32),
    (_blocks, 1, 1, 1 << 14, 0, 8),
    (_shared, 4, 2, 64, 0, 8), (_shared, 4, 4, 64, 0, 8), (_shared, 17, 1, 64, 0, 32), (_shared, 8, 16, 16, 0, 32),
    (_shared, 17, 1, 8, 16, 8), (_shared, 17, 1, 8, 17, 32),
])
def test_most_steps(lib, call, G, Nq, Hkv, few, tile):
    """(B + 4) Hkv tiles (steps + 2) < 2^31, at the largest B (few: at this one, by the largest table) that the rule takes and at the
    next.  An alignment error, which is looked for later, shows that a call passes it."""
    tiles, block = -(-G * Nq // tile), 16 if call is _blocks else 1
    most = lambda B, tokens: (B + 4) * Hkv * tiles * (-(-(tokens + block) // 64) + 2) < 1 << 31
    tokens = 1 << 18
    if few:
        steps = ((1 << 31) - 1) // ((few + 4) * Hkv * tiles) - 2
        tokens = min(steps * 64 - block, 1 << 30) // 32 * 32
        pairs = [(few, tokens)] + ([(few, tokens + 64)] if tokens + 64 <= 1 << 30 else [])
    else:
        B = ((1 << 31) - 1) // (Hkv * tiles * (-(-(tokens + block) // 64) + 2)) - 4
        pairs = [(B, tokens), (B + 1, tokens)]
    for B, tokens in pairs:
        got = call(lib, B=B, Hq=G * Hkv, Hkv=Hkv, Nq=Nq, maxp=tokens // 32, pages=8, table=2)
        assert got == (ALI if most(B, tokens) else UNS), (B, tokens)


def test_workspaces():
    """Sizes for what the calls take, none for what they refuse; large enough for the partial results of every CTA."""
    f = fa.fa_select_blocks_workspace_bytes
    assert f(2, 3, 100) >= 2 * 3 * 100 * 12 and f(0, 1, 1) == f(1, 0, 1) == f(1, 1, 0) == f(1, 1, (1 << 30) + 1) == 0
    for g in (fa.fa_decode_blocks_workspace_bytes, fa.fa_decode_shared_workspace_bytes):
        assert g(4, 32, 8, 1, 128) >= 304 * 8 * 129 * 4
        for bad in ((0, 4, 2, 1, 64), (1, 0, 2, 1, 64), (1, 3, 2, 1, 64), (1, 4, 0, 1, 64), (1, 4, 2, 0, 64), (1, 4, 2, 17, 64),
                    (1, 4, 2, 1, 96), (1 << 23, 4, 2, 1, 64)):
            assert g(*bad) == 0, bad
    assert fa.fa_decode_shared_workspace_bytes(64, 32, 8, 2, 128) >= 152 * 256 * 129 * 4


def test_conveniences_refuse_tensors():
    """What the binding checks needs no GPU where it looks at types and devices first."""
    x = torch.zeros((1, 2, 16, 64), dtype=torch.bfloat16)
    i = torch.zeros((1, 1), dtype=torch.int32)
    n = torch.zeros((1,), dtype=torch.int32)
    bounds = torch.zeros((1, 2, 1, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        fa.cache_append(x, x, x, x, i, n)
    with pytest.raises(ValueError, match="CUDA"):
        fa.select_blocks(x, bounds, i, n, block=16, keep=1)
    with pytest.raises(ValueError, match="CUDA"):
        fa.decode_blocks(x, x, x, i, n, torch.zeros((1, 2, 1), dtype=torch.int32), block=16)
    with pytest.raises(ValueError, match="CUDA"):
        fa.decode_shared(x, x, x, i, n, n)
    with pytest.raises(TypeError):
        fa.decode_shared(None, None, x, i, n, n)
