"""The long-context operators as a serving program chains them: without a wait of the host, captured and replayed, on other
streams, with wide tables and far pages."""
import math

import numpy as np
import pytest
import torch

from oracle import paged as op
from tests.paged_common import DEV, bf16, check_rows, f64, ints, ok, random_pages, table_of, to_gpu

pytestmark = pytest.mark.gpu
ONE, PAIR = 2.0 ** -8, 2.0 ** -16


@pytest.mark.parametrize("d,Hkv,G,page,block", [(128, 4, 4, 64, 32), (64, 8, 1, 16, 8), (128, 2, 16, 32, 4), (64, 2, 3, 48, 4)])
def test_serving_steps(cuda_lib, d, Hkv, G, page, block):
    """Prompts, then steps of one and three tokens: append with bounds, selection, attention over the selected blocks and over
    everything, each against float64 on what the cache then holds."""
    fa, B, scale = cuda_lib, 4, 1.0 / math.sqrt(d)
    rng = np.random.default_rng(d + G)
    prompts, steps = [300, 1, 77, 160], [1, 3, 1]
    maxp = -(-(max(prompts) + sum(steps)) // page)
    pages = B * maxp + 1
    c = random_pages(5, pages, Hkv, page, d, block)
    table = table_of(6, B, maxp, pages)
    g, tab = to_gpu(c), ints(table)
    turns = fa.rope_table(fa.rope_frequencies(d)[0])
    lens = np.zeros(B, dtype=np.int32)
    for N, new in [(max(prompts), prompts)] + [(n, None) for n in steps]:
        k, v = bf16(rng, (B, Hkv, N, d), 0.3).to(DEV), bf16(rng, (B, Hkv, N, d), 0.3).to(DEV)
        fa.cache_append(k, v, g["k"], g["v"], tab, ints(lens), None if new is None else ints(new), turns=turns, bounds=g["b"])
        pos = (ints(lens)[:, None] + torch.arange(N, device=DEV)).int().contiguous()
        op.append(c, table, lens, f64(fa.rope(k, turns, pos)), f64(v), new)
        lens = lens + (N if new is None else np.array(new, dtype=np.int32))
        Nq = 1 if new is not None else N
        q = fa.rope(bf16(rng, (B, Hkv * G, Nq, d), 0.3).to(DEV), turns, (ints(lens)[:, None] - Nq + torch.arange(Nq, device=DEV)).int().contiguous())
        keep = 6
        lists = fa.select_blocks(q, g["b"], tab, ints(lens), block=block, keep=keep, first=1, recent=2)
        want = op.select(f64(q), c["b"], table, lens, block, keep, 1, 2)
        assert np.array_equal(lists.cpu().numpy(), want)
        o, lse = fa.decode_blocks(q, g["k"], g["v"], tab, ints(lens), lists, block=block)
        check_rows(o, lse, op.attend(f64(q), c, table, lens, scale, op.tokens_of(want, block)), PAIR)
        o, lse = fa.decode_shared(q, g["k"], g["v"], tab, ints(lens), ints([0]))
        check_rows(o, lse, op.attend(f64(q), c, table, lens, scale), PAIR)
    ok(fa)


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("d,Hkv,G,B,shared", [(128, 4, 4, 5, 320), (64, 2, 8, 40, 1000), (128, 8, 4, 32, 700)])
def test_chain_without_waits_is_the_chain_with_them(cuda_lib, d, Hkv, G, B, shared, captured):
    """Append, selection, both attentions, over and over: bit for bit those of the same calls with the device idle in between,
    also captured and replayed, and on a side stream.  (40 x 8 rows go through the matrix kernel of the prefix.)"""
    fa, page, block, steps = cuda_lib, 32, 16, 5
    rng = np.random.default_rng(d + B)
    full = shared // page
    lens0 = shared + rng.integers(0, 60, B).astype(np.int32)
    own = 4
    c = random_pages(3, full + B * own, Hkv, page, d, block)
    p = rng.permutation(full + B * own).astype(np.int32)
    table = np.ascontiguousarray(np.concatenate([np.tile(p[:full], (B, 1)), p[full:].reshape(B, own)], 1))
    tab, n_shared = ints(table), ints([full * page])
    turns = fa.rope_table(fa.rope_frequencies(d)[0])
    kv = [[bf16(rng, (B, Hkv, 2, d), 0.3).to(DEV) for _ in range(2)] for _ in range(steps)]
    qs = [bf16(rng, (B, Hkv * G, 2, d), 0.3).to(DEV) for _ in range(steps)]

    def program(g, lens, wait):
        out = []
        for i in range(steps):
            fa.cache_append(kv[i][0], kv[i][1], g["k"], g["v"], tab, lens, turns=turns, bounds=g["b"])
            wait()
            lens = lens + 2
            wait()
            lists = fa.select_blocks(qs[i], g["b"], tab, lens, block=block, keep=9, first=1, recent=2)
            wait()
            out += [lists, *fa.decode_blocks(qs[i], g["k"], g["v"], tab, lens, lists, block=block)]
            wait()
            out += fa.decode_shared(qs[i], g["k"], g["v"], tab, lens, n_shared)
            wait()
        return out + [g["k"], g["v"], g["b"]]

    want = program(to_gpu(c), ints(lens0), torch.cuda.synchronize)
    g, lens = to_gpu(c), ints(lens0)
    start = {n: g[n].clone() for n in g}
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = program(g, lens, lambda: None)
    for turn in range(4):
        for n in g:
            g[n].copy_(start[n])
        torch.cuda.synchronize()
        if captured:
            graph.replay()
        elif turn % 2:
            with torch.cuda.stream(side):
                got = program(g, lens, lambda: None)
        else:
            got = program(g, lens, lambda: None)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    ok(fa)


def test_streams_given_to_the_calls(cuda_lib):
    """stream= puts a call, and what it allocates, on that stream; another device's is refused by the framework's check."""
    fa, Hkv, d, page, block = cuda_lib, 2, 64, 16, 16
    rng = np.random.default_rng(0)
    c = random_pages(1, 8, Hkv, page, d, block)
    table, lens = table_of(2, 2, 4, 8), [50, 20]
    q, kn = bf16(rng, (2, 4, 1, d), 0.3).to(DEV), bf16(rng, (2, Hkv, 3, d), 0.3).to(DEV)
    a, b = to_gpu(c), to_gpu(c)
    s = torch.cuda.Stream()

    def calls(g, stream):
        fa.cache_append(kn, kn, g["k"], g["v"], ints(table), ints(lens), bounds=g["b"], stream=stream)
        n = ints(np.array(lens) + 3)
        lists = fa.select_blocks(q, g["b"], ints(table), n, block=block, keep=2, stream=stream)
        return [lists, *fa.decode_blocks(q, g["k"], g["v"], ints(table), n, lists, block=block, stream=stream),
                *fa.decode_shared(q, g["k"], g["v"], ints(table), n, ints([16]), stream=stream)]
    want = calls(a, None)
    torch.cuda.synchronize()
    for stream in (s, s.cuda_stream, 0):
        b = to_gpu(c)
        torch.cuda.synchronize()
        got = calls(b, stream)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got + [b["k"], b["v"], b["b"]], want + [a["k"], a["v"], a["b"]]))


def test_workspaces_given_to_the_calls(cuda_lib):
    """A workspace of the stated size is enough and whatever it holds; a smaller or unaligned one is refused."""
    fa, Hkv, G, d, page, block, B = cuda_lib, 2, 4, 128, 16, 8, 20
    rng = np.random.default_rng(3)
    c = random_pages(4, B * 5, Hkv, page, d, block)
    table, lens = table_of(5, B, 5, B * 5), rng.integers(1, 80, B)
    g, q = to_gpu(c), bf16(rng, (B, Hkv * G, 1, d), 0.3).to(DEV)
    table[:, :2] = table[0, :2]
    tab, n = ints(table), ints(lens)
    calls = [(fa.fa_select_blocks_workspace_bytes(B, Hkv, 5 * page // block),
              lambda w: [fa.select_blocks(q, g["b"], tab, n, block=block, keep=4, workspace=w)]),
             (fa.fa_decode_blocks_workspace_bytes(B, Hkv * G, Hkv, 1, d),
              lambda w: fa.decode_blocks(q, g["k"], g["v"], tab, n, ints(np.tile(np.arange(10), (B, Hkv, 1))), block=block, workspace=w)),
             (fa.fa_decode_shared_workspace_bytes(B, Hkv * G, Hkv, 1, d),
              lambda w: fa.decode_shared(q, g["k"], g["v"], tab, n, ints([20]), workspace=w))]
    for size, f in calls:
        want = f(None)
        for fill in (0, 255):
            w = torch.full((size,), fill, dtype=torch.uint8, device=DEV)
            assert all(torch.equal(a, b) for a, b in zip(f(w), want))
        with pytest.raises(fa.FAError) as err:
            f(torch.empty(size - 1 - size % 16, dtype=torch.uint8, device=DEV)[:max(1, size // 4)])
        assert err.value.status == fa.FA_ERR_WORKSPACE
        with pytest.raises(fa.FAError) as err:
            f(torch.empty(size + 32, dtype=torch.uint8, device=DEV)[4:])
        assert err.value.status == fa.FA_ERR_ALIGNMENT
    ok(fa)


def test_wide_tables(cuda_lib):
    """Tables far wider than the sequences: the prefix goes through its matrix kernel at any number of rows, the selection's
    scores through the workspace."""
    fa, Hkv, G, d, page, block = cuda_lib, 8, 4, 128, 64, 4
    rng = np.random.default_rng(8)
    for B, shared in ((32, 1000), (12, 129), (33, 640)):
        full, wide = shared // page, 2051
        lens = shared + rng.integers(1, 100, B)
        lens[3] = 0
        own = -(-(shared + 100) // page) - full
        c = random_pages(9, full + B * own, Hkv, page, d)
        p = rng.permutation(full + B * own).astype(np.int32)
        table = np.full((B, wide), -1, dtype=np.int32)
        table[:, :full] = p[:full]
        table[:, full:full + own] = p[full:].reshape(B, own)
        if shared % page:
            for n in c:
                c[n][table[:, full], :, :shared % page] = c[n][table[0, full], :, :shared % page]
        g, q = to_gpu(c), bf16(rng, (B, Hkv * G, 1, d), 0.3)
        o, lse = fa.decode_shared(q.to(DEV), g["k"], g["v"], ints(table), ints(lens), ints([shared]))
        ok(fa)
        check_rows(o, lse, op.attend(f64(q), c, table, lens, 1 / math.sqrt(d)), ONE)
    # 32816 blocks of the table, an odd number of them; 300 query rows, several tiles of them
    lens = [4000, 77, 0]
    for G, Nq, wide in ((4, 1, 2051), (75, 4, 63)):
        c = random_pages(10, 3 * 63, 1, page, d, block)
        table = np.full((3, wide), -1, dtype=np.int32)
        table[:, :63] = rng.permutation(3 * 63).reshape(3, 63)
        q, bounds = bf16(rng, (3, G, Nq, d), 0.3), to_gpu(c)["b"]
        got = fa.select_blocks(q.to(DEV), bounds, ints(table), ints(lens), block=block, keep=33, first=1, recent=1)
        ok(fa)
        assert np.array_equal(got.cpu().numpy(), op.select(f64(q), c["b"], table, lens, block, 33, 1, 1))


def test_far_pages(cuda_lib):
    """Pages beyond 2^32 bytes and 2^31 elements."""
    fa, Hkv, d, page, block = cuda_lib, 8, 128, 256, 32
    pages = (1 << 31) // (Hkv * d * page) + 6
    kp = torch.zeros((pages, Hkv, page, d), dtype=torch.bfloat16, device=DEV)
    vp = torch.zeros_like(kp)
    bounds = torch.zeros((pages, Hkv, page // block, 2, d), dtype=torch.bfloat16, device=DEV)
    rng = np.random.default_rng(4)
    n = [700, 650]
    far = np.array([[pages - 1, pages - 3, pages - 5], [pages - 1, pages - 3, pages - 2]], dtype=np.int32)
    k, v = (bf16(rng, (2, Hkv, 700, d), 0.3).to(DEV) for _ in "kv")
    k[1, :, :512], v[1, :, :512] = k[0, :, :512], v[0, :, :512]
    fa.cache_append(k[:1], v[:1], kp, vp, ints(far[:1]), ints([0]), bounds=bounds)
    fa.cache_append(k[1:, :, 512:], v[1:, :, 512:], kp, vp, ints(far[1:]), ints([512]), ints([138]), bounds=bounds)
    small = {"k": f64(kp[-6:]), "v": f64(vp[-6:]), "b": f64(bounds[-6:])}
    near = far - (pages - 6)
    q = bf16(rng, (2, Hkv * 4, 1, d), 0.3)
    lists = fa.select_blocks(q.to(DEV), bounds, ints(far), ints(n), block=block, keep=7, recent=2)
    want = op.select(f64(q), small["b"], near, n, block, 7, 0, 2)
    assert np.array_equal(lists.cpu().numpy(), want)
    o, lse = fa.decode_blocks(q.to(DEV), kp, vp, ints(far), ints(n), lists, block=block)
    check_rows(o, lse, op.attend(f64(q), small, near, n, 1 / math.sqrt(d), op.tokens_of(want, block)), PAIR)
    o, lse = fa.decode_shared(q.to(DEV), kp, vp, ints(far), ints(n), ints([512]))
    check_rows(o, lse, op.attend(f64(q), small, near, n, 1 / math.sqrt(d)), ONE)
    many = torch.cat([q] * 20)                             # 160 rows: the matrix kernel
    o, lse = fa.decode_shared(many.to(DEV), kp, vp, ints(np.tile(far, (20, 1))), ints(n * 20), ints([512]))
    check_rows(o[:2], lse[:2], op.attend(f64(q), small, near, n, 1 / math.sqrt(d)), ONE)
    check_rows(o[38:], lse[38:], op.attend(f64(q), small, near, n, 1 / math.sqrt(d)), ONE)
    ok(fa)


def test_append_raises_version_counters(cuda_lib):
    fa, Hkv, d, page = cuda_lib, 1, 64, 16
    g = to_gpu(random_pages(1, 2, Hkv, page, d, 8))
    k = torch.zeros((1, Hkv, 1, d), dtype=torch.bfloat16, device=DEV)
    before = {n: g[n]._version for n in g}
    fa.cache_append(k, k, g["k"], g["v"], ints([[0, 1]]), ints([3]))
    assert g["k"]._version > before["k"] and g["v"]._version > before["v"] and g["b"]._version == before["b"]
    fa.cache_append(k, k, g["k"], g["v"], ints([[0, 1]]), ints([3]), bounds=g["b"])
    assert g["b"]._version > before["b"]
    with torch.inference_mode():
        fa.cache_append(k, k, g["k"], g["v"], ints([[0, 1]]), ints([3]), bounds=g["b"])
    ok(fa)


def test_conveniences_refuse(cuda_lib):
    fa, Hkv, d, page = cuda_lib, 2, 64, 16
    g = to_gpu(random_pages(1, 4, Hkv, page, d, 8))
    k = torch.zeros((1, Hkv, 1, d), dtype=torch.bfloat16, device=DEV)
    q = torch.zeros((1, 4, 1, d), dtype=torch.bfloat16, device=DEV)
    tab, n = ints([[0, 1]]), ints([3])
    bad = [
        lambda: fa.cache_append(k.float(), k, g["k"], g["v"], tab, n),
        lambda: fa.cache_append(k[:, :1], k, g["k"], g["v"], tab, n),
        lambda: fa.cache_append(k, k, g["k"], g["v"][:3], tab, n),
        lambda: fa.cache_append(k, k, g["k"], g["v"], tab.long(), n),
        lambda: fa.cache_append(k, k, g["k"], g["v"], tab, n, bounds=g["b"].float()),
        lambda: fa.cache_append(k, k, g["k"], g["v"], tab, n, bounds=g["b"][:, :, :, :1]),
        lambda: fa.cache_append(k, k, g["k"], g["v"], tab, n, new_lens=ints([1, 1])),
        lambda: fa.select_blocks(q, g["b"][0], tab, n, block=8, keep=2),
        lambda: fa.select_blocks(q[..., :32], g["b"], tab, n, block=8, keep=2),
        lambda: fa.select_blocks(q.transpose(1, 2), g["b"], tab, ints([3, 3]), block=8, keep=2),
        lambda: fa.decode_blocks(q, g["k"], g["v"], tab, n, ints([[[0]]]), block=8),
        lambda: fa.decode_blocks(q, g["k"], g["v"], tab, n, torch.zeros((1, Hkv, 2), device=DEV), block=8),
        lambda: fa.decode_shared(q, g["k"], g["v"], tab, n, ints([1, 2])),
        lambda: fa.decode_shared(q, g["k"], g["v"], tab, n, torch.zeros((1,), dtype=torch.int32)),
        lambda: fa.decode_shared(q, g["k"].transpose(1, 2), g["v"], tab, n, ints([1])),
    ]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    for f, status in [(lambda: fa.select_blocks(q, g["b"], tab, n, block=8, keep=0), fa.FA_ERR_INVALID_ARG),
                      (lambda: fa.select_blocks(q, g["b"], tab, n, block=8, keep=2, first=2, recent=1), fa.FA_ERR_INVALID_ARG),
                      (lambda: fa.decode_blocks(q, g["k"], g["v"], tab, n, ints([[[0], [0]]]), block=7), fa.FA_ERR_INVALID_ARG),
                      (lambda: fa.decode_blocks(q, g["k"], g["v"], tab, n, ints([[[0], [0]]]), block=8, scale=0.0), fa.FA_ERR_INVALID_ARG)]:
        with pytest.raises(fa.FAError) as err:
            f()
        assert err.value.status == status
    ok(fa)


def test_selection_refuses_before_it_takes_memory(cuda_lib):
    """Lists of 2^31 - 1 blocks for 64 kv heads would be half a terabyte; a long list that is all right is filled with -1."""
    fa, Hkv, d = cuda_lib, 64, 64
    bounds = torch.zeros((2, Hkv, 2, 2, d), dtype=torch.bfloat16, device=DEV)
    q = torch.zeros((1, Hkv, 17, d), dtype=torch.bfloat16, device=DEV)
    tab, n, most = ints([[1, 0]]), ints([20]), 2 ** 31 - 1
    for f, status in [(lambda: fa.select_blocks(q[:, :, 0].contiguous(), bounds, tab, n, block=8, keep=most, first=-1), fa.FA_ERR_INVALID_ARG),
                      (lambda: fa.select_blocks(q[:, :, 0].contiguous(), bounds, tab, n, block=0, keep=most), fa.FA_ERR_INVALID_ARG),
                      (lambda: fa.select_blocks(q, bounds, tab, n, block=8, keep=most), fa.FA_ERR_UNSUPPORTED)]:
        with pytest.raises(fa.FAError) as err:
            f()
        assert err.value.status == status
    got = fa.select_blocks(q[:, :, 0].contiguous(), bounds, tab, n, block=8, keep=100000)
    assert (got[..., :3] == ints([0, 1, 2])).all() and (got[..., 3:] == -1).all()
    ok(fa)
