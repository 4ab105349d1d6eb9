"""The serving-cache calls as a program chains them: one behind the other without a wait of the host, on any stream,
with sequences that pause."""
import numpy as np
import pytest
import torch

from oracle import cache as oc
from tests.cache_fp8_common import DEV, args, assert_same_cache, bf16, copy, f64, ints, random_cache, table_of, to_gpu

pytestmark = pytest.mark.gpu


def _ok(fa):
    st, detail = fa.fa_get_last_device_error()
    assert st == 0, detail


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("d,Hkv,G,page,sb", [(128, 4, 4, 64, 32), (64, 8, 1, 16, 8), (128, 2, 16, 32, 32)])
def test_chain_without_waits_is_the_chain_with_them(cuda_lib, d, Hkv, G, page, sb, captured):
    """Append (whose blocks' scales grow), decode with weights and eviction, twice over, then a second round on the
    evicted cache: every output and the whole cache are bit for bit those of the same calls with the device idle in
    between.  Each kernel reads what the one before wrote: scales, lengths, weights."""
    fa, B, steps = cuda_lib, 5, 6
    rng = np.random.default_rng(d + Hkv)
    lens0 = np.array([333, 7, 0, 129, 500], dtype=np.int32)
    maxp, newp = -(-520 // page), -(-200 // page)
    c = random_cache(3, B * (maxp + newp), Hkv, page, sb, d)
    both = table_of(4, B, maxp + newp, B * (maxp + newp))
    tab, new = ints(both[:, :maxp]), ints(both[:, maxp:])
    turns = fa.rope_table(10000.0 ** (-2.0 * np.arange(d // 2) / d))
    kv = [[(bf16(rng, (B, Hkv, 3, d), 0.3) * 1.5 ** i).to(DEV) for _ in range(2)] for i in range(steps)]
    qs = [bf16(rng, (B, Hkv * G, 1, d), 0.3).to(DEV) for _ in range(steps)]

    def program(g, lens, w, wait):
        out, t = [], tab
        for i in range(steps):
            fa.cache_append_fp8(kv[i][0], kv[i][1], *args(g), t, lens, turns=turns)
            wait()
            lens = lens + 3
            wait()
            out += fa.decode_paged_fp8(fa.rope(qs[i], turns, (lens - 1)[:, None].contiguous()), *args(g), t, lens, weights=w)
            wait()
            if i == steps // 2:
                lens, w, kept = fa.cache_evict_fp8(*args(g), t, lens, w, new, 150, 20)
                wait()
                out, t = out + [kept], new
        return out + [lens, w] + list(args(g))

    want = program(to_gpu(c), ints(lens0), torch.zeros((B, Hkv, maxp * page), device=DEV), torch.cuda.synchronize)
    g, lens, w = to_gpu(c), ints(lens0), torch.zeros((B, Hkv, maxp * page), device=DEV)
    start = [t.clone() for t in args(g)]
    if captured:
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            got = program(g, lens, w, lambda: None)
    for _ in range(5):
        for t, s in zip(args(g), start):
            t.copy_(s)
        w.zero_()
        if captured:
            graph.replay()
        else:
            got = program(g, lens, w, lambda: None)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    _ok(fa)


def test_stream_handles(cuda_lib):
    """0 is the default stream, as for the framework's other calls, and any other handle itself."""
    x = torch.zeros((1, 1, 8, 64), dtype=torch.bfloat16, device=DEV)
    s = torch.cuda.Stream()
    for stream, handle in ((0, 0), (s, s.cuda_stream), (s.cuda_stream, s.cuda_stream), (torch.cuda.default_stream(), 0)):
        with cuda_lib._on_stream(stream, x):
            assert torch.cuda.current_stream().cuda_stream == handle
    want = torch.zeros((1, 1, 8, 64), dtype=torch.bfloat16, device=DEV)
    turns = cuda_lib.rope_table([0.5] * 32)
    for i in range(20):                      # ordered behind what the default stream does before it
        x.fill_(i + 1)
        y = cuda_lib.rope(x, turns, positions=ints([[0] * 8]), stream=0)
        assert torch.equal(y, want + (i + 1))


def test_append_leaves_paused_sequences_alone(cuda_lib):
    """A sequence without new tokens is not touched, even in the middle of a block: neither its scale (here a subnormal
    one, which a write would raise) nor its table, whose pages may be gone."""
    Hkv, d, page, sb = 2, 64, 16, 8
    rng = np.random.default_rng(1)
    c = random_cache(2, 6, Hkv, page, sb, d)
    c["ks"][1] = 2.0 ** -140
    table = np.array([[0, 3], [1, -1], [-1, -1]], dtype=np.int32)
    k = bf16(rng, (3, Hkv, 4, d))
    for lens, new in (([5, 3, 20], [4, 0, 0]), ([8, 11, 0], [0, 0, 0])):
        g = to_gpu(c)
        cuda_lib.cache_append_fp8(k.to(DEV), k.to(DEV), *args(g), ints(table), ints(lens), ints(new))
        _ok(cuda_lib)
        ref = copy(c)
        oc.append(ref, table, lens, f64(k), f64(k), new)
        assert_same_cache(g, ref)
