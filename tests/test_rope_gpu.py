"""fa_rope against float64: layouts, partial and interleaved rotation, far and negative positions, its gradient."""
import numpy as np
import pytest
import torch

import exact_tiled_attention_21_gb300 as fa_mod
from oracle import cache as oc
from tests.cache_fp8_common import DEV, bf16, f64, ints

pytestmark = pytest.mark.gpu


def _check(y, x, pos, freq, inter, mag, inverse, what=""):
    """cos and sin are within 2^-20 (of a unit), products and the sum in fp32 (three roundings of 2^-24, all of at
    most |x1| + |x2|, inside the other half of 2^-19), then one bf16 rounding of at most 2^-8 |y|."""
    ref = oc.rope(f64(x), pos, freq, inter, mag, inverse)
    size, half = np.zeros_like(ref), len(freq)
    a = np.abs(f64(x))
    for i in range(half):
        p, q = (2 * i, 2 * i + 1) if inter else (i, i + half)
        size[..., p] = size[..., q] = (a[..., p] + a[..., q]) * abs(mag)
    err = np.abs(f64(y) - ref) - (2.0 ** -8 * np.abs(ref) + 2.0 ** -19 * size)
    assert err.max() <= 0, "%s: off by %g more than its bound" % (what, err.max())
    assert np.array_equal(f64(y)[..., 2 * half:], f64(x)[..., 2 * half:]), what


def _positions(rng, B, N, far):
    return (rng.integers(-far, far + 1, (B, 1)) + np.arange(N)).astype(np.int32)


@pytest.mark.parametrize("B,H,N,d,rot,inter,far,mag", [
    (1, 1, 1, 64, 16, False, 0, 1.0),
    (1, 1, 1, 128, 128, True, 2 ** 31 - 2, 1.25),
    (2, 3, 37, 128, 128, False, 131072, 1.0),
    (3, 5, 9, 64, 64, True, 1000, 0.5),
    (2, 9, 33, 128, 48, False, 10 ** 6, 1.2079),
    (2, 8, 65, 64, 32, True, 100, 1.0),
    (1, 40, 130, 128, 16, True, 5, -1.0),
    (32, 32, 1, 128, 128, False, 131072, 1.0),
    (1, 13, 1000, 128, 112, False, 4000, 1.0),
])
@pytest.mark.parametrize("inverse", [False, True])
def test_rope_parity(cuda_lib, B, H, N, d, rot, inter, far, mag, inverse):
    rng = np.random.default_rng(B * 1000 + N + rot)
    freq = 10000.0 ** (-2.0 * np.arange(rot // 2) / rot)
    x = bf16(rng, (B, H, N, d)).to(DEV)
    pos = _positions(rng, B, N, min(far, 2 ** 31 - 1 - N))
    table = cuda_lib.rope_table(freq)
    kept = x.clone()
    y = cuda_lib.rope(x, table, ints(pos), inter, mag, inverse)
    assert torch.equal(x, kept) and y.is_contiguous()
    _check(y, x, pos, freq, inter, mag, inverse)
    # other layouts hold the same bits: token-major, and inside a wider projection, in and out
    wide = torch.full((B, N, H + 3, d), 7.0, dtype=torch.bfloat16, device=DEV)
    wide[:, :, 1:1 + H] = x.transpose(1, 2)
    view = wide[:, :, 1:1 + H].transpose(1, 2)
    assert torch.equal(cuda_lib.rope(view, table, ints(pos), inter, mag, inverse), y)
    out = torch.zeros((B, N, H, d), dtype=torch.bfloat16, device=DEV)
    cuda_lib.rope(view, table, ints(pos), inter, mag, inverse, out=out.transpose(1, 2))
    assert torch.equal(out.transpose(1, 2), y)
    # in place, leaving the projection's other columns alone
    cuda_lib.rope(view, table, ints(pos), inter, mag, inverse, out=view)
    assert torch.equal(view, y)
    assert (wide[:, :, :1] == 7).all() and (wide[:, :, 1 + H:] == 7).all()


def test_rope_default_positions_and_broadcast_input(cuda_lib):
    rng = np.random.default_rng(3)
    freq, _ = cuda_lib.rope_frequencies(64, scaling="yarn", factor=8.0, original_context=4096)
    table = cuda_lib.rope_table(freq)
    x = bf16(rng, (1, 1, 50, 64)).to(DEV)
    y = cuda_lib.rope(x, table)
    _check(y, x, np.arange(50)[None], freq, False, 1.0, False)
    many = cuda_lib.rope(x.expand(3, 7, 50, 64), table)   # strides of 0 are read, not written
    assert torch.equal(many, y.expand(3, 7, 50, 64))


def test_rope_gradient_against_differences(cuda_lib):
    """<g, J v> = <J^T g, v> with J v from two rotations (the map is linear), and the oracle's transpose."""
    rng = np.random.default_rng(8)
    for inter in (False, True):
        freq = 10000.0 ** (-2.0 * np.arange(24) / 48)
        table = cuda_lib.rope_table(freq)
        x, v, g = (bf16(rng, (2, 3, 40, 64), 0.0).to(DEV) for _ in range(3))
        pos = _positions(rng, 2, 40, 9000)
        step = x + v
        jv = f64(cuda_lib.rope(step, table, ints(pos), inter, 1.5)) - f64(cuda_lib.rope(x, table, ints(pos), inter, 1.5))
        dx = cuda_lib.rope(g, table, ints(pos), inter, 1.5, inverse=True)
        real = f64(step) - f64(x)
        lhs, rhs = (f64(g) * jv).sum(), (f64(dx) * real).sum()
        # three results rounded to bf16 (2^-8 each of their size), summed with the other factor's magnitudes
        size = 2.0 ** -8 * ((np.abs(f64(g)) * 1.5 * 2 * (np.abs(f64(step)).max() + np.abs(f64(x)).max())).sum()
                            + (np.abs(f64(dx)) * np.abs(real)).sum())
        assert abs(lhs - rhs) <= size
        _check(dx, g, pos, freq, inter, 1.5, True)


def test_rope_large_tensor(cuda_lib):
    """More than 2^32 bytes: offsets stay right at the end."""
    H, N, d = 40, 460000, 128
    x = torch.zeros((1, H, N, d), dtype=torch.bfloat16, device=DEV)
    tail = bf16(np.random.default_rng(1), (1, 2, 100, d)).to(DEV)
    x[:, -2:, -100:] = tail
    freq = 10000.0 ** (-2.0 * np.arange(64) / 128)
    table = cuda_lib.rope_table(freq)
    cuda_lib.rope(x, table, out=x)
    _check(x[:, -2:, -100:], tail, np.arange(N - 100, N)[None], freq, False, 1.0, False)
    assert (x[:, :2, :100] == 0).all()


def test_rope_special_values(cuda_lib):
    """Infinities and NaN stay in their pair."""
    freq = 10000.0 ** (-2.0 * np.arange(8) / 16)
    table = cuda_lib.rope_table(freq)
    x = bf16(np.random.default_rng(2), (1, 1, 3, 64)).to(DEV)
    x[0, 0, 1, 2] = float("nan")
    x[0, 0, 1, 40] = float("inf")
    y = cuda_lib.rope(x, table)
    assert y[0, 0, 1, [2, 10]].isnan().all() and y[0, 0, 1, 40].isinf()
    assert int((~y.isfinite()).sum()) == 3


def test_rope_on_a_side_stream_and_in_a_graph(cuda_lib):
    rng = np.random.default_rng(4)
    table = cuda_lib.rope_table(10000.0 ** (-2.0 * np.arange(32) / 64))
    x = bf16(rng, (2, 4, 300, 64)).to(DEV)
    pos = ints(_positions(rng, 2, 300, 5000))
    want = cuda_lib.rope(x, table, pos)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = [cuda_lib.rope(x, table, pos, stream=s) for _ in range(3)]
    got.append(cuda_lib.rope(x, table, pos, stream=s.cuda_stream))
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(g, want) for g in got)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = cuda_lib.rope(x, table, pos)
    pos += 7
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, cuda_lib.rope(x, table, pos))


def test_rope_refusals(cuda_lib):
    table = cuda_lib.rope_table([1.0] * 32)
    x = torch.zeros((1, 2, 8, 64), dtype=torch.bfloat16, device=DEV)
    for call in (lambda: cuda_lib.rope(x.float(), table), lambda: cuda_lib.rope(x[..., ::2], table),
                 lambda: cuda_lib.rope(x, table.int()), lambda: cuda_lib.rope(x, table, ints([[0] * 7])),
                 lambda: cuda_lib.rope(x, table, out=x[:, :1]), lambda: cuda_lib.rope(x[0], table)):
        with pytest.raises(ValueError):
            call()
    for call, st in ((lambda: cuda_lib.rope(x, table[:12]), fa_mod.FA_ERR_UNSUPPORTED),
                     (lambda: cuda_lib.rope(x, cuda_lib.rope_table([1.0] * 40)), fa_mod.FA_ERR_INVALID_ARG),
                     (lambda: cuda_lib.rope(x[:, :1], table, out=x[:, :1, :1].expand(1, 1, 8, 64)), fa_mod.FA_ERR_INVALID_ARG),
                     (lambda: cuda_lib.rope(torch.zeros((1, 2, 8, 68), dtype=x.dtype, device=DEV)[..., :64], table),
                      fa_mod.FA_ERR_ALIGNMENT)):
        with pytest.raises(fa_mod.FAError) as e:
            call()
        assert e.value.status == st
