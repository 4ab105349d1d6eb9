"""fa_decode_paged_fp8 where one token takes almost all the weight and a long flat tail has all the value."""
import math

import numpy as np
import pytest
import torch

from oracle import cache as oc
from tests.cache_fp8_common import DEV, args, f64, ints, to_gpu

pytestmark = pytest.mark.gpu


def _check_tail(o, ref):
    """A weight of the value product is rounded to fp16 relative to a reference that puts the largest one of its warp
    at 2^11 or above: half a step is 2^-11 of a normal weight and 2^-25 of a subnormal one, so 2^-36 of the largest
    p vs.  Scores and sums as in check_decode: rel = 2^-17 A + 2^-21, sums 2^-18.  The result's own rounding 2^-8."""
    o_ref, _, A, PV, T = ref
    rel = 2.0 ** -17 * A + 2.0 ** -21
    bound = 2.0 ** -8 * np.abs(o_ref) + (2.0 ** -11 + rel[..., None] + 2.0 ** -18) * PV + 2.0 ** -36 * T
    over = np.abs(f64(o) - o_ref) / bound
    assert over.max() <= 1, "%g times its bound at %s, off by %g of itself" % (
        over.max(), np.unravel_index(over.argmax(), over.shape), (np.abs(f64(o) - o_ref) / np.abs(o_ref)).max())


@pytest.mark.parametrize("spread", [0.0, 0.3])
@pytest.mark.parametrize("gap", [16.0, 20.4, 22.0, 23.6, 24.6, 25.2])
@pytest.mark.parametrize("rows,d", [(1, 128), (4, 64), (16, 128), (32, 64)])
def test_decode_flat_tail_behind_a_sink(cuda_lib, rows, d, gap, spread):
    """The first key is `gap` octaves above the others and has no value; the others' values have one sign, so that
    errors of their weights add up instead of cancelling.  More sequences (all of the same pages) than CTAs: each has
    one CTA for all of its keys, and the warp that holds the first key holds a quarter or half of the others."""
    n, page, sb, B = 65536 + 77, 64, 64, 640
    maxp = -(-n // page)
    rng = np.random.default_rng(int(gap * 10) + rows)
    c = {m: np.zeros((maxp, 1, page, d), dtype=np.uint8) for m in ("k", "v")}
    c |= {m: np.full((maxp, 1, 1), 2.0 ** -8) for m in ("ks", "vs")}
    c["v"][:] = oc.to_e4m3(rng.uniform(100, 440, c["v"].shape))
    c["v"][0, 0, 0] = 0
    table = np.arange(maxp, dtype=np.int32)[None]
    # q = 1 in every column: a key's score in octaves is its sum / sqrt(d) log2(e); the sink's column 0 holds 448 times a
    # scale of its own block, the tail's column 1 a few steps of `spread`
    q = torch.ones((1, rows, 1, d), dtype=torch.bfloat16)
    octave = math.log2(math.e) / math.sqrt(d)
    first = np.zeros((page, d))
    first[0, 0] = gap / octave
    c["ks"][0] = np.float32(gap / octave / 448)
    c["k"][0, 0] = oc.to_e4m3(first / c["ks"][0, 0, 0])
    if spread:
        tail = np.zeros((maxp - 1, 1, page, d))
        tail[..., 1] = rng.standard_normal((maxp - 1, 1, page)) * spread / octave
        c["ks"][1:] = 2.0 ** -7
        c["k"][1:] = oc.to_e4m3(tail * 2.0 ** 7)
    o, lse = cuda_lib.decode_paged_fp8(q.expand(B, -1, -1, -1).contiguous().to(DEV), *args(to_gpu(c)),
                                       ints(np.repeat(table, B, 0)), ints([n] * B))
    assert cuda_lib.fa_get_last_device_error()[0] == 0
    _check_tail(o, oc.decode(f64(q)[:, :1], c, table, [n], 1 / math.sqrt(d)))   # all sequences and rows are alike
