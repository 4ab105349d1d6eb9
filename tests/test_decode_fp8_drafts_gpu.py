"""fa_decode_paged_fp8 where some of the new tokens hold nothing of use: what a query does not see does not reach it."""
import math

import numpy as np
import pytest
import torch

from oracle import cache as oc
from tests.cache_fp8_common import DEV, args, bf16, check_decode, copy, f64, ints, random_cache, table_of, to_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G,Nq,lens", [
    (1, 2, [2, 1, 50]), (2, 4, [4, 33, 131]), (1, 16, [16, 40, 130]), (4, 4, [100, 3, 257]), (8, 4, [129, 64, 3000]),
    (5, 5, [130, 35, 9]), (3, 16, [140, 15, 1040]), (16, 5, [300, 132, 4]), (2, 16, [5000, 128, 144])])
def test_decode_nan_in_tokens_that_a_query_does_not_see(cuda_lib, G, Nq, lens, d):
    """A draft padded to Nq tokens: the keys and values of its last ones are NaN.  The queries before them get what they
    get with zeros there; those that see one show it, and a NaN in one value in its column only."""
    Hkv, page, sb = 2, 16, 8
    maxp = -(-max(lens) // page)
    B = len(lens)
    c = random_cache(Nq + d, B * maxp, Hkv, page, sb, d)
    table = table_of(4, B, maxp, B * maxp)
    q = bf16(np.random.default_rng(G), (B, Hkv * G, Nq, d), 0.3)
    run = lambda x: cuda_lib.decode_paged_fp8(q.to(DEV), *args(to_gpu(x)), ints(table), ints(lens))
    for first in {1, Nq // 2, Nq - 1} - {0}:                 # the first padded token of the Nq
        zero, nan_v, nan_kv = copy(c), copy(c), copy(c)
        for b, n in enumerate(lens):
            for t in range(max(first, Nq - n), Nq):
                j = n - Nq + t
                at = (table[b, j // page], slice(None), j % page)
                nan_v["v"][at] = nan_kv["v"][at] = nan_kv["k"][at] = 0x7F if t % 2 else 0xFF
                zero["v"][at] = zero["k"][at] = nan_v["k"][at] = 0
        ref = tuple(x[:, :, :first] for x in oc.decode(f64(q), zero, table, lens, 1 / math.sqrt(d)))
        got = [run(x) for x in (zero, nan_v, nan_kv)]
        for o, lse in got:
            check_decode(o[:, :, :first], lse[:, :, :first], ref)
        assert torch.equal(got[1][0][:, :, :first], got[0][0][:, :, :first])
        for o, _ in got[1:]:
            for b, n in enumerate(lens):
                seen = list(range(max(first, Nq - n), Nq))
                assert o[b, :, seen].isnan().all()
    # a NaN in one value of one token: that column of the queries that see it, and nothing else
    for back in {0, 1, Nq - 1}:
        bad, zero = copy(c), copy(c)
        for b, n in enumerate(lens):
            if n > back:
                at = (table[b, (n - 1 - back) // page], 1, (n - 1 - back) % page, 37)
                bad["v"][at], zero["v"][at] = 0x7F, 0
        o, oz = run(bad)[0], run(zero)[0]
        want = torch.zeros_like(o, dtype=torch.bool)
        for b, n in enumerate(lens):
            if n > back:
                want[b, G:, Nq - 1 - back:, 37] = True
        assert torch.equal(o.isnan(), want)
        assert torch.equal(o.masked_fill(want, 0), oz.masked_fill(want, 0))
    assert cuda_lib.fa_get_last_device_error()[0] == 0
