"""fa_decode_paged_fp8 with accumulated weights over tables and batches of many sizes."""
import numpy as np
import pytest
import torch

from oracle import cache as oc
from tests.cache_fp8_common import DEV, args, bf16, check_decode, f64, ints, random_cache, table_of, to_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Hq,Nq", [(8, 1), (10, 3), (32, 2)])
def test_decode_wide_table_with_weights(cuda_lib, Hq, Nq):
    """Weights over a table of far more pages than the sequences use: the bits of a narrow one, and nothing behind the
    sequences changes."""
    lens, Hkv, page = [300, 0, 129], 2, 16
    maxp = -(-max(lens) // page)
    c = random_cache(7, 3 * maxp, Hkv, page, 8, 128)
    table = table_of(8, 3, maxp, 3 * maxp)
    q = bf16(np.random.default_rng(9), (3, Hq, Nq, 128), 0.3).to(DEV)
    wide = np.full((3, 5000), -7, dtype=np.int32)
    wide[:, :maxp] = table
    g, got = to_gpu(c), []
    for tab in (table, wide):
        w = torch.full((3, Hkv, tab.shape[1] * page), 0.5, device=DEV)
        got.append(cuda_lib.decode_paged_fp8(q, *args(g), ints(tab), ints(lens), weights=w) + (w,))
    assert cuda_lib.fa_get_last_device_error()[0] == 0
    narrow, broad = got
    assert torch.equal(narrow[0], broad[0]) and torch.equal(narrow[1], broad[1])
    assert torch.equal(narrow[2], broad[2][..., :maxp * page]) and (broad[2][..., maxp * page:] == 0.5).all()


@pytest.mark.parametrize("Hq,Nq", [(4, 1), (8, 3)])
def test_decode_batch_of_hundreds(cuda_lib, Hq, Nq):
    """700 sequences, more than one scan of lengths holds and more than there are CTAs, a third of them empty."""
    B, Hkv, page, d = 700, 2, 16, 64
    rng = np.random.default_rng(3)
    lens = np.where(rng.random(B) < 0.33, 0, rng.integers(1, 90, B)).astype(np.int32)
    maxp = 6
    c = random_cache(5, 40, Hkv, page, 8, d)
    table = rng.integers(0, 40, (B, maxp)).astype(np.int32)          # pages are shared: they are only read
    q = bf16(rng, (B, Hq, Nq, d), 0.3)
    w, w_ref = torch.zeros((B, Hkv, maxp * page), device=DEV), np.zeros((B, Hkv, maxp * page))
    o, lse = cuda_lib.decode_paged_fp8(q.to(DEV), *args(to_gpu(c)), ints(table), ints(lens), weights=w)
    assert cuda_lib.fa_get_last_device_error()[0] == 0
    check_decode(o, lse, oc.decode(f64(q), c, table, lens, 0.125, w_ref), w, w_ref)
