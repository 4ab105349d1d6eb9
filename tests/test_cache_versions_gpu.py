"""The version counters of what the serving-cache calls write in place."""
import numpy as np
import pytest
import torch

from tests.cache_fp8_common import DEV, args, bf16, ints, random_cache, table_of, to_gpu

pytestmark = pytest.mark.gpu


def test_writes_raise_version_counters(cuda_lib):
    """What a call writes in place counts as changed, so that autograd refuses a gradient from the old values."""
    rng = np.random.default_rng(0)
    x, g = bf16(rng, (2, 3, 37, 64)).to(DEV), bf16(rng, (2, 3, 37, 64)).to(DEV)
    table, pos = cuda_lib.rope_table(10000.0 ** (-2.0 * np.arange(16) / 32)), ints(rng.integers(0, 5000, (2, 37)))
    p = torch.ones_like(g).requires_grad_()
    y = (p * x).sum()                        # x is kept for the gradient of p
    cuda_lib.rope(x, table, pos, out=x)
    with pytest.raises(RuntimeError):
        y.backward()
    Hkv, page, d = 2, 16, 64
    pool = to_gpu(random_cache(1, 8, Hkv, page, 8, d))
    tab, new = ints(table_of(2, 1, 3, 6)), ints([[6, 7]])
    w = torch.zeros((1, Hkv, 48), device=DEV)
    k = g[:1, :Hkv, :5].contiguous()
    before = lambda: [t._version for t in args(pool) + (w,)]
    v0 = before()
    cuda_lib.cache_append_fp8(k, k, *args(pool), tab, ints([0]))
    v1 = before()
    assert all(b > a for a, b in zip(v0[:4], v1[:4])) and v1[4] == v0[4]
    q = g[:1, :Hkv, :1].contiguous()
    cuda_lib.decode_paged_fp8(q, *args(pool), tab, ints([5]))
    assert before() == v1
    cuda_lib.decode_paged_fp8(q, *args(pool), tab, ints([5]), weights=w)
    v2 = before()
    assert v2[:4] == v1[:4] and v2[4] > v1[4]
    cuda_lib.cache_evict_fp8(*args(pool), tab, ints([5]), w, new, 3)
    v3 = before()
    assert all(b > a for a, b in zip(v2[:4], v3[:4])) and v3[4] == v2[4]
    with torch.inference_mode():             # tensors without a counter are written as they were
        pool = to_gpu(random_cache(1, 8, Hkv, page, 8, d))
        z = x.detach().clone()
    cuda_lib.cache_append_fp8(k, k, *args(pool), tab, ints([0]))
    cuda_lib.rope(z, table, pos, out=z)
