"""Rescaling a block of another writer's scale (no power of two) at the ends of fp32's range."""
import numpy as np
import pytest
import torch

from oracle import cache as oc
from tests.cache_fp8_common import DEV, args, assert_same_cache, bf16, f64, ints, random_cache, to_gpu

pytestmark = pytest.mark.gpu


def _ok(fa):
    st, detail = fa.fa_get_last_device_error()
    assert st == 0, detail


# Pairs of block scales (no powers of two) whose products with e4m3's 448 overflow fp32, or whose values are so small
# that those products lose bits.
ENDS = [(1.1e36, 1.9e36), (7.7e35, 3.0e38), (np.float32(3 * 2.0 ** -149), np.float32(5 * 2.0 ** -149)),
        (np.float32(1.7e-41), np.float32(2.9e-41))]


@pytest.mark.parametrize("small,large", ENDS)
def test_evict_rescales_at_the_ends_of_the_range(cuda_lib, small, large):
    Hkv, d, page, sb, n = 1, 64, 16, 8, 48
    c = random_cache(3, 6, Hkv, page, sb, d)
    rng = np.random.default_rng(4)
    c["k"][:] = rng.integers(0, 127, c["k"].shape)          # every magnitude, 448 among them
    c["v"][:] = rng.integers(128, 255, c["v"].shape)
    for m in ("ks", "vs"):
        c[m][:, :, 0], c[m][:, :, 1] = np.float64(np.float32(small)), np.float64(np.float32(large))
    table, new = np.array([[0, 1, 2]], dtype=np.int32), np.array([[5, 4]], dtype=np.int32)
    w = rng.random((1, Hkv, n)).astype(np.float32)
    g = to_gpu(c)
    cuda_lib.cache_evict_fp8(*args(g), ints(table), ints([n]), torch.from_numpy(w).to(DEV), ints(new), 30, 3)
    _ok(cuda_lib)
    oc.evict(c, table, np.array([n]), w, new, 30, 3)
    assert_same_cache(g, c)


def test_append_rescales_at_the_top_of_the_range(cuda_lib):
    """Earlier tokens under a foreign scale of 1.1e36, new ones near bf16's largest number (scale 2^120)."""
    Hkv, d, page, sb = 1, 64, 16, 16
    rng = np.random.default_rng(5)
    c = random_cache(6, 2, Hkv, page, sb, d)
    c["k"][:] = rng.integers(0, 127, c["k"].shape)
    c["v"][:] = c["k"]
    for m in ("ks", "vs"):
        c[m][:] = np.float64(np.float32(1.1e36))
    k = (bf16(rng, (1, Hkv, 3, d), 0.0).clamp(-3, 3) * 1e38).to(torch.bfloat16)
    k[0, 0, 1, 7] = 3.3e38
    g, table = to_gpu(c), np.array([[1]], dtype=np.int32)
    cuda_lib.cache_append_fp8(k.to(DEV), k.to(DEV), *args(g), ints(table), ints([9]))
    _ok(cuda_lib)
    oc.append(c, table, [9], f64(k), f64(k))
    assert_same_cache(g, c)
