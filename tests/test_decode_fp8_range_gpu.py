"""fa_decode_paged_fp8 where the values are at the ends of bf16's range."""
import math

import numpy as np
import pytest

from oracle import cache as oc
from tests.cache_fp8_common import DEV, args, bf16, check_decode, f64, ints, random_cache, table_of, to_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [1, 8, 12, 32, 40])
@pytest.mark.parametrize("n", [1, 100, 3000])
@pytest.mark.parametrize("d", [64, 128])
def test_decode_values_at_the_ends_of_the_range(cuda_lib, d, n, rows):
    """O is a mean of the values: it neither overflows where they are near bf16's largest number, nor is lost where
    every block has the smallest scale."""
    page, sb = 32, 32
    maxp = -(-n // page)
    c = random_cache(n + rows, maxp + 1, 1, page, sb, d)
    table = table_of(3, 1, maxp, maxp + 1)
    q = bf16(np.random.default_rng(rows), (1, rows, 1, d), 0.0)
    for scale, byte in ((2.0 ** 120, 224.0), (2.0 ** -126, 1.0)):
        c["vs"][:] = scale
        c["v"][:] = oc.to_e4m3(np.full(c["v"].shape, byte))
        c["v"][..., ::3] |= 0x80
        o, lse = cuda_lib.decode_paged_fp8(q.to(DEV), *args(to_gpu(c)), ints(table), ints([n]))
        check_decode(o, lse, oc.decode(f64(q), c, table, [n], 1 / math.sqrt(d)), what="scale %g" % scale)
    assert cuda_lib.fa_get_last_device_error()[0] == 0
