"""How far fa_decode_shared rounds softmax weights: own tokens' to 16 bits in every form of the call, shared ones' to bf16 in the
prefix's kernel and to 16 bits in the list of few rows."""
import math

import numpy as np
import pytest
import torch

from oracle import paged as op
from tests.paged_common import DEV, bf16, check_rows, f64, ints, ok, to_gpu
from tests.test_decode_shared_gpu import ONE, PAIR, _case

# (B, Hkv, G, Nq, d, shared, tokens of the table at least): what the prefix's kernel takes is more than 128 rows of all sequences, or
# a wide table
KERNEL = [
    (40, 2, 4, 1, 128, 300, 0),
    (40, 2, 8, 1, 64, 300, 0),
    (20, 2, 4, 4, 128, 600, 0),        # 16 rows of a sequence
    (33, 3, 1, 9, 64, 300, 0),
    (7, 2, 8, 4, 64, 1500, 0),         # 32
    (44, 3, 6, 4, 128, 260, 0),        # own tokens in a kernel of their own
    (3, 2, 4, 1, 128, 100, 40000),
]
FEW = [(3, 2, 4, 1, 128, 100, 0), (5, 2, 8, 2, 64, 900, 0), (2, 1, 4, 8, 128, 300, 0)]


def _inputs(B, Hkv, G, Nq, d, shared, wide, values):
    """A few own tokens, so that the roundings of their weights do not average out; values: of the shared tokens too, else zeros."""
    rng = np.random.default_rng(B + d)
    lens = shared + rng.integers(Nq, Nq + 6, B)
    c, table = _case(B + d, lens, shared, Hkv, 8, d)
    if not values:
        for t in range(shared):
            c["v"][table[:, t // 8], :, t % 8] = 0.0
    if wide:
        table = np.concatenate([table, np.zeros((B, -(-wide // 8)), dtype=np.int32)], 1)
    q = bf16(rng, (B, Hkv * G, Nq, d), 0.3)
    return q, c, table, lens, op.attend(f64(q), c, table, lens, 1.0 / math.sqrt(d))


def _rounded(q, c, table, lens, scale, first):
    """O with the weights of tokens from `first` on, relative to the row's largest, as one bf16 each."""
    B, Hq, Nq, d = q.shape
    Hkv, page = c["k"].shape[1:3]
    o = np.zeros(q.shape)
    for b in range(B):
        n = int(lens[b])
        j = np.arange(n)
        pg, at = table[b][j // page].astype(np.int64), j % page
        for h in range(Hq):
            K, V = c["k"][pg, h // (Hq // Hkv), at], c["v"][pg, h // (Hq // Hkv), at]
            for t in range(Nq):
                see = j <= n - Nq + t
                x = K[see] @ f64(q)[b, h, t] * scale
                p = np.exp(x - x.max())
                w = np.where(j[see] >= first, f64(torch.from_numpy(p).to(torch.bfloat16)), p)
                o[b, h, t] = w @ V[see] / p.sum()
    return o


@pytest.mark.parametrize("case", [KERNEL[0], KERNEL[3], FEW[0]])
def test_the_bounds_tell_one_bf16_from_two(case):
    q, c, table, lens, ref = _inputs(*case, False)
    lse = torch.from_numpy(ref[1])
    exact = torch.from_numpy(ref[0]).to(torch.bfloat16)
    check_rows(exact, lse, ref, PAIR)
    one = torch.from_numpy(_rounded(q, c, table, lens, 1.0 / math.sqrt(case[4]), case[5])).to(torch.bfloat16)
    check_rows(one, lse, ref, ONE)
    with pytest.raises(AssertionError, match="O exceeds"):
        check_rows(one, lse, ref, PAIR)


def _run(fa, q, c, table, lens, shared):
    g = to_gpu(c)
    o, lse = fa.decode_shared(q.to(DEV), g["k"], g["v"], ints(table), ints(lens), ints([shared]))
    ok(fa)
    return o, lse


@pytest.mark.gpu
@pytest.mark.parametrize("case", KERNEL)
def test_own_tokens_beside_a_prefix(cuda_lib, case):
    """The shared tokens' values are zeros, so that only the own tokens' weights reach O."""
    q, c, table, lens, ref = _inputs(*case, False)
    check_rows(*_run(cuda_lib, q, c, table, lens, case[5]), ref, PAIR)


@pytest.mark.gpu
@pytest.mark.parametrize("case", FEW)
def test_all_tokens_of_few_rows(cuda_lib, case):
    q, c, table, lens, ref = _inputs(*case, True)
    check_rows(*_run(cuda_lib, q, c, table, lens, case[5]), ref, PAIR)
