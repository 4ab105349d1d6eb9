"""fa_decode_shared where a kv head's query rows end in a tile of at most 128: CTAs that go from such an item to one of 256 rows
of the next kv head; and its workspaces."""
import math

import numpy as np
import pytest
import torch

from oracle import paged as op
from tests.paged_common import DEV, bf16, check_rows, f64, ints, ok, to_gpu
from tests.test_decode_shared_gpu import ONE, _case

pytestmark = pytest.mark.gpu


# Rows of a kv head are 1 to 128 more than a multiple of 256; with 152 SMs the division gives fewer CTAs than items, whose shares
# cross from a short tile of at least two steps to the next kv head's first in 10 to 29 places.
@pytest.mark.parametrize("B,Hkv,G,Nq,d,shared,most", [
    (300, 32, 1, 1, 64, 256, 8),
    (300, 12, 1, 1, 128, 390, 8),
    (300, 12, 1, 1, 64, 650, 8),
    (150, 20, 1, 2, 64, 300, 8),       # drafts
    (150, 20, 1, 2, 128, 300, 8),
    (75, 24, 2, 2, 128, 300, 8),
    (8, 80, 4, 9, 64, 520, 16),        # more than 32 rows of a sequence: own tokens in a kernel of their own
    (8, 80, 4, 9, 128, 520, 16),
])
def test_short_last_tiles(cuda_lib, B, Hkv, G, Nq, d, shared, most):
    rng = np.random.default_rng(B + d)
    lens = shared + rng.integers(Nq, max(most, Nq) + 1, B)
    lens[1] = 0
    c, table = _case(B + d, lens, shared, Hkv, 8, d)
    q, g = bf16(rng, (B, Hkv * G, Nq, d), 0.3), to_gpu(c)
    args = (q.to(DEV), g["k"], g["v"], ints(table), ints(lens), ints([shared]))
    o, lse = cuda_lib.decode_shared(*args)
    ok(cuda_lib)
    check_rows(o, lse, op.attend(f64(q), c, table, lens, 1.0 / math.sqrt(d)), ONE)
    for _ in range(20):                # whichever of the CTA's warps comes first
        again = cuda_lib.decode_shared(*args)
        assert torch.equal(again[0], o) and torch.equal(again[1], lse)
    ok(cuda_lib)


@pytest.mark.parametrize("B,Hkv,G,Nq,d,shared", [
    (3, 2, 4, 1, 128, 100),            # one list of steps
    (40, 2, 4, 1, 128, 300),           # own tokens in the prefix's kernel, one tile of rows and two
    (40, 2, 8, 1, 64, 300),
    (70, 2, 9, 4, 128, 300),           # in a kernel of their own
])
def test_a_workspace_of_16_byte_alignment(cuda_lib, B, Hkv, G, Nq, d, shared):
    """What a call needs of its workspace is 16-byte alignment and the stated size; nothing is written beside it."""
    rng = np.random.default_rng(B + d)
    lens = shared + rng.integers(Nq, 40, B)
    c, table = _case(3, lens, shared, Hkv, 8, d)
    q, g = bf16(rng, (B, Hkv * G, Nq, d), 0.3), to_gpu(c)
    args = (q.to(DEV), g["k"], g["v"], ints(table), ints(lens), ints([shared]))
    o, lse = cuda_lib.decode_shared(*args)
    check_rows(o, lse, op.attend(f64(q), c, table, lens, 1.0 / math.sqrt(d)), ONE)
    size = cuda_lib.fa_decode_shared_workspace_bytes(B, Hkv * G, Hkv, Nq, d)
    for at in (16, 32, 48, 208):
        room = torch.full((size + 512,), 0xA5, dtype=torch.uint8, device=DEV)
        w = room[at:at + size]
        assert w.data_ptr() % 32 == at % 32
        again = cuda_lib.decode_shared(*args, workspace=w)
        assert torch.equal(again[0], o) and torch.equal(again[1], lse)
        assert (room[:at] == 0xA5).all() and (room[at + size:] == 0xA5).all()
    ok(cuda_lib)
