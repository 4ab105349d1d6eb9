"""The serving-cache calls as the first ones of a process, under capture: nothing that they set up on the host breaks it."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import torch
import exact_tiled_attention_21_gb300 as fa
dev = torch.device("cuda", 0)
i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)
kp, vp = (torch.zeros((8, 2, 16, 64), dtype=torch.uint8, device=dev) for _ in range(2))
ks, vs = (torch.zeros((8, 2, 2), device=dev) for _ in range(2))
k = torch.randn((1, 2, 20, 64), device=dev).to(torch.bfloat16)
q = torch.randn((1, 8, 1, 64), device=dev).to(torch.bfloat16)
turns, table, new = fa.rope_table([0.1] * 32), i32([[3, 1, 5]]), i32([[0, 7]])
zero, lens, w = i32([0]), i32([20]), torch.zeros((1, 2, 48), device=dev)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    qr = fa.rope(q, turns, lens.view(1, 1))
    fa.cache_append_fp8(k, k, kp, vp, ks, vs, table, zero, turns=turns)
    o, lse = fa.decode_paged_fp8(qr, kp, vp, ks, vs, table, lens, weights=w)
    out = fa.cache_evict_fp8(kp, vp, ks, vs, table, lens, w, new, 10, 4)
graph.replay()
torch.cuda.synchronize()
assert o.isfinite().all() and lse.isfinite().all() and abs(float(w.sum()) - 8.0) < 1e-3
assert int(out[0]) == 10 and fa.fa_get_last_device_error()[0] == 0
print("captured")
"""


def test_first_calls_under_capture(cuda_lib):
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stdout + r.stderr
