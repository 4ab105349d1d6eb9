"""Which rows the merge of fa_decode_shared leaves as they are: find_parts of csrc/fa_decode_rows.cuh, compiled for the host."""
import os
import subprocess

from exact_tiled_attention_21_gb300 import _build

SOURCE = r"""
#include <cstdio>
#include "fa_decode_rows.cuh"
int main() {
    using namespace fa;
    // one kv head; sequences 0 and 1 take part in a prefix of 100 tokens, 2 is shorter, 3 empty; own tokens in one segment, but for
    // sequence 1's
    const int lens[4] = {105, 300, 60, 0}, shared = 100, ends[8] = {0, 0, 0, 2, 2, 2, -7, 9};
    const int noted[2][2] = {{0, 4}, {-1, 77}};  // the prefix's first and last CTA, and what a kernel that gave up left
    for (const auto& pre : noted) {
        Params a;
        a.shared = &shared;
        a.lens = lens;
        a.ends = const_cast<int*>(ends);
        a.pre_ends = pre;
        a.B = 4, a.Hkv = 1, a.Nq = 1, a.rows = 4, a.row_tiles = 1, a.max_pages = 40;
        a.page = FastDiv(16);
        a.joint = 0, a.pre_rows = 128, a.pre_tiles = 1, a.pre_item = 0, a.pre_workers = 5;
        for (int b = 0; b < 4; ++b) {
            const Parts x = find_parts<false>(a, b, 0, 0, 0);
            printf("%d %d %d ", x.n, x.pn, (int)x.done);
        }
    }
}
"""


def test_rows_beside_a_prefix_that_left_no_parts_are_still_written(tmp_path):
    """decode_rows writes a row itself only if no prefix belongs to it; the merge decides by the same, whether the prefix's kernel
    noted its parts or gave up."""
    src, exe = str(tmp_path / "parts.cu"), str(tmp_path / "parts")
    with open(src, "w") as f:
        f.write(SOURCE)
    subprocess.run([_build.nvcc()] + _build.ARCH + _build.FLAGS + ["-I" + _build.CSRC, "-o", exe, src], check=True,
                   capture_output=True, text=True)
    got = subprocess.run([exe], check=True, capture_output=True, text=True).stdout.split()
    # (own segments, the prefix's, written already) of each sequence
    want = [1, 5, 0, 3, 5, 0, 1, 0, 1, 0, 0, 0] + [1, 0, 0, 3, 0, 0, 1, 0, 1, 0, 0, 0]
    assert list(map(int, got)) == want
