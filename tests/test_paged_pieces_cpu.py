"""The arithmetic that cuts a sequence into pieces, compiled for the host, at
the sizes that the paged cache admits (2^30 slots: 2^25 tiles of 32 keys, 2^24
of 64) against whole numbers without a limit."""
import os
import random
import subprocess

from long_context_hybrid_kv_b200 import build as B

PROGRAM = r"""
#include <stdio.h>
#include "ds4a_paged.cuh"
int main() {
  int j, n, p;
  while (scanf("%d %d %d", &j, &n, &p) == 3) printf("%d\n", ds4a::paged_piece(j, n, p));
  return 0;
}
"""


def test_pieces_begin_where_whole_numbers_say(tmp_path):
    src, exe = tmp_path / "pieces.cu", tmp_path / "pieces"
    src.write_text(PROGRAM)
    subprocess.run([B.NVCC, *B.ARCH, "-std=c++17", "-I", B.INCLUDE, "-I", B.CSRC, "--expt-relaxed-constexpr", str(src), "-o",
                    str(exe)], check=True, capture_output=True)
    rng = random.Random(1)
    most = 1 << 25
    cases = [(j, n, p) for n in (2, 5, 296, 1000, 14_500_000, 15_625_000, most - 1, most) for p in (1, 2, 65, 147, 148, 295, 296)
             if p <= n for j in range(p + 1)]
    for _ in range(20000):
        p = rng.randint(1, 296)
        cases.append((rng.randint(0, p), rng.randint(p, most), p))
    out = subprocess.run([str(exe)], input="\n".join("%d %d %d" % c for c in cases), capture_output=True, text=True,
                         check=True, env={**os.environ, "CUDA_VISIBLE_DEVICES": ""}).stdout.split()
    assert len(out) == len(cases)
    for (j, n, p), got in zip(cases, out):
        assert int(got) == j * n // p, (j, n, p)
    # (the 32-bit product that this replaces: wrong at 500 million slots)
    assert ((275 * 15_625_000) & 0xFFFFFFFF) // 296 != 275 * 15_625_000 // 296
