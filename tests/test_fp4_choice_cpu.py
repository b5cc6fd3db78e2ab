"""Which kernel and tile the 4-bit product picks (its host function, compiled here): the sizes that
tests/test_gpu_fp4.py multiplies reach every outcome that any size has."""

import os
import random
import subprocess

import diffusion_transformer_gb300 as D
from tests.test_gpu_fp4 import CLUSTER_SIZES, SIZES

CSRC = os.path.join(os.path.dirname(D.library_path), "csrc")
PROGRAM = """
#include <cstdio>
#include "fp4_choice.h"
int main() {
  int M, N, K, rows32;
  while (scanf("%d %d %d %d", &M, &N, &K, &rows32) == 4) {
    const dit::Fp4Choice c = dit::fp4_choose(M, N, K, rows32 != 0, 152);
    printf("%d %d %d\\n", c.bn, c.parts, int(c.swap));
  }
}
"""


def _choices(tmp_path, asked):
    src, exe = tmp_path / "choose.cpp", tmp_path / "choose"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", CSRC, "-o", str(exe), str(src)], check=True, capture_output=True)
    text = "".join("%d %d %d %d\n" % q for q in asked)
    out = subprocess.run([str(exe)], input=text, capture_output=True, text=True, check=True).stdout.splitlines()
    assert len(out) == len(asked)
    return [tuple(int(v) for v in line.split()) for line in out]


def test_the_gpu_tests_reach_every_kernel_and_tile(tmp_path):
    # as tests/test_gpu_fp4.py calls it: fp32 and bf16 rows one after another, and bf16 rows off 32 bytes
    asked = [(M, N, K, int(M == 1 or N % per == 0)) for M, N, K in SIZES + CLUSTER_SIZES for per in (8, 16)]
    asked += [(M, N, K, 0) for M, N, K in SIZES + CLUSTER_SIZES]
    reached = set(_choices(tmp_path, asked))
    rng = random.Random(1)
    log = lambda hi: int(round(2 ** rng.uniform(0, hi)))  # noqa: E731
    anywhere = set(_choices(tmp_path, [(log(14), log(15), log(15), rng.randrange(2)) for _ in range(200000)]))
    assert len(anywhere) >= 18 and reached >= anywhere, sorted(anywhere - reached)


def test_choices_hold_for_any_size(tmp_path):
    most = 1 << 30
    asked = [(M, N, K, r) for M in (1, 16, 17, 1000, most) for N in (1, 128, 5000, most) for K in (1, 256, 70000, most)
             for r in (0, 1) if M * K < 1 << 41 and N * K < 1 << 41 and M * N < 1 << 39]
    for (M, N, K, r), (bn, parts, swap) in zip(asked, _choices(tmp_path, asked)):
        assert parts in (0, 1, 2, 4, 8) and parts <= -(-K // 256)
        if parts:
            assert bn in (16, 32, 64, 128) and -(-M // bn) <= 65535 and (bn == 128 or M <= bn)
        else:
            assert bn in (128, 192, 256) and (swap or r)
