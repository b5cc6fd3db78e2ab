"""Where the scale bytes of a 4-bit matrix stand, from the functions the kernels address them with (compiled here
for the host), against the layout that the header describes, up to the largest sizes it allows."""

import os
import subprocess

import pytest

import diffusion_transformer_gb300 as D

CSRC = os.path.join(os.path.dirname(D.library_path), "csrc")
PROGRAM = """
#include <cstdio>
#include "fp4_layout.h"
int main() {
  int fmt, cols, row, block;
  while (scanf("%d %d %d %d", &fmt, &cols, &row, &block) == 4)
    printf("%lld\\n", dit::fp4_scale_row(fmt, row, cols) + (long long)dit::fp4_scale_block(block));
}
"""
MOST = 1 << 30


def _offsets(tmp_path, asked):
    src, exe = tmp_path / "at.cpp", tmp_path / "at"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-I", CSRC, "-o", str(exe), str(src)], check=True, capture_output=True)
    text = "".join("%d %d %d %d\n" % q for q in asked)
    out = subprocess.run([str(exe)], input=text, capture_output=True, text=True, check=True).stdout.split()
    return [int(v) for v in out]


@pytest.mark.parametrize("fmt,size", [(D.DIT_FP4_NV, 16), (D.DIT_FP4_MX, 32)], ids=["nv", "mx"])
def test_scale_offsets_up_to_the_largest_sizes(tmp_path, fmt, size):
    asked = []
    for cols in (1, 5 * size + 1, (1 << 24) * size - 1, (1 << 24) * size + 16, MOST - 7, MOST):
        last = (cols - 1) // size
        for row in (0, 31, 32, 127, 128, 1000, MOST - 1):
            for block in sorted({0, last // 2, max(0, last - 1), last, last // 4 * 4}):
                asked.append((fmt, cols, row, block))
    got = _offsets(tmp_path, asked)
    assert len(got) == len(asked)
    for (_, cols, row, block), at in zip(asked, got):
        tiles = -(-cols // (4 * size))
        want = ((row // 128) * tiles + block // 4) * 512 + 16 * (row % 32) + 4 * (row % 128 // 32) + block % 4
        assert at == want, (cols, row, block)
        if row < 1 << 20:
            assert at < D.dit_fp4_scale_bytes(fmt, row + 1, cols)
