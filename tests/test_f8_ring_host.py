"""The scale ring of the 8-bit products on CTA pairs, from its own header on the host: no row
that a sum warp reads lies outside the chunk it belongs to.  (Behind the ring are the barriers of
the kernel, beside a chunk the one that is being filled.)"""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include <cstddef>
#include <cstdio>
#include "f8_ring.cuh"
using Ring = qlora::f8::PairRing;
int main() {
  const long a = offsetof(Ring, a), b = offsetof(Ring, b);
  Ring r;
  for (unsigned chunk = 0; chunk < 4; ++chunk)
    for (unsigned i = 0; i <= qlora::f8::kChunk; ++i) {  // the read behind the last block too
      const char* base = reinterpret_cast<const char*>(&r);
      const long ra = a + Ring::a_at(chunk, 0) + i * Ring::a_at(0, 1);
      const long rb = b + Ring::b_at(chunk, 0) + i * Ring::b_at(0, 1);
      const long a0 = reinterpret_cast<const char*>(&r.a[chunk & 1]) - base;
      const long b0 = reinterpret_cast<const char*>(&r.b[chunk & 1]) - base;
      const bool in = ra >= a0 && ra + (long)sizeof(r.a[0][0]) <= a0 + (long)sizeof(r.a[0]) &&
                      rb >= b0 && rb + (long)sizeof(r.b[0][0]) <= b0 + (long)sizeof(r.b[0]);
      std::printf("%u %u %d\n", chunk, i, in ? 1 : 0);
    }
}
"""


def test_pair_ring_reads_stay_in_their_chunk(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no g++")
    src, exe = tmp_path / "ring.cpp", tmp_path / "ring"
    src.write_text(PROGRAM)
    csrc = os.path.join(ROOT, "bit_nf4_quantized_17_b200", "csrc")
    subprocess.run([cxx, "-std=c++17", "-I", csrc, "-o", str(exe), str(src)], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout
    rows = [tuple(map(int, x.split())) for x in out.splitlines()]
    assert len(rows) == 4 * 17
    assert [r for r in rows if not r[2]] == []
