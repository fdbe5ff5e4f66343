// Scales of the 8-bit products on their way to the epilogue warps: a ring of two chunks of
// kChunk blocks in shared memory.  Plain C++, so that its layout can be checked on the host.
#pragma once

#include <cstdint>

namespace qlora {
namespace f8 {

constexpr int kChunk = 16;

// A's scales of ROWS rows and B's of COLS block columns.  SPARE rows end each chunk and are
// never written: where the sums of a block cover the latency of the next one's scales, the
// last block of a chunk reads a row further as well, and what it reads is not used.
template <int ROWS, int COLS, int SPARE = 0>
struct ScaleRing {
  float a[2][kChunk + SPARE][ROWS];
  float b[2][kChunk + SPARE][COLS];

  // Byte offsets of block i's rows from those of block 0 of the first chunk.
  static constexpr uint32_t a_at(uint32_t chunk, uint32_t i) {
    return ((chunk & 1u) * (kChunk + SPARE) + i) * ROWS * 4u;
  }
  static constexpr uint32_t b_at(uint32_t chunk, uint32_t i) {
    return ((chunk & 1u) * (kChunk + SPARE) + i) * COLS * 4u;
  }
};

// The ring of the CTA pairs (f8_gemm2.cu).
using PairRing = ScaleRing<128, 2, 1>;

}  // namespace f8
}  // namespace qlora
