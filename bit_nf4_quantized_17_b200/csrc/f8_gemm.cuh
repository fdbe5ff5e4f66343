// Pieces shared by the 8-bit product kernels (f8_gemm.cu, f8_gemm2.cu).
#pragma once

#include "f8.cuh"
#include "f8_ring.cuh"
#include "tc_common.cuh"
#include "tc_ptx.cuh"

namespace qlora {
namespace f8 {

constexpr long long kTimeoutCycles = 4000000000ll;  // ~2 s at 1.9 GHz

struct GemmArgs {
  int32_t m, n;                // rows (tokens) and columns of C
  int32_t kb_total, kb_per;    // 128-deep blocks, blocks per split
  int32_t n_tiles;             // tiles along the P x Q grid's fast axis
  int32_t stages;
  int32_t b_mn;                // B MN-major: its contraction axis is its rows
  int32_t ext_tiles, ext_half, ext_last_steps, ext_mn;
  int32_t c_f32;
  int32_t b_ready;             // B may be read before the launches ahead are done
  int32_t c_tma;               // C leaves through TMA stores (CTA pairs)
  const float* sa;             // A's scales, [kb][m]
  const float* sb;             // B's scales: block column nb at sb[nb * sb_n + kb * sb_k]
  int64_t sb_n, sb_k;
  void* c;
  int64_t c_ld;
  uint32_t idesc, idesc_ext;
};

// The scale ring (f8_ring.cuh) is filled by one warp with 4-byte asynchronous copies (any
// alignment), so that no epilogue warp waits for global memory and a block's scales are two
// or three shared-memory loads, issued a block ahead.
static __device__ __forceinline__ void cp_async4(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(ptx::smem_u32(dst)), "l"(src)
               : "memory");
}
// One arrival of the calling thread on `bar` once its copies so far have landed.
static __device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(ptx::smem_u32(bar))
               : "memory");
}
static __device__ __forceinline__ void cp_async_wait_all() {
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// Fills one chunk: blocks [kb, kb + kChunk) below kb_end, A's rows from `row`, B's
// scale columns from `col` (of `cols`).  Rows and columns past the end repeat the
// last one: what they scale is not stored.  All lanes of one warp; `full` counts 32.
template <int ROWS, int COLS, int SPARE>
static __device__ __forceinline__ void fill_scales(const GemmArgs& p,
                                                   ScaleRing<ROWS, COLS, SPARE>* ring, int slot,
                                                   int kb, int kb_end, int row, int col, int cols,
                                                   int lane, uint64_t* full) {
  const int n = min(kChunk, kb_end - kb);
  for (int i = 0; i < n; ++i) {
    const float* sa = p.sa + static_cast<int64_t>(kb + i) * p.m;
#pragma unroll
    for (int r = 0; r < (ROWS + 31) / 32; ++r)
      if (r * 32 + lane < ROWS)
        cp_async4(&ring->a[slot][i][r * 32 + lane], sa + min(row + r * 32 + lane, p.m - 1));
  }
  if (lane < n) {
#pragma unroll
    for (int c = 0; c < COLS; ++c)
      cp_async4(&ring->b[slot][lane][c],
                p.sb + static_cast<int64_t>(min(col + c, cols - 1)) * p.sb_n +
                    (kb + lane) * p.sb_k);
  }
  cp_async_arrive(full);
}

// acc[at ..] += s r, two sums in a register pair and instruction.
template <int N>
static __device__ __forceinline__ void add64(uint64_t (&acc)[N], int at, const uint32_t (&r)[64],
                                             float s) {
  uint64_t ss;
  asm("mov.b64 %0, {%1, %1};" : "=l"(ss) : "f"(s));
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    uint64_t x;
    asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "r"(r[2 * j]), "r"(r[2 * j + 1]));
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc[at + j]) : "l"(x), "l"(ss));
  }
}

// N consecutive columns of a row of C from column c0 (N = 4 or 16)
template <int N>
static __device__ __forceinline__ void store_run(const GemmArgs& p, int64_t row, int64_t c0,
                                          const float* v) {
  if (row >= p.m || c0 >= p.n) return;
  const int64_t at = row * p.c_ld + c0;
  const bool whole = c0 + N <= p.n;
  if (p.c_f32) {
    float* o = static_cast<float*>(p.c) + at;
    if (whole && (p.c_ld & 3) == 0) {
#pragma unroll
      for (int j = 0; j < N; j += 4)
        *reinterpret_cast<float4*>(o + j) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
    } else {
#pragma unroll
      for (int j = 0; j < N; ++j)
        if (c0 + j < p.n) o[j] = v[j];
    }
  } else {
    __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.c) + at;
    if (whole && N == 16 && (p.c_ld & 7) == 0) {
      uint32_t w[N / 2];
#pragma unroll
      for (int j = 0; j < N / 2; ++j) w[j] = tc::pack_bf16x2(v[2 * j], v[2 * j + 1]);
#pragma unroll
      for (int j = 0; j < N / 8; ++j)
        reinterpret_cast<uint4*>(o)[j] =
            make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
    } else if (whole && N == 4 && (p.c_ld & 3) == 0) {
      *reinterpret_cast<uint2*>(o) =
          make_uint2(tc::pack_bf16x2(v[0], v[1]), tc::pack_bf16x2(v[2], v[3]));
    } else {
#pragma unroll
      for (int j = 0; j < N; ++j)
        if (c0 + j < p.n) o[j] = __float2bfloat16_rn(v[j]);
    }
  }
}

// The fields of the arguments that do not depend on the kernel.
GemmArgs gemm_args(const qlora_f8& a, const qlora_f8& b, bool trans_b, void* c, bool c_f32,
                   const F8Lora& l);

}  // namespace f8

// f8_gemm2.cu: the product on CTA pairs, for sizes whose 256 x 256 tiles fill the GPU.
qlora_status f8_gemm_pairs(const qlora_f8& a, const qlora_f8& b, bool trans_b, void* c, bool c_f32,
                           const F8Lora& lora, cudaStream_t s);
// f8_gemm_pow2.cu: the same where every scale of a and b is a power of two.
qlora_status f8_gemm_pow2(const qlora_f8& a, const qlora_f8& b, bool trans_b, void* c, bool c_f32,
                          const F8Lora& lora, cudaStream_t s);

}  // namespace qlora
