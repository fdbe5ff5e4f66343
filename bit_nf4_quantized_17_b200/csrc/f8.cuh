// Matrices held in 8-bit floating point with one scale per block of 128:
// internal declarations of the quantiser, the products and the rank-r gradient.
#pragma once

#include <cuda_fp8.h>

#include "internal.cuh"
#include "kernels.cuh"

namespace qlora {

// Scale blocks along one axis of `n` elements.
inline int64_t f8_blocks(int64_t n) { return ceil_div(n, 128); }

// f8_gemm.cu: SMs of the current device.
namespace f8 {
int sm_count();
}

// abi_f8.cu: shape and pointer checks of a qlora_f8.
qlora_status check_f8(const qlora_f8& q);

// f8_quantize.cu
qlora_status launch_f8_quantize(const void* X, int32_t x_dtype, const qlora_f8& q, cudaStream_t s);
qlora_status launch_f8_dequantize(const qlora_f8& q, void* out, int32_t out_dtype,
                                  cudaStream_t s);

// f8_front.cu: 8 bits of bf16 X (into x8, by rows) and one LoRA factor in one launch:
// U = X A^T with A r x K, or (along) U = X A with A K x r.  K = x8.cols, r multiples of 8.
// f8_front_takes: where it is the faster form.
struct FrontOp {
  const void* x;
  const void* a;
  int32_t r;
  bool along;
  bool encode;    // false: x8 gives the sizes only
  float* u;       // U (M x r fp32) or NULL
  float sc;
  void* su;       // sc U as bf16 [hi | lo], lora_span(r) columns each
  void* ut;       // U^T as three bf16 terms, ut_lo rows apart, rows of ut_ld; or NULL
  int64_t ut_ld;
  int32_t ut_lo;
};
bool f8_front_takes(int64_t M, int64_t K, int32_t r);
qlora_status f8_front(const FrontOp& f, const qlora_f8& x8, cudaStream_t s);
// f8_front_wide.cu: the same for many tokens.
qlora_status f8_front_wide(const FrontOp& f, const qlora_f8& x8, DeviceStatus* st,
                           cudaStream_t s);

// The LoRA term of a product, added as extra stages of the same accumulators:
// C += hi . R + lo . R with [hi | lo] = L (m x 2 lora_span(r) bf16) and R (bf16)
// B (n x r, K-major) in the forward, A (r x n, MN-major) in the backward.
struct F8Lora {
  const void* L;
  const void* R;
  int32_t r;  // 0 = no LoRA term
  // The launches ahead of the product belong to the same call and write neither B nor R,
  // and the first of them began when everything before it was done: B may be read at once.
  bool b_ready = false;
};

// f8_gemm.cu: C (m x n, row-major, bf16 or fp32) = A . B^T (trans_b) or A . B,
// A by rows, B by tiles, plus the LoRA term.  Any sizes; m >= 1.
qlora_status f8_gemm(const qlora_f8& a, const qlora_f8& b, bool trans_b, void* c, bool c_f32,
                     const F8Lora& lora, cudaStream_t s);

// f8_gemm.cu: clusters of such a launch (all CTAs along z) that run at once.  A cluster lies
// within one group of SMs: of size 8 at one CTA per SM fewer than 16 do.
int f8_resident_clusters(const void* fn, const cudaLaunchConfig_t& cfg);

// f8_grad_b.cu: dB (N x r fp32) = sc dY^T U (added to dB when accumulate), dY M x N bf16, U
// M x r fp32, r and N multiples of 8.  ut: room for U^T as three bf16 terms, lora_rows(r) rows
// each of ld_u elements (a multiple of 8, at least M).
qlora_status f8_grad_b(const void* dY, int64_t N, const float* U, int64_t M, int32_t r, float sc,
                       bool accumulate, void* ut, int64_t ld_u, float* dB, DeviceStatus* st,
                       cudaStream_t s);

// f8_grad.cu: dA (r x d_in fp32) = sc V^T X^ from X kept by rows in 8 bits (added to
// dA when accumulate).  More than 16 tokens: V^T as three bf16 terms, lora_rows(r)
// rows apart, ld_v elements a row; r a multiple of 8 up to 256.  Up
// to 16 tokens: V (M x r fp32), r and d_in multiples of 8.
qlora_status f8_grad_a(const void* vt, int64_t ld_v, const qlora_f8& x, int32_t r, float sc,
                       bool accumulate, float* dA, DeviceStatus* st, cudaStream_t s);
qlora_status f8_small_grad_a(const float* V, const qlora_f8& x, int r, float sc, bool accumulate,
                             float* dA, cudaStream_t s);

}  // namespace qlora
