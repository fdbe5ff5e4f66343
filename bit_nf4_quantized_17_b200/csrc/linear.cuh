// Forward / backward orchestration of the QLoRA linear layer.
#pragma once

#include "internal.cuh"
#include "kernels.cuh"

namespace qlora {

// Pieces shared by the linear layers over the NF4 and the 8-bit base.
inline size_t align256(size_t b) { return (b + 255) & ~size_t(255); }
inline int64_t pad8(int64_t v) { return (v + 7) / 8 * 8; }
inline float lora_scale(float alpha, int32_t r) { return alpha / static_cast<float>(r); }

struct SideStream {
  cudaStream_t stream = nullptr;
  cudaEvent_t fork = nullptr, join = nullptr;
};
qlora_status side_stream(SideStream** out);

ReduceArgs reduce_args(const float* part, int splits, int64_t rows, int cols, int pcols);
qlora_status rank_product(const void* A, bool a_mn, int64_t m_rows, int64_t kdim, int64_t ld_a,
                          const void* B, int64_t ld_b, int32_t b_rows, int32_t n_cols,
                          float* part, int splits, const ReduceArgs& out, DeviceStatus* st,
                          cudaStream_t s);

#define QLORA_TRY(x)                      \
  do {                                    \
    qlora_status _st = (x);               \
    if (_st != QLORA_OK) return _st;      \
  } while (0)

struct LinearPlan {
  size_t fwd_workspace;
  size_t bwd_workspace;
};

LinearPlan plan_linear(int64_t M, int64_t N, int64_t K, int32_t r);

// Options of the adapter branch.
//  - Several adapters: r = n_adapters * r_adapter (A and B stacked along the
//    rank); seg[m] is the adapter of token m, and the reductions that produce
//    U and V zero the columns of the other adapters, so every later step (the
//    fused GEMMs' LoRA stages, dA, dB) sees only each token's own adapter.
//    One adapter: seg == nullptr and r_adapter == r.  The scale is
//    alpha / r_adapter.
//  - LoRA dropout: the adapter branch reads x_drop = X (.) D instead of X,
//    keep = 1 / (1 - p), and the LoRA part of dX is masked by D (mask != nullptr).
//    Without dropout x_drop = X, keep = 1 and mask = nullptr.
//  - Input kept in 8 bits (backward only): dA reads x8 instead of X (or of
//    x_drop, whose kept form it then is); x_buf is for the CUDA-core path to
//    restore it (M x K bf16), and above 16 tokens on the tensor cores for V^T.
struct LoraOpts {
  int32_t r_adapter;
  const int32_t* seg;
  const void* x_drop;
  const uint8_t* mask;
  float keep;
  const qlora_f8* x8 = nullptr;
  void* x_buf = nullptr;
};

bool linear_multi_supported(int64_t M, int64_t N, int64_t K, int32_t r);

// Bytes behind the backward's workspace for an M x K input that is kept in 8 bits (x_buf).
size_t f8_input_bytes(int64_t M, int64_t N, int64_t K, int32_t r);

// f8_linear.cu: the layer over an 8-bit base (tiles).  r, N and K multiples of 8.
LinearPlan plan_f8_linear(int64_t M, int64_t N, int64_t K, int32_t r);
qlora_status f8_linear_forward(const qlora_f8& W, const void* A, const void* B, int32_t r,
                               float alpha, const void* X, const qlora_f8& x8, void* Y,
                               float* U_save, void* workspace, cudaStream_t s);
qlora_status f8_linear_backward(const qlora_f8& W, const void* A, const void* B, int32_t r,
                                float alpha, const qlora_f8& x8, const float* U, const void* dY,
                                int32_t grad_format, void* dX, float* dA, float* dB,
                                bool accumulate, void* workspace, cudaStream_t s);

qlora_status linear_forward(const qlora_nf4& W, const LevelTable& t, const void* A,
                            const void* B, int32_t r, float alpha, const void* X, int64_t M,
                            void* Y, float* U_save, void* workspace, cudaStream_t s,
                            const LoraOpts& o);

qlora_status linear_backward(const qlora_nf4& W, const LevelTable& t, const void* A,
                             const void* B, int32_t r, float alpha, const void* X,
                             const float* U, const void* dY, int64_t M, void* dX, float* dA,
                             float* dB, bool accumulate, void* workspace, cudaStream_t s,
                             const LoraOpts& o);

}  // namespace qlora
