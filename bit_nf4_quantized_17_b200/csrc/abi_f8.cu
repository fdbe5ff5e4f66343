// C ABI of the 8-bit operators: argument checks on the host, then launches on
// the caller's stream.  See include/qlora.h for the contract of each call.
#include "f8.cuh"
#include "linear.cuh"

using namespace qlora;

namespace qlora {

static constexpr int64_t kMaxElems = int64_t(1) << 36;
static constexpr int64_t kMaxSide = int64_t(1) << 30;  // tile coordinates stay inside 32 bits

static qlora_status check_f8_shape(int64_t rows, int64_t cols, int32_t layout) {
  if (rows < 0 || cols < 1 || rows > kMaxSide || cols > kMaxSide) return QLORA_ERR_SHAPE;
  if (rows > kMaxElems / cols) return QLORA_ERR_SHAPE;
  if (layout != QLORA_F8_ROWS && layout != QLORA_F8_TILES) return QLORA_ERR_UNSUPPORTED;
  return QLORA_OK;
}

qlora_status check_f8(const qlora_f8& q) {
  const qlora_status st = check_f8_shape(q.rows, q.cols, q.layout);
  if (st != QLORA_OK) return st;
  if (q.format != QLORA_E4M3 && q.format != QLORA_E5M2) return QLORA_ERR_UNSUPPORTED;
  if (q.pow2 != 0 && q.pow2 != 1) return QLORA_ERR_UNSUPPORTED;
  if (q.ld < q.cols || q.ld % 16 != 0 || q.ld > (int64_t(1) << 32)) return QLORA_ERR_SHAPE;
  if (q.rows == 0) return QLORA_OK;
  if (!q.codes || !q.scales) return QLORA_ERR_NULL;
  if (!aligned16(q.codes) || !aligned16(q.scales)) return QLORA_ERR_ALIGN;
  return QLORA_OK;
}

}  // namespace qlora

extern "C" {

qlora_status qlora_f8_sizes(int64_t rows, int64_t cols, int32_t layout, int64_t* ld,
                            size_t* codes_bytes, size_t* scales_bytes) {
  const qlora_status st = check_f8_shape(rows, cols, layout);
  if (st != QLORA_OK) return st;
  const int64_t l = ceil_div(cols, 16) * 16;
  const int64_t blocks = (layout == QLORA_F8_ROWS ? rows : f8_blocks(rows)) * f8_blocks(cols);
  if (ld) *ld = l;
  if (codes_bytes) *codes_bytes = static_cast<size_t>(rows * l);
  if (scales_bytes) *scales_bytes = static_cast<size_t>(4 * blocks);
  return QLORA_OK;
}

qlora_status qlora_f8_quantize(const void* X, int32_t x_dtype, const qlora_f8* q, void* stream) {
  const NvtxRange nvtx("qlora_f8_quantize");
  if (!q) return QLORA_ERR_NULL;
  const qlora_status st = check_f8(*q);
  if (st != QLORA_OK) return st;
  if (x_dtype != QLORA_F32 && x_dtype != QLORA_BF16) return QLORA_ERR_UNSUPPORTED;
  if (q->rows == 0) return QLORA_OK;
  if (!X) return QLORA_ERR_NULL;
  if (!aligned16(X)) return QLORA_ERR_ALIGN;
  return launch_f8_quantize(X, x_dtype, *q, static_cast<cudaStream_t>(stream));
}

qlora_status qlora_f8_dequantize(const qlora_f8* q, void* X_out, int32_t out_dtype,
                                 void* stream) {
  const NvtxRange nvtx("qlora_f8_dequantize");
  if (!q) return QLORA_ERR_NULL;
  const qlora_status st = check_f8(*q);
  if (st != QLORA_OK) return st;
  if (out_dtype != QLORA_F32 && out_dtype != QLORA_BF16) return QLORA_ERR_UNSUPPORTED;
  if (q->rows == 0) return QLORA_OK;
  if (!X_out) return QLORA_ERR_NULL;
  if (!aligned16(X_out)) return QLORA_ERR_ALIGN;
  return launch_f8_dequantize(*q, X_out, out_dtype, static_cast<cudaStream_t>(stream));
}

qlora_status qlora_f8_matmul(const qlora_f8* A, const qlora_f8* B, int32_t trans_b, void* C,
                             int32_t c_dtype, void* stream) {
  const NvtxRange nvtx("qlora_f8_matmul");
  if (!A || !B) return QLORA_ERR_NULL;
  qlora_status st = check_f8(*A);
  if (st != QLORA_OK) return st;
  if ((st = check_f8(*B)) != QLORA_OK) return st;
  if (A->layout != QLORA_F8_ROWS || B->layout != QLORA_F8_TILES) return QLORA_ERR_UNSUPPORTED;
  if (c_dtype != QLORA_F32 && c_dtype != QLORA_BF16) return QLORA_ERR_UNSUPPORTED;
  if (A->cols != (trans_b ? B->cols : B->rows)) return QLORA_ERR_SHAPE;
  if (B->rows == 0) return QLORA_ERR_SHAPE;
  const int64_t n = trans_b ? B->rows : B->cols;
  if (A->rows > kMaxElems / n) return QLORA_ERR_SHAPE;
  if (A->rows == 0) return QLORA_OK;
  if (!C) return QLORA_ERR_NULL;
  if (!aligned16(C)) return QLORA_ERR_ALIGN;
  return f8_gemm(*A, *B, trans_b != 0, C, c_dtype == QLORA_F32, F8Lora{nullptr, nullptr, 0},
                 static_cast<cudaStream_t>(stream));
}

qlora_status qlora_f8_linear_workspace(int64_t M, int64_t N, int64_t K, int32_t r,
                                       size_t* fwd_bytes, size_t* bwd_bytes) {
  if (M < 0 || N < 1 || K < 1 || r < 1 || r > 256 || M > kMaxSide || N > kMaxSide || K > kMaxSide)
    return QLORA_ERR_SHAPE;
  const LinearPlan p = plan_f8_linear(M, N, K, r);
  if (fwd_bytes) *fwd_bytes = p.fwd_workspace;
  if (bwd_bytes) *bwd_bytes = p.bwd_workspace;
  return QLORA_OK;
}

static qlora_status check_f8_linear(const qlora_f8* W, const void* A, const void* B, int32_t r,
                                    const qlora_f8* X8, const void* workspace,
                                    size_t workspace_bytes, bool bwd) {
  if (!W || !A || !B || !X8 || !workspace) return QLORA_ERR_NULL;
  qlora_status st = check_f8(*W);
  if (st != QLORA_OK) return st;
  if ((st = check_f8(*X8)) != QLORA_OK) return st;
  if (W->layout != QLORA_F8_TILES || X8->layout != QLORA_F8_ROWS) return QLORA_ERR_UNSUPPORTED;
  if (W->rows < 1 || X8->cols != W->cols || r < 1 || r > 256) return QLORA_ERR_SHAPE;
  // TMA reads bf16 rows of r, N and K elements: multiples of 16 bytes
  if (r % 8 != 0 || W->rows % 8 != 0 || W->cols % 8 != 0) return QLORA_ERR_UNSUPPORTED;
  if (!aligned16(A) || !aligned16(B) || !aligned16(workspace)) return QLORA_ERR_ALIGN;
  const LinearPlan p = plan_f8_linear(X8->rows, W->rows, W->cols, r);
  if (workspace_bytes < (bwd ? p.bwd_workspace : p.fwd_workspace)) return QLORA_ERR_WORKSPACE;
  return QLORA_OK;
}

qlora_status qlora_f8_linear_fwd(const qlora_f8* W, const void* A, const void* B, int32_t r,
                                 float alpha, const void* X, const qlora_f8* X8, void* Y,
                                 float* U_save, void* workspace, size_t workspace_bytes,
                                 void* stream) {
  const NvtxRange nvtx("qlora_f8_linear_fwd");
  const qlora_status st = check_f8_linear(W, A, B, r, X8, workspace, workspace_bytes, false);
  if (st != QLORA_OK) return st;
  if (X8->rows == 0) return QLORA_OK;
  if (!X || !Y) return QLORA_ERR_NULL;
  if (!aligned16(X) || !aligned16(Y) || !aligned16(U_save)) return QLORA_ERR_ALIGN;
  return f8_linear_forward(*W, A, B, r, alpha, X, *X8, Y, U_save, workspace,
                           static_cast<cudaStream_t>(stream));
}

// No tokens: the gradients of A and B are zero (or stay as they are).
static qlora_status no_tokens(float* dA, float* dB, int64_t r, int64_t N, int64_t K,
                              int32_t accumulate, cudaStream_t s) {
  if (accumulate) return QLORA_OK;
  if (cudaMemsetAsync(dA, 0, sizeof(float) * r * K, s) != cudaSuccess ||
      cudaMemsetAsync(dB, 0, sizeof(float) * r * N, s) != cudaSuccess)
    return QLORA_ERR_CUDA;
  return QLORA_OK;
}

qlora_status qlora_f8_linear_bwd(const qlora_f8* W, const void* A, const void* B, int32_t r,
                                 float alpha, const qlora_f8* X8, const float* U, const void* dY,
                                 int32_t grad_format, void* dX, float* dA, float* dB,
                                 int32_t accumulate, void* workspace, size_t workspace_bytes,
                                 void* stream) {
  const NvtxRange nvtx("qlora_f8_linear_bwd");
  const qlora_status st = check_f8_linear(W, A, B, r, X8, workspace, workspace_bytes, true);
  if (st != QLORA_OK) return st;
  if (grad_format != QLORA_E4M3 && grad_format != QLORA_E5M2) return QLORA_ERR_UNSUPPORTED;
  if (!dA || !dB || (X8->rows > 0 && (!U || !dY))) return QLORA_ERR_NULL;
  if (!aligned16(U) || !aligned16(dY) || !aligned16(dX) || !aligned16(dA) || !aligned16(dB))
    return QLORA_ERR_ALIGN;  // (a NULL dX counts as aligned)
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (X8->rows == 0) return no_tokens(dA, dB, r, W->rows, W->cols, accumulate, s);
  return f8_linear_backward(*W, A, B, r, alpha, *X8, U, dY, grad_format, dX, dA, dB,
                            accumulate != 0, workspace, s);
}

}  // extern "C"
