// C ABI of the 8-bit operators: argument checks on the host, then launches on
// the caller's stream.  See include/qlora.h for the contract of each call.
#include "f8.cuh"

using namespace qlora;

namespace qlora {

static constexpr int64_t kMaxElems = int64_t(1) << 36;

static qlora_status check_f8_shape(int64_t rows, int64_t cols, int32_t layout) {
  if (rows < 0 || cols < 1 || rows > 0x7fffffff || cols > 0x7fffff00) return QLORA_ERR_SHAPE;
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

}  // extern "C"
