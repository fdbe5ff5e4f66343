// Forward and backward of the linear layer over an 8-bit base weight.
//
// The base W (tiles of 128 x 128) takes the place of the NF4 weight; the LoRA
// branch is the same ("LoRA 与 QLoRA：把大模型微调拆成可负担的工程", 2 and 6):
//   forward   X^ = 8 bits of X (by rows; kept for the backward), U = X A^T,
//             Y = X^ W^T + s U B^T
//   backward  dY^ = 8 bits of dY (by rows), V = dY B, dX = dY^ W + s V A,
//             dB = s dY^T U, dA = s V^T X^
// Both large products run on the tensor cores in 8 bits, with the LoRA term as
// extra bf16 stages of the same accumulators; the rank-r products read X and dY
// in bf16, except dA, which reads the kept X^.
#include <algorithm>

#include "f8.cuh"
#include "linear.cuh"

namespace qlora {
namespace {

// Workspace (byte offsets; the status word is first).
//   forward   sU [hi | lo]
//   backward  sV [hi | lo] | V (fp32, few tokens) or V^T (three bf16 terms) |
//             U^T (three bf16 terms) | dY codes | dY scales
struct Layout {
  size_t su, fwd_end;
  size_t sv, vt, ut, dy_codes, dy_scales, bwd_end;
  int64_t dy_ld;
};

Layout layout(int64_t M, int64_t N, int32_t r) {
  Layout L{};
  if (M < 1) M = 1;  // no tokens: no work, but a workspace with a status word
  const int64_t span = lora_span(r), r16 = lora_rows(r), mp = pad8(M);
  L.su = kStatusBytes;
  L.fwd_end = L.su + align256(2 * M * 2 * span);
  L.sv = kStatusBytes;
  L.vt = L.sv + align256(2 * M * 2 * span);
  L.ut = L.vt + align256(std::max<size_t>(2 * 3 * r16 * mp, sizeof(float) * M * r));
  L.dy_codes = L.ut + align256(2 * 3 * r16 * mp);
  L.dy_ld = ceil_div(N, 16) * 16;
  L.dy_scales = L.dy_codes + align256(M * L.dy_ld);
  L.bwd_end = L.dy_scales + align256(sizeof(float) * f8_blocks(N) * M);
  return L;
}

}  // namespace

LinearPlan plan_f8_linear(int64_t M, int64_t N, int64_t K, int32_t r) {
  (void)K;
  const Layout L = layout(M, N, r);
  return LinearPlan{L.fwd_end, L.bwd_end};
}

qlora_status f8_linear_forward(const qlora_f8& W, const void* A, const void* B, int32_t r,
                               float alpha, const void* X, const qlora_f8& x8, void* Y,
                               float* U_save, void* workspace, cudaStream_t s) {
  const int64_t M = x8.rows, N = W.rows, K = W.cols;
  const Layout L = layout(M, N, r);
  const float sc = lora_scale(alpha, r);
  char* ws = static_cast<char*>(workspace);
  auto* st = reinterpret_cast<DeviceStatus*>(ws);
  char* su = ws + L.su;
  // U = X A^T -> U_save (fp32) and sU = s U as bf16 hi + lo; the 8 bits of X
  const FrontOp f{X, A, r, false, true, U_save, sc, su, nullptr, 0, 0};
  QLORA_TRY(f8_front_takes(M, K, r) ? f8_front(f, x8, s) : f8_front_wide(f, x8, st, s));
  // starts beside what is ahead of it in this call and reads W at once
  return f8_gemm(x8, W, true, Y, false, F8Lora{su, B, r, true}, s);
}

qlora_status f8_linear_backward(const qlora_f8& W, const void* A, const void* B, int32_t r,
                                float alpha, const qlora_f8& x8, const float* U, const void* dY,
                                int32_t grad_format, void* dX, float* dA, float* dB,
                                bool accumulate, void* workspace, cudaStream_t s) {
  const int64_t M = x8.rows, N = W.rows, K = W.cols;
  const Layout L = layout(M, N, r);
  const float sc = lora_scale(alpha, r);
  const int32_t r16 = lora_rows(r);
  const int64_t mp = pad8(M);
  char* ws = static_cast<char*>(workspace);
  auto* st = reinterpret_cast<DeviceStatus*>(ws);
  char *sv = ws + L.sv, *vt = ws + L.vt, *ut = ws + L.ut;
  float* v = reinterpret_cast<float*>(vt);  // few tokens: V in fp32
  const bool small = M <= kSmallM;
  const qlora_f8 dy8{M, N, L.dy_ld, QLORA_F8_ROWS, grad_format, x8.pow2, 0,
                     reinterpret_cast<uint8_t*>(ws + L.dy_codes),
                     reinterpret_cast<float*>(ws + L.dy_scales)};
  // dX on the caller's stream; beside it dB, which needs only inputs, and dA after V
  SideStream* ss = nullptr;
  QLORA_TRY(side_stream(&ss));
  const cudaStream_t s2 = ss->stream;
  auto fork = [&]() -> bool {
    return cudaEventRecord(ss->fork, s) == cudaSuccess &&
           cudaStreamWaitEvent(s2, ss->fork, 0) == cudaSuccess;
  };
  // V = dY B -> sV = s V as [hi | lo], and V (fp32) or V^T in terms; the 8 bits of dY
  auto v_work = [&]() -> qlora_status {
    const FrontOp f{dY, B, r, true, dX != nullptr, small ? v : nullptr, sc, sv,
                    small ? nullptr : vt, mp, r16};
    return f8_front_takes(M, N, r) ? f8_front(f, dy8, s) : f8_front_wide(f, dy8, st, s);
  };
  auto grad_b = [&]() -> qlora_status {
    if (small) return small_grad_b(dY, U, static_cast<int>(M), N, r, sc, accumulate, dB, s2);
    return f8_grad_b(dY, N, U, M, r, sc, accumulate, ut, mp, dB, st, s2);
  };
  auto all_work = [&]() -> qlora_status {
    QLORA_TRY(v_work());
    QLORA_TRY(grad_b());
    if (!fork()) return QLORA_ERR_CUDA;
    if (dX) QLORA_TRY(f8_gemm(dy8, W, false, dX, false, F8Lora{sv, A, r, true}, s));
    if (small) return f8_small_grad_a(v, x8, r, sc, accumulate, dA, s2);
    return f8_grad_a(vt, mp, x8, r, sc, accumulate, dA, st, s2);
  };
  if (!fork()) return QLORA_ERR_CUDA;
  const qlora_status done = all_work();
  // join on every path, so that nothing of this call runs past it on the side stream
  const bool joined = cudaEventRecord(ss->join, s2) == cudaSuccess &&
                      cudaStreamWaitEvent(s, ss->join, 0) == cudaSuccess;
  if (done != QLORA_OK) return done;
  return joined ? QLORA_OK : QLORA_ERR_CUDA;
}

}  // namespace qlora
