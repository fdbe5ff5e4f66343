// Launches of f8_front_kernel (f8_front.cuh).
#include <algorithm>

#include "f8_front.cuh"

namespace qlora {

// Where every warp has one block at most (16 tokens x 16 ranks x 128 columns) the launch is
// one latency.  Forward of the layer with this kernel and with f8_front_wide's: 24 x 4096 x
// 4096 at rank 16 11.7 and 14.6 us, 128 of them at rank 64 16.3 and 18.6, 256 18.9 and
// 20.4.  With more blocks (256 x 8192 x 8192 at rank 64: 42.6 and 36.8) or tokens (512 x
// 4096 x 4096 at rank 16: 27.3 and 22) reading X and A once each wins.
bool f8_front_takes(int64_t M, int64_t K, int32_t r) {
  return M <= 16 ||
         (M <= 256 && ceil_div(M, 16) * f8_blocks(K) * ceil_div(r, kRanks) <= 148 * kMaxWarps);
}

qlora_status f8_front(const FrontOp& f, const qlora_f8& x8, cudaStream_t s) {
  const int64_t M = x8.rows, K = x8.cols;
  if (M < 1 || K % 8 != 0 || f.r % 8 != 0) return QLORA_ERR_UNSUPPORTED;
  FrontArgs p{};
  p.x = static_cast<const __nv_bfloat16*>(f.x);
  p.a = static_cast<const __nv_bfloat16*>(f.a);
  p.codes = f.encode ? x8.codes : nullptr;
  p.scales = x8.scales;
  p.k = K;
  p.ld = x8.ld;
  p.m = M;
  p.r = f.r;
  p.kbs = static_cast<int32_t>(f8_blocks(K));
  p.pow2 = x8.pow2;
  p.span = lora_span(f.r);
  p.u = f.u;
  p.su = static_cast<__nv_bfloat16*>(f.su);
  p.sc = f.sc;
  p.ut = static_cast<__nv_bfloat16*>(f.ut);
  p.ut_ld = f.ut_ld;
  p.ut_lo = f.ut_lo;
  p.per = static_cast<int32_t>(ceil_div(p.kbs, kMaxCtas));
  const int ctas = static_cast<int>(ceil_div(p.kbs, p.per));
  const int64_t groups = p.span / kRanks;  // those past the last rank write zeros
  // a warp per 16 tokens and block of 128 columns, as far as all run at once; then
  // more tokens per CTA and more blocks per warp
  int64_t blocks;
  int slices;
  for (p.tiles = 1;; p.tiles *= 2) {
    blocks = ceil_div(M, 16 * p.tiles);
    slices = std::min(kMaxWarps / p.tiles, p.per);
    if (p.tiles == 8 || ctas * groups * blocks * p.tiles * slices <= 148 * kMaxWarps) break;
  }
  const bool e5 = x8.format == QLORA_E5M2, two = M > 8;
  const void* fn = f.along ? front_along_kernel(e5, two) : front_kernel<false>(e5, two);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas), static_cast<unsigned>(groups),
                     static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(static_cast<unsigned>(32 * p.tiles * slices));
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(ctas);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  void* args[] = {&p};
  const int kind = f.encode ? QLORA_KERNEL_QUANTIZE : QLORA_KERNEL_LORA_GEMM;
  count_launch();
  timing_mark(kind, s, true);
  const cudaError_t e = cudaLaunchKernelExC(&cfg, fn, args);
  timing_mark(kind, s, false);
  if (e != cudaSuccess) {
    (void)cudaGetLastError();
    return QLORA_ERR_CUDA;
  }
  return after_launch("f8_front", s);
}

}  // namespace qlora
