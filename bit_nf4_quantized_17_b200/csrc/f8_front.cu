// Launches of f8_front_kernel (f8_front.cuh).
#include <algorithm>

#include "f8_front.cuh"

namespace qlora {

// Up to 16 tokens this kernel is the faster form at any size, with f8_front_wide_kernel's rows
// mostly empty: forward of the layer with this one and with that, one token x 4096 x 4096 at
// rank 16 9.4 and 13.0 us, 16 x 8192 x 8192 at rank 64 14.5 and 22.5, 16 x 1024 x 20000 at
// rank 256 21.0 and 36.2.  Up to 256 tokens it is where every warp has one block at most (16
// tokens x 16 ranks x 128 columns), so that the launch is one latency: 24 x 4096 x 4096 at
// rank 16 11.7 and 15.2, 128 x 4096 x 4096 at rank 64 15.4 and 18.8, 256 of them 18.6 and 20.5.
// With more blocks (256 x 8192 x 8192 at rank 64: 39.7 and 36.5; 128 x 1024 x 8192 at rank 256:
// 33.7 and 27.3) or tokens reading X and A once each wins.
bool f8_front_takes(int64_t M, int64_t K, int32_t r) {
  if (M <= 16 || M > 256) return M <= 16;
  return ceil_div(M, 16) * f8_blocks(K) * ceil_div(r, kRanks) <= f8::sm_count() * kMaxWarps;
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
  const int64_t warps = static_cast<int64_t>(f8::sm_count()) * kMaxWarps;
  int64_t blocks;
  int slices;
  for (p.tiles = 1;; p.tiles *= 2) {
    blocks = ceil_div(M, 16 * p.tiles);
    slices = std::min(kMaxWarps / p.tiles, p.per);
    if (p.tiles == 8 || ctas * groups * blocks * p.tiles * slices <= warps) break;
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
