// dB = s dY^T U of the layer over an 8-bit base, for more than 16 tokens.
//
//   dB[n][j] = s sum_m dY[m][n] U[m][j]
//
// D = dY^T U per 128 columns of dY on the tensor cores (tcgen05.mma kind::f16, M = 128, N =
// rc ranks <= 128), the contraction over tokens split over a cluster and summed in distributed
// shared memory in split order, as in gemm_rank.cu.  U is fp32 and enters as three bf16 terms
// (two would leave dB off by 2.5e-6 relative), with the accumulators of f8_grad.cu: several
// in turn for the first term, one for the small products of the other two.  Relative to fp64
// at rank 16, 4096 columns: 4096 tokens 2.4e-7, 65536 4.8e-7 (2.6e-6 and 1.9e-5 with two
// terms in one accumulator).
//
// Bound by latency at a few thousand tokens (loads two to five stages deep, the start and the
// sum across the cluster): 4096 x 4096 at rank 16 cold in 13.7 us, 34 MB from DRAM (38% of
// HBM); 2048 x 8192 at rank 64 17.4 us (30%).  Above rank 64 U's terms from L2, 6 bytes a rank and
// token for each 128 columns, weigh too.
//
// Roles (192 threads): warp 0 TMA producer, warp 1 TMEM owner and MMA issuer, warps 2-5 drain
// and sum.  Every wait is bounded; a wait that gives up reports QLORA_ERR_DEVICE_TIMEOUT and
// leaves NaN in its rows of dB.
#include <cudaTypedefs.h>

#include <algorithm>

#include "f8.cuh"
#include "f8_codec.cuh"
#include "f8_splits.cuh"
#include "linear.cuh"
#include "tc_common.cuh"
#include "tc_ptx.cuh"

namespace qlora {
namespace {

constexpr int kThreads = 192;
constexpr int kABytes = 16384;  // 64 tokens x 128 columns of dY, two 64-column halves
constexpr int kTerms = 3;       // of U
constexpr int kMaxStages = 8;
constexpr int kBesideBytes = 1024 + 8 * (2 * kMaxStages + 1) + 8;  // alignment, barriers, two words
constexpr long long kTimeoutCycles = 4000000000ll;

struct GradBArgs {
  int32_t n;                    // columns of dY
  int32_t kt0, kt_end, kt_per;  // 64-token tiles of this launch, tiles per split
  int32_t r, rc, term_rows;     // rank, ranks per chunk (a multiple of 16), rows of a term of U^T
  int32_t stages, area;         // of tiles; their bytes (the partial sums reuse them)
  int32_t accs, tmem_cols;      // accumulators of the first term (a power of two), TMEM columns
  float* dB;
  float sc;
  int32_t accumulate;
  uint32_t idesc;
  DeviceStatus* st;
};

__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr));
  return v;
}

__global__ void __launch_bounds__(kThreads, 2)
f8_grad_b_kernel(const __grid_constant__ CUtensorMap tmY, const __grid_constant__ CUtensorMap tmU,
                 const GradBArgs p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  // [stages x (dY | U^T)], reused as the fp32 partial sums
  const int stage_bytes = kABytes + kTerms * p.rc * 128;
  float* red = reinterpret_cast<float*>(smem);  // [128][rc + 4]
  const int red_ld = p.rc + 4;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + p.area);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  uint64_t* full = reinterpret_cast<uint64_t*>(tmem_slot + 2);
  uint64_t* empty = full + kMaxStages;
  uint64_t* accum = empty + kMaxStages;

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int S = static_cast<int>(gridDim.z), z = static_cast<int>(blockIdx.z);  // a cluster's
  const int n0 = blockIdx.x * 128;
  const int j0 = blockIdx.y * p.rc;  // first rank of the chunk
  const int t0 = p.kt0 + z * p.kt_per;
  const int tn = max(0, min(p.kt_per, p.kt_end - t0));

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      ptx::mbar_init(&full[s], 1);
      ptx::mbar_init(&empty[s], 1);
    }
    ptx::mbar_init(accum, 1);
    *abort_flag = 0;
    ptx::fence_mbar_init();
    ptx::prefetch_tmap(&tmY);
    ptx::prefetch_tmap(&tmU);
  }
  if (warp == 1) {
    ptx::tmem_alloc(tmem_slot, p.tmem_cols);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0 && ptx::elect_one()) {
    // ------------------------------------------------------ TMA producer
    int s = 0, issued = 0;
    uint32_t ph = 1;
    uint8_t* sp = smem;
    for (int i = 0, m = t0 * 64; i < tn; ++i, m += 64) {
      if (!ptx::mbar_wait(&empty[s], ph, kTimeoutCycles, abort_flag)) break;
      ptx::mbar_arrive_expect_tx(&full[s], stage_bytes);
      ptx::tma_load_2d(&tmY, &full[s], sp, n0, m);
      ptx::tma_load_2d(&tmY, &full[s], sp + 8192, n0 + 64, m);
#pragma unroll
      for (int t = 0; t < kTerms; ++t)
        ptx::tma_load_2d(&tmU, &full[s], sp + kABytes + t * p.rc * 128, m, t * p.term_rows + j0);
      ++issued;
      sp += stage_bytes;
      if (++s == p.stages) {
        s = 0;
        ph ^= 1;
        sp = smem;
      }
    }
    // never leave with copies in flight into this CTA's shared memory
    for (int i = (issued > p.stages ? issued - p.stages : 0); i < issued; ++i)
      ptx::mbar_wait(&full[i % p.stages], (i / p.stages) & 1, kTimeoutCycles, nullptr);
  } else if (warp == 1 && ptx::elect_one()) {
    // ------------------------------------------------------ MMA issuer
    const uint64_t term = static_cast<uint64_t>(p.rc * 128) >> 4;
    const uint32_t rest = tmem + p.accs * p.rc;
    const uint32_t y_addr = ptx::smem_u32(smem);
    // dY: MN-major, two 64-column halves 8192 bytes apart, 16 tokens (2048 bytes) a step
    const uint64_t a0 = ptx::sw128_desc(y_addr, 8192, 1024);
    const uint64_t b0 = ptx::sw128_desc(y_addr + kABytes, 16, 1024);
    int s = 0;
    uint32_t ph = 0;
    uint64_t off = 0;
    for (int i = 0; i < tn; ++i) {
      if (!ptx::mbar_wait(&full[s], ph, kTimeoutCycles, abort_flag)) break;
      ptx::tc_fence_after();
      const uint32_t d = tmem + (i & (p.accs - 1)) * p.rc;
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) {
        const uint64_t a = a0 + off + ((2048 * ks) >> 4), b = b0 + off + ((32 * ks) >> 4);
        ptx::umma_bf16(d, a, b, p.idesc, i >= p.accs || ks != 0 ? 1u : 0u);
        ptx::umma_bf16(rest, a, b + term, p.idesc, (i | ks) != 0 ? 1u : 0u);
        ptx::umma_bf16(rest, a, b + 2 * term, p.idesc, 1u);
      }
      ptx::umma_commit(&empty[s]);
      off += stage_bytes >> 4;
      if (++s == p.stages) {
        s = 0;
        ph ^= 1;
        off = 0;
      }
    }
    ptx::umma_commit(accum);
    ptx::mbar_wait(accum, 0, kTimeoutCycles, nullptr);  // MMAs done before TMEM is freed
  }
  __syncthreads();  // every copy has landed and every MMA has read its tiles
  // ---------------------------------------- partial sums to shared memory
  if (warp >= 2) {
    const int quarter = warp & 3;  // TMEM lanes 32 quarter .. + 31
    const int row = 32 * quarter + lane;
    bool ok = tn > 0 && ptx::mbar_wait(accum, 0, kTimeoutCycles, abort_flag);
    ok = __all_sync(0xffffffffu, ok && !*abort_flag);
    if (ok) ptx::tc_fence_after();
    const uint32_t at = tmem + (static_cast<uint32_t>(32 * quarter) << 16);
    const int used = min(p.accs, tn);
    for (int c = 0; c < p.rc; c += 16) {
      float v[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) v[j] = 0.0f;
      // the small products first
      for (int a = used; ok && a >= 0; --a) {
        uint32_t r[16];
        ptx::tmem_ld_x16(at + (a == used ? p.accs : a) * p.rc + c, r);
        ptx::tmem_ld_wait(r);
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] += __uint_as_float(r[j]);
      }
      float* dst = red + row * red_ld + c;
#pragma unroll
      for (int j = 0; j < 16; j += 4)
        *reinterpret_cast<float4*>(dst + j) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  // a wait of this CTA gave up: its sums are not whole (the status word may not be read)
  if (*abort_flag)
    for (int e = threadIdx.x; e < 128 * red_ld; e += kThreads) red[e] = __int_as_float(0x7fffffff);
  ptx::cluster_sync();
  // ---------------------------------------- sum over the splits, in order
  // runs of four ranks (r is a multiple of 8), dealt to the CTAs of the cluster
  const int runs = min(p.rc, p.r - j0) >> 2, rows = min(128, p.n - n0);
  for (int e = z * kThreads + static_cast<int>(threadIdx.x); e < rows * runs; e += S * kThreads) {
    const int i = e / runs, j = 4 * (e - i * runs);
    const uint32_t off = static_cast<uint32_t>(i * red_ld + j) * 4u;
    float4 f[8];
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (q < S) f[q] = ld_cluster_f32x4(ptx::cluster_addr(red, static_cast<uint32_t>(q)) + off);
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      if (q < S) {
        v.x += f[q].x;
        v.y += f[q].y;
        v.z += f[q].z;
        v.w += f[q].w;
      }
    }
    float4* dst = reinterpret_cast<float4*>(p.dB + static_cast<int64_t>(n0 + i) * p.r + j0 + j);
    float4 o = make_float4(p.sc * v.x, p.sc * v.y, p.sc * v.z, p.sc * v.w);
    if (p.accumulate) {
      const float4 d = *dst;
      o = make_float4(d.x + o.x, d.y + o.y, d.z + o.z, d.w + o.w);
    }
    *dst = o;
  }
  // no CTA leaves (or frees TMEM) while the others may still read its sums
  __syncthreads();
  ptx::cluster_sync();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, p.tmem_cols);
  }
  if (threadIdx.x == 0 && *abort_flag) report(p.st, QLORA_ERR_DEVICE_TIMEOUT, 160u);
}

// ------------------------------------------------------------ U^T in terms
// A CTA turns 64 tokens x 32 ranks: whole lines in, whole lines out.
__global__ void __launch_bounds__(256)
terms_kernel(const float* __restrict__ u, int64_t m, int r, __nv_bfloat16* __restrict__ ut,
             int64_t ld, int64_t term) {
  __shared__ float tile[32][65];
  const int64_t m0 = static_cast<int64_t>(blockIdx.x) * 64;
  const int j0 = blockIdx.y * 32;
  for (int e = threadIdx.x; e < 64 * 8; e += 256) {
    const int i = e >> 3, j = 4 * (e & 7);
    if (m0 + i >= m || j0 + j >= r) continue;  // r is a multiple of 4
    const float4 f = __ldg(reinterpret_cast<const float4*>(u + (m0 + i) * r + j0 + j));
    tile[j][i] = f.x;
    tile[j + 1][i] = f.y;
    tile[j + 2][i] = f.z;
    tile[j + 3][i] = f.w;
  }
  __syncthreads();
  for (int e = threadIdx.x; e < 64 * 32; e += 256) {
    const int j = e >> 6, i = e & 63;
    if (m0 + i >= m || j0 + j >= r) continue;
    const Terms t = terms_of(tile[j][i]);
    __nv_bfloat16* dst = ut + (j0 + j) * ld + m0 + i;
    dst[0] = t.hi;
    dst[term] = t.mid;
    dst[2 * term] = t.lo;
  }
}

}  // namespace

qlora_status f8_grad_b(const void* dY, int64_t N, const float* U, int64_t M, int32_t r, float sc,
                       bool accumulate, void* ut, int64_t ld_u, float* dB, DeviceStatus* st,
                       cudaStream_t s) {
  const int32_t r16 = lora_rows(r);
  count_launch();
  const dim3 grid(static_cast<unsigned>(ceil_div(M, 64)), static_cast<unsigned>(ceil_div(r, 32)));
  terms_kernel<<<grid, 256, 0, s>>>(U, M, r, static_cast<__nv_bfloat16*>(ut), ld_u, ld_u * r16);
  QLORA_TRY(after_launch("f8_grad_b terms", s));
  GradBArgs p{};
  const int chunks = r16 > 128 ? 2 : 1;
  p.rc = static_cast<int32_t>(ceil_div(r16, 16 * chunks) * 16);
  CUtensorMap my, mu;
  if (!make_map(&my, dY, true, N, M, N, 64, 64, true) ||
      !make_map(&mu, ut, true, M, 2 * r16 + r, ld_u, 64, static_cast<uint32_t>(p.rc), true))
    return QLORA_ERR_CUDA;
  p.n = static_cast<int32_t>(N);
  p.r = r;
  p.term_rows = r16;
  p.dB = dB;
  p.sc = sc;
  p.idesc = ptx::idesc_bf16(128, p.rc, 1, 0);
  p.st = st;
  const void* kernel = reinterpret_cast<const void*>(f8_grad_b_kernel);
  const qlora_status cs = ensure_smem(kernel, kCtaMaxSmem);
  if (cs != QLORA_OK) return cs;
  // two CTAs an SM where two stages fit beside another's, else one; as many stages as do
  const int stage_bytes = kABytes + kTerms * p.rc * 128;
  const bool two = 2 * stage_bytes + kBesideBytes <= kCtaHalfSmem;
  p.stages =
      std::min(kMaxStages, ((two ? kCtaHalfSmem : kCtaMaxSmem) - kBesideBytes) / stage_bytes);
  p.area = std::max(p.stages * stage_bytes, 128 * (p.rc + 4) * 4);
  int max_accs = 1;
  while ((2 * max_accs + 1) * p.rc <= (two ? 256 : 512)) max_accs *= 2;
  const int64_t kt_total = ceil_div(M, 64), tiles = ceil_div(N, 128);
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 1;
  attr[0].val.clusterDim.y = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // One launch in n splits over `per` tiles each: its shared memory and grid.
  auto plan = [&](int n, int64_t per) {
    p.kt_per = static_cast<int32_t>(per);
    for (p.accs = 1; p.accs < max_accs && 4 * per > kChain * p.accs;) p.accs *= 2;
    for (p.tmem_cols = 32; p.tmem_cols < (p.accs + 1) * p.rc;) p.tmem_cols *= 2;
    cfg.dynamicSmemBytes = std::max(p.area + kBesideBytes, p.tmem_cols * kSmemPerColumn - 1024);
    attr[0].val.clusterDim.z = static_cast<unsigned>(n);
    cfg.gridDim = dim3(static_cast<unsigned>(tiles), chunks, n);
  };
  // At least 8 tiles a split: this launch runs beside dX's kernel, whose CTAs wait for whole
  // SMs (backward of 1024 x 4096 x 4096 at rank 16 in 1, 2 and 4 splits 37.6, 37.0 and 41.2 us,
  // at rank 64 41.1, 45.3 and 48.1; without dX 27.9, 23.3 and 22.3).  The costs, in us without
  // dX: 4096 tokens x 4096 at rank 64 in 2, 4 and 8 splits 51.6, 36.5 and 36.7, 8192 at rank
  // 16 59.6, 49.1 and 43.1, 4096 x 11008 at rank 64 in 2, 3 and 6 69.4, 55.2 and 61.8.
  int splits = 1;
  int64_t launches = 1;
  choose_splits(kernel, cfg, tiles * chunks, kt_total, 8, two, max_accs, SplitCost{17, 40, 6, 60},
                plan, &splits, &launches);
  const int64_t each = ceil_div(kt_total, launches);
  plan(splits, ceil_div(each, splits));
  for (int64_t kt0 = 0; kt0 < kt_total; kt0 += each) {
    p.kt0 = static_cast<int32_t>(kt0);
    p.kt_end = static_cast<int32_t>(std::min(kt_total, kt0 + each));
    p.accumulate = accumulate || kt0 > 0 ? 1 : 0;
    count_launch();
    timing_mark(QLORA_KERNEL_LORA_GEMM, s, true);
    const cudaError_t e = cudaLaunchKernelEx(&cfg, f8_grad_b_kernel, my, mu, p);
    timing_mark(QLORA_KERNEL_LORA_GEMM, s, false);
    if (e != cudaSuccess) {
      (void)cudaGetLastError();
      return QLORA_ERR_CUDA;
    }
    QLORA_TRY(after_launch("f8_grad_b", s));
  }
  return QLORA_OK;
}

}  // namespace qlora
