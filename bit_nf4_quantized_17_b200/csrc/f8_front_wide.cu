// The work of f8_front_kernel for many tokens: 8 bits of X by rows (definitions:
// f8_quantize.cu) and the LoRA factor U = X A^T (or V = dY B) from one read of X.
//
// A CTA takes 128 tokens and a share of the contraction: X and the factor's operand come
// by TMA in 64-column tiles (128-byte swizzle).  One thread multiplies them into several TMEM
// accumulators in turn (tcgen05.mma, N = the rank rounded up): sums there are cut off, not
// rounded, and shorter chains lose less (U of 2048 x 8192 at rank 64 against fp64: 3.2e-7,
// 1.4e-6 in one accumulator; 0.3 us).  Four (two above rank 128), more as far as TMEM goes
// where a chain were longer than 32 MMAs, and more splits where longer than 64 (16384 tokens x
// 22016 at rank 64: 8.9e-7, 6.0e-6 in four accumulators and one split).  Beside it two groups of four warps
// take the 128-column blocks in turn, a thread a row: the block's 64 words of X in
// registers give its scale and codes, which leave through shared memory and TMA stores.
// The shares are summed in distributed shared memory in order, as in gemm_rank.cu.  Every wait
// is bounded; one that gives up reports QLORA_ERR_DEVICE_TIMEOUT and leaves NaN in the factor
// of its tokens.
//
// Bound by latency within a block (load, maximum, encoding, store, two groups deep) and
// by the sum across the cluster: 19 us alone and cold for 2048 x 8192 at rank 64, 8 of
// them for its bytes.  Forward of the layer against the NF4 layer's rank product and the
// quantiser as two launches: 2048 x 8192 x 8192 in 140.5 us (145.6), 4096 x 4096 x 11008
// in 197 (214), 1024 x 4096 x 4096 at rank 16 in 28.4 (30.6).  Three groups that encode
// gain 0.2 to 1 us at ranks up to 64, where their code tiles fit.
#include <cudaTypedefs.h>

#include <algorithm>

#include "f8.cuh"
#include "f8_codec.cuh"
#include "tc_common.cuh"
#include "tc_ptx.cuh"

namespace qlora {
namespace {

constexpr int kThreads = 384;  // TMA, MMA, two idle warps; two groups of four that encode
constexpr int kXBytes = 16384;  // 128 rows x 64 bf16
constexpr int kCodeBytes = 16384;
constexpr int kMaxStages = 8;
constexpr int kStageBudget = 192 * 1024;
constexpr int kMaxSmem = 1024 + kStageBudget + 2 * kCodeBytes + 256;
constexpr int kChain = 32, kMaxChain = 64;  // MMAs into one accumulator: wanted, at most
constexpr long long kTimeoutCycles = 4000000000ll;

struct WideArgs {
  int32_t m, kt_total, k_tiles;  // tokens; 64-column tiles, tiles per split (even)
  int32_t b_mn, bn;              // operand of the factor MN-major; MMA N
  int32_t b_bytes, stage_bytes, stages, red_ld, area;
  int32_t accs, acc_cols;        // accumulators, TMEM columns of one (powers of two)
  int32_t encode;                // 0: U alone
  float* scales;                 // [kb][m]
  int32_t pow2, r, span;
  float* u;                      // m x r or NULL
  __nv_bfloat16* su;             // m x [span | span]
  float sc;
  __nv_bfloat16* ut;             // three terms, ut_lo rows apart, or NULL
  int64_t ut_ld;
  int32_t ut_lo;
  DeviceStatus* st;
};

__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr));
  return v;
}

__device__ __forceinline__ void sync_group(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

__device__ __forceinline__ float word_value(uint32_t w, int half) {
  return __uint_as_float(half ? (w & 0xffff0000u) : (w << 16));
}

// 64 columns of a row of a tile: chunk c of 16 bytes lies at c ^ (row mod 8)
__device__ __forceinline__ void load_row(const uint8_t* tile, int row, uint32_t (&w)[32]) {
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    const uint4 v =
        *reinterpret_cast<const uint4*>(tile + row * 128 + ((c ^ (row & 7)) << 4));
    w[4 * c] = v.x;
    w[4 * c + 1] = v.y;
    w[4 * c + 2] = v.z;
    w[4 * c + 3] = v.w;
  }
}

// codes of 64 columns, chunks c0 .. c0 + 3 of the row of a code tile
template <bool E5M2>
__device__ __forceinline__ void store_codes(uint8_t* tile, int row, int c0, float inv,
                                            const uint32_t (&w)[32]) {
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    uint32_t o[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint32_t w0 = w[8 * c + 2 * q], w1 = w[8 * c + 2 * q + 1];
      o[q] = encode4<E5M2>(word_value(w0, 0), word_value(w0, 1), word_value(w1, 0),
                           word_value(w1, 1), inv);
    }
    *reinterpret_cast<uint4*>(tile + row * 128 + (((c0 + c) ^ (row & 7)) << 4)) =
        make_uint4(o[0], o[1], o[2], o[3]);
  }
}

template <bool E5M2>
__global__ void __launch_bounds__(kThreads, 1)
f8_front_wide_kernel(const __grid_constant__ CUtensorMap tmX,
                     const __grid_constant__ CUtensorMap tmB,
                     const __grid_constant__ CUtensorMap tmC, const WideArgs p) {
  // the product may start: it reads what this launch writes after its own wait
  ptx::grid_launch_dependents();
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  // [stages x (X | B)], reused as the fp32 partial tile once all of them are read
  float* red = reinterpret_cast<float*>(smem);
  uint8_t* codes = smem + p.area;  // a tile per group
  uint64_t* full = reinterpret_cast<uint64_t*>(codes + 2 * kCodeBytes);
  uint64_t* empty = full + kMaxStages;
  uint64_t* accum = empty + kMaxStages;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(accum + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t S = gridDim.z, z = blockIdx.z;  // the cluster spans z
  const int m0 = blockIdx.x * 128;
  const int kt0 = static_cast<int>(z) * p.k_tiles;
  const int kn = max(0, min(p.k_tiles, p.kt_total - kt0));

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      ptx::mbar_init(&full[s], 1);
      ptx::mbar_init(&empty[s], p.encode ? 5 : 1);  // the MMAs, and four warps that encode
    }
    ptx::mbar_init(accum, 1);
    *abort_flag = 0;
    ptx::fence_mbar_init();
    ptx::prefetch_tmap(&tmX);
    ptx::prefetch_tmap(&tmB);
    ptx::prefetch_tmap(&tmC);
  }
  if (warp == 1) {
    ptx::tmem_alloc(tmem_slot, p.accs * p.acc_cols);
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
    uint8_t* sx = smem;
    for (int k = kt0 * 64, i = 0; i < kn; ++i, k += 64) {
      if (!ptx::mbar_wait(&empty[s], ph, kTimeoutCycles, abort_flag)) break;
      ptx::mbar_arrive_expect_tx(&full[s], kXBytes + p.b_bytes);
      ptx::tma_load_2d(&tmX, &full[s], sx, k, m0);
      if (p.b_mn) {
        for (int h = 0; h < p.bn; h += 64)
          ptx::tma_load_2d(&tmB, &full[s], sx + kXBytes + h * 128, h, k);
      } else {
        ptx::tma_load_2d(&tmB, &full[s], sx + kXBytes, k, 0);
      }
      ++issued;
      sx += p.stage_bytes;
      if (++s == p.stages) {
        s = 0;
        ph ^= 1;
        sx = smem;
      }
    }
    // never leave with copies in flight into this CTA's shared memory
    for (int i = (issued > p.stages ? issued - p.stages : 0); i < issued; ++i)
      ptx::mbar_wait(&full[i % p.stages], (i / p.stages) & 1, kTimeoutCycles, nullptr);
  } else if (warp == 1 && ptx::elect_one()) {
    // ------------------------------------------------------ MMA issuer
    const uint32_t idesc = ptx::idesc_bf16(128, p.bn, 0, p.b_mn);
    const uint32_t x_addr = ptx::smem_u32(smem);
    const uint64_t x0 = ptx::sw128_desc(x_addr, 16, 1024);
    const uint64_t b0 = ptx::sw128_desc(x_addr + kXBytes, p.b_mn ? 8192 : 16, 1024);
    const uint64_t bs = p.b_mn ? (2048 >> 4) : (32 >> 4);
    int s = 0;
    uint32_t ph = 0;
    uint64_t off = 0;
    for (int i = 0; i < kn; ++i) {
      if (!ptx::mbar_wait(&full[s], ph, kTimeoutCycles, abort_flag)) break;
      ptx::tc_fence_after();
      const uint64_t xd = x0 + off, bd = b0 + off;
      const uint32_t d = tmem + (i & (p.accs - 1)) * p.acc_cols;
      ptx::umma_bf16(d, xd, bd, idesc, i >= p.accs ? 1u : 0u);
      ptx::umma_bf16(d, xd + (32 >> 4), bd + bs, idesc, 1u);
      ptx::umma_bf16(d, xd + 2 * (32 >> 4), bd + 2 * bs, idesc, 1u);
      ptx::umma_bf16(d, xd + 3 * (32 >> 4), bd + 3 * bs, idesc, 1u);
      ptx::umma_commit(&empty[s]);
      off += p.stage_bytes >> 4;
      if (++s == p.stages) {
        s = 0;
        ph ^= 1;
        off = 0;
      }
    }
    ptx::umma_commit(accum);
    ptx::mbar_wait(accum, 0, kTimeoutCycles, nullptr);  // MMAs done before TMEM is freed
  } else if (warp >= 4) {
    // ------------------------------------------------------ 8 bits of X
    const int group = (warp - 4) >> 2, quarter = warp & 3;
    const int row = 32 * quarter + lane;
    const bool leader = quarter == 0 && lane == 0;
    uint8_t* out = codes + group * kCodeBytes;
    int s = 0;
    uint32_t ph = 0;
    bool ok = true;
    auto step = [&]() {
      if (++s == p.stages) {
        s = 0;
        ph ^= 1;
      }
    };
    // A wait that gives up sets the flag that ends all others; the loop runs on, so that
    // the group's barriers stay in step.
    auto take = [&](uint32_t (&w)[32]) {
      ok = ptx::mbar_wait(&full[s], ph, kTimeoutCycles, abort_flag) && ok;
      load_row(smem + s * p.stage_bytes, row, w);
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&empty[s]);
      step();
    };
    if (group == 1) {
      step();
      step();
    }
    for (int i = 2 * group; p.encode && i < kn; i += 4) {
      uint32_t w0[32], w1[32];
      take(w0);
      float a = amax_words<__nv_bfloat16>(w0);
      if (i + 1 < kn) {
        take(w1);
        a = fmaxf(a, amax_words<__nv_bfloat16>(w1));
      } else {
#pragma unroll
        for (int j = 0; j < 32; ++j) w1[j] = 0u;
      }
      step();  // the other group's block
      step();
      const int kb = (kt0 + i) >> 1;
      const float sc = block_scale_of(a, E5M2, p.pow2 != 0);
      const float inv = __fdiv_rn(1.0f, sc);
      if (m0 + row < p.m) p.scales[static_cast<int64_t>(kb) * p.m + m0 + row] = sc;
      if (leader) ptx::bulk_wait_read();  // the store before has read the tile
      sync_group(1 + group, 128);
      store_codes<E5M2>(out, row, 0, inv, w0);
      store_codes<E5M2>(out, row, 4, inv, w1);
      ptx::fence_proxy_async_smem();
      sync_group(1 + group, 128);
      if (leader && ok) {
        ptx::tma_store_2d(&tmC, out, kb * 128, m0);
        ptx::bulk_commit();
      }
    }
    if (leader) ptx::bulk_wait_all();
    // -------------------------------------------- partial tile -> shared memory
    sync_group(3, 256);  // every tile of X has been read
    ok = kn > 0 && ptx::mbar_wait(accum, 0, kTimeoutCycles, abort_flag);
    ok = __all_sync(0xffffffffu, ok && !*abort_flag);
    if (ok) ptx::tc_fence_after();
    for (int c = group; c < p.bn / 16; c += 2) {
      float v[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) v[j] = 0.0f;
      for (int a = 0; ok && a < min(p.accs, kn); ++a) {
        uint32_t r[16];
        ptx::tmem_ld_x16(tmem + (static_cast<uint32_t>(32 * quarter) << 16) + a * p.acc_cols +
                             16 * c, r);
        ptx::tmem_ld_wait(r);
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] += __uint_as_float(r[j]);
      }
      float* dst = red + static_cast<size_t>(row) * p.red_ld + 16 * c;
#pragma unroll
      for (int j = 0; j < 16; j += 4)
        *reinterpret_cast<float4*>(dst + j) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  // a wait of this CTA gave up: its sums are not whole (the status word may not be read)
  if (*abort_flag)
    for (int e = threadIdx.x; e < 128 * p.red_ld; e += kThreads)
      red[e] = __int_as_float(0x7fffffff);
  ptx::cluster_sync();

  // --------------------------- sum over the splits, in order, and store
  if (warp >= 4) {
    const int slice = (128 + static_cast<int>(S) - 1) / static_cast<int>(S);
    const int i0 = static_cast<int>(z) * slice;
    const int rows = max(0, min(min(slice, 128 - i0), p.m - m0 - i0));
    const int quads = p.span >> 2;
    uint32_t peer[8];
#pragma unroll
    for (int q = 0; q < 8; ++q)
      peer[q] = q < static_cast<int>(S) ? ptx::cluster_addr(red, static_cast<uint32_t>(q)) : 0u;
    for (int e = threadIdx.x - 128; e < rows * quads; e += 256) {
      const int i = i0 + e / quads, j = 4 * (e - (e / quads) * quads);
      const int64_t row = m0 + i;
      float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      if (j < p.r) {  // r is a multiple of 8; columns past it are zero
        const uint32_t off = static_cast<uint32_t>((i * p.red_ld + j) * 4);
        float4 h[8];
#pragma unroll
        for (int q = 0; q < 8; ++q)
          if (q < static_cast<int>(S)) h[q] = ld_cluster_f32x4(peer[q] + off);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          if (q < static_cast<int>(S)) {
            v[0] += h[q].x;
            v[1] += h[q].y;
            v[2] += h[q].z;
            v[3] += h[q].w;
          }
        }
        if (p.u)
          *reinterpret_cast<float4*>(p.u + row * p.r + j) = make_float4(v[0], v[1], v[2], v[3]);
        if (p.ut) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const Terms t = terms_of(v[q]);
            p.ut[(j + q) * p.ut_ld + row] = t.hi;
            p.ut[(p.ut_lo + j + q) * p.ut_ld + row] = t.mid;
            p.ut[(2 * p.ut_lo + j + q) * p.ut_ld + row] = t.lo;
          }
        }
      }
      uint32_t hi[2], lo[2];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const float f0 = p.sc * v[2 * q], f1 = p.sc * v[2 * q + 1];
        const __nv_bfloat162 hh = __floats2bfloat162_rn(f0, f1);
        const __nv_bfloat162 ll =
            __floats2bfloat162_rn(f0 - __low2float(hh), f1 - __high2float(hh));
        hi[q] = *reinterpret_cast<const uint32_t*>(&hh);
        lo[q] = *reinterpret_cast<const uint32_t*>(&ll);
      }
      __nv_bfloat16* o = p.su + row * 2 * p.span + j;
      *reinterpret_cast<uint2*>(o) = make_uint2(hi[0], hi[1]);
      *reinterpret_cast<uint2*>(o + p.span) = make_uint2(lo[0], lo[1]);
    }
  }
  // no CTA leaves (or frees TMEM) while the others may still read its tile
  __syncthreads();
  ptx::cluster_sync();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, p.accs * p.acc_cols);
  }
  if (threadIdx.x == 0 && *abort_flag) report(p.st, QLORA_ERR_DEVICE_TIMEOUT, 150u);
}

}  // namespace

qlora_status f8_front_wide(const FrontOp& f, const qlora_f8& x8, DeviceStatus* st,
                           cudaStream_t s) {
  const int64_t M = x8.rows, K = x8.cols;
  if (M < 1 || K % 8 != 0 || f.r % 8 != 0 || f.r > 256) return QLORA_ERR_UNSUPPORTED;
  const int64_t m_tiles = ceil_div(M, 128);
  WideArgs p{};
  p.m = static_cast<int32_t>(M);
  p.kt_total = static_cast<int32_t>(ceil_div(K, 64));
  p.b_mn = f.along ? 1 : 0;
  p.span = lora_span(f.r);
  p.bn = f.along ? p.span : lora_rows(f.r);
  p.b_bytes = p.bn * 128;
  p.stage_bytes = kXBytes + p.b_bytes;
  // a multiple of 4, so that a stage's tiles all go to the same group: it has seen every
  // phase of the barriers that it waits on
  p.stages = kMaxStages * p.stage_bytes <= kStageBudget ? kMaxStages : 4;
  p.acc_cols = 32;
  while (p.acc_cols < p.bn) p.acc_cols *= 2;
  const int max_accs = 512 / p.acc_cols;
  p.red_ld = p.bn + 4;
  p.area = static_cast<int32_t>(
      ceil_div(std::max(p.stages * p.stage_bytes, 128 * p.red_ld * 4), 1024) * 1024);
  p.encode = f.encode ? 1 : 0;
  p.scales = x8.scales;
  p.pow2 = x8.pow2;
  p.r = f.r;
  p.u = f.u;
  p.su = static_cast<__nv_bfloat16*>(f.su);
  p.sc = f.sc;
  p.ut = static_cast<__nv_bfloat16*>(f.ut);
  p.ut_ld = f.ut_ld;
  p.ut_lo = f.ut_lo;
  p.st = st;
  CUtensorMap mx, mb, mc;
  bool ok = make_map(&mx, f.x, true, K, M, K, 64, 128, true) &&
            (f.along ? make_map(&mb, f.a, true, f.r, K, f.r, 64, 64, true)
                     : make_map(&mb, f.a, true, K, f.r, K, 64, static_cast<uint32_t>(p.bn), true));
  mc = mx;
  // zeros up to the next multiple of 16 columns
  if (f.encode)
    ok = ok && make_map(&mc, x8.codes, false, ceil_div(K, 16) * 16, M, x8.ld, 128, 128, true);
  if (!ok) return QLORA_ERR_CUDA;
  const bool e5 = x8.format == QLORA_E5M2;
  const void* fn = e5 ? reinterpret_cast<const void*>(f8_front_wide_kernel<true>)
                      : reinterpret_cast<const void*>(f8_front_wide_kernel<false>);
  const qlora_status cs = ensure_smem(fn, kMaxSmem);
  if (cs != QLORA_OK) return cs;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 1;
  attr[0].val.clusterDim.y = 1;
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = 1024 + p.area + 2 * kCodeBytes + 256;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // as many splits as run at once, at least 4 blocks each
  const int64_t kbs = f8_blocks(K);
  const int sms = f8::sm_count();
  int splits = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({8, sms / m_tiles, kbs / 4})));
  // no fewer than keep a chain at kMaxChain MMAs, four a tile
  const int least = static_cast<int>(
      std::min<int64_t>(8, ceil_div(p.kt_total, kMaxChain / 4 * max_accs)));
  for (splits = std::max(splits, least);; --splits) {
    attr[0].val.clusterDim.z = static_cast<unsigned>(splits);
    cfg.gridDim = dim3(static_cast<unsigned>(m_tiles), 1u, static_cast<unsigned>(splits));
    if (splits == least || m_tiles <= f8_resident_clusters(fn, cfg)) break;
  }
  p.k_tiles = 2 * static_cast<int32_t>(ceil_div(kbs, splits));
  for (p.accs = std::min(4, max_accs); p.accs < max_accs && 4 * p.k_tiles > kChain * p.accs;)
    p.accs *= 2;
  void* args[] = {&mx, &mb, &mc, &p};
  count_launch();
  const int kind = f.encode ? QLORA_KERNEL_QUANTIZE : QLORA_KERNEL_LORA_GEMM;
  timing_mark(kind, s, true);
  const cudaError_t e = cudaLaunchKernelExC(&cfg, fn, args);
  timing_mark(kind, s, false);
  if (e != cudaSuccess) {
    (void)cudaGetLastError();
    return QLORA_ERR_CUDA;
  }
  return after_launch("f8_front_wide", s);
}

}  // namespace qlora
