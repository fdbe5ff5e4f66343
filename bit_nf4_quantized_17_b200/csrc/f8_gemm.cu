// Matrix product in 8-bit floating point with a scale for each block of 128.
//
//   C[m][n] = sum_kb sA[kb][m] sB[kb, n / 128] sum_{k in block kb} a[m][k] b[n][k]
//             (+ sum_j L[m][j] R[n][j], the LoRA term)
// A is held by rows (a scale per row and 128 contraction elements), B by tiles
// (a scale per 128 x 128).  The scales change along the contraction, so a
// block's product is not added to the next one's on the tensor core: each
// 128-deep block goes into a TMEM accumulator of its own (4 MMAs of kind
// f8f6f4), and the epilogue warps add it, times its scales, to fp32 sums in
// registers while the tensor core works on the next block.
//
// One CTA computes a 128 x BN tile from a 128-row operand P and a BN-row
// operand Q; both roles can be played by A and B:
//   * P = A, Q = B (BN = 128): thread = output row, one scale per thread and block;
//   * SWAP, for few tokens: P = B, Q = A (BN = 16, 32, 64): the 128 rows of the
//     MMA are output columns, no MMA row is wasted on tokens that do not exist,
//     and B, whose bytes bound the product, is read once.  A thread holds one
//     output column and all BN tokens; the tokens' scales live one per lane and
//     are passed round by shuffles.
// B is read in place in both directions of the layer: K-major (C = A B^T) or
// MN-major (C = A B).
// Where the tiles would leave SMs idle the contraction is split over the CTAs
// of a cluster (up to 8) and the fp32 partial tiles are summed in distributed
// shared memory in split order (deterministic).
//
// Roles: warp 0 TMA producer, warp 1 TMEM owner and MMA issuer, the other 4 or
// 8 warps drain the accumulators.  Every wait is bounded; the call has no
// status word, so a CTA whose wait gives up writes NaN to its part.
#include <cudaTypedefs.h>

#include <algorithm>

#include "f8_gemm.cuh"

namespace qlora {
namespace {

using f8::GemmArgs;
using f8::kTimeoutCycles;
using f8::store_run;

constexpr int kPBytes = 16384;                      // 128 rows x 128 bytes
constexpr int kMaxStages = 12;

__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr));
  return v;
}

template <int BN, bool SWAP>
struct Cfg {
  static constexpr int kEpi = BN >= 128 ? 8 : 4;  // epilogue warps
  static constexpr int kThreads = 64 + 32 * kEpi;
  static constexpr int kCols = BN / (kEpi / 4);   // accumulator columns per thread
  static constexpr int kBufs = BN >= 128 ? 2 : 4; // TMEM accumulators in flight
  static constexpr int kTmem = BN * kBufs;        // 64, 128 or 256 columns
  static constexpr int kQBytes = BN * 128;
  static constexpr int kStage = kPBytes + kQBytes;
  // fp32 partial tile: rows of tokens, padded against bank conflicts
  static constexpr int kRedLd = SWAP ? 128 + 4 : BN + 4;
  static constexpr int kRedBytes = (SWAP ? BN : 128) * kRedLd * 4;
};

template <int BN, bool SWAP>
__global__ void __launch_bounds__(Cfg<BN, SWAP>::kThreads, 1)
f8_gemm_kernel(const __grid_constant__ CUtensorMap tmP, const __grid_constant__ CUtensorMap tmQ,
               const __grid_constant__ CUtensorMap tmP2, const __grid_constant__ CUtensorMap tmQ2,
               const GemmArgs p) {
  using C = Cfg<BN, SWAP>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  // [stages x (P | Q)], reused as the fp32 partial tile once every MMA is done
  const int area = max(p.stages * C::kStage, C::kRedBytes);
  float* red = reinterpret_cast<float*>(smem);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + area);
  uint64_t* empty = full + kMaxStages;
  uint64_t* acc_full = empty + kMaxStages;
  uint64_t* acc_empty = acc_full + C::kBufs;
  uint64_t* drain = acc_empty + C::kBufs;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t S = gridDim.z, z = blockIdx.z;  // the cluster spans z
  // tile of P (128 rows) and of Q (BN rows)
  const int qt = SWAP ? blockIdx.x / p.n_tiles : blockIdx.x % p.n_tiles;
  const int pt = SWAP ? blockIdx.x % p.n_tiles : blockIdx.x / p.n_tiles;
  const int p0 = pt * 128, q0 = qt * BN;
  const int kb0 = static_cast<int>(z) * p.kb_per;
  const int kn = max(0, min(p.kb_per, p.kb_total - kb0));
  // the LoRA stages belong to the last split
  const int ext = (z == S - 1) ? p.ext_tiles : 0;
  const int total = kn + ext;
  const int bufs_used = kn + (ext ? 1 : 0);  // accumulators drained, in order
  const bool p_mn = SWAP && p.b_mn, q_mn = !SWAP && p.b_mn;
  const bool p2_mn = SWAP && p.ext_mn, q2_mn = !SWAP && p.ext_mn;

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      ptx::mbar_init(&full[s], 1);
      ptx::mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < C::kBufs; ++b) {
      ptx::mbar_init(&acc_full[b], 1);
      ptx::mbar_init(&acc_empty[b], C::kEpi);
    }
    ptx::mbar_init(drain, 1);
    *abort_flag = 0;
    ptx::fence_mbar_init();
    ptx::prefetch_tmap(&tmP);
    ptx::prefetch_tmap(&tmQ);
  }
  if (warp == 1) {
    ptx::tmem_alloc(tmem_slot, C::kTmem);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  float acc[C::kCols];
#pragma unroll
  for (int j = 0; j < C::kCols; ++j) acc[j] = 0.0f;
  // TMEM lanes of a warp are those of its number mod 4
  const int quarter = warp & 3;
  const int half = (warp - 2) >> 2;  // column half of an 8-warp epilogue
  bool ok = true;

  if (warp == 0 && lane == 0) {
    // ------------------------------------------------------ TMA producer
    int issued = 0;
    for (int i = 0; i < total; ++i) {
      const int s = i % p.stages;
      if (!ptx::mbar_wait(&empty[s], ((i / p.stages) & 1) ^ 1, kTimeoutCycles, abort_flag)) break;
      uint8_t* sp = smem + s * C::kStage;
      uint8_t* sq = sp + kPBytes;
      ptx::mbar_arrive_expect_tx(&full[s], C::kStage);
      if (i < kn) {
        const int k = (kb0 + i) * 128;
        if (p_mn)
          ptx::tma_load_2d(&tmP, &full[s], sp, p0, k);
        else
          ptx::tma_load_2d(&tmP, &full[s], sp, k, p0);
        if (q_mn)
          ptx::tma_load_2d(&tmQ, &full[s], sq, q0, k);
        else
          ptx::tma_load_2d(&tmQ, &full[s], sq, k, q0);
      } else {
        // L columns [64 t, 64 t + 64) of [hi | lo], R at ranks 64 (t mod half)
        const int t = i - kn;
        const int kl = t * 64, kr = (t % p.ext_half) * 64;
        if (SWAP) {
          if (p2_mn) {
            ptx::tma_load_2d(&tmP2, &full[s], sp, p0, kr);
            ptx::tma_load_2d(&tmP2, &full[s], sp + 8192, p0 + 64, kr);
          } else {
            ptx::tma_load_2d(&tmP2, &full[s], sp, kr, p0);
          }
          ptx::tma_load_2d(&tmQ2, &full[s], sq, kl, q0);
        } else {
          ptx::tma_load_2d(&tmP2, &full[s], sp, kl, p0);
          if (q2_mn) {
#pragma unroll
            for (int h = 0; h < (BN + 63) / 64; ++h)
              ptx::tma_load_2d(&tmQ2, &full[s], sq + 8192 * h, q0 + 64 * h, kr);
          } else {
            ptx::tma_load_2d(&tmQ2, &full[s], sq, kr, q0);
          }
        }
      }
      ++issued;
    }
    // never leave with copies in flight into this CTA's shared memory
    for (int i = (issued > p.stages ? issued - p.stages : 0); i < issued; ++i)
      ptx::mbar_wait(&full[i % p.stages], (i / p.stages) & 1, kTimeoutCycles, nullptr);
  } else if (warp == 1 && lane == 0) {
    // ------------------------------------------------------ MMA issuer
    int i = 0;
    for (; i < total; ++i) {
      const int s = i % p.stages;
      const int t = i - kn;             // LoRA stage, when >= 0
      const int u = t > 0 ? kn : i;     // accumulator use: all LoRA stages share one
      const int b = u % C::kBufs;
      if (t <= 0 && !ptx::mbar_wait(&acc_empty[b], ((u / C::kBufs) & 1) ^ 1, kTimeoutCycles,
                                    abort_flag))
        break;
      if (!ptx::mbar_wait(&full[s], (i / p.stages) & 1, kTimeoutCycles, abort_flag)) break;
      ptx::tc_fence_after();
      const uint32_t p_addr = ptx::smem_u32(smem + s * C::kStage);
      const uint32_t q_addr = p_addr + kPBytes;
      const uint32_t d = tmem + b * BN;
      if (t < 0) {
        // MN-major 8-bit tiles: 128 contraction rows of 128 bytes, 32 rows a step
        const uint64_t pd = ptx::sw128_desc(p_addr, p_mn ? kPBytes : 16, 1024);
        const uint64_t qd = ptx::sw128_desc(q_addr, q_mn ? kPBytes : 16, 1024);
        const uint64_t ps = p_mn ? (4096 >> 4) : (32 >> 4);
        const uint64_t qs = q_mn ? (4096 >> 4) : (32 >> 4);
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
          ptx::umma_f8(d, pd + ps * ks, qd + qs * ks, p.idesc, ks ? 1u : 0u);
      } else {
        const uint64_t pd = ptx::sw128_desc(p_addr, p2_mn ? 8192 : 16, 1024);
        const uint64_t qd = ptx::sw128_desc(q_addr, q2_mn ? 8192 : 16, 1024);
        const uint64_t ps = p2_mn ? (2048 >> 4) : (32 >> 4);
        const uint64_t qs = q2_mn ? (2048 >> 4) : (32 >> 4);
        const int steps = (t % p.ext_half) == p.ext_half - 1 ? p.ext_last_steps : 4;
        for (int ks = 0; ks < steps; ++ks)
          ptx::umma_bf16(d, pd + ps * ks, qd + qs * ks, p.idesc_ext, (t | ks) != 0 ? 1u : 0u);
      }
      ptx::umma_commit(&empty[s]);
      if (t < 0 || i == total - 1) ptx::umma_commit(&acc_full[b]);
    }
    if (i < total) {
      // gave up: what was issued is done before shared memory and TMEM go
      ptx::umma_commit(drain);
      ptx::mbar_wait(drain, 0, kTimeoutCycles, nullptr);
    }
  } else if (warp >= 2) {
    // ------------------------------------------------------ epilogue warps
    const uint32_t lane_base = static_cast<uint32_t>(32 * quarter) << 16;
    const int row = 32 * quarter + lane;  // row of the P tile
    // scales of block i of this split: SWAP keeps token q0 + lane (+ 32) per
    // lane, otherwise the thread's own row; times B's scale of the tile
    constexpr int kSc = SWAP ? (BN + 31) / 32 : 1;
    const float* sb = p.sb + static_cast<int64_t>((SWAP ? p0 : q0) >> 7) * p.sb_n;
    auto scale_of = [&](int i, float (&sv)[kSc]) {
      if (i >= kn) return;
      const int64_t kb = kb0 + i;
      const float w = __ldg(sb + kb * p.sb_k);
#pragma unroll
      for (int h = 0; h < kSc; ++h) {
        const int tok = SWAP ? q0 + 32 * h + lane : p0 + row;
        sv[h] = tok < p.m ? __ldg(p.sa + kb * p.m + tok) * w : 0.0f;
      }
    };
    constexpr int kAhead = 4;  // blocks whose scales are on their way
    float sv[kAhead][kSc];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) scale_of(u, sv[u]);
    for (int i0 = 0; i0 < bufs_used && ok; i0 += kAhead) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int i = i0 + u;
        if (i < bufs_used && ok) {
          const int b = i % C::kBufs;
          ok = ptx::mbar_wait(&acc_full[b], (i / C::kBufs) & 1, kTimeoutCycles, abort_flag);
          ok = __all_sync(0xffffffffu, ok);
          if (ok) {
            ptx::tc_fence_after();
            const uint32_t at = tmem + lane_base + b * BN + half * C::kCols;
            const bool lora = i == kn;
            uint32_t r[2][16];
            ptx::tmem_ld_x16(at, r[0]);
#pragma unroll
            for (int c = 0; c < C::kCols / 16; ++c) {
              ptx::tmem_ld_wait(r[c & 1]);
              if (c + 1 < C::kCols / 16) ptx::tmem_ld_x16(at + 16 * (c + 1), r[(c + 1) & 1]);
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                float s;
                if (SWAP)
                  s = __shfl_sync(0xffffffffu, sv[u][(16 * c + j) / 32], (16 * c + j) & 31);
                else
                  s = sv[u][0];
                if (lora) s = 1.0f;
                acc[16 * c + j] = fmaf(__uint_as_float(r[c & 1][j]), s, acc[16 * c + j]);
              }
            }
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&acc_empty[b]);
            scale_of(i + kAhead, sv[u]);
          }
        }
      }
    }
    ok = __all_sync(0xffffffffu, ok && !*abort_flag);
    if (!ok) {
#pragma unroll
      for (int j = 0; j < C::kCols; ++j) acc[j] = __int_as_float(0x7fffffff);
    }
    if (S == 1) {
      if (SWAP) {
        const int64_t col = static_cast<int64_t>(p0) + row;
#pragma unroll
        for (int j = 0; j < C::kCols; ++j) {
          const int64_t tok = static_cast<int64_t>(q0) + j;
          if (col < p.n && tok < p.m) {
            if (p.c_f32)
              static_cast<float*>(p.c)[tok * p.c_ld + col] = acc[j];
            else
              static_cast<__nv_bfloat16*>(p.c)[tok * p.c_ld + col] = __float2bfloat16_rn(acc[j]);
          }
        }
      } else {
#pragma unroll
        for (int c = 0; c < C::kCols / 16; ++c)
          store_run<16>(p, static_cast<int64_t>(p0) + row,
                        static_cast<int64_t>(q0) + half * C::kCols + 16 * c, acc + 16 * c);
      }
    }
  }
  if (S > 1) {
    // ---------------- partial tiles to shared memory, summed in split order
    // the stages are reused: the last block's wait above says that every MMA of
    // this CTA has read them, and the producer that every copy has landed
    ptx::tc_fence_before();
    __syncthreads();
    if (warp >= 2) {
      const int row = 32 * quarter + lane;
      if (SWAP) {
#pragma unroll
        for (int j = 0; j < C::kCols; ++j) red[j * C::kRedLd + row] = acc[j];
      } else {
#pragma unroll
        for (int j = 0; j < C::kCols; j += 4)
          *reinterpret_cast<float4*>(red + row * C::kRedLd + half * C::kCols + j) =
              make_float4(acc[j], acc[j + 1], acc[j + 2], acc[j + 3]);
      }
    }
    __syncthreads();
    ptx::cluster_sync();
    // runs of 4 consecutive columns of C, dealt to the CTAs of the cluster
    constexpr int kRuns = 128 * BN / 4, kPerRow = (SWAP ? 128 : BN) / 4;
    for (int e = static_cast<int>(z) * C::kThreads + threadIdx.x; e < kRuns;
         e += static_cast<int>(S) * C::kThreads) {
      const int tr = e / kPerRow, cc = (e % kPerRow) * 4;
      const int64_t tok = static_cast<int64_t>(SWAP ? q0 : p0) + tr;
      if (tok >= p.m) continue;
      const uint32_t off = static_cast<uint32_t>(tr * C::kRedLd + cc) * 4u;
      float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (uint32_t q = 0; q < 8; ++q) {
        if (q < S) {
          const float4 f = ld_cluster_f32x4(ptx::cluster_addr(red, q) + off);
          v[0] += f.x;
          v[1] += f.y;
          v[2] += f.z;
          v[3] += f.w;
        }
      }
      store_run<4>(p, tok, static_cast<int64_t>(SWAP ? p0 : q0) + cc, v);
    }
    // no CTA leaves while the others may still read its tile
    __syncthreads();
    ptx::cluster_sync();
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, C::kTmem);
  }
}

template <int BN, bool SWAP>
qlora_status launch(const qlora_f8& a, const qlora_f8& b, bool trans_b, GemmArgs p,
                    const F8Lora& l, int splits, cudaStream_t s) {
  using C = Cfg<BN, SWAP>;
  const int64_t m = p.m, n = p.n;
  CUtensorMap ma, mb, ml, mr;
  const uint32_t a_rows = SWAP ? BN : 128, b_rows = SWAP ? 128 : BN;
  bool ok = make_map(&ma, a.codes, false, a.cols, m, a.ld, 128, a_rows, true) &&
            (trans_b ? make_map(&mb, b.codes, false, b.cols, n, b.ld, 128, b_rows, true)
                     : make_map(&mb, b.codes, false, n, b.rows, b.ld, 128, 128, true));
  if (l.r > 0) {
    const int64_t ld = 2 * lora_span(l.r);
    ok = ok && make_map(&ml, l.L, true, ld, m, ld, 64, a_rows, true) &&
         (p.ext_mn ? make_map(&mr, l.R, true, n, l.r, n, 64, 64, true)
                   : make_map(&mr, l.R, true, l.r, n, l.r, 64, b_rows, true));
  } else {
    ml = ma;
    mr = mb;
  }
  if (!ok) return QLORA_ERR_CUDA;
  const int fa = a.format == QLORA_E5M2 ? 1 : 0, fb = b.format == QLORA_E5M2 ? 1 : 0;
  p.idesc = SWAP ? ptx::idesc_f8(fb, fa, 128, BN, p.b_mn, 0)
                 : ptx::idesc_f8(fa, fb, 128, BN, 0, p.b_mn);
  p.idesc_ext = SWAP ? ptx::idesc_bf16(128, BN, p.ext_mn, 0)
                     : ptx::idesc_bf16(128, BN, 0, p.ext_mn);
  p.kb_per = static_cast<int32_t>(ceil_div(p.kb_total, splits));
  // the stages that fit; no more than a split has blocks
  const int64_t want = p.kb_per + p.ext_tiles;
  p.stages = static_cast<int32_t>(
      std::min<int64_t>({kMaxStages, want, (200 * 1024) / C::kStage}));
  const int64_t p_tiles = ceil_div(SWAP ? n : m, 128), q_tiles = ceil_div(SWAP ? m : n, BN);
  p.n_tiles = static_cast<int32_t>(SWAP ? p_tiles : q_tiles);
  if (p_tiles * q_tiles > 0x7fffffff) return QLORA_ERR_SHAPE;
  const void* fn = reinterpret_cast<const void*>(f8_gemm_kernel<BN, SWAP>);
  const qlora_status cs = ensure_smem(fn, 220 * 1024);
  if (cs != QLORA_OK) return cs;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p_tiles * q_tiles), 1, static_cast<unsigned>(splits));
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = 1024 + std::max(p.stages * C::kStage, C::kRedBytes) + 512;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 1;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = static_cast<unsigned>(splits);
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  count_launch();
  const cudaError_t e = cudaLaunchKernelEx(&cfg, f8_gemm_kernel<BN, SWAP>, SWAP ? mb : ma,
                                           SWAP ? ma : mb, SWAP ? mr : ml, SWAP ? ml : mr, p);
  if (e != cudaSuccess) {
    (void)cudaGetLastError();
    return QLORA_ERR_CUDA;
  }
  return after_launch("f8_gemm", s);
}

// Contraction splits for `tiles` output tiles: as many CTAs as there are SMs,
// a cluster of at most 8, at least 4 blocks each.
int split_count(int64_t tiles, int64_t kb) {
  int dev = 0, sms = 148;
  if (cudaGetDevice(&dev) == cudaSuccess)
    (void)cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  const int64_t s = std::min<int64_t>({8, sms / tiles, kb / 4});
  return static_cast<int>(std::max<int64_t>(1, s));
}

}  // namespace

f8::GemmArgs f8::gemm_args(const qlora_f8& a, const qlora_f8& b, bool trans_b, void* c, bool c_f32,
                           const F8Lora& l) {
  GemmArgs p{};
  p.m = static_cast<int32_t>(a.rows);
  p.n = static_cast<int32_t>(trans_b ? b.rows : b.cols);
  p.kb_total = static_cast<int32_t>(f8_blocks(a.cols));
  p.b_mn = trans_b ? 0 : 1;
  p.sa = a.scales;
  p.sb = b.scales;
  const int64_t b_kb = f8_blocks(b.cols);
  p.sb_n = trans_b ? b_kb : 1;
  p.sb_k = trans_b ? 1 : b_kb;
  p.c = c;
  p.c_ld = p.n;
  p.c_f32 = c_f32 ? 1 : 0;
  if (l.r > 0) {
    p.ext_half = (l.r + 63) / 64;
    p.ext_tiles = 2 * p.ext_half;
    p.ext_last_steps = ((l.r - 64 * (p.ext_half - 1)) + 15) / 16;
    p.ext_mn = trans_b ? 0 : 1;
  }
  return p;
}

qlora_status f8_gemm(const qlora_f8& a, const qlora_f8& b, bool trans_b, void* c, bool c_f32,
                     const F8Lora& l, cudaStream_t s) {
  const GemmArgs p = f8::gemm_args(a, b, trans_b, c, c_f32, l);
  const int64_t m = p.m, n = p.n;
  if (m <= 64) {
    const int splits = split_count(ceil_div(n, 128), p.kb_total);
    if (m <= 16) return launch<16, true>(a, b, trans_b, p, l, splits, s);
    if (m <= 32) return launch<32, true>(a, b, trans_b, p, l, splits, s);
    return launch<64, true>(a, b, trans_b, p, l, splits, s);
  }
  const int64_t tiles = ceil_div(n, 128) * ceil_div(m, 128);
  if (tiles > 148) return f8_gemm_pairs(a, b, trans_b, c, c_f32, l, s);
  return launch<128, false>(a, b, trans_b, p, l, split_count(tiles, p.kb_total), s);
}

}  // namespace qlora
