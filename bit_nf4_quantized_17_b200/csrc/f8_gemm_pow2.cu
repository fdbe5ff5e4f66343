// Matrix product in 8-bit floating point whose scales are powers of two, on CTA
// pairs: the large form for matrices with pow2 set (same product as f8_gemm2.cu, same
// LoRA term).
//
// The tensor core multiplies by such scales itself (tcgen05.mma.kind::mxf8f6f4 with
// block_scale: one 8-bit exponent per row and 32 contraction elements), so the whole
// contraction is summed in one fp32 TMEM accumulator and the registers see each sum
// once, at the end, instead of once per 128-deep block.  Four MMAs of a block share
// an exponent.
//
// Exponents in TMEM (scale vector 1X): row r of an operand has a 32-bit word in lane r % 32,
// column r / 32, the same in each of the four lane quarters; an MMA picks one of its
// bytes.  The bytes of a word are four consecutive blocks here, so a group of four blocks
// takes 4 columns for A's 128 rows of a CTA and 6 (of 8) for the tile's 192 rows of B.
// Four warps, one a quarter, build the words from the fp32 scales (exponent bits) and store
// them with tcgen05.st, up to four groups ahead.
//
// Bound: 2048 x 8192 x 8192 in 100 us in bursts (2.75 PFLOP/s, fp32 scales 125 us), 119 us
// sustained under the 1 kW power cap; 4096^3 in 52 us.
//
// A pair computes 256 x 192 tiles: two accumulators of 192 columns (one is drained
// while the next tile is summed) and the exponents fit the 512 TMEM columns, and
// 192 divides better into rounds than 256: 2048 x 8192 is 3.75 rounds' work instead
// of 4.  MN-major B is loaded 128 columns wide, of which 96 are used.
//
// Roles per CTA (512 threads): warp 0 TMA producer, warp 1 TMEM and, in the even
// CTA, the MMA issuer, warps 4-7 exponents, warps 8-15 drain.  TMA loads of both
// CTAs count on the even CTA's barriers (no multicast).  Every wait is bounded; a CTA whose
// wait gives up writes NaN to what it had not finished.
#include <cudaTypedefs.h>

#include <algorithm>

#include "f8_gemm.cuh"

namespace qlora {
namespace {

using f8::GemmArgs;
using f8::kTimeoutCycles;
using f8::store_run;

constexpr int kBN = 192;
constexpr int kHalf = kBN / 2;               // B rows a CTA provides
constexpr int kDrain = 8;                    // drain warps
constexpr int kThreads = 32 * (8 + kDrain);
constexpr int kStages = 6;
constexpr int kOpBytes = 16384;              // 128 rows x 128 bytes (B: 96, or 128 if MN-major)
constexpr int kStageBytes = 2 * kOpBytes;
constexpr int kGroups = 4;                   // exponent groups (of four blocks) in TMEM
constexpr int kGroupCols = 12;               // TMEM columns of one: 4 for A, 8 for B
constexpr int kExpCol = 2 * kBN;             // first of them
constexpr int kOutBytes = 4096;              // a warp's part of C on its way: 32 rows x 128 bytes
constexpr int kSmemBytes = 1024 + kStages * kStageBytes + kDrain * kOutBytes + 256;
constexpr int kTileGroup = 16;               // row tiles per column tile before the next one

__device__ __forceinline__ void tile_at(const GemmArgs& p, int m_tiles, int t, int* mt, int* nt) {
  const int per = kTileGroup * p.n_tiles;
  const int g = t / per, in = t - g * per;
  const int rows = min(kTileGroup, m_tiles - g * kTileGroup);
  *nt = in / rows;
  *mt = g * kTileGroup + in - *nt * rows;
}

// A scale's bits.  The launch ahead may write the scales while this one is already resident,
// so they are not read-only for this kernel's life: a plain load, not one through the
// read-only path, and volatile, so that it stays behind the dependency wait.
__device__ __forceinline__ uint32_t scale_bits(const float* s) {
  uint32_t u;
  asm volatile("ld.global.b32 %0, [%1];" : "=r"(u) : "l"(s));
  return u;
}
// Four scales' exponents as the bytes of a word.
__device__ __forceinline__ uint32_t exponents(const uint32_t (&u)[4]) {
  uint32_t w = 0u;
#pragma unroll
  for (int j = 0; j < 4; ++j) w |= ((u[j] >> 23) & 0xffu) << (8 * j);
  return w;
}

__global__ void __launch_bounds__(kThreads, 1)
f8_pow2_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
               const __grid_constant__ CUtensorMap tmL, const __grid_constant__ CUtensorMap tmR,
               const __grid_constant__ CUtensorMap tmC, const GemmArgs p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* out_stage = smem + kStages * kStageBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(out_stage + kDrain * kOutBytes);  // even CTA's count
  uint64_t* empty = full + kStages;
  uint64_t* exp_full = empty + kStages;    // even CTA's: both CTAs' exponent warps
  uint64_t* exp_empty = exp_full + kGroups;
  uint64_t* acc_full = exp_empty + kGroups;
  uint64_t* acc_empty = acc_full + 2;      // even CTA's: both CTAs' drain warps
  uint64_t* drain = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t rank = ptx::cluster_ctarank();
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const int m_tiles = (p.m + 255) / 256;
  const int tiles = m_tiles * p.n_tiles;
  const int kn = p.kb_total;

  ptx::grid_launch_dependents();
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      ptx::mbar_init(&full[s], 1);
      ptx::mbar_init(&empty[s], 1);
    }
    for (int g = 0; g < kGroups; ++g) {
      ptx::mbar_init(&exp_full[g], 2 * 4);
      ptx::mbar_init(&exp_empty[g], 1);
    }
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(&acc_full[b], 1);
      ptx::mbar_init(&acc_empty[b], 2 * kDrain);
    }
    ptx::mbar_init(drain, 1);
    *abort_flag = 0;
    ptx::fence_mbar_init();
    ptx::prefetch_tmap(&tmA);
    ptx::prefetch_tmap(&tmB);
  }
  if (warp == 1) {
    ptx::tmem_alloc_pair(tmem_slot, 512);
    ptx::tmem_relinquish_pair();
  }
  ptx::tc_fence_before();
  // both CTAs' barriers exist before either CTA signals the other's
  ptx::cluster_sync();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0 && ptx::elect_one()) {
    // ------------------------------------------------------ TMA producer
    // (the launch may start before the one ahead of it is done: see f8_gemm.cu)
    ptx::grid_dependency_wait();
    int it = 0, s = 0;
    uint32_t ph = 1;
    bool ok = true;
    const uint32_t bar0 = ptx::cluster_addr(&full[0], 0);
    const uint32_t b_bytes = p.b_mn ? kOpBytes : kHalf * 128;
    const uint32_t r_bytes = p.ext_mn ? kOpBytes : kHalf * 128;
    auto next = [&]() {
      ++it;
      if (++s == kStages) {
        s = 0;
        ph ^= 1;
      }
    };
    for (int t = pair; t < tiles && ok; t += pairs) {
      int mt, nt;
      tile_at(p, m_tiles, t, &mt, &nt);
      const int m0 = mt * 256 + static_cast<int>(rank) * 128;
      const int n0 = nt * kBN + static_cast<int>(rank) * kHalf;
      for (int i = 0, k = 0; i < kn; ++i, k += 128) {
        ok = ptx::mbar_wait(&empty[s], ph, kTimeoutCycles, abort_flag);
        if (!ok) break;
        uint8_t* sa = smem + s * kStageBytes;
        const uint32_t bar = bar0 + 8u * s;
        if (rank == 0) ptx::mbar_arrive_expect_tx(&full[s], 2 * (kOpBytes + b_bytes));
        ptx::tma_load_2d_pair(&tmA, bar, sa, k, m0);
        if (p.b_mn)
          ptx::tma_load_2d_pair(&tmB, bar, sa + kOpBytes, n0, k);
        else
          ptx::tma_load_2d_pair(&tmB, bar, sa + kOpBytes, k, n0);
        next();
      }
      for (int x = 0, h = 0; x < p.ext_tiles && ok; ++x) {
        ok = ptx::mbar_wait(&empty[s], ph, kTimeoutCycles, abort_flag);
        if (!ok) break;
        uint8_t* sa = smem + s * kStageBytes;
        uint8_t* sb = sa + kOpBytes;
        const uint32_t bar = bar0 + 8u * s;
        if (rank == 0) ptx::mbar_arrive_expect_tx(&full[s], 2 * (kOpBytes + r_bytes));
        const int kr = h * 64;
        if (++h == p.ext_half) h = 0;
        ptx::tma_load_2d_pair(&tmL, bar, sa, x * 64, m0);
        if (p.ext_mn) {
          ptx::tma_load_2d_pair(&tmR, bar, sb, n0, kr);
          ptx::tma_load_2d_pair(&tmR, bar, sb + 8192, n0 + 64, kr);
        } else {
          ptx::tma_load_2d_pair(&tmR, bar, sb, kr, n0);
        }
        next();
      }
    }
    // never leave with copies in flight: they all count on the even CTA's barriers
    if (rank == 0)
      for (int i = (it > kStages ? it - kStages : 0); i < it; ++i)
        ptx::mbar_wait(&full[i % kStages], (i / kStages) & 1, kTimeoutCycles, nullptr);
  } else if (warp == 1 && rank == 0 && ptx::elect_one()) {
    // ------------------------------------------------------ MMA issuer (even CTA)
    const uint32_t a_addr = ptx::smem_u32(smem), b_addr = a_addr + kOpBytes;
    const uint64_t ad0 = ptx::sw128_desc(a_addr, 16, 1024);
    const uint64_t bd0 = ptx::sw128_desc(b_addr, p.b_mn ? kOpBytes : 16, 1024);
    const uint64_t rd0 = ptx::sw128_desc(b_addr, p.ext_mn ? 8192 : 16, 1024);
    const uint64_t bs = p.b_mn ? (4096 >> 4) : (32 >> 4);
    const uint64_t rs = p.ext_mn ? (2048 >> 4) : (32 >> 4);
    int s = 0, g = 0;
    uint32_t ph = 0, b = 0, bph = 1, gph = 0;
    uint64_t off = 0;
    bool ok = true;
    auto next = [&]() {
      off += kStageBytes >> 4;
      if (++s == kStages) {
        s = 0;
        ph ^= 1;
        off = 0;
      }
    };
    for (int t = pair; t < tiles && ok; t += pairs) {
      ok = ptx::mbar_wait(&acc_empty[b], bph, kTimeoutCycles, abort_flag);
      if (!ok) break;
      const uint32_t d = tmem + b * kBN;
      for (int i = 0; i < kn; ++i) {
        ok = ptx::mbar_wait(&full[s], ph, kTimeoutCycles, abort_flag);
        if (ok && (i & 3) == 0) ok = ptx::mbar_wait(&exp_full[g], gph, kTimeoutCycles, abort_flag);
        if (!ok) break;
        ptx::tc_fence_after();
        const uint64_t ad = ad0 + off, bd = bd0 + off;
        const uint32_t ea = tmem + kExpCol + g * kGroupCols, eb = ea + 4;
        // the byte of the words that this block's exponents are in
        const uint32_t idesc = p.idesc | (static_cast<uint32_t>(i & 3) << 4) |
                               (static_cast<uint32_t>(i & 3) << 29);
        ptx::umma_mxf8_pair(d, ad, bd, idesc, ea, eb, i ? 1u : 0u);
        ptx::umma_mxf8_pair(d, ad + 2, bd + bs, idesc, ea, eb, 1u);
        ptx::umma_mxf8_pair(d, ad + 4, bd + 2 * bs, idesc, ea, eb, 1u);
        ptx::umma_mxf8_pair(d, ad + 6, bd + 3 * bs, idesc, ea, eb, 1u);
        ptx::umma_commit_pair(&empty[s]);
        next();
        if ((i & 3) == 3 || i == kn - 1) {
          ptx::umma_commit_pair(&exp_empty[g]);
          if (++g == kGroups) {
            g = 0;
            gph ^= 1;
          }
        }
      }
      for (int x = 0, h = 0; x < p.ext_tiles && ok; ++x) {
        ok = ptx::mbar_wait(&full[s], ph, kTimeoutCycles, abort_flag);
        if (!ok) break;
        ptx::tc_fence_after();
        const int steps = ++h == p.ext_half ? p.ext_last_steps : 4;
        if (h == p.ext_half) h = 0;
        for (int ks = 0; ks < steps; ++ks)
          ptx::umma_bf16_pair(d, ad0 + off + 2 * ks, rd0 + off + rs * ks, p.idesc_ext, 1u);
        ptx::umma_commit_pair(&empty[s]);
        next();
      }
      if (!ok) break;
      ptx::umma_commit_pair(&acc_full[b]);
      b ^= 1;
      if (b == 0) bph ^= 1;
    }
    // what was issued is done before shared memory and TMEM go
    ptx::umma_commit_pair(drain);
    ptx::mbar_wait(drain, 0, kTimeoutCycles, nullptr);
  } else if (warp >= 4 && warp < 8) {
    // ------------------------------------------------------ exponents
    ptx::grid_dependency_wait();
    const uint32_t base = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16) + kExpCol;
    const uint32_t leader = ptx::cluster_addr(&exp_full[0], 0);
    const int nbs = (p.n + 127) >> 7;
    int g = 0;
    uint32_t ph = 1;
    bool ok = true;
    for (int t = pair; t < tiles && ok; t += pairs) {
      int mt, nt;
      tile_at(p, m_tiles, t, &mt, &nt);
      const int row0 = mt * 256 + static_cast<int>(rank) * 128 + lane;
      for (int k0 = 0; k0 < kn; k0 += 4) {
        // rows and columns past the end repeat the last one: their products are not stored;
        // blocks past the end are not multiplied
        // (all loads before the first use); a tile's 192 columns lie in two column blocks of
        // B, from 0 or 64 into the first
        uint32_t ra[4][4], rb[2][4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int64_t kb = min(k0 + j, kn - 1);
#pragma unroll
          for (int c = 0; c < 4; ++c)
            ra[c][j] = scale_bits(p.sa + kb * p.m + min(row0 + 32 * c, p.m - 1));
#pragma unroll
          for (int b = 0; b < 2; ++b)
            rb[b][j] =
                scale_bits(p.sb + min(((nt * kBN) >> 7) + b, nbs - 1) * p.sb_n + kb * p.sb_k);
        }
        uint32_t wa[4], wb[8];
#pragma unroll
        for (int c = 0; c < 4; ++c) wa[c] = exponents(ra[c]);
        const uint32_t first = exponents(rb[0]), second = exponents(rb[1]);
#pragma unroll
        for (int c = 0; c < 8; ++c)
          wb[c] = ((nt * kBN) & 127) + 32 * min(c, 5) < 128 ? first : second;
        ok = ptx::mbar_wait(&exp_empty[g], ph, kTimeoutCycles, abort_flag);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        ptx::tc_fence_after();
        ptx::tmem_st_x4(base + g * kGroupCols, wa);
        ptx::tmem_st_x8(base + g * kGroupCols + 4, wb);
        ptx::tmem_st_wait();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive_cluster(leader + 8u * g);
        if (++g == kGroups) {
          g = 0;
          ph ^= 1;
        }
      }
    }
  } else if (warp >= 8) {
    // ------------------------------------------------------ drain
    const int quarter = warp & 3, h = (warp - 8) >> 2;  // columns [96 h, 96 h + 96)
    const uint32_t lane_base = static_cast<uint32_t>(32 * quarter) << 16;
    const uint32_t free_base = ptx::cluster_addr(&acc_empty[0], 0);
    uint8_t* stage = out_stage + (warp - 8) * kOutBytes;
    uint32_t use = 0;
    bool ok = true;
    for (int t = pair; t < tiles; t += pairs, ++use) {
      int mt, nt;
      tile_at(p, m_tiles, t, &mt, &nt);
      if (ok) ok = ptx::mbar_wait(&acc_full[use & 1], (use >> 1) & 1, kTimeoutCycles, abort_flag);
      ok = __all_sync(0xffffffffu, ok && !*abort_flag);
      if (ok) ptx::tc_fence_after();
      const int row0 = mt * 256 + static_cast<int>(rank) * 128 + 32 * quarter;
      const int col0 = nt * kBN + kHalf * h;
#pragma unroll
      for (int c = 0; c < 3; ++c) {  // 32 columns
        uint32_t r[32];
        if (ok) {
          ptx::tmem_ld_x32(tmem + lane_base + (use & 1) * kBN + kHalf * h + 32 * c, r);
          ptx::tmem_ld_wait(r);
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) r[j] = 0x7fffffffu;  // NaN
        }
        if (c == 2) {
          // everything is in registers: the accumulator may be overwritten
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0 && ok) ptx::mbar_arrive_cluster(free_base + 8u * (use & 1));
        }
        const int col = col0 + 32 * c;
        if (p.c_tma) {
          if (lane == 0) ptx::bulk_wait_read();
          __syncwarp();
          if (p.c_f32) {
#pragma unroll
            for (int q = 0; q < 8; ++q)
              *reinterpret_cast<uint4*>(stage + lane * 128 + 16 * (q ^ (lane & 7))) =
                  make_uint4(r[4 * q], r[4 * q + 1], r[4 * q + 2], r[4 * q + 3]);
          } else {
            // 64 bytes a row, 64-byte swizzle
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              uint32_t w[4];
#pragma unroll
              for (int j = 0; j < 4; ++j)
                w[j] = tc::pack_bf16x2(__uint_as_float(r[8 * q + 2 * j]),
                                       __uint_as_float(r[8 * q + 2 * j + 1]));
              *reinterpret_cast<uint4*>(stage + lane * 64 + 16 * (q ^ ((lane >> 1) & 3))) =
                  make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
          ptx::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0 && row0 < p.m && col < p.n) {
            // (an fp32 C is described as pairs of 16-bit columns)
            ptx::tma_store_2d(&tmC, stage, p.c_f32 ? 2 * col : col, row0);
            ptx::bulk_commit();
          }
        } else {
          float v[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j]);
          store_run<16>(p, row0 + lane, col, v);
          store_run<16>(p, row0 + lane, col + 16, v + 16);
        }
      }
    }
    if (lane == 0) ptx::bulk_wait_read();  // before shared memory goes
  }
  ptx::tc_fence_before();
  __syncthreads();
  // neither CTA leaves (or frees TMEM) while the pair may still touch it
  ptx::cluster_sync();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc_pair(tmem, 512);
  }
}

}  // namespace

qlora_status f8_gemm_pow2(const qlora_f8& a, const qlora_f8& b, bool trans_b, void* c, bool c_f32,
                          const F8Lora& l, cudaStream_t s) {
  GemmArgs p = f8::gemm_args(a, b, trans_b, c, c_f32, l);
  const int64_t m = p.m, n = p.n;
  CUtensorMap ma, mb, ml, mr, mc;
  bool ok = make_map(&ma, a.codes, false, a.cols, m, a.ld, 128, 128, true) &&
            (trans_b ? make_map(&mb, b.codes, false, b.cols, n, b.ld, 128, kHalf, true)
                     : make_map(&mb, b.codes, false, n, b.rows, b.ld, 128, 128, true));
  if (l.r > 0) {
    const int64_t ld = 2 * lora_span(l.r);
    ok = ok && make_map(&ml, l.L, true, ld, m, ld, 64, 128, true) &&
         (p.ext_mn ? make_map(&mr, l.R, true, n, l.r, n, 64, 64, true)
                   : make_map(&mr, l.R, true, l.r, n, l.r, 64, kHalf, true));
  } else {
    ml = ma;
    mr = mb;
  }
  // C through TMA stores where its rows start on 16 bytes: 32 columns a box
  const int64_t words = c_f32 ? 2 * n : n;
  mc = ma;
  p.c_tma = words % 8 == 0 ? 1 : 0;
  if (p.c_tma) ok = ok && make_map(&mc, c, true, words, m, words, c_f32 ? 64 : 32, 32, true);
  if (!ok) return QLORA_ERR_CUDA;
  const int fa = a.format == QLORA_E5M2 ? 1 : 0, fb = b.format == QLORA_E5M2 ? 1 : 0;
  p.idesc = ptx::idesc_mxf8(fa, fb, 256, kBN, 0, p.b_mn);
  p.idesc_ext = ptx::idesc_bf16(256, kBN, 0, p.ext_mn);
  p.n_tiles = static_cast<int32_t>(ceil_div(n, kBN));
  const int64_t tiles = ceil_div(m, 256) * p.n_tiles;
  if (tiles > 0x3fffffff) return QLORA_ERR_SHAPE;
  const qlora_status cs = ensure_smem(reinterpret_cast<const void*>(f8_pow2_kernel), kSmemBytes);
  if (cs != QLORA_OK) return cs;
  const int64_t pairs = std::max<int64_t>(1, std::min<int64_t>(tiles, f8::sm_count() / 2));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * pairs));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  count_launch();
  const cudaError_t e = cudaLaunchKernelEx(&cfg, f8_pow2_kernel, ma, mb, ml, mr, mc, p);
  if (e != cudaSuccess) {
    (void)cudaGetLastError();
    return QLORA_ERR_CUDA;
  }
  return after_launch("f8_gemm_pow2", s);
}

}  // namespace qlora
