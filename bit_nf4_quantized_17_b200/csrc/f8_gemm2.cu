// Matrix product in 8-bit floating point with a scale for each block of 128, on
// CTA pairs: the large form of f8_gemm.cu (same product, same LoRA term).
//
// A cluster of two CTAs computes 256 x 256 tiles of C with pair MMAs
// (tcgen05.mma.cta_group::2, M = 256, issued by the even CTA): each CTA holds its 128
// rows of A and half of the B tile, and its TMEM receives its 128 rows' sums.  A
// 128-deep block is two products of N = 128 (64 columns of either CTA's half each),
// 256 cycles apiece, into one of two TMEM accumulators of their own (four in all:
// the 512 columns).  Four warps drain each half: 128 fp32 sums a thread, times the
// block's scales, in packed multiply-adds (two a register pair: no faster per
// sum than scalar ones, but they leave every other issue slot to the MMA issuer,
// which shares an SM quarter with two of these warps: 326 against 338 us below).
// Halves rather than one N = 256 product per block keep the MMAs and the sums of
// either group out of step with each other (one product: 340 us), and the tensor
// cores work on two accumulators while two are drained.  With one thread a row and
// 128 columns a thread needs one scale of A and two of B per block.
//
// ptxas: 168 registers at launch, 40 bytes of stack (80 of spill stores, 160 of loads in the
// code).  They come with the block of the LoRA term: without it there are none.
//
// Bound: 2048 x 8192 x 22016 takes 322 us in bursts (2.3 PFLOP/s), the same MMAs
// without sums 250 us; sustained, the 1 kW power cap lowers the clock to 1.48 GHz
// and it takes 384 us.  4096^3: 70 us.
//
// The kernel is persistent: a pair takes tiles pair, pair + pairs, ..., and
// while its sum warps store a tile the next tile's first blocks run.  Tiles go
// down 16 row tiles before the next column tile, so that the pairs at work share a few
// columns of B and rows of A that stay in L2.
//
// Roles per CTA (384 threads): warp 0 TMA producer, warp 1 TMEM and, in the
// even CTA, the MMA issuer, warp 2 the scales, warps 4-11 the sums.  The sums and the
// words on their way are 192 registers a thread: the role warps hand theirs over
// (40 against 232).  TMA loads of both CTAs count on the even CTA's barriers (no
// multicast).  Every wait is bounded; a CTA whose wait gives up writes NaN to what it
// had not finished.
#include <cudaTypedefs.h>

#include <algorithm>

#include "f8_gemm.cuh"

namespace qlora {
namespace {

using f8::GemmArgs;
using f8::kTimeoutCycles;
using f8::add64;
using f8::store_run;

constexpr int kEpi = 8;
constexpr int kRoleWarps = 4;                // TMA, MMA, scales, one idle
constexpr int kThreads = 32 * (kRoleWarps + kEpi);
constexpr int kRoleRegs = 40, kSumRegs = 232;  // registers a thread, from 168 at launch
constexpr int kStages = 5;
constexpr int kOpBytes = 16384;              // 128 rows x 128 bytes: A, and this CTA's half of B
constexpr int kStageBytes = 2 * kOpBytes;
using Ring = f8::PairRing;
constexpr int kOutBytes = 4096;              // a warp's part of C on its way: 32 rows x 128 bytes
constexpr int kSmemBytes = 1024 + kStages * kStageBytes + kEpi * kOutBytes + sizeof(Ring) + 256;
constexpr int kGroup = 16;                   // row tiles per column tile before the next one

__device__ __forceinline__ void tile_at(const GemmArgs& p, int m_tiles, int t, int* mt, int* nt) {
  const int per = kGroup * p.n_tiles;
  const int g = t / per, in = t - g * per;
  const int rows = min(kGroup, m_tiles - g * kGroup);
  *nt = in / rows;
  *mt = g * kGroup + in - *nt * rows;
}

__global__ void __launch_bounds__(kThreads, 1)
f8_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
               const __grid_constant__ CUtensorMap tmL, const __grid_constant__ CUtensorMap tmR,
               const __grid_constant__ CUtensorMap tmC, const GemmArgs p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* out_stage = smem + kStages * kStageBytes;
  Ring* ring = reinterpret_cast<Ring*>(out_stage + kEpi * kOutBytes);
  uint64_t* full = reinterpret_cast<uint64_t*>(ring + 1);  // even CTA's count
  uint64_t* empty = full + kStages;
  uint64_t* acc_full = empty + kStages;
  uint64_t* acc_empty = acc_full + 4;  // even CTA's: both CTAs' warps
  uint64_t* sc_full = acc_empty + 4;
  uint64_t* sc_empty = sc_full + 2;
  uint64_t* drain = sc_empty + 2;
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
    for (int b = 0; b < 4; ++b) {
      ptx::mbar_init(&acc_full[b], 1);
      ptx::mbar_init(&acc_empty[b], kEpi);
    }
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(&sc_full[b], 32);
      ptx::mbar_init(&sc_empty[b], kEpi);
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

  // (The loops of the two issuing threads step the stage, its phase and the
  // descriptors with adds only: see f8_gemm.cu.)
  if (warp < kRoleWarps) {
  ptx::setmaxnreg_dec<kRoleRegs>();
  if (warp == 0 && ptx::elect_one()) {
    // ------------------------------------------------------ TMA producer
    // the launch may start before the one ahead of it is done: everything before
    // this touched no memory of the caller's, everything after follows these loads
    ptx::grid_dependency_wait();
    int it = 0, s = 0;
    uint32_t ph = 1;
    bool ok = true;
    const uint32_t bar0 = ptx::cluster_addr(&full[0], 0);
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
      const int n0 = nt * 256 + static_cast<int>(rank) * 128;  // this CTA's half of B
      for (int i = 0, k = 0; i < kn; ++i, k += 128) {
        ok = ptx::mbar_wait(&empty[s], ph, kTimeoutCycles, abort_flag);
        if (!ok) break;
        uint8_t* sa = smem + s * kStageBytes;
        const uint32_t bar = bar0 + 8u * s;
        if (rank == 0) ptx::mbar_arrive_expect_tx(&full[s], 2 * kStageBytes);
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
        if (rank == 0) ptx::mbar_arrive_expect_tx(&full[s], 2 * kStageBytes);
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
    // the second 64 of this CTA's 128 B rows (columns of C): 64 rows of 128 bytes
    // further where K-major, 64 bytes further in every row where MN-major; the LoRA
    // operand's 64 columns are a box of their own either way
    const uint64_t bh = p.b_mn ? (64 >> 4) : (8192 >> 4), rh = 8192 >> 4;
    const uint32_t idesc = p.idesc;
    int s = 0;
    uint32_t ph = 0, b = 0, bph = 1;  // b: accumulator 0 or 2 of a block's first half
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
    auto next_acc = [&]() {
      b ^= 2;
      if (b == 0) bph ^= 1;
    };
    for (int t = pair; t < tiles && ok; t += pairs) {
      for (int i = 0; i < kn; ++i) {
        // the operands first: they are there long before the accumulator is free
        ok = ptx::mbar_wait(&full[s], ph, kTimeoutCycles, abort_flag) &&
             ptx::mbar_wait(&acc_empty[b], bph, kTimeoutCycles, abort_flag);
        if (!ok) break;
        ptx::tc_fence_after();
        const uint64_t ad = ad0 + off, bd = bd0 + off;
        uint32_t d = tmem + b * 128;
        ptx::umma_f8_pair(d, ad, bd, idesc, 0u);
        ptx::umma_f8_pair(d, ad + 2, bd + bs, idesc, 1u);
        ptx::umma_f8_pair(d, ad + 4, bd + 2 * bs, idesc, 1u);
        ptx::umma_f8_pair(d, ad + 6, bd + 3 * bs, idesc, 1u);
        ptx::umma_commit_pair(&acc_full[b]);
        ok = ptx::mbar_wait(&acc_empty[b + 1], bph, kTimeoutCycles, abort_flag);
        if (!ok) break;
        ptx::tc_fence_after();
        d += 128;
        ptx::umma_f8_pair(d, ad, bd + bh, idesc, 0u);
        ptx::umma_f8_pair(d, ad + 2, bd + bh + bs, idesc, 1u);
        ptx::umma_f8_pair(d, ad + 4, bd + bh + 2 * bs, idesc, 1u);
        ptx::umma_f8_pair(d, ad + 6, bd + bh + 3 * bs, idesc, 1u);
        ptx::umma_commit_pair(&acc_full[b + 1]);
        ptx::umma_commit_pair(&empty[s]);
        next();
        next_acc();
      }
      if (p.ext_tiles && ok) {
        // every LoRA stage goes into one pair of accumulators
        ok = ptx::mbar_wait(&acc_empty[b], bph, kTimeoutCycles, abort_flag) &&
             ptx::mbar_wait(&acc_empty[b + 1], bph, kTimeoutCycles, abort_flag);
        for (int x = 0, h = 0; x < p.ext_tiles && ok; ++x) {
          ok = ptx::mbar_wait(&full[s], ph, kTimeoutCycles, abort_flag);
          if (!ok) break;
          ptx::tc_fence_after();
          const int steps = ++h == p.ext_half ? p.ext_last_steps : 4;
          if (h == p.ext_half) h = 0;
          for (int ks = 0; ks < steps; ++ks) {
            const uint64_t ad = ad0 + off + 2 * ks, rd = rd0 + off + rs * ks;
            const uint32_t acc = (x | ks) != 0 ? 1u : 0u;
            ptx::umma_bf16_pair(tmem + b * 128, ad, rd, p.idesc_ext, acc);
            ptx::umma_bf16_pair(tmem + b * 128 + 128, ad, rd + rh, p.idesc_ext, acc);
          }
          ptx::umma_commit_pair(&empty[s]);
          next();
        }
        if (!ok) break;
        ptx::umma_commit_pair(&acc_full[b]);
        ptx::umma_commit_pair(&acc_full[b + 1]);
        next_acc();
      }
    }
    // what was issued is done before shared memory and TMEM go
    ptx::umma_commit_pair(drain);
    ptx::mbar_wait(drain, 0, kTimeoutCycles, nullptr);
  } else if (warp == 2) {
    // ------------------------------------------------------ scales
    ptx::grid_dependency_wait();
    int chunk = 0;
    bool ok = true;
    for (int t = pair; t < tiles && ok; t += pairs) {
      int mt, nt;
      tile_at(p, m_tiles, t, &mt, &nt);
      for (int kb = 0; kb < kn; kb += f8::kChunk, ++chunk) {
        ok = ptx::mbar_wait(&sc_empty[chunk & 1], ((chunk >> 1) & 1) ^ 1, kTimeoutCycles,
                            abort_flag);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        f8::fill_scales(p, ring, chunk & 1, kb, kn, mt * 256 + static_cast<int>(rank) * 128,
                        2 * nt, (p.n + 127) >> 7, lane, &sc_full[chunk & 1]);
      }
    }
    f8::cp_async_wait_all();
  }
  } else {
    // ------------------------------------------------------ sums
    ptx::setmaxnreg_inc<kSumRegs>();
    // warps 4-7 add the accumulators of the first half of each block, warps 8-11
    // those of the second: columns [64 h, 64 h + 64) and [128 + 64 h, ...) of the tile
    const int quarter = warp & 3, h = (warp - kRoleWarps) >> 2;
    const int lrow = 32 * quarter + lane;
    const uint32_t tmem_base = tmem + (static_cast<uint32_t>(32 * quarter) << 16) + h * 128;
    const uint32_t full_base = ptx::smem_u32(&acc_full[h]);
    const uint32_t free_base = ptx::cluster_addr(&acc_empty[h], 0);
    const uint32_t sa_base = ptx::smem_u32(&ring->a[0][0][lrow]);
    const uint32_t sb_base = ptx::smem_u32(&ring->b[0][0][0]);
    // two sums a register pair: one instruction multiplies and adds both
    uint64_t acc[64];
    uint32_t use = 0, chunk = 0;
    bool ok = true, ready = false;
    // Adds one finished accumulator, its first 64 columns times s0, the others times s1.
    auto add_block = [&](float s0, float s1, auto&& prefetch) {
      if (!ready) {
        ok = ptx::mbar_wait(&acc_full[2 * (use & 1) + h], (use >> 1) & 1, kTimeoutCycles,
                            abort_flag);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) return;
      }
      ptx::tc_fence_after();
      const uint32_t at = tmem_base + (use & 1) * 256, release = free_base + (use & 1) * 16;
      ++use;
      uint32_t r[64];
      ptx::tmem_ld_x64(at, r);
      ptx::tmem_ld_wait(r);
      add64(acc, 0, r, s0);
      ptx::tmem_ld_x64(at + 64, r);
      ptx::tmem_ld_wait(r);
      // everything is in registers: the accumulator may be overwritten
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive_cluster(release);
      // the test of the next one, and its scales, take their time while these are
      // added: next to the MMAs' operand reads an access to shared memory takes
      // 100 to 250 cycles
      const bool next = ptx::mbar_test_wait_at(full_base + (use & 1) * 16, (use >> 1) & 1);
      prefetch();
      add64(acc, 32, r, s1);
      ready = __all_sync(0xffffffffu, next);
    };
    for (int t = pair; t < tiles; t += pairs) {
      int mt, nt;
      tile_at(p, m_tiles, t, &mt, &nt);
#pragma unroll
      for (int j = 0; j < 64; ++j) acc[j] = 0ull;
      for (int k0 = 0; k0 < kn && ok; k0 += f8::kChunk, ++chunk) {
        ok = ptx::mbar_wait(&sc_full[chunk & 1], (chunk >> 1) & 1, kTimeoutCycles, abort_flag);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        uint32_t pa = sa_base + Ring::a_at(chunk, 0);
        uint32_t pb = sb_base + Ring::b_at(chunk, 0);
        float sa = ptx::lds_f32(pa);
        float2 sb = ptx::lds_f32x2(pb);
        const int n = min(f8::kChunk, kn - k0);
        for (int i = 0; i < n && ok; ++i) {
          const float s0 = sa * sb.x, s1 = sa * sb.y;
          // the next block's scales, on their way while this one is added (past the
          // last block of a chunk: the ring's spare row, not used)
          pa += Ring::a_at(0, 1);
          pb += Ring::b_at(0, 1);
          add_block(s0, s1, [&]() {
            sa = ptx::lds_f32(pa);
            sb = ptx::lds_f32x2(pb);
          });
        }
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&sc_empty[chunk & 1]);
      }
      if (p.ext_tiles && ok) add_block(1.0f, 1.0f, []() {});  // the LoRA term
      ok = __all_sync(0xffffffffu, ok && !*abort_flag);
      const int row0 = mt * 256 + static_cast<int>(rank) * 128 + 32 * quarter;
      const int col0 = nt * 256 + 64 * h;
      // value j of the thread's row: column col0 + j, or col0 + 64 + j from 64 on
      auto value = [&](int j) -> float {
        float lo, hi;
        asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(acc[j / 2]));
        return ok ? (j & 1 ? hi : lo) : __int_as_float(0x7fffffff);
      };
      if (p.c_tma) {
        // through shared memory, 128 bytes of each row at a time: the copy engine
        // writes whole lines while the next tile is multiplied (stores from the
        // registers, 16 bytes of 32 rows an instruction, took 2 us a tile)
        uint8_t* stage = out_stage + (warp - kRoleWarps) * kOutBytes;
#pragma unroll
        for (int c = 0; c < 4; ++c) {       // 32 columns
          const bool first = p.c_f32 || (c & 1) == 0;
          if (first) {
            if (lane == 0) ptx::bulk_wait_read();
            __syncwarp();
          }
          if (p.c_f32) {
#pragma unroll
            for (int q = 0; q < 8; ++q)
              *reinterpret_cast<float4*>(stage + lane * 128 + 16 * (q ^ (lane & 7))) =
                  make_float4(value(32 * c + 4 * q), value(32 * c + 4 * q + 1),
                              value(32 * c + 4 * q + 2), value(32 * c + 4 * q + 3));
          } else {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              uint32_t w[4];
#pragma unroll
              for (int j = 0; j < 4; ++j)
                w[j] = tc::pack_bf16x2(value(32 * c + 8 * q + 2 * j),
                                       value(32 * c + 8 * q + 2 * j + 1));
              *reinterpret_cast<uint4*>(stage + lane * 128 +
                                        16 * ((4 * (c & 1) + q) ^ (lane & 7))) =
                  make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
          if (p.c_f32 || (c & 1)) {
            ptx::fence_proxy_async_smem();
            __syncwarp();
            const int col = col0 + 128 * (c >> 1) + (p.c_f32 ? 32 * (c & 1) : 0);
            if (lane == 0 && row0 < p.m && col < p.n) {
              // (an fp32 C is described as pairs of 16-bit columns)
              ptx::tma_store_2d(&tmC, stage, p.c_f32 ? 2 * col : col, row0);
              ptx::bulk_commit();
            }
          }
        }
      } else {
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          float v[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) v[j] = value(16 * c + j);
          store_run<16>(p, row0 + lane, col0 + 128 * (c >> 2) + 16 * (c & 3), v);
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

qlora_status f8_gemm_pairs(const qlora_f8& a, const qlora_f8& b, bool trans_b, void* c, bool c_f32,
                           const F8Lora& l, cudaStream_t s) {
  GemmArgs p = f8::gemm_args(a, b, trans_b, c, c_f32, l);
  const int64_t m = p.m, n = p.n;
  CUtensorMap ma, mb, ml, mr;
  bool ok = make_map(&ma, a.codes, false, a.cols, m, a.ld, 128, 128, true) &&
            (trans_b ? make_map(&mb, b.codes, false, b.cols, n, b.ld, 128, 128, true)
                     : make_map(&mb, b.codes, false, n, b.rows, b.ld, 128, 128, true));
  if (l.r > 0) {
    const int64_t ld = 2 * lora_span(l.r);
    ok = ok && make_map(&ml, l.L, true, ld, m, ld, 64, 128, true) &&
         (p.ext_mn ? make_map(&mr, l.R, true, n, l.r, n, 64, 64, true)
                   : make_map(&mr, l.R, true, l.r, n, l.r, 64, 128, true));
  } else {
    ml = ma;
    mr = mb;
  }
  // C through TMA stores where its rows start on 16 bytes
  const int64_t words = c_f32 ? 2 * n : n;
  CUtensorMap mc = ma;
  p.c_tma = words % 8 == 0 ? 1 : 0;
  if (p.c_tma) ok = ok && make_map(&mc, c, true, words, m, words, 64, 32, true);
  if (!ok) return QLORA_ERR_CUDA;
  const int fa = a.format == QLORA_E5M2 ? 1 : 0, fb = b.format == QLORA_E5M2 ? 1 : 0;
  p.idesc = ptx::idesc_f8(fa, fb, 256, 128, 0, p.b_mn);
  p.idesc_ext = ptx::idesc_bf16(256, 128, 0, p.ext_mn);
  p.n_tiles = static_cast<int32_t>(ceil_div(n, 256));
  const int64_t tiles = ceil_div(m, 256) * p.n_tiles;
  if (tiles > 0x3fffffff) return QLORA_ERR_SHAPE;
  const void* fn = reinterpret_cast<const void*>(f8_pair_kernel);
  const qlora_status cs = ensure_smem(fn, kSmemBytes);
  if (cs != QLORA_OK) return cs;
  // the sum warps' larger share comes out of the registers of the launch: a build that
  // launches with fewer would wait for them forever
  constexpr int kRegsTag = 1;
  int regs = 0;
  if (!cached_value(fn, kRegsTag, &regs)) {
    cudaFuncAttributes attr;
    if (cudaFuncGetAttributes(&attr, f8_pair_kernel) != cudaSuccess) {
      (void)cudaGetLastError();
      return QLORA_ERR_CUDA;
    }
    regs = attr.numRegs;
    store_value(fn, kRegsTag, regs);
  }
  if (regs * kThreads < 32 * (kRoleWarps * kRoleRegs + kEpi * kSumRegs))
    return QLORA_ERR_UNSUPPORTED;
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
  cfg.attrs = attr;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.numAttrs = 2;
  count_launch();
  const cudaError_t e = cudaLaunchKernelEx(&cfg, f8_pair_kernel, ma, mb, ml, mr, mc, p);
  if (e != cudaSuccess) {
    (void)cudaGetLastError();
    return QLORA_ERR_CUDA;
  }
  return after_launch("f8_gemm_pairs", s);
}

}  // namespace qlora
