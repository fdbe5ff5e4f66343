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
//   * SWAP, for few tokens: P = B, Q = A (BN = 16, 32): the 128 rows of the
//     MMA are output columns, no MMA row is wasted on tokens that do not exist,
//     and B, whose bytes bound the product, is read once.  A thread holds one
//     output column and all BN tokens.
// B is read in place in both directions of the layer: K-major (C = A B^T) or
// MN-major (C = A B).
// Where the tiles would leave SMs idle the contraction is split over the CTAs
// of a cluster (up to 8) and the fp32 partial tiles are summed in distributed
// shared memory in split order (deterministic).
//
// Roles: warp 0 TMA producer, warp 1 TMEM owner and MMA issuer, warp 2 the
// scales, the 4 or 8 warps from warp 4 on drain the accumulators.  Every wait is
// bounded; the call has no status word, so a CTA whose wait gives up writes NaN to its
// part.
//
// Bound by the bytes of B for few tokens (1 x 11008 x 4096 in 11 us from HBM, 45 MB), by
// its fixed costs (launch, first loads, cluster sum: 6 us) up to a few hundred.
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
  static_assert(SWAP ? BN <= 32 : BN == 128, "the column split of the epilogue");
  static constexpr int kEpi = BN >= 128 ? 8 : 4;  // epilogue warps
  static constexpr int kPerSm = SWAP ? 2 : 1;
  static constexpr int kThreads = 128 + 32 * kEpi;  // TMA, MMA, scales, one idle; the sums
  static constexpr int kCols = BN / (kEpi / 4);   // accumulator columns per thread
  // TMEM accumulators in flight (two of 128 columns: 22 us instead of 18.8 for
  // 256 x 11008 x 4096)
  static constexpr int kBufs = 4;
  static constexpr int kTmem = BN * kBufs;        // 64, 128 or 256 columns
  using Ring = f8::ScaleRing<SWAP ? BN : 128, 1>;
  static constexpr int kQBytes = BN * 128;
  static constexpr int kStage = kPBytes + kQBytes;
  // fp32 partial tile: rows of tokens, padded against bank conflicts
  static constexpr int kRedLd = SWAP ? 128 + 4 : BN + 4;
  static constexpr int kRedBytes = (SWAP ? BN : 128) * kRedLd * 4;
};

template <int BN, bool SWAP>
__global__ void __launch_bounds__(Cfg<BN, SWAP>::kThreads, Cfg<BN, SWAP>::kPerSm)
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
  auto* ring = reinterpret_cast<typename C::Ring*>(smem + area);
  uint64_t* full = reinterpret_cast<uint64_t*>(ring + 1);
  uint64_t* empty = full + kMaxStages;
  uint64_t* acc_full = empty + kMaxStages;
  uint64_t* acc_empty = acc_full + C::kBufs;
  uint64_t* sc_full = acc_empty + C::kBufs;
  uint64_t* sc_empty = sc_full + 2;
  uint64_t* drain = sc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t S = gridDim.z, z = blockIdx.z;  // the cluster spans z
  // tile of P (128 rows) and of Q (BN rows)
  const int qt = blockIdx.x % p.n_tiles, pt = blockIdx.x / p.n_tiles;
  const int p0 = pt * 128, q0 = qt * BN;
  const int kb0 = static_cast<int>(z) * p.kb_per;
  const int kn = max(0, min(p.kb_per, p.kb_total - kb0));
  // the LoRA stages belong to the last split
  const int ext = (z == S - 1) ? p.ext_tiles : 0;
  const bool p_mn = SWAP && p.b_mn, q_mn = !SWAP && p.b_mn;
  const bool p2_mn = SWAP && p.ext_mn, q2_mn = !SWAP && p.ext_mn;

  ptx::grid_launch_dependents();
  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      ptx::mbar_init(&full[s], 1);
      ptx::mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < C::kBufs; ++b) {
      ptx::mbar_init(&acc_full[b], 1);
      ptx::mbar_init(&acc_empty[b], C::kEpi);
    }
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(&sc_full[b], 32);
      ptx::mbar_init(&sc_empty[b], C::kEpi);
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
  const int half = (warp - 4) >> 2;  // column half of an 8-warp epilogue
  bool ok = true;

  // One thread issues all copies and one all MMAs: their loops step the stage, its
  // phase and the descriptors with adds only.  (Dividing by the runtime stage count
  // in them cost 600 and 1100 cycles a block, more than the block's bytes or MMAs.)
  if (warp == 0 && ptx::elect_one()) {
    // ------------------------------------------------------ TMA producer
    auto load_p = [&](int st, uint8_t* dst, int k) {
      if (p_mn)
        ptx::tma_load_2d(&tmP, &full[st], dst, p0, k);
      else
        ptx::tma_load_2d(&tmP, &full[st], dst, k, p0);
    };
    auto load_q = [&](int st, uint8_t* dst, int k) {
      if (q_mn)
        ptx::tma_load_2d(&tmQ, &full[st], dst + kPBytes, q0, k);
      else
        ptx::tma_load_2d(&tmQ, &full[st], dst + kPBytes, k, q0);
    };
    // The launch may start before those ahead of it are done.  Until they are it reads
    // nothing but a B that they do not write: as many of its tiles as there are stages
    // (decoding: often all), so that the weight streams in under their latency.
    const int early = p.b_ready ? min(kn, p.stages) : 0;
    for (int i = 0, k = kb0 * 128; i < early; ++i, k += 128) {
      ptx::mbar_arrive_expect_tx(&full[i], C::kStage);
      if (SWAP)
        load_p(i, smem + i * C::kStage, k);
      else
        load_q(i, smem + i * C::kStage, k);
    }
    ptx::grid_dependency_wait();
    int s = 0, issued = 0;
    uint32_t ph = 1;
    bool go = true;
    uint8_t* sp = smem;
    auto next = [&]() {
      ++issued;
      sp += C::kStage;
      if (++s == p.stages) {
        s = 0;
        ph ^= 1;
        sp = smem;
      }
    };
    for (int i = 0, k = kb0 * 128; i < kn; ++i, k += 128) {
      if (i >= early) {
        go = ptx::mbar_wait(&empty[s], ph, kTimeoutCycles, abort_flag);
        if (!go) break;
        ptx::mbar_arrive_expect_tx(&full[s], C::kStage);
      }
      if (!SWAP || i >= early) load_p(s, sp, k);
      if (SWAP || i >= early) load_q(s, sp, k);
      next();
    }
    for (int t = 0, h = 0; t < ext && go; ++t) {
      go = ptx::mbar_wait(&empty[s], ph, kTimeoutCycles, abort_flag);
      if (!go) break;
      uint8_t* sq = sp + kPBytes;
      ptx::mbar_arrive_expect_tx(&full[s], C::kStage);
      // L columns [64 t, 64 t + 64) of [hi | lo], R at ranks 64 (t mod half)
      const int kl = t * 64, kr = h * 64;
      if (++h == p.ext_half) h = 0;
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
          for (int j = 0; j < (BN + 63) / 64; ++j)
            ptx::tma_load_2d(&tmQ2, &full[s], sq + 8192 * j, q0 + 64 * j, kr);
        } else {
          ptx::tma_load_2d(&tmQ2, &full[s], sq, kr, q0);
        }
      }
      next();
    }
    // never leave with copies in flight into this CTA's shared memory
    for (int i = (issued > p.stages ? issued - p.stages : 0); i < issued; ++i)
      ptx::mbar_wait(&full[i % p.stages], (i / p.stages) & 1, kTimeoutCycles, nullptr);
  } else if (warp == 1 && ptx::elect_one()) {
    // ------------------------------------------------------ MMA issuer
    int s = 0, b = 0;
    uint32_t ph = 0, bph = 1;
    bool go = true;
    // descriptors of stage 0; a stage further is kStage / 16 more (see gemm_tc2.cu)
    const uint32_t p_addr = ptx::smem_u32(smem), q_addr = p_addr + kPBytes;
    // MN-major 8-bit tiles: 128 contraction rows of 128 bytes, 32 rows a step
    const uint64_t pd0 = ptx::sw128_desc(p_addr, p_mn ? kPBytes : 16, 1024);
    const uint64_t qd0 = ptx::sw128_desc(q_addr, q_mn ? kPBytes : 16, 1024);
    const uint64_t ps = p_mn ? (4096 >> 4) : (32 >> 4), qs = q_mn ? (4096 >> 4) : (32 >> 4);
    const uint32_t idesc = p.idesc;
    uint64_t off = 0;
    auto next = [&]() {
      off += C::kStage >> 4;
      if (++s == p.stages) {
        s = 0;
        ph ^= 1;
        off = 0;
      }
    };
    for (int i = 0; i < kn; ++i) {
      go = ptx::mbar_wait(&acc_empty[b], bph, kTimeoutCycles, abort_flag) &&
           ptx::mbar_wait(&full[s], ph, kTimeoutCycles, abort_flag);
      if (!go) break;
      ptx::tc_fence_after();
      const uint32_t d = tmem + b * BN;
      const uint64_t pd = pd0 + off, qd = qd0 + off;
      ptx::umma_f8(d, pd, qd, idesc, 0u);
      ptx::umma_f8(d, pd + ps, qd + qs, idesc, 1u);
      ptx::umma_f8(d, pd + 2 * ps, qd + 2 * qs, idesc, 1u);
      ptx::umma_f8(d, pd + 3 * ps, qd + 3 * qs, idesc, 1u);
      ptx::umma_commit(&empty[s]);
      ptx::umma_commit(&acc_full[b]);
      next();
      if (++b == C::kBufs) {
        b = 0;
        bph ^= 1;
      }
    }
    if (ext && go) {
      // every LoRA stage goes into one accumulator
      go = ptx::mbar_wait(&acc_empty[b], bph, kTimeoutCycles, abort_flag);
      const uint64_t p2d = ptx::sw128_desc(p_addr, p2_mn ? 8192 : 16, 1024);
      const uint64_t q2d = ptx::sw128_desc(q_addr, q2_mn ? 8192 : 16, 1024);
      const uint64_t p2s = p2_mn ? (2048 >> 4) : (32 >> 4), q2s = q2_mn ? (2048 >> 4) : (32 >> 4);
      for (int t = 0, h = 0; t < ext && go; ++t) {
        go = ptx::mbar_wait(&full[s], ph, kTimeoutCycles, abort_flag);
        if (!go) break;
        ptx::tc_fence_after();
        const int steps = ++h == p.ext_half ? p.ext_last_steps : 4;
        if (h == p.ext_half) h = 0;
        for (int ks = 0; ks < steps; ++ks)
          ptx::umma_bf16(tmem + b * BN, p2d + off + p2s * ks, q2d + off + q2s * ks, p.idesc_ext,
                         (t | ks) != 0 ? 1u : 0u);
        ptx::umma_commit(&empty[s]);
        next();
      }
      if (go) ptx::umma_commit(&acc_full[b]);
    }
    if (!go) {
      // gave up: what was issued is done before shared memory and TMEM go
      ptx::umma_commit(drain);
      ptx::mbar_wait(drain, 0, kTimeoutCycles, nullptr);
    }
  } else if (warp == 2) {
    // ------------------------------------------------------ scales
    ptx::grid_dependency_wait();
    for (int kb = 0, c = 0; kb < kn; kb += f8::kChunk, ++c) {
      bool go = ptx::mbar_wait(&sc_empty[c & 1], ((c >> 1) & 1) ^ 1, kTimeoutCycles, abort_flag);
      go = __all_sync(0xffffffffu, go);
      if (!go) break;
      f8::fill_scales(p, ring, c & 1, kb0 + kb, kb0 + kn, SWAP ? q0 : p0, (SWAP ? p0 : q0) >> 7,
                      (p.n + 127) >> 7, lane, &sc_full[c & 1]);
    }
    f8::cp_async_wait_all();
  } else if (warp >= 4) {
    // ------------------------------------------------------ epilogue warps
    const int row = 32 * quarter + lane;  // row of the P tile
    const uint32_t tmem_base = tmem + (static_cast<uint32_t>(32 * quarter) << 16) + half * C::kCols;
    int use = 0;
    auto wait_acc = [&]() {
      ok = ptx::mbar_wait(&acc_full[use % C::kBufs], (use / C::kBufs) & 1, kTimeoutCycles,
                          abort_flag);
      ok = __all_sync(0xffffffffu, ok);
      if (ok) ptx::tc_fence_after();
    };
    auto release_acc = [&]() {
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&acc_empty[use % C::kBufs]);
      ++use;
    };
    // Adds one finished accumulator: each column (SWAP: token) j times s[j] sb with
    // the tokens' scales s in shared memory, or the thread's row times sb.
    uint64_t pairs[SWAP ? 1 : 32];
#pragma unroll
    for (int j = 0; j < (SWAP ? 1 : 32); ++j) pairs[j] = 0ull;
    auto add_block = [&](const float* s, float sb) {
      wait_acc();
      if (!ok) return;
      const uint32_t at = tmem_base + (use % C::kBufs) * BN;
      if (!SWAP) {
        uint32_t r[64];
        ptx::tmem_ld_x64(at, r);
        ptx::tmem_ld_wait(r);
        release_acc();
        f8::add64(pairs, 0, r, sb);
      } else {
        uint32_t r[C::kCols / 16][16];
#pragma unroll
        for (int c = 0; c < C::kCols / 16; ++c) ptx::tmem_ld_x16(at + 16 * c, r[c]);
#pragma unroll
        for (int c = 0; c < C::kCols / 16; ++c) ptx::tmem_ld_wait(r[c]);
        release_acc();
#pragma unroll
        for (int j = 0; j < C::kCols; j += 4) {
          float4 f = make_float4(1.0f, 1.0f, 1.0f, 1.0f);
          if (s) f = *reinterpret_cast<const float4*>(s + j);  // one address for all lanes
          acc[j] = fmaf(__uint_as_float(r[j / 16][j % 16]), f.x * sb, acc[j]);
          acc[j + 1] = fmaf(__uint_as_float(r[j / 16][j % 16 + 1]), f.y * sb, acc[j + 1]);
          acc[j + 2] = fmaf(__uint_as_float(r[j / 16][j % 16 + 2]), f.z * sb, acc[j + 2]);
          acc[j + 3] = fmaf(__uint_as_float(r[j / 16][j % 16 + 3]), f.w * sb, acc[j + 3]);
        }
      }
    };
    for (int k0 = 0, chunk = 0; k0 < kn && ok; k0 += f8::kChunk, ++chunk) {
      const int slot = chunk & 1;
      ok = ptx::mbar_wait(&sc_full[slot], (chunk >> 1) & 1, kTimeoutCycles, abort_flag);
      ok = __all_sync(0xffffffffu, ok);
      const int n = min(f8::kChunk, kn - k0);
      float sa = SWAP ? 1.0f : ring->a[slot][0][row], sb = ring->b[slot][0][0];
      for (int i = 0; i < n && ok; ++i) {
        const float s = sa * sb;
        // the next block's scales (the last read of a chunk is not used)
        const int ni = min(i + 1, f8::kChunk - 1);
        if (!SWAP) sa = ring->a[slot][ni][row];
        sb = ring->b[slot][ni][0];
        add_block(ring->a[slot][i], s);
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&sc_empty[slot]);
    }
    if (ext && ok) add_block(nullptr, 1.0f);  // the LoRA term
    if (!SWAP) {
#pragma unroll
      for (int j = 0; j < 32; ++j)
        asm("mov.b64 {%0, %1}, %2;"
            : "=f"(acc[(2 * j) % C::kCols]), "=f"(acc[(2 * j + 1) % C::kCols])
            : "l"(pairs[SWAP ? 0 : j]));
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
    if (warp >= 4) {
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

// Contraction splits for `tiles` output tiles on `slots` CTAs: as many as run at
// once (a cluster holds at most 8), at least 4 blocks each.  (More splits than fit at
// once never pay: clusters wait for whole groups of free SMs.  64 x 11008 x 4096, 86
// tiles on 148 SMs: 14 us unsplit, 40 us in 5 splits.)
int split_count(int64_t tiles, int64_t kb, int64_t slots) {
  const int64_t s = std::min<int64_t>({8, slots / tiles, kb / 4});
  return static_cast<int>(std::max<int64_t>(1, s));
}

template <int BN, bool SWAP>
qlora_status launch(const qlora_f8& a, const qlora_f8& b, bool trans_b, GemmArgs p,
                    const F8Lora& l, cudaStream_t s) {
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
  const int64_t p_tiles = ceil_div(SWAP ? n : m, 128), q_tiles = ceil_div(SWAP ? m : n, BN);
  p.n_tiles = static_cast<int32_t>(q_tiles);
  if (p_tiles * q_tiles > 0x7fffffff) return QLORA_ERR_SHAPE;
  const void* fn = reinterpret_cast<const void*>(f8_gemm_kernel<BN, SWAP>);
  const qlora_status cs = ensure_smem(fn, 220 * 1024);
  if (cs != QLORA_OK) return cs;
  const int sms = f8::sm_count();
  const int64_t tiles = p_tiles * q_tiles;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(C::kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 1;
  attr[0].val.clusterDim.y = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  for (int splits = split_count(tiles, p.kb_total, C::kPerSm * sms);; --splits) {
    p.kb_per = static_cast<int32_t>(ceil_div(p.kb_total, splits));
    // the stages that fit beside as many CTAs as an SM gets; no more than a split has blocks
    const int64_t want = p.kb_per + p.ext_tiles;
    const bool two = C::kPerSm == 2 && tiles * splits > sms;
    p.stages = static_cast<int32_t>(
        std::min<int64_t>({kMaxStages, want, ((two ? 100 : 200) * 1024) / C::kStage}));
    cfg.gridDim = dim3(static_cast<unsigned>(tiles), 1, static_cast<unsigned>(splits));
    cfg.dynamicSmemBytes =
        1024 + std::max(p.stages * C::kStage, C::kRedBytes) + sizeof(typename C::Ring) + 512;
    attr[0].val.clusterDim.z = static_cast<unsigned>(splits);
    // A cluster lies within one group of SMs, so of size 8 at one CTA per SM fewer than 16
    // run at once: 256 x 1024 x 4096, 16 tiles, took 14.2 us in 8 splits and takes 7.9 in
    // as many as do.  Two CTAs per SM read for one another while some wait: 16 x 11008 x
    // 4096, 86 tiles, 7.8 us in 3 splits, 10.3 in the 2 that would all be resident.
    if (C::kPerSm == 2 || splits == 1 || tiles <= f8_resident_clusters(fn, cfg)) break;
  }
  count_launch();
  const cudaError_t e = cudaLaunchKernelEx(&cfg, f8_gemm_kernel<BN, SWAP>, SWAP ? mb : ma,
                                           SWAP ? ma : mb, SWAP ? mr : ml, SWAP ? ml : mr, p);
  if (e != cudaSuccess) {
    (void)cudaGetLastError();
    return QLORA_ERR_CUDA;
  }
  return after_launch("f8_gemm", s);
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
  p.b_ready = l.b_ready ? 1 : 0;
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
  if (m <= 16) return launch<16, true>(a, b, trans_b, p, l, s);
  if (m <= 32) return launch<32, true>(a, b, trans_b, p, l, s);
  // whichever ends soonest: rounds of tiles times what a 128-deep block of a tile takes
  // (0.32 us for 128 x 128 on a CTA, 0.46 for 256 x 256 on a pair, 0.28 for 256 x 192 on a
  // pair with power-of-two scales).  At k = 4096: 384 x 11008 in 26 us on CTAs, 42 on
  // pairs; 4096 x 4096 in 112, 70 and 52 us; 1024 x 4096 in 21 on pairs, 22.5 as powers.
  const int sms = f8::sm_count();
  const int64_t tiles = ceil_div(n, 128) * ceil_div(m, 128), m2 = ceil_div(m, 256);
  if (tiles > sms) {
    const int64_t pairs = sms / 2;
    const int64_t one = 32 * ceil_div(tiles, sms);
    const int64_t two = 46 * ceil_div(m2 * ceil_div(n, 256), pairs);
    const int64_t pow2 = 28 * ceil_div(m2 * ceil_div(n, 192), pairs);
    if (a.pow2 && b.pow2 && pow2 < std::min(one, two))
      return f8_gemm_pow2(a, b, trans_b, c, c_f32, l, s);
    if (two < one) return f8_gemm_pairs(a, b, trans_b, c, c_f32, l, s);
  }
  return launch<128, false>(a, b, trans_b, p, l, s);
}

int f8_resident_clusters(const void* fn, const cudaLaunchConfig_t& cfg) {
  // one answer per kernel, device, cluster size and KB of shared memory
  const int tag = 16 + static_cast<int>(cfg.gridDim.z) +
                  256 * static_cast<int>(cfg.dynamicSmemBytes >> 10);
  int n = 0;
  if (cached_value(fn, tag, &n)) return n;
  if (cudaOccupancyMaxActiveClusters(&n, fn, &cfg) != cudaSuccess) {
    (void)cudaGetLastError();
    n = 0;
  }
  store_value(fn, tag, n);
  return n;
}

int f8::sm_count() {
  int dev = 0, sms = 148;
  if (cudaGetDevice(&dev) == cudaSuccess)
    (void)cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return sms;
}

}  // namespace qlora
