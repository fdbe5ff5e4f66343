// dA = s V^T X^ from an input X that was kept in 8 bits (by rows): the one product
// of the backward pass that reads X.
//
//   dA[j][k] = s sum_m V[m][j] X^[m][k],   X^[m][k] = bf16(code[m][k] scale[k / 128][m])
//
// It cannot do without the read of the codes, one byte per element of X.  The scale
// changes along the contraction (m), so it has to be applied to an operand: the
// codes are expanded to bf16 on their way into the tensor core's operand tiles,
// as the restored activations would be, and no bf16 copy of X is written.
//
// Bound by latency: a tile's way through load, expansion and MMAs two stages deep, the start
// and the sum across the cluster.  Cold, 4096 x 4096 at rank 16 in 18.5 us: 17.7 MB from DRAM
// (15% of HBM), tensor pipe 4% and issue 17% active; 2048 x 8192 at rank 64 20 us, 14% and 25%.
// Above rank 64 V's terms from L2, 6 bytes a rank and token for each 128 columns, weigh too.
//
// More than 16 tokens: D = X^T V^T per 128 columns of X on the tensor cores
// (tcgen05.mma kind::f16, M = 128, N = rc ranks <= 128), the contraction split over a cluster
// and summed in distributed shared memory in split order, as in gemm_rank.cu.  V is fp32: it
// enters as three bf16 terms (24 bits; two would leave dA off by 2.5e-6 relative).  Sums in
// TMEM are cut off, not rounded, which adds up along a chain of MMAs: the first term's
// products go tile by tile in turn into as many accumulators as keep its chains at 16 MMAs
// (256 tokens), as far as TMEM goes, the small products of the other two into one more, and
// tokens past 48 MMAs a chain (64 above rank 64) are a launch of their own that adds to dA.
// Relative to fp64 at rank 16, 4096 columns: 4096 tokens 4.3e-7, 65536 8.8e-7 (2.7e-6 and
// 2.0e-5 with two terms in one accumulator and launch).
//
// Roles (384 threads): warp 0 loads codes, warp 2 loads V^T, warp 1 owns TMEM and issues the
// MMAs, warps 4-11 expand in two groups (group g takes 64-token tiles i % 2 == g) and drain.
// Every wait is bounded; a wait that gives up reports QLORA_ERR_DEVICE_TIMEOUT and leaves NaN
// in its columns of dA.
//
// Up to 16 tokens: CUDA cores, bound by writing dA; a thread takes 16 columns of 4
// ranks, so that each code is expanded once for 4 ranks.
#include <cudaTypedefs.h>

#include <algorithm>

#include "f8.cuh"
#include "f8_splits.cuh"
#include "linear.cuh"
#include "tc_common.cuh"
#include "tc_ptx.cuh"

namespace qlora {
namespace {

constexpr int kThreads = 384;
constexpr int kABytes = 16384;     // 64 tokens x 128 columns in bf16, two 64-column halves
constexpr int kCodeBytes = 8192;   // 64 tokens x 128 codes
// even numbers: a slot's tiles all go to the same group, which has seen every phase of the
// barriers that it waits on
constexpr int kCodeSlots = 4;
constexpr int kStages = 2;
static_assert(kCodeSlots % 2 == 0 && kStages % 2 == 0, "each slot and stage has one group");
constexpr int kMaxVStages = 8;
// Shared memory beside the tiles: their alignment to 1024 bytes from 128, and two words and
// the barriers, of which those that free a stage of V are A's where both have two stages (at
// rank 64 two CTAs then fit an SM to the byte).
constexpr int kAlignSlack = 1024 - 128;
constexpr int barrier_bytes(int v_stages) {
  return 8 + 8 * (2 * kCodeSlots + 2 * kStages + 1 + (v_stages == kStages ? 1 : 2) * v_stages);
}
static_assert(barrier_bytes(kStages) == 128, "see above");
constexpr int kTerms = 3;          // of V
constexpr long long kTimeoutCycles = 4000000000ll;

struct GradArgs {
  const float* scales;   // [kb][m]
  int32_t m, k;          // tokens, columns of X
  int32_t kt0, kt_end, kt_per;  // 64-token tiles of this launch, tiles per split
  int32_t r, rc, lo_row;     // rank, ranks per chunk (a multiple of 16), rows of a term of V^T
  int32_t v_stages;      // of V^T tiles
  int32_t area;          // bytes of the tiles (the partial sums reuse them)
  int32_t accs, tmem_cols;   // accumulators of the first term (a power of two), TMEM columns
  float* dA;
  float sc;
  int32_t accumulate;
  uint32_t idesc;
  DeviceStatus* st;
};

// 4 codes times a scale as 4 bf16
template <bool E5M2>
__device__ __forceinline__ uint2 expand4(uint32_t c, float s) {
  constexpr __nv_fp8_interpretation_t kF = E5M2 ? __NV_E5M2 : __NV_E4M3;
  const float2 a = __half22float2(__half2(
      __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(c & 0xffffu), kF)));
  const float2 b = __half22float2(
      __half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(c >> 16), kF)));
  return make_uint2(tc::pack_bf16x2(__fmul_rn(a.x, s), __fmul_rn(a.y, s)),
                    tc::pack_bf16x2(__fmul_rn(b.x, s), __fmul_rn(b.y, s)));
}

template <bool E5M2>
__global__ void __launch_bounds__(kThreads, 2)
f8_grad_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmV,
               const GradArgs p) {
  extern __shared__ __align__(128) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  // [kStages x A] [codes] [v_stages x V^T], reused as the fp32 partial sums
  const int v_bytes = kTerms * p.rc * 128;
  uint8_t* codes = smem + kStages * kABytes;
  uint8_t* vtile = codes + kCodeSlots * kCodeBytes;
  float* red = reinterpret_cast<float*>(smem);  // [rc][132]: 128 columns of X each
  constexpr int kRedLd = 132;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + p.area);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  uint64_t* code_full = reinterpret_cast<uint64_t*>(tmem_slot + 2);
  uint64_t* code_empty = code_full + kCodeSlots;
  uint64_t* full_a = code_empty + kCodeSlots;
  uint64_t* empty = full_a + kStages;
  uint64_t* accum = empty + kStages;
  uint64_t* full_b = accum + 1;
  const bool shared = p.v_stages == kStages;  // one barrier frees A's and V's stage
  uint64_t* empty_b = shared ? empty : full_b + p.v_stages;

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t S = gridDim.z, z = blockIdx.z;
  const int kb = blockIdx.x, k0 = kb * 128;
  const int j0 = blockIdx.y * p.rc;  // first rank of the chunk
  const int t0 = p.kt0 + static_cast<int>(z) * p.kt_per;
  const int tn = max(0, min(p.kt_per, p.kt_end - t0));

  if (threadIdx.x == 0) {
    for (int s = 0; s < kCodeSlots; ++s) {
      ptx::mbar_init(&code_full[s], 1);
      ptx::mbar_init(&code_empty[s], 4);
    }
    for (int s = 0; s < kStages; ++s) {
      ptx::mbar_init(&full_a[s], 4);
      ptx::mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < p.v_stages; ++s) {
      ptx::mbar_init(&full_b[s], 1);
      if (!shared) ptx::mbar_init(&empty_b[s], 1);
    }
    ptx::mbar_init(accum, 1);
    *abort_flag = 0;
    ptx::fence_mbar_init();
    ptx::prefetch_tmap(&tmX);
    ptx::prefetch_tmap(&tmV);
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
    // ------------------------------------------------------ codes
    int issued = 0;
    for (int i = 0; i < tn; ++i) {
      const int s = i % kCodeSlots;
      if (!ptx::mbar_wait(&code_empty[s], ((i / kCodeSlots) & 1) ^ 1, kTimeoutCycles, abort_flag))
        break;
      ptx::mbar_arrive_expect_tx(&code_full[s], kCodeBytes);
      ptx::tma_load_2d(&tmX, &code_full[s], codes + s * kCodeBytes, k0, (t0 + i) * 64);
      ++issued;
    }
    // never leave with copies in flight into this CTA's shared memory
    for (int i = (issued > kCodeSlots ? issued - kCodeSlots : 0); i < issued; ++i)
      ptx::mbar_wait(&code_full[i % kCodeSlots], (i / kCodeSlots) & 1, kTimeoutCycles, nullptr);
  } else if (warp == 2 && ptx::elect_one()) {
    // ------------------------------------------------------ V^T: the chunk's rows of each term
    int issued = 0, s = 0;
    uint32_t ph = 1;
    for (int i = 0; i < tn; ++i) {
      if (!ptx::mbar_wait(&empty_b[s], ph, kTimeoutCycles, abort_flag)) break;
      uint8_t* sv = vtile + s * v_bytes;
      ptx::mbar_arrive_expect_tx(&full_b[s], v_bytes);
#pragma unroll
      for (int t = 0; t < kTerms; ++t)
        ptx::tma_load_2d(&tmV, &full_b[s], sv + t * p.rc * 128, (t0 + i) * 64, t * p.lo_row + j0);
      ++issued;
      if (++s == p.v_stages) {
        s = 0;
        ph ^= 1;
      }
    }
    // (none of these is more than v_stages back)
    for (int i = (issued > p.v_stages ? issued - p.v_stages : 0); i < issued; ++i)
      ptx::mbar_wait(&full_b[i % p.v_stages], (i / p.v_stages) & 1, kTimeoutCycles, nullptr);
  } else if (warp == 1 && ptx::elect_one()) {
    // ------------------------------------------------------ MMA issuer
    const uint64_t term = static_cast<uint64_t>(p.rc * 128) >> 4;
    const uint32_t rest = tmem + p.accs * p.rc;
    // A: MN-major, two 64-column halves 8192 bytes apart, 16 tokens (2048 bytes) a step
    const uint64_t a0 = ptx::sw128_desc(ptx::smem_u32(smem), 8192, 1024);
    const uint64_t b0 = ptx::sw128_desc(ptx::smem_u32(vtile), 16, 1024);
    int vs = 0;
    uint32_t vph = 0;
    uint64_t off = 0;
    for (int i = 0; i < tn; ++i) {
      const int s = i % kStages;
      if (!ptx::mbar_wait(&full_b[vs], vph, kTimeoutCycles, abort_flag) ||
          !ptx::mbar_wait(&full_a[s], (i / kStages) & 1, kTimeoutCycles, abort_flag))
        break;
      ptx::tc_fence_after();
      const uint64_t ad = a0 + s * (kABytes >> 4), bd = b0 + off;
      const uint32_t d = tmem + (i & (p.accs - 1)) * p.rc;
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) {
        const uint64_t a = ad + ((2048 * ks) >> 4), b = bd + ((32 * ks) >> 4);
        ptx::umma_bf16(d, a, b, p.idesc, i >= p.accs || ks != 0 ? 1u : 0u);
        ptx::umma_bf16(rest, a, b + term, p.idesc, (i | ks) != 0 ? 1u : 0u);
        ptx::umma_bf16(rest, a, b + 2 * term, p.idesc, 1u);
      }
      ptx::umma_commit(&empty[s]);
      if (!shared) ptx::umma_commit(&empty_b[vs]);
      off += v_bytes >> 4;
      if (++vs == p.v_stages) {
        vs = 0;
        vph ^= 1;
        off = 0;
      }
    }
    ptx::umma_commit(accum);
    ptx::mbar_wait(accum, 0, kTimeoutCycles, nullptr);  // MMAs done before TMEM is freed
  } else if (warp >= 4) {
    // ------------------------------------------------------ expansion
    const int grp = (warp - 4) >> 2, td = (threadIdx.x - 128) & 127;
    const int row = td & 63, h = td >> 6;  // token of the tile, half of its 128 columns
    const float* sx = p.scales + static_cast<int64_t>(kb) * p.m;
    auto scale_at = [&](int i) -> float {  // clamped: codes past the last token are zero
      return __ldg(sx + min((t0 + i) * 64 + row, p.m - 1));
    };
    float next = grp < tn ? scale_at(grp) : 0.0f;
    for (int i = grp; i < tn; i += 2) {
      const int s = i % kCodeSlots, st = i % kStages;
      if (!ptx::mbar_wait(&code_full[s], (i / kCodeSlots) & 1, kTimeoutCycles, abort_flag)) break;
      const uint8_t* src = codes + s * kCodeBytes + row * 128;
      uint4 c[4];
#pragma unroll
      for (int q = 0; q < 4; ++q)
        c[q] = *reinterpret_cast<const uint4*>(src + 16 * ((4 * h + q) ^ (row & 7)));
      const float sc = next;
      if (i + 2 < tn) next = scale_at(i + 2);
      // the next copy into the slot writes through the async proxy: order these
      // reads before it, then release the slot
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&code_empty[s]);
      uint4 o[8];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint2 e0 = expand4<E5M2>(c[q].x, sc), e1 = expand4<E5M2>(c[q].y, sc);
        const uint2 e2 = expand4<E5M2>(c[q].z, sc), e3 = expand4<E5M2>(c[q].w, sc);
        o[2 * q] = make_uint4(e0.x, e0.y, e1.x, e1.y);
        o[2 * q + 1] = make_uint4(e2.x, e2.y, e3.x, e3.y);
      }
      if (!ptx::mbar_wait(&empty[st], ((i / kStages) & 1) ^ 1, kTimeoutCycles, abort_flag)) break;
      uint8_t* dst = smem + st * kABytes + h * 8192 + row * 128;
#pragma unroll
      for (int j = 0; j < 8; ++j) *reinterpret_cast<uint4*>(dst + 16 * (j ^ (row & 7))) = o[j];
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&full_a[st]);
    }
  }
  __syncthreads();
  // ---------------------------------------- partial sums to shared memory, transposed
  if (warp >= 4) {
    const int i = 32 * (warp & 3) + lane;  // column of X in the tile
    bool ok = tn > 0 && ptx::mbar_wait(accum, 0, kTimeoutCycles, abort_flag);
    ok = __all_sync(0xffffffffu, ok && !*abort_flag);
    if (ok) ptx::tc_fence_after();
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
    const int used = min(p.accs, tn);
    for (int c = 16 * ((warp - 4) >> 2); c < p.rc; c += 32) {
      float v[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) v[j] = 0.0f;
      // the small products first
      for (int a = used; ok && a >= 0; --a) {
        uint32_t r[16];
        ptx::tmem_ld_x16(lane_base + (a == used ? p.accs : a) * p.rc + c, r);
        ptx::tmem_ld_wait(r);
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] += __uint_as_float(r[j]);
      }
#pragma unroll
      for (int j = 0; j < 16; ++j) red[(c + j) * kRedLd + i] = v[j];
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  // a wait of this CTA gave up: its sums are not whole (the status word may not be read)
  if (*abort_flag)
    for (int e = threadIdx.x; e < p.rc * kRedLd; e += kThreads)
      red[e] = __int_as_float(0x7fffffff);
  ptx::cluster_sync();
  // ---------------------------------------- sum over the splits, in order
  const int cols = min(p.rc, p.r - j0);
  for (int e = static_cast<int>(z) * kThreads + threadIdx.x; e < cols * 128;
       e += static_cast<int>(S) * kThreads) {
    const int j = e >> 7, i = e & 127;
    if (k0 + i >= p.k) continue;
    float v = 0.0f;
#pragma unroll
    for (uint32_t q = 0; q < 8; ++q) {
      if (q < S) {
        v += ptx::ld_cluster_f32(ptx::cluster_addr(red, q) + 4u * (j * kRedLd + i));
      }
    }
    float* dst = p.dA + static_cast<int64_t>(j0 + j) * p.k + k0 + i;
    *dst = p.accumulate ? *dst + p.sc * v : p.sc * v;
  }
  // no CTA leaves (or frees TMEM) while the others may still read its sums
  __syncthreads();
  ptx::cluster_sync();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, p.tmem_cols);
  }
  if (threadIdx.x == 0 && *abort_flag) report(p.st, QLORA_ERR_DEVICE_TIMEOUT, 140u);
}

// ------------------------------------------------------------ up to 16 tokens
template <int MM, bool E5M2>
__global__ void __launch_bounds__(128)
f8_grad_small_kernel(const uint8_t* __restrict__ codes, const float* __restrict__ scales,
                     int64_t ld, int M, int K, const float* __restrict__ V, int r, float sc,
                     int accumulate, float* __restrict__ dA) {
  const int k16 = (K + 15) / 16;
  const int e = blockIdx.x * 128 + threadIdx.x;
  if (e >= k16) return;
  const int k = 16 * e, j = 4 * blockIdx.y;  // 16 columns, 4 ranks
  const float* sx = scales + static_cast<int64_t>(k >> 7) * M;
  float acc[4][16];
#pragma unroll
  for (int q = 0; q < 4; ++q)
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[q][i] = 0.0f;
#pragma unroll
  for (int m = 0; m < MM; ++m) {
    if (m >= M) break;
    const uint4 c = __ldg(reinterpret_cast<const uint4*>(codes + m * ld + k));
    const float s = __ldg(sx + m);
    const float4 v = __ldg(reinterpret_cast<const float4*>(V + m * r + j));
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint2 b = expand4<E5M2>(w[q], s);
      const float x[4] = {__uint_as_float(b.x << 16), __uint_as_float(b.x & 0xffff0000u),
                          __uint_as_float(b.y << 16), __uint_as_float(b.y & 0xffff0000u)};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[0][4 * q + i] = fmaf(v.x, x[i], acc[0][4 * q + i]);
        acc[1][4 * q + i] = fmaf(v.y, x[i], acc[1][4 * q + i]);
        acc[2][4 * q + i] = fmaf(v.z, x[i], acc[2][4 * q + i]);
        acc[3][4 * q + i] = fmaf(v.w, x[i], acc[3][4 * q + i]);
      }
    }
  }
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    float* dst = dA + static_cast<int64_t>(j + q) * K + k;
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      if (k + i >= K) continue;  // K is a multiple of 8
      float4 o = make_float4(sc * acc[q][i], sc * acc[q][i + 1], sc * acc[q][i + 2],
                             sc * acc[q][i + 3]);
      if (accumulate) {
        const float4 d = *reinterpret_cast<const float4*>(dst + i);
        o = make_float4(d.x + o.x, d.y + o.y, d.z + o.z, d.w + o.w);
      }
      *reinterpret_cast<float4*>(dst + i) = o;
    }
  }
}

template <int MM>
void launch_small(const qlora_f8& x, const float* V, int r, float sc, int acc, float* dA,
                  cudaStream_t s) {
  const int K = static_cast<int>(x.cols), M = static_cast<int>(x.rows);
  const dim3 grid(static_cast<unsigned>(ceil_div(ceil_div(K, 16), 128)), r / 4);
  if (x.format == QLORA_E5M2)
    f8_grad_small_kernel<MM, true><<<grid, 128, 0, s>>>(x.codes, x.scales, x.ld, M, K, V, r, sc,
                                                        acc, dA);
  else
    f8_grad_small_kernel<MM, false><<<grid, 128, 0, s>>>(x.codes, x.scales, x.ld, M, K, V, r, sc,
                                                         acc, dA);
}

}  // namespace

qlora_status f8_small_grad_a(const float* V, const qlora_f8& x, int r, float sc, bool accumulate,
                             float* dA, cudaStream_t s) {
  if (x.rows < 1 || x.rows > kSmallM || x.cols % 8 != 0 || r % 8 != 0) return QLORA_ERR_UNSUPPORTED;
  const int acc = accumulate ? 1 : 0;
  count_launch();
  if (x.rows == 1) launch_small<1>(x, V, r, sc, acc, dA, s);
  else if (x.rows <= 4) launch_small<4>(x, V, r, sc, acc, dA, s);
  else launch_small<16>(x, V, r, sc, acc, dA, s);
  return after_launch("f8_small_grad_a", s);
}

qlora_status f8_grad_a(const void* vt, int64_t ld_v, const qlora_f8& x, int32_t r, float sc,
                       bool accumulate, float* dA, DeviceStatus* st, cudaStream_t s) {
  const int64_t M = x.rows, K = x.cols;
  const int32_t r16 = lora_rows(r);
  GradArgs p{};
  const int chunks = r16 > 128 ? 2 : 1;
  p.rc = static_cast<int32_t>(ceil_div(r16, 16 * chunks) * 16);
  CUtensorMap mx, mv;
  if (!make_map(&mx, x.codes, false, K, M, x.ld, 128, 64, true) ||
      !make_map(&mv, vt, true, M, 2 * r16 + r, ld_v, 64, static_cast<uint32_t>(p.rc), true))
    return QLORA_ERR_CUDA;
  p.scales = x.scales;
  p.m = static_cast<int32_t>(M);
  p.k = static_cast<int32_t>(K);
  p.r = r;
  p.lo_row = r16;
  p.dA = dA;
  p.sc = sc;
  p.idesc = ptx::idesc_bf16(128, p.rc, 1, 0);
  p.st = st;
  const bool e5 = x.format == QLORA_E5M2;
  auto* fn = e5 ? f8_grad_kernel<true> : f8_grad_kernel<false>;
  const void* kernel = reinterpret_cast<const void*>(fn);
  const qlora_status cs = ensure_smem(kernel, kCtaMaxSmem);
  if (cs != QLORA_OK) return cs;
  // Two CTAs an SM where two stages of V fit beside the rest, else one; as many stages as do.
  // TMEM columns likewise: half of them where two share an SM.
  constexpr int kFixed = kStages * kABytes + kCodeSlots * kCodeBytes;
  const int v_bytes = kTerms * p.rc * 128;
  auto need = [&](int stages) {
    p.area = std::max(kFixed + stages * v_bytes, p.rc * 132 * 4);
    return kAlignSlack + p.area + barrier_bytes(stages);
  };
  const bool two = need(kStages) <= kCtaHalfSmem;
  p.v_stages = kMaxVStages;
  while (need(p.v_stages) > (two ? kCtaHalfSmem : kCtaMaxSmem)) --p.v_stages;
  const int smem = need(p.v_stages);
  int max_accs = 1;
  while ((2 * max_accs + 1) * p.rc <= (two ? 256 : 512)) max_accs *= 2;
  const int64_t kt_total = ceil_div(M, 64);
  const int64_t tiles = ceil_div(K, 128);
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
    cfg.dynamicSmemBytes = std::max(smem, p.tmem_cols * kSmemPerColumn - 1024);
    attr[0].val.clusterDim.z = static_cast<unsigned>(n);
    cfg.gridDim = dim3(static_cast<unsigned>(tiles), chunks, n);
  };
  // Splits of the tokens, at least 4 tiles each: whichever ends soonest.  In tenths of a tile's
  // time a launch takes 60 and, a round of clusters that run at once, 10 a tile (17 where two
  // CTAs share an SM), 40 for the start and 6 a split for the sum.  Backward without dX, d_in
  // 4096, rank 16, in 4 and in 8 splits: 4096 tokens 34.4 and 33.7 us, 8192 57.3 and 52.7;
  // 2048 at rank 64 34.1 and 34.6; d_in 2048, rank 128, 4096 tokens, in 6 and 8 (two
  // rounds) 66.4 and 76.6; d_in 8192, rank 256, 8192 tokens in one launch of 4 and in four of
  // 1 437 and 470.
  int splits = 1;
  int64_t launches = 1;
  choose_splits(kernel, cfg, tiles * chunks, kt_total, 4, two, max_accs, SplitCost{17, 40, 6, 60},
                plan, &splits, &launches);
  const int64_t each = ceil_div(kt_total, launches);
  plan(splits, ceil_div(each, splits));
  for (int64_t kt0 = 0; kt0 < kt_total; kt0 += each) {
    p.kt0 = static_cast<int32_t>(kt0);
    p.kt_end = static_cast<int32_t>(std::min(kt_total, kt0 + each));
    p.accumulate = accumulate || kt0 > 0 ? 1 : 0;
    count_launch();
    timing_mark(QLORA_KERNEL_LORA_GEMM, s, true);
    const cudaError_t e = cudaLaunchKernelEx(&cfg, fn, mx, mv, p);
    timing_mark(QLORA_KERNEL_LORA_GEMM, s, false);
    if (e != cudaSuccess) {
      (void)cudaGetLastError();
      return QLORA_ERR_CUDA;
    }
    QLORA_TRY(after_launch("f8_grad_a", s));
  }
  return QLORA_OK;
}

}  // namespace qlora
