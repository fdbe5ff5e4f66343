// What the 8-bit layer needs of X (or dY) before its product, for up to a few hundred
// tokens, in one launch: 8 bits by rows (definitions: f8_quantize.cu) and the LoRA factor
//   U[m][j] = sum_k X[m][k] A[j][k]       V[m][j] = sum_k dY[m][k] B[k][j]  (ALONG)
// as fp32, as the product's operand, s U in bf16 [hi | lo], and transposed for dA.
//
// A warp takes a block of 128 columns of 16 tokens (one 16-byte load per row and 32
// columns and lane) and 16 ranks of the other operand, all loads before the first use.
// The same registers give the block's scale (two shuffles across the four lanes of a
// row), its codes, and the operands of the matrix instructions: a lane's 8 consecutive
// columns are taken as columns 2t, 2t+1, 2t+8, 2t+9 of two steps, for both operands alike,
// which only reorders the sum.  B's rows are turned by ldmatrix on the way.  The
// contraction is spread over the warps of up to 8 CTAs of a cluster, the partial sums are
// added in a fixed order (warps, then CTAs).
//
// Bound by latency: one load from HBM or L2, the sum across the cluster and the launch.
// Forward of the layer, per call in a sequence, against the two launches of the NF4
// layer's rank product and the quantiser: 8 x 4096 x 11008 at rank 64 in 14.3 us (19.3),
// 16 x 8192 x 8192 in 18.3 (23.8), 8 x 4096 x 4096 at rank 16 in 10.0 (11.3), one token
// of it in 9.5 (9.2); the product alone takes 11.5, 14.8, 7.4 and 6.5.  Backward of 16 x
// 8192 x 8192 in 25.4 (30.3), 24 x 4096 x 4096 at rank 16 in 20.0 (23.9).
// (16 tokens x 16 ranks x 128 columns are 16 matrix instructions of mma.sync, done
// between the loads' arrivals; tcgen05 would need the operands in shared memory first.)
#pragma once

#include "f8.cuh"
#include "f8_codec.cuh"
#include "tc_ptx.cuh"

namespace qlora {
namespace {

constexpr int kMaxWarps = 16;
constexpr int kMaxCtas = 8;
constexpr int kRanks = 16;  // per CTA

struct FrontArgs {
  const __nv_bfloat16* x;  // M x K
  const __nv_bfloat16* a;  // r x K, or K x r (ALONG)
  uint8_t* codes;          // NULL: no 8 bits wanted
  float* scales;           // [kb][M]
  int64_t k, ld, m;
  int32_t r, kbs, per;     // 128-column blocks, blocks per CTA
  int32_t tiles;           // 16-token tiles per CTA (warps w, w + tiles, ... share one)
  int32_t pow2, span;
  float* u;                // M x r or NULL
  __nv_bfloat16* su;       // M x [span | span]
  float sc;
  __nv_bfloat16* ut;       // ALONG: U^T as three terms or NULL: rows of ut_ld, terms ut_lo rows apart
  int64_t ut_ld;
  int32_t ut_lo;
};

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Four 8 x 8 tiles of shared memory, rows along the contraction: a lane receives
// contraction rows 2t, 2t + 1 of column g of each.
__device__ __forceinline__ void load_tiles_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// Byte offset of row `pos` of an 8 x 8 tile among those of 32 contraction rows i, half h:
// tile (e, n) holds rows 8t + 4h + 2e + {0, 1} (pos = 2t, 2t + 1) of ranks 8n .. 8n + 7.
// The exclusive or spreads the stores of neighbouring rows over the banks.
__device__ __forceinline__ int tile_offset(int i, int h, int e, int n, int pos) {
  return 1024 * i + 512 * h + 256 * e + 128 * n + 16 * (pos ^ (2 * (n + 2 * e)));
}

// A block of the second operand whose rows run along the contraction, as a lane's loads
// bring it, turned into operands through 2 KB of the warp's, 64 rows at a time.
constexpr int kTurnBytes = 2048;
__device__ __forceinline__ void turn_tiles(uint32_t (&a)[2][16], uint8_t* mine, int lane) {
  const uint32_t base = ptx::smem_u32(mine);
#pragma unroll
  for (int s = 0; s < 4; s += 2) {
    __syncwarp();  // the rows before have been read
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const int k = 16 * n + (lane >> 1);  // of the 32
        const int at =
            tile_offset(i, (k >> 2) & 1, (k >> 1) & 1, lane & 1, 2 * (k >> 3) + (k & 1));
        const uint32_t* w = &a[n][4 * (s + i)];
        *reinterpret_cast<uint4*>(mine + at) = make_uint4(w[0], w[1], w[2], w[3]);
      }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t b[4];  // (e, n) = (0, 0), (1, 0), (0, 1), (1, 1)
        load_tiles_t(base + tile_offset(i, h, (lane >> 3) & 1, lane >> 4, lane & 7), b);
        const int at = 4 * (s + i) + 2 * h;
        a[0][at] = b[0];
        a[0][at + 1] = b[1];
        a[1][at] = b[2];
        a[1][at + 1] = b[3];
      }
  }
}

__device__ __forceinline__ float word_value(uint32_t w, int half) {
  return __uint_as_float(half ? (w & 0xffff0000u) : (w << 16));
}

// TWO: more than 8 tokens (a lane holds rows g and g + 8).  ALONG: the second operand's
// rows run along the contraction (V = dY B): it passes through shared memory.
template <bool E5M2, bool TWO, bool ALONG>
__global__ void __launch_bounds__(32 * kMaxWarps) f8_front_kernel(const FrontArgs p) {
  // the product may start: it reads what this launch writes after its own wait
  ptx::grid_launch_dependents();
  constexpr int kHalves = TWO ? 2 : 1;
  using Red = float[16][kRanks + 1];
  __shared__ __align__(128) uint8_t area[kMaxWarps * (ALONG ? kTurnBytes : sizeof(Red))];
  Red* red = reinterpret_cast<Red*>(area);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int tile = warp % p.tiles, slice = warp / p.tiles;
  const int slices = static_cast<int>(blockDim.x >> 5) / p.tiles;
  const int64_t tile0 = static_cast<int64_t>(blockIdx.z) * p.tiles;
  const int64_t row0 = 16 * (tile0 + tile);
  const int j0 = blockIdx.y * kRanks;
  const int kb_end = min(static_cast<int>(blockIdx.x + 1) * p.per, p.kbs);
  const int64_t k16 = (p.k + 15) / 16 * 16;
  float acc[2][4] = {};
  for (int kb = blockIdx.x * p.per + slice; kb < kb_end; kb += slices) {
    // the CTAs of the rank blocks share the encoding; those past the last rank only encode
    const bool encode = kb % gridDim.y == blockIdx.y && (!ALONG || p.codes);
    if (j0 >= p.r && !encode) continue;
    const int64_t k0 = static_cast<int64_t>(kb) * 128 + 8 * t;
    uint32_t x[kHalves][16], a[2][16];  // 4 x 8 columns
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t k = k0 + 32 * i;  // K is a multiple of 8: 8 columns are inside or not
#pragma unroll
      for (int h = 0; h < kHalves; ++h) {
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (k < p.k && row0 + g + 8 * h < p.m)
          v = __ldg(reinterpret_cast<const uint4*>(p.x + (row0 + g + 8 * h) * p.k + k));
        x[h][4 * i] = v.x;
        x[h][4 * i + 1] = v.y;
        x[h][4 * i + 2] = v.z;
        x[h][4 * i + 3] = v.w;
      }
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if constexpr (ALONG) {
          // 16 rows an instruction, both halves of a row's 16 ranks side by side
          const int64_t row = static_cast<int64_t>(kb) * 128 + 32 * i + 16 * n + (lane >> 1);
          const int j = j0 + 8 * (lane & 1);
          if (row < p.k && j < p.r) v = __ldg(reinterpret_cast<const uint4*>(p.a + row * p.r + j));
        } else if (k < p.k && j0 + 8 * n + g < p.r) {
          v = __ldg(reinterpret_cast<const uint4*>(p.a + (j0 + 8 * n + g) * p.k + k));
        }
        a[n][4 * i] = v.x;
        a[n][4 * i + 1] = v.y;
        a[n][4 * i + 2] = v.z;
        a[n][4 * i + 3] = v.w;
      }
    }
    if (ALONG) turn_tiles(a, area + kTurnBytes * warp, lane);
#pragma unroll
    for (int i = 0; i < 16; i += 2)
#pragma unroll
      for (int n = 0; n < 2; ++n)
        mma_bf16(acc[n], x[0][i], TWO ? x[kHalves - 1][i] : 0u, x[0][i + 1],
                 TWO ? x[kHalves - 1][i + 1] : 0u, a[n][i], a[n][i + 1]);
    if (!encode) continue;
#pragma unroll
    for (int h = 0; h < kHalves; ++h) {
      const int64_t row = row0 + g + 8 * h;
      float m = amax_words<__nv_bfloat16>(x[h]);
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
      const float s = block_scale_of(m, E5M2, p.pow2 != 0);
      const float inv = __fdiv_rn(1.0f, s);
      if (row >= p.m) continue;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t c[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const uint32_t w0 = x[h][4 * i + 2 * q], w1 = x[h][4 * i + 2 * q + 1];
          c[q] = encode4<E5M2>(word_value(w0, 0), word_value(w0, 1), word_value(w1, 0),
                               word_value(w1, 1), inv);
        }
        const int64_t k = k0 + 32 * i;  // zeros up to the next multiple of 16
        if (k < k16)
          *reinterpret_cast<uint2*>(p.codes + row * p.ld + k) = make_uint2(c[0], c[1]);
      }
      if (t == 0) p.scales[static_cast<int64_t>(kb) * p.m + row] = s;
    }
  }
  if (ALONG) __syncthreads();  // red takes the place of the tiles
  // acc[n]: tokens g (0, 1) and g + 8 (2, 3), ranks 8 n + 2 t, + 1
#pragma unroll
  for (int n = 0; n < 2; ++n)
#pragma unroll
    for (int q = 0; q < 4; ++q) red[warp][g + 8 * (q >> 1)][8 * n + 2 * t + (q & 1)] = acc[n][q];
  __syncthreads();
  const int64_t left = p.m - 16 * tile0;
  const int rows = static_cast<int>(left < 16 * p.tiles ? left : 16 * p.tiles);
  if (slices > 1) {
    for (int e = threadIdx.x; e < rows * kRanks; e += blockDim.x) {
      const int m = e / kRanks, j = e % kRanks;
      float v = red[m >> 4][m & 15][j];
      for (int w = 1; w < slices; ++w) v += red[(m >> 4) + w * p.tiles][m & 15][j];
      red[m >> 4][m & 15][j] = v;
    }
  }
  ptx::cluster_sync();
  const int ctas = static_cast<int>(gridDim.x);  // the cluster spans x
  for (int e = static_cast<int>(ptx::cluster_ctarank()) + ctas * static_cast<int>(threadIdx.x);
       e < rows * kRanks; e += ctas * static_cast<int>(blockDim.x)) {
    const int m = e / kRanks, j = j0 + e % kRanks;
    const float* at = &red[m >> 4][m & 15][e % kRanks];
    float y[kMaxCtas];
#pragma unroll
    for (int q = 0; q < kMaxCtas; ++q)
      y[q] = q < ctas ? ptx::ld_cluster_f32(ptx::cluster_addr(at, q)) : 0.0f;
    float v = 0.0f;
#pragma unroll
    for (int q = 0; q < kMaxCtas; ++q)
      if (q < ctas) v += y[q];
    const int64_t row = 16 * tile0 + m;
    if (j < p.r && p.u) p.u[row * p.r + j] = v;
    if (ALONG && j < p.r && p.ut) {
      const Terms t = terms_of(v);
      p.ut[j * p.ut_ld + row] = t.hi;
      p.ut[(p.ut_lo + j) * p.ut_ld + row] = t.mid;
      p.ut[(2 * p.ut_lo + j) * p.ut_ld + row] = t.lo;
    }
    if (j < p.span) {  // zeros past the last rank
      const float f = j < p.r ? p.sc * v : 0.0f;
      const __nv_bfloat16 hi = __float2bfloat16_rn(f);
      __nv_bfloat16* o = p.su + row * 2 * p.span + j;
      o[0] = hi;
      o[p.span] = j < p.r ? __float2bfloat16_rn(f - __bfloat162float(hi)) : hi;
    }
  }
  ptx::cluster_sync();  // the others may still read red
}

template <bool ALONG>
const void* front_kernel(bool e5m2, bool two) {
  return e5m2 ? (two ? reinterpret_cast<const void*>(f8_front_kernel<true, true, ALONG>)
                     : reinterpret_cast<const void*>(f8_front_kernel<true, false, ALONG>))
              : (two ? reinterpret_cast<const void*>(f8_front_kernel<false, true, ALONG>)
                     : reinterpret_cast<const void*>(f8_front_kernel<false, false, ALONG>));
}

}  // namespace

// f8_front_along.cu
const void* front_along_kernel(bool e5m2, bool two);

}  // namespace qlora
