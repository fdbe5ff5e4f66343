// Block quantiser to 8-bit floating point, and its inverse.
//
// For a block of values x (one row by 128 columns, or 128 x 128) and the
// format's largest value F (448 for e4m3, 57344 for e5m2):
//   a = max |x| over the finite values,
//   s = max(RN(a / F), 2^-126),  or, for power-of-two scales, the smallest
//       power of two p >= 2^-126 with a <= F p,
//   c = RN8(RN32(x * RN32(1 / s))),   value = c * s.
// One product with the reciprocal takes the place of a division per value; with
// a power-of-two scale both forms are exact and c is the one rounding of x / s.
// The floor 2^-126 keeps s and 1 / s normal numbers (a block of zeros gets it).
// NaN and infinities become the format's NaN: the value times zero is added,
// which changes no finite value and turns an infinity, which the conversion
// would saturate, into NaN.
//
// Both directions are bound by HBM: 2 bytes read and 1 written per value from
// bf16 (the other way round when restoring), 4 and 1 from fp32, plus 4 bytes per block.
// 8192 x 11008, warm launches over four matrices, floor 41.2 us from bf16 and 68.7 from fp32: by
// rows 41.3 and 73.6, by tiles 42.3 and 89.5 (an fp32 tile is 64 registers a thread: two
// CTAs an SM, whose load and store phases overlap less), restored 42.0 and 69.6, from tiles
// 41.7 and 69.2.  (Four CTAs an SM cost the bf16 tiles of odd rows, 2-byte loads, 48 bytes of
// spills; no other instance has any.)
#include <cuda_fp8.h>

#include "f8.cuh"
#include "f8_codec.cuh"

namespace qlora {
namespace {

constexpr int kThreads = 256;
constexpr int kRestoreRows = 2;  // rows a thread restores (1, 2, 4: 20.4, 19.0, 19.4 us)

struct QArgs {
  const void* x;
  uint8_t* codes;
  float* scales;
  int64_t rows, cols, ld;
  int64_t kb;     // 128-column blocks
  int32_t pow2;
};

// 16 consecutive values of a row from column c0, zeros past the last column.
// VEC: every row starts on 16 bytes and cols is a multiple of one 16-byte load.
template <typename T, bool VEC>
struct Load16;

template <bool VEC>
struct Load16<__nv_bfloat16, VEC> {
  uint32_t w[8];
  __device__ __forceinline__ void load(const __nv_bfloat16* x, int64_t row_off, int64_t c0,
                                       int64_t cols) {
    if (VEC) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (c0 + 8 * h < cols) v = __ldg(reinterpret_cast<const uint4*>(x + row_off + c0 + 8 * h));
        w[4 * h] = v.x;
        w[4 * h + 1] = v.y;
        w[4 * h + 2] = v.z;
        w[4 * h + 3] = v.w;
      }
    } else {
      const unsigned short* p = reinterpret_cast<const unsigned short*>(x) + row_off;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t lo = c0 + 2 * j < cols ? __ldg(p + c0 + 2 * j) : 0u;
        const uint32_t hi = c0 + 2 * j + 1 < cols ? __ldg(p + c0 + 2 * j + 1) : 0u;
        w[j] = lo | (hi << 16);
      }
    }
  }
  __device__ __forceinline__ float get(int j) const {
    return __uint_as_float((j & 1) ? (w[j >> 1] & 0xffff0000u) : (w[j >> 1] << 16));
  }
};

template <bool VEC>
struct Load16<float, VEC> {
  uint32_t w[16];
  __device__ __forceinline__ void load(const float* x, int64_t row_off, int64_t c0, int64_t cols) {
    if (VEC) {
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (c0 + 4 * h < cols) v = __ldg(reinterpret_cast<const uint4*>(x + row_off + c0 + 4 * h));
        w[4 * h] = v.x;
        w[4 * h + 1] = v.y;
        w[4 * h + 2] = v.z;
        w[4 * h + 3] = v.w;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 16; ++j)
        w[j] = c0 + j < cols ? __float_as_uint(__ldg(x + row_off + c0 + j)) : 0u;
    }
  }
  __device__ __forceinline__ float get(int j) const { return __uint_as_float(w[j]); }
};

template <bool E5M2, typename L>
__device__ __forceinline__ void store16(const L& v, float inv, const QArgs& p, int64_t row,
                                        int64_t c0) {
  if (row >= p.rows || c0 >= p.cols) return;
  uint32_t o[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    o[j] = encode4<E5M2>(v.get(4 * j), v.get(4 * j + 1), v.get(4 * j + 2), v.get(4 * j + 3), inv);
  // ld is a multiple of 16 and at least cols: the 16 bytes stay inside the row
  *reinterpret_cast<uint4*>(p.codes + row * p.ld + c0) = make_uint4(o[0], o[1], o[2], o[3]);
}

// A scale per row and 128 columns.  A warp takes 512 consecutive columns of a
// row (8 lanes per block: the maximum is 3 shuffles), a CTA ROWS rows of them;
// its scales leave through shared memory, so that a block column's scales of
// consecutive rows are one store.
template <typename T, bool E5M2, bool VEC, int ROWS>
__global__ void __launch_bounds__(kThreads) f8_rows_kernel(const QArgs p) {
  // the product that follows may start: it waits for the end of this launch before it
  // reads what this one writes
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  constexpr int kPer = ROWS / 8;  // rows per warp
  __shared__ float sc[4][ROWS];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const unsigned groups = static_cast<unsigned>((p.kb + 3) / 4);
  const int64_t kbg = blockIdx.x % groups;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x / groups) * ROWS;
  const int64_t c0 = kbg * 512 + lane * 16;
  const T* x = static_cast<const T*>(p.x);
  Load16<T, VEC> v[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int64_t row = row0 + warp + 8 * i;
    v[i].load(x, row * p.cols, c0, row < p.rows ? p.cols : 0);
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    float a = amax_words<T>(v[i].w);
#pragma unroll
    for (int d = 1; d < 8; d <<= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, d));
    const float s = block_scale_of(a, E5M2, p.pow2 != 0);
    store16<E5M2>(v[i], __fdiv_rn(1.0f, s), p, row0 + warp + 8 * i, c0);
    if ((lane & 7) == 0) sc[lane >> 3][warp + 8 * i] = s;
  }
  __syncthreads();
  for (int t = threadIdx.x; t < 4 * ROWS; t += kThreads) {
    const int b = t / ROWS, i = t % ROWS;
    if (kbg * 4 + b < p.kb && row0 + i < p.rows)
      p.scales[(kbg * 4 + b) * p.rows + row0 + i] = sc[b][i];
  }
}

// 16 bytes of values of a row from column c0 (8 bf16 or 4 fp32), zeros past the last
// column, as fp32.
template <typename T, bool VEC>
struct Load1 {
  static constexpr int kN = 16 / sizeof(T);
  uint32_t w[4];
  __device__ __forceinline__ void load(const T* x, int64_t row_off, int64_t c0, int64_t cols) {
    if (VEC) {
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      if (c0 < cols) v = __ldg(reinterpret_cast<const uint4*>(x + row_off + c0));
      w[0] = v.x;
      w[1] = v.y;
      w[2] = v.z;
      w[3] = v.w;
    } else if (sizeof(T) == 2) {
      const unsigned short* p = reinterpret_cast<const unsigned short*>(x) + row_off;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t lo = c0 + 2 * j < cols ? __ldg(p + c0 + 2 * j) : 0u;
        const uint32_t hi = c0 + 2 * j + 1 < cols ? __ldg(p + c0 + 2 * j + 1) : 0u;
        w[j] = lo | (hi << 16);
      }
    } else {
      const uint32_t* p = reinterpret_cast<const uint32_t*>(x) + row_off;
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = c0 + j < cols ? __ldg(p + c0 + j) : 0u;
    }
  }
  __device__ __forceinline__ float get(int j) const {
    if (sizeof(T) == 4) return __uint_as_float(w[j]);
    return __uint_as_float((j & 1) ? (w[j >> 1] & 0xffff0000u) : (w[j >> 1] << 16));
  }
};

// A scale per 128 x 128 tile: one CTA a tile, its values in registers between
// the maximum and the encoding; a warp takes 16 rows, 16 bytes a lane and load.
template <typename T, bool E5M2, bool VEC>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 4 : 2) f8_tiles_kernel(const QArgs p) {
  using L = Load1<T, VEC>;
  constexpr int kLanes = 128 / L::kN, kRows = 32 / kLanes, kLoads = 16 / kRows;
  __shared__ float red[8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const unsigned kbs = static_cast<unsigned>(p.kb);
  const int64_t kb = blockIdx.x % kbs, rb = blockIdx.x / kbs;
  const int64_t c0 = kb * 128 + (lane % kLanes) * L::kN;
  const int64_t row0 = rb * 128 + warp * 16 + lane / kLanes;
  const T* x = static_cast<const T*>(p.x);
  L v[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int64_t row = row0 + kRows * i;
    v[i].load(x, row * p.cols, c0, row < p.rows ? p.cols : 0);
  }
  float a = 0.0f;
#pragma unroll
  for (int i = 0; i < kLoads; ++i) a = fmaxf(a, amax_words<T>(v[i].w));
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, d));
  if (lane == 0) red[warp] = a;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 8; ++w) a = fmaxf(a, red[w]);
  const float s = block_scale_of(a, E5M2, p.pow2 != 0);
  const float inv = __fdiv_rn(1.0f, s);
  // codes up to the next multiple of 16 columns: zeros past the last one
  const int64_t end = (p.cols + 15) / 16 * 16;
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int64_t row = row0 + kRows * i;
    if (row >= p.rows || c0 >= end) continue;
    uint8_t* dst = p.codes + row * p.ld + c0;
    const uint32_t lo = encode4<E5M2>(v[i].get(0), v[i].get(1), v[i].get(2), v[i].get(3), inv);
    if (sizeof(T) == 4) {
      *reinterpret_cast<uint32_t*>(dst) = lo;
    } else {
      constexpr int q = L::kN - 4;  // 4
      const uint32_t hi =
          encode4<E5M2>(v[i].get(q), v[i].get(q + 1), v[i].get(q + 2), v[i].get(q + 3), inv);
      *reinterpret_cast<uint2*>(dst) = make_uint2(lo, hi);
    }
  }
  if (threadIdx.x == 0) p.scales[rb * p.kb + kb] = s;
}

template <bool E5M2>
__device__ __forceinline__ float2 decode2(uint32_t u16) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(u16),
                                                   E5M2 ? __NV_E5M2 : __NV_E4M3);
  return __half22float2(__half2(h));
}

// N (4 or 8) codes from p, 4 or 8 bytes at once.
template <int N>
__device__ __forceinline__ void load_codes(const uint8_t* p, uint32_t (&w)[N / 4]) {
  if (N == 8) {
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
    w[0] = v.x;
    w[N / 4 - 1] = v.y;
  } else {
    w[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
  }
}

// Restores values: a warp takes 512 consecutive columns of a row in spans of one
// 16-byte store per lane, so that each store instruction writes whole lines (16
// codes a lane, two stores 32 bytes apart, took 24.8 us for 8192 x 4096 into
// bf16).  kRows rows a thread are read before the first is written.
template <typename T, bool E5M2, bool VEC, bool TILES>
__global__ void __launch_bounds__(kThreads) f8_restore_kernel(const QArgs p, T* out) {
  constexpr int kN = 16 / sizeof(T), kSpans = 512 / (32 * kN), kRows = kRestoreRows;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const unsigned groups = static_cast<unsigned>((p.kb + 3) / 4);
  const int64_t col0 = static_cast<int64_t>(blockIdx.x % groups) * 512 + lane * kN;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x / groups) * (8 * kRows);
  uint32_t code[kRows][kSpans][kN / 4];
  float sc[kRows][kSpans];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int64_t row = row0 + warp + 8 * i;
#pragma unroll
    for (int h = 0; h < kSpans; ++h) {
      const int64_t c = col0 + h * 32 * kN;
      if (row < p.rows && c < p.cols) {
        load_codes<kN>(p.codes + row * p.ld + c, code[i][h]);
        const int64_t kb = c >> 7;
        sc[i][h] = __ldg(p.scales + (TILES ? (row >> 7) * p.kb + kb : kb * p.rows + row));
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int64_t row = row0 + warp + 8 * i;
#pragma unroll
    for (int h = 0; h < kSpans; ++h) {
      const int64_t c = col0 + h * 32 * kN;
      if (row >= p.rows || c >= p.cols) continue;
      float f[kN];
#pragma unroll
      for (int j = 0; j < kN / 2; ++j) {
        const float2 d = decode2<E5M2>((code[i][h][j >> 1] >> (16 * (j & 1))) & 0xffffu);
        f[2 * j] = __fmul_rn(d.x, sc[i][h]);
        f[2 * j + 1] = __fmul_rn(d.y, sc[i][h]);
      }
      T* o = out + row * p.cols + c;
      if (!VEC) {
#pragma unroll
        for (int j = 0; j < kN; ++j)
          if (c + j < p.cols) {
            if (sizeof(T) == 2)
              reinterpret_cast<__nv_bfloat16*>(o)[j] = __float2bfloat16_rn(f[j]);
            else
              reinterpret_cast<float*>(o)[j] = f[j];
          }
      } else if (sizeof(T) == 2) {
        uint32_t u[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const __nv_bfloat162 v =
              __floats2bfloat162_rn(f[(2 * j) % kN], f[(2 * j + 1) % kN]);
          u[j] = *reinterpret_cast<const uint32_t*>(&v);
        }
        *reinterpret_cast<uint4*>(o) = make_uint4(u[0], u[1], u[2], u[3]);
      } else {
        *reinterpret_cast<float4*>(o) = make_float4(f[0], f[1], f[2], f[3]);
      }
    }
  }
}

template <typename T, bool E5M2, bool VEC>
qlora_status quantize_as(const QArgs& p, bool tiles, cudaStream_t s) {
  const int64_t groups = (p.kb + 3) / 4;
  // 8 rows a CTA while 32 would leave SMs without work
  const bool few = ceil_div(p.rows, 32) * groups < 296;
  const int64_t grid = tiles ? p.kb * f8_blocks(p.rows) : groups * ceil_div(p.rows, few ? 8 : 32);
  if (grid > 0x7fffffff) return QLORA_ERR_SHAPE;
  const unsigned g = static_cast<unsigned>(grid);
  count_launch();
  timing_mark(QLORA_KERNEL_QUANTIZE, s, true);
  if (tiles)
    f8_tiles_kernel<T, E5M2, VEC><<<g, kThreads, 0, s>>>(p);
  else if (few)
    f8_rows_kernel<T, E5M2, VEC, 8><<<g, kThreads, 0, s>>>(p);
  else
    f8_rows_kernel<T, E5M2, VEC, 32><<<g, kThreads, 0, s>>>(p);
  timing_mark(QLORA_KERNEL_QUANTIZE, s, false);
  return after_launch("f8_quantize", s);
}

template <typename T, bool E5M2, bool VEC>
qlora_status restore_as(const QArgs& p, bool tiles, void* out, cudaStream_t s) {
  const int64_t grid = (p.kb + 3) / 4 * ceil_div(p.rows, 8 * kRestoreRows);
  if (grid > 0x7fffffff) return QLORA_ERR_SHAPE;
  const unsigned g = static_cast<unsigned>(grid);
  count_launch();
  if (tiles)
    f8_restore_kernel<T, E5M2, VEC, true><<<g, kThreads, 0, s>>>(p, static_cast<T*>(out));
  else
    f8_restore_kernel<T, E5M2, VEC, false><<<g, kThreads, 0, s>>>(p, static_cast<T*>(out));
  return after_launch("f8_restore", s);
}

QArgs args_of(const qlora_f8& q, const void* x) {
  return QArgs{x, q.codes, q.scales, q.rows, q.cols, q.ld, f8_blocks(q.cols), q.pow2};
}

}  // namespace

qlora_status launch_f8_quantize(const void* X, int32_t x_dtype, const qlora_f8& q,
                                cudaStream_t s) {
  const QArgs p = args_of(q, X);
  const bool tiles = q.layout == QLORA_F8_TILES, e5 = q.format == QLORA_E5M2;
  if (x_dtype == QLORA_BF16) {
    const bool vec = q.cols % 8 == 0;
    if (vec)
      return e5 ? quantize_as<__nv_bfloat16, true, true>(p, tiles, s)
                : quantize_as<__nv_bfloat16, false, true>(p, tiles, s);
    return e5 ? quantize_as<__nv_bfloat16, true, false>(p, tiles, s)
              : quantize_as<__nv_bfloat16, false, false>(p, tiles, s);
  }
  const bool vec = q.cols % 4 == 0;
  if (vec)
    return e5 ? quantize_as<float, true, true>(p, tiles, s)
              : quantize_as<float, false, true>(p, tiles, s);
  return e5 ? quantize_as<float, true, false>(p, tiles, s)
            : quantize_as<float, false, false>(p, tiles, s);
}

qlora_status launch_f8_dequantize(const qlora_f8& q, void* out, int32_t out_dtype,
                                  cudaStream_t s) {
  const QArgs p = args_of(q, nullptr);
  const bool tiles = q.layout == QLORA_F8_TILES, e5 = q.format == QLORA_E5M2;
  if (out_dtype == QLORA_BF16) {
    const bool vec = q.cols % 8 == 0;
    if (vec)
      return e5 ? restore_as<__nv_bfloat16, true, true>(p, tiles, out, s)
                : restore_as<__nv_bfloat16, false, true>(p, tiles, out, s);
    return e5 ? restore_as<__nv_bfloat16, true, false>(p, tiles, out, s)
              : restore_as<__nv_bfloat16, false, false>(p, tiles, out, s);
  }
  const bool vec = q.cols % 4 == 0;
  if (vec)
    return e5 ? restore_as<float, true, true>(p, tiles, out, s)
              : restore_as<float, false, true>(p, tiles, out, s);
  return e5 ? restore_as<float, true, false>(p, tiles, out, s)
            : restore_as<float, false, false>(p, tiles, out, s);
}

}  // namespace qlora
