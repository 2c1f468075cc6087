// Codes of 8-bit floating point with an fp32 scale for each block of 128: the
// operands of the products in gemm_f8.cu.  Entry point, host plan and kernels;
// the contract is in include/tcg.h.
//
// A block's largest magnitude a gives its scale a / F (F the format's largest
// value) and the codes rn(F x / a).  F x is exact for 16-bit x, and the
// quotient is computed to the last bit where it matters: y = F x * (1 / a), then
// one correction y + (F x - y a) / a, whose residual an fma gives exactly.  An
// exact tie between two codes therefore stays one (with y alone, or x divided by
// the rounded scale, 1 of 300 such ties went the other way), and other quotients
// of 16-bit values lie at least 2^-13 (bf16) or 2^-16 (f16) of themselves off a tie.
// Those of fp32 values may lie as close as 2^-50, and F x has up to 27 bits: see
// encode_f32.
//
// All three kernels read X once, keep it on the SM between the maximum and the
// codes, and are bound by HBM.  Rows: a half warp (16-bit types) or a warp holds a
// block's row, a warp takes 8 rows so that their 8 loads are in flight together and
// the 8 scales, neighbours in memory, leave as one sector: 16384 x 8192 bf16 63 us,
// 6.4 TB/s.  Columns: a warp holds 128 rows of 32 or 16 columns: 16384 x 4096 bf16
// 35.6 us, 5.7 TB/s, 16384 x 16384 123.5 us, 6.6 TB/s (rows: 34.0 and 121.8).  Squares:
// a CTA holds a block: 8192 x 8192 bf16 34.6 us, 5.8 TB/s.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "common.h"
#include "ptx.cuh"
#include "ptx_moe.cuh"

namespace tcg {

namespace {

constexpr int BLOCK = 128;
constexpr int MAX_GROUPS = 1024;
constexpr int64_t MAX_EXTENT = int64_t{1} << 30;
constexpr int ROW_WARPS = 4;
constexpr int ROWS = 8;  // rows of a warp
constexpr int COL_WARPS = 4;
constexpr int SQUARE_THREADS = 256;

// 16 bytes of X: V values of type T.  Maxima are taken of the words as they are
// (pairs of 16-bit values at a time): converted first, the values took twice the
// registers, and kept them until the codes.
template <class T>
struct Word {
  static constexpr int V = 16 / static_cast<int>(sizeof(T));
  uint32_t w[4];

  __device__ __forceinline__ void load(const T* from, int n, bool aligned) {  // the first n values, then zeros
    if (aligned) {
      const uint4 v = n > 0 ? *reinterpret_cast<const uint4*>(from) : make_uint4(0, 0, 0, 0);
      w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = j < n ? reinterpret_cast<const uint32_t*>(from)[j] : 0u;
    } else {
      const uint16_t* h = reinterpret_cast<const uint16_t*>(from);
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = (2 * j < n ? h[2 * j] : 0u) | (2 * j + 1 < n ? h[2 * j + 1] : 0u) << 16;
    }
  }

  __device__ __forceinline__ float value(int j) const {
    if constexpr (std::is_same<T, float>::value)
      return __uint_as_float(w[j]);
    else if constexpr (std::is_same<T, __half>::value)
      return __half2float(__ushort_as_half(static_cast<uint16_t>(w[j / 2] >> (16 * (j % 2)))));
    else
      return __uint_as_float(j % 2 ? w[j / 2] & 0xffff0000u : w[j / 2] << 16);
  }
};

// The larger magnitudes of a word (already positive) and another; NaN are passed over.
template <class T>
__device__ __forceinline__ uint32_t most(uint32_t a, uint32_t x) {
  if constexpr (std::is_same<T, float>::value) {
    return __float_as_uint(fmaxf(__uint_as_float(a), fabsf(__uint_as_float(x))));
  } else {
    using T2 = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;
    const T2 m = __hmax2(*reinterpret_cast<const T2*>(&a), __habs2(*reinterpret_cast<const T2*>(&x)));
    return *reinterpret_cast<const uint32_t*>(&m);
  }
}

// The largest value of a word.
template <class T>
__device__ __forceinline__ float largest_in(uint32_t a) {
  Word<T> x;
  x.w[0] = a;
  if constexpr (std::is_same<T, float>::value)
    return x.value(0);
  else
    return fmaxf(x.value(0), x.value(1));
}

// How the values of a block become codes.
struct Coder {
  float by;     // x * by is F x (a in normal range)
  float a, inv; // divided by a
};

template <bool WIDE>
__device__ __forceinline__ float largest() { return WIDE ? 57344.0f : 448.0f; }

template <bool WIDE>
__device__ __forceinline__ Coder make_coder(float amax, bool pow2, float& scale) {
  const float F = largest<WIDE>();
  if (amax == 0.0f) {
    scale = 1.0f;
    return {1.0f, 1.0f, 1.0f};
  }
  if (isinf(amax)) {  // finite values become 0, infinities NaN
    scale = amax;
    return {0.0f, 1.0f, 1.0f};
  }
  scale = fmaxf(amax / F, 0x1p-126f);
  if (pow2) {
    // F = 1.75 * 2^8 or 1.75 * 2^15: the power is decided by amax's significand
    int e;
    const float m = frexpf(amax, &e);  // [0.5, 1)
    const int k = max(e - (m <= 0.875f ? 9 : 8) - (WIDE ? 7 : 0), -126);
    scale = ldexpf(1.0f, k);
    return {ldexpf(1.0f, -k), 1.0f, 1.0f};
  }
  if (scale == 0x1p-126f) return {0x1p126f, 1.0f, 1.0f};
  // kept away from the ends of fp32's range, where F x and 1 / a would leave it
  const float pre = amax > 0x1p64f ? 0x1p-32f : amax < 0x1p-64f ? 0x1p32f : 1.0f;
  const float a = amax * pre;
  return {F * pre, a, 1.0f / a};
}

// Factors of fp32 x that give a little less and a little more than F x / a.  Each
// product is within four roundings, 2^-22 of itself, of its own.  A power of two (by of
// `pow2`, zeros and the smallest blocks; F has three significant bits) is exact.
struct Bounds {
  float below, above;
};
__device__ __forceinline__ Bounds bounds(const Coder& c) {
  if ((__float_as_uint(c.by) & 0x7fffffu) == 0) return {c.by, c.by};
  const float k = c.by * c.inv;
  return {k * (1.0f - 0x1p-21f), k * (1.0f + 0x1p-21f)};
}
__device__ __forceinline__ Bounds from_lane(const Bounds& b, int lane) {
  return {__shfl_sync(0xffffffffu, b.below, lane), __shfl_sync(0xffffffffu, b.above, lane)};
}

__device__ __forceinline__ Coder from_lane(const Coder& c, int lane) {
  return {__shfl_sync(0xffffffffu, c.by, lane), __shfl_sync(0xffffffffu, c.a, lane), __shfl_sync(0xffffffffu, c.inv, lane)};
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi));
  return v;
}
__device__ __forceinline__ void unpair(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}

// F x / a of 16-bit x, so close that rounding it to a code rounds F x / a itself.
__device__ __forceinline__ float quotient(float x, const Coder& c) {
  const float n = x * c.by;
  const float y = n * c.inv;
  return fmaf(fmaf(-y, c.a, n), c.inv, y);
}

// Rounding to odd: of the two fp32 values around z + rest (rest the less of z's last
// bit) the one whose last bit is set, unless rest is 0.  Ties have few bits, so that a
// quotient beside one stays on its side.
__device__ __forceinline__ float to_odd(float z, float rest) {
  const uint32_t bits = __float_as_uint(z);
  const int32_t step = static_cast<int32_t>(__float_as_uint(rest) ^ bits) >> 31 | 1;  // towards zero or away from it
  return __uint_as_float(rest != 0.0f && !(bits & 1u) ? bits + step : bits);
}

// Four codes, the first in the low byte.
template <bool WIDE>
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
  constexpr __nv_fp8_interpretation_t I = WIDE ? __NV_E5M2 : __NV_E4M3;
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, I);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, I);
  return lo | hi << 16;
}

// Four codes of fp32 values, if `sure`: the same from a little less and from a little
// more than F x / a.  Where they differ (1 of 2^16 values, and ties) store_exact_codes
// decides.  8192 x 8192 fp32, rows, columns and squares: 49.7, 54.1 and 57.8 us; where one
// value of 300 is a tie (bf16 values) 54, 69 and 63, where every word has one (small
// integers) 78, 92 and 85, about as much as with store_exact_codes throughout.
template <bool WIDE, class F>
__device__ __forceinline__ uint32_t encode_f32(const Word<float>& x, F&& bound, bool& sure) {
  float lo[4], hi[4];
#pragma unroll
  for (int j = 0; j < 4; j += 2) {
    const Bounds a = bound(j), b = bound(j + 1);
    const uint64_t v = pair(x.value(j), x.value(j + 1));
    unpair(mul2(v, pair(a.below, b.below)), lo[j], lo[j + 1]);
    unpair(mul2(v, pair(a.above, b.above)), hi[j], hi[j + 1]);
  }
  const uint32_t code = encode4<WIDE>(lo[0], lo[1], lo[2], lo[3]);
  sure = code == encode4<WIDE>(hi[0], hi[1], hi[2], hi[3]);
  return code;
}

// The first n of a word's V codes.
template <int V>
__device__ __forceinline__ void put_codes(const uint32_t (&code)[V / 4], uint8_t* q, int n, bool aligned) {
  if (!aligned) {
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (j < n) q[j] = static_cast<uint8_t>(code[j / 4] >> (8 * (j % 4)));
  } else if (n > 0) {
    if constexpr (V == 8)
      *reinterpret_cast<uint2*>(q) = make_uint2(code[0], code[1]);
    else
      *reinterpret_cast<uint32_t*>(q) = code[0];
  }
}

// What the codes of a type's values are made with.
template <class T>
using Maker = typename std::conditional<std::is_same<T, float>::value, Bounds, Coder>::type;
template <class T>
__device__ __forceinline__ Maker<T> maker(const Coder& c) {
  if constexpr (std::is_same<T, float>::value)
    return bounds(c);
  else
    return c;
}

// V codes of a word; true if store_exact_codes has to replace them.
template <bool WIDE, class T, class F>
__device__ __forceinline__ bool store_codes(const Word<T>& x, uint8_t* q, int n, bool aligned, F&& coder) {
  constexpr int V = Word<T>::V;
  uint32_t code[V / 4];
  bool sure = true;
  if constexpr (std::is_same<T, float>::value) {
    code[0] = encode_f32<WIDE>(x, coder, sure);
  } else {
#pragma unroll
    for (int j = 0; j < V; j += 4)
      code[j / 4] = encode4<WIDE>(quotient(x.value(j), coder(j)), quotient(x.value(j + 1), coder(j + 1)),
                                  quotient(x.value(j + 2), coder(j + 2)), quotient(x.value(j + 3), coder(j + 3)));
  }
  put_codes<V>(code, q, n, aligned);
  return !sure;
}

// F x = m + low exactly; z is one of the two fp32 values around (m + low) / a, and the
// sign of the rest is exact (multiples of z's and a's last bits, less than 2^25 of them).
template <bool WIDE, class F>
__device__ __forceinline__ void store_exact_codes(const Word<float>& x, uint8_t* q, int n, bool aligned, F&& coder) {
  float z[4], rest[4];
  const uint64_t minus = pair(-1.0f, -1.0f);
#pragma unroll
  for (int j = 0; j < 4; j += 2) {
    const Coder a = coder(j), b = coder(j + 1);
    const uint64_t v = pair(x.value(j), x.value(j + 1)), inv = pair(a.inv, b.inv), less = pair(-a.a, -b.a);
    const uint64_t m = mul2(v, pair(a.by, b.by));
    const uint64_t less_low = fma2(v, pair(-a.by, -b.by), m);
    const uint64_t y = mul2(m, inv);
    const uint64_t zz = fma2(fma2(less_low, minus, fma2(y, less, m)), inv, y);
    unpair(zz, z[j], z[j + 1]);
    unpair(fma2(less_low, minus, fma2(zz, less, m)), rest[j], rest[j + 1]);
  }
  const uint32_t code[1] = {encode4<WIDE>(to_odd(z[0], rest[0]), to_odd(z[1], rest[1]), to_odd(z[2], rest[2]), to_odd(z[3], rest[3]))};
  put_codes<4>(code, q, n, aligned);
}

// ----------------------------------------------------------------------- rows
//
// A word a lane, 16 or 32 lanes a block.  ALIGNED: X in 16-byte words, Q in words of
// V bytes, and C whole words.
template <class T, bool WIDE, bool ALIGNED>
__global__ void __launch_bounds__(32 * ROW_WARPS) row_kernel(int64_t R, int64_t C, const T* __restrict__ X,
                                                             int64_t ldx, bool pow2, uint8_t* __restrict__ Q,
                                                             int64_t ldq, float* __restrict__ scale,
                                                             int64_t ld_scale, int64_t col_warps) {
  constexpr int V = Word<T>::V;
  constexpr int LANES = BLOCK / V;
  const int lane = threadIdx.x & 31;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * ROW_WARPS + (threadIdx.x >> 5);
  const int64_t r0 = w / col_warps * ROWS;
  const int64_t c = (w % col_warps) * 32 * V + lane * V;
  const int n = static_cast<int>(max(int64_t{0}, min(static_cast<int64_t>(V), C - c)));
  griddep_wait();
  if (r0 >= R) return;
  const int rows = static_cast<int>(min(static_cast<int64_t>(ROWS), R - r0));
  Word<T> x[ROWS];
#pragma unroll
  for (int i = 0; i < ROWS; ++i) x[i].load(X + (r0 + i) * ldx + c, i < rows ? n : 0, ALIGNED);
  // a lane makes the coder of one row, for all lanes of its block (each of them all
  // eight: as many instructions as the codes; 16384 x 8192 bf16 95 us, 71 so)
  float mine = 0.0f;
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) m = most<T>(m, x[i].w[j]);
    float a = largest_in<T>(m);
#pragma unroll
    for (int d = LANES / 2; d; d >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, d));
    if (lane % ROWS == i) mine = a;
  }
  float s;
  const Coder my = make_coder<WIDE>(mine, pow2, s);
  const Maker<T> make = maker<T>(my);
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const Maker<T> k = from_lane(make, lane / LANES * LANES + i);
    const bool d = i < rows && store_codes<WIDE>(x[i], Q + (r0 + i) * ldq + c, n, ALIGNED, [&](int) { return k; });
    if constexpr (std::is_same<T, float>::value) {
      if (__any_sync(0xffffffffu, d)) {
        const Coder e = from_lane(my, lane / LANES * LANES + i);
        if (d) store_exact_codes<WIDE>(x[i], Q + (r0 + i) * ldq + c, n, ALIGNED, [&](int) { return e; });
      }
    }
  }
  const int64_t block = (c - lane % LANES * V) / BLOCK;
  if (lane % LANES < rows && block * BLOCK < C) scale[block * ld_scale + r0 + lane % LANES] = s;
  griddep_launch_dependents();
}

// -------------------------------------------------------------------- columns

// A warp takes 128 rows by four times V columns: lane 4 g + w holds rows g + 8 i and
// columns V w .. + V.  Its maxima and coders go through shuffles alone, so warps never
// wait for one another (as CTAs of 128 x 64 with barriers, 16385 x 4096 bf16 took 55
// to 67 us).  ALIGNED: between maxima and codes the words stay in shared memory, each
// lane's its own, so that 24 warps of an SM have loads in flight (in registers there is
// room for 12; 8192 x 8192 fp32 70 us, 57 so).  One tile a warp: with runs of tiles,
// and each lane's next words copied while it codes, 16384 x 16384 bf16 took 143 us
// instead of 124; with as many CTAs as fit and equal shares for all 20 to 30 % more.
template <class T, bool WIDE, bool ALIGNED>
__global__ void __launch_bounds__(32 * COL_WARPS, ALIGNED ? 6 : 3)
    column_kernel(int64_t R, int64_t C, const T* __restrict__ X, int64_t ldx, bool pow2, int G,
                  const int32_t* __restrict__ offsets, uint8_t* __restrict__ Q, int64_t ldq, float* __restrict__ scale,
                  int64_t ld_scale, int64_t across) {
  constexpr int V = Word<T>::V;
  constexpr int COLS = 4 * V, PER = BLOCK / 8;
  constexpr int UNROLL = ALIGNED ? 4 : PER;  // addresses of all sixteen words would spill
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g8 = lane >> 2, w4 = lane & 3;
  const int64_t slot = blockIdx.x / across;  // the block's row of scales
  const int64_t c = ((blockIdx.x % across) * COL_WARPS + warp) * COLS + V * w4;
  const int n = static_cast<int>(max(int64_t{0}, min(static_cast<int64_t>(V), C - c)));
  griddep_wait();
  int64_t lo = slot * BLOCK, end = R;
  if (offsets) {
    // block j of group g has slot offsets[g] / 128 + g + j; the slots of groups rise.  (For
    // any offsets slot >= g, as some group of an index >= g was met, so that lo below is
    // first % 128 + (slot - g) * 128 >= 0.)
    int g = -1, first = 0, next = 0;
    for (int i = lane; i < G; i += 32) {
      const int o = min(max(offsets[i], 0), static_cast<int>(R)), o1 = offsets[i + 1];
      if (o / BLOCK + i <= slot) ++g, first = o, next = o1;
    }
    g = __reduce_add_sync(0xffffffffu, g) + 31;
    if (g < 0) return;
    first = __shfl_sync(0xffffffffu, first, g);  // lane g % 32 met g last
    end = min(max(__shfl_sync(0xffffffffu, next, g), first), static_cast<int>(R));
    lo = first + (slot - first / BLOCK - g) * BLOCK;
  }
  if (lo >= end || c - V * w4 >= C) return;  // a slot that no group uses keeps its value
  const int rows = static_cast<int>(min(static_cast<int64_t>(BLOCK), end - lo));
  __shared__ uint4 kept[ALIGNED ? COL_WARPS : 1][ALIGNED ? PER : 1][32];
  Word<T> x[ALIGNED ? 1 : PER];
  const auto word = [&](int i) -> const Word<T>& {
    if constexpr (ALIGNED) {
      const uint4 v = kept[warp][i][lane];
      x[0].w[0] = v.x, x[0].w[1] = v.y, x[0].w[2] = v.z, x[0].w[3] = v.w;
      return x[0];
    } else {
      return x[i];
    }
  };
#pragma unroll UNROLL
  for (int i = 0; i < PER; ++i) {
    const bool exists = n > 0 && g8 + 8 * i < rows;
    const T* from = X + (lo + g8 + 8 * i) * ldx + c;
    if constexpr (ALIGNED)
      copy_16(smem_u32(&kept[warp][i][lane]), exists ? from : X, exists ? 16 : 0);
    else
      x[i].load(from, exists ? n : 0, false);
  }
  if constexpr (ALIGNED) asm volatile("cp.async.wait_all;" ::: "memory");
  Word<T> top = {};  // of the columns
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const Word<T>& v = word(i);
#pragma unroll
    for (int j = 0; j < 4; ++j) top.w[j] = most<T>(top.w[j], v.w[j]);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int d = 16; d >= 4; d >>= 1) top.w[j] = most<T>(top.w[j], __shfl_xor_sync(0xffffffffu, top.w[j], d));
  float mine = 0.0f;  // the largest of column V w4 + g8
#pragma unroll
  for (int j = 0; j < V; ++j)
    if (g8 % V == j) mine = top.value(j);
  float s;
  const Coder my = make_coder<WIDE>(mine, pow2, s);
  if (g8 < V && c + g8 < C) scale[slot * ld_scale + c + g8] = s;
  const Maker<T> make = maker<T>(my);
  Maker<T> k[V];
#pragma unroll
  for (int j = 0; j < V; ++j) k[j] = from_lane(make, 4 * j + w4);
#pragma unroll UNROLL
  for (int i = 0; i < PER; ++i) {
    const Word<T>& v = word(i);
    if constexpr (!std::is_same<T, float>::value) {
      if (g8 + 8 * i < rows)
        store_codes<WIDE>(v, Q + (lo + g8 + 8 * i) * ldq + c, n, ALIGNED, [&](int j) { return k[j]; });
    } else {
      uint8_t* q = Q + (lo + g8 + 8 * i) * ldq + c;
      const bool doubt = g8 + 8 * i < rows && store_codes<WIDE>(v, q, n, ALIGNED, [&](int j) { return k[j]; });
      if (__any_sync(0xffffffffu, doubt)) {
        Coder exact[V];
#pragma unroll
        for (int j = 0; j < V; ++j) exact[j] = from_lane(my, 4 * j + w4);
        if (doubt) store_exact_codes<WIDE>(v, q, n, ALIGNED, [&](int j) { return exact[j]; });
      }
    }
  }
  griddep_launch_dependents();
}

// -------------------------------------------------------------------- squares

// A block a CTA, in words of 16 bytes.  Four CTAs an SM of 16-bit values (8192 x 8192:
// 34.6 us; three 41, five 44), two of fp32 (58 us; one 92, three 68).
template <class T, bool WIDE, bool ALIGNED>
__global__ void __launch_bounds__(SQUARE_THREADS, ALIGNED && sizeof(T) == 2 ? 4 : 2)
    square_kernel(int64_t R, int64_t C, const T* __restrict__ X, int64_t ldx, bool pow2, uint8_t* __restrict__ Q,
                  int64_t ldq, float* __restrict__ scale, int64_t ld_scale, int64_t col_tiles) {
  constexpr int V = Word<T>::V;
  constexpr int ACROSS = BLOCK / V, DOWN = SQUARE_THREADS / ACROSS, PER = BLOCK / DOWN;
  __shared__ float top[SQUARE_THREADS / 32];
  const int t = threadIdx.x;
  const int64_t lo = blockIdx.x / col_tiles * BLOCK, tile = blockIdx.x % col_tiles;
  const int64_t c = tile * BLOCK + V * (t % ACROSS);
  const int n = static_cast<int>(max(int64_t{0}, min(static_cast<int64_t>(V), C - c)));
  const int rows = static_cast<int>(min(static_cast<int64_t>(BLOCK), R - lo));
  griddep_wait();
  Word<T> x[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int row = t / ACROSS + DOWN * i;
    x[i].load(X + (lo + row) * ldx + c, row < rows ? n : 0, ALIGNED);
  }
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) w = most<T>(w, x[i].w[j]);
  float m = largest_in<T>(w), s;
#pragma unroll
  for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
  if ((t & 31) == 0) top[t >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < SQUARE_THREADS / 32; ++i) m = fmaxf(m, top[i]);
  const Coder k = make_coder<WIDE>(m, pow2, s);
  if (t == 0) scale[blockIdx.x / col_tiles * ld_scale + tile] = s;
  const Maker<T> make = maker<T>(k);
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int row = t / ACROSS + DOWN * i;
    uint8_t* q = Q + (lo + row) * ldq + c;
    const bool doubt = row < rows && store_codes<WIDE>(x[i], q, n, ALIGNED, [&](int) { return make; });
    if constexpr (std::is_same<T, float>::value)
      if (doubt) store_exact_codes<WIDE>(x[i], q, n, ALIGNED, [&](int) { return k; });
  }
  griddep_launch_dependents();
}

// ----------------------------------------------------------------------- host

template <class... Params, class... Args>
int launch(void (*kernel)(Params...), int64_t grid, int threads, cudaStream_t s, Args... args) {
  if (grid > INT32_MAX) return TCG_ERR_UNSUPPORTED;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
  cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (int rc = record_cuda(cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...))) return rc;
  set_launch_count(1);
  return TCG_OK;
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

template <class T, bool WIDE, bool ALIGNED>
int run_typed(tcg_f8_blocks blocks, bool pow2, int64_t R, int64_t C, const T* X, int64_t ldx, int G,
              const int32_t* offsets, uint8_t* Q, int64_t ldq, float* scale, int64_t ld_scale, cudaStream_t s) {
  if (blocks == TCG_F8_ROW) {
    constexpr int64_t V = Word<T>::V;
    const int64_t col_warps = ceil_div(C, 32 * V);
    return launch(row_kernel<T, WIDE, ALIGNED>, ceil_div(ceil_div(R, ROWS) * col_warps, ROW_WARPS), 32 * ROW_WARPS, s,
                  R, C, X, ldx, pow2, Q, ldq, scale, ld_scale, col_warps);
  }
  if (blocks == TCG_F8_SQUARE) {
    const int64_t tiles = ceil_div(C, BLOCK);
    return launch(square_kernel<T, WIDE, ALIGNED>, ceil_div(R, BLOCK) * tiles, SQUARE_THREADS, s, R, C, X, ldx, pow2, Q,
                  ldq, scale, ld_scale, tiles);
  }
  const int64_t slots = offsets ? R / BLOCK + G : ceil_div(R, BLOCK);
  const int64_t across = ceil_div(C, COL_WARPS * 64 / static_cast<int64_t>(sizeof(T)));
  return launch(column_kernel<T, WIDE, ALIGNED>, slots * across, 32 * COL_WARPS, s, R, C, X, ldx, pow2, G, offsets, Q,
                ldq, scale, ld_scale, across);
}

int run_quantize(tcg_input q_type, tcg_f8_blocks blocks, int pow2, int64_t R, int64_t C, tcg_dtype x_type,
                 const void* X, int64_t ldx, int G, const int32_t* offsets, void* Q, int64_t ldq, float* scale,
                 int64_t ld_scale, cudaStream_t s) {
  set_launch_count(0);
  if (q_type != TCG_IN_E4M3 && q_type != TCG_IN_E5M2) return TCG_ERR_INVALID;
  if (blocks < TCG_F8_ROW || blocks > TCG_F8_SQUARE || x_type < TCG_F32 || x_type > TCG_BF16) return TCG_ERR_INVALID;
  if (R < 0 || C < 0 || G < 1) return TCG_ERR_INVALID;
  if (offsets ? blocks != TCG_F8_COLUMN : G != 1) return TCG_ERR_INVALID;
  if (R >= MAX_EXTENT || C >= MAX_EXTENT || G > MAX_GROUPS) return TCG_ERR_UNSUPPORTED;
  if (R == 0 || C == 0) return TCG_OK;
  const int64_t across = blocks == TCG_F8_ROW ? R : blocks == TCG_F8_COLUMN ? C : ceil_div(C, BLOCK);
  if (ldx == 0) ldx = C;
  if (ldq == 0) ldq = C;
  if (ld_scale == 0) ld_scale = across;
  if (!X || !Q || !scale || ldx < C || ldq < C || ld_scale < across) return TCG_ERR_INVALID;
  const int64_t size = x_type == TCG_F32 ? 4 : 2;
  const auto at = [](const void* p) { return reinterpret_cast<uintptr_t>(p); };
  if (at(X) % size || at(scale) % 4 || at(offsets) % 4) return TCG_ERR_ALIGNMENT;
  int dev;
  if (int rc = current_device_checked(&dev)) return rc;
  const int64_t V = 16 / size;  // elements of a 16-byte word
  const bool aligned = at(X) % 16 == 0 && ldx % V == 0 && C % V == 0 && at(Q) % V == 0 && ldq % V == 0;
  const auto typed = [&](auto z) {
    using T = decltype(z);
    const T* x = static_cast<const T*>(X);
    uint8_t* q = static_cast<uint8_t*>(Q);
    const bool p = pow2 != 0;
    if (q_type == TCG_IN_E5M2)
      return aligned ? run_typed<T, true, true>(blocks, p, R, C, x, ldx, G, offsets, q, ldq, scale, ld_scale, s)
                     : run_typed<T, true, false>(blocks, p, R, C, x, ldx, G, offsets, q, ldq, scale, ld_scale, s);
    return aligned ? run_typed<T, false, true>(blocks, p, R, C, x, ldx, G, offsets, q, ldq, scale, ld_scale, s)
                   : run_typed<T, false, false>(blocks, p, R, C, x, ldx, G, offsets, q, ldq, scale, ld_scale, s);
  };
  if (x_type == TCG_F32) return typed(float{});
  if (x_type == TCG_F16) return typed(__half{});
  return typed(__nv_bfloat16{});
}

}  // namespace

}  // namespace tcg

using namespace tcg;

extern "C" {

int tcg_f8_quantize(tcg_input q_type, tcg_f8_blocks blocks, int pow2, int64_t R, int64_t C, tcg_dtype x_type,
                    const void* X, int64_t ldx, int G, const int32_t* offsets, void* Q, int64_t ldq, float* scale,
                    int64_t ld_scale, void* stream) {
  return guarded([&] {
    return run_quantize(q_type, blocks, pow2, R, C, x_type, X, ldx, G, offsets, Q, ldq, scale, ld_scale,
                        static_cast<cudaStream_t>(stream));
  });
}

}  // extern "C"
