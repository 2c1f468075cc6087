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
// of 16-bit values lie at least 2^-13 off a tie.
//
// Both kernels read X once, keep it in registers between the maximum and the
// codes, and are bound by HBM.  Rows: a half warp (16-bit types) or a warp holds
// a block's row, a warp takes 8 rows so that their 8 loads are in flight
// together and the 8 scales, neighbours in memory, leave as one sector.  Columns
// and squares: a CTA holds 128 x 128.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "common.h"
#include "ptx.cuh"

namespace tcg {

namespace {

constexpr int BLOCK = 128;
constexpr int MAX_GROUPS = 1024;
constexpr int64_t MAX_EXTENT = int64_t{1} << 30;
constexpr int ROW_WARPS = 4;
constexpr int ROWS = 8;  // rows of a warp
constexpr int TILE_THREADS = 256;

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }

// How the values of a block become codes.
struct Coder {
  float by;     // x * by is F x (a in normal range), exact but for fp32's last bit
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

__device__ __forceinline__ float quotient(float x, const Coder& c) {
  const float n = x * c.by;
  const float y = n * c.inv;
  return fmaf(fmaf(-y, c.a, n), c.inv, y);
}

// Four codes, the first in the low byte.
template <bool WIDE>
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
  constexpr __nv_fp8_interpretation_t I = WIDE ? __NV_E5M2 : __NV_E4M3;
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, I);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, I);
  return lo | hi << 16;
}

// NaN are passed over
__device__ __forceinline__ float most(float a, float x) { return fmaxf(a, fabsf(x)); }

// ----------------------------------------------------------------------- rows
//
// V elements a lane, 128 / V lanes a block.  ALIGNED: X in 16-byte words, Q in
// words of V bytes.
template <class T, bool WIDE, bool ALIGNED>
__global__ void __launch_bounds__(32 * ROW_WARPS) row_kernel(int64_t R, int64_t C, const T* __restrict__ X,
                                                             int64_t ldx, bool pow2, uint8_t* __restrict__ Q,
                                                             int64_t ldq, float* __restrict__ scale,
                                                             int64_t ld_scale, int64_t col_warps) {
  constexpr int V = ALIGNED ? 16 / static_cast<int>(sizeof(T)) : 4;
  constexpr int LANES = BLOCK / V;  // 16 or 32
  const int lane = threadIdx.x & 31;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * ROW_WARPS + (threadIdx.x >> 5);
  const int64_t r0 = w / col_warps * ROWS;
  const int64_t c = (w % col_warps) * 32 * V + lane * V;
  griddep_wait();
  if (r0 >= R) return;
  const int rows = static_cast<int>(min(static_cast<int64_t>(ROWS), R - r0));
  float x[ROWS][V];
  uint4 raw[ALIGNED ? ROWS : 1];
  if constexpr (ALIGNED) {
#pragma unroll
    for (int i = 0; i < ROWS; ++i)
      raw[i] = i < rows && c < C ? *reinterpret_cast<const uint4*>(X + (r0 + i) * ldx + c) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      const T* v = reinterpret_cast<const T*>(&raw[i]);
#pragma unroll
      for (int j = 0; j < V; ++j) x[i][j] = to_f32(v[j]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < ROWS; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j) x[i][j] = i < rows && c + j < C ? to_f32(X[(r0 + i) * ldx + c + j]) : 0.0f;
  }
  float mine = 0.0f;  // the scale of row lane % LANES
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    float a = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) a = most(a, x[i][j]);
#pragma unroll
    for (int d = LANES / 2; d; d >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, d));
    float s;
    const Coder k = make_coder<WIDE>(a, pow2, s);
    if (lane % LANES == i) mine = s;
    if (i < rows && c < C) {
      uint8_t* q = Q + (r0 + i) * ldq + c;
      uint32_t code[V / 4];
#pragma unroll
      for (int j = 0; j < V; j += 4)
        code[j / 4] = encode4<WIDE>(quotient(x[i][j], k), quotient(x[i][j + 1], k), quotient(x[i][j + 2], k),
                                    quotient(x[i][j + 3], k));
      if constexpr (ALIGNED && V == 8) {
        *reinterpret_cast<uint2*>(q) = make_uint2(code[0], code[1]);
      } else if constexpr (ALIGNED) {
        *reinterpret_cast<uint32_t*>(q) = code[0];
      } else {
#pragma unroll
        for (int j = 0; j < V; ++j)
          if (c + j < C) q[j] = static_cast<uint8_t>(code[0] >> (8 * j));
      }
    }
  }
  const int64_t block = (c - lane % LANES * V) / BLOCK;
  if (lane % LANES < rows && block * BLOCK < C) scale[block * ld_scale + r0 + lane % LANES] = mine;
  griddep_launch_dependents();
}

// --------------------------------------------------------- columns and squares

// A tile of up to 128 x 128: thread t holds rows t / 16 + 16 i and columns
// 8 (t % 16) .. + 8.  SQUARE: one block; else a block a column.
template <class T, bool WIDE, bool ALIGNED, bool SQUARE>
__global__ void __launch_bounds__(TILE_THREADS) tile_kernel(int64_t R, int64_t C, const T* __restrict__ X, int64_t ldx,
                                                            bool pow2, int G, const int32_t* __restrict__ offsets,
                                                            uint8_t* __restrict__ Q, int64_t ldq,
                                                            float* __restrict__ scale, int64_t ld_scale,
                                                            int64_t col_tiles) {
  __shared__ float top[TILE_THREADS / 32][BLOCK];
  const int t = threadIdx.x;
  const int64_t slot = blockIdx.x / col_tiles;  // the block's row of scales
  const int64_t tile = blockIdx.x % col_tiles;
  const int64_t c = tile * BLOCK + 8 * (t & 15);
  griddep_wait();
  int64_t lo = slot * BLOCK, end = R;
  if (offsets) {
    // block j of group g has slot offsets[g] / 128 + g + j; the slots of groups rise
    int below = 0;
    for (int g = t; g < G; g += TILE_THREADS) {
      const int64_t o = min(max(static_cast<int64_t>(offsets[g]), int64_t{0}), R);
      below += o / BLOCK + g <= slot;
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) below += __shfl_xor_sync(0xffffffffu, below, d);
    int* count = reinterpret_cast<int*>(&top[0][0]);
    if ((t & 31) == 0) count[t >> 5] = below;
    __syncthreads();
    int g = -1;
    for (int i = 0; i < TILE_THREADS / 32; ++i) g += count[i];
    __syncthreads();
    if (g < 0) return;
    const int64_t first = min(max(static_cast<int64_t>(offsets[g]), int64_t{0}), R);
    end = min(max(static_cast<int64_t>(offsets[g + 1]), first), R);
    lo = first + (slot - first / BLOCK - g) * BLOCK;
  }
  if (lo >= end) return;  // a slot that no group uses keeps its value
  const int rows = static_cast<int>(min(static_cast<int64_t>(BLOCK), end - lo));
  // kept in its own type: fp32 values took 64 registers, and a CTA more an SM
  struct alignas(16) Row {
    T v[8];
  } x[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int row = (t >> 4) + 16 * i;
    const T* from = X + (lo + row) * ldx + c;
    if constexpr (ALIGNED) {
      constexpr int V = 16 / static_cast<int>(sizeof(T));
#pragma unroll
      for (int h = 0; h < 8; h += V)
        *reinterpret_cast<uint4*>(&x[i].v[h]) =
            row < rows && c + h < C ? *reinterpret_cast<const uint4*>(from + h) : make_uint4(0, 0, 0, 0);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) x[i].v[j] = row < rows && c + j < C ? from[j] : T(0.0f);
    }
  }
  float a[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    a[j] = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) a[j] = most(a[j], to_f32(x[i].v[j]));
  }
  float s[8];
  Coder k[SQUARE ? 1 : 8];
  if constexpr (SQUARE) {
    float m = a[0];
#pragma unroll
    for (int j = 1; j < 8; ++j) m = fmaxf(m, a[j]);
#pragma unroll
    for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    if ((t & 31) == 0) top[0][t >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < TILE_THREADS / 32; ++i) m = fmaxf(m, top[0][i]);
    k[0] = make_coder<WIDE>(m, pow2, s[0]);
    if (t == 0) scale[slot * ld_scale + tile] = s[0];
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) a[j] = fmaxf(a[j], __shfl_xor_sync(0xffffffffu, a[j], 16));
    if ((t & 31) < 16) {
      *reinterpret_cast<float4*>(&top[t >> 5][8 * (t & 15)]) = make_float4(a[0], a[1], a[2], a[3]);
      *reinterpret_cast<float4*>(&top[t >> 5][8 * (t & 15) + 4]) = make_float4(a[4], a[5], a[6], a[7]);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < TILE_THREADS / 32; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) a[j] = fmaxf(a[j], top[i][8 * (t & 15) + j]);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      k[j] = make_coder<WIDE>(a[j], pow2, s[j]);
      if (t < 16 && c + j < C) scale[slot * ld_scale + c + j] = s[j];
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int row = (t >> 4) + 16 * i;
    if (row >= rows) break;
    uint8_t* q = Q + (lo + row) * ldq + c;
    uint32_t code[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float y[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) y[j] = quotient(to_f32(x[i].v[4 * h + j]), k[SQUARE ? 0 : 4 * h + j]);
      code[h] = encode4<WIDE>(y[0], y[1], y[2], y[3]);
    }
    if constexpr (ALIGNED) {
      if (sizeof(T) == 2) {
        if (c < C) *reinterpret_cast<uint2*>(q) = make_uint2(code[0], code[1]);
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (c + 4 * h < C) *reinterpret_cast<uint32_t*>(q + 4 * h) = code[h];
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (c + j < C) q[j] = static_cast<uint8_t>(code[j / 4] >> (8 * (j % 4)));
    }
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
    constexpr int64_t V = ALIGNED ? 16 / sizeof(T) : 4;
    const int64_t col_warps = ceil_div(C, 32 * V);
    return launch(row_kernel<T, WIDE, ALIGNED>, ceil_div(ceil_div(R, ROWS) * col_warps, ROW_WARPS), 32 * ROW_WARPS, s,
                  R, C, X, ldx, pow2, Q, ldq, scale, ld_scale, col_warps);
  }
  const int64_t tiles = ceil_div(C, BLOCK), slots = offsets ? R / BLOCK + G : ceil_div(R, BLOCK);
  if (blocks == TCG_F8_SQUARE)
    return launch(tile_kernel<T, WIDE, ALIGNED, true>, slots * tiles, TILE_THREADS, s, R, C, X, ldx, pow2, G, offsets,
                  Q, ldq, scale, ld_scale, tiles);
  return launch(tile_kernel<T, WIDE, ALIGNED, false>, slots * tiles, TILE_THREADS, s, R, C, X, ldx, pow2, G, offsets, Q,
                ldq, scale, ld_scale, tiles);
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
