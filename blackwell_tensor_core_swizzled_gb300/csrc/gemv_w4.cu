// Few rows of 16-bit activations against 4-bit matrices with group scales.
// Entry point and kernel; the contract is in include/tcg.h.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "common.h"

namespace tcg {

namespace {

constexpr int MAX_GROUPS = 1024;
constexpr int64_t MAX_EXTENT = int64_t{1} << 30;

__device__ __forceinline__ float decode_e2m1(uint32_t c) {
  const float mag = (c & 6) ? (1.0f + 0.5f * static_cast<float>(c & 1)) * static_cast<float>(1 << ((c & 6) >> 1)) * 0.5f
                            : 0.5f * static_cast<float>(c & 1);
  return (c & 8) ? -mag : mag;
}
__device__ __forceinline__ float decode_e8m0(uint32_t b) {
  return b == 0 ? __uint_as_float(0x00400000u) : b == 255 ? __uint_as_float(0x7FC00000u) : __uint_as_float(b << 23);
}
// unsigned E4M3: the sign bit set is NaN
__device__ __forceinline__ float decode_ue4m3(uint32_t b) {
  if (b >= 0x7Fu) return __uint_as_float(0x7FC00000u);
  const uint32_t e = b >> 3, m = b & 7u;
  return e ? __uint_as_float(((e + 120u) << 23) | (m << 20)) : static_cast<float>(m) * 0x1p-9f;
}

// One warp per output (row r, column n): lanes stride over the 32-code chunks.
__global__ void __launch_bounds__(256) gemv_kernel(const tcg_gemv_w4_args a) {
  const int64_t o = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (o >= a.R * a.N) return;
  const int lane = threadIdx.x & 31;
  const int64_t r = o / a.N, n = o % a.N;
  int g = 0;
  bool found = true;
  if (a.offsets) {
    int64_t hi = 0;
    found = false;
    for (int i = 0; i <= a.G && !found; ++i) {
      const int64_t lo = hi;
      hi = min(max(static_cast<int64_t>(a.offsets[i]), hi), a.R);
      if (i > 0 && r >= lo && r < hi) {
        found = true;
        g = i - 1;
      }
    }
  }
  float acc = 0.0f;
  if (found) {
    const uint8_t* b = a.B + (g * a.stride_b + n * a.ldb) / 2;
    for (int64_t k = 2 * lane; k < a.K; k += 64) {
      const uint32_t byte = b[k / 2];
      const int64_t si = g * a.stride_scale + n * a.ld_scale + k / a.group;
      float s, z = 0.0f;
      if (a.format == TCG_W4_INT4) {
        s = a.in_type == TCG_IN_BF16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(a.scale)[si])
                                     : __half2float(static_cast<const __half*>(a.scale)[si]);
        z = a.zero ? static_cast<float>(a.zero[si]) : 8.0f;
      } else {
        const uint32_t sb = static_cast<const uint8_t*>(a.scale)[si];
        s = a.format == TCG_W4_MXF4 ? decode_e8m0(sb) : decode_ue4m3(sb);
      }
      for (int i = 0; i < 2; ++i) {
        const uint32_t c = (byte >> (4 * i)) & 15u;
        const float v = a.format == TCG_W4_INT4 ? static_cast<float>(c) - z : decode_e2m1(c);
        const float x = a.in_type == TCG_IN_BF16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(a.A)[r * a.lda + k + i])
                                                 : __half2float(static_cast<const __half*>(a.A)[r * a.lda + k + i]);
        acc += v * x * s;  // the scale last: v * s alone could overflow where x is 0
      }
    }
  }
  for (int d = 16; d > 0; d >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, d);
  if (lane) return;
  if (found && a.alpha) acc *= a.alpha[g];
  const int64_t i = r * a.ldd + n;
  if (a.d_type == TCG_F32)
    static_cast<float*>(a.D)[i] = acc;
  else if (a.d_type == TCG_F16)
    static_cast<__half*>(a.D)[i] = __float2half_rn(acc);
  else
    static_cast<__nv_bfloat16*>(a.D)[i] = __float2bfloat16_rn(acc);
}

int run_gemv(const tcg_gemv_w4_args* args, cudaStream_t s) {
  set_launch_count(0);
  if (!args) return TCG_ERR_INVALID;
  tcg_gemv_w4_args a = *args;
  if (a.format < TCG_W4_INT4 || a.format > TCG_W4_NVF4) return TCG_ERR_INVALID;
  if (a.in_type != TCG_IN_F16 && a.in_type != TCG_IN_BF16) return TCG_ERR_INVALID;
  if (a.d_type < TCG_F32 || a.d_type > TCG_BF16) return TCG_ERR_INVALID;
  if (a.R < 0 || a.N < 0 || a.K < 0 || a.G < 1) return TCG_ERR_INVALID;
  if (a.R >= MAX_EXTENT || a.N >= MAX_EXTENT || a.K >= MAX_EXTENT || a.G > MAX_GROUPS) return TCG_ERR_UNSUPPORTED;
  if (a.format != TCG_W4_INT4) {
    const int block = a.format == TCG_W4_MXF4 ? 32 : 16;
    if (a.group == 0) a.group = block;
    if (a.group != block || a.zero) return TCG_ERR_INVALID;
  } else if (a.group != 32 && a.group != 64 && a.group != 128) {
    return a.group <= 0 ? TCG_ERR_INVALID : TCG_ERR_UNSUPPORTED;
  }
  if (!a.offsets && a.G != 1) return TCG_ERR_INVALID;
  if (a.R == 0 || a.N == 0) return TCG_OK;
  if (a.ldd == 0) a.ldd = a.N;
  if (!a.D || a.ldd < a.N) return TCG_ERR_INVALID;
  if (reinterpret_cast<uintptr_t>(a.D) % (a.d_type == TCG_F32 ? 4 : 2)) return TCG_ERR_ALIGNMENT;
  if ((reinterpret_cast<uintptr_t>(a.offsets) | reinterpret_cast<uintptr_t>(a.alpha)) % 4) return TCG_ERR_ALIGNMENT;
  if (a.K > 0) {
    if (a.K % 32 || a.K % a.group) return TCG_ERR_ALIGNMENT;
    if (a.lda == 0) a.lda = a.K;
    if (a.ldb == 0) a.ldb = a.K;
    if (a.ld_scale == 0) a.ld_scale = a.K / a.group;
    if (a.lda < a.K || a.ldb < a.K || a.ld_scale < a.K / a.group) return TCG_ERR_INVALID;
    if (a.stride_b == 0) a.stride_b = a.N * a.ldb;
    if (a.stride_scale == 0) a.stride_scale = a.N * a.ld_scale;
    if (!a.A || !a.B || !a.scale || a.stride_b < 0 || a.stride_scale < 0) return TCG_ERR_INVALID;
    if (reinterpret_cast<uintptr_t>(a.A) % 16 || a.lda % 8 || reinterpret_cast<uintptr_t>(a.B) % 16 || a.ldb % 32 ||
        a.stride_b % 32)
      return TCG_ERR_ALIGNMENT;
    if (a.format == TCG_W4_INT4 && reinterpret_cast<uintptr_t>(a.scale) % 2) return TCG_ERR_ALIGNMENT;
  }
  int dev;
  if (int rc = current_device_checked(&dev)) return rc;
  if (a.R * a.N > (int64_t{1} << 33)) return TCG_ERR_UNSUPPORTED;
  gemv_kernel<<<static_cast<unsigned>((a.R * a.N + 7) / 8), 256, 0, s>>>(a);
  if (int rc = record_cuda(cudaGetLastError())) return rc;
  set_launch_count(1);
  return TCG_OK;
}

}  // namespace

}  // namespace tcg

using namespace tcg;

extern "C" int tcg_gemv_w4(const tcg_gemv_w4_args* args, void* stream) {
  return guarded([&] { return run_gemv(args, static_cast<cudaStream_t>(stream)); });
}
