// Products of sorted rows with their group's matrix, and the gradient of the
// matrices.  Entry points and kernels; the contract is in include/tcg.h.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "common.h"

namespace tcg {

namespace {

constexpr int MAX_GROUPS = 1024;
constexpr int64_t MAX_EXTENT = int64_t{1} << 30;

struct GroupedArgs {
  const void *A, *B;
  const int32_t* offsets;
  void* D;
  int64_t R, N, K, lda, ldb, stride_b, ldd, stride_d;
  int G;
  int bf16, mn, d_type;
};

__device__ __forceinline__ float load16(const void* p, int64_t i, int bf16) {
  return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i])
              : __half2float(static_cast<const __half*>(p)[i]);
}

__device__ __forceinline__ void store_out(void* p, int64_t i, int type, float v) {
  if (type == TCG_F32)
    static_cast<float*>(p)[i] = v;
  else if (type == TCG_F16)
    static_cast<__half*>(p)[i] = __float2half_rn(v);
  else
    static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
}

// offsets[g] as the kernels use it: never below the previous one, never past R
__device__ __forceinline__ int64_t clamp_offset(int64_t o, int64_t lo, int64_t R) {
  return o < lo ? lo : o > R ? R : o;
}

// 64 x 64 tiles of C = P^T Q over a contracted range, 256 threads, 4 x 4 each.
// Forward: one block per (row tile, column tile), each row of the tile with
// its own group, the tile walked group by group.
__global__ void __launch_bounds__(256) grouped_kernel(const GroupedArgs a) {
  __shared__ float sa[16][65], sb[16][65];
  __shared__ int64_t bounds[2];
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int64_t r0 = static_cast<int64_t>(blockIdx.y) * 64, n0 = static_cast<int64_t>(blockIdx.x) * 64;
  float out[4][4] = {};
  int64_t prev = 0;
  for (int g = 0; g < a.G; ++g) {
    if (threadIdx.x == 0) {
      bounds[0] = clamp_offset(a.offsets[g], prev, a.R);
      bounds[1] = clamp_offset(a.offsets[g + 1], bounds[0], a.R);
    }
    __syncthreads();
    const int64_t lo = bounds[0], hi = bounds[1];
    prev = lo;
    __syncthreads();
    if (hi <= r0 || lo >= r0 + 64 || lo == hi) continue;
    float acc[4][4] = {};
    for (int64_t k0 = 0; k0 < a.K; k0 += 16) {
      for (int i = threadIdx.x; i < 1024; i += 256) {
        const int kk = i & 15, m = i >> 4;
        sa[kk][m] = r0 + m < a.R && k0 + kk < a.K ? load16(a.A, (r0 + m) * a.lda + k0 + kk, a.bf16) : 0.0f;
        const int64_t n = n0 + m, k = k0 + kk;
        sb[kk][m] = n < a.N && k < a.K ? load16(a.B, g * a.stride_b + (a.mn ? k * a.ldb + n : n * a.ldb + k), a.bf16) : 0.0f;
      }
      __syncthreads();
      for (int kk = 0; kk < 16; ++kk)
        for (int i = 0; i < 4; ++i)
          for (int j = 0; j < 4; ++j) acc[i][j] += sa[kk][ty + 16 * i] * sb[kk][tx + 16 * j];
      __syncthreads();
    }
    for (int i = 0; i < 4; ++i) {
      const int64_t r = r0 + ty + 16 * i;
      if (r >= lo && r < hi)
        for (int j = 0; j < 4; ++j) out[i][j] = acc[i][j];
    }
  }
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int64_t r = r0 + ty + 16 * i, n = n0 + tx + 16 * j;
      if (r < a.R && n < a.N) store_out(a.D, r * a.ldd + n, a.d_type, out[i][j]);
    }
}

// Matrix gradient: one block per (k tile, n tile, group); A = DY, B = A.
__global__ void __launch_bounds__(256) grouped_wgrad_kernel(const GroupedArgs a) {
  __shared__ float sa[16][65], sb[16][65];
  __shared__ int64_t bounds[2];
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int64_t k0 = static_cast<int64_t>(blockIdx.x) * 64, n0 = static_cast<int64_t>(blockIdx.y) * 64;
  const int g = blockIdx.z;
  if (threadIdx.x == 0) {
    int64_t lo = 0, hi = 0;
    for (int i = 0; i <= g + 1; ++i) {
      lo = hi;
      hi = clamp_offset(a.offsets[i], hi, a.R);
    }
    bounds[0] = lo;
    bounds[1] = hi;
  }
  __syncthreads();
  const int64_t lo = bounds[0], hi = bounds[1];
  float acc[4][4] = {};
  for (int64_t r0 = lo; r0 < hi; r0 += 16) {
    for (int i = threadIdx.x; i < 1024; i += 256) {
      const int m = i & 63, rr = i >> 6;
      sa[rr][m] = r0 + rr < hi && n0 + m < a.N ? load16(a.A, (r0 + rr) * a.lda + n0 + m, a.bf16) : 0.0f;
      sb[rr][m] = r0 + rr < hi && k0 + m < a.K ? load16(a.B, (r0 + rr) * a.ldb + k0 + m, a.bf16) : 0.0f;
    }
    __syncthreads();
    for (int rr = 0; rr < 16; ++rr)
      for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) acc[i][j] += sa[rr][ty + 16 * i] * sb[rr][tx + 16 * j];
    __syncthreads();
  }
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int64_t n = n0 + ty + 16 * i, k = k0 + tx + 16 * j;
      if (n < a.N && k < a.K) store_out(a.D, g * a.stride_d + n * a.ldd + k, a.d_type, acc[i][j]);
    }
}

// ---------------------------------------------------------------------- host

int check_problem(tcg_input in_type, int64_t R, int64_t N, int64_t K, int G, tcg_dtype d_type) {
  if (in_type != TCG_IN_F16 && in_type != TCG_IN_BF16) return TCG_ERR_INVALID;
  if (R < 0 || N < 0 || K < 0 || G < 1 || d_type < TCG_F32 || d_type > TCG_BF16) return TCG_ERR_INVALID;
  if (R >= MAX_EXTENT || N >= MAX_EXTENT || K >= MAX_EXTENT || G > MAX_GROUPS) return TCG_ERR_UNSUPPORTED;
  return TCG_OK;
}

// 16-bit operand rows the tensor-map rules apply to: ld >= inner, 16 bytes
int check_operand16(const void* p, int64_t inner, int64_t* ld) {
  if (*ld == 0) *ld = inner;
  if (!p || *ld < inner || *ld < 1) return TCG_ERR_INVALID;
  return reinterpret_cast<uintptr_t>(p) % 16 || *ld % 8 ? TCG_ERR_ALIGNMENT : TCG_OK;
}

int check_output(const void* p, int64_t inner, int64_t* ld, tcg_dtype type) {
  if (*ld == 0) *ld = inner;
  if (!p || *ld < inner) return TCG_ERR_INVALID;
  return reinterpret_cast<uintptr_t>(p) % (type == TCG_F32 ? 4 : 2) ? TCG_ERR_ALIGNMENT : TCG_OK;
}

int check_offsets(const int32_t* p) {
  if (!p) return TCG_ERR_INVALID;
  return reinterpret_cast<uintptr_t>(p) % 4 ? TCG_ERR_ALIGNMENT : TCG_OK;
}

int run_grouped(tcg_input in_type, int64_t R, int64_t N, int64_t K, int G, const void* A, int64_t lda,
                const int32_t* offsets, const void* B, tcg_major b_major, int64_t ldb, int64_t stride_b, void* D,
                tcg_dtype d_type, int64_t ldd, cudaStream_t s) {
  set_launch_count(0);
  if (int rc = check_problem(in_type, R, N, K, G, d_type)) return rc;
  if (b_major != TCG_K_MAJOR && b_major != TCG_MN_MAJOR) return TCG_ERR_INVALID;
  if (R == 0 || N == 0) return TCG_OK;
  if (int rc = check_output(D, N, &ldd, d_type)) return rc;
  if (int rc = check_offsets(offsets)) return rc;
  if (K > 0) {
    const int64_t inner = b_major == TCG_K_MAJOR ? K : N, outer = b_major == TCG_K_MAJOR ? N : K;
    if (int rc = check_operand16(A, K, &lda)) return rc;
    if (int rc = check_operand16(B, inner, &ldb)) return rc;
    if (stride_b == 0) stride_b = outer * ldb;
    if (stride_b < 0) return TCG_ERR_INVALID;
    if (stride_b % 8) return TCG_ERR_ALIGNMENT;
  }
  int dev;
  if (int rc = current_device_checked(&dev)) return rc;
  GroupedArgs a{A, B, offsets, D, R, N, K, lda, ldb, stride_b, ldd, 0, G, in_type == TCG_IN_BF16,
                b_major == TCG_MN_MAJOR, d_type};
  grouped_kernel<<<dim3(static_cast<unsigned>((N + 63) / 64), static_cast<unsigned>((R + 63) / 64)), 256, 0, s>>>(a);
  if (int rc = record_cuda(cudaGetLastError())) return rc;
  set_launch_count(1);
  return TCG_OK;
}

int run_wgrad(tcg_input in_type, int64_t R, int64_t N, int64_t K, int G, const void* DY, int64_t lddy, const void* A,
              int64_t lda, const int32_t* offsets, void* DW, tcg_dtype dw_type, int64_t lddw, int64_t stride_dw,
              cudaStream_t s) {
  set_launch_count(0);
  if (int rc = check_problem(in_type, R, N, K, G, dw_type)) return rc;
  if (N == 0 || K == 0) return TCG_OK;
  if (int rc = check_output(DW, K, &lddw, dw_type)) return rc;
  if (stride_dw == 0) stride_dw = N * lddw;
  if (stride_dw < 0) return TCG_ERR_INVALID;
  if (int rc = check_offsets(offsets)) return rc;
  if (R > 0) {
    if (int rc = check_operand16(DY, N, &lddy)) return rc;
    if (int rc = check_operand16(A, K, &lda)) return rc;
  }
  int dev;
  if (int rc = current_device_checked(&dev)) return rc;
  GroupedArgs a{DY, A, offsets, DW, R, N, K, lddy, lda, 0, lddw, stride_dw, G, in_type == TCG_IN_BF16, 0, dw_type};
  grouped_wgrad_kernel<<<dim3(static_cast<unsigned>((K + 63) / 64), static_cast<unsigned>((N + 63) / 64),
                              static_cast<unsigned>(G)), 256, 0, s>>>(a);
  if (int rc = record_cuda(cudaGetLastError())) return rc;
  set_launch_count(1);
  return TCG_OK;
}

}  // namespace

}  // namespace tcg

using namespace tcg;

extern "C" {

int tcg_gemm_grouped(tcg_input in_type, int64_t R, int64_t N, int64_t K, int G, const void* A, int64_t lda,
                     const int32_t* offsets, const void* B, tcg_major b_major, int64_t ldb, int64_t stride_b,
                     void* D, tcg_dtype d_type, int64_t ldd, void* stream) {
  return guarded([&] {
    return run_grouped(in_type, R, N, K, G, A, lda, offsets, B, b_major, ldb, stride_b, D, d_type, ldd,
                       static_cast<cudaStream_t>(stream));
  });
}

int tcg_gemm_grouped_wgrad(tcg_input in_type, int64_t R, int64_t N, int64_t K, int G, const void* DY, int64_t lddy,
                           const void* A, int64_t lda, const int32_t* offsets, void* DW, tcg_dtype dw_type,
                           int64_t lddw, int64_t stride_dw, void* stream) {
  return guarded([&] {
    return run_wgrad(in_type, R, N, K, G, DY, lddy, A, lda, offsets, DW, dw_type, lddw, stride_dw,
                     static_cast<cudaStream_t>(stream));
  });
}

}  // extern "C"
