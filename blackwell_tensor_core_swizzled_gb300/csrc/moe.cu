// Mixture-of-experts routing: the order of the tokens' choices by expert, the
// copy of token rows to their sorted positions, the weighted sum back, and its
// gradient.  Entry points and kernels; the contract is in include/tcg.h.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "common.h"

namespace tcg {

namespace {

constexpr int MAX_EXPERTS = 1024;

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <class T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// ---------------------------------------------------------------------- sort
//
// A stable counting sort: rank of entry i in bucket e (its expert, or E when
// dropped) = entries of smaller buckets + entries of e before i.  Every warp
// owns a contiguous range of entries; counts[w][e] is first the number of
// entries of e in warp w's range, then (exclusive sums over warps and
// buckets) the rank of the warp's next entry of e.  Within 32 entries the
// lanes of one bucket find each other with match_any and take consecutive
// ranks in lane order, so the order never depends on timing.
constexpr int SORT_WARPS = 32;

__device__ __forceinline__ int bucket_of(int expert, int E) {
  return static_cast<unsigned>(expert) < static_cast<unsigned>(E) ? expert : E;
}

__global__ void __launch_bounds__(32 * SORT_WARPS) sort_kernel(int n, int E, const int32_t* __restrict__ expert,
                                                               int32_t* __restrict__ offsets,
                                                               int32_t* __restrict__ position,
                                                               int32_t* __restrict__ source) {
  extern __shared__ int counts[];  // [SORT_WARPS][E + 1]
  __shared__ int warp_sum[32];
  const int NB = E + 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < SORT_WARPS * NB; i += blockDim.x) counts[i] = 0;
  __syncthreads();
  const int per = ((n + SORT_WARPS - 1) / SORT_WARPS + 31) / 32 * 32;  // entries per warp, whole rounds
  const int lo = min(n, warp * per), hi = min(n, lo + per);
  int* mine = counts + warp * NB;
  for (int i0 = lo; i0 < hi; i0 += 32) {
    const int i = i0 + lane;
    const int b = i < hi ? bucket_of(expert[i], E) : -1;
    const unsigned same = __match_any_sync(0xffffffffu, b);
    if (b >= 0 && lane == __ffs(same) - 1) mine[b] += __popc(same);
    __syncwarp();
  }
  __syncthreads();
  // exclusive sums over the warps for each bucket, then over the buckets: the
  // thread of bucket b (NB <= 1025: the thread of bucket 0 also takes 1024)
  int total = 0;
  const int b = threadIdx.x;
  if (b < NB) {
    for (int w = 0; w < SORT_WARPS; ++w) {
      const int c = counts[w * NB + b];
      counts[w * NB + b] = total;
      total += c;
    }
  }
  int incl = total;
  for (int d = 1; d < 32; d <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += v;
  }
  if (lane == 31) warp_sum[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    int s = warp_sum[lane];
    for (int d = 1; d < 32; d <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, s, d);
      if (lane >= d) s += v;
    }
    warp_sum[lane] = s;
  }
  __syncthreads();
  const int start = incl - total + (warp ? warp_sum[warp - 1] : 0);
  if (b < NB) {
    offsets[b] = start;  // offsets[E] = start of the dropped bucket
    for (int w = 0; w < SORT_WARPS; ++w) counts[w * NB + b] += start;
  }
  if (NB > 1024 && b == 0) {  // bucket 1024: the dropped entries of E = 1024
    int t = warp_sum[31];
    offsets[1024] = t;
    for (int w = 0; w < SORT_WARPS; ++w) {
      const int c = counts[w * NB + 1024];
      counts[w * NB + 1024] = t;
      t += c;
    }
  }
  __syncthreads();
  for (int i0 = lo; i0 < hi; i0 += 32) {
    const int i = i0 + lane;
    const int e = i < hi ? bucket_of(expert[i], E) : -1;
    const unsigned same = __match_any_sync(0xffffffffu, e);
    if (e >= 0) {
      const int p = mine[e] + __popc(same & ((1u << lane) - 1u));
      position[i] = e < E ? p : -1 - p;
      source[p] = i;
    }
    __syncwarp();
    if (e >= 0 && lane == __ffs(same) - 1) mine[e] += __popc(same);
    __syncwarp();
  }
}

// ------------------------------------------------------- dispatch and combine

template <class T>
__global__ void dispatch_kernel(int topk, int64_t H, const T* __restrict__ X, int64_t ldx,
                                const int32_t* __restrict__ position, T* __restrict__ Xs, int64_t ldxs) {
  const int64_t i = blockIdx.x;
  const int p = position[i];
  const T* src = X + (i / topk) * ldx;
  T* dst = Xs + static_cast<int64_t>(p < 0 ? -1 - p : p) * ldxs;
  for (int64_t h = threadIdx.x; h < H; h += blockDim.x) dst[h] = p < 0 ? from_f32<T>(0.0f) : src[h];
}

template <class T>
__global__ void combine_kernel(int topk, int64_t H, const T* __restrict__ Ys, int64_t ldys,
                               const int32_t* __restrict__ position, const float* __restrict__ weight,
                               T* __restrict__ Y, int64_t ldy) {
  const int64_t t = blockIdx.x;
  for (int64_t h = threadIdx.x; h < H; h += blockDim.x) {
    float acc = 0.0f;
    for (int j = 0; j < topk; ++j) {
      const int p = position[t * topk + j];
      if (p >= 0) acc += (weight ? weight[t * topk + j] : 1.0f) * to_f32(Ys[static_cast<int64_t>(p) * ldys + h]);
    }
    Y[t * ldy + h] = from_f32<T>(acc);
  }
}

template <class T>
__global__ void __launch_bounds__(256) combine_grad_kernel(int topk, int64_t H, const T* __restrict__ dY, int64_t lddy,
                                                           const T* __restrict__ Ys, int64_t ldys,
                                                           const int32_t* __restrict__ position,
                                                           const float* __restrict__ weight, T* __restrict__ dYs,
                                                           int64_t lddys, float* __restrict__ dweight) {
  const int64_t i = blockIdx.x;
  const int p = position[i];
  const int64_t row = p < 0 ? -1 - p : p;
  const T* g = dY + (i / topk) * lddy;
  const float w = weight ? weight[i] : 1.0f;
  float dot = 0.0f;
  for (int64_t h = threadIdx.x; h < H; h += blockDim.x) {
    const float d = p < 0 ? 0.0f : to_f32(g[h]);
    dYs[row * lddys + h] = from_f32<T>(p < 0 ? 0.0f : w * d);
    if (Ys && p >= 0) dot += d * to_f32(Ys[row * ldys + h]);
  }
  if (!dweight) return;
  __shared__ float part[8];
  for (int d = 16; d > 0; d >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, d);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = dot;
  __syncthreads();
  if (threadIdx.x == 0) {
    float s = 0.0f;
    for (int k = 0; k < 8; ++k) s += part[k];
    dweight[i] = s;
  }
}

// ---------------------------------------------------------------------- host

constexpr int64_t MAX_ENTRIES = int64_t{1} << 30;

int check_route(tcg_dtype type, int64_t T, int topk, int64_t H) {
  if (type < TCG_F32 || type > TCG_BF16 || T < 0 || topk < 1 || H < 0) return TCG_ERR_INVALID;
  if (topk > 64 || T * topk >= MAX_ENTRIES || T >= MAX_ENTRIES || H >= MAX_ENTRIES) return TCG_ERR_UNSUPPORTED;
  return TCG_OK;
}

// One matrix argument: base and leading dimension (0 = H).
int check_rows(const void* p, int64_t H, int64_t* ld, tcg_dtype type) {
  if (*ld == 0) *ld = H;
  if (!p || *ld < H) return TCG_ERR_INVALID;
  if (reinterpret_cast<uintptr_t>(p) % (type == TCG_F32 ? 4 : 2)) return TCG_ERR_ALIGNMENT;
  return TCG_OK;
}

int check_words(const void* p) {
  if (!p) return TCG_ERR_INVALID;
  return reinterpret_cast<uintptr_t>(p) % 4 ? TCG_ERR_ALIGNMENT : TCG_OK;
}

int launched(int launches) {
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return record_cuda(e);
  set_launch_count(launches);
  return TCG_OK;
}

int run_sort(int64_t T, int topk, int E, const int32_t* expert, int32_t* offsets, int32_t* position, int32_t* source,
             cudaStream_t s) {
  set_launch_count(0);
  if (T < 0 || topk < 1 || E < 1) return TCG_ERR_INVALID;
  if (E > MAX_EXPERTS || T >= MAX_ENTRIES || topk >= MAX_ENTRIES || T * topk >= MAX_ENTRIES)
    return TCG_ERR_UNSUPPORTED;
  if (int rc = check_words(offsets)) return rc;
  if (T > 0) {
    if (int rc = check_words(expert)) return rc;
    if (int rc = check_words(position)) return rc;
    if (int rc = check_words(source)) return rc;
  }
  int dev;
  if (int rc = current_device_checked(&dev)) return rc;
  const int smem = SORT_WARPS * (E + 1) * 4;
  if (int rc = record_cuda(cudaFuncSetAttribute(sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)))
    return rc;
  sort_kernel<<<1, 32 * SORT_WARPS, smem, s>>>(static_cast<int>(T * topk), E, expert, offsets, position, source);
  return launched(1);
}

template <class F>
void for_type(tcg_dtype type, F&& f) {
  if (type == TCG_F32)
    f(float{});
  else if (type == TCG_F16)
    f(__half{});
  else
    f(__nv_bfloat16{});
}

int run_dispatch(tcg_dtype type, int64_t T, int topk, int64_t H, const void* X, int64_t ldx, const int32_t* position,
                 void* Xs, int64_t ldxs, cudaStream_t s) {
  set_launch_count(0);
  if (int rc = check_route(type, T, topk, H)) return rc;
  if (T == 0 || H == 0) return TCG_OK;
  if (int rc = check_rows(X, H, &ldx, type)) return rc;
  if (int rc = check_rows(Xs, H, &ldxs, type)) return rc;
  if (int rc = check_words(position)) return rc;
  int dev;
  if (int rc = current_device_checked(&dev)) return rc;
  for_type(type, [&](auto z) {
    using E = decltype(z);
    dispatch_kernel<E><<<static_cast<unsigned>(T * topk), 256, 0, s>>>(topk, H, static_cast<const E*>(X), ldx, position,
                                                                       static_cast<E*>(Xs), ldxs);
  });
  return launched(1);
}

int run_combine(tcg_dtype type, int64_t T, int topk, int64_t H, const void* Ys, int64_t ldys, const int32_t* position,
                const float* weight, void* Y, int64_t ldy, cudaStream_t s) {
  set_launch_count(0);
  if (int rc = check_route(type, T, topk, H)) return rc;
  if (T == 0 || H == 0) return TCG_OK;
  if (int rc = check_rows(Ys, H, &ldys, type)) return rc;
  if (int rc = check_rows(Y, H, &ldy, type)) return rc;
  if (int rc = check_words(position)) return rc;
  if (reinterpret_cast<uintptr_t>(weight) % 4) return TCG_ERR_ALIGNMENT;
  int dev;
  if (int rc = current_device_checked(&dev)) return rc;
  for_type(type, [&](auto z) {
    using E = decltype(z);
    combine_kernel<E><<<static_cast<unsigned>(T), 256, 0, s>>>(topk, H, static_cast<const E*>(Ys), ldys, position,
                                                               weight, static_cast<E*>(Y), ldy);
  });
  return launched(1);
}

int run_combine_grad(tcg_dtype type, int64_t T, int topk, int64_t H, const void* dY, int64_t lddy, const void* Ys,
                     int64_t ldys, const int32_t* position, const float* weight, void* dYs, int64_t lddys,
                     float* dweight, cudaStream_t s) {
  set_launch_count(0);
  if (int rc = check_route(type, T, topk, H)) return rc;
  if ((Ys == nullptr) != (dweight == nullptr)) return TCG_ERR_INVALID;
  if (T == 0 || (H == 0 && !dweight)) return TCG_OK;
  if (dweight) {
    if (int rc = check_words(dweight)) return rc;
    if (int rc = check_rows(Ys, H, &ldys, type)) return rc;
  }
  if (int rc = check_rows(dY, H, &lddy, type)) return rc;
  if (int rc = check_rows(dYs, H, &lddys, type)) return rc;
  if (int rc = check_words(position)) return rc;
  if (reinterpret_cast<uintptr_t>(weight) % 4) return TCG_ERR_ALIGNMENT;
  int dev;
  if (int rc = current_device_checked(&dev)) return rc;
  for_type(type, [&](auto z) {
    using E = decltype(z);
    combine_grad_kernel<E><<<static_cast<unsigned>(T * topk), 256, 0, s>>>(
        topk, H, static_cast<const E*>(dY), lddy, static_cast<const E*>(Ys), ldys, position, weight,
        static_cast<E*>(dYs), lddys, dweight);
  });
  return launched(1);
}

}  // namespace

}  // namespace tcg

using namespace tcg;

extern "C" {

int tcg_moe_sort(int64_t T, int topk, int E, const int32_t* expert, int32_t* offsets, int32_t* position,
                 int32_t* source, void* stream) {
  return guarded([&] { return run_sort(T, topk, E, expert, offsets, position, source, static_cast<cudaStream_t>(stream)); });
}

int tcg_moe_dispatch(tcg_dtype type, int64_t T, int topk, int64_t H, const void* X, int64_t ldx,
                     const int32_t* position, void* Xs, int64_t ldxs, void* stream) {
  return guarded([&] {
    return run_dispatch(type, T, topk, H, X, ldx, position, Xs, ldxs, static_cast<cudaStream_t>(stream));
  });
}

int tcg_moe_combine(tcg_dtype type, int64_t T, int topk, int64_t H, const void* Ys, int64_t ldys,
                    const int32_t* position, const float* weight, void* Y, int64_t ldy, void* stream) {
  return guarded([&] {
    return run_combine(type, T, topk, H, Ys, ldys, position, weight, Y, ldy, static_cast<cudaStream_t>(stream));
  });
}

int tcg_moe_combine_grad(tcg_dtype type, int64_t T, int topk, int64_t H, const void* dY, int64_t lddy,
                         const void* Ys, int64_t ldys, const int32_t* position, const float* weight, void* dYs,
                         int64_t lddys, float* dweight, void* stream) {
  return guarded([&] {
    return run_combine_grad(type, T, topk, H, dY, lddy, Ys, ldys, position, weight, dYs, lddys, dweight,
                            static_cast<cudaStream_t>(stream));
  });
}

}  // extern "C"
