// Mixture-of-experts routing: the order of the tokens' choices by expert, the
// copy of token rows to their sorted positions, the weighted sum back, and its
// gradient.  Entry points and kernels; the contract is in include/tcg.h.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "common.h"
#include "once.h"
#include "ptx.cuh"

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
// dropped) = entries of smaller buckets + entries of e before i.  A cluster of
// SORT_CTAS CTAs sorts (one CTA up to SORT_ONE entries, where the cluster's
// barriers would cost more than they save); every warp owns a contiguous range
// of entries.  counts[w][e] is first the number of entries of e in warp w's
// range; exclusive sums over the warps of a CTA, the CTAs of the cluster (read
// from their shared memory) and the buckets turn it into the rank of the
// warp's next entry of e.  Within 32 entries the lanes of one bucket find each
// other with a vote for every bit of the bucket's number (match_any walks the
// distinct values one by one) and take consecutive ranks in lane order, so the
// order never depends on timing.
//
// It is bound by the latency of its rounds, so the entries are spread: 65536
// of 64 experts take 8.9 us on 16 CTAs, 12.6 on 8 (1 M entries 78 and 150);
// below SORT_ONE one CTA is quicker (144 entries 3.1 us; 2048 5.6 on 16).
constexpr int SORT_WARPS = 32;
constexpr int SORT_CTAS = 16;  // above 8: opted in to
constexpr int SORT_ONE = 2048;
constexpr int SORT_ROUNDS = 8;

__device__ __forceinline__ int bucket_of(int expert, int E) {
  return static_cast<unsigned>(expert) < static_cast<unsigned>(E) ? expert : E;
}

__device__ __forceinline__ int ld_cluster_s32(uint32_t addr) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}

// Lanes whose bucket is this lane's; buckets below 2^bits, -1 matches -1.
__device__ __forceinline__ unsigned same_bucket(int b, int bits) {
  unsigned same = __ballot_sync(0xffffffffu, b < 0);
  if (b >= 0) same = ~same;
  for (int i = 0; i < bits; ++i) {
    const unsigned ones = __ballot_sync(0xffffffffu, (b >> i) & 1);
    same &= (b >> i) & 1 ? ones : ~ones;
  }
  return same;
}

// Exclusive sum of one value a thread over the CTA's 32 warps; total to all.
__device__ __forceinline__ int block_scan(int v, int* warp_sum, int* total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int incl = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += o;
  }
  if (lane == 31) warp_sum[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    int w = warp_sum[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, w, d);
      if (lane >= d) w += o;
    }
    warp_sum[lane] = w;
  }
  __syncthreads();
  *total = warp_sum[31];
  return incl - v + (warp ? warp_sum[warp - 1] : 0);
}

template <int CTAS>
__global__ void __launch_bounds__(32 * SORT_WARPS) sort_kernel(int n, int E, const int32_t* __restrict__ expert,
                                                               int32_t* __restrict__ offsets,
                                                               int32_t* __restrict__ position,
                                                               int32_t* __restrict__ source) {
  extern __shared__ int counts[];  // [SORT_WARPS][E + 1], then this CTA's counts [E + 1]
  __shared__ int warp_sum[32];
  const int NB = E + 1;
  int* cta_counts = counts + SORT_WARPS * NB;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = CTAS > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  for (int i = threadIdx.x; i < SORT_WARPS * NB; i += blockDim.x) counts[i] = 0;
  __syncthreads();
  griddep_wait();
  griddep_launch_dependents();
  const int parts = CTAS * SORT_WARPS;
  const int per = ((n + parts - 1) / parts + 31) / 32 * 32;  // entries per warp, whole rounds
  const int64_t from = static_cast<int64_t>(rank * SORT_WARPS + warp) * per;
  const int lo = static_cast<int>(min(static_cast<int64_t>(n), from));
  const int hi = static_cast<int>(min(static_cast<int64_t>(n), from + per));
  int* mine = counts + warp * NB;
  const int bits = 32 - __clz(E);  // of the largest bucket, E
  // SORT_ROUNDS rounds of 32 entries are read at once
  int buckets[SORT_ROUNDS];
  auto read = [&](int i0) {
#pragma unroll
    for (int r = 0; r < SORT_ROUNDS; ++r) {
      const int i = i0 + 32 * r + lane;
      buckets[r] = i < hi ? bucket_of(expert[i], E) : -1;
    }
  };
  for (int i0 = lo; i0 < hi; i0 += 32 * SORT_ROUNDS) {
    read(i0);
#pragma unroll
    for (int r = 0; r < SORT_ROUNDS; ++r) {
      if (i0 + 32 * r >= hi) break;
      const unsigned same = same_bucket(buckets[r], bits);
      if (buckets[r] >= 0 && lane == __ffs(same) - 1) mine[buckets[r]] += __popc(same);
      __syncwarp();
    }
  }
  __syncthreads();
  // over the warps, for each bucket (a thread each; NB <= 1025: two for the first)
  for (int b = threadIdx.x; b < NB; b += 32 * SORT_WARPS) {
    int total = 0;
#pragma unroll 8
    for (int w = 0; w < SORT_WARPS; ++w) {
      const int c = counts[w * NB + b];
      counts[w * NB + b] = total;
      total += c;
    }
    cta_counts[b] = total;
  }
  if constexpr (CTAS > 1)
    cluster_sync();
  else
    __syncthreads();
  // over the cluster's CTAs and the buckets; bucket 1024 follows the others
  int carry = 0;
  for (int b0 = 0; b0 < NB; b0 += 32 * SORT_WARPS) {
    const int b = b0 + static_cast<int>(threadIdx.x);
    int total = 0, before = 0;
    if (b < NB) {
      if constexpr (CTAS > 1) {
        const uint32_t at = smem_u32(cta_counts + b);
#pragma unroll
        for (int r = 0; r < CTAS; ++r) {
          const int c = ld_cluster_s32(mapa_shared(at, r));
          if (r < rank) before += c;
          total += c;
        }
      } else {
        total = cta_counts[b];
      }
    }
    int sum;
    const int start = carry + block_scan(total, warp_sum, &sum);
    carry += sum;
    if (b < NB) {
      if (rank == 0) offsets[b] = start;  // offsets[E]: the start of the dropped entries
#pragma unroll 8
      for (int w = 0; w < SORT_WARPS; ++w) counts[w * NB + b] += start + before;
    }
    __syncthreads();
  }
  for (int i0 = lo; i0 < hi; i0 += 32 * SORT_ROUNDS) {
    if (hi - lo > 32 * SORT_ROUNDS) read(i0);
#pragma unroll
    for (int r = 0; r < SORT_ROUNDS; ++r) {
      if (i0 + 32 * r >= hi) break;
      const int i = i0 + 32 * r + lane, e = buckets[r];
      const unsigned same = same_bucket(e, bits);
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
  if constexpr (CTAS > 1) cluster_sync();  // peers have read this CTA's counts
}

// ------------------------------------------------------- dispatch and combine
//
// All three walk the tokens, so that a token's own row moves once and its
// topk sorted rows once each; what bounds them is those bytes.  A thread takes
// a pack of a row at a time (16 bytes where bases and rows allow, else one
// element).  16384 tokens of 4096 bf16 and 4 choices: dispatch 100 us, combine
// 101 us (6.7 TB/s both, the rate of a plain copy).

template <class T, bool WIDE>
struct Pack {
  static constexpr int N = WIDE ? 16 / sizeof(T) : 1;
  T v[N];
  __device__ __forceinline__ static Pack load(const T* p) {
    Pack r;
    if constexpr (WIDE)
      *reinterpret_cast<uint4*>(r.v) = __ldcs(reinterpret_cast<const uint4*>(p));
    else
      r.v[0] = *p;
    return r;
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (WIDE)
      __stcs(reinterpret_cast<uint4*>(p), *reinterpret_cast<const uint4*>(v));
    else
      *p = v[0];
  }
};

constexpr int MOVE_THREADS = 256;
constexpr int COMBINE_THREADS = 128;
constexpr int GRAD_THREADS = 128;
constexpr int GRAD_ROWS = 2;  // its gradient: choices at a time

// Sorted row of a position, and whether the entry is kept; positions outside
// the sorted rows (not a result of the sort) are left alone.
struct Place {
  int64_t row;
  bool kept, valid;
};
__device__ __forceinline__ Place place(int p, int64_t rows) {
  Place r;
  r.kept = p >= 0;
  r.row = r.kept ? p : -1 - static_cast<int64_t>(p);
  r.valid = r.row < rows;
  return r;
}

// Grid: (tokens, parts of a row).
template <class T, bool WIDE>
__global__ void __launch_bounds__(MOVE_THREADS) dispatch_kernel(int topk, int64_t rows, int64_t H,
                                                                const T* __restrict__ X, int64_t ldx,
                                                                const int32_t* __restrict__ position,
                                                                T* __restrict__ Xs, int64_t ldxs) {
  using P = Pack<T, WIDE>;
  griddep_wait();
  griddep_launch_dependents();
  const int64_t t = blockIdx.x;
  const int32_t* pos = position + t * topk;
  const T* src = X + t * ldx;
  const int64_t step = static_cast<int64_t>(gridDim.y) * MOVE_THREADS * P::N;
  for (int64_t h = (static_cast<int64_t>(blockIdx.y) * MOVE_THREADS + threadIdx.x) * P::N; h < H; h += step) {
    const P x = P::load(src + h);
    for (int j = 0; j < topk; ++j) {
      const Place d = place(pos[j], rows);
      if (!d.valid) continue;
      P y = x;
      if (!d.kept)
#pragma unroll
        for (int i = 0; i < P::N; ++i) y.v[i] = from_f32<T>(0.0f);
      y.store(Xs + d.row * ldxs + h);
    }
  }
}

// ROWS choices at a time of PACKS packs.
template <class T, bool WIDE, int ROWS, int PACKS>
__global__ void __launch_bounds__(COMBINE_THREADS) combine_kernel(int topk, int64_t rows, int64_t H,
                                                               const T* __restrict__ Ys, int64_t ldys,
                                                               const int32_t* __restrict__ position,
                                                               const float* __restrict__ weight, T* __restrict__ Y,
                                                               int64_t ldy) {
  using P = Pack<T, WIDE>;
  griddep_wait();
  griddep_launch_dependents();
  const int64_t t = blockIdx.x;
  const int32_t* pos = position + t * topk;
  const float* wt = weight ? weight + t * topk : nullptr;
  constexpr int64_t STRIDE = static_cast<int64_t>(COMBINE_THREADS) * P::N;  // between a thread's packs
  const int64_t step = static_cast<int64_t>(gridDim.y) * STRIDE * PACKS;
  for (int64_t h = blockIdx.y * STRIDE * PACKS + static_cast<int64_t>(threadIdx.x) * P::N; h < H; h += step) {
    float acc[PACKS][P::N] = {};
    for (int j0 = 0; j0 < topk; j0 += ROWS) {
      // positions and weights first, so that the rows' loads follow each other
      int64_t row[ROWS];  // -1: none
      float w[ROWS];
#pragma unroll
      for (int j = 0; j < ROWS; ++j) {
        row[j] = j0 + j < topk ? pos[j0 + j] : -1;
        w[j] = j0 + j < topk && wt ? wt[j0 + j] : 1.0f;
      }
      P y[ROWS][PACKS];
#pragma unroll
      for (int j = 0; j < ROWS; ++j) {
        if (row[j] >= rows) row[j] = -1;
#pragma unroll
        for (int k = 0; k < PACKS; ++k)
          if (row[j] >= 0 && h + k * STRIDE < H) y[j][k] = P::load(Ys + row[j] * ldys + h + k * STRIDE);
      }
#pragma unroll
      for (int j = 0; j < ROWS; ++j)
#pragma unroll
        for (int k = 0; k < PACKS; ++k)
          if (row[j] >= 0)
#pragma unroll
            for (int i = 0; i < P::N; ++i) acc[k][i] = fmaf(w[j], to_f32(y[j][k].v[i]), acc[k][i]);
    }
#pragma unroll
    for (int k = 0; k < PACKS; ++k) {
      if (h + k * STRIDE >= H) break;
      P out;
#pragma unroll
      for (int i = 0; i < P::N; ++i) out.v[i] = from_f32<T>(acc[k][i]);
      out.store(Y + t * ldy + h + k * STRIDE);
    }
  }
}

// One block a token: dYs rows and (dweight) the dots, GRAD_ROWS choices at a
// time, the token's own row coming from the caches again after the first ones.
// Few choices and small blocks are what keeps the streams of reads and writes
// of an SM apart: at 8191 x 8 x 4096 bf16 2 choices and 128 threads take 185
// us, 4 and 256 221, 8 and 256 336, 1 and 128 232.  A thread's terms are added in the order of h, then the warp's lanes
// and the block's warps in a fixed order.
template <class T, bool WIDE>
__global__ void __launch_bounds__(GRAD_THREADS) combine_grad_kernel(int topk, int64_t rows, int64_t H,
                                                                    const T* __restrict__ dY, int64_t lddy,
                                                                    const T* __restrict__ Ys, int64_t ldys,
                                                                    const int32_t* __restrict__ position,
                                                                    const float* __restrict__ weight,
                                                                    T* __restrict__ dYs, int64_t lddys,
                                                                    float* __restrict__ dweight) {
  using P = Pack<T, WIDE>;
  __shared__ float part[GRAD_THREADS / 32][GRAD_ROWS];
  griddep_wait();
  griddep_launch_dependents();
  const int64_t t = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const T* g = dY + t * lddy;
  for (int j0 = 0; j0 < topk; j0 += GRAD_ROWS) {
    Place s[GRAD_ROWS];
    float w[GRAD_ROWS], dot[GRAD_ROWS] = {};
#pragma unroll
    for (int j = 0; j < GRAD_ROWS; ++j) {
      s[j] = Place{0, false, false};
      w[j] = 0.0f;
      if (j0 + j < topk) {
        s[j] = place(position[t * topk + j0 + j], rows);
        if (s[j].kept) w[j] = weight ? weight[t * topk + j0 + j] : 1.0f;
      }
    }
    for (int64_t h = static_cast<int64_t>(threadIdx.x) * P::N; h < H; h += GRAD_THREADS * P::N) {
      P y[GRAD_ROWS];
#pragma unroll
      for (int j = 0; j < GRAD_ROWS; ++j)
        if (dweight && s[j].kept && s[j].valid) y[j] = P::load(Ys + s[j].row * ldys + h);
      const P d = P::load(g + h);
#pragma unroll
      for (int j = 0; j < GRAD_ROWS; ++j) {
        if (!s[j].valid) continue;
        P o;
#pragma unroll
        for (int i = 0; i < P::N; ++i) {
          const float v = to_f32(d.v[i]);
          o.v[i] = from_f32<T>(s[j].kept ? w[j] * v : 0.0f);
          if (dweight && s[j].kept) dot[j] = fmaf(v, to_f32(y[j].v[i]), dot[j]);
        }
        o.store(dYs + s[j].row * lddys + h);
      }
    }
    if (!dweight) continue;
#pragma unroll
    for (int j = 0; j < GRAD_ROWS; ++j) {
#pragma unroll
      for (int k = 16; k > 0; k >>= 1) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], k);
      if (lane == 0) part[warp][j] = dot[j];
    }
    __syncthreads();
    if (threadIdx.x < GRAD_ROWS && j0 + static_cast<int>(threadIdx.x) < topk) {
      float sum = 0.0f;
#pragma unroll
      for (int k = 0; k < GRAD_THREADS / 32; ++k) sum += part[k][threadIdx.x];
      dweight[t * topk + j0 + threadIdx.x] = sum;
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------- host

constexpr int64_t MAX_ENTRIES = int64_t{1} << 30;

int check_route(tcg_dtype type, int64_t T, int topk, int64_t H) {
  if (type < TCG_F32 || type > TCG_BF16 || T < 0 || topk < 1 || H < 0) return TCG_ERR_INVALID;
  if (topk > 64 || T >= MAX_ENTRIES || T * topk >= MAX_ENTRIES || H >= MAX_ENTRIES) return TCG_ERR_UNSUPPORTED;
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

// Launch as a programmatic dependent of the stream's previous kernel (every
// kernel here waits with griddepcontrol.wait before it touches memory).
template <class... Params, class... Args>
int launch(void (*kernel)(Params...), dim3 grid, int threads, int smem, int cluster, cudaStream_t s, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  if (int rc = record_cuda(cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...))) return rc;
  set_launch_count(1);
  return TCG_OK;
}

// Both sort kernels' shared-memory attribute, once a device.
constexpr int sort_smem(int E) { return (SORT_WARPS + 1) * (E + 1) * 4; }
OncePerDevice<cudaError_t> g_sort;

cudaError_t sort_setup(int dev) {
  return g_sort(dev, [] {
    cudaError_t e =
        cudaFuncSetAttribute(sort_kernel<1>, cudaFuncAttributeMaxDynamicSharedMemorySize, sort_smem(MAX_EXPERTS));
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(sort_kernel<SORT_CTAS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               sort_smem(MAX_EXPERTS));
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(sort_kernel<SORT_CTAS>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    return e;
  });
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
  if (int rc = record_cuda(sort_setup(dev))) return rc;
  const int n = static_cast<int>(T * topk);
  if (n <= SORT_ONE)
    return launch(sort_kernel<1>, dim3(1), 32 * SORT_WARPS, sort_smem(E), 1, s, n, E, expert, offsets, position, source);
  return launch(sort_kernel<SORT_CTAS>, dim3(SORT_CTAS), 32 * SORT_WARPS, sort_smem(E), SORT_CTAS, s, n, E, expert,
                offsets, position, source);
}

// f(element type's value, whether rows move as 16-byte words)
template <class F>
int for_type(tcg_dtype type, bool wide, F&& f) {
  if (type == TCG_F32) return wide ? f(float{}, std::true_type{}) : f(float{}, std::false_type{});
  if (type == TCG_F16) return wide ? f(__half{}, std::true_type{}) : f(__half{}, std::false_type{});
  return wide ? f(__nv_bfloat16{}, std::true_type{}) : f(__nv_bfloat16{}, std::false_type{});
}

// Rows of H elements whose starts are all 16-byte aligned.
bool wide_rows(tcg_dtype type, int64_t H, const void* a, int64_t lda, const void* b, int64_t ldb) {
  const int per = type == TCG_F32 ? 4 : 8;
  return H % per == 0 && lda % per == 0 && ldb % per == 0 &&
         (reinterpret_cast<uintptr_t>(a) | reinterpret_cast<uintptr_t>(b)) % 16 == 0;
}

// Blocks a token's row is split into: one, unless there are so few tokens that
// SMs would idle.
unsigned row_parts(int64_t T, int64_t H, tcg_dtype type, bool wide, int threads, int dev) {
  const int64_t packs = wide ? H / (type == TCG_F32 ? 4 : 8) : H;
  const int64_t most = std::max<int64_t>(1, (packs + threads - 1) / threads);
  return static_cast<unsigned>(std::min<int64_t>(most, std::max<int64_t>(1, 4 * device_sms(dev) / T)));
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
  const bool wide = wide_rows(type, H, X, ldx, Xs, ldxs);
  const unsigned parts = row_parts(T, H, type, wide, MOVE_THREADS, dev);
  return for_type(type, wide, [&](auto z, auto w) {
    using E = decltype(z);
    return launch(dispatch_kernel<E, decltype(w)::value>, dim3(static_cast<unsigned>(T), parts), MOVE_THREADS, 0, 1, s,
                  topk, T * topk, H, static_cast<const E*>(X), ldx, position, static_cast<E*>(Xs), ldxs);
  });
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
  const bool wide = wide_rows(type, H, Ys, ldys, Y, ldy);
  const unsigned parts = row_parts(T, H, type, wide, COMBINE_THREADS, dev);
  return for_type(type, wide, [&](auto z, auto w) {
    using E = decltype(z);
    constexpr bool W = decltype(w)::value;
    // Few tokens want their rows' latencies side by side (64 tokens x 8 x 4096
    // bf16 2.2 us, 3.1 two by two).  With more, two choices keep the rows that
    // are read together few: 16384 x 4 101 us, 139 four by four, 169 eight;
    // 2432 x 8 32 us, 35 eight; 1216 x 8 19 either way.
    const auto kernel = topk > 4 && parts > 1 ? combine_kernel<E, W, 8, 1> : combine_kernel<E, W, 2, 2>;
    return launch(kernel, dim3(static_cast<unsigned>(T), parts), COMBINE_THREADS, 0, 1, s, topk, T * topk, H,
                  static_cast<const E*>(Ys), ldys, position, weight, static_cast<E*>(Y), ldy);
  });
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
  const bool wide = wide_rows(type, H, dY, lddy, dYs, lddys) && (!Ys || wide_rows(type, H, Ys, ldys, Ys, ldys));
  return for_type(type, wide, [&](auto z, auto w) {
    using E = decltype(z);
    return launch(combine_grad_kernel<E, decltype(w)::value>, dim3(static_cast<unsigned>(T)), GRAD_THREADS, 0, 1, s, topk,
                  T * topk, H, static_cast<const E*>(dY), lddy, static_cast<const E*>(Ys), ldys, position, weight,
                  static_cast<E*>(dYs), lddys, dweight);
  });
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
