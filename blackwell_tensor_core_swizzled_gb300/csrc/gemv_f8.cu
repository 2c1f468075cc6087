// Few rows of 8-bit codes against 8-bit matrices with a scale for each 128 x 128:
// what tcg_gemm_f8 and tcg_gemm_f8_grouped run where a matrix meets few rows.
//
//     D[r, n] = sum_b SA[b, r] SB[n / 128, b] sum_{k in block b} A[r, k] B[g][n, k]
//
// The matrices' bytes from HBM are the bound, so that reads have to be in flight
// without a pause.  A unit is 16 rows n of a matrix against up to 8 rows r, over the
// whole contraction (a group's further rows are units of their own, next to it: the
// matrix then comes from L2).  One warp brings the matrix in stages of 1 KB of each row
// (eight slabs of 16 rows by 128 bytes, one copy) into a ring, across units;
// another the codes and scales of the rows r.  Each of eight warps takes one slab,
// which is one block of the scales: four mma.m16n8k32 of the codes as they are, and
// one fp32 multiply-add of each sum by the two scales' product.  The
// warps' sums are added in shared memory, in order.  (tcgen05 wants tiles of 128
// rows n: too few of them for all SMs, and 500 cycles a block between its waits and
// commits where few columns take the pipe 50: 1 x 8192 x 8192 19 us there, 15 here;
// 1 x 4096 x 4096 11 and 7.)  1 x 8192 x 8192 runs at 4.5 TB/s, 5 us of its 15 being
// the start: launch, cold code, the first bytes; 1 x 16384 x 4096 16.3 us.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstring>

#include "common.h"
#include "once.h"
#include "ptx.cuh"
#include "ptx_moe.cuh"
#include "wait.cuh"

namespace tcg {

namespace {

constexpr int BLOCK = 128;
constexpr int WARPS = 8;  // that multiply; two more bring matrices, and rows with their scales
constexpr int THREADS = 32 * (WARPS + 2);
constexpr int CHUNK = BLOCK * WARPS;  // bytes of a row in a stage
constexpr int SLAB_BYTES = 16 * 128;
constexpr int TILE_BYTES = SLAB_BYTES * WARPS;
constexpr int MAX_STAGES = 4;  // (5 and 6 are 3 % slower)
constexpr int MAX_SMEM = 232448;
constexpr int COLUMNS = 8;  // rows r of a unit

struct Gemv8Params {
  CUtensorMap slab, edge;  // of B: [G][128-byte slabs][N][128], and [G][N][K] in single slabs for the last stage
  const int32_t* offsets;  // or null: one group of all R rows
  int G, R, N, K;
  int stages;
  const uint8_t* A;
  int64_t lda;
  const float* SA;
  int64_t ld_sa;
  const float* SB;
  int64_t sb_group, sb_row;
  void* D;
  int64_t ldd;
  int d_type;
  unsigned long long* err;
  uint64_t timeout_ns;
};

// Shared memory behind the ring of the matrix' stages: rows' codes and scales by
// stage, sums, groups.
struct Layout {
  static constexpr int X_ROW = CHUNK + 16;  // 16 bytes on: eight rows' words lie in different banks
  int x_stage, scales;  // bytes of a stage's rows, and where its scales begin in it
  int x, sums, seg, pre, bars, bytes;
  __host__ __device__ Layout(int R, int G, int stages) {
    const int columns = R < COLUMNS ? R : COLUMNS;
    scales = X_ROW * columns;
    x_stage = scales + 4 * WARPS * (COLUMNS + 2);  // [slab][rows' scales, the matrix' own, one unused]
    int at = stages * TILE_BYTES;
    auto take = [&](int n) {
      const int here = at;
      at += (n + 15) / 16 * 16;
      return here;
    };
    x = take(stages * x_stage);
    sums = take(WARPS * 8 * 17 * 4);
    seg = take(4 * (G + 1));
    pre = take(4 * (G + 1));
    bars = take(2 * MAX_STAGES * 8 + 16);
    bytes = at + 1024;  // the ring starts on a swizzle period
  }
};

template <bool WIDE>
__device__ __forceinline__ void mma_16832(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
  if constexpr (WIDE)
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.f32.e5m2.e5m2.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float ld_shared_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ float2 ld_shared_2f32(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr));
  return v;
}
__device__ __forceinline__ void workers_sync() { asm volatile("bar.sync 1, %0;" ::"n"(32 * WARPS) : "memory"); }
__device__ __forceinline__ bool workers_agree(bool ok) {
  uint32_t all;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\tbar.red.and.pred q, 1, %2, p;\n\tselp.b32 %0, 1, 0, q;\n\t}"
      : "=r"(all)
      : "r"(static_cast<uint32_t>(ok)), "n"(32 * WARPS)
      : "memory");
  return all != 0;
}

// One unit: rows r0 .. + columns of group g against rows n0 .. + 16 of its matrix.
struct Unit {
  int g, r0, columns, n0;
};

template <bool WIDE>
__global__ void __launch_bounds__(THREADS, 2) gemv_f8_kernel(const __grid_constant__ Gemv8Params p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (sbase - raw);
  const Layout at(p.R, p.G, p.stages);
  int* seg = reinterpret_cast<int*>(gbase + at.seg);
  int* pre = reinterpret_cast<int*>(gbase + at.pre);
  float* sums = reinterpret_cast<float*>(gbase + at.sums);
  const uint32_t bar0 = sbase + at.bars;
  auto full_bar = [&](uint32_t s) { return bar0 + 8u * s; };
  auto empty_bar = [&](uint32_t s) { return bar0 + 8u * (MAX_STAGES + s); };
  volatile uint32_t* abort_flag = reinterpret_cast<uint32_t*>(gbase + at.bars + 16 * MAX_STAGES);
  const WaitCtx wctx{p.timeout_ns, p.err, abort_flag};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t stages = static_cast<uint32_t>(p.stages);
  const int tiles = (p.N + 15) / 16;

  if (threadIdx.x == 0) {
    if (p.K >= 128) prefetch_tmap(&p.slab);
    if (p.K > 0) prefetch_tmap(&p.edge);
    for (uint32_t s = 0; s < stages; ++s) {
      mbar_init(full_bar(s), 1 + 32);  // the matrix' bytes, the lanes' copies of rows and scales
      mbar_init(empty_bar(s), WARPS);
    }
    *abort_flag = 0u;
    fence_mbarrier_init();
  }
  // a programmatic dependent of the previous kernel: no global access before
  griddep_wait();
  griddep_launch_dependents();
  // offsets, each clamped to [the previous one, R], and the units before each group
  if (warp == 0) {
    int run_max = 0, run_units = 0;
    for (int g0 = 0; g0 <= p.G; g0 += 32) {
      const int g = g0 + lane;
      int v = g > p.G ? 0 : p.offsets ? min(max(p.offsets[g], 0), p.R) : g ? p.R : 0;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, v, d);
        if (lane >= d) v = max(v, o);
      }
      v = max(v, run_max);
      int before = __shfl_up_sync(0xffffffffu, v, 1);
      if (lane == 0) before = run_max;
      int units = g >= 1 && g <= p.G ? (v - before + COLUMNS - 1) / COLUMNS * tiles : 0;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, units, d);
        if (lane >= d) units += o;
      }
      units += run_units;
      if (g <= p.G) {
        seg[g] = v;
        pre[g] = units;
      }
      run_max = __shfl_sync(0xffffffffu, v, 31);
      run_units = __shfl_sync(0xffffffffu, units, 31);
    }
  }
  __syncthreads();
  const int units = p.K > 0 ? pre[p.G] : 0;
  const int chunks = (p.K + CHUNK - 1) / CHUNK;
  auto decode = [&](int u) {
    int a = 0, b = p.G;  // pre[a] <= u < pre[b]
    while (b - a > 1) {
      const int mid = (a + b) >> 1;
      if (pre[mid] <= u)
        a = mid;
      else
        b = mid;
    }
    // the row blocks of a group sweep its matrix together
    const int rows = seg[a + 1] - seg[a], blocks = (rows + COLUMNS - 1) / COLUMNS, v = u - pre[a];
    const int block = v % blocks;
    return Unit{a, seg[a] + block * COLUMNS, min(COLUMNS, rows - block * COLUMNS), v / blocks * 16};
  };

  if (warp == WARPS) {
    // --------------------------------------------------- producer of matrices
    uint32_t s = 0, ph = 0, sent = 0;
    bool ok = true;
    for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
      const Unit t = decode(u);
      for (int c = 0; c < chunks; ++c) {
        if (!wait_inline(empty_bar(s), ph ^ 1u, wctx, SITE_PROD_EMPTY)) {
          ok = false;
          break;
        }
        if (lane == 0) {
          const uint32_t to = sbase + s * TILE_BYTES;
          if (p.K % 128 == 0 || c + 1 < chunks) {
            mbar_arrive_expect_tx(full_bar(s), TILE_BYTES);
            tma_load_4d(to, &p.slab, 0, t.n0, c * WARPS, t.g, full_bar(s));
          } else {
            const int n = min(WARPS, (p.K - c * CHUNK + 127) / 128);
            mbar_arrive_expect_tx(full_bar(s), static_cast<uint32_t>(SLAB_BYTES * n));
            for (int w = 0; w < n; ++w)
              tma_load3<1>(to + SLAB_BYTES * w, &p.edge, c * CHUNK + 128 * w, t.n0, t.g, full_bar(s));
          }
        }
        __syncwarp();
        ++sent;
        if (++s == stages) {
          s = 0;
          ph ^= 1u;
        }
      }
    }
    if (!ok && lane == 0) {
      // let the copies in flight land before the CTA can exit
      const uint32_t out = min(sent, stages);
      for (uint32_t j = sent - out; j < sent; ++j) {
        const uint64_t t0 = globaltimer();
        while (!mbar_try_wait(full_bar(j % stages), (j / stages) & 1u) && globaltimer() - t0 < 20000000ull) {
        }
      }
    }
    return;
  }
  if (warp == WARPS + 1) {
    // ----------------------------------------- producer of rows and of scales
    uint32_t s = 0, ph = 0;
    for (int u = blockIdx.x; u < units; u += gridDim.x) {
      const Unit t = decode(u);
      // the lanes share out the rows: 32, 16, 8 or 4 of a row, or all rows in turns
      const int shift = t.columns > 4 ? 2 : t.columns > 2 ? 3 : t.columns > 1 ? 4 : 5;
      const int per_turn = 32 >> shift, index = lane >> shift, piece = lane & ((1 << shift) - 1);
      const float* sb = p.SB + t.g * p.sb_group + (t.n0 / BLOCK) * p.sb_row;
      for (int c = 0; c < chunks; ++c) {
        if (!wait_inline(empty_bar(s), ph ^ 1u, wctx, SITE_PROD_EMPTY)) {
          asm volatile("cp.async.wait_all;" ::: "memory");
          return;
        }
        const uint32_t to = sbase + at.x + s * at.x_stage;
        for (int col = index; col < t.columns; col += per_turn) {
          const uint8_t* from = p.A + (t.r0 + col) * p.lda + c * CHUNK;
#pragma unroll 4
          for (int v = piece; v < CHUNK / 16; v += 1 << shift)
            copy_16(to + col * Layout::X_ROW + 16u * v, from + 16 * v, min(max(p.K - c * CHUNK - 16 * v, 0), 16));
        }
        for (int i = lane; i < WARPS * (t.columns + 1); i += 32) {
          const int slab = i & (WARPS - 1), col = i / WARPS, b = c * WARPS + slab;
          const bool exists = b * BLOCK < p.K;
          const float* from = col < t.columns ? p.SA + b * p.ld_sa + t.r0 + col : sb + b;
          copy_f32(to + at.scales + 4u * (slab * (COLUMNS + 2) + (col < t.columns ? col : COLUMNS)), from, exists);
        }
        copies_arrive(full_bar(s));
        if (++s == stages) {
          s = 0;
          ph ^= 1u;
        }
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    return;
  }

  // ----------------------------------------------------------------- workers
  const int g = lane >> 2, c4 = lane & 3;
  uint32_t s = 0, ph = 0;
  for (int u = blockIdx.x; u < units; u += gridDim.x) {
    const Unit t = decode(u);
    float acc[4] = {};
    bool ok = true;
    for (int c = 0; c < chunks; ++c) {
      ok = wait_inline(full_bar(s), ph, wctx, SITE_MMA_FULL);
      if (!ok) break;
      if (c * CHUNK + BLOCK * warp < p.K) {
        const uint32_t slab = sbase + s * TILE_BYTES + SLAB_BYTES * warp;
        const uint32_t x = sbase + at.x + s * at.x_stage + BLOCK * warp;
        const uint32_t sc = sbase + at.x + s * at.x_stage + at.scales + 4u * warp * (COLUMNS + 2);
        const float scale = ld_shared_f32(sc + 4u * COLUMNS);
        uint4 a[2][2];  // this lane's 16-byte chunks c4 and c4 + 4 of rows g and g + 8
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int r = 0; r < 2; ++r) a[h][r] = ld_shared_v4(slab + 128u * (g + 8 * r) + 16u * ((c4 + 4 * h) ^ g));
        float part[4] = {};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          // the same 16 k of row r = g (of rows that do not exist: anything)
          const uint4 b = ld_shared_v4(x + min(g, p.R - 1) * Layout::X_ROW + 16u * (c4 + 4 * h));
          mma_16832<WIDE>(part, a[h][0].x, a[h][1].x, a[h][0].y, a[h][1].y, b.x, b.y);
          mma_16832<WIDE>(part, a[h][0].z, a[h][1].z, a[h][0].w, a[h][1].w, b.z, b.w);
        }
        const float2 sa = ld_shared_2f32(sc + 8u * c4);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] = fmaf(part[i], (i & 1 ? sa.y : sa.x) * scale, acc[i]);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty_bar(s));
      if (++s == stages) {
        s = 0;
        ph ^= 1u;
      }
    }
    if (!workers_agree(ok)) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) sums[(warp * 8 + 2 * c4 + (i & 1)) * 17 + g + 8 * (i >> 1)] = acc[i];
    workers_sync();
    const int row = threadIdx.x & 15, col = threadIdx.x >> 4, n = t.n0 + row;
    if (col < t.columns && n < p.N) {
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) v += sums[(w * 8 + col) * 17 + row];
      const int64_t to = (t.r0 + col) * p.ldd + n;
      if (p.d_type == OUT_F32)
        static_cast<float*>(p.D)[to] = v;
      else if (p.d_type == OUT_BF16)
        static_cast<__nv_bfloat16*>(p.D)[to] = __float2bfloat16_rn(v);
      else
        static_cast<__half*>(p.D)[to] = __float2half_rn(v);
    }
    workers_sync();
  }
  // rows of no group (and all rows when K is 0): zero
  const int first = seg[0], end = p.K > 0 ? seg[p.G] : first;
  for (int r = blockIdx.x; r < p.R; r += gridDim.x) {
    if (r >= first && r < end) {
      r += (end - 1 - r) / gridDim.x * gridDim.x;  // the last row below `end` this block meets
      continue;
    }
    for (int n = threadIdx.x; n < p.N; n += 32 * WARPS) {
      const int64_t i = r * p.ldd + n;
      if (p.d_type == OUT_F32)
        static_cast<float*>(p.D)[i] = 0.0f;
      else
        static_cast<uint16_t*>(p.D)[i] = 0;
    }
  }
}

using Kernel = void (*)(const Gemv8Params);
OncePerDevice<cudaError_t> g_setup;

}  // namespace

int run_gemv_f8(tcg_input type, int64_t R, int64_t N, int64_t K, int G, const void* A, int64_t lda, const float* SA,
                int64_t ld_sa, const int32_t* offsets, const void* B, int64_t ldb, int64_t stride_b, const float* SB,
                int64_t ld_sb, int64_t stride_sb, void* D, tcg_dtype d_type, int64_t ldd, int dev, cudaStream_t s) {
  if (int rc = record_cuda(g_setup(dev, [] {
        const auto smem = [](Kernel k) { return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, MAX_SMEM); };
        const cudaError_t e = smem(gemv_f8_kernel<false>);
        return e == cudaSuccess ? smem(gemv_f8_kernel<true>) : e;
      })))
    return rc;
  Gemv8Params p;
  std::memset(&p, 0, sizeof p);
  if (K > 0) {
    if (K >= 128)
      if (int rc = make_slab_map(&p.slab, B, 128, N, K / 128, G, ldb, stride_b, 16, WARPS)) return rc;
    if (int rc = make_byte_map(&p.edge, B, K, N, G, ldb, stride_b, 128, 16)) return rc;
  }
  p.offsets = offsets;
  p.G = G;
  p.R = static_cast<int>(R);
  p.N = static_cast<int>(N);
  p.K = static_cast<int>(K);
  p.A = static_cast<const uint8_t*>(A);
  p.lda = lda;
  p.SA = SA;
  p.ld_sa = ld_sa;
  p.SB = SB;
  p.sb_group = stride_sb;
  p.sb_row = ld_sb;
  p.D = D;
  p.ldd = ldd;
  p.d_type = d_type;
  p.err = device_error_word(dev);
  p.timeout_ns = wait_timeout_ns();
  // two CTAs share an SM
  p.stages = MAX_STAGES;
  while (p.stages > 1 && Layout(p.R, G, p.stages).bytes > MAX_SMEM / 2 - 1024) --p.stages;
  const int64_t units = (R / COLUMNS + std::min<int64_t>(G, R)) * ((N + 15) / 16);
  if (units > INT32_MAX / 2) return TCG_ERR_UNSUPPORTED;
  const int64_t grid = std::max<int64_t>(1, std::min<int64_t>(units, 2 * device_sms(dev)));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
  cfg.blockDim = dim3(THREADS, 1, 1);
  cfg.dynamicSmemBytes = static_cast<size_t>(Layout(p.R, G, p.stages).bytes);
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (int rc = record_cuda(cudaLaunchKernelEx(&cfg, type == TCG_IN_E5M2 ? gemv_f8_kernel<true> : gemv_f8_kernel<false>, p))) return rc;
  set_launch_count(1);
  record_gemv_f8_plan(COLUMNS, p.stages, static_cast<int>(grid));
  return TCG_OK;
}

}  // namespace tcg
