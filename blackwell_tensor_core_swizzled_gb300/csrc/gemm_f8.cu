// Products of 8-bit floating point with an fp32 scale for each block of 128, on
// the tensor cores: dense, by group, and the matrices' gradient by group.  Entry
// points, host plan and kernel; the contract is in include/tcg.h.
//
// No MMA kind takes fp32 scales.  So the sum of a block of 128 k is one accumulator
// in tensor memory (four MMAs of 32 k), and the epilogue's warps add it, scaled, to
// sums in their registers while the MMAs fill the next accumulator: 128 x 256 sums
// of a CTA are 128 registers of 256 threads.  All of it in fp32: one rounding of the
// scales' product and one of each addition (BOTH: of each scaling too).
//
// One kernel in three forms.  P has the MMA's rows, 128 for each CTA, and Q its
// columns:
//
//             tile        P                     Q                     scales
//   ROWS      256 x 256   A, rows r             B or B[g], rows n     A's by row, B's square
//   COLUMNS   128 x 64    B or B[g], rows n     A, rows r             A's by row, B's square
//   BOTH      256 x 256   B, rows n             A, rows r             by row on either side
//   (weight)  256 x 256   A, columns k, MN      DY, columns n, MN     by column of either
//
// ROWS: a lane holds one row, so that one factor, the product of the two scales,
// serves all of its 128 columns.  (The first form, rows on the columns' side and a
// factor for each read from shared memory by every lane, took 851 us for
// 8192 x 8192 x 8192.)
// COLUMNS: few rows cost few columns, any multiple of 16; the result is stored
// transposed.  Where its tiles leave SMs idle, two or four CTAs share a tile's
// contraction and add their sums through the cluster's shared memory.
// BOTH: a multiply and a multiply-add of each element.  The contraction of the
// weight product is ragged: rows of the next group within the last block are
// overwritten with zeros in shared memory up to the next multiple of 32, and the
// MMAs beyond are not issued.
//
// What bounds them: a block of a pair's 256 x 256 takes the tensor pipe 512 cycles,
// its 32 KB for each SM about 500 of what L2 delivers, and the epilogue's multiply-adds
// 256 (BOTH: 512) beside as many of reads from tensor memory.  8192 x 8192 x 8192 takes
// 409 us in bursts, 2.69 PFLOP/s (345 if the multiply-adds are left out, so much is the
// operands' delivery); back to back for seconds the power limit holds the clock at 1.91
// GHz and it takes about 445.  The weight gradient of 4096 x 4096 over 8191 rows takes
// 184 us, 1.50 PFLOP/s (136 without the multiply-adds, 105 without the reads as well):
// scaling both ways, and 16 % for the last of 3.4 waves of tiles.  More warps for the
// epilogue (12, 16), an accumulator in two halves with barriers of their own (an MMA of
// 128 columns takes most of the time of 256: 565 us), reads of tensor memory a step
// ahead, or one warp's arrival for all made them slower; four staging tiles a warp
// instead of two, at one ring stage less, 331 -> 341 us where stores count most.
//
// One warp decodes the tile list and copies the blocks' scales ahead into a shared
// ring, one each brings P and Q, one issues the MMAs.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstring>
#include <type_traits>

#include "common.h"
#include "desc.cuh"
#include "gemm_kernel.cuh"
#include "ptx.cuh"
#include "ptx_moe.cuh"
#include "tmem_ldst.cuh"
#include "wait.cuh"

namespace tcg {

namespace {

constexpr int MAX_GROUPS = 1024;
constexpr int64_t MAX_EXTENT = int64_t{1} << 30;
constexpr int BLOCK = 128;  // k of a scale, and of a ring stage
constexpr int STAGING_BYTES = 2048;
constexpr int TILES = 4;   // decoded tiles ahead of the warps that work on them
constexpr int SLOTS = 8;   // blocks whose scales are in shared memory
constexpr int BAND = 8;    // column tiles that sweep a group's row tiles together

// What has a scale for each block: the columns (and 128 rows together), rows and
// columns, or the rows (and 128 columns together).
enum Scaling : int { COLUMNS = 0, BOTH = 1, ROWS = 2 };

struct F8Params {
  CUtensorMap tmap_p;    // [G or 1][rows][128-byte boxes]
  CUtensorMap tmap_q;    // Q in boxes of a full tile's rows (MN-major: 128 k)
  CUtensorMap tmap_q16;  // K-major Q in boxes of 16 rows, for partial tiles
  CUtensorMap tmap_d;    // output [G or 1][c][m] in boxes of 32 m and 32 rows (fp32: 16)
  int d_tma;
  const int32_t* offsets;  // or null: one group of all R
  int G, R;
  int weight;    // the contraction runs over the group's rows
  int p_mn, q_mn;
  int M;         // extent of m
  int C;         // weight: extent of c
  int K;         // contraction length unless weight
  int m_tiles;
  int split;     // COLUMNS: CTAs of a cluster that share a unit's contraction (1, 2 or 4)
  // scales of single rows or columns: [block][row], b * fine_b + row
  const float* fine;
  int64_t fine_b;
  // BOTH: P's, likewise; else one for 128: g * other_group + (row / 128) * other_row + b * other_b
  const float* other;
  int64_t other_group, other_row, other_b;
  uint64_t p_hi, q_hi;
  uint32_t p_kstep, q_kstep;  // 16-byte units per 32 of the contraction
  uint32_t idesc;             // without N
  void* D;
  int64_t ldd, stride_d;
  int d_type, d_size;
  unsigned long long* err;
  uint64_t timeout_ns;
};

// kind::f8f6f4 (E4M3 / E5M2), D fp32 in TMEM, A and B from shared descriptors.
template <int CG>
__device__ __forceinline__ void mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accum) {
  if constexpr (CG == 2)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accum)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accum)
        : "memory");
}

template <bool MORE, int N>
__device__ __forceinline__ void set_registers() {
  if constexpr (MORE)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
  else
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t pair(uint32_t lo, uint32_t hi) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "r"(lo), "r"(hi));
  return v;
}
__device__ __forceinline__ void unpair(uint64_t v, uint32_t& lo, uint32_t& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=r"(lo), "=r"(hi) : "l"(v));
}
// sum += {lo, hi} * f (* row), two fp32 operations an instruction.  Volatile, so
// that none moves before the wait for the tensor-memory read of lo and hi.
__device__ __forceinline__ void add_scaled(uint64_t& sum, uint32_t lo, uint32_t hi, uint64_t f) {
  asm volatile("{\n\t.reg .b64 v;\n\tmov.b64 v, {%1, %2};\n\tfma.rn.f32x2 %0, v, %3, %0;\n\t}"
               : "+l"(sum)
               : "r"(lo), "r"(hi), "l"(f));
}
__device__ __forceinline__ void add_scaled(uint64_t& sum, uint32_t lo, uint32_t hi, uint64_t f, uint64_t row) {
  asm volatile(
      "{\n\t.reg .b64 v;\n\tmov.b64 v, {%1, %2};\n\tmul.rn.f32x2 v, v, %3;\n\tfma.rn.f32x2 %0, v, %4, %0;\n\t}"
      : "+l"(sum)
      : "r"(lo), "r"(hi), "l"(f), "l"(row));
}

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ void st_cluster_2x64(uint32_t addr, uint64_t a, uint64_t b) {
  asm volatile("st.shared::cluster.v2.b64 [%0], {%1, %2};" ::"r"(addr), "l"(a), "l"(b) : "memory");
}
__device__ __forceinline__ void ld_shared_2x64(uint32_t addr, uint64_t& a, uint64_t& b) {
  asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(a), "=l"(b) : "r"(addr) : "memory");
}
__device__ __forceinline__ uint64_t ld_shared_b64(uint32_t addr) {
  uint64_t v;
  asm volatile("ld.shared.b64 %0, [%1];" : "=l"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint16_t ld_shared_u16(uint32_t addr) {
  uint16_t v;
  asm volatile("ld.shared.b16 %0, [%1];" : "=h"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float ld_shared_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
template <int CG, int BN, int STAGES, Scaling MODE>
struct F8Cfg {
  static constexpr int PARTS = 2;  // epilogue warps that share a lane quadrant's columns
  static constexpr int EPI_WARPS = 4 * PARTS;
  static constexpr int THREADS = 32 * (4 + EPI_WARPS);
  static constexpr int P_BYTES = 128 * 128;
  static constexpr int Q_ROWS = BN / CG;
  static constexpr int Q_BYTES = Q_ROWS * 128;
  static constexpr int STAGE_BYTES = P_BYTES + Q_BYTES;
  static constexpr int STAGING = 2;  // staging tiles for each epilogue warp
  // accumulators; of 64 columns four (256 rows over 64 groups of 4096 x 1024 56.5 us with two, 54.9
  // with four or eight)
  static constexpr int ACCS = 512 / BN < 4 ? 512 / BN : 4;
  static constexpr int EPI_OFF = STAGES * STAGE_BYTES;
  static constexpr int SC_OFF = EPI_OFF + EPI_WARPS * STAGING * STAGING_BYTES;
  // a block's scales: Q's of the columns, then P's of the rows or of all; ROWS: P's of
  // the rows, then Q's of 128 columns each
  static constexpr int SLOT_BYTES = 4 * (MODE == ROWS ? 128 + 4 : BN + (MODE == BOTH ? 128 : 4));
  // split contractions: fragments of two column parts and four lane quadrants
  static constexpr int RED_OFF = (SC_OFF + SLOTS * SLOT_BYTES + 127) / 128 * 128;
  static constexpr int BAR_OFF = RED_OFF + (MODE == COLUMNS ? EPI_WARPS * 4096 : 0);
  // full[S], empty[S], rag[S], peer[S], acc_full[A], acc_empty[A], drain, tile_full[T], tile_empty[T],
  // scale_full[L], scale_empty[L], reduced
  static constexpr int NUM_BARS = 4 * STAGES + 1 + 2 * ACCS + 2 * TILES + 2 * SLOTS + 1;
  static constexpr int TILE_OFF = (BAR_OFF + NUM_BARS * 8 + 8 + 15) / 16 * 16;  // tmem slot + abort flag before it
  static constexpr int SEG_OFF = TILE_OFF + TILES * 48;
  static constexpr int SMEM_BYTES = 1024 + SEG_OFF + 2 * (MAX_GROUPS + 1) * 4;
  static_assert(Q_BYTES % 1024 == 0, "swizzle period");
  static_assert(SMEM_BYTES <= 232448, "dynamic shared memory");
  static_assert(ACCS >= 2, "the next accumulator is filled meanwhile");
};

// One unit: a tile of one group.
struct alignas(16) FTile {
  int g;
  int lo;     // first row of the group
  int m0;     // first m of the tile (of the pair's tile)
  int c0;     // first column within the group (weight: within C)
  int ncols;  // columns of the tile that exist
  int mma_n;  // columns the MMA computes
  int nkb;    // blocks of the contraction (0: the tile is zero)
  int last;   // depth of the last block
  int rows;   // ROWS: rows of the group from m0 on
  int kb0;    // first block of this CTA
};
static_assert(sizeof(FTile) <= 48, "tile ring");

// A group's n ragged columns (ROWS: rows): tiles of `per` each, the last shorter.
template <int CG, int BN, Scaling MODE>
__device__ __forceinline__ void split_ragged(int n, bool whole, int& tiles, int& per) {
  if constexpr (MODE == ROWS) {
    per = 128 * CG;
  } else {
    const int t = (n + BN - 1) / BN;
    const int step = whole ? BN : 16 * CG;
    per = t ? ((n + t - 1) / t + step - 1) / step * step : step;
  }
  tiles = (n + per - 1) / per;
}

// seg[0..G]: clamped offsets; pre[0..G]: units of the groups before (unless weight).
template <int CG, int BN, Scaling MODE>
__device__ __forceinline__ FTile decode_unit(const F8Params& p, const int* seg, const int* pre, int u) {
  FTile t;
  int v, tiles, per, n;
  if (p.weight) {
    split_ragged<CG, BN, MODE>(p.C, true, tiles, per);
    const int per_group = tiles * p.m_tiles;
    t.g = u / per_group;
    v = u - t.g * per_group;
    n = p.C;
  } else {
    int a = 0, b = p.G;  // pre[a] <= u < pre[b]
    while (b - a > 1) {
      const int mid = (a + b) >> 1;
      if (pre[mid] <= u)
        a = mid;
      else
        b = mid;
    }
    t.g = a;
    v = u - pre[a];
    n = seg[a + 1] - seg[a];
    split_ragged<CG, BN, MODE>(n, p.q_mn, tiles, per);
  }
  t.lo = seg[t.g];
  const int depth = p.weight ? seg[t.g + 1] - t.lo : p.K;
  const int band = v / (BAND * p.m_tiles);
  const int first = band * BAND;
  const int width = min(tiles - first, BAND);
  v -= first * p.m_tiles;
  const int ragged = (first + v % width) * per;
  if constexpr (MODE == ROWS) {
    t.m0 = ragged;
    t.c0 = (v / width) * BN;
    t.rows = n - ragged;
    t.ncols = min(BN, p.M - t.c0);
  } else {
    t.m0 = (v / width) * (128 * CG);
    t.c0 = ragged;
    t.rows = 0;
    t.ncols = min(per, n - t.c0);
  }
  t.mma_n = p.weight || p.q_mn ? BN : (t.ncols + 16 * CG - 1) / (16 * CG) * (16 * CG);
  t.nkb = (depth + BLOCK - 1) / BLOCK;
  t.last = depth - BLOCK * (t.nkb - 1);
  t.kb0 = 0;
  if constexpr (MODE == COLUMNS) {
    const int per_cta = (t.nkb + p.split - 1) / p.split;
    t.kb0 = min(t.nkb, per_cta * static_cast<int>(cluster_ctarank()));
    t.nkb = min(per_cta, t.nkb - t.kb0);
  }
  return t;
}

template <int CG, int BN, int STAGES, Scaling MODE>
__global__ void __launch_bounds__(F8Cfg<CG, BN, STAGES, MODE>::THREADS, 1) f8_kernel(const __grid_constant__ F8Params p) {
  using C = F8Cfg<CG, BN, STAGES, MODE>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (sbase - raw);
  const uint32_t bar0 = sbase + C::BAR_OFF;
  auto full_bar = [&](uint32_t s) { return bar0 + 8u * s; };
  auto empty_bar = [&](uint32_t s) { return bar0 + 8u * (STAGES + s); };
  auto rag_bar = [&](uint32_t s) { return bar0 + 8u * (2 * STAGES + s); };
  auto peer_bar = [&](uint32_t s) { return bar0 + 8u * (3 * STAGES + s); };
  auto accf_bar = [&](uint32_t b) { return bar0 + 8u * (4 * STAGES + b); };
  auto acce_bar = [&](uint32_t b) { return bar0 + 8u * (4 * STAGES + C::ACCS + b); };
  const uint32_t drain_bar = bar0 + 8u * (4 * STAGES + 2 * C::ACCS);
  const uint32_t after = drain_bar + 8u;
  auto tile_full = [&](uint32_t i) { return after + 8u * i; };
  auto tile_empty = [&](uint32_t i) { return after + 8u * (TILES + i); };
  auto scf_bar = [&](uint32_t i) { return after + 8u * (2 * TILES + i); };
  auto sce_bar = [&](uint32_t i) { return after + 8u * (2 * TILES + SLOTS + i); };
  const uint32_t red_bar = after + 8u * (2 * TILES + 2 * SLOTS);
  auto slot_at = [&](uint32_t i) { return sbase + C::SC_OFF + i * C::SLOT_BYTES; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + C::BAR_OFF + 8 * C::NUM_BARS);
  volatile uint32_t* abort_flag = tmem_slot + 1;
  int* seg = reinterpret_cast<int*>(gbase + C::SEG_OFF);
  int* pre = seg + p.G + 1;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = (CG == 2) ? cluster_ctarank() : 0u;
  const int across = MODE == COLUMNS ? p.split : CG;  // CTAs of a cluster
  const int cluster_id = blockIdx.x / across;
  const int num_clusters = gridDim.x / across;
  const WaitCtx wctx{p.timeout_ns, p.err, abort_flag};

  // the maps exist unless the contraction is empty
  if (warp == 0 && lane == 0 && (p.weight ? p.R : p.K) > 0) {
    prefetch_tmap(&p.tmap_p);
    prefetch_tmap(&p.tmap_q);
    if (MODE == COLUMNS) prefetch_tmap(&p.tmap_q16);
  }
  if (threadIdx.x == 96) {
    for (uint32_t s = 0; s < STAGES; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
      mbar_init(rag_bar(s), 1);
      mbar_init(peer_bar(s), 1);
    }
    for (uint32_t b = 0; b < C::ACCS; ++b) {
      mbar_init(accf_bar(b), 1);
      mbar_init(acce_bar(b), C::EPI_WARPS * CG);
    }
    mbar_init(drain_bar, 1);
    mbar_init(red_bar, C::EPI_WARPS);
    for (uint32_t i = 0; i < TILES; ++i) {
      mbar_init(tile_full(i), 1);
      mbar_init(tile_empty(i), 3 + C::EPI_WARPS);
    }
    for (uint32_t i = 0; i < SLOTS; ++i) {
      mbar_init(scf_bar(i), 32);
      mbar_init(sce_bar(i), C::EPI_WARPS);
    }
    *abort_flag = 0u;
    fence_mbarrier_init();
  }
  // a programmatic dependent of the previous kernel: no global access before
  griddep_wait();
  if (warp == 2) {
    tmem_alloc<CG>(smem_u32(tmem_slot), 512);
    tmem_relinquish<CG>();
  }
  // offsets, each clamped to [the previous one, R], and the units before each group
  if (p.offsets) {
    for (int g = threadIdx.x; g <= p.G; g += C::THREADS) seg[g] = p.offsets[g];
  } else if (threadIdx.x < 2) {
    seg[threadIdx.x] = threadIdx.x ? p.R : 0;
  }
  __syncthreads();
  if (warp == 3) {
    int run_max = 0, run_units = 0;
    for (int g0 = 0; g0 <= p.G; g0 += 32) {
      const int g = g0 + lane;
      int v = g <= p.G ? min(max(seg[g], 0), p.R) : 0;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, v, d);
        if (lane >= d) v = max(v, o);
      }
      v = max(v, run_max);
      int before = __shfl_up_sync(0xffffffffu, v, 1);
      if (lane == 0) before = run_max;
      // units of group g - 1
      int tiles = 0, per, units = 0;
      if (g >= 1 && g <= p.G && !p.weight) {
        split_ragged<CG, BN, MODE>(v - before, p.q_mn, tiles, per);
        units = tiles * p.m_tiles;
      }
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
  tc_fence_before();
  __syncthreads();
  if (across > 1) cluster_sync();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  griddep_launch_dependents();
  int total_units;
  if (p.weight) {
    int tiles, per;
    split_ragged<CG, BN, MODE>(p.C, true, tiles, per);
    total_units = p.G * tiles * p.m_tiles;
  } else {
    total_units = p.K > 0 ? pre[p.G] : 0;
  }

  // The n-th tile of this CTA, decoded by warp 3.
  FTile* tiles = reinterpret_cast<FTile*>(gbase + C::TILE_OFF);
  auto fetch = [&](uint32_t n, FTile& t) {
    const uint32_t i = n % TILES;
    if (!wait_inline(tile_full(i), (n / TILES) & 1u, wctx, SITE_PROD_EMPTY)) return false;
    t = tiles[i];
    __syncwarp();
    if (lane == 0) mbar_arrive(tile_empty(i));
    return true;
  };

  // of the 384 x 168 registers at launch few for the four warps that feed, more for
  // those that hold sums
  if (warp < 4) {
    set_registers<false, 56>();
    if (warp == 3) {
      // ------------------------------------------- tile list and blocks' scales
      uint32_t n = 0, it = 0;
      auto publish = [&](int u, FTile& t) {
        t = decode_unit<CG, BN, MODE>(p, seg, pre, u);
        const uint32_t i = n % TILES;
        if (!wait_inline(tile_empty(i), ((n / TILES) & 1u) ^ 1u, wctx, SITE_PROD_EMPTY)) return false;
        if (lane == 0) {
          tiles[i] = t;
          mbar_arrive(tile_full(i));
        }
        __syncwarp();
        ++n;
        return true;
      };
      FTile t, next;
      bool ok = cluster_id >= total_units || publish(cluster_id, next);
      for (int u = cluster_id; u < total_units && ok; u += num_clusters) {
        t = next;
        // the tile after this one, ahead of this one's scales
        if (u + num_clusters < total_units && !publish(u + num_clusters, next)) break;
        const int b0 = p.weight ? t.lo / BLOCK + t.g : t.kb0;
        const int m0 = t.m0 + static_cast<int>(rank) * 128;
        // single scales of `n` columns or rows, and those of the other operand
        const int n = MODE == ROWS ? t.rows - static_cast<int>(rank) * 128 : t.ncols;
        const float* fine = p.fine + b0 * p.fine_b + (p.weight ? t.c0 : MODE == ROWS ? t.lo + m0 : t.lo + t.c0);
        const float* other = MODE == BOTH   ? p.other + b0 * p.other_b + m0
                             : MODE == ROWS ? p.other + t.g * p.other_group + (t.c0 / BLOCK + lane) * p.other_row
                                            : p.other + t.g * p.other_group + (m0 / BLOCK) * p.other_row + b0 * p.other_b;
        constexpr int FINE = MODE == ROWS ? 128 : BN;
        for (int kb = 0; kb < t.nkb; ++kb, ++it) {
          const uint32_t i = it % SLOTS;
          if (!wait_inline(sce_bar(i), ((it / SLOTS) & 1u) ^ 1u, wctx, SITE_PROD_EMPTY)) {
            ok = false;
            break;
          }
          const uint32_t at = slot_at(i) + 4u * lane;
#pragma unroll
          for (int k = 0; k < FINE / 32; ++k)
            if (lane + 32 * k < FINE) copy_f32(at + 128u * k, fine + lane + 32 * k, lane + 32 * k < n);
          if constexpr (MODE == BOTH) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              copy_f32(at + 4u * FINE + 128u * k, other + lane + 32 * k, m0 + lane + 32 * k < p.M);
          } else if (lane < (MODE == ROWS ? BN / BLOCK : 1)) {
            copy_f32(at + 4u * FINE, other, (MODE == ROWS ? t.c0 + BLOCK * lane : m0) < p.M);
          }
          copies_arrive(scf_bar(i));
          fine += p.fine_b;
          other += p.other_b;
        }
      }
      // none in flight when the CTA ends
      asm volatile("cp.async.wait_all;" ::: "memory");
    } else if (warp != 1) {
      // ---------------------------------------------- producers, of P and of Q
      const bool brings_p = warp == 0;
      uint32_t it = 0, s = 0, ph = 0, n = 0;
      bool ok = true;
      for (int u = cluster_id; u < total_units && ok; u += num_clusters) {
        FTile t;
        ok = fetch(n++, t);
        if (!ok) break;
        const int half = t.mma_n / CG;
        const int m0 = t.m0 + static_cast<int>(rank) * 128;
        const int c0 = t.c0 + static_cast<int>(rank) * half;
        // the group is in the rows of the one operand and the matrix of the other
        const int p_row = MODE == ROWS ? t.lo + m0 : m0, p_mat = MODE == ROWS || p.weight ? 0 : t.g;
        const int q_row = MODE == ROWS || p.weight ? c0 : t.lo + c0, q_mat = MODE == ROWS ? t.g : 0;
        const bool boxed = MODE == ROWS || p.weight || p.q_mn || half == C::Q_ROWS;  // Q in one box
        const uint32_t tx = C::P_BYTES + static_cast<uint32_t>(boxed ? C::Q_BYTES : half * 128);
        for (int kb = 0; kb < t.nkb; ++kb) {
          if (!wait_inline(empty_bar(s), ph ^ 1u, wctx, SITE_PROD_EMPTY)) {
            ok = false;
            break;
          }
          if (elect_one()) {
            const uint32_t sp = sbase + s * C::STAGE_BYTES;
            const uint32_t sq = sp + C::P_BYTES;
            const int k0 = BLOCK * (t.kb0 + kb);
            const uint32_t fb = (CG == 2) ? mapa_shared(full_bar(s), 0) : full_bar(s);
            if (p.weight && kb == t.nkb - 1 && (t.last & 31)) {
              // the warp that zeroes the rows past the group's end waits for
              // this CTA's bytes alone; full[s] just marks the stage
              const int r0 = t.lo + k0;
              if (brings_p) {
                if (rank == 0) mbar_arrive(full_bar(s));
                mbar_arrive_expect_tx(rag_bar(s), tx);
                tma_load3<1>(sp, &p.tmap_p, m0, r0, 0, rag_bar(s));
              } else {
                tma_load3<1>(sq, &p.tmap_q, c0, r0, 0, rag_bar(s));
              }
            } else if (brings_p) {
              if (rank == 0) mbar_arrive_expect_tx(full_bar(s), tx * CG);
              if (!p.p_mn)
                tma_load3<CG>(sp, &p.tmap_p, k0, p_row, p_mat, fb);
              else
                tma_load3<CG>(sp, &p.tmap_p, p_row, p.weight ? t.lo + k0 : k0, p_mat, fb);
            } else if (p.q_mn) {
              tma_load3<CG>(sq, &p.tmap_q, q_row, p.weight ? t.lo + k0 : k0, q_mat, fb);
            } else if (boxed) {
              tma_load3<CG>(sq, &p.tmap_q, k0, q_row, q_mat, fb);
            } else {
              for (int i = 0; i < half; i += 16) tma_load3<CG>(sq + 128 * i, &p.tmap_q16, k0, q_row + i, q_mat, fb);
            }
          }
          __syncwarp();
          ++it;
          if (++s == STAGES) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
      if (!ok && elect_one()) {
        // let the copies in flight land before the CTA can exit: full[s] counts
        // the leader's and (for a pair) the peer's; ragged stages are waited
        // for by time, as the peer's are
        const uint32_t n_out = it < static_cast<uint32_t>(STAGES) ? it : static_cast<uint32_t>(STAGES);
        if ((CG == 1 || rank == 0) && !p.weight && brings_p) {
          for (uint32_t j = it - n_out; j < it; ++j) {
            const uint64_t t0 = globaltimer();
            while (!mbar_try_wait(full_bar(j % STAGES), (j / STAGES) & 1u) && globaltimer() - t0 < 20000000ull) {
            }
          }
        } else {
          const uint64_t t0 = globaltimer();
          while (globaltimer() - t0 < 2000000ull) {
          }
        }
      }
      __syncwarp();
    } else {
      // --------------------------------- MMA issuer (leader), row zeroing (both)
      const uint64_t p_desc0 = sdesc(sbase, p.p_hi);
      const uint64_t q_desc0 = sdesc(sbase + C::P_BYTES, p.q_hi);
      uint32_t s = 0, ph = 0, n = 0, tcount = 0, rag_ph = 0;  // rag_ph: one parity bit per stage
      bool ok = true;
      for (int u = cluster_id; u < total_units && ok; u += num_clusters) {
        FTile t;
        ok = fetch(n++, t);
        if (!ok) break;
        const bool issue = CG == 1 || rank == 0;
        const uint32_t idesc = p.idesc | (static_cast<uint32_t>(t.mma_n >> 3) << 17);
        for (int kb = 0; kb < t.nkb; ++kb) {
          const bool last = kb == t.nkb - 1;
          const bool ragged = p.weight && last && (t.last & 31);
          const uint32_t b = tcount % C::ACCS;
          if (issue && !wait_inline(acce_bar(b), ((tcount / C::ACCS) & 1u) ^ 1u, wctx, SITE_MMA_ACC_EMPTY)) {
            ok = false;
            break;
          }
          ++tcount;
          const uint32_t d_tmem = tmem_base + b * BN;
          if (issue && !wait_inline(full_bar(s), ph, wctx, SITE_MMA_FULL)) {
            ok = false;
            break;
          }
          if (ragged) {
            const uint32_t par = (rag_ph >> s) & 1u;
            rag_ph ^= 1u << s;
            if (!wait_inline(rag_bar(s), par, wctx, SITE_MMA_FULL)) {
              ok = false;
              break;
            }
            // rows [last, next multiple of 32) of P and Q; a row's 128 bytes are
            // the same under the swizzle
            const uint32_t sp = sbase + s * C::STAGE_BYTES;
            const int rows = 32 - (t.last & 31);
            for (int i = lane; i < 2 * rows * 8; i += 32) {
              const int ch = i / (rows * 8), rr = i - ch * rows * 8;
              st_shared_v4((ch ? sp + C::P_BYTES : sp) + 128u * (t.last + (rr >> 3)) + 16u * (rr & 7), 0u, 0u, 0u, 0u);
            }
            fence_proxy_async_shared();
            __syncwarp();
            if constexpr (CG == 2) {
              if (rank != 0) {
                if (lane == 0) mbar_arrive_cluster(mapa_shared(peer_bar(s), 0));
              } else if (!wait_inline(peer_bar(s), par, wctx, SITE_MMA_FULL) || !mbar_try_wait_cluster(peer_bar(s), par)) {
                ok = false;
                break;
              }
            }
          }
          if (issue) {
            tc_fence_after();
            if (elect_one()) {
              const uint64_t st = (s * static_cast<uint32_t>(C::STAGE_BYTES)) >> 4;
              const int steps = p.weight && last ? (t.last + 31) >> 5 : 4;
#pragma unroll
              for (int j = 0; j < 4; ++j)
                if (j < steps)
                  mma_f8<CG>(d_tmem, p_desc0 + st + j * p.p_kstep, q_desc0 + st + j * p.q_kstep, idesc, j ? 1u : 0u);
              tc_commit<CG>(empty_bar(s));
              tc_commit<CG>(accf_bar(b));
            }
            __syncwarp();
          }
          if (++s == STAGES) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
      if (!ok && (CG == 1 || rank == 0) && elect_one()) {
        tc_commit<CG>(drain_bar);
        const uint64_t t0 = globaltimer();
        while (!mbar_try_wait(drain_bar, 0) && globaltimer() - t0 < 20000000ull) {
        }
      }
      __syncwarp();
    }
  } else {
    // ------------------------------------------------------------ epilogue
    set_registers<true, 224>();
    const int q = warp & 3;            // TMEM lane quadrant
    const int part = (warp - 4) >> 2;  // 32-column chunks part, part + PARTS, ...
    constexpr int ACROSS = 32 * C::PARTS;  // a warp's chunks of 32 columns lie so far apart
    constexpr int MINE = (BN + ACROSS - 1) / ACROSS;
    uint32_t tcount = 0, n = 0, stores = 0;
    const uint32_t buf0 = sbase + C::EPI_OFF + static_cast<uint32_t>((warp - 4) * C::STAGING * STAGING_BYTES);
    // the staging tile to fill next: its last store has read it
    auto staging = [&] {
      if (stores >= C::STAGING) {
        if (lane == 0) bulk_wait_group_read<C::STAGING - 1>();
        __syncwarp();
      }
      return buf0 + stores % C::STAGING * STAGING_BYTES;
    };
    auto send = [&](uint32_t buf, int m0, int c, int g) {
      fence_proxy_async_shared();
      __syncwarp();
      if (lane == 0) {
        tma_store_3d(&p.tmap_d, buf, m0, c, g);
        bulk_commit_group();
      }
      ++stores;
    };
    const uint32_t lanes = tmem_base + (static_cast<uint32_t>(32 * q) << 16);
    for (int u = cluster_id; u < total_units; u += num_clusters) {
      FTile t;
      if (!fetch(n++, t)) break;
      if constexpr (MODE == ROWS) {
        constexpr int COLS = BN / C::PARTS, CHUNKS = COLS / 32, STEP = 2;
        const int c_warp = COLS * part;  // this warp's columns of the tile
        const int mine = (t.ncols - c_warp + 31) / 32;
        uint64_t sum[CHUNKS][16];  // pairs of columns
#pragma unroll
        for (int i = 0; i < CHUNKS; ++i)
#pragma unroll
          for (int k = 0; k < 16; ++k) sum[i][k] = 0ull;
        bool done = true;
        for (int kb = 0; kb < t.nkb; ++kb, ++tcount) {
          const uint32_t b = tcount % C::ACCS, slot = tcount % SLOTS;
          done = wait_inline(scf_bar(slot), (tcount / SLOTS) & 1u, wctx, SITE_EPI_ACC_FULL);
          if (!done) break;
          const uint32_t at = slot_at(slot);
          const float f = ld_shared_f32(at + 4u * (32 * q + lane)) * ld_shared_f32(at + 4u * (128 + c_warp / BLOCK));
          const uint64_t ff = pair(__float_as_uint(f), __float_as_uint(f));
          done = wait_inline(accf_bar(b), (tcount / C::ACCS) & 1u, wctx, SITE_EPI_ACC_FULL);
          if (!done) break;
          tc_fence_after();
#pragma unroll
          for (int i = 0; i < CHUNKS; i += STEP) {
            if (i >= mine) break;
            uint32_t r[STEP][32];
#pragma unroll
            for (int j = 0; j < STEP; ++j) tmem_ld_32x32b_x32(lanes + b * BN + c_warp + 32 * (i + j), r[j]);
            tc_wait_ld();
#pragma unroll
            for (int j = 0; j < STEP; ++j)
#pragma unroll
              for (int k = 0; k < 16; ++k) add_scaled(sum[i + j][k], r[j][2 * k], r[j][2 * k + 1], ff);
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(sce_bar(slot));
            if constexpr (CG == 2)
              mbar_arrive_relaxed(mapa_shared(acce_bar(b), 0));  // no memory to order, only TMEM reads
            else
              mbar_arrive(acce_bar(b));
          }
        }
        if (!done) break;
        const int m_warp = static_cast<int>(rank) * 128 + 32 * q;  // the warp's first row in the tile
        const int rows = min(32, t.rows - m_warp);
        const int row0 = t.lo + t.m0 + m_warp;
        if (rows <= 0) continue;
        if (p.d_tma && p.d_type != OUT_F32) {
          // What most calls take, apart from the rest: instructions that are fetched once a
          // tile have to be few and in a row (12289 rows, 64 groups, 4096 x 2048, f16, MN-major:
          // 189 us in one loop with the other paths, 163 so).
          const auto store = [&](auto bf) {
#pragma unroll
            for (int i = 0; i < CHUNKS; ++i) {
              if (i >= mine) break;
              const int n0 = t.c0 + c_warp + 32 * i;
              const uint32_t buf = staging();
#pragma unroll
              for (uint32_t j = 0; j < 4; ++j) {
                uint32_t w[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  uint32_t lo, hi;
                  unpair(sum[i][4 * j + k], lo, hi);
                  w[k] = decltype(bf)::value ? pack_bf16(lo, hi) : pack_f16(lo, hi);
                }
                st_shared_v4(buf + 64u * lane + 16u * (j ^ ((static_cast<uint32_t>(lane) >> 1) & 3u)), w[0], w[1], w[2],
                             w[3]);
              }
              if (rows == 32) {  // columns clip at the map's end, a group's rows do not
                send(buf, n0, row0, 0);
                continue;
              }
              __syncwarp();
              const int word = lane & 3;
#pragma unroll
              for (int k = 0; k < 32; k += 8) {
                const int r = k + (lane >> 2);
                const uint4 v = ld_shared_v4(buf + 64u * r + 16u * (word ^ ((r >> 1) & 3)));
                if (r < rows && n0 + 8 * word < p.M)
                  *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.D) + (row0 + r) * p.ldd + n0 + 8 * word) = v;
              }
              __syncwarp();
            }
          };
          if (p.d_type == OUT_BF16)
            store(std::true_type{});
          else
            store(std::false_type{});
          continue;
        }
#pragma unroll
        for (int i = 0; i < CHUNKS; ++i) {
          if (i >= mine) break;
          const int n0 = t.c0 + c_warp + 32 * i;
          const bool boxed = p.d_tma && rows == 32;
          uint8_t* dst = static_cast<uint8_t*>(p.D) + (static_cast<int64_t>(row0) * p.ldd + n0 + lane) * p.d_size;
          if (p.d_type == OUT_F32) {
            // two staging tiles of 16 rows
            if (lane == 0) bulk_wait_group_read<0>();
            __syncwarp();
            const uint32_t row = static_cast<uint32_t>(lane) & 15u;
            const uint32_t to = buf0 + STAGING_BYTES * (static_cast<uint32_t>(lane) >> 4) + 128u * row;
#pragma unroll
            for (uint32_t j = 0; j < 8; ++j) {
              uint32_t w[4];
              unpair(sum[i][2 * j], w[0], w[1]);
              unpair(sum[i][2 * j + 1], w[2], w[3]);
              st_shared_v4(to + 16u * (j ^ (row & 7u)), w[0], w[1], w[2], w[3]);
            }
            if (boxed) {
              send(buf0, n0, row0, 0);
              send(buf0 + STAGING_BYTES, n0, row0 + 16, 0);
              continue;
            }
            __syncwarp();
            if (p.d_tma) {
              const int word = lane & 7;
              for (int k = 0; k < rows; k += 4) {
                const int r = k + (lane >> 3);
                const uint4 v = ld_shared_v4(buf0 + 128u * r + 16u * (word ^ (r & 7)));
                if (r < rows && n0 + 4 * word < p.M)
                  *reinterpret_cast<uint4*>(static_cast<float*>(p.D) + (row0 + r) * p.ldd + n0 + 4 * word) = v;
              }
              __syncwarp();
              continue;
            }
            for (int k = 0; k < rows; ++k) {
              const uint32_t from = buf0 + 128u * k + 16u * ((static_cast<uint32_t>(lane) >> 2) ^ (k & 7u)) + 4u * (lane & 3u);
              if (n0 + lane < p.M) *reinterpret_cast<float*>(dst + k * p.ldd * 4) = ld_shared_f32(from);
            }
            __syncwarp();
            continue;
          }
          const uint32_t buf = staging();
          const bool bf = p.d_type == OUT_BF16;
#pragma unroll
          for (uint32_t j = 0; j < 4; ++j) {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t lo, hi;
              unpair(sum[i][4 * j + k], lo, hi);
              w[k] = bf ? pack_bf16(lo, hi) : pack_f16(lo, hi);
            }
            st_shared_v4(buf + 64u * lane + 16u * (j ^ ((static_cast<uint32_t>(lane) >> 1) & 3u)), w[0], w[1], w[2], w[3]);
          }
          __syncwarp();
          for (int k = 0; k < rows; ++k) {
            const uint32_t from = buf + 64u * k + 16u * ((static_cast<uint32_t>(lane) >> 3) ^ ((k >> 1) & 3u)) + 2u * (lane & 7u);
            if (n0 + lane < p.M) *reinterpret_cast<uint16_t*>(dst + k * p.ldd * 2) = ld_shared_u16(from);
          }
          __syncwarp();
        }
      } else {
        uint64_t sum[MINE][2][8];  // chunk, 16 rows, pairs of columns as in the fragment
#pragma unroll
        for (int i = 0; i < MINE; ++i)
#pragma unroll
          for (int k = 0; k < 16; ++k) sum[i][k >> 3][k & 7] = 0ull;
        const int mine = (t.ncols - 32 * part + ACROSS - 1) / ACROSS;  // this warp's chunks of 32 columns that exist
        bool done = true;
        for (int kb = 0; kb < t.nkb; ++kb, ++tcount) {
          const uint32_t b = tcount % C::ACCS, slot = tcount % SLOTS;
          done = wait_inline(scf_bar(slot), (tcount / SLOTS) & 1u, wctx, SITE_EPI_ACC_FULL) &&
                 wait_inline(accf_bar(b), (tcount / C::ACCS) & 1u, wctx, SITE_EPI_ACC_FULL);
          if (!done) break;
          tc_fence_after();
          const uint32_t at = slot_at(slot);
          uint64_t row[MODE == BOTH ? 4 : 1];  // P's factors of this lane's rows lane / 4 + 8 h (or of all), twice
#pragma unroll
          for (int h = 0; h < (MODE == BOTH ? 4 : 1); ++h) {
            const uint32_t r = __float_as_uint(ld_shared_f32(at + 4u * (MODE == BOTH ? BN + 32 * q + 8 * h + (lane >> 2) : BN)));
            row[h] = pair(r, r);
          }
          // chunks' fragments of 16 rows by 32 columns, STEP chunks (or the one) at a time
          const uint32_t from = lanes + b * BN + 32 * part;
          constexpr int STEP = MINE < 2 ? MINE : 2;
#pragma unroll
          for (int i0 = 0; i0 < MINE; i0 += STEP) {
            if (i0 >= mine) break;
            uint32_t r[STEP][2][16];
#pragma unroll
            for (int i = 0; i < STEP; ++i)
#pragma unroll
              for (int h = 0; h < 2; ++h)
                tmem_ld_16x256b_x4(from + ACROSS * (i0 + i) + (static_cast<uint32_t>(h) << 20), r[i][h]);
#pragma unroll
            for (int i = 0; i < STEP; ++i) {
              uint64_t f[4];  // factors of this lane's columns 8 j + 2 (lane % 4), + 1
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                f[j] = ld_shared_b64(at + 4u * (32 * part + ACROSS * (i0 + i) + 8 * j + 2 * (lane & 3)));
                if constexpr (MODE != BOTH) f[j] = mul2(f[j], row[0]);
              }
              if (i == 0) tc_wait_ld();
#pragma unroll
              for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                  if constexpr (MODE == BOTH)
                    add_scaled(sum[i0 + i][h][k], r[i][h][2 * k], r[i][h][2 * k + 1], f[k / 2], row[2 * h + (k & 1)]);
                  else
                    add_scaled(sum[i0 + i][h][k], r[i][h][2 * k], r[i][h][2 * k + 1], f[k / 2]);
                }
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(sce_bar(slot));
            if constexpr (CG == 2)
              mbar_arrive_relaxed(mapa_shared(acce_bar(b), 0));  // no memory to order, only TMEM reads
            else
              mbar_arrive(acce_bar(b));
          }
        }
        if (!done) break;
        if constexpr (MODE == COLUMNS) {
          if (p.split > 1) {
            // Every CTA of the cluster sends a lane quadrant's sums to the one CTA that
            // adds them, in the order of the blocks, and stores them.  A cluster has
            // one unit at most, so the buffer is written once.
            const int quads = 4 / p.split, owner = q / quads, from = static_cast<int>(cluster_ctarank());
            const uint32_t mine_at = sbase + C::RED_OFF + 4096u * ((q % quads * p.split + from) * 2 + part) + 16u * lane;
            if (mine > 0) {
              const uint32_t to = mapa_shared(mine_at, static_cast<uint32_t>(owner));
#pragma unroll
              for (int v = 0; v < 8; ++v) st_cluster_2x64(to + 512u * v, sum[0][v >> 2][2 * (v & 3)], sum[0][v >> 2][2 * (v & 3) + 1]);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(mapa_shared(red_bar, static_cast<uint32_t>(owner)));
            if (from != owner) continue;
            if (!wait_inline(red_bar, 0u, wctx, SITE_EPI_ACC_FULL) || !mbar_try_wait_cluster(red_bar, 0u)) break;
            if (mine <= 0) continue;
            for (int r = 0; r < p.split; ++r) {
              const uint32_t at = mine_at + 4096u * 2 * (r - from);
#pragma unroll
              for (int v = 0; v < 8; ++v) {
                uint64_t a, b;
                ld_shared_2x64(at + 512u * v, a, b);
                uint64_t &x = sum[0][v >> 2][2 * (v & 3)], &y = sum[0][v >> 2][2 * (v & 3) + 1];
                x = r ? add2(x, a) : a;
                y = r ? add2(y, b) : b;
              }
            }
          }
        }
        const int m_warp = t.m0 + static_cast<int>(rank) * 128 + 32 * q;
        const int row0 = p.weight ? t.c0 : t.lo + t.c0, outer = p.weight ? t.g : 0;
        const int64_t pitch = p.ldd * p.d_size;
        const bool m_ok = m_warp + lane < p.M;
        uint8_t* dst = static_cast<uint8_t*>(p.D) + static_cast<int64_t>(row0) * pitch +
                       (p.weight ? t.g * p.stride_d * p.d_size : 0) + static_cast<int64_t>(m_warp + lane) * p.d_size;
        if (mine <= 0 || m_warp >= p.M) continue;
        // half a chunk, 16 rows of 32 m
        const auto fill_f32 = [&](uint32_t buf, int i, int g) {
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            const uint32_t m = 8u * h + (static_cast<uint32_t>(lane) >> 2);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              uint32_t lo, hi;
              unpair(sum[i][h >> 1][2 * (2 * g + j) + (h & 1)], lo, hi);
              const uint32_t at = 8u * j + 2u * (lane & 3);
              st_shared_u32(buf + 128u * at + 16u * ((m >> 2) ^ (at & 7u)) + 4u * (m & 3u), lo);
              st_shared_u32(buf + 128u * (at + 1) + 16u * ((m >> 2) ^ ((at + 1) & 7u)) + 4u * (m & 3u), hi);
            }
          }
        };
        // stmatrix turns 8 m of 8 columns into 8 rows of 16 bytes: lane 8k + n
        // addresses row 8j + n, m 8k..8k+7; a row's four 16-byte words are swizzled
        const uint32_t k8 = static_cast<uint32_t>(lane) >> 3, n8 = static_cast<uint32_t>(lane) & 7u;
        const auto fill_16 = [&](uint32_t buf, int i, bool bf) {
#pragma unroll
          for (uint32_t j = 0; j < 4; ++j) {
            const uint32_t to = 8u * j + n8;
            uint32_t w[4];
#pragma unroll
            for (int h = 0; h < 4; ++h) {
              uint32_t lo, hi;
              unpair(sum[i][h >> 1][2 * j + (h & 1)], lo, hi);
              w[h] = bf ? pack_bf16(lo, hi) : pack_f16(lo, hi);
            }
            stmatrix_x4_trans(buf + 64u * to + 16u * (k8 ^ ((to >> 1) & 3u)), w[0], w[1], w[2], w[3]);
          }
        };
        // rows of a matrix clip at the map's end, rows of a group do not
        if (p.d_tma && (p.weight || 32 * part + ACROSS * (mine - 1) + 32 <= t.ncols)) {
          // whole boxes, apart from the rest as above (the matrices' gradient of 32 experts of
          // 2048 x 4096 354 us in one loop with the other paths, 331 so)
          const int row = row0 + 32 * part;
          const auto store = [&](auto type) {
            constexpr int TYPE = decltype(type)::value;
#pragma unroll
            for (int i = 0; i < MINE; ++i) {
              if (i >= mine) break;
#pragma unroll
              for (int g = 0; g < (TYPE == OUT_F32 ? 2 : 1); ++g) {
                const uint32_t buf = staging();
                if constexpr (TYPE == OUT_F32)
                  fill_f32(buf, i, g);
                else
                  fill_16(buf, i, TYPE == OUT_BF16);
                send(buf, m_warp, row + ACROSS * i + 16 * g, outer);
              }
            }
          };
          if (p.d_type == OUT_F32)
            store(std::integral_constant<int, OUT_F32>{});
          else if (p.d_type == OUT_BF16)
            store(std::integral_constant<int, OUT_BF16>{});
          else
            store(std::integral_constant<int, OUT_F16>{});
          continue;
        }
#pragma unroll
        for (int i = 0; i < MINE; ++i) {
          const int c = 32 * part + ACROSS * i;
          if (i >= mine) break;
          if (p.d_type == OUT_F32) {
#pragma unroll
            for (int g = 0; g < 2; ++g) {
              const uint32_t buf = staging();
              fill_f32(buf, i, g);
              __syncwarp();
              for (int k = 0; k < 16; ++k) {
                const uint32_t m = static_cast<uint32_t>(lane);
                if (m_ok && c + 16 * g + k < t.ncols)
                  *reinterpret_cast<float*>(dst + (c + 16 * g + k) * pitch) =
                      ld_shared_f32(buf + 128u * k + 16u * ((m >> 2) ^ (k & 7u)) + 4u * (m & 3u));
              }
              __syncwarp();
            }
            continue;
          }
          const uint32_t buf = staging();
          fill_16(buf, i, p.d_type == OUT_BF16);
          __syncwarp();
          for (int n = 0; n < 32; ++n)
            if (m_ok && c + n < t.ncols)
              *reinterpret_cast<uint16_t*>(dst + (c + n) * pitch) =
                  ld_shared_u16(buf + 64u * n + 16u * (k8 ^ ((static_cast<uint32_t>(n) >> 1) & 3u)) + 2u * n8);
          __syncwarp();
        }
      }
    }
    if (lane == 0) bulk_wait_group_all();
    __syncwarp();
    if (!p.weight) {
      // rows of no group (and all rows when K is 0): zero
      const int t = threadIdx.x - 128;
      const int first = seg[0], end = p.K > 0 ? seg[p.G] : first;
      for (int r = blockIdx.x; r < p.R; r += gridDim.x) {
        if (r >= first && r < end) {
          r += (end - 1 - r) / gridDim.x * gridDim.x;  // the last row below `end` this block meets
          continue;
        }
        for (int m = t; m < p.M; m += 32 * C::EPI_WARPS) {
          const int64_t i = r * p.ldd + m;
          if (p.d_type == OUT_F32)
            static_cast<float*>(p.D)[i] = 0.0f;
          else
            static_cast<uint16_t*>(p.D)[i] = 0;
        }
      }
    }
  }

  // ------------------------------------------------------------ teardown
  tc_fence_before();
  cta_barrier_unaligned();
  __syncwarp();
  if (across > 1) cluster_sync();
  tc_fence_after();
  if (warp == 2) tmem_dealloc<CG>(tmem_base, 512);
}

// ---------------------------------------------------------------------- host

template <int CG, int BN, int STAGES, Scaling MODE>
KernelInfo variant() {
  using C = F8Cfg<CG, BN, STAGES, MODE>;
  return {reinterpret_cast<const void*>(&f8_kernel<CG, BN, STAGES, MODE>), C::SMEM_BYTES, CG, BN, KIND_F16, C::THREADS};
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
bool misaligned(const void* p, unsigned n) { return reinterpret_cast<uintptr_t>(p) % n != 0; }

int check_problem(tcg_input in_type, int64_t R, int64_t N, int64_t K, int G, tcg_dtype d_type) {
  if (in_type != TCG_IN_E4M3 && in_type != TCG_IN_E5M2) return TCG_ERR_INVALID;
  if (R < 0 || N < 0 || K < 0 || G < 1 || d_type < TCG_F32 || d_type > TCG_BF16) return TCG_ERR_INVALID;
  if (R >= MAX_EXTENT || N >= MAX_EXTENT || K >= MAX_EXTENT || G > MAX_GROUPS) return TCG_ERR_UNSUPPORTED;
  return TCG_OK;
}

// A matrix of codes: rows of `inner`, 16-byte aligned
int check_codes(const void* p, int64_t inner, int64_t* ld) {
  if (*ld == 0) *ld = inner;
  if (!p || *ld < inner || *ld < 1) return TCG_ERR_INVALID;
  return misaligned(p, 16) || *ld % 16 ? TCG_ERR_ALIGNMENT : TCG_OK;
}

int check_scales(const float* p, int64_t inner, int64_t* ld) {
  if (*ld == 0) *ld = inner;
  if (!p || *ld < inner) return TCG_ERR_INVALID;
  return misaligned(p, 4) ? TCG_ERR_ALIGNMENT : TCG_OK;
}

int check_output(const void* p, int64_t inner, int64_t* ld, tcg_dtype type) {
  if (*ld == 0) *ld = inner;
  if (!p || *ld < inner) return TCG_ERR_INVALID;
  return misaligned(p, type == TCG_F32 ? 4 : 2) ? TCG_ERR_ALIGNMENT : TCG_OK;
}

// An operand: `groups` matrices of `rows` rows along the output, `depth` codes
// each; MN-major: of `depth` rows.
struct Operand {
  const void* codes;
  bool mn;
  int64_t ld, stride, groups, rows, depth;
};

// Fills what the operands' majors decide: descriptors, steps and maps.
int set_operands(F8Params* p, const KernelInfo& ki, tcg_input type, const Operand& P, const Operand& Q) {
  p->p_mn = P.mn;
  p->q_mn = Q.mn;
  p->p_hi = P.mn ? sdesc_hi(128 * BLOCK, 1024, SW_128B) : sdesc_hi(16, 1024, SW_128B);
  p->q_hi = Q.mn ? sdesc_hi(128 * BLOCK, 1024, SW_128B) : sdesc_hi(16, 1024, SW_128B);
  p->p_kstep = P.mn ? 32 * 128 / 16 : 32 / 16;
  p->q_kstep = Q.mn ? 32 * 128 / 16 : 32 / 16;
  const uint32_t format = type == TCG_IN_E5M2 ? MXF_E5M2 : MXF_E4M3;
  // kind::f8f6f4's descriptor: D fp32, then formats, majors and sizes as of kind::f16
  p->idesc = (1u << 4) | (format << 7) | (format << 10) | (static_cast<uint32_t>(P.mn) << 15) |
             (static_cast<uint32_t>(Q.mn) << 16) | (static_cast<uint32_t>(128 * ki.cta_group >> 4) << 24);
  if (P.depth == 0) return TCG_OK;
  const auto map = [](CUtensorMap* m, const Operand& o, uint32_t rows) {
    return o.mn ? make_byte_map(m, o.codes, o.rows, o.depth, o.groups, o.ld, o.stride, 128, BLOCK)
                : make_byte_map(m, o.codes, o.depth, o.rows, o.groups, o.ld, o.stride, 128, rows);
  };
  if (int rc = map(&p->tmap_p, P, 128)) return rc;
  if (int rc = map(&p->tmap_q, Q, static_cast<uint32_t>(ki.bn / ki.cta_group))) return rc;
  return Q.mn ? TCG_OK : map(&p->tmap_q16, Q, 16);
}

// Launches the variant on all SMs (or on fewer, never more than `units`
// clusters), as a programmatic dependent of the stream's previous kernel.
int launch_f8(const KernelInfo& ki, F8Params& p, int dev, int64_t units, cudaStream_t s) {
  if (units > INT32_MAX / 2) return TCG_ERR_UNSUPPORTED;
  int clusters = 0;
  if (int rc = max_resident_clusters(dev, ki, &clusters)) return rc;
  const int cg = std::max(ki.cta_group, p.split);
  if (p.split > 1) clusters = static_cast<int>(units);
  p.d_size = p.d_type == TCG_F32 ? 4 : 2;
  // TMA stores where the output's rows and matrices are 16-byte aligned and
  // end on such a boundary
  const int64_t low = reinterpret_cast<int64_t>(p.D) | p.ldd * p.d_size | p.stride_d * p.d_size |
                      static_cast<int64_t>(p.M) * p.d_size;
  p.d_tma = low % 16 == 0;
  if (p.d_tma) {
    const uint64_t rows = static_cast<uint64_t>(p.weight ? p.C : p.R), outer = p.weight ? p.G : 1;
    if (int rc = make_store_map(&p.tmap_d, p.D, static_cast<tcg_dtype>(p.d_type), p.M, rows, outer, p.ldd,
                                p.weight ? p.stride_d : p.R * p.ldd, 128))
      return rc;
  }
  p.err = device_error_word(dev);
  p.timeout_ns = wait_timeout_ns();
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(cg * std::max<int64_t>(1, std::min<int64_t>(units, clusters))), 1, 1);
  cfg.blockDim = dim3(static_cast<unsigned>(ki.threads), 1, 1);
  cfg.dynamicSmemBytes = ki.smem_bytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cg;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cg > 1 ? 2 : 1;
  void* args[] = {&p};
  if (int rc = record_cuda(cudaLaunchKernelExC(&cfg, ki.func, args))) return rc;
  set_launch_count(1);
  record_f8_plan(p.offsets != nullptr, ki.cta_group, ki.bn, p.split, static_cast<int>(cfg.gridDim.x) / cg);
  return TCG_OK;
}

// How a product of R rows in G groups is run.
struct Plan {
  KernelInfo ki;
  Scaling mode;
};

// A few rows a group stream the matrices (gemv_f8.cu) where the tiles of 128 x 64 are
// few for the SMs; many keep every SM reading, and streaming passes over the matrix of
// a popular group again for each eight of its rows.  Tiles and streamed, us:
//     up to two rows a group, and a tile an SM for each 800 of K, but at least 2 and at most 7
//       1 x 8192 x 8192 18.9 and 15.8; 32 rows over 16 groups of 4096 x 4096 52.9 and 46.4 (3.4 tiles
//       an SM), 96 over 48 of 2048 x 4096 73.7 and 69.1 (5.1), 96 over 48 of 2048 x 8192 138.9 and 121.9;
//       beyond, 128 over 64 of 4096 x 1024 53.8 and 80.4 (13.5; all rows in one group 8.9 and 27.2),
//       256 over 128 of 4096 x 4096 319 and 360 (27; 17.5 and 132), 64 over 32 of 2048 x 2048 30.4 and 31.9 (3.4)
//     up to eight, below 64 MB of matrices and up to 1.5 tiles an SM
//       8 x 4096 x 4096 11.5 and 8.7, 64 rows over 8 groups of 2992 x 2048 17.7 and 15.8 (1.3);
//       beyond, 8 x 8192 x 8192 18.9 and 21.5, 512 over 64 of 512 x 512 12.3 and 13.5 (1.7)
// Only the average is known here: all of 32 rows in one of 16 groups of 4096 x 4096 take
// 20.8 streamed and 14.7 in tiles.
bool few_rows(int64_t R, int G, int64_t N, int64_t K, int sms) {
  const int64_t tiles = G * ceil_div(N, 128);
  if (R <= 2 * static_cast<int64_t>(G)) return tiles <= sms * std::min(std::max(K / 800.0, 2.0), 7.0);
  return R <= 8 * static_cast<int64_t>(G) && N * K < (int64_t{1} << 26) / G && 2 * tiles <= 3 * sms;
}

// Tiles of 128 x 64 for up to 64 rows a group, and where there are no more of them
// than SMs: 128 x 4096 x 4096 in 13.8 us (256 x 256: 21.0), 256 x 4096 x 4096 16.4
// (21.3), 128 x 8192 x 8192 26.8 (35.5), 512 x 2048 x 8192 26.4 (34.8); beyond, 300 x
// 4096 x 4096 takes 19.8 with 256 x 256.  Here too the average decides: 2048 rows over 32
// groups of 4096 x 2048 take 50 us if even (256 x 256: 65), 65 (72) with half of them in
// one group and 43 (23) with all.
Plan choose(int64_t R, int64_t N, int G, int dev, bool a_mn, bool square) {
  if (!square) return {variant<2, 256, 5, BOTH>(), BOTH};
  const bool idle = (ceil_div(R, 64) + G - 1) * ceil_div(N, 128) <= device_sms(dev);
  if (!a_mn && (R <= 64 * static_cast<int64_t>(G) || idle)) return {variant<1, 64, 6, COLUMNS>(), COLUMNS};
  return {variant<2, 256, 5, ROWS>(), ROWS};
}

// A's rows and scales against B's, for the dense and the grouped product.
int run_rows(const Plan& plan, F8Params& p, int dev, tcg_input type, const Operand& A, const float* SA, int64_t ld_sa,
             const Operand& B, const float* SB, int64_t ld_sb, int64_t stride_sb, int64_t groups, cudaStream_t s) {
  const bool rows = plan.mode == ROWS;
  const int cg = plan.ki.cta_group;
  p.m_tiles = static_cast<int>(ceil_div(p.M, rows ? plan.ki.bn : 128 * cg));
  if (int rc = rows ? set_operands(&p, plan.ki, type, A, B) : set_operands(&p, plan.ki, type, B, A)) return rc;
  p.fine = SA;
  p.fine_b = ld_sa;
  p.other = SB;
  p.other_group = stride_sb;
  p.other_row = B.mn ? 1 : ld_sb;
  p.other_b = plan.mode == BOTH || B.mn ? ld_sb : 1;
  // an upper bound of the units: a full tile per so many rows, and a partial one more for each group
  const int64_t per = rows ? 128 * cg : plan.ki.bn;
  const int64_t units = (ceil_div(p.R, per) + groups - 1) * p.m_tiles;
  // Where the tiles leave SMs idle, 2 or 4 CTAs share one's contraction (at least
  // four blocks each).
  p.split = 1;
  if (plan.mode == COLUMNS)
    while (p.split < 4 && units * p.split * 2 <= device_sms(dev) && p.K >= 8 * BLOCK * p.split) p.split *= 2;
  return launch_f8(plan.ki, p, dev, units, s);
}

int run_dense(tcg_input type, int64_t M, int64_t N, int64_t K, const void* A, tcg_major a_major, int64_t lda,
              const float* SA, int64_t ld_sa, const void* B, tcg_major b_major, int64_t ldb, const float* SB,
              int64_t ld_sb, int sb_square, void* D, tcg_dtype d_type, int64_t ldd, cudaStream_t s) {
  begin_product();
  if (int rc = check_problem(type, M, N, K, 1, d_type)) return rc;
  if (a_major != TCG_K_MAJOR && a_major != TCG_MN_MAJOR) return TCG_ERR_INVALID;
  if (b_major != TCG_K_MAJOR && b_major != TCG_MN_MAJOR) return TCG_ERR_INVALID;
  if (M == 0 || N == 0) return TCG_OK;
  if (int rc = check_output(D, N, &ldd, d_type)) return rc;
  const bool a_mn = a_major == TCG_MN_MAJOR, b_mn = b_major == TCG_MN_MAJOR;
  const int64_t kb = ceil_div(K, BLOCK), nb = ceil_div(N, BLOCK);
  if (K > 0) {
    if (int rc = check_codes(A, a_mn ? M : K, &lda)) return rc;
    if (int rc = check_codes(B, b_mn ? N : K, &ldb)) return rc;
    if (int rc = check_scales(SA, M, &ld_sa)) return rc;
    if (int rc = check_scales(SB, !sb_square ? N : b_mn ? nb : kb, &ld_sb)) return rc;
  }
  int dev;
  if (int rc = current_device_checked(&dev)) return rc;
  if (sb_square && !a_mn && !b_mn && few_rows(M, 1, N, K, device_sms(dev)))
    return run_gemv_f8(type, M, N, K, 1, A, lda, SA, ld_sa, nullptr, B, ldb, N * ldb, SB, ld_sb, 0, D, d_type, ldd, dev, s);
  F8Params p;
  std::memset(&p, 0, sizeof p);
  p.G = 1;
  p.R = static_cast<int>(M);
  p.M = static_cast<int>(N);
  p.K = static_cast<int>(K);
  p.D = D;
  p.ldd = ldd;
  p.d_type = d_type;
  return run_rows(choose(M, N, 1, dev, a_mn, sb_square), p, dev, type, {A, a_mn, lda, (a_mn ? K : M) * lda, 1, M, K}, SA, ld_sa,
                  {B, b_mn, ldb, (b_mn ? K : N) * ldb, 1, N, K}, SB, ld_sb, 0, 1, s);
}

int run_grouped(tcg_input type, int64_t R, int64_t N, int64_t K, int G, const void* A, int64_t lda, const float* SA,
                int64_t ld_sa, const int32_t* offsets, const void* B, tcg_major b_major, int64_t ldb, int64_t stride_b,
                const float* SB, int64_t ld_sb, int64_t stride_sb, void* D, tcg_dtype d_type, int64_t ldd,
                cudaStream_t s) {
  begin_product();
  if (int rc = check_problem(type, R, N, K, G, d_type)) return rc;
  if (b_major != TCG_K_MAJOR && b_major != TCG_MN_MAJOR) return TCG_ERR_INVALID;
  if (R == 0 || N == 0) return TCG_OK;
  if (int rc = check_output(D, N, &ldd, d_type)) return rc;
  if (!offsets) return TCG_ERR_INVALID;
  if (misaligned(offsets, 4)) return TCG_ERR_ALIGNMENT;
  const bool mn = b_major == TCG_MN_MAJOR;
  const int64_t kb = ceil_div(K, BLOCK), nb = ceil_div(N, BLOCK);
  if (K > 0) {
    if (int rc = check_codes(A, K, &lda)) return rc;
    if (int rc = check_codes(B, mn ? N : K, &ldb)) return rc;
    if (stride_b == 0) stride_b = (mn ? K : N) * ldb;
    if (stride_b < 0) return TCG_ERR_INVALID;
    if (stride_b % 16) return TCG_ERR_ALIGNMENT;
    if (int rc = check_scales(SA, R, &ld_sa)) return rc;
    if (int rc = check_scales(SB, mn ? nb : kb, &ld_sb)) return rc;
    if (stride_sb == 0) stride_sb = (mn ? kb : nb) * ld_sb;
    if (stride_sb < 0) return TCG_ERR_INVALID;
  }
  int dev;
  if (int rc = current_device_checked(&dev)) return rc;
  if (!mn && few_rows(R, G, N, K, device_sms(dev)))
    return run_gemv_f8(type, R, N, K, G, A, lda, SA, ld_sa, offsets, B, ldb, stride_b, SB, ld_sb, stride_sb, D, d_type,
                       ldd, dev, s);
  F8Params p;
  std::memset(&p, 0, sizeof p);
  p.offsets = offsets;
  p.G = G;
  p.R = static_cast<int>(R);
  p.M = static_cast<int>(N);
  p.K = static_cast<int>(K);
  p.D = D;
  p.ldd = ldd;
  p.d_type = d_type;
  return run_rows(choose(R, N, G, dev, false, true), p, dev, type, {A, false, lda, R * lda, 1, R, K}, SA, ld_sa,
                  {B, mn, ldb, stride_b, G, N, K}, SB, ld_sb, stride_sb, std::min<int64_t>(G, R), s);
}

int run_wgrad(tcg_input type, int64_t R, int64_t N, int64_t K, int G, const void* DY, int64_t lddy, const float* SDY,
              int64_t ld_sdy, const void* A, int64_t lda, const float* SA, int64_t ld_sa, const int32_t* offsets,
              void* DW, tcg_dtype dw_type, int64_t lddw, int64_t stride_dw, cudaStream_t s) {
  begin_product();
  if (int rc = check_problem(type, R, N, K, G, dw_type)) return rc;
  if (N == 0 || K == 0) return TCG_OK;
  if (int rc = check_output(DW, K, &lddw, dw_type)) return rc;
  if (stride_dw == 0) stride_dw = N * lddw;
  if (stride_dw < 0) return TCG_ERR_INVALID;
  if (!offsets) return TCG_ERR_INVALID;
  if (misaligned(offsets, 4)) return TCG_ERR_ALIGNMENT;
  if (R > 0) {
    if (int rc = check_codes(DY, N, &lddy)) return rc;
    if (int rc = check_codes(A, K, &lda)) return rc;
    if (int rc = check_scales(SDY, N, &ld_sdy)) return rc;
    if (int rc = check_scales(SA, K, &ld_sa)) return rc;
  }
  int dev;
  if (int rc = current_device_checked(&dev)) return rc;
  const KernelInfo ki = variant<2, 256, 5, BOTH>();
  F8Params p;
  std::memset(&p, 0, sizeof p);
  p.offsets = offsets;
  p.G = G;
  p.R = static_cast<int>(R);
  p.weight = p.split = 1;
  p.M = static_cast<int>(K);
  p.C = static_cast<int>(N);
  p.m_tiles = static_cast<int>(ceil_div(K, 128 * ki.cta_group));
  if (int rc = set_operands(&p, ki, type, {A, true, lda, R * lda, 1, K, R}, {DY, true, lddy, R * lddy, 1, N, R})) return rc;
  p.fine = SDY;
  p.fine_b = ld_sdy;
  p.other = SA;
  p.other_b = ld_sa;
  p.D = DW;
  p.ldd = lddw;
  p.stride_d = stride_dw;
  p.d_type = dw_type;
  return launch_f8(ki, p, dev, static_cast<int64_t>(G) * ceil_div(N, ki.bn) * p.m_tiles, s);
}

}  // namespace

}  // namespace tcg

using namespace tcg;

extern "C" {

int tcg_gemm_f8(tcg_input in_type, int64_t M, int64_t N, int64_t K, const void* A, tcg_major a_major, int64_t lda,
                const float* SA, int64_t ld_sa, const void* B, tcg_major b_major, int64_t ldb, const float* SB,
                int64_t ld_sb, int sb_square, void* D, tcg_dtype d_type, int64_t ldd, void* stream) {
  return guarded([&] {
    return run_dense(in_type, M, N, K, A, a_major, lda, SA, ld_sa, B, b_major, ldb, SB, ld_sb, sb_square, D, d_type, ldd,
                     static_cast<cudaStream_t>(stream));
  });
}

int tcg_gemm_f8_grouped(tcg_input in_type, int64_t R, int64_t N, int64_t K, int G, const void* A, int64_t lda,
                        const float* SA, int64_t ld_sa, const int32_t* offsets, const void* B, tcg_major b_major,
                        int64_t ldb, int64_t stride_b, const float* SB, int64_t ld_sb, int64_t stride_sb, void* D,
                        tcg_dtype d_type, int64_t ldd, void* stream) {
  return guarded([&] {
    return run_grouped(in_type, R, N, K, G, A, lda, SA, ld_sa, offsets, B, b_major, ldb, stride_b, SB, ld_sb, stride_sb,
                       D, d_type, ldd, static_cast<cudaStream_t>(stream));
  });
}

int tcg_gemm_f8_grouped_wgrad(tcg_input in_type, int64_t R, int64_t N, int64_t K, int G, const void* DY, int64_t lddy,
                              const float* SDY, int64_t ld_sdy, const void* A, int64_t lda, const float* SA,
                              int64_t ld_sa, const int32_t* offsets, void* DW, tcg_dtype dw_type, int64_t lddw,
                              int64_t stride_dw, void* stream) {
  return guarded([&] {
    return run_wgrad(in_type, R, N, K, G, DY, lddy, SDY, ld_sdy, A, lda, SA, ld_sa, offsets, DW, dw_type, lddw, stride_dw,
                     static_cast<cudaStream_t>(stream));
  });
}

}  // extern "C"
