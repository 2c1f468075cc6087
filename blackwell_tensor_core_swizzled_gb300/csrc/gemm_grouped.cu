// Products of sorted rows with their group's matrix, and the gradient of the
// matrices, on the tensor cores.  Entry points, host plan and kernel; the
// contract is in include/tcg.h.
//
// One kernel serves all three products.  It computes C[m, c] = sum_k P[m, k]
// Q[c, k] in tiles of 128 * CG rows m by up to BN columns c and stores it
// transposed, element (m, c) at out[c * ldd + m]:
//
//             P (MMA rows)              Q (MMA columns)      contraction
//   forward   B[g], rows n, K-major     the group's rows r   K
//   input     B[g], rows n, MN-major    the group's rows r   K
//   weight    A, columns k, MN-major    DY, columns n        the group's rows
//
// The ragged extent of a product, the group's rows, is thus on the MMA's N
// side, which any multiple of 16 (32 for a CTA pair) up to 256 may have: a
// tile with few rows costs few columns and nothing is padded in memory.  A
// group's rows are split evenly into as few tiles of at most BN as they need.
//
// Outputs leave in blocks of 32 m by 32 columns (fp32: 16) through a shared
// staging tile and a TMA store, rows of the tile being output rows; a block
// that a group's end cuts and outputs that are not 16-byte aligned are stored
// by the lanes, an output row an instruction.  (Blocks of 64 m by pairs of
// warps, and fp32 ones of 32 columns, were 1 and 15 % slower.)
//
// In the weight product the contraction is ragged: the last 64-row block of a
// group also loads rows of the next group.  The MMAs of 16 rows beyond the
// end are not issued, and the rows of the last partial 16 are overwritten with
// zeros in shared memory (both operands: the neighbour's rows may hold
// infinities) before the MMA reads them.
//
// fp32 outputs: the tensor core cuts a running sum's last bits at every step, an
// error that grows with the contraction (2.6e-6 of the result at 4096).  So
// every few blocks (at most CHAIN) the MMAs change to the other accumulator, and
// the epilogue adds the finished one to sums in its registers (rounded), while
// the next is computed.  The error stays that of one chain, 4.7e-7 at 512 and at
// 16384; plain fp32 products are at 1.6e-7 to 6.1e-7.  16-bit outputs round far
// more than that and take the whole contraction in one accumulator: at 4096,
// 0.2 % of bf16 values round to the other neighbour than a plain fp32 sum's do,
// and both are as far from the exact result (1.66e-3).
//
// What bounds it: many rows a group, the tensor cores (32768 rows x 4096 x 4096
// of one group 558 us, where the dense kernel takes 537; 65536 x 2048 x 4096 in
// 32 groups 1.64 to 1.76 PFLOP/s with the clock); few, the matrices' bytes from
// HBM (96 us for 537 MB: 5.6 TB/s); the matrices' gradient in fp32, the stores:
// a warp's block of 2 KB leaves in some 700 cycles, which for all SMs is HBM's
// rate, but nothing leaves while the same warps add a chain, and every 512 rows
// begin one more (32 groups of 2048 x 4096: 64 rows 172 us fp32, 6.2 TB/s, and
// 102 bf16; 512 rows each 236 and 190; the same rows unevenly, spread 0.5, 291
// to 328 and 241).  (The pair kernels spill 24 bytes.)
//
// The structure is the dense kernel's: a persistent CTA (or pair) per SM, TMA
// producer warps, an MMA warp, two accumulators in TMEM, epilogue warps.
// The tile list depends on offsets, which only the device knows, so each CTA
// reads them once and keeps the running tile count per group in shared memory;
// a warp turns unit indexes into tiles by a binary search, ahead of the others.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstring>

#include "common.h"
#include "desc.cuh"
#include "gemm_kernel.cuh"
#include "ptx.cuh"
#include "ptx_moe.cuh"
#include "tmem_ldst.cuh"

namespace tcg {

namespace {

constexpr int MAX_GROUPS = 1024;
constexpr int64_t MAX_EXTENT = int64_t{1} << 30;
constexpr int EPI_WARPS = 8;
constexpr int STAGING_BYTES = 2048;
constexpr int TILES = 4;  // decoded tiles ahead of the warps that work on them
constexpr int GROUPED_THREADS = 32 * (4 + EPI_WARPS);
// fp32 outputs: blocks of the contraction summed by the tensor core at most
// (16384 x 2048 x 4096 in 32 groups: 8 blocks 233 us, 4 299, 16 229, all 226)
constexpr int CHAIN = 8;
// column tiles of a group that sweep its row tiles together (1, 4, 8 and 16
// are within 4 % of each other at 32 groups of 2048 x 4096)
constexpr int BAND = 8;

struct GroupedParams {
  CUtensorMap tmap_p;    // [G or 1][rows][64-element boxes]
  CUtensorMap tmap_q;    // Q in boxes of a full tile's rows (MN-major: 64)
  CUtensorMap tmap_q16;  // K-major Q in boxes of 16 rows, for partial tiles
  CUtensorMap tmap_d;    // 16-bit output [G or 1][c][m] in boxes of 32 m and 32 rows
  int d_tma;
  const int32_t* offsets;
  int G, R;
  int weight;    // the contraction runs over the group's rows
  int p_mn;      // P is MN-major
  int M;         // extent of m
  int C;         // weight: extent of c
  int K;         // forward, input: contraction length
  int m_tiles;
  uint64_t p_hi, q_hi;
  uint32_t p_kstep, q_kstep;  // 16-byte units per 16 of the contraction
  uint32_t idesc;             // without N
  void* D;
  int64_t ldd, stride_d;
  int d_type, d_size;
  int pairs;  // 16-bit outputs: two m at a time are 4-byte aligned, and M is even
  unsigned long long* err;
  uint64_t timeout_ns;
};

template <int CG, int BN, int STAGES, int GROUPS>
struct GroupedCfg {
  static constexpr int P_BYTES = 128 * 128;
  static constexpr int Q_ROWS = BN / CG;
  static constexpr int Q_BYTES = Q_ROWS * 128;
  static constexpr int STAGE_BYTES = P_BYTES + Q_BYTES;
  // two staging tiles for each epilogue warp
  static constexpr int EPI_OFF = STAGES * STAGE_BYTES;
  static constexpr int BAR_OFF = EPI_OFF + EPI_WARPS * 2 * STAGING_BYTES;
  // full[S], empty[S], rag[S], peer[S], acc_full[2], acc_empty[2], drain, tile_full[T], tile_empty[T]
  static constexpr int NUM_BARS = 4 * STAGES + 5 + 2 * TILES;
  static constexpr int TILE_OFF = (BAR_OFF + NUM_BARS * 8 + 8 + 15) / 16 * 16;  // tmem slot + abort flag before it
  static constexpr int SEG_OFF = TILE_OFF + TILES * 48;
  static constexpr int SMEM_BYTES = 1024 + SEG_OFF + 2 * (GROUPS + 1) * 4;
  static_assert(Q_BYTES % 1024 == 0, "swizzle period");
  static_assert(SMEM_BYTES <= 232448, "dynamic shared memory");
  static_assert(2 * BN <= 512, "two accumulators");
};

// One unit: a tile of one group.
struct alignas(16) GTile {
  int g;
  int lo;     // first row of the group
  int m0;     // first m of the tile (of the pair's tile)
  int c0;     // first column within the group (weight: within C)
  int ncols;  // columns of the tile that exist
  int mma_n;  // columns the MMA computes
  int nkb;    // 64-deep blocks of the contraction (0: the tile is zero)
  int last;   // depth of the last block
  int chain;  // blocks one accumulator takes
};

// A group's columns n: tiles of `per` columns each, the last one shorter.
template <int CG, int BN>
__device__ __forceinline__ void split_columns(int n, int& tiles, int& per) {
  const int t = (n + BN - 1) / BN;
  per = t ? ((n + t - 1) / t + 16 * CG - 1) / (16 * CG) * (16 * CG) : 16 * CG;
  tiles = (n + per - 1) / per;
}

// seg[0..G]: clamped offsets; pre[0..G]: units of the groups before (forward).
template <int CG, int BN>
__device__ __forceinline__ GTile decode_unit(const GroupedParams& p, const int* seg, const int* pre, int u) {
  GTile t;
  int v, tiles, per, n;
  if (p.weight) {
    split_columns<CG, BN>(p.C, tiles, per);
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
    split_columns<CG, BN>(n, tiles, per);
  }
  t.lo = seg[t.g];
  const int depth = p.weight ? seg[t.g + 1] - t.lo : p.K;
  const int band = v / (BAND * p.m_tiles);
  const int first = band * BAND;
  const int width = min(tiles - first, BAND);
  v -= first * p.m_tiles;
  t.m0 = (v / width) * (128 * CG);
  t.c0 = (first + v % width) * per;
  t.ncols = min(per, n - t.c0);
  t.mma_n = (t.ncols + 16 * CG - 1) / (16 * CG) * (16 * CG);
  t.nkb = (depth + 63) >> 6;
  t.last = depth - 64 * (t.nkb - 1);
  // fp32 outputs: equal chains of at most CHAIN blocks (with 8 and then 1, nine
  // blocks left the short chain's epilogue uncovered: 17 % of the product's time)
  t.chain = max(1, t.nkb);
  if (p.d_type == OUT_F32 && t.nkb > CHAIN) {
    const int chains = (t.nkb + CHAIN - 1) / CHAIN;
    t.chain = (t.nkb + chains - 1) / chains;
  }
  return t;
}

// Store up to 32 accumulator columns of one warp: lane = m, register i =
// column i, whose row of the output starts i * pitch bytes after `dst` (this
// lane's element of the first).  Addresses advance by additions alone: as a
// multiplication for each column they took more of the epilogue than the
// stores.  16-bit outputs in pairs: neighbouring lanes exchange halves, so that
// an even lane stores two m of column i and an odd one two m of column i + 1.
__device__ __forceinline__ void store_columns(uint8_t* dst, int64_t pitch, int ncols, bool m_ok, int type, bool pairs,
                                              int lane, const uint32_t (&r)[32]) {
  if (type == OUT_F32) {
#pragma unroll
    for (int i = 0; i < 32; ++i, dst += pitch) {
      if (i >= ncols) break;
      if (m_ok) __stcs(reinterpret_cast<uint32_t*>(dst), r[i]);
    }
    return;
  }
  const bool bf = type == OUT_BF16;
  if (pairs) {
    const uint32_t pick = (lane & 1) ? 0x3276u : 0x5410u;
    dst += (lane & 1) ? pitch - 2 : 0;
    pitch *= 2;
#pragma unroll
    for (int i = 0; i < 32; i += 2, dst += pitch) {
      if (i >= ncols) break;
      const uint32_t h = bf ? pack_bf16(r[i], r[i + 1]) : pack_f16(r[i], r[i + 1]);
      const uint32_t o = __shfl_xor_sync(0xffffffffu, h, 1);
      if (m_ok && ((lane & 1) == 0 || i + 1 < ncols)) *reinterpret_cast<uint32_t*>(dst) = __byte_perm(h, o, pick);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 32; i += 2, dst += 2 * pitch) {
      if (i >= ncols) break;
      const uint32_t h = bf ? pack_bf16(r[i], r[i + 1]) : pack_f16(r[i], r[i + 1]);
      if (m_ok) *reinterpret_cast<uint16_t*>(dst) = static_cast<uint16_t>(h);
      if (m_ok && i + 1 < ncols) *reinterpret_cast<uint16_t*>(dst + pitch) = static_cast<uint16_t>(h >> 16);
    }
  }
}

template <int CG, int BN, int STAGES, int GROUPS>
__global__ void __launch_bounds__(GROUPED_THREADS, 1) grouped_kernel(const __grid_constant__ GroupedParams p) {
  using C = GroupedCfg<CG, BN, STAGES, GROUPS>;
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
  auto acce_bar = [&](uint32_t b) { return bar0 + 8u * (4 * STAGES + 2 + b); };
  const uint32_t drain_bar = bar0 + 8u * (4 * STAGES + 4);
  auto tile_full = [&](uint32_t i) { return bar0 + 8u * (4 * STAGES + 5 + i); };
  auto tile_empty = [&](uint32_t i) { return bar0 + 8u * (4 * STAGES + 5 + TILES + i); };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + C::BAR_OFF + 8 * C::NUM_BARS);
  volatile uint32_t* abort_flag = tmem_slot + 1;
  int* seg = reinterpret_cast<int*>(gbase + C::SEG_OFF);
  int* pre = seg + p.G + 1;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = (CG == 2) ? cluster_ctarank() : 0u;
  const int cluster_id = blockIdx.x / CG;
  const int num_clusters = gridDim.x / CG;
  const WaitCtx wctx{p.timeout_ns, p.err, abort_flag};

  // the maps exist unless the contraction is empty
  if (warp == 0 && lane == 0 && (p.weight ? p.R : p.K) > 0) {
    prefetch_tmap(&p.tmap_p);
    prefetch_tmap(&p.tmap_q);
    if (!p.weight) prefetch_tmap(&p.tmap_q16);
  }
  if (threadIdx.x == 96) {
    for (uint32_t s = 0; s < STAGES; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
      mbar_init(rag_bar(s), 1);
      mbar_init(peer_bar(s), 1);
    }
    for (uint32_t b = 0; b < 2; ++b) {
      mbar_init(accf_bar(b), 1);
      mbar_init(acce_bar(b), EPI_WARPS * CG);
    }
    mbar_init(drain_bar, 1);
    for (uint32_t i = 0; i < TILES; ++i) {
      mbar_init(tile_full(i), 1);
      mbar_init(tile_empty(i), 3 + EPI_WARPS);
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
  for (int g = threadIdx.x; g <= p.G; g += GROUPED_THREADS) seg[g] = p.offsets[g];
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
        split_columns<CG, BN>(v - before, tiles, per);
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
  if constexpr (CG == 2) cluster_sync();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  griddep_launch_dependents();
  int total_units;
  if (p.weight) {
    int tiles, per;
    split_columns<CG, BN>(p.C, tiles, per);
    total_units = p.G * tiles * p.m_tiles;
  } else {
    total_units = p.K > 0 ? pre[p.G] : 0;
  }

  // The n-th tile of this CTA, decoded by warp 3: half a dozen divisions, 1150
  // cycles of each tile of a small contraction when every warp did its own.
  GTile* tiles = reinterpret_cast<GTile*>(gbase + C::TILE_OFF);
  auto fetch = [&](uint32_t n, GTile& t) {
    const uint32_t i = n % TILES;
    if (!wait_uniform(tile_full(i), (n / TILES) & 1u, wctx, SITE_PROD_EMPTY)) return false;
    t = tiles[i];
    __syncwarp();
    if (lane == 0) mbar_arrive(tile_empty(i));
    return true;
  };

  if (warp == 3) {
    // ------------------------------------------------------------ tile list
    uint32_t n = 0;
    for (int u = cluster_id; u < total_units; u += num_clusters, ++n) {
      const GTile t = decode_unit<CG, BN>(p, seg, pre, u);
      const uint32_t i = n % TILES;
      if (!wait_uniform(tile_empty(i), ((n / TILES) & 1u) ^ 1u, wctx, SITE_PROD_EMPTY)) break;
      if (lane == 0) {
        tiles[i] = t;
        mbar_arrive(tile_full(i));
      }
      __syncwarp();
    }
  } else if (warp == 0 || warp == 2) {
    // ---------------------------------------------- producers, of P and of Q:
    // one thread takes 150 cycles a copy, and the matrices' gradient has four
    // to a block whose MMAs take 512
    const bool brings_p = warp == 0;
    uint32_t it = 0, s = 0, ph = 0, n = 0;
    bool ok = true;
    for (int u = cluster_id; u < total_units && ok; u += num_clusters) {
      GTile t;
      ok = fetch(n++, t);
      if (!ok) break;
      const int half = t.mma_n / CG;
      const int m0 = t.m0 + static_cast<int>(rank) * 128;
      const int c0 = t.c0 + static_cast<int>(rank) * half;
      const int q_chunks = (half + 63) >> 6;
      const uint32_t tx = C::P_BYTES + static_cast<uint32_t>(p.weight ? q_chunks * 8192 : half * 128);
      for (int kb = 0; kb < t.nkb; ++kb) {
        if (!wait_uniform(empty_bar(s), ph ^ 1u, wctx, SITE_PROD_EMPTY)) {
          ok = false;
          break;
        }
        if (elect_one()) {
          const uint32_t sp = sbase + s * C::STAGE_BYTES;
          const uint32_t sq = sp + C::P_BYTES;
          const int k0 = 64 * kb;
          const uint32_t fb = (CG == 2) ? mapa_shared(full_bar(s), 0) : full_bar(s);
          if (p.weight && kb == t.nkb - 1 && (t.last & 15)) {
            // the warp that zeroes the rows past the group's end waits for
            // this CTA's bytes alone; full[s] just marks the stage
            const int r0 = t.lo + k0;
            if (brings_p) {
              if (rank == 0) mbar_arrive(full_bar(s));
              mbar_arrive_expect_tx(rag_bar(s), tx);
              for (int i = 0; i < 2; ++i) tma_load3<1>(sp + 8192 * i, &p.tmap_p, m0 + 64 * i, r0, 0, rag_bar(s));
            } else {
              for (int i = 0; i < q_chunks; ++i) tma_load_2d(sq + 8192 * i, &p.tmap_q, c0 + 64 * i, r0, rag_bar(s));
            }
          } else if (brings_p) {
            if (rank == 0) mbar_arrive_expect_tx(full_bar(s), tx * CG);
            if (!p.p_mn) {
              tma_load3<CG>(sp, &p.tmap_p, k0, m0, t.g, fb);
            } else {
              for (int i = 0; i < 2; ++i)
                tma_load3<CG>(sp + 8192 * i, &p.tmap_p, m0 + 64 * i, p.weight ? t.lo + k0 : k0, p.weight ? 0 : t.g, fb);
            }
          } else if (p.weight) {
            for (int i = 0; i < q_chunks; ++i) tma_load<CG>(sq + 8192 * i, &p.tmap_q, c0 + 64 * i, t.lo + k0, fb);
          } else if (half == C::Q_ROWS) {
            tma_load<CG>(sq, &p.tmap_q, k0, t.lo + c0, fb);
          } else {
            for (int i = 0; i < half; i += 16) tma_load<CG>(sq + 128 * i, &p.tmap_q16, k0, t.lo + c0 + i, fb);
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
  } else if (warp == 1) {
    // --------------------------------- MMA issuer (leader), row zeroing (both)
    const uint64_t p_desc0 = sdesc(sbase, p.p_hi);
    const uint64_t q_desc0 = sdesc(sbase + C::P_BYTES, p.q_hi);
    uint32_t s = 0, ph = 0, n = 0, tcount = 0, rag_ph = 0;  // rag_ph: one parity bit per stage
    bool ok = true;
    for (int u = cluster_id; u < total_units && ok; u += num_clusters) {
      GTile t;
      ok = fetch(n++, t);
      if (!ok) break;
      if (t.nkb == 0) continue;
      const bool issue = CG == 1 || rank == 0;
      const uint32_t idesc = p.idesc | (static_cast<uint32_t>(t.mma_n >> 3) << 17);
      uint32_t b = 0, d_tmem = 0;
      int link = 0;  // blocks in the accumulator
      for (int kb = 0; kb < t.nkb; ++kb) {
        const bool last = kb == t.nkb - 1;
        const bool ragged = p.weight && last && (t.last & 15);
        if (issue && link == 0) {
          b = tcount & 1u;
          if (!wait_uniform(acce_bar(b), ((tcount >> 1) & 1u) ^ 1u, wctx, SITE_MMA_ACC_EMPTY)) {
            ok = false;
            break;
          }
          tc_fence_after();
          ++tcount;
          d_tmem = tmem_base + b * BN;
        }
        if (issue && !wait_uniform(full_bar(s), ph, wctx, SITE_MMA_FULL)) {
          ok = false;
          break;
        }
        if (ragged) {
          const uint32_t par = (rag_ph >> s) & 1u;
          rag_ph ^= 1u << s;
          if (!warp_wait(rag_bar(s), par, wctx, SITE_MMA_FULL)) {
            ok = false;
            break;
          }
          // rows [last, next multiple of 16) of the two P chunks and the Q
          // chunks; a row's 128 bytes are the same under the swizzle
          const uint32_t sp = sbase + s * C::STAGE_BYTES;
          const int rows = 16 - (t.last & 15);
          const int chunks = 2 + ((t.mma_n / CG + 63) >> 6);
          for (int i = lane; i < chunks * rows * 8; i += 32) {
            const int ch = i / (rows * 8), rr = i - ch * rows * 8;
            const uint32_t at = (ch < 2 ? sp + 8192u * ch : sp + C::P_BYTES + 8192u * (ch - 2)) + 128u * (t.last + (rr >> 3)) +
                                16u * (rr & 7);
            st_shared_v4(at, 0u, 0u, 0u, 0u);
          }
          fence_proxy_async_shared();
          __syncwarp();
          if constexpr (CG == 2) {
            if (rank != 0) {
              if (lane == 0) mbar_arrive_cluster(mapa_shared(peer_bar(s), 0));
            } else if (!warp_wait(peer_bar(s), par, wctx, SITE_MMA_FULL) || !mbar_try_wait_cluster(peer_bar(s), par)) {
              ok = false;
              break;
            }
          }
        }
        if (issue) {
          tc_fence_after();
          if (elect_one()) {
            const uint64_t st = (s * static_cast<uint32_t>(C::STAGE_BYTES)) >> 4;
            const int steps = last ? (t.last + 15) >> 4 : 4;
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (j < steps)
                mma_f16<CG>(d_tmem, p_desc0 + st + j * p.p_kstep, q_desc0 + st + j * p.q_kstep, idesc,
                            (link | j) ? 1u : 0u);
            tc_commit<CG>(empty_bar(s));
            if (last || link == t.chain - 1) tc_commit<CG>(accf_bar(b));
          }
          __syncwarp();
        }
        if (++link == t.chain) link = 0;
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
  } else if (warp >= 4) {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;            // TMEM lane quadrant
    const int part = (warp - 4) >> 2;  // 32-column chunks part, part + 2, ...
    uint32_t tcount = 0;
    const uint32_t buf0 = sbase + C::EPI_OFF + static_cast<uint32_t>((warp - 4) * 2 * STAGING_BYTES);
    uint32_t stores = 0;
    // the staging tile to fill next: its store before the last has read it
    auto staging = [&] {
      if (stores >= 2) {
        if (lane == 0) bulk_wait_group_read<1>();
        __syncwarp();
      }
      return buf0 + (stores & 1u) * STAGING_BYTES;
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
    uint32_t n = 0;
    for (int u = cluster_id; u < total_units; u += num_clusters) {
      GTile t;
      if (!fetch(n++, t)) break;
      const int m_warp = t.m0 + static_cast<int>(rank) * 128 + 32 * q;
      // output rows of the map: all c of a matrix clip at its end, rows of a
      // group do not
      const int row0 = p.weight ? t.c0 : t.lo + t.c0, outer = p.weight ? t.g : 0;
      const int m = t.m0 + static_cast<int>(rank) * 128 + 32 * q + lane;
      const bool m_ok = m < p.M;
      const int64_t pitch = p.ldd * p.d_size;
      uint8_t* dst = static_cast<uint8_t*>(p.D) + (p.weight ? t.g * p.stride_d * p.d_size + t.c0 * pitch : (t.lo + t.c0) * pitch) +
                     static_cast<int64_t>(m) * p.d_size;
      if (t.nkb == 0) {
        const uint32_t zero[32] = {};
        for (int c = 32 * part; c < t.ncols; c += 64)
          store_columns(dst + c * pitch, pitch, t.ncols - c, m_ok, p.d_type, p.pairs, lane, zero);
        continue;
      }
      const uint32_t lanes = tmem_base + (static_cast<uint32_t>(32 * q) << 16);
      auto release = [&](uint32_t b) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if constexpr (CG == 2)
            mbar_arrive_relaxed(mapa_shared(acce_bar(b), 0));  // no memory to order, only TMEM reads
          else
            mbar_arrive(acce_bar(b));
        }
      };
      if (p.d_type == OUT_F32) {
        constexpr int MINE = (BN + 63) / 64;  // blocks of 32 columns of this warp
        float sum[MINE][32] = {};
        bool done = true;
        for (int kb = 0; kb < t.nkb; kb += t.chain, ++tcount) {
          const uint32_t b = tcount & 1u;
          done = warp_wait(accf_bar(b), (tcount >> 1) & 1u, wctx, SITE_EPI_ACC_FULL);
          if (!done) break;
          tc_fence_after();
#pragma unroll
          for (int i = 0; i < MINE; ++i) {
            const int c = 32 * part + 64 * i;
            if (c >= t.ncols) break;
#pragma unroll
            for (int h = 0; h < 32; h += 16) {  // 16 at a time: registers
              uint32_t r[16];
              ldx_32x32b_x16(lanes + b * BN + c + h, r);
              tc_wait_ld();
#pragma unroll
              for (int k = 0; k < 16; ++k) sum[i][h + k] += __uint_as_float(r[k]);
            }
          }
          release(b);
        }
        if (!done) break;
#pragma unroll
        for (int i = 0; i < MINE; ++i) {
          const int c = 32 * part + 64 * i;
          if (c >= t.ncols) break;
          if (!p.d_tma || !(p.weight || c + 32 <= t.ncols)) {
#pragma unroll
            for (int k = 0; k < 32; ++k)
              if (m_ok && c + k < t.ncols) __stcs(reinterpret_cast<float*>(dst + (c + k) * pitch), sum[i][k]);
            continue;
          }
          if (m_warp >= p.M) break;
#pragma unroll
          for (int h = 0; h < 32; h += 16) {  // a staging tile holds 16 rows of 32 m
            const uint32_t buf = staging();
#pragma unroll
            for (int k = 0; k < 16; ++k) st_shared_u32(buf + 128u * k + 4u * lane, __float_as_uint(sum[i][h + k]));
            send(buf, m_warp, row0 + c + h, outer);
          }
        }
        continue;
      }
      const uint32_t b = tcount & 1u;
      if (!warp_wait(accf_bar(b), (tcount >> 1) & 1u, wctx, SITE_EPI_ACC_FULL)) break;
      ++tcount;
      tc_fence_after();
      const uint32_t tb = lanes + b * BN;
#pragma unroll 1
      for (int c = 32 * part; c < t.ncols; c += 64) {
        if (p.d_tma && (p.weight || c + 32 <= t.ncols)) {
          if (m_warp >= p.M) break;
          // fragments of 16 m each; stmatrix turns 8 m of 8 columns into 8
          // rows of 16 bytes: lane 8k + i addresses row 8j + i, m 8k..8k+7
          uint32_t lo[16], hi[16];
          tmem_ld_16x256b_x4(tb + c, lo);
          tmem_ld_16x256b_x4(tb + c + (16u << 16), hi);
          tc_wait_ld();
          const uint32_t buf = staging();
          const bool bf = p.d_type == OUT_BF16;
          const uint32_t k = static_cast<uint32_t>(lane) >> 3, i = static_cast<uint32_t>(lane) & 7u;
#pragma unroll
          for (uint32_t j = 0; j < 4; ++j) {
            const uint32_t row = 8u * j + i;
            auto pk = [&](uint32_t a, uint32_t b) { return bf ? pack_bf16(a, b) : pack_f16(a, b); };
            stmatrix_x4_trans(buf + 64u * row + 16u * (k ^ ((row >> 1) & 3u)), pk(lo[4 * j], lo[4 * j + 1]),
                              pk(lo[4 * j + 2], lo[4 * j + 3]), pk(hi[4 * j], hi[4 * j + 1]),
                              pk(hi[4 * j + 2], hi[4 * j + 3]));
          }
          send(buf, m_warp, row0 + c, outer);
          continue;
        }
        uint32_t r[32];
        tmem_ld_32x32b_x32(tb + c, r);
        tc_wait_ld();
        store_columns(dst + c * pitch, pitch, t.ncols - c, m_ok, p.d_type, p.pairs, lane, r);
      }
      release(b);
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
        for (int m = t; m < p.M; m += 32 * EPI_WARPS) {
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
  if constexpr (CG == 2) cluster_sync();
  tc_fence_after();
  if (warp == 2) tmem_dealloc<CG>(tmem_base, 512);
}

// ---------------------------------------------------------------------- host

struct Variant {
  KernelInfo ki;
  int bn;
};

template <int CG, int BN, int STAGES, int GROUPS>
Variant variant() {
  using C = GroupedCfg<CG, BN, STAGES, GROUPS>;
  return {KernelInfo{reinterpret_cast<const void*>(&grouped_kernel<CG, BN, STAGES, GROUPS>), C::SMEM_BYTES, CG, BN,
                     KIND_F16, GROUPED_THREADS},
          BN};
}

// CTA pairs; more than 184 groups' tile counts take a ring stage's memory (32
// groups of 2048 x 4096, 16384 rows: fp32 matrices' gradient 2 % slower with
// five stages than with six, rows' gradient 3 %).
Variant pair_variant(int G) { return G <= 184 ? variant<2, 256, 6, 184>() : variant<2, 256, 5, MAX_GROUPS>(); }

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

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Launches the variant on all SMs (or on fewer, never more than `units`
// clusters), as a programmatic dependent of the stream's previous kernel.
int launch_grouped(const Variant& v, GroupedParams& p, int dev, int64_t units, cudaStream_t s) {
  int clusters = 0;
  if (int rc = max_resident_clusters(dev, v.ki, &clusters)) return rc;
  const int cg = v.ki.cta_group;
  p.d_size = p.d_type == TCG_F32 ? 4 : 2;
  p.pairs = reinterpret_cast<uintptr_t>(p.D) % 4 == 0 && p.ldd % 2 == 0 && p.stride_d % 2 == 0 && p.M % 2 == 0;
  // TMA stores where the output's rows and matrices are 16-byte aligned and
  // end on such a boundary (a store is cut at 16-byte steps: rows of 513 bf16
  // were written up to their 516th element)
  const int64_t low = reinterpret_cast<int64_t>(p.D) | p.ldd * p.d_size | p.stride_d * p.d_size |
                      static_cast<int64_t>(p.M) * p.d_size;
  p.d_tma = low % 16 == 0;
  if (p.d_tma) {
    const uint64_t rows = static_cast<uint64_t>(p.weight ? p.C : p.R), outer = p.weight ? p.G : 1;
    if (int rc = make_store_map(&p.tmap_d, p.D, static_cast<tcg_dtype>(p.d_type), p.M, rows, outer, p.ldd, p.weight ? p.stride_d : p.R * p.ldd))
      return rc;
  }
  p.err = device_error_word(dev);
  p.timeout_ns = wait_timeout_ns();
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(cg * std::max<int64_t>(1, std::min<int64_t>(units, clusters))), 1, 1);
  cfg.blockDim = dim3(GROUPED_THREADS, 1, 1);
  cfg.dynamicSmemBytes = v.ki.smem_bytes;
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
  if (int rc = record_cuda(cudaLaunchKernelExC(&cfg, v.ki.func, args))) return rc;
  set_launch_count(1);
  record_grouped_plan(cg, v.bn, static_cast<int>(cfg.gridDim.x) / cg);
  return TCG_OK;
}

int run_grouped(tcg_input in_type, int64_t R, int64_t N, int64_t K, int G, const void* A, int64_t lda,
                const int32_t* offsets, const void* B, tcg_major b_major, int64_t ldb, int64_t stride_b, void* D,
                tcg_dtype d_type, int64_t ldd, cudaStream_t s) {
  begin_product();
  if (int rc = check_problem(in_type, R, N, K, G, d_type)) return rc;
  if (b_major != TCG_K_MAJOR && b_major != TCG_MN_MAJOR) return TCG_ERR_INVALID;
  if (R == 0 || N == 0) return TCG_OK;
  if (int rc = check_output(D, N, &ldd, d_type)) return rc;
  if (int rc = check_offsets(offsets)) return rc;
  const bool mn = b_major == TCG_MN_MAJOR;
  if (K > 0) {
    if (int rc = check_operand16(A, K, &lda)) return rc;
    if (int rc = check_operand16(B, mn ? N : K, &ldb)) return rc;
    if (stride_b == 0) stride_b = (mn ? K : N) * ldb;
    if (stride_b < 0) return TCG_ERR_INVALID;
    if (stride_b % 8) return TCG_ERR_ALIGNMENT;
  }
  int dev;
  if (int rc = current_device_checked(&dev)) return rc;
  const bool bf16 = in_type == TCG_IN_BF16;
  // Few rows a group stream the matrices: CTAs of 128 x 64 are then quicker
  // than pairs of 256 x 256, which win once a group takes two narrow tiles (32
  // groups of 2048 x 4096: 16 rows a group 96 us and 104, 64 103 and 106, 80
  // 133 and 108, 128 168 and 112).  Only the average is known here: 512 rows all
  // in one of the 32 groups 24 us and 27, 128 in each of four 25 and 27, but 2048
  // all in one 77 and 29.
  const bool wide = R > 64 * static_cast<int64_t>(G);
  const Variant v = wide ? pair_variant(G) : variant<1, 64, 7, MAX_GROUPS>();
  const int cg = v.ki.cta_group;
  GroupedParams p;
  std::memset(&p, 0, sizeof p);
  if (K > 0) {
    if (int rc = mn ? make_operand_map(&p.tmap_p, B, bf16, N, K, G, ldb, stride_b, 64)
                    : make_operand_map(&p.tmap_p, B, bf16, K, N, G, ldb, stride_b, 128))
      return rc;
    if (int rc = make_operand_map(&p.tmap_q, A, bf16, K, R, 0, lda, 0, static_cast<uint32_t>(v.bn / cg))) return rc;
    if (int rc = make_operand_map(&p.tmap_q16, A, bf16, K, R, 0, lda, 0, 16)) return rc;
  }
  p.offsets = offsets;
  p.G = G;
  p.R = static_cast<int>(R);
  p.p_mn = mn;
  p.M = static_cast<int>(N);
  p.K = static_cast<int>(K);
  p.m_tiles = static_cast<int>(ceil_div(N, 128 * cg));
  p.p_hi = mn ? sdesc_hi(8192, 1024, SW_128B) : sdesc_hi(16, 1024, SW_128B);
  p.p_kstep = mn ? 2048 / 16 : 32 / 16;
  p.q_hi = sdesc_hi(16, 1024, SW_128B);
  p.q_kstep = 32 / 16;
  p.idesc = idesc_f16(bf16, true, mn, false, 128 * cg, 0);
  p.D = D;
  p.ldd = ldd;
  p.d_type = d_type;
  // an upper bound of the units: a full tile per BN rows and one more per group
  const int64_t units = (R / v.bn + std::min<int64_t>(G, R)) * 2 * p.m_tiles;
  if (units > INT32_MAX / 2) return TCG_ERR_UNSUPPORTED;
  return launch_grouped(v, p, dev, units, s);
}

int run_wgrad(tcg_input in_type, int64_t R, int64_t N, int64_t K, int G, const void* DY, int64_t lddy, const void* A,
              int64_t lda, const int32_t* offsets, void* DW, tcg_dtype dw_type, int64_t lddw, int64_t stride_dw,
              cudaStream_t s) {
  begin_product();
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
  const bool bf16 = in_type == TCG_IN_BF16;
  const Variant v = pair_variant(G);
  const int cg = v.ki.cta_group;
  GroupedParams p;
  std::memset(&p, 0, sizeof p);
  if (R > 0) {
    if (int rc = make_operand_map(&p.tmap_p, A, bf16, K, R, 1, lda, R * lda, 64)) return rc;
    if (int rc = make_operand_map(&p.tmap_q, DY, bf16, N, R, 0, lddy, 0, 64)) return rc;
  }
  p.offsets = offsets;
  p.G = G;
  p.R = static_cast<int>(R);
  p.weight = 1;
  p.p_mn = 1;
  p.M = static_cast<int>(K);
  p.C = static_cast<int>(N);
  p.m_tiles = static_cast<int>(ceil_div(K, 128 * cg));
  p.p_hi = p.q_hi = sdesc_hi(8192, 1024, SW_128B);
  p.p_kstep = p.q_kstep = 2048 / 16;
  p.idesc = idesc_f16(bf16, true, true, true, 128 * cg, 0);
  p.D = DW;
  p.ldd = lddw;
  p.stride_d = stride_dw;
  p.d_type = dw_type;
  const int64_t units = static_cast<int64_t>(G) * 2 * ceil_div(N, v.bn) * p.m_tiles;
  if (units > INT32_MAX / 2) return TCG_ERR_UNSUPPORTED;
  return launch_grouped(v, p, dev, units, s);
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
