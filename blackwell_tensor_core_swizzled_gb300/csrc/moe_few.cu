// A whole mixture-of-experts layer for a few tokens in two kernels.  Entry point,
// host plan and kernels; the contract is in include/tcg.h.
//
//     y[t] = sum_e w[t, e] W2[e] (silu(W1[e] x[t]) * (W3[e] x[t]))
//
// Few tokens read each chosen expert's matrices once, so HBM bounds both
// kernels, and what counts is that reads are always in flight.  The first makes
// w h of every (expert, token) pair, the second multiplies by W2 and sums over a
// token's experts.
//
// Every CTA finds the chosen experts by itself (a token mask for each), so no
// kernel sorts.  A unit is 16 rows: of one expert's W1 and W3, or of y, whose
// CTA then passes through all experts, so that sums over experts need neither
// atomics nor memory.  Eight tokens of an expert at a time: further ones pass over
// its rows again, which then come from L2.  One warp brings the rows in stages of
// 1 KB of each (eight 128-byte slabs of 16 rows, one copy) into a ring, across units,
// another x and the scales; each of eight warps takes one slab, decodes it in
// registers and multiplies it with mma.m16n8k16, tokens on the 8 columns: the tensor
// cores are idle most of the time either way (7 to 12 % active), and tcgen05 would
// want 8-bit weights against 8-bit activations, or decoded ones in shared memory, at
// four times the bytes.
//
// Measured: 1 token x 8 of 128 experts of 4096 x 1024 E4M3, bf16, 30 us (a start of 5
// for each kernel, half of the second's hidden; 100 MB at 6.8 TB/s are 14.8); 32 tokens
// x 4 of 32 f16 experts of 4096 x 2048, 254 us, 6.2 TB/s; 8 tokens x 8 of 64 experts of
// 4096 x 1024 E4M3 104 us, 5.1 TB/s.  With more tokens an expert than eight the passes
// from L2 count: 32 x 8 of 64 such experts 202 us.
//
// The second kernel starts while the first runs (it needs half an SM): its lists
// are made and its ring is full when the first ends.
//
// h is kept as two 16-bit values, h = hi + lo, both multiplied: one value of x's
// type would add an error as large as that of rounding y (2.4e-3 instead of
// 1.7e-3 of bf16 outputs' norm).  In f16 lo is stored 2^11 times as large: as it is,
// what hi leaves of an h of less than 2^-3 would lie below f16's normal range, and of
// 2^-17 (a small weight of an ordinary activation) 2^-8 would be lost.  2^-22 of h is
// lost now, or 2^-36.
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
constexpr int MAX_TOKENS = 64;
constexpr int MAX_TOPK = 64;
constexpr int MAX_EXPERTS = 1024;
constexpr int64_t MAX_EXTENT = int64_t{1} << 29;  // rows' bytes are counted in 32 bits
constexpr int WARPS = 8;                    // that multiply; two more bring weights, and x and scales
constexpr int FEW_THREADS = 32 * (WARPS + 2);
constexpr int SLAB_BYTES = 16 * 128;
constexpr int MAX_STAGES = 6;
constexpr int MAX_SMEM = 232448;

struct FewParams {
  CUtensorMap slab[2];  // [E][128-byte slabs][rows][128]: W1 and W3, or W2
  CUtensorMap edge[2];  // [E][rows][bytes] in single slabs, for a last stage whose rows end inside a slab
  const int32_t* expert;
  const float* weight;
  int T, topk, E;
  int K, N;        // length of the weights' rows, and their number
  int row_bytes;
  int matrices, stages;
  const uint16_t* X;  // [T][K]; second kernel: hi [pairs][K]
  int64_t ldx;
  uint16_t *hi, *lo;  // [pairs][ldh]
  int64_t ldh;
  int64_t lo_at;  // lo - hi
  const float* S[2];  // 8-bit weights' scales of 128 x 128
  int64_t ld_s, stride_s;
  void* Y;
  int64_t ldy;
  int y_type;
  unsigned long long* err;
  uint64_t timeout_ns;
};

// What one pass over an expert's rows is for: up to eight of its tokens.
struct Job {
  int expert, first, tokens, block;  // first: its first pair; block: of the expert's tokens, by eights
};

// Slabs of 128 bytes of each row in a stage: one a warp, or, where h comes in two
// parts for more than eight tokens against 8-bit weights (33 KB to 16 KB of them), one
// for two warps, so that two CTAs fit an SM: 32 tokens x 8 of 64 experts of 4096 x 1024
// 202 us, 229 with whole stages (16 tokens, where two CTAs fit either way, 60 and 58;
// one token, if its few columns came so too, 31.8 and 30.3).
__host__ __device__ constexpr int slabs_a_stage(bool second, int size, bool direct) {
  return second && size == 1 && !direct ? WARPS / 2 : WARPS;
}

// Shared memory from the sizes: ring stages of weights, then of x and scales,
// then lists.
struct Layout {
  int stage;               // bytes of a stage's weights
  int x_row, x_part, x_stage;  // of x: a column, hi or lo of all columns, a stage with its scales
  int x, sums, masks, list, jobs, token, weight, bars, bytes;
  __host__ __device__ Layout(int T, int topk, int E, bool second, int size, int matrices, int stages) {
    const int pairs = T * topk, most = pairs < E ? pairs : E, slabs = slabs_a_stage(second, size, T <= 8);
    stage = SLAB_BYTES * slabs * matrices;
    x_row = 128 * slabs / size * 2 + (size == 1 ? 16 : 64);  // so that a quarter warp's words lie in different banks
    x_part = x_row * (T < 8 ? T : 8);
    x_stage = x_part * (second ? 2 : 1) + 2 * WARPS * 4;
    int at = stages * stage;
    auto take = [&](int n) {
      const int here = at;
      at += (n + 15) / 16 * 16;
      return here;
    };
    x = take(stages * x_stage);
    sums = take(second ? WARPS * T * 16 * 4 : WARPS * 2 * 8 * 17 * 4);
    masks = take(8 * E);
    list = take(4 * most);
    jobs = take(16 * (most + pairs / 8));
    token = take(pairs);
    weight = take(second ? 0 : 4 * pairs);
    bars = take(2 * MAX_STAGES * 8 + 8 * 4 + 16);
    bytes = at + 1024;  // the ring starts on a swizzle period
  }
};

// ---------------------------------------------------------------- arithmetic

template <bool BF16>
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (BF16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Four E4M3 codes as two pairs of 16-bit values, by conversion to f16; bf16 has
// none from E4M3, so values go on through fp32, whose upper halves they fit.
// (Shifting the codes' bits into place took 12 instructions, with the test for
// NaN that it needs, where this takes 8.)
template <bool BF16>
__device__ __forceinline__ void decode4(uint32_t w, uint32_t& p, uint32_t& q) {
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(p) : "h"(static_cast<uint16_t>(w)));
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(q) : "h"(static_cast<uint16_t>(w >> 16)));
  if constexpr (BF16) {
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&p));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&q));
    p = __byte_perm(__float_as_uint(a.x), __float_as_uint(a.y), 0x7632);
    q = __byte_perm(__float_as_uint(b.x), __float_as_uint(b.y), 0x7632);
  }
}


// What lo is multiplied by where it is stored.  hi leaves at most 2^-11 of itself, 2^4,
// so that lo stays within f16's range; bf16 has fp32's.
template <bool BF16>
__device__ __forceinline__ constexpr float lo_factor() { return BF16 ? 1.0f : 2048.0f; }

template <bool BF16>
__device__ __forceinline__ float to_f32(uint16_t v) {
  if constexpr (BF16)
    return __uint_as_float(static_cast<uint32_t>(v) << 16);
  else
    return __half2float(__ushort_as_half(v));
}

template <bool BF16>
__device__ __forceinline__ uint16_t round16(float v) {
  if constexpr (BF16)
    return __bfloat16_as_ushort(__float2bfloat16_rn(v));
  else
    return __half_as_ushort(__float2half_rn(v));
}

__device__ __forceinline__ float ld_shared_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr));
  return v;
}

// all but the producer of weights
__device__ __forceinline__ void consumers_sync() { asm volatile("bar.sync 2, %0;" ::"n"(32 * (WARPS + 1)) : "memory"); }
__device__ __forceinline__ void workers_sync() { asm volatile("bar.sync 1, %0;" ::"n"(32 * WARPS) : "memory"); }

// The same; true if all are.
__device__ __forceinline__ bool workers_agree(bool ok) {
  uint32_t all;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\tbar.red.and.pred q, 1, %2, p;\n\tselp.b32 %0, 1, 0, q;\n\t}"
      : "=r"(all)
      : "r"(static_cast<uint32_t>(ok)), "n"(32 * WARPS)
      : "memory");
  return all != 0;
}

// -------------------------------------------------------------------- kernels

// W8: weights are E4M3 with scales, else of x's type.  SECOND: W2 and the sum over
// experts, else W1, W3 and the activation.  DIRECT (SECOND, up to eight tokens):
// columns are tokens, whatever the expert, so that the sums stay in registers.
template <bool BF16, bool W8, bool SECOND, bool DIRECT>
__global__ void __launch_bounds__(FEW_THREADS, 2) few_kernel(const __grid_constant__ FewParams p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (sbase - raw);
  constexpr int SLABS = slabs_a_stage(SECOND, W8 ? 1 : 2, DIRECT);
  constexpr int CHUNK = 128 * SLABS;  // bytes of a row in a stage
  constexpr int TILE_BYTES = SLAB_BYTES * SLABS;
  const Layout at(p.T, p.topk, p.E, SECOND, W8 ? 1 : 2, p.matrices, p.stages);
  const int stage_bytes = at.stage, stages = p.stages;
  unsigned long long* masks = reinterpret_cast<unsigned long long*>(gbase + at.masks);
  int* list = reinterpret_cast<int*>(gbase + at.list);   // the chosen experts
  Job* job = reinterpret_cast<Job*>(gbase + at.jobs);
  uint8_t* token = gbase + at.token;                     // a pair's token
  float* weight = reinterpret_cast<float*>(gbase + at.weight);
  float* sums = reinterpret_cast<float*>(gbase + at.sums);
  const uint32_t bar0 = sbase + at.bars;
  auto full_bar = [&](uint32_t s) { return bar0 + 8u * s; };
  auto empty_bar = [&](uint32_t s) { return bar0 + 8u * (MAX_STAGES + s); };
  int* counts = reinterpret_cast<int*>(gbase + at.bars + 16 * MAX_STAGES);  // of eight ranges of experts
  volatile uint32_t* abort_flag = reinterpret_cast<uint32_t*>(gbase + at.bars + 16 * MAX_STAGES + 32);
  const WaitCtx wctx{p.timeout_ns, p.err, abort_flag};

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int pairs = p.T * p.topk;
  if (threadIdx.x == 0) {
    for (int i = 0; i < p.matrices && p.row_bytes > 0; ++i) {
      if (p.row_bytes >= 128) prefetch_tmap(&p.slab[i]);
      prefetch_tmap(&p.edge[i]);
    }
    for (int s = 0; s < stages; ++s) {
      mbar_init(full_bar(s), 1 + 32);  // the weights' bytes, the lanes' copies of x and scales
      mbar_init(empty_bar(s), WARPS);
    }
    *abort_flag = 0u;
    fence_mbarrier_init();
  }
  for (int e = threadIdx.x; e < p.E; e += FEW_THREADS) masks[e] = 0ull;
  // The first kernel waits for what is before it.  The second starts after all
  // CTAs of the first have, so that the choices and weights it reads ahead are
  // complete; only h is not.
  // (Rows of no length need no first kernel.)
  if (!SECOND || p.row_bytes == 0) griddep_wait();
  if constexpr (!SECOND) griddep_launch_dependents();
  __syncthreads();
  for (int i = threadIdx.x; i < pairs; i += FEW_THREADS) {
    const unsigned e = static_cast<unsigned>(p.expert[i]);
    if (e < static_cast<unsigned>(p.E)) atomicOr(&masks[e], 1ull << (i / p.topk));
  }
  __syncthreads();
  // the chosen experts in rising order, each of eight warps 128 of them
  unsigned votes[4];
  if (warp < 8) {
    int n = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = 128 * warp + 32 * i + lane;
      votes[i] = __ballot_sync(0xffffffffu, e < p.E && masks[e] != 0ull);
      n += __popc(votes[i]);
    }
    if (lane == 0) counts[warp] = n;
  }
  __syncthreads();
  int chosen = 0;
#pragma unroll
  for (int w = 0; w < 8; ++w) {
    if (w == warp) {
      int n = chosen;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (votes[i] >> lane & 1) list[n + __popc(votes[i] & ((1u << lane) - 1u))] = 128 * warp + 32 * i + lane;
        n += __popc(votes[i]);
      }
    }
    chosen += counts[w];
  }
  __syncthreads();
  // the pairs (experts rising, their tokens rising) and the jobs
  int* job_count = counts + 7;
  if (warp == 0) {
    int pairs_run = 0, jobs_run = 0;
    for (int a0 = 0; a0 < chosen; a0 += 32) {
      const int e = a0 + lane < chosen ? list[a0 + lane] : -1;
      const int n = e >= 0 ? __popcll(masks[e]) : 0, blocks = (n + 7) / 8;
      int pairs_to = n, jobs_to = blocks;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, pairs_to, d), q = __shfl_up_sync(0xffffffffu, jobs_to, d);
        if (lane >= d) pairs_to += o, jobs_to += q;
      }
      for (int i = 0; i < blocks; ++i)
        job[jobs_run + jobs_to - blocks + i] = {e, pairs_run + pairs_to - n + 8 * i, min(8, n - 8 * i), i};
      pairs_run += __shfl_sync(0xffffffffu, pairs_to, 31);
      jobs_run += __shfl_sync(0xffffffffu, jobs_to, 31);
    }
    __syncwarp();
    if (lane == 0) *job_count = jobs_run;
  }
  __syncthreads();
  const int jobs = *job_count;

  const int tiles = (p.N + 15) / 16;
  const int units = SECOND ? tiles : jobs * tiles;
  const int chunks = (p.row_bytes + CHUNK - 1) / CHUNK;
  const int passes = SECOND ? jobs : 1;  // over rows, of a unit
  // slabs of chunk c that exist
  auto slabs_of = [&](int c) { return min(SLABS, (p.row_bytes - c * CHUNK + 127) / 128); };

  if (warp == WARPS) {
    // --------------------------------------------------- producer of weights
    uint32_t s = 0, ph = 0, sent = 0;
    bool ok = true;
    for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
      const int n0 = (SECOND ? u : u % tiles) * 16;
      for (int i = 0; i < passes && ok; ++i) {
        const int e = job[SECOND ? i : u / tiles].expert;
        for (int c = 0; c < chunks; ++c) {
          if (!wait_inline(empty_bar(s), ph ^ 1u, wctx, SITE_PROD_EMPTY)) {
            ok = false;
            break;
          }
          if (lane == 0) {
            const uint32_t to = sbase + s * stage_bytes;
            if (p.row_bytes % 128 == 0 || c + 1 < chunks) {
              mbar_arrive_expect_tx(full_bar(s), static_cast<uint32_t>(stage_bytes));
              for (int m = 0; m < p.matrices; ++m)
                tma_load_4d(to + TILE_BYTES * m, &p.slab[m], 0, n0, c * SLABS, e, full_bar(s));
            } else {
              const int n = slabs_of(c);
              mbar_arrive_expect_tx(full_bar(s), static_cast<uint32_t>(SLAB_BYTES * n * p.matrices));
              for (int m = 0; m < p.matrices; ++m)
                for (int w = 0; w < n; ++w)
                  tma_load3<1>(to + TILE_BYTES * m + SLAB_BYTES * w, &p.edge[m], c * CHUNK + 128 * w, n0, e, full_bar(s));
            }
          }
          __syncwarp();
          ++sent;
          if (++s == static_cast<uint32_t>(stages)) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
    }
    if (!ok && lane == 0) {
      // let the copies in flight land before the CTA can exit
      const uint32_t out = min(sent, static_cast<uint32_t>(stages));
      for (uint32_t j = sent - out; j < sent; ++j) {
        const uint64_t t0 = globaltimer();
        while (!mbar_try_wait(full_bar(j % stages), (j / stages) & 1u) && globaltimer() - t0 < 20000000ull) {
        }
      }
    }
    return;
  }

  // the pairs' tokens and weights
  for (int j = warp < WARPS ? warp : jobs; j < jobs; j += WARPS) {
    const Job a = job[j];
    const unsigned long long mask = masks[a.expert];
    for (int t = lane; t < p.T; t += 32) {
      const int rank = __popcll(mask & ((1ull << t) - 1)) - 8 * a.block;
      if ((mask >> t & 1) && rank >= 0 && rank < 8) {
        token[a.first + rank] = static_cast<uint8_t>(t);
        if constexpr (!SECOND) {
          float w = 0.0f;  // a token that names an expert twice gets it with both weights
          for (int i = 0; i < p.topk; ++i)
            if (p.expert[t * p.topk + i] == a.expert) w += p.weight ? p.weight[t * p.topk + i] : 1.0f;
          weight[a.first + rank] = w;
        }
      }
    }
  }
  consumers_sync();
  constexpr int SIZE = W8 ? 1 : 2;
  constexpr int CODES = 16 / SIZE;         // weights of 16 bytes
  constexpr int WORDS = CODES / 2;         // of x against them
  constexpr int M = SECOND ? 1 : 2;
  constexpr int PARTS = SECOND ? 2 : 1;    // hi and lo
  constexpr bool LO_SCALED = SECOND && lo_factor<BF16>() != 1.0f;
  constexpr int CHAINS = LO_SCALED ? 2 : 1;          // sums of hi, and of lo as it is stored
  constexpr bool APART = W8 || DIRECT;               // a stage's sums are added to the others apart
  if constexpr (SECOND) {
    griddep_wait();
    griddep_launch_dependents();
  }
  if (warp == WARPS + 1) {
    // ------------------------------------------- producer of x and of scales:
    // a stage's x of the job's tokens and its scales come as far
    // ahead as its weights (loaded by the workers, a stage ahead or at once,
    // their latency under HBM's load was half of all time)
    uint32_t s = 0, ph = 0;
    for (int u = blockIdx.x; u < units; u += gridDim.x) {
      const int n0 = (SECOND ? u : u % tiles) * 16;
      for (int i = 0; i < passes; ++i) {
        const Job a = job[SECOND ? i : u / tiles];
        const int64_t scale_at = a.expert * p.stride_s + (n0 / BLOCK) * p.ld_s;
        // the lanes share out 1, 2, 4 or 8 tokens (one warp takes 2000 cycles a stage
        // if it passes over eight columns one by one)
        const int first = a.first, tokens = a.tokens;
        const int shift = tokens > 4 ? 2 : tokens > 2 ? 3 : tokens > 1 ? 4 : 5;  // log2 of a token's lanes
        const int index = lane >> shift, piece = lane & ((1 << shift) - 1);
        const bool exists = index < tokens;
        const int t = exists ? token[first + index] : 0;
        const uint16_t* x = (SECOND ? p.hi : p.X) + (SECOND ? first + index : t) * p.ldx;
        const uint32_t col = DIRECT ? t : index;
        for (int c = 0; c < chunks; ++c) {
          if (!wait_inline(empty_bar(s), ph ^ 1u, wctx, SITE_PROD_EMPTY)) {
            asm volatile("cp.async.wait_all;" ::: "memory");
            return;
          }
          const uint32_t to = sbase + at.x + s * at.x_stage;
          constexpr int PIECES = CHUNK / SIZE / 8;  // 16-byte words of a column
          if (exists) {
#pragma unroll
            for (int q = 0; q < PARTS; ++q)
#pragma unroll 4
              for (int v = piece; v < PIECES; v += 1 << shift) {
                const int k = c * (CHUNK / SIZE) + 8 * v;
                copy_16(to + q * at.x_part + col * at.x_row + 16u * v, x + (q ? p.lo_at : 0) + k, k < p.K ? 16 : 0);
              }
          }
          if constexpr (W8) {
            const int m = lane >> 3, slab = c * SLABS + (lane & 7);
            if (m < p.matrices && (lane & 7) < SLABS)
              copy_f32(to + PARTS * at.x_part + 4u * lane, p.S[m] + scale_at + slab, slab * 128 < p.row_bytes);
          }
          copies_arrive(full_bar(s));
          if (++s == static_cast<uint32_t>(stages)) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    return;
  }

  // ----------------------------------------------------------------- workers
  const int g = lane >> 2, c4 = lane & 3;
  constexpr int SHARE = WARPS / SLABS;  // warps of a slab, each half of its rows' bytes
  const int mine = warp / SHARE;        // this warp's slab
  uint32_t s = 0, ph = 0;
  float acc[CHAINS][M][4];
  bool ok = true;
  // This warp's share of a job: adds to acc.
  auto multiply = [&](const Job& a) {
    // DIRECT: which of this lane's sums (columns 2 c4, + 1) belong to the expert's
    // tokens; the others' columns hold anything
    const uint32_t columns = DIRECT ? 5u * (static_cast<uint32_t>(masks[a.expert]) >> (2 * c4) & 3u) : 15u;
    for (int c = 0; c < chunks; ++c) {
      if (!wait_inline(full_bar(s), ph, wctx, SITE_MMA_FULL)) {
        ok = false;
        return;
      }
      if (c * CHUNK + 128 * mine < p.row_bytes) {
        const uint32_t xs = sbase + at.x + s * at.x_stage;
        float sc[M];
        if constexpr (W8) {
#pragma unroll
          for (int m = 0; m < M; ++m) sc[m] = ld_shared_f32(xs + PARTS * at.x_part + 32u * m + 4u * mine);
        }
#pragma unroll
        for (int i = 0; i < 2 / SHARE; ++i) {
          const int h = SHARE == 1 ? i : warp & 1;
          const int k = mine * (128 / SIZE) + CODES * (c4 + 4 * h);  // of the stage
          uint4 x[PARTS][WORDS / 4];
#pragma unroll
          for (int q = 0; q < PARTS; ++q)
#pragma unroll
            for (int v = 0; v < WORDS / 4; ++v)
              x[q][v] = ld_shared_v4(xs + q * at.x_part + min(g, p.T - 1) * at.x_row + 2u * k + 16u * v);
          uint32_t A[M][CODES / 4][4];  // fragments of this lane's 16-byte chunk of rows g and g + 8
#pragma unroll
          for (int m = 0; m < M; ++m) {
            if (m >= p.matrices) break;
            const uint32_t slab = sbase + s * stage_bytes + TILE_BYTES * m + SLAB_BYTES * mine;
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const uint4 v = ld_shared_v4(slab + 128u * (g + 8 * r) + 16u * ((c4 + 4 * h) ^ g));
              const uint32_t w[4] = {v.x, v.y, v.z, v.w};
              if constexpr (W8) {
#pragma unroll
                for (int i = 0; i < 4; ++i) decode4<BF16>(w[i], A[m][i][r], A[m][i][2 + r]);
              } else {
#pragma unroll
                for (int i = 0; i < 2; ++i) A[m][i][r] = w[2 * i], A[m][i][2 + r] = w[2 * i + 1];
              }
            }
          }
          float part[CHAINS][M][4] = {};
#pragma unroll
          for (int q = 0; q < PARTS; ++q) {
            const uint32_t* w = reinterpret_cast<const uint32_t*>(&x[q][0]);
#pragma unroll
            for (int i = 0; i < CODES / 4; ++i) {
#pragma unroll
              for (int m = 0; m < M; ++m)
                if (m < p.matrices) mma_16816<BF16>(APART ? part[q % CHAINS][m] : acc[q % CHAINS][m], A[m][i], w[2 * i], w[2 * i + 1]);
            }
          }
          if constexpr (APART) {
#pragma unroll
            for (int m = 0; m < M; ++m)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                float& to = acc[0][m][i];
                const float v = LO_SCALED ? fmaf(part[CHAINS - 1][m][i], 1.0f / lo_factor<BF16>(), part[0][m][i]) : part[0][m][i];
                if (!DIRECT || (columns >> i & 1)) to = W8 ? fmaf(v, sc[m], to) : to + v;
              }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty_bar(s));
      if (++s == static_cast<uint32_t>(stages)) {
        s = 0;
        ph ^= 1u;
      }
    }
  };
  auto clear = [&] {
#pragma unroll
    for (int j = 0; j < CHAINS; ++j)
#pragma unroll
      for (int m = 0; m < M; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[j][m][i] = 0.0f;
  };
  // W2's sum i of this lane
  auto sum_of = [&](int i) {
    return LO_SCALED && !APART ? fmaf(acc[CHAINS - 1][0][i], 1.0f / lo_factor<BF16>(), acc[0][0][i]) : acc[0][0][i];
  };

  if constexpr (!SECOND) {
    for (int u = blockIdx.x; u < units; u += gridDim.x) {
      const Job a = job[u / tiles];
      const int n0 = (u % tiles) * 16;
      clear();
      multiply(a);
      if (!workers_agree(ok)) return;
      // [warp][matrix][column][row]
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) sums[((warp * 2 + m) * 8 + 2 * c4 + (i & 1)) * 17 + g + 8 * (i >> 1)] = acc[0][m][i];
      workers_sync();
      const int row = threadIdx.x & 15, col = threadIdx.x >> 4;
      if (col < a.tokens && n0 + row < p.N) {
        float v[2] = {};
#pragma unroll
        for (int w = 0; w < WARPS; ++w)
#pragma unroll
          for (int m = 0; m < 2; ++m) v[m] += sums[((w * 2 + m) * 8 + col) * 17 + row];
        const int pair = a.first + col;
        const float silu = v[0] / (1.0f + expf(-v[0]));
        const float h = (p.matrices > 1 ? silu * v[1] : silu) * weight[pair];
        const uint16_t hi = round16<BF16>(h);
        const float rest = h - to_f32<BF16>(hi);
        const int64_t to = pair * p.ldh + n0 + row;
        p.hi[to] = hi;
        p.lo[to] = isfinite(rest) ? round16<BF16>(rest * lo_factor<BF16>()) : static_cast<uint16_t>(0);
      }
      workers_sync();
    }
  } else {
    float* own = sums + warp * p.T * 16;
    for (int u = blockIdx.x; u < units; u += gridDim.x) {
      const int n0 = u * 16;
      clear();
      if constexpr (DIRECT) {
        for (int j = 0; j < jobs && ok; ++j) multiply(job[j]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int t = 2 * c4 + (i & 1);
          if (t < p.T) own[t * 16 + g + 8 * (i >> 1)] = sum_of(i);
        }
      } else {
        for (int i = lane; i < p.T * 16; i += 32) own[i] = 0.0f;
        __syncwarp();
        for (int j = 0; j < jobs && ok; ++j) {
          const Job a = job[j];
          multiply(a);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int col = 2 * c4 + (i & 1);
            if (col < a.tokens) own[token[a.first + col] * 16 + g + 8 * (i >> 1)] += sum_of(i);
          }
          clear();
          __syncwarp();
        }
      }
      if (!workers_agree(ok)) return;
      for (int i = threadIdx.x; i < p.T * 16; i += 32 * WARPS) {
        const int t = i >> 4, n = n0 + (i & 15);
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) v += sums[w * p.T * 16 + i];
        if (n < p.N) {
          const int64_t to = t * p.ldy + n;
          if (p.y_type == OUT_F32)
            static_cast<float*>(p.Y)[to] = v;
          else
            static_cast<uint16_t*>(p.Y)[to] = p.y_type == OUT_BF16 ? round16<true>(v) : round16<false>(v);
        }
      }
      workers_sync();
    }
  }
}

// ----------------------------------------------------------------------- host

using Kernel = void (*)(const FewParams);
OncePerDevice<cudaError_t> g_setup;

template <bool BF16, bool W8>
Kernel pick(bool second, int T) {
  return !second ? few_kernel<BF16, W8, false, false>
         : T <= 8 ? few_kernel<BF16, W8, true, true>
                  : few_kernel<BF16, W8, true, false>;
}

Kernel pick(bool second, bool bf16, bool w8, int T) {
  if (bf16) return w8 ? pick<true, true>(second, T) : pick<true, false>(second, T);
  return w8 ? pick<false, true>(second, T) : pick<false, false>(second, T);
}

cudaError_t setup(int dev) {
  return g_setup(dev, [] {
    for (int i = 0; i < 4; ++i)
      for (Kernel k : {pick(false, i & 1, i & 2, 1), pick(true, i & 1, i & 2, 1), pick(true, i & 1, i & 2, MAX_TOKENS)}) {
        const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, MAX_SMEM);
        if (e != cudaSuccess) return e;
      }
    return cudaSuccess;
  });
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
bool misaligned(const void* p, unsigned n) { return reinterpret_cast<uintptr_t>(p) % n != 0; }

int launch(Kernel kernel, const FewParams& p, int64_t grid, int smem, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
  cfg.blockDim = dim3(FEW_THREADS, 1, 1);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return record_cuda(cudaLaunchKernelEx(&cfg, kernel, p));
}

// Maps of one matrix of each expert: `rows` rows of `bytes`, `ld` bytes apart.
int weight_maps(FewParams* p, int i, const void* W, int64_t bytes, int64_t rows, int64_t ld, int64_t stride,
                int slabs) {
  if (bytes >= 128)
    if (int rc = make_slab_map(&p->slab[i], W, 128, rows, bytes / 128, p->E, ld, stride, 16, slabs)) return rc;
  return make_byte_map(&p->edge[i], W, bytes, rows, p->E, ld, stride, 128, 16);
}

// Weights [E][rows][length] of `size` bytes: whole 16-byte words
int check_weights(const void* W, int64_t rows, int64_t length, int size, int64_t* ld, int64_t* stride) {
  if (*ld == 0) *ld = length;
  if (*stride == 0) *stride = rows * *ld;
  if (!W || *ld < length || *stride < 0) return TCG_ERR_INVALID;
  return misaligned(W, 16) || *ld * size % 16 || *stride * size % 16 || length * size % 16 ? TCG_ERR_ALIGNMENT : TCG_OK;
}

int check_scales(const float* S, int64_t rows, int64_t length, int64_t* ld, int64_t* stride) {
  if (*ld == 0) *ld = ceil_div(length, BLOCK);
  if (*stride == 0) *stride = ceil_div(rows, BLOCK) * *ld;
  if (!S || *ld < ceil_div(length, BLOCK) || *stride < 0) return TCG_ERR_INVALID;
  return misaligned(S, 4) ? TCG_ERR_ALIGNMENT : TCG_OK;
}

// How a kernel runs: ring stages, shared memory and CTAs an SM.
struct Shape {
  int stages, smem, ctas;
};

// Two CTAs share an SM where half its memory holds 24 KB of weights and more: twice
// the warps hide their latencies (1 token x 8 of 128 experts of 4096 x 1024, E4M3:
// 30 us, 43 with one; 32 tokens x 4 of 32 f16 experts of 4096 x 2048 18 % less than
// with one).
// Else one has what fits.
Shape shape(int T, int topk, int E, bool second, int size, int matrices) {
  const auto at = [&](int n) { return Layout(T, topk, E, second, size, matrices, n); };
  for (int n = MAX_STAGES / matrices; n * at(n).stage >= 24 << 10; --n)
    if (at(n).bytes <= MAX_SMEM / 2 - 1024) return {n, at(n).bytes, 2};
  for (int n = MAX_STAGES / matrices;; --n)  // one stage fits whatever the lists (140 KB at most)
    if (at(n).bytes <= MAX_SMEM) return {n, at(n).bytes, 1};
}

int64_t work_bytes(int64_t T, int topk, int64_t I) {
  if (T < 0 || T > MAX_TOKENS || topk < 1 || topk > MAX_TOPK || I < 0 || I >= MAX_EXTENT) return -1;
  return 4 * T * topk * I;
}

int run_few(const tcg_moe_few_args* args, cudaStream_t s) {
  begin_product();
  if (!args) return TCG_ERR_INVALID;
  tcg_moe_few_args a = *args;
  if (a.x_type != TCG_IN_F16 && a.x_type != TCG_IN_BF16) return TCG_ERR_INVALID;
  if (a.w_type != a.x_type && a.w_type != TCG_IN_E4M3) return TCG_ERR_INVALID;
  if (a.T < 0 || a.H < 0 || a.I < 0 || a.topk < 1 || a.E < 1 || a.y_type < TCG_F32 || a.y_type > TCG_BF16)
    return TCG_ERR_INVALID;
  if (a.T > MAX_TOKENS || a.topk > MAX_TOPK || a.E > MAX_EXPERTS || a.H >= MAX_EXTENT || a.I >= MAX_EXTENT)
    return TCG_ERR_UNSUPPORTED;
  if (a.T == 0 || a.H == 0) return TCG_OK;
  const bool w8 = a.w_type == TCG_IN_E4M3;
  const int size = w8 ? 1 : 2;
  if (a.ldy == 0) a.ldy = a.H;
  if (!a.Y || a.ldy < a.H || !a.expert) return TCG_ERR_INVALID;
  if (misaligned(a.Y, a.y_type == TCG_F32 ? 4 : 2) || misaligned(a.expert, 4) || misaligned(a.weight, 4))
    return TCG_ERR_ALIGNMENT;
  if (a.I > 0) {
    if (a.ldx == 0) a.ldx = a.H;
    if (!a.X || a.ldx < a.H || !a.work) return TCG_ERR_INVALID;
    if (misaligned(a.X, 16) || a.ldx % 8 || misaligned(a.work, 16)) return TCG_ERR_ALIGNMENT;
    int64_t ld = a.ld1, stride = a.stride1;
    if (int rc = check_weights(a.W1, a.I, a.H, size, &ld, &stride)) return rc;
    if (a.W3 && misaligned(a.W3, 16)) return TCG_ERR_ALIGNMENT;
    a.ld1 = ld, a.stride1 = stride;
    if (int rc = check_weights(a.W2, a.H, a.I, size, &a.ld2, &a.stride2)) return rc;
    if (w8) {
      if (int rc = check_scales(a.S1, a.I, a.H, &a.ld_s1, &a.stride_s1)) return rc;
      if (a.W3 && !a.S3) return TCG_ERR_INVALID;
      if (misaligned(a.S3, 4)) return TCG_ERR_ALIGNMENT;
      if (int rc = check_scales(a.S2, a.H, a.I, &a.ld_s2, &a.stride_s2)) return rc;
    }
  }
  int dev;
  if (int rc = current_device_checked(&dev)) return rc;
  if (int rc = record_cuda(setup(dev))) return rc;
  const bool bf16 = a.x_type == TCG_IN_BF16;
  const int T = static_cast<int>(a.T), sms = device_sms(dev);
  const int64_t pairs = a.T * a.topk;
  FewParams p;
  std::memset(&p, 0, sizeof p);
  p.expert = a.expert;
  p.weight = a.weight;
  p.T = T;
  p.topk = a.topk;
  p.E = a.E;
  p.hi = static_cast<uint16_t*>(a.work);
  p.lo = p.hi + pairs * a.I;
  p.ldh = a.I;
  p.lo_at = pairs * a.I;
  p.err = device_error_word(dev);
  p.timeout_ns = wait_timeout_ns();
  FewParams q = p;
  int launches = 0;
  if (a.I > 0) {
    p.K = static_cast<int>(a.H);
    p.N = static_cast<int>(a.I);
    p.row_bytes = p.K * size;
    p.matrices = a.W3 ? 2 : 1;
    if (int rc = weight_maps(&p, 0, a.W1, p.row_bytes, a.I, a.ld1 * size, a.stride1 * size, WARPS)) return rc;
    if (a.W3)
      if (int rc = weight_maps(&p, 1, a.W3, p.row_bytes, a.I, a.ld1 * size, a.stride1 * size, WARPS)) return rc;
    p.X = static_cast<const uint16_t*>(a.X);
    p.ldx = a.ldx;
    p.S[0] = a.S1;
    p.S[1] = a.S3;
    p.ld_s = a.ld_s1;
    p.stride_s = a.stride_s1;
    if (int rc = weight_maps(&q, 0, a.W2, a.I * size, a.H, a.ld2 * size, a.stride2 * size, slabs_a_stage(true, size, T <= 8)))
      return rc;
    const int64_t units = std::min<int64_t>(a.E + pairs / 8, pairs) * ceil_div(a.I, 16);
    if (units > INT32_MAX) return TCG_ERR_UNSUPPORTED;
    const Shape h = shape(T, a.topk, a.E, false, size, p.matrices);
    p.stages = h.stages;
    if (int rc = launch(pick(false, bf16, w8, T), p, std::min<int64_t>(units, h.ctas * sms), h.smem, s)) return rc;
    ++launches;
  }
  q.K = static_cast<int>(a.I);
  q.N = static_cast<int>(a.H);
  q.row_bytes = q.K * size;
  q.matrices = 1;
  const Shape h = shape(T, a.topk, a.E, true, size, 1);
  q.stages = h.stages;
  q.ldx = q.ldh;
  q.S[0] = a.S2;
  q.ld_s = a.ld_s2;
  q.stride_s = a.stride_s2;
  q.Y = a.Y;
  q.ldy = a.ldy;
  q.y_type = a.y_type;
  if (int rc = launch(pick(true, bf16, w8, T), q, std::min<int64_t>(ceil_div(a.H, 16), h.ctas * sms), h.smem, s)) return rc;
  set_launch_count(launches + 1);
  return TCG_OK;
}

}  // namespace

}  // namespace tcg

using namespace tcg;

extern "C" {

int64_t tcg_moe_few_work_bytes(int64_t T, int topk, int64_t I) { return work_bytes(T, topk, I); }

int tcg_moe_few(const tcg_moe_few_args* args, void* stream) {
  return guarded([&] { return run_few(args, static_cast<cudaStream_t>(stream)); });
}

}  // extern "C"
