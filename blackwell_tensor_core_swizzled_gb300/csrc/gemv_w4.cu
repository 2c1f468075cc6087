// Few rows of 16-bit activations against 4-bit matrices with group scales.
// Entry point, host plan and kernel; the contract is in include/tcg.h.
//
// The work is to stream the codes: N K / 2 bytes a matrix against a few rows.
// Codes are decoded to f16 in registers (every E2M1 value, and code - zero of
// INT4, is exact there) and multiplied by mma m16n8k16 with fp32
// accumulation: 16 matrix rows by 8 activation rows, so that up to 8 rows cost
// the decoding once.  (A 64 x 64-bit product on tcgen05 would take the decoded
// codes through shared or tensor memory first; the register path has no such
// stop, and at 8 rows the mma rate is a third of what HBM can feed.)  A
// group's sum is multiplied by its scale in fp32: the scale meets sums, not
// weights, which keeps every product exact.
//
// A warp owns a slab of 256 of K for KSL slabs and walks down the matrix in
// tiles of 16 rows; its activations stay in registers for all of them.  A
// team of warps covers K (across a cluster of CTAs when the slabs are more
// than a CTA's warps), adds its warps' sums in a fixed order through shared
// memory, and takes an equal share of the tiles.  Tiles arrive by cp.async
// into a ring private to the warp: no barrier stands between load and use.
//
// bf16 activations are brought into f16's range by a power of two per row and
// slab (the largest finite value to [2^14, 2^15)), undone on each group's fp32
// sum before its scale (the other order could overflow on the way): exact for values down to 2^-29 of the slab's largest; smaller ones
// round at 2^-39 of it, below the fp32 sums' own rounding of that largest
// value's product.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstring>
#include <mutex>

#include "common.h"
#include "ptx.cuh"

namespace tcg {

namespace {

constexpr int MAX_GROUPS = 1024;
constexpr int64_t MAX_EXTENT = int64_t{1} << 30;

constexpr int WARPS = 16;
constexpr int THREADS = 32 * WARPS;
constexpr int SLAB = 256;          // K per warp and tile: 128 bytes of codes
constexpr int TILE_N = 16;         // matrix rows per tile
constexpr int STAGES = 4;          // ring stages per warp
constexpr int CODE_BYTES = TILE_N * SLAB / 2;
constexpr int SCALE_PITCH = 20;    // bytes: up to 16 of scales, from a 4-byte boundary
constexpr int ZERO_PITCH = 12;     // up to 8 of zero points
constexpr int STAGE_BYTES = CODE_BYTES + TILE_N * (SCALE_PITCH + ZERO_PITCH);
constexpr int PART_PITCH = 20;     // floats between activation rows of a partial tile
constexpr int ROUND = 16;          // units a cluster sums before its CTAs meet

struct GemvParams {
  int R, N, K, G;
  int group_shift;   // log2 of K per scale
  const uint8_t* A;  // 16-bit elements
  int64_t lda;
  const int32_t* offsets;
  const uint8_t* B;
  int64_t ldb, stride_b;  // bytes
  const uint8_t* scale;
  int64_t ld_scale, stride_scale, scale_bytes;  // bytes; size of the array
  const uint8_t* zero;
  int64_t ld_zero, stride_zero, zero_bytes;
  int scale_words, zero_words;  // 4-byte words that hold a row's slab of scales, zero points
  const float* alpha;
  void* D;
  int d_type;
  int64_t ldd;
  int tiles;        // 16-row tiles of a matrix
  int slabs;        // ceil(K / 256)
  int team_warps;   // warps of a team in one CTA
  int teams;        // teams in a CTA
};

template <int NT>
struct GemvSmem {
  static constexpr int RING = WARPS * STAGES * STAGE_BYTES;
  static constexpr int PART = 2 * WARPS * 8 * NT * PART_PITCH * 4;  // two tiles of every warp
  static constexpr int SUM = ROUND * 8 * NT * 16 * 4;               // a cluster CTA's sums of a round
  static constexpr int SEG = 2 * (MAX_GROUPS + 1) * 4;
  static constexpr int BYTES = RING + PART + SUM + SEG;
  static_assert(BYTES <= 232448, "dynamic shared memory");
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds8(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// the eight E2M1 codes of a word as four f16 pairs, in order
__device__ __forceinline__ void e2m1_word(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}
__device__ __forceinline__ void e2m1_half(uint32_t w, uint32_t (&h)[2]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t}"
      : "=r"(h[0]), "=r"(h[1])
      : "r"(w));
}
__device__ __forceinline__ uint32_t hsub2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}

// The eight unsigned codes of a word minus the zero point, as f16 pairs
// (0,4) (1,5) (2,6) (3,7).  A code in the low bits of a half under the
// exponent of 1024 is 1024 + code; four bits higher it is 1024 + 16 code,
// which fma brings back: (1024 + 16 code) / 16 - (64 + zero), exact.  z1024
// holds 1024 + zero twice.
__device__ __forceinline__ void int4_word(uint32_t w, uint32_t z1024, uint32_t (&h)[4]) {
  constexpr uint32_t K1024 = 0x64006400u, SIXTEENTH = 0x2C002C00u, K960 = 0x63806380u;
  const uint32_t w8 = w >> 8;
  const uint32_t nz = hsub2(K960, z1024);  // -(64 + zero)
  h[0] = hsub2((w & 0x000F000Fu) | K1024, z1024);
  h[1] = hfma2((w & 0x00F000F0u) | K1024, SIXTEENTH, nz);
  h[2] = hsub2((w8 & 0x000F000Fu) | K1024, z1024);
  h[3] = hfma2((w8 & 0x00F000F0u) | K1024, SIXTEENTH, nz);
}

__device__ __forceinline__ float half_bits(uint32_t h) { return __half2float(__ushort_as_half(static_cast<uint16_t>(h))); }

// Barrier of a team's warps in a CTA (two warps or more: at most 8 teams)
__device__ __forceinline__ void team_sync(int team, int warps) {
  if (warps == 1)
    __syncwarp();
  else
    asm volatile("barrier.sync %0, %1;" ::"r"(team + 1), "r"(32 * warps) : "memory");
}

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr));
  return v;
}

__device__ __forceinline__ void store_d(const GemvParams& p, int64_t i, float v) {
  if (p.d_type == TCG_F32)
    static_cast<float*>(p.D)[i] = v;
  else if (p.d_type == TCG_F16)
    static_cast<__half*>(p.D)[i] = __float2half_rn(v);
  else
    static_cast<__nv_bfloat16*>(p.D)[i] = __float2bfloat16_rn(v);
}

// A row block: up to 8 * NT rows of one group.
struct RowBlock {
  int g, row0, rows;
};

template <int NT>
__device__ __forceinline__ RowBlock row_block(const GemvParams& p, const int* seg, const int* pre, int rb) {
  constexpr int ROWS = 8 * NT;
  if (!p.offsets) return {0, rb * ROWS, min(ROWS, p.R - rb * ROWS)};
  int a = 0, b = p.G;  // pre[a] <= rb < pre[b]
  while (b - a > 1) {
    const int mid = (a + b) >> 1;
    if (pre[mid] <= rb)
      a = mid;
    else
      b = mid;
  }
  const int row0 = seg[a] + (rb - pre[a]) * ROWS;
  return {a, row0, min(ROWS, seg[a + 1] - row0)};
}

// The activations of a row block for one slab as B fragments.  Lane (g, c) =
// (lane / 4, lane % 4) holds row 8 nt + g; `frag[ch][nt]` covers 32 of K in
// the order in which the codes' words decode.  Returns (bf16) the factors that
// undo the scaling for the accumulator's columns 2c and 2c + 1.
template <int FMT, bool BF16, int NT>
__device__ __forceinline__ void load_fragments(const GemvParams& p, const RowBlock& rb, int slab, int lane,
                                               uint32_t (&frag)[8][NT][4], float (&undo)[NT][2]) {
  const int g = lane >> 2, c = lane & 3;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int r = 8 * nt + g;
    const uint8_t* row = p.A + 2 * (static_cast<int64_t>(rb.row0 + r) * p.lda + slab * SLAB);
    uint32_t v[8][4];
#pragma unroll
    for (int ch = 0; ch < 8; ++ch) {
      const bool in = r < rb.rows && slab * SLAB + 32 * ch < p.K;
      if (FMT == TCG_W4_NVF4) {  // 4 of each group of 16
        uint2 x = make_uint2(0u, 0u), y = x;
        if (in) {
          x = *reinterpret_cast<const uint2*>(row + 64 * ch + 8 * c);
          y = *reinterpret_cast<const uint2*>(row + 64 * ch + 32 + 8 * c);
        }
        v[ch][0] = x.x;
        v[ch][1] = x.y;
        v[ch][2] = y.x;
        v[ch][3] = y.y;
      } else {  // 8 consecutive
        uint4 x = make_uint4(0u, 0u, 0u, 0u);
        if (in) x = *reinterpret_cast<const uint4*>(row + 64 * ch + 16 * c);
        v[ch][0] = x.x;
        v[ch][1] = x.y;
        v[ch][2] = x.z;
        v[ch][3] = x.w;
      }
    }
    if (BF16) {
      // the largest magnitude of the row's slab; max drops NaN, and infinities
      // are looked past when there are any
      uint32_t m2 = 0;
#pragma unroll
      for (int ch = 0; ch < 8; ++ch)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          asm("max.bf16x2 %0, %0, %1;" : "+r"(m2) : "r"(v[ch][i] & 0x7FFF7FFFu));
      uint32_t m = max(m2 & 0xFFFFu, m2 >> 16);
      if (m >= 0x7F80u) {
        m = 0;
#pragma unroll
        for (int ch = 0; ch < 8; ++ch)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t lo = v[ch][i] & 0x7FFFu, hi = (v[ch][i] >> 16) & 0x7FFFu;
            if (lo < 0x7F80u) m = max(m, lo);
            if (hi < 0x7F80u) m = max(m, hi);
          }
      }
      m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
      const int e = 141 - static_cast<int>(m >> 7);  // 2^e brings the largest to [2^14, 2^15)
      const int s = min(e, 126);
      const float up = __uint_as_float(static_cast<uint32_t>(s + 127) << 23);
      const float down = __uint_as_float(static_cast<uint32_t>(127 - s) << 23);
#pragma unroll
      for (int ch = 0; ch < 8; ++ch)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const __half2 h = __floats2half2_rn(__uint_as_float(v[ch][i] << 16) * up,
                                              __uint_as_float(v[ch][i] & 0xFFFF0000u) * up);
          v[ch][i] = *reinterpret_cast<const uint32_t*>(&h);
        }
      // the factors of rows 2c and 2c + 1, held by the lanes of those rows
      undo[nt][0] = __shfl_sync(0xffffffffu, down, 8 * c);
      undo[nt][1] = __shfl_sync(0xffffffffu, down, 8 * c + 4);
    }
#pragma unroll
    for (int ch = 0; ch < 8; ++ch) {
      if (FMT == TCG_W4_INT4) {  // pairs (0,4) (1,5) (2,6) (3,7)
        frag[ch][nt][0] = __byte_perm(v[ch][0], v[ch][2], 0x5410);
        frag[ch][nt][1] = __byte_perm(v[ch][0], v[ch][2], 0x7632);
        frag[ch][nt][2] = __byte_perm(v[ch][1], v[ch][3], 0x5410);
        frag[ch][nt][3] = __byte_perm(v[ch][1], v[ch][3], 0x7632);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) frag[ch][nt][i] = v[ch][i];
      }
    }
  }
}

// One tile's slab: acc[nt] += (codes . activations) * scales; `stage` is its
// ring stage, ms / mz the byte offsets of rows g and g + 8's scales and zero
// points from their 4-byte boundary.
template <int FMT, bool BF16, int NT>
__device__ __forceinline__ void tile_slab(const GemvParams& p, uint32_t stage, int lane, int chunks, uint32_t ms0,
                                          uint32_t ms1, uint32_t mz0, uint32_t mz1, const uint32_t (&frag)[8][NT][4],
                                          const float (&undo)[NT][2], float (&acc)[NT][4]) {
  auto add = [&](int nt, const float (&part)[4], float f0, float f1) {
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[nt][i] += (BF16 ? part[i] * undo[nt][i & 1] : part[i]) * (i < 2 ? f0 : f1);
  };
  const uint32_t g = lane >> 2, c = lane & 3;
  const uint32_t code0 = stage + 128u * g, code1 = code0 + 1024u;
  const uint32_t sc0 = stage + CODE_BYTES + SCALE_PITCH * g + ms0, sc1 = stage + CODE_BYTES + SCALE_PITCH * (g + 8) + ms1;
  uint32_t b0[4], b1[4];  // scale bytes of rows g and g + 8
  if (FMT != TCG_W4_INT4) {
    constexpr int W = FMT == TCG_W4_MXF4 ? 2 : 4;
    const uint32_t a0 = sc0 - ms0, a1 = sc1 - ms1;
    uint32_t lo0 = lds32(a0), lo1 = lds32(a1);
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const uint32_t hi0 = lds32(a0 + 4 * i + 4), hi1 = lds32(a1 + 4 * i + 4);
      b0[i] = __funnelshift_r(lo0, hi0, 8 * ms0);
      b1[i] = __funnelshift_r(lo1, hi1, 8 * ms1);
      lo0 = hi0;
      lo1 = hi1;
    }
    if (FMT == TCG_W4_NVF4) {
      // unsigned E4M3: a byte with the top bit set is NaN (0xFF)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t t0 = b0[i] & 0x80808080u, t1 = b1[i] & 0x80808080u;
        b0[i] |= t0 - (t0 >> 7);
        b1[i] |= t1 - (t1 >> 7);
      }
    }
  }
#pragma unroll
  for (int ch = 0; ch < 8; ++ch) {
    if (ch >= chunks) break;
    const uint32_t at = ((ch ^ g) & 7u) * 16u;
    if (FMT == TCG_W4_NVF4) {
      // scales 2 ch and 2 ch + 1 of both rows
      uint32_t s0, s1;
      const uint32_t w0 = b0[ch / 2] >> (16 * (ch & 1)), w1 = b1[ch / 2] >> (16 * (ch & 1));
      asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(s0) : "r"(w0));
      asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(s1) : "r"(w1));
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        uint32_t h0[2], h1[2];
        e2m1_half(lds16(code0 + at + 8 * q + 2 * c), h0);
        e2m1_half(lds16(code1 + at + 8 * q + 2 * c), h1);
        const float f0 = half_bits(q ? s0 >> 16 : s0), f1 = half_bits(q ? s1 >> 16 : s1);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float part[4] = {};
          mma16816(part, h0[0], h1[0], h0[1], h1[1], frag[ch][nt][2 * q], frag[ch][nt][2 * q + 1]);
          add(nt, part, f0, f1);
        }
      }
    } else {
      uint32_t h0[4], h1[4];
      float f0, f1;
      const uint32_t w0 = lds32(code0 + at + 4 * c), w1 = lds32(code1 + at + 4 * c);
      if (FMT == TCG_W4_MXF4) {
        e2m1_word(w0, h0);
        e2m1_word(w1, h1);
        // both rows' e8m0 bytes to bf16 pairs, exact (0 is 2^-127, 255 NaN)
        const uint32_t pair = __byte_perm(b0[ch / 4], b1[ch / 4], (ch & 3) | ((4 + (ch & 3)) << 4));
        uint32_t s;
        asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.bf16x2.ue8m0x2 %0, lo;\n\t}" : "=r"(s) : "r"(pair));
        f0 = __uint_as_float(s << 16);
        f1 = __uint_as_float(s & 0xFFFF0000u);
      } else {
        const uint32_t gi = static_cast<uint32_t>(32 * ch) >> p.group_shift;
        const uint32_t s0 = lds16(sc0 + 2 * gi), s1 = lds16(sc1 + 2 * gi);
        f0 = BF16 ? __uint_as_float(s0 << 16) : half_bits(s0);
        f1 = BF16 ? __uint_as_float(s1 << 16) : half_bits(s1);
        uint32_t z0 = 8, z1 = 8;
        if (p.zero) {
          const uint32_t zb = stage + CODE_BYTES + TILE_N * SCALE_PITCH + gi;
          z0 = lds8(zb + ZERO_PITCH * g + mz0);
          z1 = lds8(zb + ZERO_PITCH * (g + 8) + mz1);
        }
        int4_word(w0, 0x64006400u + z0 * 0x10001u, h0);
        int4_word(w1, 0x64006400u + z1 * 0x10001u, h1);
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float part[4] = {};
        mma16816(part, h0[0], h1[0], h0[1], h1[1], frag[ch][nt][0], frag[ch][nt][1]);
        mma16816(part, h0[2], h1[2], h0[3], h1[3], frag[ch][nt][2], frag[ch][nt][3]);
        add(nt, part, f0, f1);
      }
    }
  }
}

template <int FMT, bool BF16, int NT, int KSL>
__global__ void __launch_bounds__(THREADS, 1) gemv_kernel(const __grid_constant__ GemvParams p) {
  using S = GemvSmem<NT>;
  extern __shared__ __align__(16) uint8_t smem[];
  float* part = reinterpret_cast<float*>(smem + S::RING);
  float* sums = reinterpret_cast<float*>(smem + S::RING + S::PART);
  int* seg = reinterpret_cast<int*>(smem + S::RING + S::PART + S::SUM);
  int* pre = seg + p.G + 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;
  uint32_t cluster_size;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(cluster_size));
  const int rank = static_cast<int>(cluster_ctarank());
  const int team = warp / p.team_warps, wk = warp - team * p.team_warps;
  const bool idle = team >= p.teams;  // warps left over when teams do not fill the CTA
  const int num_teams = static_cast<int>(gridDim.x / cluster_size) * p.teams;
  // neighbouring teams sit in different CTAs, so that few tiles spread over all
  // (a cluster has one team; its CTAs' spare warps follow it to the cluster's barriers)
  const int team_id = (cluster_size > 1 ? 0 : team) * static_cast<int>(gridDim.x / cluster_size) +
                      static_cast<int>(blockIdx.x / cluster_size);

  griddep_wait();
  griddep_launch_dependents();
  int blocks;
  if (p.offsets) {
    constexpr int ROWS = 8 * NT;
    for (int i = threadIdx.x; i <= p.G; i += THREADS) seg[i] = p.offsets[i];
    __syncthreads();
    if (warp == 0) {  // clamp to [previous, R]; row blocks before each group
      int run_max = 0, run_blocks = 0;
      for (int i0 = 0; i0 <= p.G; i0 += 32) {
        const int i = i0 + lane;
        int v = i <= p.G ? min(max(seg[i], 0), p.R) : 0;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int o = __shfl_up_sync(0xffffffffu, v, d);
          if (lane >= d) v = max(v, o);
        }
        v = max(v, run_max);
        int before = __shfl_up_sync(0xffffffffu, v, 1);
        if (lane == 0) before = run_max;
        int n = i >= 1 && i <= p.G ? (v - before + ROWS - 1) / ROWS : 0;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int o = __shfl_up_sync(0xffffffffu, n, d);
          if (lane >= d) n += o;
        }
        n += run_blocks;
        if (i <= p.G) {
          seg[i] = v;
          pre[i] = n;
        }
        run_max = __shfl_sync(0xffffffffu, v, 31);
        run_blocks = __shfl_sync(0xffffffffu, n, 31);
      }
    }
    __syncthreads();
    blocks = pre[p.G];
    // rows of no group give zero
    const int first = seg[0], end = seg[p.G];
    for (int r = blockIdx.x; r < p.R; r += gridDim.x) {
      if (r >= first && r < end) continue;
      for (int n = threadIdx.x; n < p.N; n += THREADS) store_d(p, r * p.ldd + n, 0.0f);
    }
  } else {
    blocks = (p.R + 8 * NT - 1) / (8 * NT);
  }

  const int64_t units = static_cast<int64_t>(blocks) * p.tiles;
  const bool no_team = idle && cluster_size == 1;
  const int64_t u0 = no_team ? 0 : units * team_id / num_teams;
  const int64_t u1 = no_team ? 0 : units * (team_id + 1) / num_teams;
  // this warp's slabs: slab0 + sl * slab_step, each pass
  const int slab_step = p.team_warps * static_cast<int>(cluster_size);
  const int slab0 = rank * p.team_warps + wk;
  const int passes = (p.slabs + slab_step * KSL - 1) / (slab_step * KSL);
  const uint32_t ring = smem_u32(smem) + warp * STAGES * STAGE_BYTES;

  // ---- ring: steps (unit, pass, slab) in order; the load cursor runs ahead
  int64_t lu = idle ? u1 : u0;
  int ltile = 0, lpass = 0, lsl = 0, lrb = -1, lgroup = 0;
  if (u0 < u1) {
    lrb = static_cast<int>(u0 / p.tiles);
    ltile = static_cast<int>(u0 - static_cast<int64_t>(lrb) * p.tiles);
    lgroup = row_block<NT>(p, seg, pre, lrb).g;
  }
  uint32_t lstage = 0;
  auto issue = [&] {
    if (lu < u1) {
      const int slab = slab0 + (lpass * KSL + lsl) * slab_step;
      if (slab < p.slabs) {
        const uint32_t st = ring + lstage * STAGE_BYTES;
        const int n0 = ltile * TILE_N;
        const uint8_t* base = p.B + lgroup * p.stride_b + slab * (SLAB / 2);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = (lane >> 3) + 4 * i, ch = lane & 7;
          const bool in = n0 + row < p.N && slab * SLAB + 32 * ch < p.K;
          cp_async16(st + 128 * row + ((ch ^ row) & 7) * 16, in ? base + (n0 + row) * p.ldb + 16 * ch : p.B, in ? 16 : 0);
        }
        auto words = [&](uint32_t dst, int pitch, int count, const uint8_t* array, int64_t at, int64_t ld, int64_t size) {
          for (int i = lane; i < TILE_N * count; i += 32) {
            const int row = i / count, w = i - row * count;
            const int64_t off = ((at + (n0 + row) * ld) & ~int64_t{3}) + 4 * w;
            const bool in = n0 + row < p.N && off < size;
            cp_async4(dst + row * pitch + 4 * w, in ? array + off : array,
                      in ? static_cast<uint32_t>(min(int64_t{4}, size - off)) : 0u);
          }
        };
        const int64_t per = FMT == TCG_W4_INT4 ? 2 : 1;
        const int64_t s_at = lgroup * p.stride_scale + per * ((slab * SLAB) >> p.group_shift);
        words(st + CODE_BYTES, SCALE_PITCH, p.scale_words, p.scale, s_at, p.ld_scale, p.scale_bytes);
        if (FMT == TCG_W4_INT4 && p.zero)
          words(st + CODE_BYTES + TILE_N * SCALE_PITCH, ZERO_PITCH, p.zero_words, p.zero,
                lgroup * p.stride_zero + ((slab * SLAB) >> p.group_shift), p.ld_zero, p.zero_bytes);
      }
      if (++lsl == KSL) {
        lsl = 0;
        if (++lpass == passes) {
          lpass = 0;
          ++lu;
          if (++ltile == p.tiles) {
            ltile = 0;
            ++lrb;
            if (lu < u1) lgroup = row_block<NT>(p, seg, pre, lrb).g;
          }
        }
      }
      if (++lstage == STAGES) lstage = 0;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll 1
  for (int i = 0; i < STAGES - 1; ++i) issue();

  uint32_t frag[KSL][8][NT][4];
  float undo[KSL][NT][2];
  RowBlock rb{0, 0, 0};
  int have = -1;  // row block whose fragments are loaded
  uint32_t stage = 0;
  int buf = 0;
  int crb = lrb, ctile = 0;
  if (u0 < u1) {
    crb = static_cast<int>(u0 / p.tiles);
    ctile = static_cast<int>(u0 - static_cast<int64_t>(crb) * p.tiles);
  }
  // one round, or for a cluster (whose CTAs share one unit range) rounds of ROUND units
  for (int64_t r0 = u0, r1; r0 < u1; r0 = r1) {
    r1 = cluster_size > 1 ? min(u1, r0 + ROUND) : u1;
    for (int64_t u = idle ? r1 : r0; u < r1; ++u) {
      float acc[NT][4] = {};
      for (int pass = 0; pass < passes; ++pass) {
        if (have != crb || passes > 1) {
          rb = row_block<NT>(p, seg, pre, crb);
          have = crb;
#pragma unroll
          for (int sl = 0; sl < KSL; ++sl)
            load_fragments<FMT, BF16, NT>(p, rb, slab0 + (pass * KSL + sl) * slab_step, lane, frag[sl], undo[sl]);
        }
#pragma unroll
        for (int sl = 0; sl < KSL; ++sl) {
          issue();
          asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 1) : "memory");
          __syncwarp();
          const int slab = slab0 + (pass * KSL + sl) * slab_step;
          if (slab < p.slabs) {
            const int n0 = ctile * TILE_N;
            const uint32_t per = FMT == TCG_W4_INT4 ? 2u : 1u;
            const uint32_t gi = static_cast<uint32_t>(slab * SLAB) >> p.group_shift;
            const uint32_t s_at = static_cast<uint32_t>(rb.g * p.stride_scale) + per * gi;
            const uint32_t z_at = static_cast<uint32_t>(rb.g * p.stride_zero) + gi;
            const uint32_t lds = static_cast<uint32_t>(p.ld_scale), ldz = static_cast<uint32_t>(p.ld_zero);
            const uint32_t ra = static_cast<uint32_t>(n0 + g), rc = ra + 8;
            const int chunks = min(8, (p.K - slab * SLAB) >> 5);
            const uint32_t st = ring + stage * STAGE_BYTES;
            tile_slab<FMT, BF16, NT>(p, st, lane, chunks, (s_at + ra * lds) & 3u, (s_at + rc * lds) & 3u,
                                     (z_at + ra * ldz) & 3u, (z_at + rc * ldz) & 3u, frag[sl], undo[sl], acc);
          }
          __syncwarp();  // the stage is refilled by the next issue
          if (++stage == STAGES) stage = 0;
        }
      }
      // the team's sum, activation row major with 16 matrix rows each
      float* mine = part + ((buf * WARPS + warp) * 8 * NT) * PART_PITCH;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) mine[(8 * nt + 2 * c + (i & 1)) * PART_PITCH + g + 8 * (i >> 1)] = acc[nt][i];
      team_sync(team, p.team_warps);
      const float* base = part + ((buf * WARPS + team * p.team_warps) * 8 * NT) * PART_PITCH;
      for (int j = wk * 32 + lane; j < 128 * NT; j += 32 * p.team_warps) {
        const int row = j >> 4, n = j & 15;
        float s = 0.0f;
        for (int w = 0; w < p.team_warps; ++w) s += base[(w * 8 * NT + row) * PART_PITCH + n];
        if (cluster_size > 1) {
          sums[(u - r0) * 128 * NT + j] = s;
        } else if (row < rb.rows && ctile * TILE_N + n < p.N) {
          store_d(p, (rb.row0 + row) * p.ldd + ctile * TILE_N + n, p.alpha ? s * p.alpha[rb.g] : s);
        }
      }
      buf ^= 1;
      if (++ctile == p.tiles) {
        ctile = 0;
        ++crb;
      }
    }
    if (cluster_size > 1) {
      cluster_sync();
      // the round's outputs, spread over the cluster's threads
      const int count = static_cast<int>(r1 - r0) * 128 * NT;
      for (int j = rank * THREADS + threadIdx.x; j < count; j += cluster_size * THREADS) {
        const int64_t u = r0 + j / (128 * NT);
        const int row = (j >> 4) % (8 * NT), n = j & 15;
        const int b = static_cast<int>(u / p.tiles), tile = static_cast<int>(u - static_cast<int64_t>(b) * p.tiles);
        const RowBlock o = row_block<NT>(p, seg, pre, b);
        if (row < o.rows && tile * TILE_N + n < p.N) {
          float s = 0.0f;
          for (uint32_t k = 0; k < cluster_size; ++k) s += ld_cluster_f32(mapa_shared(smem_u32(sums + j), k));
          store_d(p, (o.row0 + row) * p.ldd + tile * TILE_N + n, p.alpha ? s * p.alpha[o.g] : s);
        }
      }
      cluster_sync();  // peers have read this CTA's sums
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// ---------------------------------------------------------------------- host

using Kernel = void (*)(GemvParams);

// Index of a variant: format, bf16, (NT, KSL) = (1, 1), (1, 2), (2, 1).
constexpr int SHAPES = 3, VARIANTS = 3 * 2 * SHAPES;
constexpr int shape_index(int nt, int ksl) { return nt == 2 ? 2 : ksl - 1; }

template <int FMT, bool BF16>
void fill(Kernel* k) {
  k[0] = gemv_kernel<FMT, BF16, 1, 1>;
  k[1] = gemv_kernel<FMT, BF16, 1, 2>;
  k[2] = gemv_kernel<FMT, BF16, 2, 1>;
}

struct Variants {
  Kernel k[VARIANTS];
  Variants() {
    fill<TCG_W4_INT4, false>(k);
    fill<TCG_W4_INT4, true>(k + SHAPES);
    fill<TCG_W4_MXF4, false>(k + 2 * SHAPES);
    fill<TCG_W4_MXF4, true>(k + 3 * SHAPES);
    fill<TCG_W4_NVF4, false>(k + 4 * SHAPES);
    fill<TCG_W4_NVF4, true>(k + 5 * SHAPES);
  }
};
const Variants g_variants;

int smem_bytes(int nt) { return nt == 2 ? GemvSmem<2>::BYTES : GemvSmem<1>::BYTES; }

// Per device, on the first call: the variants' shared-memory attribute and the
// clusters of 1, 2 and 4 CTAs that are resident at once.
constexpr int MAX_DEVICES = 64;
struct DeviceInfo {
  std::once_flag once;
  cudaError_t err = cudaSuccess;
  int clusters[3] = {0, 0, 0};
};
DeviceInfo g_info[MAX_DEVICES];

const DeviceInfo& device_info(int dev) {
  DeviceInfo& d = g_info[dev];
  std::call_once(d.once, [&] {
    for (int i = 0; i < VARIANTS && d.err == cudaSuccess; ++i)
      d.err = cudaFuncSetAttribute(reinterpret_cast<const void*>(g_variants.k[i]),
                                   cudaFuncAttributeMaxDynamicSharedMemorySize,
                                   smem_bytes(i % SHAPES == shape_index(2, 1) ? 2 : 1));
    d.clusters[0] = device_sms(dev);
    for (int i = 1; i < 3 && d.err == cudaSuccess; ++i) {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(static_cast<unsigned>(d.clusters[0] >> i << i), 1, 1);
      cfg.blockDim = dim3(THREADS, 1, 1);
      cfg.dynamicSmemBytes = smem_bytes(2);
      cudaLaunchAttribute attr;
      attr.id = cudaLaunchAttributeClusterDimension;
      attr.val.clusterDim.x = 1u << i;
      attr.val.clusterDim.y = 1;
      attr.val.clusterDim.z = 1;
      cfg.attrs = &attr;
      cfg.numAttrs = 1;
      d.err = cudaOccupancyMaxActiveClusters(&d.clusters[i],
                                             reinterpret_cast<const void*>(g_variants.k[shape_index(2, 1)]), &cfg);
    }
  });
  return d;
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
  const int64_t blocks_k = a.K / a.group;
  if (a.K > 0) {
    if (a.K % 32 || a.K % a.group) return TCG_ERR_ALIGNMENT;
    if (a.lda == 0) a.lda = a.K;
    if (a.ldb == 0) a.ldb = a.K;
    if (a.ld_scale == 0) a.ld_scale = blocks_k;
    if (a.lda < a.K || a.ldb < a.K || a.ld_scale < blocks_k) return TCG_ERR_INVALID;
    if (a.stride_b == 0) a.stride_b = a.N * a.ldb;
    if (a.stride_scale == 0) a.stride_scale = a.N * a.ld_scale;
    if (!a.A || !a.B || !a.scale || a.stride_b < 0 || a.stride_scale < 0) return TCG_ERR_INVALID;
    if (reinterpret_cast<uintptr_t>(a.A) % 16 || a.lda % 8 || reinterpret_cast<uintptr_t>(a.B) % 16 || a.ldb % 32 ||
        a.stride_b % 32)
      return TCG_ERR_ALIGNMENT;
    if ((reinterpret_cast<uintptr_t>(a.scale) | reinterpret_cast<uintptr_t>(a.zero)) % 4) return TCG_ERR_ALIGNMENT;
  }
  int dev;
  if (int rc = current_device_checked(&dev)) return rc;
  if (a.K == 0) {
    const size_t ds = a.d_type == TCG_F32 ? 4 : 2;
    if (int rc = record_cuda(cudaMemset2DAsync(a.D, static_cast<size_t>(a.ldd) * ds, 0, static_cast<size_t>(a.N) * ds,
                                               static_cast<size_t>(a.R), s)))
      return rc;
    set_launch_count(1);
    return TCG_OK;
  }
  GemvParams p;
  std::memset(&p, 0, sizeof p);
  const int es = a.format == TCG_W4_INT4 ? 2 : 1;
  p.R = static_cast<int>(a.R);
  p.N = static_cast<int>(a.N);
  p.K = static_cast<int>(a.K);
  p.G = a.G;
  p.group_shift = a.group == 16 ? 4 : a.group == 32 ? 5 : a.group == 64 ? 6 : 7;
  p.A = static_cast<const uint8_t*>(a.A);
  p.lda = a.lda;
  p.offsets = a.offsets;
  p.B = a.B;
  p.ldb = a.ldb / 2;
  p.stride_b = a.stride_b / 2;
  const int64_t scales = (a.G - 1) * a.stride_scale + (a.N - 1) * a.ld_scale + blocks_k;
  p.scale = static_cast<const uint8_t*>(a.scale);
  p.ld_scale = a.ld_scale * es;
  p.stride_scale = a.stride_scale * es;
  p.scale_bytes = scales * es;
  p.zero = a.zero;
  p.ld_zero = a.ld_scale;
  p.stride_zero = a.stride_scale;
  p.zero_bytes = scales;
  // words that hold a row's slab: one more where rows start off a 4-byte boundary
  const int seg_s = SLAB / a.group * es, seg_z = SLAB / a.group;
  p.scale_words = seg_s / 4 + (p.ld_scale % 4 || p.stride_scale % 4 ? 1 : 0);
  p.zero_words = (seg_z + 3) / 4 + (p.ld_zero % 4 || p.stride_zero % 4 ? 1 : 0);
  p.alpha = a.alpha;
  p.D = a.D;
  p.d_type = a.d_type;
  p.ldd = a.ldd;
  p.tiles = static_cast<int>((a.N + TILE_N - 1) / TILE_N);
  p.slabs = static_cast<int>((a.K + SLAB - 1) / SLAB);

  // rows per block: 16 when groups are expected to have more than 8 rows
  const int64_t active = std::min<int64_t>(a.G, a.R);
  const int nt = a.R > 8 * active ? 2 : 1;
  const int64_t units = std::max<int64_t>(active, (a.R + 8 * nt - 1) / (8 * nt)) * p.tiles;
  if (units > INT32_MAX) return TCG_ERR_UNSUPPORTED;
  // The team: KSL slabs a warp, over a cluster of `cl` CTAs.  The busiest
  // team's tiles times the slabs each of its warps takes is the time; of equal
  // ones the first below (fewer CTAs, then more slabs a warp) is taken.
  const DeviceInfo& info = device_info(dev);
  if (info.err != cudaSuccess) return record_cuda(info.err);
  int best_ksl = 1, best_cl = 1;
  int64_t best = INT64_MAX;
  for (int i = 0, cl = 1; i < 3; ++i, cl *= 2) {
    if (info.clusters[i] < 1) continue;
    for (int ksl = nt == 1 ? 2 : 1; ksl >= 1; --ksl) {
      const int want = (p.slabs + cl * ksl - 1) / (cl * ksl);
      if (cl > 1 && want <= WARPS / 2) continue;  // half a CTA would idle
      const int team_warps = std::min(WARPS, want);
      const int teams = cl > 1 ? 1 : WARPS / team_warps;
      const int64_t n = static_cast<int64_t>(info.clusters[i]) * teams;
      const int64_t passes = (p.slabs + cl * ksl * team_warps - 1) / (cl * ksl * team_warps);
      const int64_t time = (units + n - 1) / n * passes * ksl * (passes > 1 ? 2 : 1);
      if (time < best) {
        best = time;
        best_ksl = ksl;
        best_cl = cl;
      }
    }
  }
  p.team_warps = std::min(WARPS, (p.slabs + best_cl * best_ksl - 1) / (best_cl * best_ksl));
  p.teams = best_cl > 1 ? 1 : WARPS / p.team_warps;
  const bool bf16 = a.in_type == TCG_IN_BF16;
  const Kernel k = g_variants.k[(a.format * 2 + (bf16 ? 1 : 0)) * SHAPES + shape_index(nt, best_ksl)];
  cudaLaunchConfig_t cfg = {};
  const int64_t ctas = std::min<int64_t>(info.clusters[best_cl / 2], units);
  cfg.gridDim = dim3(static_cast<unsigned>(ctas * best_cl), 1, 1);
  cfg.blockDim = dim3(THREADS, 1, 1);
  cfg.dynamicSmemBytes = smem_bytes(nt);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = best_cl;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = best_cl > 1 ? 2 : 1;
  void* params[] = {&p};
  if (int rc = record_cuda(cudaLaunchKernelExC(&cfg, reinterpret_cast<const void*>(k), params))) return rc;
  set_launch_count(1);
  return TCG_OK;
}

}  // namespace

}  // namespace tcg

using namespace tcg;

extern "C" int tcg_gemv_w4(const tcg_gemv_w4_args* args, void* stream) {
  return guarded([&] { return run_gemv(args, static_cast<cudaStream_t>(stream)); });
}
