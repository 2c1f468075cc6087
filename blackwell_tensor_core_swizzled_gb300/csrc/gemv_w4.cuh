// Few rows of 16-bit activations against 4-bit matrices with group scales.
// The kernel; entry point and host plan are in gemv_w4.cu, the contract in
// include/tcg.h.
//
// The work is to stream the codes: N K / 2 bytes a matrix against a few rows.
// Codes are decoded to f16 in registers (every E2M1 value, and code - zero of
// INT4, is exact there) and multiplied by mma m16n8k16 with fp32
// accumulation: 16 matrix rows by 8 activation rows, so that up to 8 rows cost
// the decoding once.  (A tcgen05 product would take the decoded codes through
// shared or tensor memory first, four times the codes' bytes: 7 us each way for
// 16384 x 8192 at 128 bytes a cycle and SM.  For up to 8 rows, 24 us, that is
// too much; for 17 and more, which decode the matrix again for every 16 (int4
// 16384 x 8192: 16 rows 34 us, 32 rows 62), it would pay.)  Scales keep every
// product exact: NVFP4's unsigned E4M3 scale times an E2M1 value has 6
// significant bits between 2^-10 and 2688, an f16 value, so it is multiplied
// into the decoded codes and the whole contraction is one chain of mma; e8m0
// and 16-bit scales do not fit f16 that way and multiply the group's fp32 sum.
//
// Decoding, not HBM, is the first bound: integer and conversion instructions
// issue at half rate, so the 16 decoding warps do little else, and what feeds
// and empties them has warps of its own:
//   warps 0..15   a slab of 256 of K each, whose activations stay in
//                 registers, walking down the matrix 16 rows at a time (eight
//                 warps when there are 16 activation rows: their fragments
//                 take 64 registers, and what spills goes past an L1 that
//                 shared memory leaves almost nothing of; at the 96 registers
//                 that 19 warps leave, most variants of 4 and 8 rows spill a
//                 few, int4 in groups of 32 with 4 rows and nvf4 bf16 with 8
//                 up to 116 bytes)
//   the next      brings the rows of a stage to a ring: codes, scales and
//                 zero points by a TMA copy each, for all slabs at once (a
//                 copy takes its issuing thread 150 cycles; one for every
//                 warp or row would take longer than the decoding)
//   two more      add the warps' parts of a tile of two stages in a fixed
//                 order and store it while the next tile is decoded;
//   the last      brings scales and zero points whose rows TMA cannot, since
//                 they do not start on 16-byte boundaries.
// The warps cover K side by side; when K is short, the others stand below
// them and a stage has so many more rows.  Each CTA takes an equal share of
// the matrix rows.  A K of more slabs than warps is taken in passes over a
// chunk of tiles, whose sums wait in shared memory.  What lies beyond K or N
// is zero, so the inner loop has no bounds.
//
// Decoding 16 rows of 256 takes a scheduler 253 cycles in mxf4, 310 in nvf4,
// 400 in int4 (16 activation rows 520), where HBM feeds them in 370; a tile's
// hand-overs add about 100.  One token on mxf4 8192 x 8192 takes 13.0 us, of
// which 5 are the codes' bytes at HBM's rate and 5 the start: the offsets, the
// activations, the first bytes and the code itself are all fetched cold, one
// after the other.  32 rows on 64 nvf4 experts of 4096 x 4096: 45 us (5.3
// TB/s).  16 rows on int4 16384 x 8192: 33.5 us, of which the four passes are 3
// (as 65536 x 2048, one pass, 30.6): two decoding warps a scheduler, of which
// 0.7 can issue on average, leave half of its cycles empty.  With 8 rows, 24.6
// us, 1.5 of four warps can, and 63 % of the cycles issue.
//
// bf16 activations are brought into f16's range by a power of two per row and
// slab (the largest finite value to [2^14, 2^15)), undone on fp32 sums, before a
// scale that could overflow with it.  f16 then holds every value down to 2^-31
// of the slab's largest with all its bits.  Smaller ones may be all that counts
// (where the larger ones meet zero codes, or their groups a small scale), so a
// CTA that meets one, or a slab near either end of bf16's range, does its share
// once more with such slabs in bands of 32 binades each: mxf4 8192 x 8192, 1 row,
// 13 us without and 58 to 63 with them, nvf4 16384 x 8192, 8 rows, 26 and 87
// (six such values) to 115 (in all slabs).  (What looks for them costs usual
// calls 1 to 7 %, 8 rows of nvf4 11.)
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstring>

#include "common.h"
#include "gemm_kernel.cuh"
#include "ptx.cuh"
#include "ptx_moe.cuh"

namespace tcg {

namespace {

constexpr int MAX_GROUPS = 1024;
constexpr int64_t MAX_EXTENT = int64_t{1} << 30;

constexpr int SLAB = 256;          // K per warp: 128 bytes of codes
constexpr int STAGE_N = 16;        // matrix rows per stage: one mma's
// a swizzled box of rows of `span` bytes: where byte x of row r lies
__device__ __forceinline__ uint32_t box_at(uint32_t r, uint32_t x, uint32_t span) {
  const uint32_t swizzle = span == 128 ? r & 7u : span == 64 ? (r >> 1) & 3u : (r >> 2) & 1u;
  return r * span + (x ^ (swizzle << 4));
}

// What a kernel is compiled for: a format, and for INT4 its group.
enum Kind4 : int { K_INT4_32 = 0, K_INT4_64 = 1, K_INT4_128 = 2, K_MXF4 = 3, K_NVF4 = 4, KINDS4 = 5 };
constexpr bool is_int4(int k) { return k <= K_INT4_128; }
constexpr int group_of_kind(int k) { return k == K_NVF4 ? 16 : k == K_MXF4 ? 32 : 32 << k; }
constexpr int scale_bytes(int k) { return SLAB / group_of_kind(k) * (is_int4(k) ? 2 : 1); }  // of a row's slab
// room in a stage for scales, and zero points behind the first 8 KiB: 16 rows
// for a K of 8000
constexpr int SCALE_STAGE = 12 * 1024, ZERO_OFF = 8 * 1024;
constexpr int GRAIN = 2;           // matrix rows: the unit in which the CTAs share them

struct GemvParams {
  // codes as bytes in 128-byte swizzled boxes of a stage's rows: whole slabs
  // [G][K / 256][N][128], all that a stage has of them in one box; when K has
  // a part of a slab more, also rows [G][N][K / 2], one slab a box
  CUtensorMap tmap_b, tmap_part;
  // scales, zero points as bytes [G][N][bytes of a row] in swizzled boxes of a
  // stage's rows, where their rows are 16-byte aligned (`bulk`)
  CUtensorMap tmap_s, tmap_z;
  int box_s, box_z;  // bytes of a box's rows: 32, 64 or 128 (not `bulk`: from row to row)
  int one_run;       // not `bulk`: a stage's rows are copied with what lies between them, not one by one
  int R, N, K, G;
  const uint8_t* A;  // 16-bit elements
  int64_t lda;
  const int32_t* offsets;
  const uint8_t* scale;
  int64_t ld_scale, stride_scale;  // bytes
  int scale_row;                   // scales of a row
  const uint8_t* zero;
  int64_t ld_zero, stride_zero;
  int bulk;
  const float* alpha;
  void* D;
  int d_type;
  int64_t ldd;
  int grains;       // GRAIN-row units of a matrix
  int slabs;        // ceil(K / 256)
  int passes;       // of `across` slabs
  int blocks, share;  // row blocks there probably are, and then a CTA's grains
  int across;       // warps side by side along K
  int tile_rows;    // 32 down
  int down;         // warps below each other: 16 rows of a stage each
  unsigned long long* err;
  uint64_t timeout_ns;
};

// TOK activation rows per block: 4, 8 or 16.  They are the columns of one mma
// (16: of two); 4 rows take its even columns, which are half of a lane's
// accumulators, so that scaling costs half.
template <int TOK>
struct Shape {
  static constexpr int NT = TOK == 16 ? 2 : 1;        // mma column blocks
  static constexpr int STEP = TOK == 4 ? 2 : 1;       // accumulator columns between rows
  static constexpr int WARPS = TOK == 16 ? 8 : 16;    // decoding warps
  static constexpr int TILE_N = 32;                   // matrix rows a warp has of a tile: two stages
  static constexpr int OUT = TOK * TILE_N;            // sums of them
  static constexpr int CAP = (TOK == 16 ? 4096 : 1024) / OUT;  // tiles of a chunk that is passed over more than once
  static constexpr int STAGES = TOK == 16 ? 5 : 4;    // ring stages
  // buffers of parts: tile i of a chunk uses number i % PARTS, and each adding
  // warp empties one: in every pass the same warp has the tile's sums
  static constexpr int PARTS = 2;
  static constexpr int ADD_WARPS = PARTS;
  static constexpr int threads(bool bulk) { return 32 * (WARPS + 1 + ADD_WARPS + (bulk ? 0 : 1)); }
  static constexpr int PART_PITCH = TILE_N + (TOK == 4 ? 8 : 4);  // floats between a part's activation rows
  static constexpr int TILE_PART = TOK * PART_PITCH;  // floats of a warp's part
  // a stage: codes [slab][row][128 bytes]; scales, then zero points [row][pitch]
  // or as boxes
  static constexpr int CODE_BYTES = WARPS * STAGE_N * SLAB / 2;
  static constexpr int SCALES = STAGES * CODE_BYTES;
  static constexpr int PART = SCALES + STAGES * SCALE_STAGE;
  // an activation row on its way to each warp's registers
  static constexpr int ACT = PART + PARTS * WARPS * TILE_PART * 4;
  static constexpr int ACT_BYTES = TOK == 4 ? SLAB * 2 : 0;
  static constexpr int SUM = ACT + WARPS * ACT_BYTES;
  // full[STAGES], empty[STAGES], part_full[PARTS], part_free[PARTS]; and others
  // for doing the share again
  static constexpr int BARS = SUM + CAP * OUT * 4, BAR_BYTES = (2 * STAGES + 2 * PARTS) * 8;
  static constexpr int SEG = BARS + 2 * BAR_BYTES + 8;  // abort and unusual flags before it
  static constexpr int BYTES = 1024 + SEG + 2 * (MAX_GROUPS + 1) * 4;
  static_assert(BYTES <= 232448, "dynamic shared memory");
};

__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
// Bytes [src, src + len) of a tensor that starts on a 4-byte boundary to shared
// memory, as far past the 16-byte boundary dst as src is past one: a bulk copy,
// and words before and after it.  Returns the bulk copy's bytes.
__device__ __forceinline__ uint32_t copy_run(uint32_t dst, const uint8_t* src, int len, uint32_t bar) {
  const int mis = static_cast<int>(reinterpret_cast<uintptr_t>(src)) & 15;
  src -= mis;
  len += mis;
  const int head = mis ? 16 : 0, tail = max(len & ~15, head);
#pragma unroll 1
  for (int x = mis & ~3; x < min(head, len); x += 4) cp_async4(dst + x, src + x, min(4, len - x));
#pragma unroll 1
  for (int x = tail; x < len; x += 4) cp_async4(dst + x, src + x, min(4, len - x));
  if (tail > head) bulk_copy(dst + head, src + head, tail - head, bar);
  return tail - head;
}
// Loads by shared-memory address that the compiler may move between waits.
template <class T>
__device__ __forceinline__ T lds(const uint8_t* base, uint32_t off) {
  return *reinterpret_cast<const T*>(base + off);
}

// d += a b (16 x 16 by 16 x 8, f16 in, fp32 out); mma16816_zero: d = a b
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma16816_zero(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

// the eight E2M1 codes of a word as four f16 pairs, in order
__device__ __forceinline__ void e2m1_word(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}
__device__ __forceinline__ uint32_t hsub2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
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
// holds 1024 + zero twice, nz -(64 + zero).
__device__ __forceinline__ void int4_word(uint32_t w, uint32_t z1024, uint32_t nz, uint32_t (&h)[4]) {
  constexpr uint32_t K1024 = 0x64006400u, SIXTEENTH = 0x2C002C00u;
  const uint32_t w8 = w >> 8;
  h[0] = hsub2((w & 0x000F000Fu) | K1024, z1024);
  h[1] = hfma2((w & 0x00F000F0u) | K1024, SIXTEENTH, nz);
  h[2] = hsub2((w8 & 0x000F000Fu) | K1024, z1024);
  h[3] = hfma2((w8 & 0x00F000F0u) | K1024, SIXTEENTH, nz);
}

__device__ __forceinline__ float half_bits(uint32_t h) { return __half2float(__ushort_as_half(static_cast<uint16_t>(h))); }

__device__ __forceinline__ void store_d(const GemvParams& p, int64_t i, float v) {
  if (p.d_type == TCG_F32)
    static_cast<float*>(p.D)[i] = v;
  else if (p.d_type == TCG_F16)
    static_cast<__half*>(p.D)[i] = __float2half_rn(v);
  else
    static_cast<__nv_bfloat16*>(p.D)[i] = __float2bfloat16_rn(v);
}

// A row block: up to TOK rows of one group.
struct RowBlock {
  int g, row0, rows;
};

// `span`: the rows of a single block (first, last + 1), when there is but one
template <int TOK>
__device__ __noinline__ RowBlock row_block(const GemvParams& p, const int* seg, const int* pre, bool single, int2 span,
                                           int rb) {
  if (single) return {0, span.x, span.y - span.x};
  if (!p.offsets) return {0, rb * TOK, min(TOK, p.R - rb * TOK)};
  int a = 0, b = p.G;  // pre[a] <= rb < pre[b]
  while (b - a > 1) {
    const int mid = (a + b) >> 1;
    if (pre[mid] <= rb)
      a = mid;
    else
      b = mid;
  }
  const int row0 = seg[a] + (rb - pre[a]) * TOK;
  return {a, row0, min(TOK, seg[a + 1] - row0)};
}

// How a row's slab of bf16 activations is brought into f16: 2^e brings the
// largest finite one to [2^14, 2^15), and undo = 2^-e takes it back.  f16 holds
// all bits of a bf16 value from 2^-17 on.  Where smaller ones are among them,
// the slab is taken in bands, band b with those that 2^(e + 32 b) brings to
// [2^-17, 2^15) (up to 2^126, where every bf16 value is in range).
//
// 2^-e comes before the scale, which could overflow with it.  A group's sum is 0
// or in [2^-25, 2^30), so that this stays a normal number for e in [-96, 96];
// for others `after` behind the scale makes up the rest.  A slab of one band and
// such an e is a usual one.
constexpr int EXACT_BINADES = 31;  // below the largest value's, that f16 holds
constexpr int BAND_STEP = 32, MAX_UNDO = 96;
__device__ __forceinline__ float power_of_2(int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }
// Magnitude bits of two values: the running maximum, NaN dropped, and the
// minimum of each less 1 (0xFFFF: a zero)
__device__ __forceinline__ void extremes(uint32_t v, uint32_t& largest, uint32_t& smallest) {
  const uint32_t mag = v & 0x7FFF7FFFu;
  asm("max.bf16x2 %0, %0, %1;" : "+r"(largest) : "r"(mag));
  asm("{\n\t.reg .b32 t;\n\tadd.u16x2 t, %1, %2;\n\tmin.u16x2 %0, %0, t;\n\t}"
      : "+r"(smallest)
      : "r"(mag), "r"(0xFFFFFFFFu));
}
// The scaling of a row by the magnitude bits of its largest value.
struct Scaling {
  int e;
  float after;
  uint32_t low, high;  // magnitude bits of a band
};
__device__ __forceinline__ int first_exponent(uint32_t largest) { return min(141 - static_cast<int>(largest >> 7), 126); }
// Whether it wants bands or `after` (`smallest`: a lane's, as above).
__device__ __forceinline__ bool is_unusual(uint32_t largest, uint32_t smallest) {
  const int s = static_cast<int>(min(smallest & 0xFFFFu, smallest >> 16));
  return s < static_cast<int>(largest & 0x7F80u) - (EXACT_BINADES << 7) || largest >= (141 + MAX_UNDO + 1) << 7 ||
         largest - 1 < ((141 - MAX_UNDO) << 7) - 1;
}
__device__ __forceinline__ Scaling scaling_of_band(uint32_t largest, int band) {
  Scaling r;
  // magnitude bits of 2^x, 0 below bf16's subnormals, inf above its range
  const auto bits = [](int x) {
    return x > 127 ? 0x7F80u : x >= -126 ? static_cast<uint32_t>(x + 127) << 7 : x >= -133 ? 1u << (x + 133) : 0u;
  };
  const int e0 = largest ? first_exponent(largest) : 0;
  r.e = min(e0 + BAND_STEP * band, 126);
  r.after = power_of_2(min(max(r.e, -MAX_UNDO), MAX_UNDO) - r.e);
  r.low = bits(-17 - r.e);
  r.high = band ? bits(-17 - min(e0 + BAND_STEP * (band - 1), 126)) : 0x8000u;
  return r;
}
// v without the values of other bands
__device__ __forceinline__ uint32_t of_band(uint32_t v, const Scaling& r) {
  const uint32_t x = v & 0x7FFFu, y = (v >> 16) & 0x7FFFu;
  return (x >= r.low && x < r.high ? v & 0xFFFFu : 0u) | (y >= r.low && y < r.high ? v & 0xFFFF0000u : 0u);
}

// Two bf16 values times `up` as f16
__device__ __forceinline__ uint32_t to_f16(uint32_t v, float up) {
  const __half2 h = __floats2half2_rn(__uint_as_float(v << 16) * up, __uint_as_float(v & 0xFFFF0000u) * up);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// Eight elements in the order in which int4_word decodes: (0,4) (1,5) (2,6) (3,7)
__device__ __forceinline__ void order_int4(uint32_t (&f)[4]) {
  const uint32_t v0 = f[0], v1 = f[1], v2 = f[2], v3 = f[3];
  f[0] = __byte_perm(v0, v2, 0x5410);
  f[1] = __byte_perm(v0, v2, 0x7632);
  f[2] = __byte_perm(v1, v3, 0x5410);
  f[3] = __byte_perm(v1, v3, 0x7632);
}

// The activations of a row block for one slab as B fragments.  Lane (g, c) =
// (lane / 4, lane % 4) holds column 8 nt + g (TOK = 4: row g / 2, even g
// alone count); `frag[ch][nt]` covers 32 of K in the order in which the codes
// decode.  With up to 4 rows a row is read 8 elements a lane, brought into
// f16's range and passed through the warp's scratch, where element order is
// fragment order: converting them as fragments would repeat the work of the
// columns that do not count.
// undo (bf16): the factors that take the scaling back, for the accumulator's
// columns 2c and 2c + 1 (TOK = 4: row c).  Sets *unusual if the slab is not a
// usual one; the fragments are of no use then.
template <int KIND, bool BF16, int TOK, int NT = Shape<TOK>::NT>
__device__ __forceinline__ void load_fragments(const GemvParams& p, const RowBlock& rb, int slab, int lane,
                                               uint8_t* scratch, volatile uint32_t* unusual,
                                               uint32_t (&frag)[8][NT][4], float (&undo)[NT][2]) {
  const int g = lane >> 2, c = lane & 3;
  if constexpr (TOK > 4) {
    // many rows: each lane reads its own fragments, a quad shares a row
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = 8 * nt + g;
      const uint8_t* row = p.A + 2 * ((rb.row0 + r) * p.lda + slab * SLAB + 8 * c);
#pragma unroll
      for (int ch = 0; ch < 8; ++ch) {
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (r < rb.rows && slab * SLAB + 32 * ch < p.K) v = *reinterpret_cast<const uint4*>(row + 64 * ch);
        uint32_t(&f)[4] = frag[ch][nt];
        f[0] = v.x;
        f[1] = v.y;
        f[2] = v.z;
        f[3] = v.w;
      }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      undo[nt][0] = undo[nt][1] = 1.0f;
      if (BF16) {
        uint32_t m2 = 0, least = 0xFFFFFFFFu;
#pragma unroll
        for (int ch = 0; ch < 8; ++ch)
#pragma unroll
          for (int i = 0; i < 4; ++i) extremes(frag[ch][nt][i], m2, least);
        uint32_t m = max(m2 & 0xFFFFu, m2 >> 16);
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
        if (is_unusual(m, least)) *unusual = 1u;
        const int e = first_exponent(m);
        const float up = power_of_2(e), down = power_of_2(-e);
#pragma unroll
        for (int ch = 0; ch < 8; ++ch)
#pragma unroll
          for (int i = 0; i < 4; ++i) frag[ch][nt][i] = to_f16(frag[ch][nt][i], up);
        // the factors of rows 2c and 2c + 1, held by the lanes of those rows
        undo[nt][0] = __shfl_sync(0xffffffffu, down, 8 * c);
        undo[nt][1] = __shfl_sync(0xffffffffu, down, 8 * c + 4);
      }
      if (is_int4(KIND)) {
#pragma unroll
        for (int ch = 0; ch < 8; ++ch) order_int4(frag[ch][nt]);
      }
    }
  } else {
#pragma unroll
    for (int ch = 0; ch < 8; ++ch)
#pragma unroll
      for (int i = 0; i < 4; ++i) frag[ch][0][i] = 0u;
    const uint8_t* src = p.A + 2 * (rb.row0 * p.lda + slab * SLAB + 8 * lane);
    const bool in = slab * SLAB + 8 * lane < p.K;
    float down = 1.0f;  // row c's factor
    uint4 next[4];  // all rows in flight at once
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      next[r] = make_uint4(0u, 0u, 0u, 0u);
      if (in && r < rb.rows) next[r] = *reinterpret_cast<const uint4*>(src + 2 * r * p.lda);
    }
#pragma unroll 1
    for (int r = 0; r < rb.rows; ++r) {
      uint32_t v[4] = {next[0].x, next[0].y, next[0].z, next[0].w};
      next[0] = next[1];
      next[1] = next[2];
      next[2] = next[3];
      if (BF16) {
        uint32_t m2 = 0, least = 0xFFFFFFFFu;
#pragma unroll
        for (int i = 0; i < 4; ++i) extremes(v[i], m2, least);
        const uint32_t m = __reduce_max_sync(0xffffffffu, max(m2 & 0xFFFFu, m2 >> 16));
        if (is_unusual(m, least)) *unusual = 1u;
        const int e = first_exponent(m);
        const float up = power_of_2(e);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = to_f16(v[i], up);
        if (c == r) down = power_of_2(-e);
      }
      if (is_int4(KIND)) order_int4(v);
      *reinterpret_cast<uint4*>(scratch + 16 * lane) = make_uint4(v[0], v[1], v[2], v[3]);
      __syncwarp();
      if (g == 2 * r) {  // the row of this even column: 8 consecutive elements of each 32
#pragma unroll
        for (int ch = 0; ch < 8; ++ch) {
          const uint4 a = lds<uint4>(scratch, 64 * ch + 16 * c);
          uint32_t(&f)[4] = frag[ch][0];
          f[0] = a.x;
          f[1] = a.y;
          f[2] = a.z;
          f[3] = a.w;
        }
      }
      __syncwarp();
    }
    undo[0][0] = undo[0][1] = down;
    __syncwarp();
  }
}

// The same of one band of any slab: undo before the scale and `after` behind it.
// Returns whether a row has values of a later band.
template <int KIND, int TOK, int NT = Shape<TOK>::NT>
__device__ __forceinline__ bool load_band(const GemvParams& p, const RowBlock& rb, int slab, int band, int lane,
                                          uint32_t (&frag)[8][NT][4], float (&undo)[NT][2], float (&after)[NT][2]) {
  const int g = lane >> 2, c = lane & 3;
  bool later = false;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int r = TOK > 4 ? 8 * nt + g : g & 1 ? TOK : g / 2;  // the column's row; TOK: none
    const uint8_t* row = p.A + 2 * ((rb.row0 + r) * p.lda + slab * SLAB + 8 * c);
    uint32_t m2 = 0, least = 0xFFFFFFFFu;
#pragma unroll
    for (int ch = 0; ch < 8; ++ch) {
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      if (r < rb.rows && slab * SLAB + 32 * ch < p.K) v = *reinterpret_cast<const uint4*>(row + 64 * ch);
      uint32_t(&f)[4] = frag[ch][nt];
      f[0] = v.x;
      f[1] = v.y;
      f[2] = v.z;
      f[3] = v.w;
#pragma unroll
      for (int i = 0; i < 4; ++i) extremes(f[i], m2, least);
    }
    uint32_t m = max(m2 & 0xFFFFu, m2 >> 16);
    if (m >= 0x7F80u) {  // past infinities
      m = 0;
#pragma unroll
      for (int ch = 0; ch < 8; ++ch)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t lo = frag[ch][nt][i] & 0x7FFFu, hi = (frag[ch][nt][i] >> 16) & 0x7FFFu;
          if (lo < 0x7F80u) m = max(m, lo);
          if (hi < 0x7F80u) m = max(m, hi);
        }
    }
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    const Scaling s = scaling_of_band(m, band);
    const float up = power_of_2(s.e), down = power_of_2(-min(max(s.e, -MAX_UNDO), MAX_UNDO));
    least = min(least & 0xFFFFu, least >> 16);
    later |= least != 0xFFFFu && least + 1 < s.low;
#pragma unroll
    for (int ch = 0; ch < 8; ++ch) {
      uint32_t(&f)[4] = frag[ch][nt];
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i] = to_f16(of_band(f[i], s), up);
      if (is_int4(KIND)) order_int4(f);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int from = 8 * c + (TOK > 4 ? 4 * i : 0);
      undo[nt][i] = __shfl_sync(0xffffffffu, down, from);
      after[nt][i] = __shfl_sync(0xffffffffu, s.after, from);
    }
  }
  return __any_sync(0xffffffffu, later);
}

// A row's scales of a slab as words, from a byte offset that may be off a
// 4-byte boundary, and followed by another row's after `left` bytes.
template <int W, bool ALIGNED>
__device__ __forceinline__ void scale_words(const uint8_t* at, int left, uint32_t (&w)[W]) {
  if constexpr (ALIGNED) {
    if constexpr (W == 4) {
      const uint4 v = lds<uint4>(at, 0);
      w[0] = v.x;
      w[1] = v.y;
      w[2] = v.z;
      w[3] = v.w;
    } else if constexpr (W == 2) {
      const uint2 v = lds<uint2>(at, 0);
      w[0] = v.x;
      w[1] = v.y;
    } else {
      w[0] = lds<uint32_t>(at, 0);
    }
  } else {
    const uint32_t off = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(at)) & 3u;
    const uint8_t* base = at - off;
    uint32_t lo = lds<uint32_t>(base, 0);
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const uint32_t hi = lds<uint32_t>(base, 4 * i + 4);
      w[i] = __funnelshift_r(lo, hi, 8 * off);
      lo = hi;
    }
    if (left < 4 * W) {
#pragma unroll
      for (int i = 0; i < W; ++i)
        w[i] &= left >= 4 * i + 4 ? ~0u : left > 4 * i ? (1u << (8 * (left - 4 * i))) - 1u : 0u;
    }
  }
}

// 16 rows of a tile and a slab: acc[nt] = (codes . activations) * scales.
// `codes` is the first of the rows' 128-byte lines; s0, s1 (z0, z1) the slab's
// scales (zero points) of rows g and g + 8, of which `left` bytes are K's.
template <int KIND, bool BF16, int TOK, bool BULK, int NT = Shape<TOK>::NT>
__device__ __forceinline__ void rows16(const uint8_t* codes, const uint8_t* s0, const uint8_t* s1, const uint8_t* z0,
                                       const uint8_t* z1, int left, int lane, const uint32_t (&frag)[8][NT][4],
                                       const float (&undo)[NT][2], float (&acc)[NT][4]) {
  constexpr int STEP = Shape<TOK>::STEP;
  constexpr int W = scale_bytes(KIND) / 4;
  const uint32_t g = lane >> 2, c = lane & 3;
  // row g's chunk ch (32 of K, 16 bytes) lies at chunk ch ^ (g & 7)
  const uint32_t code = 144u * g + 4u * c;
  uint32_t w0[W], w1[W];
  scale_words<W, BULK>(s0, left, w0);
  scale_words<W, BULK>(s1, left, w1);
  if constexpr (KIND == K_NVF4) {
    // unsigned E4M3: a byte with the top bit set is NaN (0xFF)
    if ((w0[0] | w0[1] | w0[2] | w0[3] | w1[0] | w1[1] | w1[2] | w1[3]) & 0x80808080u) {
#pragma unroll
      for (int i = 0; i < W; ++i) {
        const uint32_t t0 = w0[i] & 0x80808080u, t1 = w1[i] & 0x80808080u;
        w0[i] |= t0 - (t0 >> 7);
        w1[i] |= t1 - (t1 >> 7);
      }
    }
    // scales go into the codes: two chains over the slab (one mma waits for
    // the last of its chain).  The lanes with c < 2 hold the codes of the
    // chunk's first group.
    const uint32_t pick = c < 2 ? 0x1010u : 0x3232u;
    float sum[2][NT][4];
#pragma unroll
    for (int ch = 0; ch < 8; ++ch) {
      const uint32_t at = code ^ (16u * ch);
      uint32_t h0[4], h1[4], f0, f1;
      e2m1_word(lds<uint32_t>(codes, at), h0);
      e2m1_word(lds<uint32_t>(codes, at + 1024), h1);
      if (ch & 1) {
        asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, b;\n\t}" : "=r"(f0) : "r"(w0[ch / 2]));
        asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, b;\n\t}" : "=r"(f1) : "r"(w1[ch / 2]));
      } else {
        asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t}" : "=r"(f0) : "r"(w0[ch / 2]));
        asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t}" : "=r"(f1) : "r"(w1[ch / 2]));
      }
      f0 = __byte_perm(f0, 0, pick);
      f1 = __byte_perm(f1, 0, pick);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        h0[i] = hmul2(h0[i], f0);
        h1[i] = hmul2(h1[i], f1);
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        if (ch == 0) {
          mma16816_zero(sum[0][nt], h0[0], h1[0], h0[1], h1[1], frag[ch][nt][0], frag[ch][nt][1]);
          mma16816_zero(sum[1][nt], h0[2], h1[2], h0[3], h1[3], frag[ch][nt][2], frag[ch][nt][3]);
        } else {
          mma16816(sum[0][nt], h0[0], h1[0], h0[1], h1[1], frag[ch][nt][0], frag[ch][nt][1]);
          mma16816(sum[1][nt], h0[2], h1[2], h0[3], h1[3], frag[ch][nt][2], frag[ch][nt][3]);
        }
      }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; i += STEP) {
        const float v = sum[0][nt][i] + sum[1][nt][i];
        acc[nt][i] = BF16 ? v * undo[nt][i & 1] : v;
      }
  } else {
    constexpr int PER = group_of_kind(KIND) / 32;  // chunks per scale
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[nt][i] = 0.0f;
    uint32_t y0 = 0x64086408u, y1 = y0, n0 = 0xD480D480u, n1 = n0;  // 1024 + zero, -(64 + zero), zero 8
    float part[2][NT][4];
#pragma unroll
    for (int ch = 0; ch < 8; ++ch) {
      const uint32_t at = code ^ (16u * ch);
      constexpr uint32_t K960 = 0x63806380u;
      const int gi = ch / PER;
      uint32_t h0[4], h1[4];
      const uint32_t c0 = lds<uint32_t>(codes, at), c1 = lds<uint32_t>(codes, at + 1024);
      if constexpr (KIND == K_MXF4) {
        e2m1_word(c0, h0);
        e2m1_word(c1, h1);
      } else {
        if (ch % PER == 0 && z0) {
          y0 = 0x64006400u + lds<uint8_t>(z0, gi) * 0x10001u;
          y1 = 0x64006400u + lds<uint8_t>(z1, gi) * 0x10001u;
          n0 = hsub2(K960, y0);
          n1 = hsub2(K960, y1);
        }
        int4_word(c0, y0, n0, h0);
        int4_word(c1, y1, n1, h1);
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        if (ch % PER == 0) {
          mma16816_zero(part[0][nt], h0[0], h1[0], h0[1], h1[1], frag[ch][nt][0], frag[ch][nt][1]);
          mma16816_zero(part[1][nt], h0[2], h1[2], h0[3], h1[3], frag[ch][nt][2], frag[ch][nt][3]);
        } else {
          mma16816(part[0][nt], h0[0], h1[0], h0[1], h1[1], frag[ch][nt][0], frag[ch][nt][1]);
          mma16816(part[1][nt], h0[2], h1[2], h0[3], h1[3], frag[ch][nt][2], frag[ch][nt][3]);
        }
      }
      if (ch % PER == PER - 1) {
        float f0, f1;
        if constexpr (KIND == K_MXF4) {
          // both rows' e8m0 bytes to bf16 pairs, exact (0 is 2^-127, 255 NaN)
          const uint32_t pair = __byte_perm(w0[gi / 4], w1[gi / 4], (gi & 3) | ((4 + (gi & 3)) << 4));
          uint32_t f;
          asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.bf16x2.ue8m0x2 %0, a;\n\t}" : "=r"(f) : "r"(pair));
          f0 = __uint_as_float(f << 16);
          f1 = __uint_as_float(f & 0xFFFF0000u);
        } else if (BF16) {
          f0 = __uint_as_float((gi & 1) ? w0[gi / 2] & 0xFFFF0000u : w0[gi / 2] << 16);
          f1 = __uint_as_float((gi & 1) ? w1[gi / 2] & 0xFFFF0000u : w1[gi / 2] << 16);
        } else {
          f0 = half_bits((gi & 1) ? w0[gi / 2] >> 16 : w0[gi / 2]);
          f1 = half_bits((gi & 1) ? w1[gi / 2] >> 16 : w1[gi / 2]);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; i += STEP) {
            const float v = part[0][nt][i] + part[1][nt][i];
            acc[nt][i] += (BF16 ? v * undo[nt][i & 1] : v) * (i < 2 ? f0 : f1);
          }
      }
    }
  }
}

// A CTA's tiles in order: chunks of tiles, for each its passes over K, for
// each the tiles.  Without a second pass all tiles are one chunk.
template <int CAP>
struct Cursor {
  int chunk, pos, end;   // grains, counted over the row blocks
  int i, pass;           // tile within the chunk, pass
  int block, n0, rows;   // the tile: row block, first matrix row, rows (0: no more)

  __device__ __forceinline__ void locate(const GemvParams& p) {
    if (pos >= end) {
      rows = 0;
      return;
    }
    block = pos < p.grains ? 0 : pos / p.grains;
    n0 = (pos - block * p.grains) * GRAIN;
    rows = min(min(p.tile_rows, (end - pos) * GRAIN), p.N - n0);
  }
  __device__ __forceinline__ void next(const GemvParams& p, int passes) {
    pos += (rows + GRAIN - 1) / GRAIN;
    n0 += rows;
    ++i;
    if (passes > 1 && (pos >= end || i == CAP)) {
      i = 0;
      if (++pass < passes) {
        pos = chunk;
      } else {
        pass = 0;
        chunk = pos;
      }
      locate(p);
    } else if (n0 < p.N && pos < end) {  // further down the same matrix
      rows = min(min(p.tile_rows, (end - pos) * GRAIN), p.N - n0);
    } else {
      locate(p);
    }
  }
};

template <int TOK, bool BULK>
__device__ __forceinline__ void init_barriers(uint32_t bars, const GemvParams& p) {
  using S = Shape<TOK>;
  const int active = p.across * p.down;
  for (int i = 0; i < S::STAGES; ++i) {
    mbar_init(bars + 8 * i, BULK ? 1 : 34);  // the copies' bytes, twice; each lane's that copies words
    mbar_init(bars + 8 * (S::STAGES + i), active);
  }
  for (int i = 0; i < S::PARTS; ++i) {
    mbar_init(bars + 8 * (2 * S::STAGES + i), active);
    mbar_init(bars + 8 * (2 * S::STAGES + S::PARTS + i), 1);
  }
  fence_mbarrier_init();
}

// A CTA's share of the matrix rows, by all its warps.  `blocks` row blocks.
template <int KIND, bool BF16, int TOK, bool BULK, bool BANDS>
__device__ __forceinline__ void do_share(const GemvParams& p, uint8_t* smem, const int* seg, const int* pre, bool single,
                                         int2 span, int blocks) {
  using S = Shape<TOK>;
  constexpr int WARPS = S::WARPS, NT = S::NT, STAGES = S::STAGES, PARTS = S::PARTS, ADD_WARPS = S::ADD_WARPS;
  const uint32_t base = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t* flags = reinterpret_cast<uint32_t*>(smem + S::SEG - 8);  // abort, unusual
  const WaitCtx wctx{p.timeout_ns, p.err, flags};
  const uint32_t full = base + S::BARS + (BANDS ? S::BAR_BYTES : 0), empty = full + 8 * STAGES,
                 part_full = empty + 8 * STAGES, part_free = part_full + 8 * PARTS;
  const int active = p.across * p.down;  // decoding warps at work
  // a CTA's share of the grains; the slab of a warp in pass i is its column + i * across
  const int ctas = static_cast<int>(gridDim.x), cta = static_cast<int>(blockIdx.x), passes = p.passes;
  const int total = blocks * p.grains, share = blocks == p.blocks ? p.share : total / ctas, more = total - share * ctas;
  Cursor<S::CAP> cu;
  cu.chunk = cu.pos = cta * share + min(cta, more);
  cu.end = cu.pos + share + (cta < more ? 1 : 0);
  cu.i = cu.pass = cu.block = cu.n0 = 0;
  cu.locate(p);
  bool ok = true;

  constexpr int SB = scale_bytes(KIND), ZB = SLAB / group_of_kind(KIND);  // a row's scales, zero points of a slab
  constexpr int ES = is_int4(KIND) ? 2 : 1;
  const int stage_rows = STAGE_N * p.down;
  // bytes of a stage's rows of scales, zero points
  const int want_s = p.across * SB, want_z = p.across * ZB;
  const bool has_zero = is_int4(KIND) && p.zero;
  if (warp == WARPS || (!BULK && warp == WARPS + 1 + ADD_WARPS)) {
    // -------------------------------------------------------------- feeding
    const bool copies = !BULK && warp != WARPS;  // scales and zero points that TMA cannot bring
    int group = 0, block = -1;
    uint32_t stage = 0, ph = 1;
    const uint32_t box = stage_rows * (SLAB / 2);  // a slab's codes
    const uint32_t bytes =
        p.across * box + (BULK ? stage_rows * ((want_s + p.box_s - 1) / p.box_s * p.box_s + (has_zero ? p.box_z : 0)) : 0);
    for (; cu.rows; cu.next(p, passes)) {
      if (cu.block != block) {
        block = cu.block;
        group = p.G == 1 ? 0 : row_block<TOK>(p, seg, pre, false, span, block).g;
      }
      const int first = cu.pass * p.across;  // slab
      const bool part = p.K % SLAB && cu.pass == passes - 1;
#pragma unroll 1
      for (int h = 0; h < cu.rows; h += stage_rows) {
        const int n0 = cu.n0 + h;
        const uint32_t bar = full + 8 * stage, codes = base + stage * S::CODE_BYTES;
        const uint32_t sdst = base + S::SCALES + stage * SCALE_STAGE, zdst = sdst + ZERO_OFF;
        ok = wait_uniform(empty + 8 * stage, ph, wctx, SITE_PROD_EMPTY);  // the stage's last readers
        if (!ok) break;
        if (!copies) {
          if (elect_one()) {
            mbar_arrive_expect_tx(bar, bytes);
            // (a part of a slab goes with the whole ones before it when K is one
            // pass; the last of several passes takes slab by slab, below)
            if (!part || (passes == 1 && p.slabs > 1)) tma_load_4d(codes, &p.tmap_b, 0, n0, first, group, bar);
            if (part && passes == 1)
              tma_load3<1>(codes + (p.slabs - 1) * box, &p.tmap_part, (p.slabs - 1) * (SLAB / 2), n0, group, bar);
            if (BULK) {
              for (int x = 0; x < want_s; x += p.box_s)
                tma_load3<1>(sdst + stage_rows * x, &p.tmap_s, first * SB + x, n0, group, bar);
              if (has_zero) tma_load3<1>(zdst, &p.tmap_z, first * ZB, n0, group, bar);
            }
          }
          __syncwarp();
          if (part && passes > 1 && lane < p.across)  // zeros beyond K
            tma_load3<1>(codes + lane * box, &p.tmap_part, (first + lane) * (SLAB / 2), n0, group, bar);
        } else {
          const int rows = min(stage_rows, cu.rows - h), runs = p.one_run ? 1 : rows;
          auto copy = [&](uint32_t dst, int pitch, const uint8_t* at, int64_t ld, int len) {
            if (p.one_run) len += (rows - 1) * pitch;
            uint32_t bulk_bytes = 0;
            for (int i = lane; i < runs; i += 32) bulk_bytes += copy_run(dst + i * pitch, at + i * ld, len, bar);
            return bulk_bytes;
          };
          uint32_t sent = copy(sdst, p.box_s, p.scale + group * p.stride_scale + n0 * p.ld_scale + first * SB, p.ld_scale,
                               min(want_s, p.scale_row * ES - first * SB));
          if (has_zero)
            sent += copy(zdst, p.box_z, p.zero + group * p.stride_zero + n0 * p.ld_zero + first * ZB, p.ld_zero,
                         min(want_z, p.scale_row - first * ZB));
          sent = __reduce_add_sync(0xffffffffu, sent);
          if (lane == 0) mbar_arrive_expect_tx(bar, sent);
          asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
        }
        if (++stage == STAGES) {
          stage = 0;
          ph ^= 1u;
        }
      }
      if (!ok) break;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (!ok && lane == 0) {
      // let the copies in flight land before the CTA can exit
      const uint64_t t0 = globaltimer();
      while (globaltimer() - t0 < 2000000ull) {
      }
    }
  } else if (warp < WARPS) {
    // ------------------------------------------------------------- decoding
    const int below = warp / p.across, wk = warp - below * p.across;
    const int g = lane >> 2, c = lane & 3, row = STAGE_N * below + g;
    if (warp >= active) cu.rows = 0;
    uint32_t frag[8][NT][4];
    float undo[NT][2], after[NT][2];
    // BANDS: a tile is gone through for each band, upwards, the next one down
    int band = 0, have_band = 0;
    bool rising = true, later = false, first = true, more = false;
    int have_block = -1, have_pass = -1, group = 0;  // whose fragments are loaded
    uint32_t stage = 0, ph = 0, buf = 0, buf_ph = ~0u;  // buf_ph: a parity bit per buffer
    const uint8_t* codes0 = smem + (wk * stage_rows + STAGE_N * below) * (SLAB / 2);
    const uint8_t *scales0 = smem + S::SCALES, *zeros0 = scales0 + ZERO_OFF;
    const int to_s1 = 8 * p.box_s, to_z1 = 8 * p.box_z;  // from row g to row g + 8
    if (BULK) {
      // 128 bytes of a row to a box; a box's rows 8 apart are swizzled alike
      const uint32_t x = wk * SB;
      scales0 += (x >> 7) * (stage_rows * 128) + box_at(row, x & 127u, p.box_s);
      zeros0 += box_at(row, wk * ZB, p.box_z);
    } else {
      scales0 += row * p.box_s + wk * SB;
      zeros0 += row * p.box_z + wk * ZB;
    }
    float* part0 = reinterpret_cast<float*>(smem + S::PART) + warp * S::TILE_PART +
                   (TOK == 4 ? c : 2 * c) * S::PART_PITCH + g;
    while (cu.rows) {
      if (have_block != cu.block || have_pass != cu.pass || (BANDS && have_band != band)) {
        const RowBlock rb = row_block<TOK>(p, seg, pre, single, span, cu.block);
        group = rb.g;
        have_block = cu.block;
        have_pass = cu.pass;
        if constexpr (BANDS) {
          if (have_band == band) {  // other activations
            band = 0;
            rising = true;
          }
          have_band = band;
          later = load_band<KIND, TOK>(p, rb, wk + cu.pass * p.across, band, lane, frag, undo, after);
        } else {
          load_fragments<KIND, BF16, TOK>(p, rb, wk + cu.pass * p.across, lane, smem + S::ACT + warp * S::ACT_BYTES,
                                         flags + 1, frag, undo);
        }
      }
      if (BANDS) more = rising ? later : band > 0;
      const int slab = wk + cu.pass * p.across;
#pragma unroll 1
      for (int h = 0; h < cu.rows; h += stage_rows) {
        ok = wait_uniform(full + 8 * stage, ph, wctx, SITE_MMA_FULL);
        if (!ok) break;
        float acc[NT][4] = {};
        if (slab < p.slabs && h + STAGE_N * below < cu.rows) {
          const uint8_t *s0 = scales0 + stage * SCALE_STAGE, *s1 = s0 + to_s1;
          const uint8_t *z0 = nullptr, *z1 = nullptr;
          if (has_zero) {
            z0 = zeros0 + stage * SCALE_STAGE;
            z1 = z0 + to_z1;
          }
          if (!BULK) {
            // each row, or the stage, starts as far past a 16-byte boundary as in memory
            const uint32_t first = static_cast<uint32_t>(cu.pass * p.across), n0 = static_cast<uint32_t>(cu.n0 + h);
            const uint32_t below_s = p.one_run ? 0 : static_cast<uint32_t>(p.ld_scale);
            const uint32_t at = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p.scale)) + first * SB +
                                n0 * static_cast<uint32_t>(p.ld_scale) + row * below_s +
                                static_cast<uint32_t>(group) * static_cast<uint32_t>(p.stride_scale);
            s0 += at & 15u;
            s1 += (at + 8u * below_s) & 15u;
            if (has_zero) {
              const uint32_t below_z = p.one_run ? 0 : static_cast<uint32_t>(p.ld_zero);
              const uint32_t zat = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p.zero)) + first * ZB +
                                   n0 * static_cast<uint32_t>(p.ld_zero) + row * below_z +
                                   static_cast<uint32_t>(group) * static_cast<uint32_t>(p.stride_zero);
              z0 += zat & 15u;
              z1 += (zat + 8u * below_z) & 15u;
            }
          }
          rows16<KIND, BF16, TOK, BULK>(codes0 + stage * S::CODE_BYTES, s0, s1, z0, z1, p.scale_row * ES - slab * SB, lane, frag, undo, acc);
        }
        __syncwarp();
        if (lane == 0 && !more) mbar_arrive(empty + 8 * stage);
        if (++stage == STAGES) {
          stage = 0;
          ph ^= 1u;
        }
        if (h == 0) {  // the buffer its parts go to
          ok = wait_uniform(part_free + 8 * buf, (buf_ph >> buf) & 1u, wctx, SITE_MMA_ACC_EMPTY);
          if (!ok) break;
        }
        float* mine = part0 + buf * (WARPS * S::TILE_PART) + (h ? STAGE_N : 0);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; i += S::STEP) {
            float& part = mine[(8 * nt + (i & 1)) * S::PART_PITCH + 8 * (i >> 1)];
            part = BANDS ? fmaf(acc[nt][i], after[nt][i & 1], first ? 0.0f : part) : acc[nt][i];
          }
      }
      if (!ok) break;
      if (BANDS && more) {  // the tile's stages again
        for (int h = 0; h < cu.rows; h += stage_rows) {
          ph ^= stage == 0 ? 1u : 0u;
          stage = stage == 0 ? STAGES - 1 : stage - 1;
        }
        band += rising ? 1 : -1;
        first = false;
        continue;
      }
      rising = !rising;
      first = true;
      __syncwarp();
      if (lane == 0) mbar_arrive(part_full + 8 * buf);
      buf_ph ^= 1u << buf;
      cu.next(p, passes);
      if (++buf == PARTS || cu.i == 0) buf = 0;
    }
  } else {
    // --------------------------------------------------------------- adding
    const int me = warp - (WARPS + 1);
    const float* parts0 = reinterpret_cast<const float*>(smem + S::PART);
    float* sums = reinterpret_cast<float*>(smem + S::SUM);
    uint32_t parity = 0;
    RowBlock o{0, 0, 0};
    int block = -1;
    float alpha = 1.0f;
    for (; ok && cu.rows; cu.next(p, passes)) {
      const int buf = cu.i % PARTS;
      if (buf != me) continue;
      if (cu.block != block) {
        block = cu.block;
        o = row_block<TOK>(p, seg, pre, single, span, block);
        if (p.alpha) alpha = p.alpha[o.g];
      }
      ok = wait_uniform(part_full + 8 * buf, parity, wctx, SITE_EPI_ACC_FULL);
      if (!ok) break;
      parity ^= 1u;
#pragma unroll 1
      for (int below = 0; below < p.down; ++below) {
        // 32 rows of the tile: 16 of each stage
        const float* parts = parts0 + (buf * WARPS + below * p.across) * S::TILE_PART;
#pragma unroll
        for (int j0 = 0; j0 < S::OUT; j0 += 128) {
          constexpr int LANES = S::TILE_N / 4;  // lanes an activation row takes
          const int row = j0 / S::TILE_N + lane / LANES, n = 4 * (lane % LANES);
          const float4* at = reinterpret_cast<const float4*>(parts + (row < TOK ? row : 0) * S::PART_PITCH + n);
          float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
          for (int w = 0; w < p.across; ++w) {
            const float4 v = at[w * (S::TILE_PART / 4)];
            s.x += v.x;
            s.y += v.y;
            s.z += v.z;
            s.w += v.w;
          }
          if (row < TOK && passes > 1) {
            float4* keep = reinterpret_cast<float4*>(sums + cu.i * S::OUT + j0 + 4 * lane);
            if (cu.pass > 0) {
              const float4 v = *keep;
              s.x += v.x;
              s.y += v.y;
              s.z += v.z;
              s.w += v.w;
            }
            *keep = s;
          }
          if (cu.pass == passes - 1 && row < o.rows) {
            const int first = (n < STAGE_N ? n : n + stage_rows - STAGE_N) + STAGE_N * below;  // row of the tile
            const int64_t d = (o.row0 + row) * p.ldd + cu.n0 + first;
            const float v[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (first + k < cu.rows) store_d(p, d + k, v[k] * alpha);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(part_free + 8 * buf);
    }
    if (!BANDS && p.offsets) {  // rows of no group give zero
      const int first = single ? span.x : seg[0], end = single ? span.y : seg[p.G];
#pragma unroll 1
      for (int r = blockIdx.x; r < p.R; r += gridDim.x) {
        if (r >= first && r < end) continue;
#pragma unroll 1
        for (int n = threadIdx.x - 32 * (WARPS + 1); n < p.N; n += 32 * ADD_WARPS) store_d(p, r * p.ldd + n, 0.0f);
      }
    }
  }
}

__device__ __forceinline__ uint8_t* aligned_smem() {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  return smem_raw + (((raw + 1023u) & ~1023u) - raw);
}

// One group of few rows: its block is there whatever the offsets say, and the
// codes need not wait for them.
template <int TOK>
__device__ __forceinline__ bool single_block(const GemvParams& p, int2* span) {
  const bool single = p.offsets && p.G == 1 && p.R <= TOK;
  *span = make_int2(0, 0);
  if (single) {
    span->x = min(max(p.offsets[0], 0), p.R);
    span->y = min(max(p.offsets[1], span->x), p.R);
  }
  return single;
}

// The share once more, since a warp has met a slab that is not usual.  (Apart,
// and with nothing kept for it: with what bands need in one loop with the
// others, that took 4 to 10 % more.)
template <int KIND, int TOK, bool BULK>
__device__ __noinline__ void do_share_in_bands(const GemvParams& p) {
  using S = Shape<TOK>;
  uint8_t* smem = aligned_smem();
  if (threadIdx.x == 0) init_barriers<TOK, BULK>(smem_u32(smem) + S::BARS + S::BAR_BYTES, p);
  __syncthreads();
  const int* seg = reinterpret_cast<const int*>(smem + S::SEG);
  const int* pre = seg + p.G + 1;
  int2 span;
  const bool single = single_block<TOK>(p, &span);
  do_share<KIND, true, TOK, BULK, true>(p, smem, seg, pre, single, span,
                                        single ? 1 : p.offsets ? pre[p.G] : (p.R + TOK - 1) / TOK);
}

// BULK: scales and zero points come by TMA (a runtime choice took 5 to 8 % of
// the kernel's time).
template <int KIND, bool BF16, int TOK, bool BULK>
__global__ void __launch_bounds__(Shape<TOK>::threads(BULK), 1) gemv_kernel(const __grid_constant__ GemvParams p) {
  using S = Shape<TOK>;
  uint8_t* smem = aligned_smem();
  volatile uint32_t* flags = reinterpret_cast<uint32_t*>(smem + S::SEG - 8);  // abort, unusual
  int* seg = reinterpret_cast<int*>(smem + S::SEG);
  int* pre = seg + p.G + 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    init_barriers<TOK, BULK>(smem_u32(smem) + S::BARS, p);
    flags[0] = flags[1] = 0u;
  }
  __syncthreads();
  griddep_wait();
  griddep_launch_dependents();
  int2 span;
  const bool single = single_block<TOK>(p, &span);
  int blocks;
  if (single) {
    blocks = 1;
  } else if (p.offsets) {
    if (warp == S::WARPS) {  // clamp to [previous, R]; row blocks before each group; four groups a lane
      int run_max = 0, run_blocks = 0;
#pragma unroll 1
      for (int i0 = 0; i0 <= p.G; i0 += 128) {
        int v[4], n[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int i = i0 + 4 * lane + k;
          v[k] = i <= p.G ? p.offsets[i] : 0;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          v[k] = min(max(v[k], 0), p.R);
          if (k) v[k] = max(v[k], v[k - 1]);
        }
        int top = v[3];
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int o = __shfl_up_sync(0xffffffffu, top, d);
          if (lane >= d) top = max(top, o);
        }
        int before = __shfl_up_sync(0xffffffffu, top, 1);
        before = lane == 0 ? run_max : max(before, run_max);
        int sum = 0, last = before;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int i = i0 + 4 * lane + k;
          v[k] = max(v[k], before);
          sum += i >= 1 && i <= p.G ? (v[k] - last + TOK - 1) / TOK : 0;
          last = v[k];
          n[k] = sum;
        }
        int all = sum;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int o = __shfl_up_sync(0xffffffffu, all, d);
          if (lane >= d) all += o;
        }
        const int mine = run_blocks + all - sum;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int i = i0 + 4 * lane + k;
          if (i <= p.G) {
            seg[i] = v[k];
            pre[i] = mine + n[k];
          }
        }
        run_max = max(run_max, __shfl_sync(0xffffffffu, top, 31));
        run_blocks += __shfl_sync(0xffffffffu, all, 31);
      }
    }
    __syncthreads();
    blocks = pre[p.G];
  } else {
    blocks = (p.R + TOK - 1) / TOK;
  }

  do_share<KIND, BF16, TOK, BULK, false>(p, smem, seg, pre, single, span, blocks);
  if constexpr (BF16) {
    __syncthreads();
    volatile uint32_t* f = reinterpret_cast<uint32_t*>(aligned_smem() + S::SEG - 8);
    if (f[1] && !f[0]) do_share_in_bands<KIND, TOK, BULK>(p);
  }
}

// Index of a variant: Kind4, bf16, TOK (4, 8, 16).
constexpr int SHAPES = 3, VARIANTS = KINDS4 * 2 * SHAPES;
constexpr int shape_index(int tok) { return tok == 16 ? 2 : tok == 8 ? 1 : 0; }

template <int KIND, bool BULK>
void fill(const void** k) {
  const auto f = [](void (*kernel)(GemvParams)) { return reinterpret_cast<const void*>(kernel); };
  k += KIND * 2 * SHAPES;
  k[0] = f(gemv_kernel<KIND, false, 4, BULK>);
  k[1] = f(gemv_kernel<KIND, false, 8, BULK>);
  k[2] = f(gemv_kernel<KIND, false, 16, BULK>);
  k[3] = f(gemv_kernel<KIND, true, 4, BULK>);
  k[4] = f(gemv_kernel<KIND, true, 8, BULK>);
  k[5] = f(gemv_kernel<KIND, true, 16, BULK>);
}

template <bool BULK>
struct Variants {
  const void* k[VARIANTS];
  Variants() {
    fill<K_INT4_32, BULK>(k);
    fill<K_INT4_64, BULK>(k);
    fill<K_INT4_128, BULK>(k);
    fill<K_MXF4, BULK>(k);
    fill<K_NVF4, BULK>(k);
  }
};

}  // namespace

// The variants whose scales come as runs (a translation unit of their own).
const void* w4_runs_kernel(int variant);

}  // namespace tcg
