// Few rows of 16-bit activations against 4-bit matrices with group scales:
// entry point and host plan.  The contract is in include/tcg.h.
#include "gemv_w4.cuh"
#include "once.h"

namespace tcg {

namespace {

// ---------------------------------------------------------------------- host

const Variants<true> g_variants;
constexpr int SHAPE_SMEM[SHAPES] = {Shape<4>::BYTES, Shape<8>::BYTES, Shape<16>::BYTES};
constexpr int SHAPE_WARPS[SHAPES] = {Shape<4>::WARPS, Shape<8>::WARPS, Shape<16>::WARPS};
constexpr int SHAPE_THREADS[SHAPES] = {Shape<4>::threads(true), Shape<8>::threads(true), Shape<16>::threads(true)};
const void* variant(int i, bool bulk) { return bulk ? g_variants.k[i] : w4_runs_kernel(i); }

// Per device, on the first call: the variants' shared-memory attribute (all of
// them, 3 ms, so that no later call, one under capture say, loads a kernel).
OncePerDevice<cudaError_t> g_setup;

cudaError_t device_setup(int dev) {
  return g_setup(dev, [] {
    for (int i = 0; i < 2 * VARIANTS; ++i)
      if (const cudaError_t e =
              cudaFuncSetAttribute(variant(i / 2, i % 2 != 0), cudaFuncAttributeMaxDynamicSharedMemorySize,
                                   SHAPE_SMEM[i / 2 % SHAPES]))
        return e;
    return cudaSuccess;
  });
}

int run_gemv(const tcg_gemv_w4_args* args, cudaStream_t s) {
  begin_product();
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
    // with one group no stride is ever taken, but a tensor map wants an aligned one
    if (a.G == 1) a.stride_scale = a.N * a.ld_scale;
  }
  int dev;
  if (int rc = current_device_checked(&dev)) return rc;
  if (a.K == 0) {
    const size_t ds = a.d_type == TCG_F32 ? 4 : 2;
    if (int rc = record_cuda(cudaMemset2DAsync(a.D, static_cast<size_t>(a.ldd) * ds, 0, static_cast<size_t>(a.N) * ds,
                                               static_cast<size_t>(a.R), s)))
      return rc;
    set_launch_count(1);
    record_zero_plan();
    return TCG_OK;
  }
  GemvParams p;
  std::memset(&p, 0, sizeof p);
  const int es = a.format == TCG_W4_INT4 ? 2 : 1;
  p.R = static_cast<int>(a.R);
  p.N = static_cast<int>(a.N);
  p.K = static_cast<int>(a.K);
  p.G = a.G;
  p.A = static_cast<const uint8_t*>(a.A);
  p.lda = a.lda;
  p.offsets = a.offsets;
  p.scale = static_cast<const uint8_t*>(a.scale);
  p.ld_scale = a.ld_scale * es;
  p.stride_scale = a.stride_scale * es;
  p.scale_row = static_cast<int>(blocks_k);
  p.zero = a.zero;
  p.ld_zero = a.ld_scale;
  p.stride_zero = a.stride_scale;
  // boxes when rows are aligned, else runs of rows where they fit a stage (mxf4,
  // 1 row: 14000 x 4096 10.8 us in boxes, 14000 x 4000 11.8 in runs; nvf4, 32
  // experts: 4096 x 4096 67, 4000 x 4064 78; int4 with zero points, 16 rows:
  // 16384 x 8192 41, 16384 x 7968 54), else row by row (one token on 8192 x 8192
  // 25 us where boxes take 13, 64 experts 180 and 46)
  // (then K is a multiple of 256, and of so much that a pass's share of a row
  // is one of 16 bytes)
  const int64_t s_low = blocks_k * es | p.ld_scale | p.stride_scale |
                        static_cast<int64_t>(reinterpret_cast<uintptr_t>(a.scale));
  const int64_t z_low = blocks_k | p.ld_zero | p.stride_zero |
                        static_cast<int64_t>(reinterpret_cast<uintptr_t>(a.zero));
  p.bulk = s_low % 16 == 0 && (!a.zero || z_low % 16 == 0);
  p.alpha = a.alpha;
  p.D = a.D;
  p.d_type = a.d_type;
  p.ldd = a.ldd;
  p.grains = static_cast<int>((a.N + GRAIN - 1) / GRAIN);
  p.err = device_error_word(dev);
  p.timeout_ns = wait_timeout_ns();
  p.slabs = static_cast<int>((a.K + SLAB - 1) / SLAB);

  // rows per block: as many as the groups are expected to have (int4 16384 x
  // 8192: 4 rows 24 us in blocks of 4 or 8, 34 of 16; 5 rows 42, 25, 34; 8 rows
  // 44, 24, 35; 9 rows 63, 45, 35; 32 rows 150, 82, 66; nvf4 8192 x 4096: 8
  // rows 14.3, 10.8, 13.5; 16 rows 21.6, 15.0, 14.3).  Only the average is known
  // here: 32 rows on 64 nvf4 experts of 4096 x 4096 take 23 us in blocks of 4
  // when one expert has them all (16: 21), 24 on four (16: 26), 67 on 32 (16:
  // 112).
  const int64_t active = std::min<int64_t>(a.G, a.R);
  const int tok = a.R > 8 * active ? 16 : a.R > 4 * active ? 8 : 4;
  // (a block for every `tok` rows and one more per group there can be at most)
  if ((a.R / tok + active) * p.grains > INT32_MAX) return TCG_ERR_UNSUPPORTED;
  if (int rc = record_cuda(device_setup(dev))) return rc;
  const int warps = SHAPE_WARPS[shape_index(tok)];
  p.across = std::min(warps, p.slabs);
  // when K is short, the other warps go below: as far as every CTA still gets
  // that many rows, and their scales fit (int4 16384 x 1024: 8.3 us, 12.2 with
  // the other warps idle)
  const int64_t blocks = std::max(active, (a.R + tok - 1) / tok);
  const int64_t wanted = (blocks * a.N / device_sms(dev) + STAGE_N - 1) / STAGE_N;
  p.down = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(warps / p.across, wanted)));
  const auto box = [](int bytes) { return bytes <= 32 ? 32 : bytes <= 64 ? 64 : 128; };
  const auto pitch = [](int bytes) { return 16 * ((bytes + 30) / 16 | 1); };  // 16 bytes to spare; rows on different banks
  const int want_z = p.across * (SLAB / a.group), want_s = want_z * es;
  const int64_t room_s = a.zero ? ZERO_OFF : SCALE_STAGE, room_z = a.zero ? SCALE_STAGE - ZERO_OFF : INT64_MAX;
  // (up to 15 bytes before a run, and a word read past it)
  const auto fits = [&](int64_t row_s, int64_t row_z) {
    return STAGE_N * p.down * row_s + 19 <= room_s && STAGE_N * p.down * row_z + 19 <= room_z;
  };
  const int down = p.down;
  p.one_run = 0;
  if (!p.bulk) {
    while (p.down > 1 && !fits(p.ld_scale, p.ld_zero)) --p.down;
    p.one_run = fits(p.ld_scale, p.ld_zero);
  }
  p.box_s = p.bulk ? box(want_s) : p.one_run ? static_cast<int>(p.ld_scale) : pitch(want_s);
  p.box_z = p.bulk ? box(want_z) : p.one_run ? static_cast<int>(p.ld_zero) : pitch(want_z);
  if (!p.one_run) {
    p.down = down;
    while (p.down > 1 && !fits(p.box_s, p.box_z)) --p.down;
  }
  p.tile_rows = 2 * STAGE_N * p.down;
  const int stage_rows = STAGE_N * p.down;
  if (p.bulk) {
    if (int rc = make_byte_map(&p.tmap_s, a.scale, blocks_k * es, a.N, a.G, p.ld_scale, p.stride_scale, p.box_s, stage_rows))
      return rc;
    if (a.zero)
      if (int rc = make_byte_map(&p.tmap_z, a.zero, blocks_k, a.N, a.G, p.ld_zero, p.stride_zero, p.box_z, stage_rows))
        return rc;
  }
  const bool part = a.K % SLAB != 0;
  if (a.K >= SLAB) {
    const int slabs = part && p.slabs == p.across ? p.across - 1 : p.across;
    if (int rc = make_slab_map(&p.tmap_b, a.B, SLAB / 2, a.N, a.K / SLAB, a.G, a.ldb / 2, a.stride_b / 2, stage_rows, slabs))
      return rc;
  }
  if (part)
    if (int rc = make_byte_map(&p.tmap_part, a.B, a.K / 2, a.N, a.G, a.ldb / 2, a.stride_b / 2, SLAB / 2, stage_rows))
      return rc;
  const int kind = a.format == TCG_W4_MXF4   ? K_MXF4
                   : a.format == TCG_W4_NVF4 ? K_NVF4
                   : a.group == 32           ? K_INT4_32
                   : a.group == 64           ? K_INT4_64
                                             : K_INT4_128;
  const void* k = variant((kind * 2 + (a.in_type == TCG_IN_BF16 ? 1 : 0)) * SHAPES + shape_index(tok), p.bulk);
  cudaLaunchConfig_t cfg = {};
  const int64_t ctas = std::min<int64_t>(device_sms(dev), (a.R / tok + active) * p.grains);
  p.passes = (p.slabs + p.across - 1) / p.across;
  p.blocks = static_cast<int>(blocks);
  p.share = static_cast<int>(blocks * p.grains / ctas);
  cfg.gridDim = dim3(static_cast<unsigned>(ctas), 1, 1);
  cfg.blockDim = dim3(static_cast<unsigned>(SHAPE_THREADS[shape_index(tok)] + (p.bulk ? 0 : 32)), 1, 1);
  cfg.dynamicSmemBytes = SHAPE_SMEM[shape_index(tok)];
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  void* params[] = {&p};
  if (int rc = record_cuda(cudaLaunchKernelExC(&cfg, k, params))) return rc;
  set_launch_count(1);
  record_w4_plan(tok, p.across, p.down, static_cast<int>(ctas), p.bulk);
  return TCG_OK;
}

}  // namespace

}  // namespace tcg

using namespace tcg;

extern "C" int tcg_gemv_w4(const tcg_gemv_w4_args* args, void* stream) {
  return guarded([&] { return run_gemv(args, static_cast<cudaStream_t>(stream)); });
}
