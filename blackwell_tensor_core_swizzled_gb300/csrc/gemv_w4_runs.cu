// The 4-bit products whose scales or zero points TMA cannot tile.
#include "gemv_w4.cuh"

namespace tcg {

namespace {
const Variants<false> g_runs;
}

const void* w4_runs_kernel(int variant) { return g_runs.k[variant]; }

}  // namespace tcg
