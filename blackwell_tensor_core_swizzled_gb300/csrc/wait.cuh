// A bounded barrier wait for kernels whose warps keep many registers or wait often.
#pragma once

#include <cstdint>

#include "gemm_kernel.cuh"
#include "ptx.cuh"

namespace tcg {

// wait_uniform without a function call (across which sums would be kept in local
// memory), and without the global timer until it has spun a while: its read took
// some 500 cycles of each wait that was not over at once.
__device__ __forceinline__ bool wait_inline(uint32_t bar, uint32_t parity, const WaitCtx& w, uint32_t site) {
  bool ok = mbar_try_wait(bar, parity);
  if (__all_sync(0xffffffffu, ok)) return true;
#pragma unroll 1
  for (int i = 0; i < 64 && !ok; ++i) ok = mbar_try_wait(bar, parity);
  if (__all_sync(0xffffffffu, ok)) return true;
  const uint64_t t0 = globaltimer();
  while (!ok) {
#pragma unroll 1
    for (int i = 0; i < 32 && !ok; ++i) ok = mbar_try_wait(bar, parity);
    if (ok || *w.abort_flag) break;
    if (globaltimer() - t0 > w.timeout_ns) {
      *w.abort_flag = 1u;
      if (w.err) atomicCAS(w.err, 0ull, make_err(1u, site));
      break;
    }
  }
  return __all_sync(0xffffffffu, ok);
}

}  // namespace tcg
