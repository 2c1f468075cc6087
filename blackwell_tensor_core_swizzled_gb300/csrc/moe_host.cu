// Host side that the mixture-of-experts operators share: tensor maps, and what
// a device holds of their kernels.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <map>
#include <mutex>
#include <string>

#include "common.h"

namespace tcg {

namespace {

constexpr int MAX_DEVICES = 64;
struct Device {
  int sms = 0;
  std::map<const void*, int> clusters;  // by kernel
};
std::mutex g_mu;
Device g_devices[MAX_DEVICES];

PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
std::once_flag g_encode_once;

bool encode_ready() {
  std::call_once(g_encode_once, [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    else
      cudaGetLastError();
  });
  return g_encode != nullptr;
}

// Tiled map swizzled over `span` bytes (128, 64, 32 or, not at all, 0), encoded
// on every call
int encode_tiled(CUtensorMap* map, CUtensorMapDataType dt, int rank, const void* base, const cuuint64_t* dims,
                 const cuuint64_t* strides, const cuuint32_t* box, uint32_t span = 128) {
  if (!encode_ready()) {
    set_error_message("cuTensorMapEncodeTiled entry point unavailable");
    return TCG_ERR_CUDA;
  }
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  const CUresult r = g_encode(map, dt, static_cast<cuuint32_t>(rank), const_cast<void*>(base), dims, strides, box, estr,
                              CU_TENSOR_MAP_INTERLEAVE_NONE,
                              span == 128  ? CU_TENSOR_MAP_SWIZZLE_128B
                              : span == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                              : span == 32 ? CU_TENSOR_MAP_SWIZZLE_32B
                                           : CU_TENSOR_MAP_SWIZZLE_NONE,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) {
    set_error_message(("cuTensorMapEncodeTiled (rank " + std::to_string(rank) + ") failed (" +
                       std::to_string(static_cast<int>(r)) + ")")
                          .c_str());
    return TCG_ERR_CUDA;
  }
  return TCG_OK;
}

}  // namespace

int make_operand_map(CUtensorMap* map, const void* base, bool bf16, uint64_t inner, uint64_t mid, uint64_t outer,
                     uint64_t stride_mid, uint64_t stride_outer, uint32_t box_mid) {
  const cuuint64_t dims[3] = {inner, mid, outer}, strides[2] = {2 * stride_mid, 2 * stride_outer};
  const cuuint32_t box[3] = {64, box_mid, 1};
  return encode_tiled(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, outer ? 3 : 2,
                      base, dims, strides, box);
}

int make_byte_map(CUtensorMap* map, const void* base, uint64_t inner, uint64_t mid, uint64_t outer,
                  uint64_t stride_mid, uint64_t stride_outer, uint32_t box_inner, uint32_t box_mid) {
  const cuuint64_t dims[3] = {inner, mid, outer}, strides[2] = {stride_mid, stride_outer};
  const cuuint32_t box[3] = {box_inner, box_mid, 1};
  return encode_tiled(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, base, dims, strides, box, box_inner);
}

int make_store_map(CUtensorMap* map, const void* base, tcg_dtype type, uint64_t inner, uint64_t mid, uint64_t outer,
                   uint64_t stride_mid, uint64_t stride_outer) {
  const bool f32 = type == TCG_F32;
  const uint64_t size = f32 ? 4 : 2;
  const cuuint64_t dims[3] = {inner, mid, outer}, strides[2] = {size * stride_mid, size * stride_outer};
  const cuuint32_t box[3] = {32, f32 ? 16u : 32u, 1};
  return encode_tiled(map,
                      f32                ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                      : type == TCG_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                         : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                      3, base, dims, strides, box, f32 ? 0 : 64);
}

int make_slab_map(CUtensorMap* map, const void* base, uint64_t inner, uint64_t mid, uint64_t slabs, uint64_t outer,
                  uint64_t stride_mid, uint64_t stride_outer, uint32_t box_mid, uint32_t box_slabs) {
  const cuuint64_t dims[4] = {inner, mid, slabs, outer}, strides[3] = {stride_mid, inner, stride_outer};
  const cuuint32_t box[4] = {static_cast<cuuint32_t>(inner), box_mid, box_slabs, 1};
  return encode_tiled(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, base, dims, strides, box);
}

int device_sms(int dev) {
  std::lock_guard<std::mutex> lk(g_mu);
  Device& d = g_devices[dev];
  if (d.sms == 0 && cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    d.sms = 0;
    return 1;
  }
  return d.sms;
}

int max_resident_clusters(int dev, const KernelInfo& ki, int* out) {
  const int sms = device_sms(dev);
  std::lock_guard<std::mutex> lk(g_mu);
  auto& known = g_devices[dev].clusters;
  const auto it = known.find(ki.func);
  if (it != known.end()) {
    *out = it->second;
    return TCG_OK;
  }
  if (int rc = record_cuda(cudaFuncSetAttribute(ki.func, cudaFuncAttributeMaxDynamicSharedMemorySize, ki.smem_bytes)))
    return rc;
  int n = std::max(1, sms / ki.cta_group);
  if (ki.cta_group > 1) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ki.cta_group * n), 1, 1);
    cfg.blockDim = dim3(static_cast<unsigned>(ki.threads), 1, 1);
    cfg.dynamicSmemBytes = static_cast<size_t>(ki.smem_bytes);
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = static_cast<unsigned>(ki.cta_group);
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int fit = 0;
    if (int rc = record_cuda(cudaOccupancyMaxActiveClusters(&fit, ki.func, &cfg))) return rc;
    n = std::max(1, std::min(n, fit));
  }
  known[ki.func] = n;
  *out = n;
  return TCG_OK;
}

}  // namespace tcg
