#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <mutex>

#include "status.h"
#include "tensor_map.h"

namespace gtp {

namespace {
PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
std::once_flag g_once;
cudaError_t g_lookup_err = cudaSuccess;
}  // namespace

gtp_status encode_tmap_3d(CUtensorMap *map, CUtensorMapDataType dtype, const void *base, uint64_t inner,
                          uint64_t middle, uint64_t outer, uint64_t row_stride_bytes, uint64_t plane_stride_bytes,
                          uint32_t box_inner, uint32_t box_middle, uint32_t box_outer) {
  std::call_once(g_once, [] {
    void *fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    g_lookup_err = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q);
    if (g_lookup_err == cudaSuccess && q == cudaDriverEntryPointSuccess)
      g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  });
  if (!g_encode) return fail(GTP_E_CUDA, "cuTensorMapEncodeTiled unavailable (%s)", cudaGetErrorString(g_lookup_err));
  const cuuint64_t dims[3] = {inner, middle, outer};
  const cuuint64_t strides[2] = {row_stride_bytes, plane_stride_bytes};
  const cuuint32_t box[3] = {box_inner, box_middle, box_outer};
  const cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = g_encode(map, dtype, 3, const_cast<void *>(base), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS)
    return fail(GTP_E_CUDA, "cuTensorMapEncodeTiled failed (%d): dims %llu x %llu x %llu, box %u x %u x %u", int(r),
                (unsigned long long)inner, (unsigned long long)middle, (unsigned long long)outer, box_inner, box_middle,
                box_outer);
  return GTP_OK;
}

}  // namespace gtp
