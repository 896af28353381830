#include "tensor_map.h"

#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <mutex>

#include "status.h"

namespace gtp {

namespace {
PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
std::once_flag g_once;
cudaError_t g_lookup_err = cudaSuccess;

// Looks the driver's encoder up once, then encodes; the caller names the shape where it is refused.
gtp_status encode(CUresult *result, CUtensorMap *map, CUtensorMapDataType dtype, cuuint32_t rank, const void *base,
                  const cuuint64_t *dims, const cuuint64_t *strides, const cuuint32_t *box, CUtensorMapSwizzle swizzle) {
  std::call_once(g_once, [] {
    void *fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    g_lookup_err = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q);
    if (g_lookup_err == cudaSuccess && q == cudaDriverEntryPointSuccess)
      g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  });
  if (!g_encode) return fail(GTP_E_CUDA, "cuTensorMapEncodeTiled unavailable (%s)", cudaGetErrorString(g_lookup_err));
  const cuuint32_t estr[3] = {1, 1, 1};
  *result = g_encode(map, dtype, rank, const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                     swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return GTP_OK;
}
}  // namespace

gtp_status encode_tmap_2d(CUtensorMap *map, CUtensorMapDataType dtype, const void *base, uint64_t inner,
                          uint64_t outer, uint64_t row_stride_bytes, uint32_t box_inner, uint32_t box_outer,
                          CUtensorMapSwizzle swizzle) {
  const cuuint64_t dims[2] = {inner, outer};
  const cuuint64_t strides[1] = {row_stride_bytes};
  const cuuint32_t box[2] = {box_inner, box_outer};
  CUresult r;
  if (gtp_status s = encode(&r, map, dtype, 2, base, dims, strides, box, swizzle)) return s;
  if (r != CUDA_SUCCESS)
    return fail(GTP_E_CUDA, "cuTensorMapEncodeTiled failed (%d): dims %llu x %llu, stride %llu, box %u x %u", int(r),
                (unsigned long long)inner, (unsigned long long)outer, (unsigned long long)row_stride_bytes, box_inner,
                box_outer);
  return GTP_OK;
}

gtp_status encode_tmap_3d(CUtensorMap *map, CUtensorMapDataType dtype, const void *base, uint64_t inner,
                          uint64_t middle, uint64_t outer, uint64_t row_stride_bytes, uint64_t plane_stride_bytes,
                          uint32_t box_inner, uint32_t box_middle, uint32_t box_outer) {
  const cuuint64_t dims[3] = {inner, middle, outer};
  const cuuint64_t strides[2] = {row_stride_bytes, plane_stride_bytes};
  const cuuint32_t box[3] = {box_inner, box_middle, box_outer};
  CUresult r;
  if (gtp_status s = encode(&r, map, dtype, 3, base, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_NONE)) return s;
  if (r != CUDA_SUCCESS)
    return fail(GTP_E_CUDA, "cuTensorMapEncodeTiled failed (%d): dims %llu x %llu x %llu, box %u x %u x %u", int(r),
                (unsigned long long)inner, (unsigned long long)middle, (unsigned long long)outer, box_inner, box_middle,
                box_outer);
  return GTP_OK;
}

}  // namespace gtp
