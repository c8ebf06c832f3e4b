// paged_map.cu -- tensor maps over the page pools.
#include <cuda.h>
#include <cudaTypedefs.h>

#include "async.cuh"

namespace kvs {

kvs_status paged_tensor_map(CUtensorMap* map, const uint16_t* pool, const PagedView& kv, int rows, int halves,
                            const char* who) {
  // through the runtime's driver entry point (the library links no driver
  // library), looked up once per process
  static const PFN_cuTensorMapEncodeTiled_v12000 encode = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q{};
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  }();
  KVS_REQUIRE(encode != nullptr, KVS_ECUDA, "%s: cuTensorMapEncodeTiled unavailable", who);
  const cuuint64_t dim[5] = {kD / 2, static_cast<cuuint64_t>(1) << kv.shift, 2, static_cast<cuuint64_t>(kv.G),
                             static_cast<cuuint64_t>(kv.num_pages)};
  const cuuint64_t stride[4] = {static_cast<cuuint64_t>(kv.token_stride) * 2, kD,
                                static_cast<cuuint64_t>(kv.head_stride) * 2,
                                static_cast<cuuint64_t>(kv.page_stride) * 2};
  const cuuint32_t box[5] = {kD / 2, static_cast<cuuint32_t>(rows), static_cast<cuuint32_t>(halves), 1, 1};
  const cuuint32_t one[5] = {1, 1, 1, 1, 1};
  const CUresult e = encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<uint16_t*>(pool), dim, stride, box,
                            one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  KVS_REQUIRE(e == CUDA_SUCCESS, KVS_ECUDA, "%s: tensor map encoding failed (%d)", who, static_cast<int>(e));
  return KVS_OK;
}

}  // namespace kvs
