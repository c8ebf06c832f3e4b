// paged_map.cu -- tensor maps over the page pools.
#include <cuda.h>
#include <cudaTypedefs.h>

#include "async.cuh"

namespace kvs {

namespace {

// cuTensorMapEncodeTiled through the runtime's driver entry point (the library
// links no driver library), looked up once per process; bf16, 128-byte swizzle.
kvs_status encode(CUtensorMap* map, const void* base, int rank, const cuuint64_t* dim, const cuuint64_t* stride,
                  const cuuint32_t* box, const char* who) {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q{};
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  }();
  KVS_REQUIRE(fn != nullptr, KVS_ECUDA, "%s: cuTensorMapEncodeTiled unavailable", who);
  const cuuint32_t one[5] = {1, 1, 1, 1, 1};
  const CUresult e = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(base), dim, stride, box, one,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  KVS_REQUIRE(e == CUDA_SUCCESS, KVS_ECUDA, "%s: tensor map encoding failed (%d)", who, static_cast<int>(e));
  return KVS_OK;
}

}  // namespace

kvs_status paged_tensor_map(CUtensorMap* map, const uint16_t* pool, const PagedView& kv, int rows, int halves,
                            const char* who) {
  const cuuint64_t dim[5] = {kD / 2, static_cast<cuuint64_t>(1) << kv.shift, 2, static_cast<cuuint64_t>(kv.G),
                             static_cast<cuuint64_t>(kv.num_pages)};
  const cuuint64_t stride[4] = {static_cast<cuuint64_t>(kv.token_stride) * 2, kD,
                                static_cast<cuuint64_t>(kv.head_stride) * 2,
                                static_cast<cuuint64_t>(kv.page_stride) * 2};
  const cuuint32_t box[5] = {kD / 2, static_cast<cuuint32_t>(rows), static_cast<cuuint32_t>(halves), 1, 1};
  return encode(map, pool, 5, dim, stride, box, who);
}

kvs_status query_tensor_map(CUtensorMap* map, const kvs_paged_prompt_args* a, int tokens) {
  const cuuint64_t dim[4] = {kD / 2, static_cast<cuuint64_t>(a->kv->G) * a->H, static_cast<cuuint64_t>(a->T), 2};
  const cuuint64_t stride[3] = {kD * 2, static_cast<cuuint64_t>(a->q_ld) * 2, kD};
  const cuuint32_t box[4] = {kD / 2, static_cast<cuuint32_t>(a->H), static_cast<cuuint32_t>(tokens), 1};
  return encode(map, a->q, 4, dim, stride, box, "paged_prompt_attn");
}

}  // namespace kvs
