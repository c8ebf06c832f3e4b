// paged.cuh -- the paged K/V cache as its kernels see it, and their launchers.
#pragma once

#include "internal.cuh"

#define KVS_PROPAGATE(expr)                \
  do {                                     \
    const kvs_status st_ = (expr);         \
    if (st_ != KVS_OK) return st_;         \
  } while (0)

namespace kvs {

// kvs_paged_kv with the page size as a shift.
struct PagedView {
  uint16_t* K;
  uint16_t* V;
  int64_t page_stride, head_stride, token_stride;
  const int32_t* table;
  int64_t table_ld;
  const int32_t* n;
  int R, G, shift, max_pages, num_pages;

  __device__ __forceinline__ int cap() const { return max_pages << shift; }
  // n[r], clamped to what the table can hold
  __device__ __forceinline__ int length(int r, int32_t* dev_status) const {
    const int v = n[r];
    if (v < 0 || v > cap()) {
      set_status(dev_status, KVS_EBOUNDS);
      return v < 0 ? 0 : cap();
    }
    return v;
  }
  // page id of token i of request r, or -1 (and KVS_EBOUNDS) for an id that is none
  __device__ __forceinline__ int page_of(int r, int i, int32_t* dev_status) const {
    const int id = __ldg(table + r * table_ld + (i >> shift));
    if (static_cast<unsigned>(id) < static_cast<unsigned>(num_pages)) return id;
    set_status(dev_status, KVS_EBOUNDS);
    return -1;
  }
  // element offset of token i's row in page id, KV head g
  __device__ __forceinline__ int64_t row(int id, int g, int i) const {
    return id * page_stride + g * head_stride + (i & ((1 << shift) - 1)) * token_stride;
  }
};

PagedView paged_view(const kvs_paged_kv* kv);

// Allows `kernel` its dynamic shared memory on the current device, the first
// time it is launched there (a launch pays for the call otherwise). Threads
// that race here set the same value.
template <auto kernel>
void allow_smem(size_t bytes) {
  static bool done[64] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 0 && dev < 64 && __atomic_load_n(&done[dev], __ATOMIC_RELAXED)) return;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes)) ==
          cudaSuccess &&
      dev >= 0 && dev < 64)
    __atomic_store_n(&done[dev], true, __ATOMIC_RELAXED);
}

kvs_status paged_append_launch(const PagedView& kv, const uint16_t* Knew, const uint16_t* Vnew, int64_t new_ld,
                               const int32_t* cu, int T, float* mass, int32_t* pos, const int32_t* seen,
                               int32_t* dev_status, cudaStream_t s);
size_t paged_decode_ws_bytes(int R, int G, int H, int weight_cap);
// test_warp >= 0: that warp gives up, and waits are bounded by wait_cycles (kvs_selftest_paged_decode_timeout)
kvs_status paged_decode_launch(const kvs_paged_decode_args* a, void* ws, int32_t* dev_status, cudaStream_t s,
                               int test_warp = -1, int64_t wait_cycles = 0);
size_t paged_prompt_ws_bytes(int R, int G, int H, int T, int cap, int window, int sinks);
size_t paged_prompt_ws_bound(int R, int G, int H, int T, int cap, int window, int sinks);  // over 1 .. T queries
// (likewise: kvs_selftest_paged_prompt_timeout)
kvs_status paged_prompt_launch(const kvs_paged_prompt_args* a, void* ws, int32_t* dev_status, cudaStream_t s,
                               int test_warp = -1, int64_t wait_cycles = 0);
size_t paged_evict_ws_bytes(int R, int G, int budget);
kvs_status paged_evict_launch(const kvs_paged_evict_args* a, void* ws, int32_t* dev_status, cudaStream_t s);

}  // namespace kvs
