// async.cuh -- mbarriers with bounded waits, TMA tile loads and the page-pool
// tensor map of the paged attention kernels.
#pragma once

#include <cuda.h>

#include "paged.cuh"

namespace kvs {

constexpr long long kWaitCycles = 2000000000ll;  // about one second

__device__ __forceinline__ uint32_t sm_addr(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ void mbar_init(uint64_t* b, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;\n" ::"r"(sm_addr(b)), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_init_fence() {
  asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t* b) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(sm_addr(b)) : "memory");
}
__device__ __forceinline__ void mbar_expect(uint64_t* b, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n" ::"r"(sm_addr(b)), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool mbar_try(uint64_t* b, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(done)
      : "r"(sm_addr(b)), "r"(parity)
      : "memory");
  return done != 0;
}
// Waits for the phase of this parity; false if it does not come. (A thread that
// was held up between its last try and the clock looks once more.)
__device__ __forceinline__ bool mbar_wait(uint64_t* b, uint32_t parity, long long cycles = kWaitCycles) {
  if (mbar_try(b, parity)) return true;
  const long long t0 = clock64();
  while (!mbar_try(b, parity))
    if (clock64() - t0 > cycles) return mbar_try(b, parity);
  return true;
}
// The page pool as a tensor [page id][head][half][token][64 elements]: `rows`
// tokens of one page and head, both 128-byte halves, to dst (the first half's
// rows, then the second's, 128-byte swizzled).
__device__ __forceinline__ void tma_page_rows(uint32_t dst, const CUtensorMap* map, int token, int half, int head,
                                              int id, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, "
      "%6}], [%7];\n" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(token), "r"(half), "r"(head), "r"(id), "r"(sm_addr(bar))
      : "memory");
}
__device__ __forceinline__ void tma_prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

// That tensor map for one pool, with boxes of `rows` tokens and `halves` halves.
kvs_status paged_tensor_map(CUtensorMap* map, const uint16_t* pool, const PagedView& kv, int rows, int halves,
                            const char* who);

// The packed queries as a tensor [half][token][head][64 elements], with boxes of
// a KV head's H heads and `tokens` tokens.
kvs_status query_tensor_map(CUtensorMap* map, const kvs_paged_prompt_args* a, int tokens);

// The tokens that a query at position p sees, as whole tiles of `kTile` tokens:
// the sinks' tiles, then those from the window's first token to p. Tiles that
// hold both are counted once.
template <int kTile>
struct VisibleTiles {
  int lo;      // first token of the window (0 without one)
  int end;     // tokens seen at most, p + 1
  int nsink;   // leading tiles with sinks, where a gap follows them
  int first;   // tile of the window's first token (0 where there is no gap)
  int count;
  __device__ __forceinline__ VisibleTiles(int n, int window, int sinks) {
    end = n;
    lo = window && n > window ? n - window : 0;
    nsink = 0;
    first = 0;
    if (lo) {
      const int s = (min(sinks, lo) + kTile - 1) / kTile;
      if (s < lo / kTile) {
        nsink = s;
        first = lo / kTile;
      }
    }
    count = nsink + (n + kTile - 1) / kTile - first;
  }
  __device__ __forceinline__ int tile(int k) const { return k < nsink ? k : first + k - nsink; }
};

}  // namespace kvs
