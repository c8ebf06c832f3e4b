// paged_decode.cu -- attention of each request's newest token over its paged
// cache, optionally with the weights added up per token.
#include "paged_simple.cuh"

namespace kvs {

namespace {

__global__ void __launch_bounds__(kSimpleThreads) paged_decode_simple_kernel(PagedView kv, kvs_paged_decode_args a,
                                                                             int32_t* dev_status) {
  pdl_wait();
  __shared__ SimpleSmem s;
  const int u = blockIdx.x, r = u / kv.G, g = u % kv.G, tid = threadIdx.x;
  const int n = kv.length(r, dev_status);
  for (int h = 0; h < a.H; ++h) {
    const size_t at = (static_cast<size_t>(u) * a.H + h) * kD + tid;
    const float q = a.q_dtype == KVS_BF16 ? bf16_bits_to_float(static_cast<const uint16_t*>(a.q)[at])
                                          : static_cast<const float*>(a.q)[at];
    __syncthreads();
    s.q[tid] = q * a.scale;
    __syncthreads();
    float lse;
    a.out[at] = simple_attend(kv, r, g, n - 1, a.window, a.sinks, s, lse, dev_status);
    if (a.lse && tid == 0) a.lse[static_cast<size_t>(u) * a.H + h] = lse;
    if (!a.mass) continue;
    for (int j = tid; j < n; j += kSimpleThreads) {
      if (a.window && j >= a.sinks && j < n - a.window) continue;
      const size_t m = static_cast<size_t>(u) * kv.cap() + j;
      const int id = kv.page_of(r, j, dev_status);
      float w = 0.f;
      if (id >= 0) {
        float acc = 0.f;
        for (int d = 0; d < kD; ++d) acc = fmaf(s.q[d], bf16_bits_to_float(kv.K[kv.row(id, g, j) + d]), acc);
        w = expf(acc - lse);
      }
      a.mass_out[m] = (h == 0 ? a.mass[m] : a.mass_out[m]) + w;
    }
  }
}

}  // namespace

size_t paged_decode_ws_bytes(int R, int G, int H, int weight_cap) {
  (void)R, (void)G, (void)H, (void)weight_cap;
  return 0;
}

kvs_status paged_decode_launch(const kvs_paged_decode_args* a, void* ws, int32_t* dev_status, cudaStream_t s) {
  (void)ws;
  const PagedView kv = paged_view(a->kv);
  launch_chained(paged_decode_simple_kernel, dim3(kv.R * kv.G), dim3(kSimpleThreads), 0, s, kv, *a, dev_status);
  return check_launch("paged_decode_attn");
}

}  // namespace kvs
