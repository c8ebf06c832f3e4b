// paged_prompt.cu -- causal attention of the newest tokens of each request (a
// prompt or a chunk of one) over its paged cache, with a sliding window and
// first tokens that stay visible.
#include <cuda_bf16.h>

#include "paged_simple.cuh"

namespace kvs {

namespace {

__global__ void __launch_bounds__(kSimpleThreads) paged_prompt_simple_kernel(PagedView kv, kvs_paged_prompt_args a,
                                                                             int32_t* dev_status) {
  pdl_wait();
  __shared__ SimpleSmem s;
  const int t = blockIdx.x, hq = blockIdx.y, g = hq / a.H, tid = threadIdx.x;
  if (t >= a.cu[kv.R]) return;
  int lo = 0, hi = kv.R;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (a.cu[mid] <= t) lo = mid;
    else hi = mid;
  }
  const int p = kv.length(lo, dev_status) - (a.cu[lo + 1] - t);
  s.q[tid] = bf16_bits_to_float(a.q[t * a.q_ld + hq * kD + tid]) * a.scale;
  __syncthreads();
  float lse;
  const float o = simple_attend(kv, lo, g, p, a.window, a.sinks, s, lse, dev_status);
  const __nv_bfloat16 v = __float2bfloat16_rn(o);
  a.out[t * a.out_ld + hq * kD + tid] = *reinterpret_cast<const uint16_t*>(&v);
  if (a.lse && tid == 0) a.lse[static_cast<size_t>(t) * kv.G * a.H + hq] = lse;
}

}  // namespace

kvs_status paged_prompt_launch(const kvs_paged_prompt_args* a, int32_t* dev_status, cudaStream_t s) {
  const PagedView kv = paged_view(a->kv);
  launch_chained(paged_prompt_simple_kernel, dim3(a->T, kv.G * a->H), dim3(kSimpleThreads), 0, s, kv, *a, dev_status);
  return check_launch("paged_prompt_attn");
}

}  // namespace kvs
