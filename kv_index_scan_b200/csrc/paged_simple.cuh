// paged_simple.cuh -- attention of one query token over a request's pages, one
// block per (token, KV head): 128 threads score 128 keys at a time, a key each,
// and then add up the values, a channel each.
#pragma once

#include "paged.cuh"

namespace kvs {

constexpr int kSimpleThreads = 128;

struct SimpleSmem {
  float q[kD];
  float w[kSimpleThreads];
  int64_t row[kSimpleThreads];
  float red[4];
};

// Softmax attention of query s.q (scaled, in shared memory) at position p.
// Returns this thread's channel of the output and sets the log-sum-exp.
__device__ __forceinline__ float simple_attend(const PagedView& kv, int r, int g, int p, int window, int sinks,
                                               SimpleSmem& s, float& lse, int32_t* dev_status) {
  const int tid = threadIdx.x;
  const float ninf = -__int_as_float(0x7f800000);
  float m = ninf, l = 0.f, o = 0.f;
  for (int j0 = 0; j0 <= p; j0 += kSimpleThreads) {
    if (window && j0 >= sinks && j0 + kSimpleThreads <= p - window + 1) continue;
    const int j = j0 + tid;
    float x = ninf;
    int64_t at = -1;
    if (j <= p && (!window || j < sinks || j > p - window)) {
      const int id = kv.page_of(r, j, dev_status);
      if (id >= 0) {
        at = kv.row(id, g, j);
        float acc = 0.f;
        for (int d = 0; d < kD; ++d) acc = fmaf(s.q[d], bf16_bits_to_float(kv.K[at + d]), acc);
        x = acc;
      }
    }
    float mx = x;
    for (int d = 16; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, d));
    __syncthreads();
    if ((tid & 31) == 0) s.red[tid >> 5] = mx;
    __syncthreads();
    const float nm = fmaxf(m, fmaxf(fmaxf(s.red[0], s.red[1]), fmaxf(s.red[2], s.red[3])));
    const float alpha = nm == ninf ? 1.f : expf(m - nm);
    s.w[tid] = at < 0 ? 0.f : expf(x - nm);
    s.row[tid] = at;
    __syncthreads();
    o *= alpha;
    l *= alpha;
    m = nm;
    for (int k = 0; k < kSimpleThreads; ++k) {
      if (s.row[k] < 0) continue;
      l += s.w[k];
      o = fmaf(s.w[k], bf16_bits_to_float(kv.V[s.row[k] + tid]), o);
    }
  }
  __syncthreads();
  lse = l > 0.f ? m + logf(l) : (m == ninf ? ninf : m + logf(l));
  return m == ninf ? 0.f : o / l;
}

}  // namespace kvs
