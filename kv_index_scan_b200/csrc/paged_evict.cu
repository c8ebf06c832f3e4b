// paged_evict.cu -- eviction from the paged cache by accumulated attention
// weight: of n > budget slots keep the protected ones (the first tokens of the
// request and its most recent) and the heaviest others, budget in all.
//
// Kept rows do not close ranks. A kept row in a slot behind the budget moves
// into a slot that an evicted row frees in front of it, j-th mover into j-th
// hole, and no other row is touched: a cache one token over its budget moves at
// most one row of each head instead of shifting all that follow the evicted
// one. Sources lie behind the budget and destinations before it, so the moves
// need no order among themselves.
//
// Two kernels. The selection (one block per (r, g)) finds the budget-th largest
// key by a radix select and lists which slot each kept one comes from; the move
// (the whole grid) copies 512 bytes for each slot whose token came from another.
#include "paged.cuh"

namespace kvs {

namespace {

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kMoveWarps = 8;

struct EvictParams {
  PagedView kv;
  const float* mass;
  const int32_t* pos;
  const int32_t* seen;
  int budget, sinks, recent;
  float* mass_out;
  int32_t* pos_out;
  int32_t* n_out;
  int32_t* src;
  int32_t* holes;  // [R*G][budget]
  int32_t* dev_status;
};

// Exclusive rank of `p` among the block's threads in thread order, and the
// total. `part` is kSelWarps ints of shared memory, free again on return.
__device__ __forceinline__ int block_rank(bool p, int* part, int& total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const unsigned m = __ballot_sync(0xFFFFFFFFu, p);
  if (lane == 0) part[warp] = __popc(m);
  __syncthreads();
  int x = part[lane];  // kSelWarps == 32
  int inc = x;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xFFFFFFFFu, inc, d);
    if (lane >= d) inc += y;
  }
  total = __shfl_sync(0xFFFFFFFFu, inc, 31);
  const int before = __shfl_sync(0xFFFFFFFFu, inc - x, warp);
  __syncthreads();
  return before + __popc(m & ((1u << lane) - 1u));
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(EvictParams p) {
  pdl_wait();
  __shared__ int hist[256];
  __shared__ int part[kSelWarps];
  __shared__ uint32_t s_prefix;
  __shared__ int s_need;
  const int u = blockIdx.x, r = u / p.kv.G;
  const int n = p.kv.length(r, p.dev_status);
  const int seen = p.seen ? p.seen[r] : n;
  const int b = p.budget;
  const size_t row = static_cast<size_t>(u) * p.kv.cap();
  const float* mass = p.mass + row;
  const int32_t* pos = p.pos ? p.pos + row : nullptr;
  float* mass_out = p.mass_out + row;
  int32_t* pos_out = p.pos_out ? p.pos_out + row : nullptr;
  int32_t* src = p.src + static_cast<size_t>(u) * b;
  int32_t* holes = p.holes + static_cast<size_t>(u) * b;
  auto put = [&](int j, int from) {
    src[j] = from;
    mass_out[j] = mass[from];
    if (pos_out) pos_out[j] = pos[from];
  };
  if (n <= b) {
    for (int j = threadIdx.x; j < b; j += kSelThreads) {
      if (j < n) put(j, j);
      else src[j] = -1;
    }
    return;
  }
  // the order of slots: protected ones above any weight, NaN below any
  auto key = [&](int j) -> uint32_t {
    const int at = pos ? pos[j] : j;
    if (at < p.sinks || at >= seen - p.recent) return 0xFFFFFFFFu;
    const float m = mass[j];
    return m != m ? 0u : ordered_key(m);
  };
  // the b-th largest key, eight bits at a time
  uint32_t prefix = 0;
  int need = b;  // still to take among the keys that share the prefix
  for (int shift = 24; shift >= 0; shift -= 8) {
    if (threadIdx.x < 256) hist[threadIdx.x] = 0;
    __syncthreads();
    for (int j = threadIdx.x; j < n; j += kSelThreads) {
      const uint32_t k = key(j);
      if (shift == 24 || (k >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&hist[(k >> shift) & 255u], 1);
    }
    __syncthreads();
    if (threadIdx.x == 0) {
      int d = 255, left = need;
      while (hist[d] < left) left -= hist[d--];
      s_prefix = prefix | (static_cast<uint32_t>(d) << shift);
      s_need = left;
    }
    __syncthreads();
    prefix = s_prefix;
    need = s_need;
  }
  // kept: keys above the cut, and of those at it the `need` lowest slots
  int ties = 0, nh = 0, nm = 0;
  for (int j0 = 0; j0 < n; j0 += kSelThreads) {
    const int j = j0 + threadIdx.x;
    const uint32_t k = j < n ? key(j) : 0u;
    const bool tie = j < n && k == prefix;
    int total;
    const int tr = ties + block_rank(tie, part, total);
    ties += total;
    const bool keep = j < n && (k > prefix || (tie && tr < need));
    const bool hole = j < b && !keep, mover = j >= b && keep;
    const int hr = nh + block_rank(hole, part, total);
    nh += total;
    const int mr = nm + block_rank(mover, part, total);
    nm += total;
    if (hole) holes[hr] = j;
    if (j < b && keep) put(j, j);
    __syncthreads();  // holes are written before a mover reads them
    if (mover) put(holes[mr], j);
  }
}

__global__ void __launch_bounds__(32 * kMoveWarps) evict_move_kernel(EvictParams p) {
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t warp0 = static_cast<int64_t>(blockIdx.x) * kMoveWarps + (threadIdx.x >> 5);
  const int64_t warps = static_cast<int64_t>(gridDim.x) * kMoveWarps;
  const int per = (p.budget + 31) / 32;
  const int64_t items = static_cast<int64_t>(p.kv.R) * p.kv.G * per;
  for (int64_t it = warp0; it < items; it += warps) {
    const int u = static_cast<int>(it / per), r = u / p.kv.G, g = u % p.kv.G;
    const int j = static_cast<int>(it % per) * 32 + lane;
    const int from = j < p.budget ? p.src[static_cast<size_t>(u) * p.budget + j] : -1;
    unsigned todo = __ballot_sync(0xFFFFFFFFu, from >= 0 && from != j);
    int64_t a = -1, b = -1;
    if (from >= 0 && from != j) {
      const int pa = p.kv.page_of(r, from, p.dev_status), pb = p.kv.page_of(r, j, p.dev_status);
      if (pa >= 0 && pb >= 0) {
        a = p.kv.row(pa, g, from);
        b = p.kv.row(pb, g, j);
      }
    }
    const bool isv = lane >= 16;
    uint16_t* pool = (isv ? p.kv.V : p.kv.K) + 8 * (lane & 15);
    while (todo) {
      const int l = __ffs(todo) - 1;
      todo &= todo - 1;
      const int64_t fa = __shfl_sync(0xFFFFFFFFu, a, l), fb = __shfl_sync(0xFFFFFFFFu, b, l);
      if (fa >= 0) *reinterpret_cast<uint4*>(pool + fb) = *reinterpret_cast<const uint4*>(pool + fa);
    }
  }
  for (int64_t r = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; r < p.kv.R;
       r += static_cast<int64_t>(gridDim.x) * blockDim.x)
    p.n_out[r] = min(p.kv.length(static_cast<int>(r), nullptr), p.budget);
}

}  // namespace

size_t paged_evict_ws_bytes(int R, int G, int budget) {
  return align_up(static_cast<size_t>(R) * G * budget * sizeof(int32_t), 16);
}

kvs_status paged_evict_launch(const kvs_paged_evict_args* a, void* ws, int32_t* dev_status, cudaStream_t s) {
  EvictParams p{};
  p.kv = paged_view(a->kv);
  p.mass = a->mass;
  p.pos = a->pos;
  p.seen = a->seen;
  p.budget = a->budget;
  p.sinks = a->sinks;
  p.recent = a->recent;
  p.mass_out = a->mass_out;
  p.pos_out = a->pos_out;
  p.n_out = a->n_out;
  p.src = a->src;
  p.holes = static_cast<int32_t*>(ws);
  p.dev_status = dev_status;
  const int RG = p.kv.R * p.kv.G;
  launch_chained(evict_select_kernel, dim3(RG), dim3(kSelThreads), 0, s, p);
  const int64_t items = static_cast<int64_t>(RG) * ((a->budget + 31) / 32);
  const int64_t want = (items + kMoveWarps - 1) / kMoveWarps;
  const int grid = static_cast<int>(want < 8ll * sm_count() ? want : 8ll * sm_count());
  launch_chained(evict_move_kernel, dim3(grid), dim3(32 * kMoveWarps), 0, s, p);
  return check_launch("kvs_paged_evict");
}

}  // namespace kvs
