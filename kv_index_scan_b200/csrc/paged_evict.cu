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
// A cluster of blocks takes each (r, g) row, so that a few long rows occupy the
// GPU as well as many short ones:
//  1. each block turns its run of the row's slots into 32-bit keys in shared
//     memory and writes the slots' own values
//     out;
//  2. the budget-th largest key by a radix select in digits of 11, 11 and 10
//     bits: histograms in shared memory, summed over the cluster by distributed
//     shared memory, every block finding the digit for itself;
//  3. each thread counts holes and movers in a contiguous piece of its block's
//     run; ranks by a scan over the block and the cluster; the two lists go to
//     the workspace;
//  4. the cluster's warps share the moves: 512 bytes each, several rows in
//     flight per warp.
// Ties at the cut go to the lower slots: only then the tied keys are ranked too.
// Bound by the moved rows' bytes, for small moves by the latency of the steps:
// 8 prompts of 16K to 64K tokens cut to 4096 (64 rows, 246,000 moves) take 68 us,
// 38 of them the moves; 128 rows of 4097 slots, one move each, 12.5 us.
#include <cooperative_groups.h>

#include "paged.cuh"

namespace kvs {

namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kMaxCluster = 8;
constexpr int kKeysMost = 22 * 1024;  // keys of a block in shared memory (two blocks share an SM)
constexpr int kFlight = 4;            // rows that a warp copies at a time (8: registers spill, 82 us for 68)
constexpr int kFewMoves = 512, kRunFew = 4096, kRunMany = 2048;
constexpr int kBatch = 8;             // slots that a thread reads at a time

constexpr uint32_t kSure = 0xFFFFFFFFu;  // key of a protected slot
constexpr uint32_t kZero = 0x80000000u;  // of a weight of zero

struct EvictParams {
  PagedView kv;
  const float* mass;
  const int32_t* pos;
  const int32_t* seen;
  int budget, sinks, recent;
  float* mass_out;
  int32_t* pos_out;
  int32_t* n_out;  // written here where it is not n itself
  int32_t* src;
  int32_t* holes;   // [R*G][budget]
  int32_t* movers;  // [R*G][budget]
  int keys_room;    // keys of shared memory a block has
  int32_t* dev_status;
};

struct EvictShared {
  int hist[3][kBins];  // one a digit: no block clears what another still reads
  unsigned long long part[2][kWarps];
  int part32[3][kWarps];
  unsigned long long count;  // of this block, read by its cluster
  int digit[3], need[3], equal[3];
};

// Sum over the block of v, and the sum of the threads before this one.
// (`part` may be written again after the block's next barrier.)
template <typename T>
__device__ __forceinline__ T scan_block(T v, T* part, T& total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  T inc = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const T y = __shfl_up_sync(0xFFFFFFFFu, inc, d);
    if (lane >= d) inc += y;
  }
  if (lane == 31) part[warp] = inc;
  __syncthreads();
  const T x = lane < kWarps ? part[lane] : T(0);
  T w = x;
#pragma unroll
  for (int d = 1; d < kWarps; d <<= 1) {
    const T y = __shfl_up_sync(0xFFFFFFFFu, w, d);
    if (lane >= d) w += y;
  }
  total = __shfl_sync(0xFFFFFFFFu, w, kWarps - 1);
  return __shfl_sync(0xFFFFFFFFu, w - x, warp) + inc - v;
}

__global__ void __launch_bounds__(kThreads, 2) paged_evict_kernel(EvictParams p) {
  extern __shared__ uint32_t evict_keys[];
  __shared__ EvictShared sm;
  const cg::cluster_group cluster = cg::this_cluster();
  const int C = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  auto sync = [&] {
    if (C == 1) __syncthreads();
    else cluster.sync();
  };
  for (int e = tid; e < 3 * kBins; e += kThreads) sm.hist[0][e] = 0;
  pdl_wait();
  pdl_trigger();
  const int u = blockIdx.x / C, r = u / p.kv.G, g = u % p.kv.G;
  const int n = p.kv.length(r, p.dev_status);
  const int seen = p.seen ? p.seen[r] : n;
  const int b = p.budget;
  const size_t row = static_cast<size_t>(u) * p.kv.cap();
  const float* mass = p.mass + row;
  const int32_t* pos = p.pos ? p.pos + row : nullptr;
  float* mass_out = p.mass_out + row;
  int32_t* pos_out = p.pos_out ? p.pos_out + row : nullptr;
  int32_t* src = p.src + static_cast<size_t>(u) * b;
  if (p.n_out && g == 0 && rank == 0 && tid == 0) p.n_out[r] = min(n, b);

  // every slot's own values; where the budget is not reached they are all
  const bool over = n > b;
  const int per = over ? (n + C - 1) / C : (b + C - 1) / C;
  const int lo = min(rank * per, over ? n : b), hi = min(lo + per, over ? n : b);
  const bool in_smem = per <= p.keys_room;
  auto key_of = [&](float m, int at) -> uint32_t {
    // protected ones above any weight, NaN below any
    if (at < p.sinks || at >= seen - p.recent) return kSure;
    return m != m ? 0u : ordered_key(m);
  };
  for (int j0 = lo + tid; j0 < hi; j0 += kBatch * kThreads) {
    // loads of a batch before its stores, which may be to the same arrays
    float m[kBatch];
    int at[kBatch];
#pragma unroll
    for (int x = 0; x < kBatch; ++x) {
      const int j = j0 + x * kThreads;
      m[x] = 0.f;
      at[x] = j;
      if (j < hi && j < n) {
        m[x] = mass[j];
        if (pos) at[x] = pos[j];
      }
    }
#pragma unroll
    for (int x = 0; x < kBatch; ++x) {
      const int j = j0 + x * kThreads;
      if (j >= hi) continue;
      if (j < b) {
        src[j] = j < n ? j : -1;
        if (j < n && mass_out != mass) mass_out[j] = m[x];
        if (j < n && pos_out != pos) pos_out[j] = at[x];
      }
      if (over && in_smem) evict_keys[j - lo] = key_of(m[x], at[x]);
    }
  }
  if (!over) return;  // (the whole cluster)
  auto key = [&](int j) { return in_smem ? evict_keys[j - lo] : key_of(mass[j], pos ? pos[j] : j); };
  __syncthreads();

  // the b-th largest key
  uint32_t cut = 0;
  int need = b, equal = 0;  // still to take among the keys that share the cut's digits, and how many do
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0), width = pass == 2 ? 10 : 11;
    int* hist = sm.hist[pass];
    // the protected (all in the first pass's top bin) and the weights of zero
    // are many: each thread counts its own
    int sure = 0, zero = 0;
#pragma unroll 4
    for (int j = lo + tid; j < hi; j += kThreads) {
      const uint32_t k = key(j);
      if (pass == 0 || (k >> (shift + width)) == (cut >> (shift + width))) {
        if (k == kSure) ++sure;
        else if (k == kZero) ++zero;
        else atomicAdd(&hist[(k >> shift) & ((1u << width) - 1u)], 1);
      }
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      sure += __shfl_xor_sync(0xFFFFFFFFu, sure, d);
      zero += __shfl_xor_sync(0xFFFFFFFFu, zero, d);
    }
    if (lane == 0 && sure) atomicAdd(&hist[(kSure >> shift) & ((1u << width) - 1u)], sure);
    if (lane == 0 && zero) atomicAdd(&hist[(kZero >> shift) & ((1u << width) - 1u)], zero);
    sync();
    // bins from the top, kOwn a thread
    constexpr int kOwn = kBins / kThreads;
    static_assert(kOwn == 4, "a thread's bins are one 16-byte load");
    const int bin = kBins - kOwn * (tid + 1);
    int h[kOwn] = {0, 0, 0, 0};
#pragma unroll
    for (int x = 0; x < kMaxCluster; ++x) {
      int4 v = make_int4(0, 0, 0, 0);
      if (x < C) v = *reinterpret_cast<const int4*>((C == 1 ? hist : cluster.map_shared_rank(hist, x)) + bin);
      h[0] += v.x;
      h[1] += v.y;
      h[2] += v.z;
      h[3] += v.w;
    }
    int all, above = scan_block(h[0] + h[1] + h[2] + h[3], sm.part32[pass], all);
#pragma unroll
    for (int e = kOwn - 1; e >= 0; --e) {
      if (above < need && above + h[e] >= need) {
        sm.digit[pass] = bin + e;
        sm.need[pass] = need - above;
        sm.equal[pass] = h[e];
      }
      above += h[e];
    }
    __syncthreads();
    cut |= static_cast<uint32_t>(sm.digit[pass]) << shift;
    need = sm.need[pass];
    equal = sm.equal[pass];
    if (equal == need) break;  // all of them: the lower digits need not be known
  }

  // this thread's piece of the block's run (an odd length: no bank conflicts)
  const int len = ((hi - lo + kThreads - 1) / kThreads) | 1;
  const int a0 = min(lo + tid * len, hi), a1 = min(a0 + len, hi);
  unsigned long long total;
  // sums over the cluster's blocks before this one, and over all of them
  auto before_us = [&](unsigned long long mine, unsigned long long& all) {
    if (tid == 0) sm.count = mine;
    sync();
    unsigned long long v = lane < C ? *cluster.map_shared_rank(&sm.count, lane) : 0ull, w = lane < rank ? v : 0ull;
#pragma unroll
    for (int d = kMaxCluster / 2; d > 0; d >>= 1) {
      v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
      w += __shfl_xor_sync(0xFFFFFFFFu, w, d);
    }
    all = __shfl_sync(0xFFFFFFFFu, v, 0);
    return __shfl_sync(0xFFFFFFFFu, w, 0);
  };
  unsigned long long last;  // holes and movers of the whole row
  int tie = 0;  // rank of the next tied key of this thread
  const bool some = equal > need;  // only some of the tied keys are kept
  if (some) {
    int t = 0;
    for (int j = a0; j < a1; ++j) t += key(j) == cut;
    const unsigned long long mine = scan_block(static_cast<unsigned long long>(t), sm.part[0], total);
    tie = static_cast<int>(before_us(total, last) + mine);
    sync();  // every block has read the counts
  }
  const int tie0 = tie;
  auto kept = [&](uint32_t k) { return some ? k > cut || (k == cut && tie++ < need) : k >= cut; };
  unsigned long long moves = 0;  // holes, and movers in the upper half
  for (int j = a0; j < a1; ++j) {
    const bool keep = kept(key(j));
    if (j < b) moves += keep ? 0ull : 1ull;
    else moves += keep ? 1ull << 32 : 0ull;
  }
  unsigned long long at = scan_block(moves, sm.part[1], total);
  at += before_us(total, last);
  {
    int h = static_cast<int>(at & 0xFFFFFFFFull), m = static_cast<int>(at >> 32);
    int32_t* holes = p.holes + static_cast<size_t>(u) * b;
    int32_t* movers = p.movers + static_cast<size_t>(u) * b;
    tie = tie0;
    for (int j = a0; j < a1; ++j) {
      const bool keep = kept(key(j));
      if (j < b && !keep) holes[h++] = j;
      if (j >= b && keep) movers[m++] = j;
    }
  }
  sync();  // the lists are written, and every block has read the counts
  const int count = static_cast<int>(last & 0xFFFFFFFFull);

  // the moves, 32 a warp at a time
  const int32_t* holes = p.holes + static_cast<size_t>(u) * b;
  const int32_t* movers = p.movers + static_cast<size_t>(u) * b;
  const bool isv = lane >= 16;
  uint16_t* pool = (isv ? p.kv.V : p.kv.K) + 8 * (lane & 15);
  // a run of up to 32 moves a warp, shorter where that lets few moves reach every warp
  const int workers = C * kWarps, me = rank * kWarps + warp;
  const int chunk = min(32, (count + workers - 1) / workers);
  for (int k0 = me * chunk; k0 < count; k0 += workers * chunk) {
    const int k = k0 + lane;
    int64_t from = -1, to = -1;
    if (lane < chunk && k < count) {
      const int h = __ldcg(holes + k), s = __ldcg(movers + k);
      src[h] = s;
      mass_out[h] = mass[s];
      if (pos_out) pos_out[h] = pos[s];
      const int ps = p.kv.page_of(r, s, p.dev_status), ph = p.kv.page_of(r, h, p.dev_status);
      if (ps >= 0 && ph >= 0) {
        from = p.kv.row(ps, g, s);
        to = p.kv.row(ph, g, h);
      }
    }
    const int here = min(chunk, count - k0);
    for (int x0 = 0; x0 < here; x0 += kFlight) {
      uint4 v[kFlight];
#pragma unroll
      for (int x = 0; x < kFlight; ++x) {
        const int64_t f = __shfl_sync(0xFFFFFFFFu, from, (x0 + x) & 31);
        if (x0 + x < here && f >= 0) v[x] = *reinterpret_cast<const uint4*>(pool + f);
      }
#pragma unroll
      for (int x = 0; x < kFlight; ++x) {
        const int64_t t = __shfl_sync(0xFFFFFFFFu, to, (x0 + x) & 31);
        if (x0 + x < here && t >= 0) *reinterpret_cast<uint4*>(pool + t) = v[x];
      }
    }
  }
}

// n cut to the budget in place, once no block needs it any more.
__global__ void evict_length_kernel(PagedView kv, int budget, int32_t* n) {
  pdl_wait();
  const int r = blockIdx.x * blockDim.x + threadIdx.x;
  if (r < kv.R) n[r] = min(kv.length(r, nullptr), budget);
}

}  // namespace

size_t paged_evict_ws_bytes(int R, int G, int budget) {
  return align_up(2 * static_cast<size_t>(R) * G * budget * sizeof(int32_t), 16);
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
  const bool in_place = a->n_out == a->kv->n;
  p.n_out = in_place ? nullptr : a->n_out;
  p.src = a->src;
  const int RG = p.kv.R * p.kv.G;
  p.holes = static_cast<int32_t*>(ws);
  p.movers = p.holes + static_cast<size_t>(RG) * a->budget;
  p.dev_status = dev_status;
  // blocks a row: enough to occupy two on every SM, each with at least so many
  // slots of the longest row there may be. Where few rows can move, the cluster's
  // barriers cost more than half a run saves (128 rows of 4097 slots, budget 4096:
  // one block a row 12.5 us, two 13.5 to 15); where many can, the moves want the blocks
  // (2 rows of 8765 slots cut to 1409: two blocks a row 21.4 us, four 14.8; 8 rows
  // of 8192 cut to 4096: 29.5 and 22.7).
  const int64_t cap = static_cast<int64_t>(a->kv->max_pages) * a->kv->page;
  const int64_t moves = cap - a->budget < a->budget ? cap - a->budget : a->budget;
  const int64_t run = moves < kFewMoves ? kRunFew : kRunMany;
  int C = 1;
  while (C < kMaxCluster && static_cast<int64_t>(RG) * C * 2 <= 2 * sm_count() && cap / (2 * C) >= run) C *= 2;
  const int64_t most = (cap + C - 1) / C;
  p.keys_room = static_cast<int>(most < kKeysMost ? most : kKeysMost);
  const size_t smem = static_cast<size_t>(p.keys_room) * sizeof(uint32_t);
  allow_smem<paged_evict_kernel>(kKeysMost * sizeof(uint32_t));
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(RG) * C);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cudaLaunchKernelEx(&cfg, paged_evict_kernel, p);
  if (in_place)
    launch_chained(evict_length_kernel, dim3((p.kv.R + 127) / 128), dim3(128), 0, s, p.kv, a->budget, a->n_out);
  return check_launch("kvs_paged_evict");
}

}  // namespace kvs
