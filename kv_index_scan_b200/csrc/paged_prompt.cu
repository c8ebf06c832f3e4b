// paged_prompt.cu -- causal attention of the newest tokens of each request (a
// prompt or a chunk of one) over its paged cache, with a sliding window and
// first tokens that stay visible.
//
// For each (token, query head) row at position p: l_j = scale * q . K_j over
// the visible tokens, out = sum_j softmax(l)_j V_j, in base 2 with an online
// softmax. 4 * 128 flops per visible (row, token) pair on the tensor cores and
// one exponential: 256 rows against 128 tokens take the tensor cores 2048
// cycles at their peak and the special function units as long.
//
//  * A block takes 256 consecutive (token, head) rows of one KV head, as two
//    tiles of 128: the heads that share a KV head share its K and V. It walks
//    the 128-token tiles that any of its rows sees, the sinks' first.
//  * One warp brings K and V by TMA, a copy per page and 128-byte half, into
//    two stages each, in the operand layout of the tensor cores (128-byte
//    swizzle). K is read K-major; V as it lies, with the tokens as K, in the
//    MN-major form.
//  * One thread issues tcgen05.mma: S = Q K^T (128 x 128, f32, in tensor
//    memory), then O += P V with P read from tensor memory. The two row tiles
//    alternate, so that one's softmax runs beside the other's products.
//  * Two groups of four warps do the softmax of one row tile each, a row per
//    thread: S from tensor memory, maximum, exponentials, P in bf16 over S's
//    columns. O is rescaled in tensor memory only when a row's maximum has
//    grown by more than 2^8 since the last time: weights up to 2^8 keep their
//    relative precision in bf16, and the sums are f32.
//  * One warp clears rows of V that no row of the block sees or that were not
//    loaded (released or bad pages, behind the last token): their weights are
//    zero, and zero times whatever lies there must not become NaN.
// Every wait is bounded; one that runs out writes KVS_ETIMEOUT, and the block
// winds down with no copy in flight and its tensor memory freed.
#include <cuda_bf16.h>

#include "async.cuh"

namespace kvs {

namespace {

constexpr int kRows = 128;                   // rows of a tile (MMA M)
constexpr int kBlockRows = 2 * kRows;
constexpr int kTok = 128;                    // tokens of a tile (MMA N of S, K of O)
constexpr int kHalfBytes = 128 * 128;        // 128 rows of one 128-byte half
constexpr int kTileBytes = 2 * kHalfBytes;   // 128 rows of 128 bf16
constexpr int kStages = 2;                   // of K, and of V
constexpr int kInfos = 4;
constexpr int kSoftWarps = 8, kLoadWarp = 8, kMmaWarp = 9, kCleanWarp = 10;
constexpr int kThreads = 32 * 12;             // three warpgroups; the last warp is idle
// registers a thread: 168 at launch; 8 * 208 + 4 * 88 = 12 * 168
constexpr int kSoftRegs = 208, kOtherRegs = 88;
constexpr float kGrow = 8.f;                 // log2 of the growth that a maximum may lag behind

struct PromptSmem {
  alignas(1024) unsigned char q[2][kTileBytes];
  unsigned char k[kStages][kTileBytes];
  unsigned char v[kStages][kTileBytes];
  uint64_t q_full, k_full[kStages], k_empty[kStages], v_full[kStages], v_empty[kStages];
  uint64_t v_clean;  // a phase for each tile that had rows to clear
  uint64_t s_full[2], p_full[2][2], o_full[2];  // p_full by tile and half of the tokens
  int groups[kInfos];  // by tile: which 16-token groups were loaded
  uint32_t tmem;
  int abort_flag;
  int item_r, item_block;
  int64_t scan[kThreads / 32];
};

struct PromptParams {
  PagedView kv;
  const uint16_t* q;
  int64_t q_ld;
  const int32_t* cu;
  int T, H, window, sinks;
  float scale_log2;  // of the magnitude of the scale
  uint32_t flip;     // sign bits of a pair of queries, turned round for a negative scale
  uint16_t* out;
  int64_t out_ld;
  float* lse;
  int32_t* dev_status;

  // the first packed row of request r, within the T there are
  __device__ __forceinline__ int start(int r) const {
    const int x = cu[r];
    if (x < 0 || x > T) set_status(dev_status, KVS_EBOUNDS);
    return min(max(x, 0), T);
  }
};

// Shared-memory matrix descriptors with the 128-byte swizzle (version 1).
// K-major: 8-row groups 1024 bytes apart.
__device__ __forceinline__ uint64_t desc_k_major(uint32_t addr) {
  return static_cast<uint64_t>((addr & 0x3FFFFu) >> 4) | (1ull << 16) | (static_cast<uint64_t>(1024 >> 4) << 32) |
         (1ull << 46) | (2ull << 61);
}
// MN-major: 64-element column blocks kHalfBytes apart, groups of 8 K rows 1024 bytes apart.
__device__ __forceinline__ uint64_t desc_mn_major(uint32_t addr) {
  return static_cast<uint64_t>((addr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(kHalfBytes >> 4) << 16) |
         (static_cast<uint64_t>(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
// f32 accumulators, bf16 operands, M = 128, N = 128; B K-major or MN-major.
constexpr uint32_t kIdesc = (1u << 4) | (1u << 7) | (1u << 10) | ((128u >> 3) << 17) | ((128u >> 4) << 24);
constexpr uint32_t kIdescMn = kIdesc | (1u << 16);

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
  return p != 0;
}
// Arrives on bar when every product issued so far is done.
__device__ __forceinline__ void mma_commit_to(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n" ::"r"(sm_addr(bar))
               : "memory");
}
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;\n" ::: "memory"); }
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;\n" ::: "memory"); }
__device__ __forceinline__ void wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory"); }
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }

// 32 columns of this warp's 32 lanes (a row per thread)
__device__ __forceinline__ void tmem_ld32(uint32_t addr, float* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
        "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15]), "=f"(r[16]),
        "=f"(r[17]), "=f"(r[18]), "=f"(r[19]), "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]), "=f"(r[24]),
        "=f"(r[25]), "=f"(r[26]), "=f"(r[27]), "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const float* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
      "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};\n" ::"r"(addr),
      "f"(r[0]), "f"(r[1]), "f"(r[2]), "f"(r[3]), "f"(r[4]), "f"(r[5]), "f"(r[6]), "f"(r[7]), "f"(r[8]), "f"(r[9]),
      "f"(r[10]), "f"(r[11]), "f"(r[12]), "f"(r[13]), "f"(r[14]), "f"(r[15]), "f"(r[16]), "f"(r[17]), "f"(r[18]),
      "f"(r[19]), "f"(r[20]), "f"(r[21]), "f"(r[22]), "f"(r[23]), "f"(r[24]), "f"(r[25]), "f"(r[26]), "f"(r[27]),
      "f"(r[28]), "f"(r[29]), "f"(r[30]), "f"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n" ::"r"(
          addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ uint32_t bf16_pair(float x, float y) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}
// two f32 in a register pair
__device__ __forceinline__ uint64_t pair(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};\n" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t v, float& x, float& y) {
  asm("mov.b64 {%0, %1}, %2;\n" : "=f"(x), "=f"(y) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
// bits [0, x) of a word
__device__ __forceinline__ uint32_t low_bits(int x) { return x <= 0 ? 0u : (x >= 32 ? 0xFFFFFFFFu : (1u << x) - 1u); }

__global__ void __launch_bounds__(kThreads, 1) paged_prompt_kernel(const PromptParams p,
                                                                   const __grid_constant__ CUtensorMap mapK,
                                                                   const __grid_constant__ CUtensorMap mapV) {
  extern __shared__ __align__(1024) unsigned char prompt_smem[];
  PromptSmem& sm = *reinterpret_cast<PromptSmem*>(prompt_smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const PagedView& kv = p.kv;
  const int G = kv.G, H = p.H;
  pdl_wait();
  pdl_trigger();

  // this block's request and rows: the blocks of all requests in order, the last ones first (they see most)
  const int g = blockIdx.x % G;
  const int order = blockIdx.x / G;
  if (tid == 0) sm.item_r = -1;
  {
    const int per = (kv.R + kThreads - 1) / kThreads;
    const int r_lo = min(kv.R, tid * per), r_hi = min(kv.R, r_lo + per);
    auto blocks_of = [&](int r) {
      return (static_cast<int64_t>(max(0, p.start(r + 1) - p.start(r))) * H + kBlockRows - 1) / kBlockRows;
    };
    int64_t mine = 0;
    for (int r = r_lo; r < r_hi; ++r) mine += blocks_of(r);
    int64_t inc = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t y = __shfl_up_sync(0xFFFFFFFFu, inc, d);
      if (lane >= d) inc += y;
    }
    if (lane == 31) sm.scan[warp] = inc;
    __syncthreads();
    int64_t total = 0, before = inc - mine;
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) before += sm.scan[w];
      total += sm.scan[w];
    }
    const int64_t x = total - 1 - order;
    if (x >= before && x < before + mine) {
      int r = r_lo;
      for (;; ++r) {
        const int64_t c = blocks_of(r);
        if (x < before + c) break;
        before += c;
      }
      sm.item_r = r;
      sm.item_block = static_cast<int>(x - before);
    }
    __syncthreads();
  }
  const int r = sm.item_r;
  if (r < 0) return;
  const int q0 = p.start(r), c = p.start(r + 1) - q0;
  const int n = kv.length(r, p.dev_status);
  const int row0 = sm.item_block * kBlockRows;             // first (token, head) row of the request
  const int rows = min(kBlockRows, c * H - row0);
  const int p_lo = n - c + row0 / H, p_hi = n - c + (row0 + rows - 1) / H;
  // tiles that any row sees
  const int end = max(0, p_hi + 1);
  const int lo = p.window && p_lo >= p.window ? p_lo - p.window + 1 : 0;
  int nsink = 0, first = 0;
  if (lo) {
    const int s = (min(p.sinks, lo) + kTok - 1) / kTok;
    if (s < lo / kTok) {
      nsink = s;
      first = lo / kTok;
    }
  }
  const int tiles = nsink + (end + kTok - 1) / kTok - first;
  // whether a tile of V has rows to clear
  auto ragged = [&](int t0, int there) {
    return there != 0xFF || t0 + kTok > end || (t0 < lo && t0 + kTok > p.sinks);
  };
  auto tile_token = [&](int i) { return (i < nsink ? i : first + i - nsink) * kTok; };

  if (tid == 0) {
    mbar_init(&sm.q_full, kSoftWarps);
    mbar_init(&sm.v_clean, 1);
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&sm.k_full[i], 1);
      mbar_init(&sm.k_empty[i], 1);
      mbar_init(&sm.v_full[i], 1);
      mbar_init(&sm.v_empty[i], 2);  // the products that read it, and the clearing warp
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.s_full[i], 1);
      mbar_init(&sm.p_full[i][0], kRows / 32);
      mbar_init(&sm.p_full[i][1], kRows / 32);
      mbar_init(&sm.o_full[i], 1);
    }
    sm.abort_flag = 0;
    mbar_init_fence();
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;\n" ::"r"(sm_addr(&sm.tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = sm.tmem;  // S of tile t at 128 t, O at 256 + 128 t

  auto fail = [&] {
    set_status(p.dev_status, KVS_ETIMEOUT);
    atomicExch(&sm.abort_flag, 1);
  };
  auto aborted = [&] { return *reinterpret_cast<volatile int*>(&sm.abort_flag) != 0; };
  auto wait = [&](uint64_t* b, uint32_t parity) {
    if (!aborted() && mbar_wait(b, parity)) return true;
    fail();
    return false;
  };

  if (warp >= kSoftWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kOtherRegs));
    if (warp == kLoadWarp) {
      // ---------------- K and V tiles ----------------
      const int box = min(1 << kv.shift, kTok), pages = kTok / box;
      const int half = lane & 1, sub = lane >> 1;
      int issued = 0;
      // this lane's page id of tile i, unchecked (nothing waits for it here); -1 where none is needed
      auto wanted = [&](int i) {
        const int t = tile_token(i) + sub * box;
        return sub < pages && t < end && (t < p.sinks || t + box > lo);
      };
      const int32_t* table = kv.table + r * kv.table_ld;
      auto look = [&](int i) { return wanted(i) ? __ldg(table + ((tile_token(i) + sub * box) >> kv.shift)) : -1; };
      int next = tiles > 0 ? look(0) : -1;
      for (int i = 0; i < tiles; ++i) {
        const int st = i % kStages;
        int id = next;
        if (i + 1 < tiles) next = look(i + 1);
        if (static_cast<unsigned>(id) >= static_cast<unsigned>(kv.num_pages)) {
          if (wanted(i)) set_status(p.dev_status, KVS_EBOUNDS);
          id = -1;
        }
        const unsigned have = __ballot_sync(0xFFFFFFFFu, id >= 0);
        const int in_page = (tile_token(i) + sub * box) & ((1 << kv.shift) - 1);
        const uint32_t at = half * kHalfBytes + sub * box * 128;
        for (int which = 0; which < 2; ++which) {
          uint64_t* full = which ? &sm.v_full[st] : &sm.k_full[st];
          int ok = 1;
          if (lane == 0) {
            if (i >= kStages) ok = wait(which ? &sm.v_empty[st] : &sm.k_empty[st], (i / kStages - 1) & 1);
            if (ok) {
              if (which == 0) {
                int there = 0;
                for (int e = 0; e < 8; ++e)
                  if (have >> (2 * (16 * e / box)) & 1u) there |= 1 << e;
                sm.groups[i % kInfos] = there;
                __threadfence_block();
              }
              if (have) mbar_expect(full, __popc(have) * box * 128);
              else mbar_arrive(full);
            }
          }
          ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
          if (!ok) break;
          if (id >= 0)
            tma_page_rows(sm_addr(which ? sm.v[st] : sm.k[st]) + at, which ? &mapV : &mapK, in_page, half, g, id, full);
          issued = 2 * i + which + 1;
        }
        if (issued < 2 * i + 2) break;
      }
      // no copy may be in flight when the block ends
      if (lane == 0)
        for (int x = max(0, issued - 2 * kStages); x < issued; ++x) {
          const int i = x / 2;
          mbar_wait(x & 1 ? &sm.v_full[i % kStages] : &sm.k_full[i % kStages], (i / kStages) & 1);
        }
    } else if (warp == kCleanWarp) {
      // ---------------- rows of V that no row of the block sees ----------------
      for (int i = 0; i < tiles; ++i) {
        const int st = i % kStages;
        int ok = 1;
        if (lane == 0) ok = wait(&sm.v_full[st], (i / kStages) & 1);
        if (!__shfl_sync(0xFFFFFFFFu, ok, 0)) break;
        const int t0 = tile_token(i), there = sm.groups[i % kInfos];
        if (ragged(t0, there)) {
          for (int x = lane; x < kTok * 16; x += 32) {
            const int row = x >> 4, t = t0 + row;
            if ((there >> (row >> 4) & 1) && t < end && (t >= lo || t < p.sinks)) continue;
            *reinterpret_cast<uint4*>(sm.v[st] + (x >> 3 & 1) * kHalfBytes + row * 128 + (x & 7) * 16) =
                make_uint4(0, 0, 0, 0);
          }
          asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.v_clean);
        }
        // the slot is not filled again before this warp has passed it: it must
        // not fall two phases of v_full behind
        if (lane == 0) mbar_arrive(&sm.v_empty[st]);
      }
    } else if (warp == kMmaWarp) {
      // ---------------- products ----------------
      // (the whole warp goes through the loop, so that descriptors stay in
      // uniform registers; one lane issues)
      if (tiles > 0) {
        const uint64_t dq = desc_k_major(sm_addr(sm.q[0])), dk = desc_k_major(sm_addr(sm.k[0])),
                       dv = desc_mn_major(sm_addr(sm.v[0]));
        const bool leader = elect_one();
        auto qk = [&](int t, int i) {
          const uint64_t a = dq + t * (kTileBytes >> 4), b = dk + (i % kStages) * (kTileBytes >> 4);
          const uint32_t d = tmem + 128 * t;
          if (leader) {
#pragma unroll
            for (int ks = 0; ks < 8; ++ks) {
              const uint64_t step = (ks >> 2) * (kHalfBytes >> 4) + (ks & 3) * 2;
              mma_ss(d, a + step, b + step, kIdesc, ks > 0);
            }
            mma_commit_to(&sm.s_full[t]);
          }
        };
        auto commit = [&](uint64_t* bar) {
          if (leader) mma_commit_to(bar);
        };
        auto wait_all = [&](uint64_t* b, uint32_t parity) { return __all_sync(0xFFFFFFFFu, wait(b, parity)) != 0; };
        int cleaned = 0;
        bool ok = wait_all(&sm.q_full, 0) && wait_all(&sm.k_full[0], 0);
        if (ok) {
          fence_after();
          qk(0, 0);
          qk(1, 0);
          commit(&sm.k_empty[0]);
        }
        for (int i = 0; i < tiles && ok; ++i) {
          const int st = i % kStages;
          ok = wait_all(&sm.v_full[st], (i / kStages) & 1);
          if (ok && ragged(tile_token(i), sm.groups[i % kInfos])) ok = wait_all(&sm.v_clean, cleaned++ & 1);
          for (int t = 0; t < 2 && ok; ++t) {
            const uint32_t d = tmem + 256 + 128 * t, a = tmem + 128 * t;
            const uint64_t b = dv + st * (kTileBytes >> 4);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              ok = ok && wait_all(&sm.p_full[t][e], i & 1);
              if (!ok) break;
              fence_after();
              if (leader) {
#pragma unroll
                for (int ks = 4 * e; ks < 4 * e + 4; ++ks)
                  mma_ts(d, a + 8 * ks, b + ks * (2048 >> 4), kIdescMn, i > 0 || ks > 0);
              }
            }
            if (!ok) break;
            if (t == 1) commit(&sm.v_empty[st]);
            if (i + 1 == tiles) {
              commit(&sm.o_full[t]);
              continue;
            }
            if (t == 0) {
              ok = wait_all(&sm.k_full[(i + 1) % kStages], ((i + 1) / kStages) & 1);
              if (!ok) break;
              fence_after();
            }
            qk(t, i + 1);
            if (t == 1) commit(&sm.k_empty[(i + 1) % kStages]);
          }
        }
        if (!ok) {  // products already issued end before the block does
          commit(&sm.o_full[0]);
          mbar_wait(&sm.o_full[0], 0);
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kSoftRegs));
    // ---------------- softmax, a row per thread ----------------
    const int t = warp >> 2;                       // row tile
    const int mine = 128 * t + (tid & 127);        // row of the block
    const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const uint32_t s_at = tmem + lanes + 128 * t, o_at = tmem + lanes + 256 + 128 * t;
    const float ninf = -__int_as_float(0x7f800000);
    // the queries, half a warp to a row, sixteen loads in flight
    const int w0 = 32 * (warp & 3), ch = lane & 15;
    // row x of the block is head v % H of token tok0 + v / H, v = row0 % H + x
    // (v < 264: the division by H is a multiplication)
    const int tok0 = row0 / H, rem = row0 - tok0 * H;
    const uint32_t by_h = 65536u / H + 1;
    auto token_of = [&](int x) { return static_cast<int>((rem + x) * by_h >> 16); };
    auto row_of = [&](int x, int64_t ld) {  // element offset of the row
      const int tk = token_of(x);
      return (q0 + tok0 + tk) * ld + (g * H + rem + x - tk * H) * kD;
    };
    {
      uint4 v[16];
#pragma unroll
      for (int x = 0; x < 16; ++x) {
        const int rr = 128 * t + w0 + 2 * x + (lane >> 4);
        v[x] = make_uint4(0, 0, 0, 0);
        if (rr < rows) v[x] = __ldg(reinterpret_cast<const uint4*>(p.q + row_of(rr, p.q_ld) + 8 * ch));
      }
#pragma unroll
      for (int x = 0; x < 16; ++x) {
        const int rr = w0 + 2 * x + (lane >> 4);
        v[x].x ^= p.flip;
        v[x].y ^= p.flip;
        v[x].z ^= p.flip;
        v[x].w ^= p.flip;
        *reinterpret_cast<uint4*>(sm.q[t] + (ch >> 3) * kHalfBytes + rr * 128 + (((ch & 7) ^ (rr & 7)) << 4)) = v[x];
      }
    }
    asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.q_full);

    const int pos = p_lo + token_of(min(mine, rows - 1));
    // the first and last position of this warp's rows
    const int p_first = p_lo + token_of(min(128 * t + w0, rows - 1));
    const int p_last = p_lo + token_of(min(128 * t + w0 + 31, rows - 1));
    float m = ninf, l = 0.f;
    bool ok = true;
    for (int i = 0; i < tiles; ++i) {
      if (!__all_sync(0xFFFFFFFFu, wait(&sm.s_full[t], i & 1))) {
        ok = false;
        break;
      }
      fence_after();
      float s[kTok];
#pragma unroll
      for (int e = 0; e < 4; ++e) tmem_ld32(s_at + 32 * e, s + 32 * e);
      wait_ld();
      const int t0 = tile_token(i), there = sm.groups[i % kInfos];
      const bool whole = there == 0xFF && t0 + kTok - 1 <= p_first &&
                         (!p.window || t0 > p_last - p.window || t0 + kTok <= p.sinks);
      if (!whole) {
        // bit j of a word: this row sees token t0 + 32 e + j
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int b = t0 + 32 * e;
          uint32_t see = low_bits(pos + 1 - b);
          if (p.window) see &= ~low_bits(pos - p.window + 1 - b) | low_bits(p.sinks - b);
          see &= (there >> (2 * e) & 1 ? 0xFFFFu : 0u) | (there >> (2 * e + 1) & 1 ? 0xFFFF0000u : 0u);
#pragma unroll
          for (int j = 0; j < 32; ++j) s[32 * e + j] = see >> j & 1u ? s[32 * e + j] : ninf;
        }
      }
      float x0 = s[0], x1 = s[1], x2 = s[2], x3 = s[3];
#pragma unroll
      for (int j = 4; j < kTok; j += 4) {
        x0 = fmaxf(x0, s[j]);
        x1 = fmaxf(x1, s[j + 1]);
        x2 = fmaxf(x2, s[j + 2]);
        x3 = fmaxf(x3, s[j + 3]);
      }
      float top = fmaxf(fmaxf(x0, x1), fmaxf(x2, x3)) * p.scale_log2;
      const bool grow = top > m + kGrow || (m == ninf && top > ninf);
      if (__any_sync(0xFFFFFFFFu, grow)) {
        const float to = grow ? top : m;
        const float a = grow ? exp2_fast(m - to) : 1.f;
        m = to;
        l *= a;
        if (i > 0) {
#pragma unroll 1
          for (int e = 0; e < 4; ++e) {
            float o[32];
            tmem_ld32(o_at + 32 * e, o);
            wait_ld();
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] *= a;
            tmem_st32(o_at + 32 * e, o);
          }
        }
      }
      const float f = m == ninf ? 0.f : m;
      const uint64_t scale2 = pair(p.scale_log2, p.scale_log2), f2 = pair(-f, -f);
      uint64_t z[2] = {0, 0};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        uint32_t w[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          float a, b;
          unpair(fma2(pair(s[32 * e + 2 * j], s[32 * e + 2 * j + 1]), scale2, f2), a, b);
          a = exp2_fast(a);
          b = exp2_fast(b);
          z[j & 1] = add2(z[j & 1], pair(a, b));
          w[j] = bf16_pair(a, b);
        }
        tmem_st16(s_at + 16 * e, w);
        if (e & 1) {  // half of the tokens: their product can begin
          wait_st();
          fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.p_full[t][e >> 1]);
        }
      }
      float z0, z1;
      unpair(add2(z[0], z[1]), z0, z1);
      l += z0 + z1;
    }
    // ---------------- the rows' output ----------------
    // through this warp's rows of the queries, which no product reads any more
    // (rounded to bf16 here), so that half a warp writes a row. (Loops that are
    // not unrolled: code that runs once a block is fetched once a block.)
    const bool done = ok && tiles > 0 && __all_sync(0xFFFFFFFFu, wait(&sm.o_full[t], 0));
    fence_after();
    const float inv = !done ? 0.f : (l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l));
    unsigned char* rows_at = sm.q[t] + w0 * 128;
#pragma unroll 1
    for (int e = 0; e < 4; ++e) {
      float o[32];
      tmem_ld32(o_at + 32 * e, o);
      wait_ld();
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint4 v = make_uint4(bf16_pair(o[8 * j] * inv, o[8 * j + 1] * inv), bf16_pair(o[8 * j + 2] * inv, o[8 * j + 3] * inv),
                             bf16_pair(o[8 * j + 4] * inv, o[8 * j + 5] * inv),
                             bf16_pair(o[8 * j + 6] * inv, o[8 * j + 7] * inv));
        if (!done) v = make_uint4(0, 0, 0, 0);  // tensor memory that nothing was written to
        *reinterpret_cast<uint4*>(rows_at + (e >> 1) * kHalfBytes + lane * 128 +
                                  (((4 * (e & 1) + j) ^ (lane & 7)) << 4)) = v;
      }
    }
    if (mine < rows && p.lse)
      p.lse[row_of(mine, static_cast<int64_t>(G) * H * kD) / kD] =
          l == 0.f ? ninf : (m + log2f(l)) * 0.6931471805599453f;
    __syncwarp();
#pragma unroll 4
    for (int x = 0; x < 16; ++x) {
      const int rr = 2 * x + (lane >> 4);
      if (128 * t + w0 + rr < rows)
        *reinterpret_cast<uint4*>(p.out + row_of(128 * t + w0 + rr, p.out_ld) + 8 * ch) =
            *reinterpret_cast<const uint4*>(rows_at + (ch >> 3) * kHalfBytes + rr * 128 + (((ch & 7) ^ (rr & 7)) << 4));
    }
  }
  fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;\n" ::"r"(tmem) : "memory");
  }
}

}  // namespace

kvs_status paged_prompt_launch(const kvs_paged_prompt_args* a, int32_t* dev_status, cudaStream_t s) {
  PromptParams p{};
  p.kv = paged_view(a->kv);
  p.q = a->q;
  p.q_ld = a->q_ld;
  p.cu = a->cu;
  p.T = a->T;
  p.H = a->H;
  p.window = a->window;
  p.sinks = a->sinks;
  p.scale_log2 = (a->scale < 0.f ? -a->scale : a->scale) * 1.4426950408889634f;
  p.flip = a->scale < 0.f ? 0x80008000u : 0u;
  p.out = a->out;
  p.out_ld = a->out_ld;
  p.lse = a->lse;
  p.dev_status = dev_status;
  const int box = a->kv->page < kTok ? a->kv->page : kTok;
  CUtensorMap mk, mv;
  kvs_status st = paged_tensor_map(&mk, a->kv->K, p.kv, box, 1, "paged_prompt_attn");
  if (st == KVS_OK) st = paged_tensor_map(&mv, a->kv->V, p.kv, box, 1, "paged_prompt_attn");
  if (st != KVS_OK) return st;
  // no more blocks than this have rows, whatever the lengths: a part block a request, and whole ones
  const int64_t whole = static_cast<int64_t>(a->T) * a->H / kBlockRows;
  const int64_t part = a->T < p.kv.R ? a->T : p.kv.R;
  const int64_t grid = (whole + part) * p.kv.G;
  KVS_REQUIRE(grid < (1ll << 31), KVS_EUNSUPPORTED, "paged_prompt_attn: T=%d rows of G=%d heads", a->T, p.kv.G);
  allow_smem<paged_prompt_kernel>(sizeof(PromptSmem));
  launch_chained(paged_prompt_kernel, dim3(static_cast<unsigned>(grid)), dim3(kThreads), sizeof(PromptSmem), s, p, mk,
                 mv);
  return check_launch("paged_prompt_attn");
}

}  // namespace kvs
