// paged_decode.cu -- attention of each request's newest token over its paged
// cache, optionally with every token's softmax weights added up.
//
// For (r, g) and query head h: l_j = scale * q_h . K_j over the visible tokens,
// out = sum_j softmax(l)_j V_j, in base 2 with an online softmax. 512 bytes of
// K and V are read per token for 4 * 128 * H flops: HBM bounds it.
//
//  * The visible tokens of all (r, g) rows are cut into units of 64 and laid
//    end to end; each block takes an equal run of them, whatever the lengths.
//    A row that lies inside one run is finished there; of a cut row, each
//    block leaves its maximum, sum and unnormalised output, and a second
//    kernel joins them. A run cuts at most the row it begins in and the row it
//    ends in, so the scratch is two partial rows a block, independent of n. That
//    kernel has a block for every row, or, with more rows than SMs, for every
//    run's end.
//  * One warp loads: a TMA copy per page and pool brings up to 64 tokens of one
//    head (both 128-byte halves, swizzled) into a ring of three 32 KB stages,
//    with what the consumers need to know about the unit beside it. Two blocks
//    share an SM (192 KB in flight).
//  * Four warps compute, 16 tokens of a unit each: S[tokens][heads] = K q^T and
//    O^T[dims][heads] += V^T P^T on mma.m16n8k16, tokens as M of the first and
//    as K of the second, the 8 columns the heads. bf16 queries are exact; f32
//    queries and the weights are split in three bf16 parts (24 bits). Each
//    16-token product is summed in the tensor core and added to the running
//    output in f32 with the rescaling as one fma: the tensor core truncates
//    its sums, and over thousands of tokens that would show.
//  * V rows that are masked or were not loaded are cleared in the registers:
//    whatever lies there (NaN too) must not meet a weight of zero.
//  * With weights wanted, the logits go to scratch (4 H bytes a token beside
//    the 512 read) and the join turns them into weights, once the row's
//    log-sum-exp is known (a kernel of its own with more than four rows an SM).
//  * Every wait is bounded; one that runs out writes KVS_ETIMEOUT. The computing
//    warps meet at a row's end, at mbarriers too: warp 0 adds up the others' parts
//    while they go on with the next row.
// Measured: 16 requests of 16K to 128K tokens, 3.70 GB: 0.60 to 0.61 ms (6.1 TB/s
// of the 6.55 a copy reaches); 32 requests seeing 4100 tokens each, 8 heads: 89.5 us
// (5.65 TB/s); 16 of 3K to 8K with weights 71.5 us; one request of 4096 tokens: 10.9
// us, 2.5 of them the join.
#include <cuda_bf16.h>

#include <algorithm>

#include "async.cuh"

namespace kvs {

namespace {

constexpr int kUnit = 64;
constexpr int kStages = 3;
constexpr int kConsumers = 4;  // warps, 16 tokens of a unit each
constexpr int kThreads = 32 * (kConsumers + 1);
constexpr int kBlocksPerSM = 2;
constexpr int kPoolBytes = kUnit * kD * 2;     // K or V of a unit
constexpr int kStageBytes = 2 * kPoolBytes;
constexpr int kMinUnits = 2;                   // units a block takes at least
constexpr int kTestUnit = 1;
constexpr int kPartRow = kD + 4;               // maximum, sum, -, -, output
constexpr int kPartSlots = 2;

// flags of a unit, beside the bits of its four 16-token groups that were loaded
constexpr int kFirst = 16, kLast = 32, kSlotShift = 6;  // slot 0: complete row, 1 + s: partial slot s

struct UnitInfo {
  int row;   // r * G + g
  int tok;   // first token
  int n;
  int flags;
};

struct DecodeSmem {
  alignas(1024) unsigned char ring[kStages][kStageBytes];
  float merge[kConsumers - 1][8][kD];
  float ml[kConsumers - 1][8][2];
  UnitInfo info[kStages];
  uint64_t full[kStages], empty[kStages];
  uint64_t parts_in, parts_out;  // the merge of a row: parts of the other warps there, and taken by warp 0
  int abort_flag;
};

struct DecodeParams {
  PagedView kv;
  const void* q;
  int H, window, sinks;
  float scale_log2;
  float* out;
  float* lse;
  const float* mass;
  float* mass_out;
  float* part;     // [blocks][kPartSlots][H][kPartRow]
  float* lse2;     // [R*G][H], base 2, of rows that one block finished (weights only)
  float* logits;   // [R*G][cap][hp], base 2 (weights only)
  int hp;          // H rounded up to 2, 4 or 8
  int blocks;
  int32_t* dev_status;
  long long wait_cycles;  // of the self-test
  int test_warp;
};

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void ldsm4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, "
      "%2, %3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(y) : "r"(x));
  return y;
}
// x and y as bf16 in one register, and what the rounding left of them
__device__ __forceinline__ uint32_t take_bf16(float& x, float& y) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
  const uint32_t b = *reinterpret_cast<const uint32_t*>(&v);
  x -= __uint_as_float(b << 16);
  y -= __uint_as_float(b & 0xFFFF0000u);
  return b;
}

// Blocks that share U units (every kernel computes the same), and the first
// unit of block b.
__device__ __forceinline__ int sharing(int64_t U, int blocks) {
  const int64_t most = (U + kMinUnits - 1) / kMinUnits;
  return most < blocks ? static_cast<int>(most) : blocks;
}
__device__ __forceinline__ int64_t first_unit(int64_t U, int b, int nb) { return U * b / nb; }
__device__ __forceinline__ int block_of_unit(int64_t U, int64_t x, int nb) {
  return static_cast<int>(((x + 1) * nb - 1) / U);
}

// Sum over the block of each thread's v, and the sum of the threads before it.
template <int kT>
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* part, int64_t& total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int64_t inc = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t y = __shfl_up_sync(0xFFFFFFFFu, inc, d);
    if (lane >= d) inc += y;
  }
  if (lane == 31) part[warp] = inc;
  __syncthreads();
  int64_t before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < kT / 32; ++w) {
    if (w < warp) before += part[w];
    total += part[w];
  }
  return before + inc - v;
}

// kTest: every wait is bounded by wait_cycles, and in every block that has as many
// units warp test_warp gives up at unit kTestUnit.
template <bool kF32Q, bool kWeights, bool kTest = false>
__global__ void __launch_bounds__(kThreads, kBlocksPerSM) paged_decode_kernel(const DecodeParams p,
                                                                              const __grid_constant__ CUtensorMap mapK,
                                                                              const __grid_constant__ CUtensorMap mapV) {
  extern __shared__ __align__(1024) unsigned char decode_smem[];
  DecodeSmem& sm = *reinterpret_cast<DecodeSmem*>(decode_smem);
  __shared__ int64_t scan_part[kThreads / 32];
  __shared__ int s_r, s_n, s_g, s_k;  // where the run begins: request, its length, KV head, tile
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const PagedView& kv = p.kv;
  const int G = kv.G;
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&sm.full[i], 1);
      mbar_init(&sm.empty[i], kConsumers);
    }
    mbar_init(&sm.parts_in, kConsumers - 1);
    mbar_init(&sm.parts_out, 1);
    sm.abort_flag = 0;
    mbar_init_fence();
    tma_prefetch_map(&mapK);
    tma_prefetch_map(&mapV);
  }
  pdl_wait();
  pdl_trigger();

  // this block's run of units, and the request it begins in
  const int per = (kv.R + kThreads - 1) / kThreads;
  const int r_lo = min(kv.R, tid * per), r_hi = min(kv.R, r_lo + per);
  int64_t mine = 0;
  int n_lo = 0;
  for (int r = r_lo; r < r_hi; ++r) {
    const int n = kv.length(r, p.dev_status);
    if (r == r_lo) n_lo = n;
    mine += VisibleTiles<kUnit>(n, p.window, p.sinks).count;
  }
  int64_t U;
  int64_t before = block_scan<kThreads>(mine, scan_part, U) * G;
  U *= G;
  const int nb = sharing(U, p.blocks);
  if (static_cast<int>(blockIdx.x) >= nb) return;
  const int64_t u0 = first_unit(U, blockIdx.x, nb), u1 = first_unit(U, blockIdx.x + 1, nb);
  if (u0 >= before && u0 < before + mine * G) {
    int r = r_lo, n = n_lo, count;
    for (;; n = kv.length(++r, nullptr)) {
      count = VisibleTiles<kUnit>(n, p.window, p.sinks).count;
      if (u0 < before + static_cast<int64_t>(count) * G) break;
      before += static_cast<int64_t>(count) * G;
    }
    const int64_t into = u0 - before;
    const int g = into >> 31 ? static_cast<int>(into / count) : static_cast<int>(into) / count;  // (64 bits are slow)
    s_r = r;
    s_n = n;
    s_g = g;
    s_k = static_cast<int>(into - static_cast<int64_t>(g) * count);
  }
  __syncthreads();
  const int units = static_cast<int>(u1 - u0);

  auto aborted = [&] { return *reinterpret_cast<volatile int*>(&sm.abort_flag) != 0; };
  // By a whole warp, every lane for itself (what the barrier guards is ordered for
  // the lanes that have seen its phase). A warp whose wait runs out leaves, and the
  // others, which may have seen the same phase come, run out of their own next
  // waits: no warp meets another at anything but such a wait.
  const long long limit = kTest ? p.wait_cycles : kWaitCycles;
  auto wait = [&](uint64_t* b, uint32_t parity) {
    if (__all_sync(0xFFFFFFFFu, mbar_try(b, parity))) return true;
    if (__all_sync(0xFFFFFFFFu, !aborted() && mbar_wait(b, parity, limit))) return true;
    if (lane == 0) {
      set_status(p.dev_status, KVS_ETIMEOUT);
      atomicExch(&sm.abort_flag, 1);
    }
    return false;
  };

  if (warp == kConsumers) {
    // ---------------- loads ----------------
    const int rows = min(1 << kv.shift, kUnit), copies = 2 * (kUnit / rows);
    const bool isv = lane & 1;
    const int sub = lane >> 1;  // this lane's page within the unit
    int r = s_r, g = s_g, k = s_k;
    VisibleTiles<kUnit> vt(s_n, p.window, p.sinks);
    const int k_start = k;
    UnitInfo next;
    int next_id;
    // the unit at (r, g, k), its flags and this lane's page
    auto look = [&](int i) {
      next.row = r * G + g;
      next.tok = vt.tile(k) * kUnit;
      next.n = vt.end;
      next.flags = 0;
      if (i == 0 || k == 0) next.flags |= kFirst;
      if (i == units - 1 || k == vt.count - 1) {
        next.flags |= kLast;
        const bool began_before = k_start > 0 && k == k_start + i;  // still the row that the run begins in
        const bool goes_on = k < vt.count - 1;
        next.flags |= (began_before ? 1 : (goes_on ? 2 : 0)) << kSlotShift;
      }
      const int t = next.tok + sub * rows;
      next_id = -1;
      if (lane < copies && t < vt.end && (t < p.sinks || t + rows > vt.lo)) next_id = kv.page_of(r, t, p.dev_status);
    };
    look(0);
    int issued = 0;
    for (int i = 0; i < units; ++i) {
      const int st = i % kStages;
      const UnitInfo info = next;
      const int id = next_id;
      if (i + 1 < units) {
        if (++k == vt.count) {
          k = 0;
          if (++g == G) {
            g = 0;
            do {
              ++r;
              vt = VisibleTiles<kUnit>(kv.length(r, nullptr), p.window, p.sinks);
            } while (vt.count == 0);
          }
        }
        look(i + 1);
      }
      const unsigned have = __ballot_sync(0xFFFFFFFFu, id >= 0);
      if (i >= kStages && !wait(&sm.empty[st], (i / kStages - 1) & 1)) break;
      if (kTest && p.test_warp == kConsumers && i == kTestUnit) break;  // (this unit never comes)
      if (lane == 0) {
        int groups = 0;  // 16-token groups that are there
        for (int e = 0; e < 4; ++e)
          if (have >> (2 * (16 * e / rows)) & 1u) groups |= 1 << e;
        sm.info[st] = {info.row, info.tok, info.n, info.flags | groups};
        if (have) mbar_expect(&sm.full[st], __popc(have) * rows * kD * 2);
        else mbar_arrive(&sm.full[st]);
      }
      __syncwarp();
      if (id >= 0) {
        const int in_page = (info.tok + sub * rows) & ((1 << kv.shift) - 1);
        tma_page_rows(sm_addr(sm.ring[st]) + (isv ? kPoolBytes : 0) + sub * rows * kD * 2, isv ? &mapV : &mapK, in_page,
                      0, info.row % G, id, &sm.full[st]);
      }
      ++issued;
    }
    // no copy may be in flight when the block ends
    if (lane == 0)
      for (int i = max(0, issued - kStages); i < issued; ++i) mbar_wait(&sm.full[i % kStages], (i / kStages) & 1, limit);
    return;
  }

  // ---------------- arithmetic ----------------
  const float ninf = -__int_as_float(0x7f800000);
  const int gq = lane >> 2, tq = lane & 3;  // fragment row and column pair
  const int hA = 2 * tq, hB = hA + 1;       // this lane's heads
  const int H = p.H;
  const int rows = min(1 << kv.shift, kUnit);
  const uint32_t half = rows * kD;  // bytes from a row's first half to its second
  const uint32_t grp = (16 * warp / rows) * rows * kD * 2 + (16 * warp % rows) * kD;
  // ldmatrix rows of this lane: K (tokens as rows) and V (tokens as columns)
  const int krow = lane & 15, kc = lane >> 4;
  const int vrow = (lane & 7) + 8 * (lane >> 4), vc = (lane >> 3) & 1;
  const uint32_t koff = grp + krow * kD, voff = kPoolBytes + grp + vrow * kD;
  constexpr int kQ = kF32Q ? 3 : 1;
  uint32_t qf[kQ][8][2];
  float o[8][4];
  float mA = ninf, mB = ninf, lA = 0.f, lB = 0.f;

  // a row's queries, head = fragment column gq
  auto load_q = [&](int row) {
#pragma unroll
    for (int ks = 0; ks < 8; ++ks)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const size_t at = (static_cast<size_t>(row) * H + min(gq, H - 1)) * kD + 16 * ks + 8 * e + 2 * tq;
        if constexpr (kF32Q) {
          float2 v = *reinterpret_cast<const float2*>(static_cast<const float*>(p.q) + at);
#pragma unroll
          for (int s = 0; s < 3; ++s) qf[s][ks][e] = take_bf16(v.x, v.y);
        } else {
          qf[0][ks][e] = *reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(p.q) + at);
        }
      }
  };
  load_q(s_r * G + s_g);  // while the first unit is on its way
  uint32_t merged = 0;    // rows, or parts of rows, that have ended here
  for (int i = 0; i < units; ++i) {
    const int st = i % kStages;
    if (!wait(&sm.full[st], (i / kStages) & 1)) break;
    if (kTest && p.test_warp == warp && i == kTestUnit) break;  // (as though the wait had run out)
    const UnitInfo info = sm.info[st];
    if (info.flags & kFirst) {
      // a new row
      if (i > 0) load_q(info.row);
      // the next row's on their way to L1 meanwhile, a line a lane (4096 rows of 256
      // tokens: 103 us became 99, 96 since)
      if (info.row + 1 < kv.R * G && lane < H * kD * (kF32Q ? 4 : 2) / 128)
        asm volatile("prefetch.global.L1 [%0];\n" ::"l"(
            static_cast<const char*>(p.q) + static_cast<size_t>(info.row + 1) * H * kD * (kF32Q ? 4 : 2) + 128 * lane));
#pragma unroll
      for (int d = 0; d < 8; ++d)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[d][e] = 0.f;
      mA = mB = ninf;
      lA = lB = 0.f;
    }
    const int t0 = info.tok + 16 * warp;
    const int lo = p.window && info.n > p.window ? info.n - p.window : 0;
    const bool there = info.flags >> warp & 1;
    auto sees = [&](int t) { return there && t < info.n && (t >= lo || t < p.sinks); };
    const bool v0 = sees(t0 + gq), v8 = sees(t0 + gq + 8);
    const bool any = __any_sync(0xFFFFFFFFu, v0 || v8);
    const bool all = __all_sync(0xFFFFFFFFu, v0 && v8);
    float s4[4] = {ninf, ninf, ninf, ninf};
    if (any) {
      const uint32_t base = sm_addr(sm.ring[st]);
      // S[tokens][heads]
      // (the lower parts of f32 queries summed apart: fewer truncations at full size)
      float sc[4] = {0.f, 0.f, 0.f, 0.f}, sl[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int ks = 0; ks < 8; ++ks) {
        uint32_t a[4];
        ldsm4(base + koff + (ks >> 2) * half + (((2 * (ks & 3) + kc) ^ (krow & 7)) << 4), a);
        mma16816(sc, a, qf[0][ks][0], qf[0][ks][1]);
#pragma unroll
        for (int s = kQ - 1; s > 0; --s) mma16816(sl, a, qf[s][ks][0], qf[s][ks][1]);
      }
      if constexpr (kF32Q)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[e] += sl[e];
      s4[0] = v0 ? sc[0] * p.scale_log2 : ninf;
      s4[1] = v0 ? sc[1] * p.scale_log2 : ninf;
      s4[2] = v8 ? sc[2] * p.scale_log2 : ninf;
      s4[3] = v8 ? sc[3] * p.scale_log2 : ninf;
      float xA = fmaxf(s4[0], s4[2]), xB = fmaxf(s4[1], s4[3]);
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) {
        xA = fmaxf(xA, __shfl_xor_sync(0xFFFFFFFFu, xA, d));
        xB = fmaxf(xB, __shfl_xor_sync(0xFFFFFFFFu, xB, d));
      }
      const float nA = fmaxf(mA, xA), nB = fmaxf(mB, xB);
      // a head whose logits are all -inf keeps its maximum there: reference 0
      const float fA = nA == ninf ? 0.f : nA, fB = nB == ninf ? 0.f : nB;
      const float alA = exp2f(mA - fA), alB = exp2f(mB - fB);
      float w4[4] = {exp2f(s4[0] - fA), exp2f(s4[1] - fB), exp2f(s4[2] - fA), exp2f(s4[3] - fB)};
      lA = lA * alA + (w4[0] + w4[2]);
      lB = lB * alB + (w4[1] + w4[3]);
      mA = nA;
      mB = nB;
      // P^T, in three parts
      uint32_t b[3][2];
#pragma unroll
      for (int s = 0; s < 3; ++s) {
        b[s][0] = transpose8x8(take_bf16(w4[0], w4[1]));
        b[s][1] = transpose8x8(take_bf16(w4[2], w4[3]));
      }
      // V rows of this lane's fragment columns, cleared where they are not seen
      const uint32_t k0 = (sees(t0 + 2 * tq) ? 0xFFFFu : 0u) | (sees(t0 + 2 * tq + 1) ? 0xFFFF0000u : 0u);
      const uint32_t k8 = (sees(t0 + 2 * tq + 8) ? 0xFFFFu : 0u) | (sees(t0 + 2 * tq + 9) ? 0xFFFF0000u : 0u);
#pragma unroll
      for (int mt = 0; mt < 8; ++mt) {
        uint32_t a[4];
        ldsm4_trans(base + voff + (mt >> 2) * half + (((2 * (mt & 3) + vc) ^ (vrow & 7)) << 4), a);
        if (!all) {
          a[0] &= k0;
          a[1] &= k0;
          a[2] &= k8;
          a[3] &= k8;
        }
        float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 2; s >= 0; --s) mma16816(c, a, b[s][0], b[s][1]);
        o[mt][0] = fmaf(o[mt][0], alA, c[0]);
        o[mt][1] = fmaf(o[mt][1], alB, c[1]);
        o[mt][2] = fmaf(o[mt][2], alA, c[2]);
        o[mt][3] = fmaf(o[mt][3], alB, c[3]);
      }
    }
    if constexpr (kWeights) {
      if (hA < p.hp) {
        float* l = p.logits + (static_cast<size_t>(info.row) * kv.cap() + t0 + gq) * p.hp + hA;
        if (t0 + gq < info.n) *reinterpret_cast<float2*>(l) = make_float2(s4[0], s4[1]);
        if (t0 + gq + 8 < info.n) *reinterpret_cast<float2*>(l + 8 * p.hp) = make_float2(s4[2], s4[3]);
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.empty[st]);

    if (info.flags & kLast) {
      // the row ends here, or this block's part of it: the warps' parts into warp 0's
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) {
        lA += __shfl_xor_sync(0xFFFFFFFFu, lA, d);
        lB += __shfl_xor_sync(0xFFFFFFFFu, lB, d);
      }
      if (warp > 0) {
        if (merged > 0 && !wait(&sm.parts_out, (merged - 1) & 1)) break;
        float(&mo)[8][kD] = sm.merge[warp - 1];
#pragma unroll
        for (int mt = 0; mt < 8; ++mt) {
          mo[hA][16 * mt + gq] = o[mt][0];
          mo[hB][16 * mt + gq] = o[mt][1];
          mo[hA][16 * mt + gq + 8] = o[mt][2];
          mo[hB][16 * mt + gq + 8] = o[mt][3];
        }
        if (gq == 0) {
          sm.ml[warp - 1][hA][0] = mA;
          sm.ml[warp - 1][hA][1] = lA;
          sm.ml[warp - 1][hB][0] = mB;
          sm.ml[warp - 1][hB][1] = lB;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.parts_in);
      } else {
        if (!wait(&sm.parts_in, merged & 1)) break;
        float MA = mA, MB = mB;
#pragma unroll
        for (int w = 0; w < kConsumers - 1; ++w) {
          MA = fmaxf(MA, sm.ml[w][hA][0]);
          MB = fmaxf(MB, sm.ml[w][hB][0]);
        }
        const float fA = MA == ninf ? 0.f : MA, fB = MB == ninf ? 0.f : MB;
        const float sA = exp2f(mA - fA), sB = exp2f(mB - fB);
        lA *= sA;
        lB *= sB;
#pragma unroll
        for (int mt = 0; mt < 8; ++mt) {
          o[mt][0] *= sA;
          o[mt][1] *= sB;
          o[mt][2] *= sA;
          o[mt][3] *= sB;
        }
#pragma unroll
        for (int w = 0; w < kConsumers - 1; ++w) {
          const float cA = exp2f(sm.ml[w][hA][0] - fA), cB = exp2f(sm.ml[w][hB][0] - fB);
          lA = fmaf(sm.ml[w][hA][1], cA, lA);
          lB = fmaf(sm.ml[w][hB][1], cB, lB);
          float(&mo)[8][kD] = sm.merge[w];
#pragma unroll
          for (int mt = 0; mt < 8; ++mt) {
            o[mt][0] = fmaf(mo[hA][16 * mt + gq], cA, o[mt][0]);
            o[mt][1] = fmaf(mo[hB][16 * mt + gq], cB, o[mt][1]);
            o[mt][2] = fmaf(mo[hA][16 * mt + gq + 8], cA, o[mt][2]);
            o[mt][3] = fmaf(mo[hB][16 * mt + gq + 8], cB, o[mt][3]);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.parts_out);
        const int slot = info.flags >> kSlotShift;
        float *dA, *dB;
        float iA = 1.f, iB = 1.f;
        if (slot == 0) {
          dA = p.out + (static_cast<size_t>(info.row) * H + hA) * kD;
          dB = dA + kD;
          iA = lA > 0.f ? 1.f / lA : (lA == 0.f ? 0.f : lA);  // nothing seen: 0; NaN stays
          iB = lB > 0.f ? 1.f / lB : (lB == 0.f ? 0.f : lB);
          if (gq == 0) {
            const float zA = lA == 0.f ? ninf : MA + log2f(lA), zB = lB == 0.f ? ninf : MB + log2f(lB);
            const size_t at = static_cast<size_t>(info.row) * H + hA;
            if (p.lse && hA < H) p.lse[at] = zA * 0.6931471805599453f;
            if (p.lse && hB < H) p.lse[at + 1] = zB * 0.6931471805599453f;
            if (kWeights && hA < H) p.lse2[at] = zA;
            if (kWeights && hB < H) p.lse2[at + 1] = zB;
          }
        } else {
          float* pp = p.part + ((static_cast<size_t>(blockIdx.x) * kPartSlots + slot - 1) * H + hA) * kPartRow;
          if (gq == 0 && hA < H) pp[0] = MA, pp[1] = lA;
          if (gq == 0 && hB < H) pp[kPartRow] = MB, pp[kPartRow + 1] = lB;
          dA = pp + 4;
          dB = dA + kPartRow;
        }
#pragma unroll
        for (int mt = 0; mt < 8; ++mt) {
          if (hA < H) {
            dA[16 * mt + gq] = o[mt][0] * iA;
            dA[16 * mt + gq + 8] = o[mt][2] * iA;
          }
          if (hB < H) {
            dB[16 * mt + gq] = o[mt][1] * iB;
            dB[16 * mt + gq + 8] = o[mt][3] * iB;
          }
        }
      }
      ++merged;
    }
  }
}

constexpr int kJoinThreads = 512;
constexpr int kJoinWarps = kJoinThreads / 32;
constexpr int kFewBatch = 8;
constexpr int kCutThreads = 256;  // with 69 registers a thread three blocks an SM
constexpr int kWeighThreads = 256, kWeighTokens = 1024, kWeighBlocksPerSM = 8;
constexpr int kWeighRowsPerSM = 4;  // with more rows the weights have a kernel of their own
constexpr int kJoinTokens = 2048;  // tokens of a row that one block turns into weights

// Parts way, way + ways, ... of a head, their maximum M, sum L and output acc
// (four channels a lane) relative to it, kFewBatch of them loaded at a time.
template <typename Part>
__device__ __forceinline__ void join_parts(Part part, int way, int ways, int parts, int lane, float& M, float& L,
                                           float4& acc) {
  const float ninf = -__int_as_float(0x7f800000);
  M = ninf;
  L = 0.f;
  acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int x0 = way; x0 < parts; x0 += kFewBatch * ways) {
    float2 ml[kFewBatch];
    float4 v[kFewBatch];
#pragma unroll
    for (int e = 0; e < kFewBatch; ++e) {
      const int x = x0 + e * ways;
      ml[e] = make_float2(ninf, 0.f);
      v[e] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (x < parts) {
        ml[e] = *reinterpret_cast<const float2*>(part(x));
        v[e] = *reinterpret_cast<const float4*>(part(x) + 4 + 4 * lane);
      }
    }
    float top = M;
#pragma unroll
    for (int e = 0; e < kFewBatch; ++e) top = fmaxf(top, ml[e].x);
    const float f = top == ninf ? 0.f : top, a = exp2f(M - f);
    M = top;
    L *= a;
    acc.x *= a;
    acc.y *= a;
    acc.z *= a;
    acc.w *= a;
#pragma unroll
    for (int e = 0; e < kFewBatch; ++e) {
      const float c = exp2f(ml[e].x - f);
      L = fmaf(c, ml[e].y, L);
      acc.x = fmaf(c, v[e].x, acc.x);
      acc.y = fmaf(c, v[e].y, acc.y);
      acc.z = fmaf(c, v[e].z, acc.z);
      acc.w = fmaf(c, v[e].w, acc.w);
    }
  }
}

// Blocks b0 .. b1 hold parts of row u (r, g); the whole block works it out. The
// lengths may be read before the wait on the attention kernel: every block of
// that kernel had waited for whatever came before it when this one was let go.
template <int kT>
__device__ __forceinline__ void blocks_of_row(const DecodeParams& p, int r, int g, const VisibleTiles<kUnit>& vt,
                                              int64_t (&scan_part)[2][kT / 32], int& b0, int& b1) {
  const PagedView& kv = p.kv;
  int64_t all = 0, before = 0;
  for (int x = threadIdx.x; x < kv.R; x += kT) {
    const int c = VisibleTiles<kUnit>(kv.length(x, nullptr), p.window, p.sinks).count;
    all += c;
    if (x < r) before += c;
  }
  int64_t U, base;
  block_scan<kT>(all, scan_part[0], U);
  block_scan<kT>(before, scan_part[1], base);
  U *= kv.G;
  base = base * kv.G + static_cast<int64_t>(g) * vt.count;
  b0 = b1 = 0;
  if (vt.count) {
    const int nb = sharing(U, p.blocks);
    b0 = block_of_unit(U, base, nb);
    b1 = block_of_unit(U, base + vt.count - 1, nb);
  }
}

// A row that nothing is seen of.
__device__ __forceinline__ void write_nothing(const DecodeParams& p, int u) {
  for (int e = threadIdx.x; e < p.H * kD; e += blockDim.x) p.out[static_cast<size_t>(u) * p.H * kD + e] = 0.f;
  if (p.lse && threadIdx.x < p.H) p.lse[static_cast<size_t>(u) * p.H + threadIdx.x] = -__int_as_float(0x7f800000);
}

// Part x of head h of a row: block b0 + x's, in its second slot where the row begins.
struct Parts {
  const float* first;
  int64_t slot;
  __device__ __forceinline__ Parts(const DecodeParams& p, int b0, int h) {
    slot = static_cast<int64_t>(p.H) * kPartRow;
    first = p.part + (static_cast<int64_t>(b0) * kPartSlots + 1) * slot + h * kPartRow;
  }
  __device__ __forceinline__ const float* operator()(int x) const {
    return x == 0 ? first : first - slot + x * kPartSlots * slot;
  }
};

// Row u's parts, of blocks b0 to b1, joined: one round of loads, eight parts of a
// head in flight a warp, and the warps' sums meet in shared memory.
template <int kT>
__device__ __forceinline__ void join_row(const DecodeParams& p, int u, int b0, int b1, float (&s_sum)[kT / 32][kD],
                                         float (&s_ml)[kT / 32][2]) {
  const float ninf = -__int_as_float(0x7f800000);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, H = p.H;
  const int shift = H <= 1 ? 0 : (H <= 2 ? 1 : (H <= 4 ? 2 : 3)), heads = 1 << shift, ways = (kT / 32) >> shift;
  const int h = warp & (heads - 1), way = warp >> shift;
  if (h < H) {
    float M, L;
    float4 acc;
    join_parts(Parts(p, b0, h), way, ways, b1 - b0 + 1, lane, M, L, acc);
    if (lane == 0) {
      s_ml[warp][0] = M;
      s_ml[warp][1] = L;
    }
    *reinterpret_cast<float4*>(&s_sum[warp][4 * lane]) = acc;
  }
  __syncthreads();
  for (int e = tid; e < H * kD; e += kT) {
    const int eh = e / kD;
    float M = ninf, L = 0.f, o = 0.f;
    for (int w = 0; w < ways; ++w) M = fmaxf(M, s_ml[w * heads + eh][0]);
    const float f = M == ninf ? 0.f : M;
    for (int w = 0; w < ways; ++w) {
      const float c = exp2f(s_ml[w * heads + eh][0] - f);
      L = fmaf(c, s_ml[w * heads + eh][1], L);
      o = fmaf(c, s_sum[w * heads + eh][e % kD], o);
    }
    p.out[static_cast<size_t>(u) * H * kD + e] = o * (L > 0.f ? 1.f / L : (L == 0.f ? 0.f : L));
    if (e % kD == 0) {
      const float z = L == 0.f ? ninf : M + log2f(L);
      if (p.lse) p.lse[static_cast<size_t>(u) * H + eh] = z * 0.6931471805599453f;
      if (p.lse2) p.lse2[static_cast<size_t>(u) * H + eh] = z;
    }
  }
}

// A block for every row, for no more rows than SMs (each then has many parts).
// The whole call, and with the kernel below: 8 rows of 4096 tokens 10.5 us, 12.3;
// 128 rows of 4096 tokens 49.6 us, 50.5; 160 rows 61.0 us either way.
__global__ void __launch_bounds__(kJoinThreads) paged_decode_join_few_kernel(const DecodeParams p) {
  __shared__ int64_t scan_part[2][kJoinWarps];
  __shared__ float s_sum[kJoinWarps][kD];
  __shared__ float s_ml[kJoinWarps][2];
  const int u = blockIdx.x, r = u / p.kv.G, g = u % p.kv.G;
  const VisibleTiles<kUnit> vt(p.kv.length(r, nullptr), p.window, p.sinks);
  int b0, b1;
  blocks_of_row<kJoinThreads>(p, r, g, vt, scan_part, b0, b1);
  pdl_wait();
  if (vt.count == 0)
    write_nothing(p, u);
  else if (b0 != b1)
    join_row<kJoinThreads>(p, u, b0, b1, s_sum, s_ml);
}

// A block for every end of a block's run, for more rows than SMs: fewer runs end
// than there are rows, and most rows lie in one run and need no joining. Block b
// joins the row that run b ends in the middle of, if the row begins in run b, and
// sees to every gridDim.x-th of the requests that nothing is seen of. 4096 rows of
// 256 tokens: the whole call 103 us (96 since), with a block for every row 129; 1024 rows of
// 1024 tokens 92 us, 99.
__global__ void __launch_bounds__(kCutThreads) paged_decode_join_cut_kernel(const DecodeParams p) {
  __shared__ int64_t scan_part[kCutThreads / 32];
  __shared__ float s_sum[kCutThreads / 32][kD];
  __shared__ float s_ml[kCutThreads / 32][2];
  __shared__ int s_u, s_b1;
  const PagedView& kv = p.kv;
  const int tid = threadIdx.x, b = blockIdx.x;
  const int own = (kv.R + kCutThreads - 1) / kCutThreads, r0 = min(kv.R, own * tid), r1 = min(kv.R, r0 + own);
  int64_t mine = 0, U;
  for (int r = r0; r < r1; ++r) mine += VisibleTiles<kUnit>(kv.length(r, nullptr), p.window, p.sinks).count;
  if (tid == 0) s_u = -1;
  int64_t base = block_scan<kCutThreads>(mine, scan_part, U) * kv.G;
  U *= kv.G;
  const int nb = sharing(U, p.blocks);
  if (b + 1 < nb) {
    const int64_t x = first_unit(U, b + 1, nb);  // the first unit of the next run
    if (x > base && x < base + mine * kv.G) {
      int64_t count = 0;
      for (int r = r0; r < r1; ++r, base += count * kv.G) {
        count = VisibleTiles<kUnit>(kv.length(r, nullptr), p.window, p.sinks).count;
        if (x >= base + count * kv.G) continue;
        const int64_t g = (x - base) / count, begin = base + g * count;
        if (begin < x && block_of_unit(U, begin, nb) == b) {
          s_u = r * kv.G + static_cast<int>(g);
          s_b1 = block_of_unit(U, begin + count - 1, nb);
        }
        break;
      }
    }
  }
  __syncthreads();
  pdl_wait();
  for (int r = b; r < kv.R; r += gridDim.x)
    if (VisibleTiles<kUnit>(kv.length(r, nullptr), p.window, p.sinks).count == 0)
      for (int g = 0; g < kv.G; ++g) write_nothing(p, r * kv.G + g);
  if (s_u >= 0) join_row<kCutThreads>(p, s_u, b, s_b1, s_sum, s_ml);
}

// The weights of tokens [chunk * kTokens, ...) of the row's visible units.
template <int kT, int kTokens>
__device__ __forceinline__ void weigh_tokens(const DecodeParams& p, int u, const VisibleTiles<kUnit>& vt,
                                             const float* lse2, int chunk) {
  const float ninf = -__int_as_float(0x7f800000);
  const size_t row = static_cast<size_t>(u) * p.kv.cap();
  float z[8];
#pragma unroll
  for (int h = 0; h < 8; ++h) z[h] = h < p.H ? lse2[h] : ninf;
#pragma unroll
  for (int e = threadIdx.x; e < kTokens; e += kT) {
    const int k = chunk * (kTokens / kUnit) + e / kUnit;
    if (k >= vt.count) break;
    const int t = vt.tile(k) * kUnit + e % kUnit;
    if (t >= vt.end || (t < vt.lo && t >= p.sinks)) continue;
    const float* l = p.logits + (row + t) * p.hp;
    const float m = p.mass[row + t];
    float w = 0.f;
    auto add = [&](float x, int h) { w += z[h] == ninf ? 0.f : exp2f(x - z[h]); };
    if (p.hp == 2) {
      const float2 v = *reinterpret_cast<const float2*>(l);
      add(v.x, 0), add(v.y, 1);
    } else {
      const float4 v = *reinterpret_cast<const float4*>(l);
      add(v.x, 0), add(v.y, 1), add(v.z, 2), add(v.w, 3);
      if (p.hp == 8) {
        const float4 y = *reinterpret_cast<const float4*>(l + 4);
        add(y.x, 4), add(y.y, 5), add(y.z, 6), add(y.w, 7);
      }
    }
    p.mass_out[row + t] = m + w;
  }
}

// Row u's parts joined (block x = 0 of the row), and its weights (every block).
__global__ void __launch_bounds__(kJoinThreads) paged_decode_weights_kernel(const DecodeParams p, int chunks) {
  __shared__ int64_t scan_part[2][kJoinWarps];
  __shared__ float s_lse2[8];
  __shared__ float s_sum[kJoinWarps][kD];
  const float ninf = -__int_as_float(0x7f800000);
  const PagedView& kv = p.kv;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int u = blockIdx.x / chunks, chunk = blockIdx.x % chunks;
  const int r = u / kv.G, g = u % kv.G, H = p.H;
  const VisibleTiles<kUnit> vt(kv.length(r, nullptr), p.window, p.sinks);
  if (chunk > 0 && static_cast<int64_t>(chunk) * (kJoinTokens / kUnit) >= vt.count) return;
  int b0, b1;
  blocks_of_row<kJoinThreads>(p, r, g, vt, scan_part, b0, b1);
  pdl_wait();
  if (vt.count == 0) {
    write_nothing(p, u);
    return;
  }
  if (b0 == b1) {
    if (tid < H) s_lse2[tid] = p.lse2[static_cast<size_t>(u) * H + tid];
  } else {
    // a head's parts are dealt to `ways` warps, each of which finds their maximum and
    // sum for itself and adds up its own outputs.
    const int parts = b1 - b0 + 1;
    const int shift = H <= 1 ? 0 : (H <= 2 ? 1 : (H <= 4 ? 2 : 3)), heads = 1 << shift, ways = kJoinWarps >> shift;
    const int h = warp & (heads - 1), way = warp >> shift;
    if (h < H) {
      const Parts part(p, b0, h);
      float M = ninf, L = 0.f;  // of the parts lane, lane + 32, ...
      for (int x = lane; x < parts; x += 32) {
        const float2 v = *reinterpret_cast<const float2*>(part(x));
        const float m = fmaxf(M, v.x), f = m == ninf ? 0.f : m;
        L = L * exp2f(M - f) + v.y * exp2f(v.x - f);
        M = m;
      }
      float f = M;
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) f = fmaxf(f, __shfl_xor_sync(0xFFFFFFFFu, f, d));
      const float top = f;
      if (f == ninf) f = 0.f;
      L *= exp2f(M - f);
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) L += __shfl_xor_sync(0xFFFFFFFFu, L, d);
      const float z = L == 0.f ? ninf : top + log2f(L);
      if (way == 0 && lane == 0) {
        s_lse2[h] = z;
        if (p.lse && chunk == 0) p.lse[static_cast<size_t>(u) * H + h] = z * 0.6931471805599453f;
      }
      if (chunk == 0) {
        const float inv = L > 0.f ? 1.f / L : (L == 0.f ? 0.f : L);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int x = way; x < parts; x += ways) {
          const float* pp = part(x);
          const float c = exp2f(pp[0] - f) * inv;
          const float4 v = *reinterpret_cast<const float4*>(pp + 4 + 4 * lane);
          acc.x = fmaf(c, v.x, acc.x);
          acc.y = fmaf(c, v.y, acc.y);
          acc.z = fmaf(c, v.z, acc.z);
          acc.w = fmaf(c, v.w, acc.w);
        }
        *reinterpret_cast<float4*>(&s_sum[warp][4 * lane]) = acc;
      }
    }
    __syncthreads();
    if (chunk == 0)
      for (int e = tid; e < H * kD; e += kJoinThreads) {
        float o = 0.f;
        for (int w = 0; w < min(ways, parts); ++w) o += s_sum[w * heads + e / kD][e % kD];
        p.out[static_cast<size_t>(u) * H * kD + e] = o;
      }
  }
  __syncthreads();
  weigh_tokens<kJoinThreads, kJoinTokens>(p, u, vt, s_lse2, chunk);
}

// The weights alone, where another kernel has joined the rows: `share` blocks a row.
// With weights, 4096 rows of 256 tokens: 143 us with the kernel above, 119 (111 since) with this
// one; 1024 rows of 1024 tokens 110 and 105; 256 rows of 1024 36 and 37.7, a launch more.
__global__ void __launch_bounds__(kWeighThreads) paged_decode_weigh_kernel(const DecodeParams p, int share) {
  __shared__ float s_lse2[8];
  const int u = blockIdx.x / share, tid = threadIdx.x;
  const VisibleTiles<kUnit> vt(p.kv.length(u / p.kv.G, nullptr), p.window, p.sinks);
  pdl_wait();
  if (vt.count == 0) return;
  if (tid < p.H) s_lse2[tid] = p.lse2[static_cast<size_t>(u) * p.H + tid];
  __syncthreads();
  for (int chunk = blockIdx.x % share; chunk <= (vt.count - 1) / (kWeighTokens / kUnit); chunk += share)
    weigh_tokens<kWeighThreads, kWeighTokens>(p, u, vt, s_lse2, chunk);
}

int decode_blocks() { return kBlocksPerSM * sm_count(); }

size_t carve(DecodeParams* p, void* ws, int R, int G, int H, int weight_cap) {
  WsCarver c(ws);
  const int hp = H <= 2 ? 2 : (H <= 4 ? 4 : 8);
  float* part = c.take<float>(static_cast<size_t>(decode_blocks()) * kPartSlots * H * kPartRow);
  float* lse2 = weight_cap ? c.take<float>(static_cast<size_t>(R) * G * H) : nullptr;
  float* logits = weight_cap ? c.take<float>(static_cast<size_t>(R) * G * weight_cap * hp) : nullptr;
  if (p) {
    p->part = part;
    p->lse2 = lse2;
    p->logits = logits;
    p->hp = hp;
  }
  return align_up(c.used, 16);
}

template <bool kF32Q, bool kWeights, bool kTest = false>
kvs_status launch(const DecodeParams& p, const CUtensorMap& mk, const CUtensorMap& mv, cudaStream_t s) {
  const int64_t cap = static_cast<int64_t>(p.kv.max_pages) << p.kv.shift;
  const int64_t chunks = kWeights ? (cap + kJoinTokens - 1) / kJoinTokens : 1, joins = chunks * p.kv.R * p.kv.G;
  KVS_REQUIRE(joins < (1ll << 31), KVS_EUNSUPPORTED, "paged_decode_attn: weights of R*G=%d rows of %lld tokens",
              p.kv.R * p.kv.G, static_cast<long long>(cap));
  allow_smem<paged_decode_kernel<kF32Q, kWeights, kTest>>(sizeof(DecodeSmem));
  launch_chained(paged_decode_kernel<kF32Q, kWeights, kTest>, dim3(p.blocks), dim3(kThreads), sizeof(DecodeSmem), s, p,
                 mk, mv);
  const int rows = p.kv.R * p.kv.G;
  if (rows <= (kWeights ? kWeighRowsPerSM : 1) * sm_count()) {
    const dim3 grid(static_cast<unsigned>(joins));
    if (kWeights)
      launch_chained(paged_decode_weights_kernel, grid, dim3(kJoinThreads), 0, s, p, static_cast<int>(chunks));
    else
      launch_chained(paged_decode_join_few_kernel, grid, dim3(kJoinThreads), 0, s, p);
  } else {
    launch_chained(paged_decode_join_cut_kernel, dim3(p.blocks), dim3(kCutThreads), 0, s, p);
    if (kWeights) {
      // blocks enough for every thread the GPU holds
      const int64_t most = (cap + kWeighTokens - 1) / kWeighTokens;
      const int64_t share = std::min<int64_t>(most, (kWeighBlocksPerSM * sm_count() + rows - 1) / rows);
      launch_chained(paged_decode_weigh_kernel, dim3(static_cast<unsigned>(rows * share)), dim3(kWeighThreads), 0, s, p,
                     static_cast<int>(share));
    }
  }
  return check_launch("paged_decode_attn");
}

}  // namespace

size_t paged_decode_ws_bytes(int R, int G, int H, int weight_cap) { return carve(nullptr, nullptr, R, G, H, weight_cap); }

kvs_status paged_decode_launch(const kvs_paged_decode_args* a, void* ws, int32_t* dev_status, cudaStream_t s,
                               int test_warp, int64_t wait_cycles) {
  DecodeParams p{};
  p.kv = paged_view(a->kv);
  p.q = a->q;
  p.H = a->H;
  p.window = a->window;
  p.sinks = a->sinks;
  p.scale_log2 = a->scale * 1.4426950408889634f;
  p.out = a->out;
  p.lse = a->lse;
  p.mass = a->mass;
  p.mass_out = a->mass_out;
  p.blocks = decode_blocks();
  p.dev_status = dev_status;
  carve(&p, ws, p.kv.R, p.kv.G, p.H, a->mass ? a->kv->max_pages * a->kv->page : 0);
  const int rows = a->kv->page < kUnit ? a->kv->page : kUnit;
  CUtensorMap mk, mv;
  KVS_PROPAGATE(paged_tensor_map(&mk, a->kv->K, p.kv, rows, 2, "paged_decode_attn"));
  KVS_PROPAGATE(paged_tensor_map(&mv, a->kv->V, p.kv, rows, 2, "paged_decode_attn"));
  p.test_warp = test_warp;
  p.wait_cycles = wait_cycles;
  if (test_warp >= 0) return launch<false, false, true>(p, mk, mv, s);
  const bool f32 = a->q_dtype == KVS_F32;
  if (f32) return a->mass ? launch<true, true>(p, mk, mv, s) : launch<true, false>(p, mk, mv, s);
  return a->mass ? launch<false, true>(p, mk, mv, s) : launch<false, false>(p, mk, mv, s);
}

}  // namespace kvs
