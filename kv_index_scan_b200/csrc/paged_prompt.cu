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
//  * An item is the (token, head) rows of as many tokens of one request and KV
//    head as fill two tiles of 128 rows (128 / H tokens a tile): the heads that
//    share a KV head share its K and V. It walks the 128-token tiles that any of
//    its rows sees, the sinks' first. Blocks are persistent, one an SM, each
//    with an equal share of the items; the next item's loads and first products
//    begin while the last one's rows are written. Where there are fewer items
//    than SMs (a few tokens over a long cache), an item's tiles are split in
//    pieces that are items themselves, and a second kernel joins the parts.
//  * One warp brings Q (a copy per row tile and 128-byte half), and K and V (a
//    copy per page and half, into two stages each) by TMA in the operand layout
//    of the tensor cores (128-byte swizzle). K is read K-major; V as it lies,
//    with the tokens as K, in the MN-major form.
//  * One thread issues tcgen05.mma: S = Q K^T (128 x 128, f32, in tensor
//    memory), then O += P V with P read from tensor memory. The two row tiles
//    alternate, so that one's softmax runs beside the other's products.
//  * Two groups of four warps do the softmax of one row tile each, a row per
//    thread: S from tensor memory, maximum, exponentials, P in bf16 over S's
//    columns. O is rescaled in tensor memory only when a row's maximum has
//    grown by more than 2^8 since the last time: weights up to 2^8 keep their
//    relative precision in bf16, and the sums are f32.
//  * Two warps clear what must not meet a weight of zero, whatever lies there:
//    rows of V that no row of the item sees or that were not loaded (released or
//    bad pages, behind the last token), and in tiles that some rows see more of
//    than others the single values that are not finite. Those are noted by token,
//    and added to the outputs of the rows that do see them at the item's end. The
//    search for them takes 1% of a long prompt's time and 3% of short items' (64
//    prompts of 300 tokens over 300: 199 us and 205 with it); without it a NaN
//    reached the queries in front of its token.
//  * The weights are rounded to bf16: the tensor cores take both operands in one
//    16-bit type, and a second product for what the rounding leaves would be half
//    as much tensor time again (full 24 bits is the decode form's choice, where
//    memory bounds). It costs an error of 2.1e-3 to 2.3e-3 against 64 bits, where
//    rounding the exact output to bf16 alone gives 1.6e-3 to 1.7e-3.
// Measured: 8192 tokens of 32 heads over 8 KV heads, causal, 0.55 TFLOP: 0.50 ms
// under the power cap (1.09 PFLOP/s; a large library product reaches 1.66 in a burst
// and 1.40 for seconds), 0.43 before it sets in; 2048 tokens over 32768 with a window
// of 4096: 158 us (0.87 PFLOP/s; 256 items for 148 SMs); 128 tokens 9.7 us; 4 tokens
// over 28676 40 us (359 before the split). The products
// with their loads alone take 0.32 and 0.09 ms: what is left is each row tile's
// chain from S through the softmax to the next S.
// Every wait is bounded; one that runs out writes KVS_ETIMEOUT, and the block
// winds down with no copy in flight and its tensor memory freed.
#include <cuda_bf16.h>

#include <algorithm>
#include <cstring>
#include <type_traits>

#include "async.cuh"

namespace kvs {

namespace {

constexpr int kRows = 128;                   // rows of a tile (MMA M)
constexpr int kTok = 128;                    // tokens of a tile (MMA N of S, K of O)
constexpr int kHalfBytes = 128 * 128;        // 128 rows of one 128-byte half
constexpr int kTileBytes = 2 * kHalfBytes;   // 128 rows of 128 bf16
constexpr int kStages = 2;                   // of K, and of V
constexpr int kInfos = 4;
constexpr int kItems = 4;                    // found ahead of the warps that work on them
constexpr int kSoftWarps = 8, kLoadWarp = 8, kMmaWarp = 9, kCleanWarp = 10, kCleanWarps = 2;
constexpr int kCutTiles = 6;                 // of an item: three at its rows' own tokens, three at their windows' first
constexpr int kNotes = 4;                    // of items (the clearing warps are at most two items ahead)
constexpr int kTakers = kSoftWarps + 1 + kCleanWarps;  // warps that take items from the loads' warp
constexpr int kThreads = 32 * 12;             // three warpgroups
// registers a thread: 168 at launch; 8 * 208 + 4 * 88 = 12 * 168
constexpr int kSoftRegs = 208, kOtherRegs = 88;
constexpr int kMaxPieces = 32;               // of an item (a lane of the join each)
constexpr int kPieceTiles = 4;               // that a piece has at least
constexpr int kTestTile = 1;
constexpr float kGrow = 8.f;                 // log2 of the growth that a maximum may lag behind

// Tokens that not all rows of an item see and that have values of V that are not
// finite, as one of the clearing warps found them in its rows of each tile (eight
// of every sixteen, a bit each).
struct Notes {
  int count, r, g;
  int tok[kCutTiles];  // the first of them
  uint32_t rows[kCutTiles][2];
};

struct PromptSmem {
  alignas(1024) unsigned char q[2][kTileBytes];
  unsigned char k[kStages][kTileBytes];
  unsigned char v[kStages][kTileBytes];
  unsigned char stage[kSoftWarps][32 * 128];  // outputs on their way
  int4 items[kItems][4];                     // the last word: whether it is an item
  uint64_t q_full, q_empty, k_full[kStages], k_empty[kStages], v_full[kStages], v_clean[kStages], v_empty[kStages];
  uint64_t item_full[kItems], item_empty[kItems];
  uint64_t s_full[2], p_full[2][2], o_full[2], drain;  // p_full by tile and half of the tokens
  Notes notes[kNotes][kCleanWarps];
  int groups[kInfos];                        // by tile: which 16-token groups were loaded
  uint32_t tmem;
  int abort_flag;
};

struct PromptParams {
  PagedView kv;
  const int32_t* cu;
  int T, H, per, window, sinks;  // per: tokens of a row tile, 128 / H
  float scale_log2;  // of the magnitude of the scale
  bool flip;         // a negative one: logits are turned round
  uint16_t* out;
  int64_t out_ld;
  float* lse;
  int pieces;        // of an item's tiles, each an item of its own (1: not split)
  float* part_o;     // [pieces][T][G*H][128], relative to the row's maximum in that piece
  float2* part_ml;   // [pieces][T][G*H]: that maximum (base 2), the sum
  int32_t* dev_status;
  long long wait_cycles;  // of the self-test
  int test_warp;

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
// 128 bytes of each head of a KV head's group and of each of a tile's tokens, to
// rows of 128 bytes (heads innermost, 128-byte swizzled).
__device__ __forceinline__ void tma_query_rows(uint32_t dst, const CUtensorMap* map, int head, int token, int half,
                                               uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
      "[%6];\n" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(head), "r"(token), "r"(half), "r"(sm_addr(bar))
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

// The rows of `per` tokens of a request and KV head for each of two row tiles,
// and the tiles of 128 tokens that any of them sees: the sinks', then those from
// the first row's window to the last row's own token.
template <bool kPieces>
struct Item {
  int r, g, q0;          // request, KV head, first packed row of the request
  int tok0, c;           // first token of the item among the request's c new ones
  int p_lo;              // its position
  int end, lo;           // tokens seen at most; first token of the first row's window
  int nsink, first;      // leading tiles with sinks; tile of the window's first token
  int piece, from, tiles;  // the item's tiles from, from + 1, ... of all

  __device__ __forceinline__ int token(int i) const {
    const int x = kPieces ? from + i : i;
    return (x < nsink ? x : first + x - nsink) * kTok;
  }
  // whether a row of the tile at t0 is seen by no row, or was not loaded
  __device__ __forceinline__ bool ragged(int t0, int there, int sinks) const {
    return there != 0xFF || t0 + kTok > end || (t0 < lo && t0 + kTok > sinks);
  }
};

// Item x of all, found by the whole warp: its pieces innermost, then the KV heads,
// the blocks of a request from its last (which sees most) to its first, the last request first.
// False behind the last one. The search goes on where the last one (for a smaller
// x) ended: below request top, with the items of the requests above it in base.
template <bool kPieces>
__device__ __forceinline__ bool find_item(const PromptParams& p, uint32_t x, int& top, uint32_t& base,
                                          Item<kPieces>& it) {
  const PagedView& kv = p.kv;
  const int lane = threadIdx.x & 31;
  uint32_t whole = x;
  if constexpr (kPieces) {
    whole = x / static_cast<uint32_t>(p.pieces);
    it.piece = static_cast<int>(x - whole * p.pieces);
  }
  const uint32_t order = whole / static_cast<uint32_t>(kv.G);
  it.g = static_cast<int>(whole - order * kv.G);
  for (; top > 0; top -= 32) {
    const int r = top - 1 - lane;
    int q0 = 0, c = 0, n = 0;
    if (r >= 0) {
      q0 = p.start(r);
      c = max(0, p.start(r + 1) - q0);
      n = kv.length(r, p.dev_status);
    }
    const uint32_t mine = (static_cast<uint32_t>(c) + 2 * p.per - 1) / (2 * p.per);
    uint32_t inc = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, inc, d);
      if (lane >= d) inc += y;
    }
    const unsigned hit = __ballot_sync(0xFFFFFFFFu, order < base + inc);
    if (hit) {
      const int l = __ffs(hit) - 1;
      const int block = static_cast<int>(__shfl_sync(0xFFFFFFFFu, base + inc, l) - 1 - order);
      it.r = top - 1 - l;
      it.q0 = __shfl_sync(0xFFFFFFFFu, q0, l);
      c = __shfl_sync(0xFFFFFFFFu, c, l);
      n = __shfl_sync(0xFFFFFFFFu, n, l);
      it.tok0 = block * 2 * p.per;
      it.c = c;
      it.p_lo = n - c + it.tok0;
      it.end = max(0, n - c + min(c, it.tok0 + 2 * p.per));
      it.lo = p.window && it.p_lo >= p.window ? it.p_lo - p.window + 1 : 0;
      it.nsink = it.first = 0;
      if (it.lo) {
        const int t = (min(p.sinks, it.lo) + kTok - 1) / kTok;
        if (t < it.lo / kTok) {
          it.nsink = t;
          it.first = it.lo / kTok;
        }
      }
      it.tiles = it.nsink + (it.end + kTok - 1) / kTok - it.first;
      if constexpr (kPieces) {
        // no more pieces than have kPieceTiles tiles each; the others are empty
        const int pieces = max(1, min(p.pieces, it.tiles / kPieceTiles)), at = min(it.piece, pieces);
        const int64_t tiles = it.tiles;
        it.from = static_cast<int>(tiles * at / pieces);
        it.tiles = static_cast<int>(tiles * min(at + 1, pieces) / pieces) - it.from;
      }
      return true;
    }
    base += __shfl_sync(0xFFFFFFFFu, inc, 31);
  }
  return false;
}

// Values of V that are not finite, of tokens that the row at position pos sees and
// others of its item do not (by a whole warp, a row a thread; pos -1: no row): read
// again from their pages and added to its outputs in tensor memory. (Out of line, as
// the next: they hardly ever run, and written in place the whole kernel took 1% longer.)
__device__ __noinline__ void add_noted(const PromptParams& p, const Notes* notes, uint32_t o_at, int pos) {
#pragma unroll 1
  for (int e = 0; e < 4; ++e) {
    float o[32];
    tmem_ld32(o_at + 32 * e, o);
    wait_ld();
#pragma unroll 1
    for (int w = 0; w < 2 * kCutTiles * kCleanWarps; ++w) {
      const Notes& n = notes[w & 1];
      const int c = w >> 2;
      uint32_t rows = c < n.count ? n.rows[c][w >> 1 & 1] : 0;
#pragma unroll 1
      while (rows) {
        const int b = 32 * (w >> 1 & 1) + __ffs(rows) - 1, j = n.tok[c] + 16 * (b >> 3) + (b & 7);
        rows &= rows - 1;
        if (j > pos || (p.window && j >= p.sinks && j <= pos - p.window)) continue;
        const int id = p.kv.page_of(n.r, j, nullptr);
        if (id < 0) continue;
        const uint4* v = reinterpret_cast<const uint4*>(p.kv.V + p.kv.row(id, n.g, j) + 32 * e);
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const uint4 q = v[y];
          const uint32_t x[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
          for (int z = 0; z < 4; ++z) {
            if ((x[z] & 0x7F80u) == 0x7F80u) o[8 * y + 2 * z] += __uint_as_float(x[z] << 16);
            if ((x[z] & 0x7F800000u) == 0x7F800000u) o[8 * y + 2 * z + 1] += __uint_as_float(x[z] & 0xFFFF0000u);
          }
        }
      }
    }
    __syncwarp();
    tmem_st32(o_at + 32 * e, o);
  }
  wait_st();
}

// Eight rows of V (16 bytes a lane, four rows of a half at v and its fellows) with
// their values that are not finite cleared, by a whole warp; the rows that had any.
__device__ __noinline__ uint32_t clear_values(uint4* v) {
  uint32_t rows = 0;
#pragma unroll 1
  for (int y = 0; y < 4; ++y) {
    uint4& w = v[(y >> 1) * (kHalfBytes / 16) + (y & 1) * 32];
    uint32_t e[4] = {w.x, w.y, w.z, w.w};
    bool bad = false;
#pragma unroll
    for (int z = 0; z < 4; ++z) {
      if ((e[z] & 0x7F80u) == 0x7F80u) e[z] &= 0xFFFF0000u, bad = true;
      if ((e[z] & 0x7F800000u) == 0x7F800000u) e[z] &= 0xFFFFu, bad = true;
    }
    if (bad) w = make_uint4(e[0], e[1], e[2], e[3]);
    const unsigned lanes = __ballot_sync(0xFFFFFFFFu, bad);
#pragma unroll
    for (int z = 0; z < 4; ++z)
      if (lanes >> (8 * z) & 0xFFu) rows |= 1u << (4 * (y & 1) + z);
  }
  return rows;
}

// kTest: every wait is bounded by wait_cycles, and in every block that has as many
// tiles warp test_warp gives up at tile kTestTile.
template <bool kPieces, bool kTest = false>
__global__ void __launch_bounds__(kThreads, 1) paged_prompt_kernel(const __grid_constant__ PromptParams p,
                                                                   const __grid_constant__ CUtensorMap mapQ,
                                                                   const __grid_constant__ CUtensorMap mapK,
                                                                   const __grid_constant__ CUtensorMap mapV) {
  extern __shared__ __align__(1024) unsigned char prompt_smem[];
  PromptSmem& sm = *reinterpret_cast<PromptSmem*>(prompt_smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const PagedView& kv = p.kv;
  const int G = kv.G, H = p.H;

  if (tid == 0) {
    mbar_init(&sm.q_full, 1);
    mbar_init(&sm.q_empty, 1);
    mbar_init(&sm.drain, 1);
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&sm.k_full[i], 1);
      mbar_init(&sm.k_empty[i], 1);
      mbar_init(&sm.v_full[i], 1);
      mbar_init(&sm.v_clean[i], kCleanWarps);
      mbar_init(&sm.v_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.s_full[i], 1);
      mbar_init(&sm.p_full[i][0], kRows / 32);
      mbar_init(&sm.p_full[i][1], kRows / 32);
      mbar_init(&sm.o_full[i], 1);
    }
    for (int i = 0; i < kItems; ++i) {
      mbar_init(&sm.item_full[i], 1);
      mbar_init(&sm.item_empty[i], kTakers);
    }
    sm.abort_flag = 0;
    mbar_init_fence();
    tma_prefetch_map(&mapQ);
    tma_prefetch_map(&mapK);
    tma_prefetch_map(&mapV);
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;\n" ::"r"(sm_addr(&sm.tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
  }
  pdl_wait();
  pdl_trigger();
  // The block's items: one of each round of gridDim.x, in the order of the
  // blocks and in the reverse in turn (items shrink along the order). The loads'
  // warp finds each while the tiles of the one before are under way, and hands it
  // on through shared memory: finding one takes 1,500 cycles and more (3,000 with
  // 148 requests), which every warp spent between two items when it found them for
  // itself, from the first request on each time. 592 items of one tile took 46.6 us
  // so and take 39; 592 of a window's six tiles 89 and 83; 512 requests of 17 tokens
  // over 100 258 and 150.
  uint32_t round = 0, base = 0;
  int top = kv.R;
  auto find = [&](Item<kPieces>& it) {
    const uint32_t at = round & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x;
    return find_item(p, round * gridDim.x + at, top, base, it);
  };
  Item<kPieces> it;
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = sm.tmem;  // S of tile t at 128 t, O at 256 + 128 t

  auto fail = [&] {
    set_status(p.dev_status, KVS_ETIMEOUT);
    atomicExch(&sm.abort_flag, 1);
  };
  auto aborted = [&] { return *reinterpret_cast<volatile int*>(&sm.abort_flag) != 0; };
  // By the whole warp, every lane for itself (what the barrier guards is ordered for
  // the lanes that have seen its phase), and first without looking whether the block
  // has given up: the products' warp waits seven times a tile, and mostly for what is
  // there.
  const long long limit = kTest ? p.wait_cycles : kWaitCycles;
  auto wait = [&](uint64_t* b, uint32_t parity) {
    if (!aborted() && mbar_wait(b, parity, limit)) return true;
    fail();
    return false;
  };
  auto wait_all = [&](uint64_t* b, uint32_t parity) {
    if (__all_sync(0xFFFFFFFFu, mbar_try(b, parity))) return true;
    return __all_sync(0xFFFFFFFFu, wait(b, parity)) != 0;
  };
  static_assert(sizeof(Item<kPieces>) < sizeof(sm.items[0]), "the last word is kept");
  auto read_item = [&](uint32_t of, Item<kPieces>& it) {
    int4 w[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) w[x] = sm.items[of % kItems][x];
    memcpy(&it, w, sizeof(it));
    return w[3].w != 0;
  };
  // by a whole warp other than the loads': the next item, false behind the last
  auto take = [&](Item<kPieces>& it, bool& ok) {
    const int slot = round % kItems;
    ok = wait_all(&sm.item_full[slot], round / kItems & 1);
    if (!ok) return false;
    const bool is = read_item(slot, it);
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.item_empty[slot]);
    ++round;
    return is;
  };
  // In every role: `at` counts the tiles, and `live` the items that have any, of
  // the whole launch; a phase of a barrier belongs to one of them.
  int at = 0, live = 0;
  bool ok = true;

  if (warp >= kSoftWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kOtherRegs));
    if (warp == kLoadWarp) {
      // ---------------- K and V tiles ----------------
      const int box = min(1 << kv.shift, kTok), pages = kTok / box;
      const int half = lane & 1, sub = lane >> 1;
      int issued = 0;  // K and V tiles
      // the next item found and handed on
      auto hand_on = [&] {
        const int slot = round % kItems;
        Item<kPieces> then;
        const bool is = find(then);
        if (round >= kItems && !wait_all(&sm.item_empty[slot], (round / kItems - 1) & 1)) return false;
        if (lane == 0) {
          int4 w[4] = {};
          memcpy(w, &then, sizeof(then));
          w[3].w = is;
#pragma unroll
          for (int x = 0; x < 4; ++x) sm.items[slot][x] = w[x];
          mbar_arrive(&sm.item_full[slot]);
        }
        ++round;
        __syncwarp();
        return true;
      };
      ok = hand_on();
      bool more = ok && read_item(0, it);
      while (more && ok) {
        // this lane's page id of tile i, unchecked (nothing waits for it here); -1 where none is needed
        auto wanted = [&](int i) {
          const int t = it.token(i) + sub * box;
          return sub < pages && t < it.end && (t < p.sinks || t + box > it.lo);
        };
        const int32_t* table = kv.table + it.r * kv.table_ld;
        auto look = [&](int i) { return wanted(i) ? __ldg(table + ((it.token(i) + sub * box) >> kv.shift)) : -1; };
        int next = it.tiles > 0 ? look(0) : -1;
        for (int i = 0; i < it.tiles && ok; ++i, ++at) {
          const int st = at % kStages;
          int id = next;
          if (i + 1 < it.tiles) next = look(i + 1);
          if (static_cast<unsigned>(id) >= static_cast<unsigned>(kv.num_pages)) {
            if (wanted(i)) set_status(p.dev_status, KVS_EBOUNDS);
            id = -1;
          }
          const unsigned have = __ballot_sync(0xFFFFFFFFu, id >= 0);
          const int in_page = (it.token(i) + sub * box) & ((1 << kv.shift) - 1);
          const uint32_t to = half * kHalfBytes + sub * box * 128;
          for (int which = 0; which < 2 && ok; ++which) {
            uint64_t* full = which ? &sm.v_full[st] : &sm.k_full[st];
            if (at >= kStages) ok = wait_all(which ? &sm.v_empty[st] : &sm.k_empty[st], (at / kStages - 1) & 1);
            if (kTest && p.test_warp == warp && at == kTestTile) ok = false;
            if (!ok) break;
            if (lane == 0) {
              if (which == 0) {
                int there = 0;
                for (int e = 0; e < 8; ++e)
                  if (have >> (2 * (16 * e / box)) & 1u) there |= 1 << e;
                sm.groups[at % kInfos] = there;
                __threadfence_block();
              }
              if (have) mbar_expect(full, __popc(have) * box * 128);
              else mbar_arrive(full);
            }
            __syncwarp();
            if (id >= 0)
              tma_page_rows(sm_addr(which ? sm.v[st] : sm.k[st]) + to, which ? &mapV : &mapK, in_page, half, it.g, id,
                            full);
            ++issued;
            if (i == 0 && which == 0) {  // the queries after the first K tile, whose place is free before theirs
              if (live > 0) ok = wait_all(&sm.q_empty, (live - 1) & 1);
              if (!ok) break;
              if (lane == 0) {
                mbar_expect(&sm.q_full, 4 * p.per * H * 128);
                for (int x = 0; x < 4; ++x)
                  tma_query_rows(sm_addr(sm.q[x >> 1]) + (x & 1) * kHalfBytes, &mapQ, it.g * H,
                                 it.q0 + it.tok0 + (x >> 1) * p.per, x & 1, &sm.q_full);
              }
              ++live;
            }
          }
          // the next item, with two tiles on their way
          if (ok && i == min(1, it.tiles - 1)) ok = hand_on();
        }
        if (ok && it.tiles <= 0) ok = hand_on();
        more = ok && read_item(round - 1, it);
      }
      // no copy may be in flight when the block ends
      if (lane == 0 && live > 0) mbar_wait(&sm.q_full, (live - 1) & 1, limit);
      if (lane == 0)
        for (int x = max(0, issued - 2 * kStages); x < issued; ++x) {
          const int i = x / 2;
          mbar_wait(x & 1 ? &sm.v_full[i % kStages] : &sm.k_full[i % kStages], (i / kStages) & 1, limit);
        }
    } else if (warp >= kCleanWarp) {
      // ---------------- what of V must not meet a weight of zero ----------------
      const int r0 = 8 * (warp - kCleanWarp);  // this warp's rows: eight of every sixteen
      while (ok && take(it, ok)) {
        Notes& notes = sm.notes[live % kNotes][warp - kCleanWarp];
        if (it.tiles > 0) {
          ++live;
          if (lane == 0) notes.count = 0;
        }
        // tokens that some rows have passed, and the first that not every row has come to
        const int passed0 = max(it.lo, p.sinks), passed1 = p.window ? it.end - p.window : 0, come = it.p_lo + 1;
        const int cut0 = passed1 > passed0 ? min(passed0, come) : come;
        for (int i = 0; i < it.tiles && ok; ++i, ++at) {
          const int st = at % kStages;
          ok = wait_all(&sm.v_full[st], (at / kStages) & 1);
          if (kTest && p.test_warp == warp && at == kTestTile) ok = false;
          if (!ok) break;
          const int t0 = it.token(i), there = sm.groups[at % kInfos];
          const bool ragged = it.ragged(t0, there, p.sinks);
          if (ragged) {
            auto clear = [&](int from, int to) {  // rows of the tile, two a step
              for (int a = (from & ~15) + r0 + (lane >> 4); a < to; a += 16)
#pragma unroll
                for (int y = a; y < a + 8; y += 2)
                  if (y >= from && y < to)
                    *reinterpret_cast<uint4*>(sm.v[st] + (lane >> 3 & 1) * kHalfBytes + y * 128 + (lane & 7) * 16) =
                        make_uint4(0, 0, 0, 0);
            };
            for (int e = 0; e < 8; ++e)
              if (!(there >> e & 1)) clear(16 * e, 16 * e + 16);
            if (t0 + kTok > it.end) clear(max(it.end - t0, 0), kTok);
            if (t0 < it.lo) clear(min(max(p.sinks - t0, 0), kTok), min(it.lo - t0, kTok));
            __syncwarp();
          }
          uint32_t rows0 = 0, rows1 = 0;
          if (t0 + kTok > cut0 && (t0 < passed1 || t0 + kTok > come)) {
            const int x0 = come - t0, x1 = it.end - t0, y0 = passed0 - t0, y1 = passed1 - t0;
#pragma unroll 1
            for (int x = 0; x < 8; ++x) {
              const int a = 16 * x + r0, b = a + 8;
              if (max(x0, a) >= min(x1, b) && max(y0, a) >= min(y1, b)) continue;
              // 16 bytes a lane, four rows of a half at a time
              uint4* v = reinterpret_cast<uint4*>(sm.v[st] + a * 128) + lane;
              uint4 w[4];
#pragma unroll
              for (int y = 0; y < 4; ++y) w[y] = v[(y >> 1) * (kHalfBytes / 16) + (y & 1) * 32];
              __nv_bfloat162 most = __floats2bfloat162_rn(0.f, 0.f);
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                const uint32_t e[4] = {w[y].x, w[y].y, w[y].z, w[y].w};
#pragma unroll
                for (int z = 0; z < 4; ++z)
                  most = __hmax2_nan(most, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&e[z])));
              }
              const uint32_t m = *reinterpret_cast<const uint32_t*>(&most);
              if (!__any_sync(0xFFFFFFFFu, (m & 0x7F80u) == 0x7F80u || (m & 0x7F800000u) == 0x7F800000u)) continue;
              const uint32_t eight = clear_values(v) << (8 * (x & 3));
              if (x < 4) rows0 |= eight;
              else rows1 |= eight;
            }
          }
          const bool found = (rows0 | rows1) != 0;
          if (found && lane == 0) {
            const int c = notes.count++;
            notes.r = it.r;
            notes.g = it.g;
            notes.tok[c] = t0 + r0;
            notes.rows[c][0] = rows0;
            notes.rows[c][1] = rows1;
          }
          if (ragged || found) {
            asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
            __syncwarp();
          }
          // (every tile goes this way: the products wait for v_clean alone, which
          // is long there when they come to it)
          if (lane == 0) mbar_arrive(&sm.v_clean[st]);
        }
      }
    } else if (warp == kMmaWarp) {
      // ---------------- products ----------------
      // (the whole warp goes through the loop, so that descriptors stay in
      // uniform registers; one lane issues)
      const uint64_t dq = desc_k_major(sm_addr(sm.q[0])), dk = desc_k_major(sm_addr(sm.k[0])),
                     dv = desc_mn_major(sm_addr(sm.v[0]));
      const bool leader = elect_one();
      auto qk = [&](int t, int x) {
        const uint64_t a = dq + t * (kTileBytes >> 4), b = dk + (x % kStages) * (kTileBytes >> 4);
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
      while (ok && take(it, ok)) {
        if (it.tiles == 0) continue;
        ok = wait_all(&sm.q_full, live & 1) && wait_all(&sm.k_full[at % kStages], (at / kStages) & 1);
        if (!ok) break;
        ++live;
        fence_after();
        qk(0, at);
        qk(1, at);
        commit(&sm.k_empty[at % kStages]);
        if (it.tiles == 1) commit(&sm.q_empty);
        for (int i = 0; i < it.tiles && ok; ++i, ++at) {
          const int st = at % kStages, after = at + 1;
          ok = wait_all(&sm.v_clean[st], (at / kStages) & 1);
          if (kTest && p.test_warp == warp && at == kTestTile) ok = false;
          for (int t = 0; t < 2 && ok; ++t) {
            const uint32_t d = tmem + 256 + 128 * t, a = tmem + 128 * t;
            const uint64_t b = dv + st * (kTileBytes >> 4);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              ok = ok && wait_all(&sm.p_full[t][e], at & 1);
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
            if (i + 1 == it.tiles) {
              commit(&sm.o_full[t]);
              continue;
            }
            if (t == 0) {
              ok = wait_all(&sm.k_full[after % kStages], (after / kStages) & 1);
              if (!ok) break;
              fence_after();
            }
            qk(t, after);
            if (t == 1) {
              commit(&sm.k_empty[after % kStages]);
              if (i + 2 == it.tiles) commit(&sm.q_empty);  // the item's last products with its queries
            }
          }
        }
      }
      if (!ok) {  // products already issued end before the block does
        commit(&sm.drain);
        mbar_wait(&sm.drain, 0, limit);
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kSoftRegs));
    // ---------------- softmax, a row per thread ----------------
    const int t = warp >> 2;                       // row tile
    const int w0 = 32 * (warp & 3);                // the warp's first row in it
    const uint32_t lanes = static_cast<uint32_t>(w0) << 16;
    const uint32_t s_at = tmem + lanes + 128 * t, o_at = tmem + lanes + 256 + 128 * t;
    const float ninf = -__int_as_float(0x7f800000);
    // row x of a tile is head x % H of its token x / H (x < 128: the division is
    // a multiplication); rows behind the tile's last token go with it
    const uint32_t by_h = 65536u / H + 1;
    auto token_of = [&](int x) { return min(static_cast<int>(x * by_h >> 16), p.per - 1); };
    bool more = take(it, ok);
    while (more && ok) {
      const int pos = it.p_lo + t * p.per + token_of(tid & 127);
      // the first and last position of this warp's rows
      const int p_first = it.p_lo + t * p.per + token_of(w0), p_last = it.p_lo + t * p.per + token_of(w0 + 31);
      float m = ninf, l = 0.f;
      for (int i = 0; i < it.tiles; ++i, ++at) {
        ok = wait_all(&sm.s_full[t], at & 1);
        if (kTest && p.test_warp == warp && at == kTestTile) ok = false;
        if (!ok) break;
        fence_after();
        const int t0 = it.token(i), there = sm.groups[at % kInfos];
        const bool whole = there == 0xFF && t0 + kTok - 1 <= p_first &&
                           (!p.window || t0 > p_last - p.window || t0 + kTok <= p.sinks);
        if (!whole || p.flip) {
          // masked in tensor memory, so that the code below is the same for
          // every tile (beside masking in its registers it ran 15% slower)
#pragma unroll 1
          for (int e = 0; e < 4; ++e) {
            // bit j: this row sees token b + j
            const int b = t0 + 32 * e;
            uint32_t see = low_bits(pos + 1 - b);
            if (p.window) see &= ~low_bits(pos - p.window + 1 - b) | low_bits(p.sinks - b);
            see &= (there >> (2 * e) & 1 ? 0xFFFFu : 0u) | (there >> (2 * e + 1) & 1 ? 0xFFFF0000u : 0u);
            float x[32];
            tmem_ld32(s_at + 32 * e, x);
            wait_ld();
#pragma unroll
            for (int j = 0; j < 32; ++j) x[j] = see >> j & 1u ? (p.flip ? -x[j] : x[j]) : ninf;
            tmem_st32(s_at + 32 * e, x);
          }
          wait_st();
        }
        float s[kTok];
#pragma unroll
        for (int e = 0; e < 4; ++e) tmem_ld32(s_at + 32 * e, s + 32 * e);
        wait_ld();
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
      // (what does not need the outputs comes before the wait for the last products)
      const int tok = it.tok0 + t * p.per, x = tid & 127;
      const bool there = x < p.per * H && tok + token_of(x) < it.c;  // whether this thread's row is there
      const int64_t token_row = static_cast<int64_t>(it.q0 + tok + token_of(x));
      const int head = it.g * H + x - token_of(x) * H;
      const bool some = ok && it.tiles > 0;  // (the next item is taken before that wait too)
      if constexpr (kPieces) {
        // a part: the row as it is, for the join
        const int64_t row = (it.piece * static_cast<int64_t>(p.T) + token_row) * G * H + head;
        more = ok && take(it, ok);
        const bool done = some && wait_all(&sm.o_full[t], live & 1);
        ok = ok && done == some;
        live += some;
        fence_after();
        if (done) {
          const Notes* notes = sm.notes[(live - 1) % kNotes];
          if (notes[0].count | notes[1].count) add_noted(p, notes, o_at, there ? pos : -1);
        }
        if (there) p.part_ml[row] = done ? make_float2(m, l) : make_float2(ninf, 0.f);
#pragma unroll 1
        for (int e = 0; e < 4 && done; ++e) {
          float o[32];
          tmem_ld32(o_at + 32 * e, o);
          wait_ld();
          if (there) {
#pragma unroll
            for (int j = 0; j < 32; j += 4)
              *reinterpret_cast<float4*>(p.part_o + row * kD + 32 * e + j) = make_float4(o[j], o[j + 1], o[j + 2], o[j + 3]);
          }
          __syncwarp();
        }
      } else {
        if (p.lse && there)
          p.lse[token_row * G * H + head] = l == 0.f ? ninf : (m + log2f(l)) * 0.6931471805599453f;
        // 64 channels at a time (rounded to bf16 here) through 128 bytes a row of
        // shared memory, 16-byte pieces exchanged so that neither side conflicts:
        // eight lanes write a row. (Not unrolled: code that runs once an item.)
        unsigned char* stage = sm.stage[warp];
        const int64_t own = there ? token_row * p.out_ld + head * kD : -1;
        int64_t to[8];
#pragma unroll
        for (int y = 0; y < 8; ++y) to[y] = __shfl_sync(0xFFFFFFFFu, own, 4 * y + (lane >> 3));
        uint16_t* out = p.out + 8 * (lane & 7);
        more = ok && take(it, ok);
        const bool done = some && wait_all(&sm.o_full[t], live & 1);
        ok = ok && done == some;
        live += some;
        fence_after();
        if (done) {
          const Notes* notes = sm.notes[(live - 1) % kNotes];
          if (notes[0].count | notes[1].count) add_noted(p, notes, o_at, there ? pos : -1);
        }
        const float inv = !done ? 0.f : (l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l));
#pragma unroll 1
        for (int e = 0; e < 2; ++e) {
          float o[64];
          tmem_ld32(o_at + 64 * e, o);
          tmem_ld32(o_at + 64 * e + 32, o + 32);
          wait_ld();
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            uint4 v = make_uint4(bf16_pair(o[8 * j] * inv, o[8 * j + 1] * inv), bf16_pair(o[8 * j + 2] * inv, o[8 * j + 3] * inv),
                                 bf16_pair(o[8 * j + 4] * inv, o[8 * j + 5] * inv),
                                 bf16_pair(o[8 * j + 6] * inv, o[8 * j + 7] * inv));
            if (!done) v = make_uint4(0, 0, 0, 0);  // tensor memory that nothing was written to
            *reinterpret_cast<uint4*>(stage + lane * 128 + ((j ^ (lane & 7)) << 4)) = v;
          }
          __syncwarp();
#pragma unroll
          for (int y = 0; y < 8; ++y) {
            const int rr = 4 * y + (lane >> 3);
            const uint4 v = *reinterpret_cast<const uint4*>(stage + rr * 128 + (((lane & 7) ^ (rr & 7)) << 4));
            if (to[y] >= 0) *reinterpret_cast<uint4*>(out + to[y] + 64 * e) = v;
          }
          __syncwarp();
        }
      }
      fence_before();  // O is read before the next item's first product is let go
    }
  }
  fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;\n" ::"r"(tmem) : "memory");
  }
}

// The pieces of every (token, query head) row joined, a row a warp.
__global__ void __launch_bounds__(256) paged_prompt_join_kernel(const PromptParams p) {
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t heads = static_cast<int64_t>(p.kv.G) * p.H, rows = heads * p.T;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (row < p.start(0) * heads || row >= p.start(p.kv.R) * heads) return;
  const float ninf = -__int_as_float(0x7f800000);
  const float2 ml = lane < p.pieces ? p.part_ml[lane * rows + row] : make_float2(ninf, 0.f);
  float M = ml.x;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, d));
  // (a piece without a token of the row's has written nothing but this)
  const bool none = ml.x == ninf && ml.y == 0.f;
  const float c = none ? 0.f : exp2f(ml.x - (M == ninf ? 0.f : M));
  float L = none ? 0.f : (ml.x == ninf ? ml.y : c * ml.y);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) L += __shfl_xor_sync(0xFFFFFFFFu, L, d);
  const float inv = L > 0.f ? 1.f / L : (L == 0.f ? 0.f : L);
  const unsigned there = __ballot_sync(0xFFFFFFFFu, !none);
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int x = 0; x < p.pieces; ++x) {
    const float w = __shfl_sync(0xFFFFFFFFu, c, x) * inv;
    if (!(there >> x & 1)) continue;
    const float4 v = *reinterpret_cast<const float4*>(p.part_o + (x * rows + row) * kD + 4 * lane);
    o.x = fmaf(w, v.x, o.x);
    o.y = fmaf(w, v.y, o.y);
    o.z = fmaf(w, v.z, o.z);
    o.w = fmaf(w, v.w, o.w);
  }
  const int64_t token = row / heads;
  *reinterpret_cast<uint2*>(p.out + token * p.out_ld + (row - token * heads) * kD + 4 * lane) =
      make_uint2(bf16_pair(o.x, o.y), bf16_pair(o.z, o.w));
  if (p.lse && lane == 0) p.lse[row] = L == 0.f ? ninf : (M + log2f(L)) * 0.6931471805599453f;
}

// No more items than this, whatever the lengths: each request's last one may be
// part empty.
int64_t most_items(int R, int G, int H, int T) {
  const int64_t per2 = 2 * (kRows / H);
  return (T + (T < R ? T : R) * (per2 - 1)) / per2 * G;
}

// Tiles of the longest item that there may be.
int64_t longest_item(int H, int64_t cap, int window, int sinks) {
  int64_t t = (cap + kTok - 1) / kTok;
  if (window) {
    const int64_t seen = (static_cast<int64_t>(window) + 2 * (kRows / H) + kTok - 1) / kTok + 1 +
                         (static_cast<int64_t>(sinks) + kTok - 1) / kTok;
    if (seen < t) t = seen;
  }
  return t;
}

// Pieces that an item's tiles are split in. In units of a tile's time (1.75 us),
// with t tiles in the longest item that there may be, a round of whole items
// takes t + 3.5, one of n pieces t / n + 5, and the join 4 (8 heads, 4 tokens over
// 28676: 359 us whole, 37 in 18 pieces; 2 heads, 1024 tokens: 20.6 whole, 23.1 in
// two): the number with the least sum of rounds. The longest item that there may be
// is the table's width: a table much wider than what it holds splits items that need
// it not (128 tokens 9.2 us and 18 from 4096 slots on, 1024 tokens 22 and 71 at 131072).
int pieces_of(int R, int G, int H, int T, int64_t cap, int window, int sinks) {
  const int64_t items = most_items(R, G, H, T), sms = sm_count(), t = longest_item(H, cap, window, sinks);
  int best = 1;
  double least = static_cast<double>((items + sms - 1) / sms) * (t + 3.5);
  for (int n = 2; n <= kMaxPieces && n * kPieceTiles <= t; ++n) {
    const double cost = static_cast<double>((items * n + sms - 1) / sms) * (static_cast<double>(t) / n + 5) + 4;
    if (cost < least) {
      least = cost;
      best = n;
    }
  }
  return best;
}

size_t carve(PromptParams* p, void* ws, int G, int H, int T, int pieces) {
  if (pieces == 1) return 0;
  WsCarver c(ws);
  const size_t rows = static_cast<size_t>(pieces) * T * G * H;
  float* o = c.take<float>(rows * kD);
  float2* ml = c.take<float2>(rows);
  if (p) {
    p->part_o = o;
    p->part_ml = ml;
  }
  return align_up(c.used, 16);
}

}  // namespace

size_t paged_prompt_ws_bytes(int R, int G, int H, int T, int cap, int window, int sinks) {
  if (R < 1 || G < 1 || H < 1 || H > 8 || T < 1) return 0;
  return carve(nullptr, nullptr, G, H, T, pieces_of(R, G, H, T, cap, window, sinks));
}

// The workspace grows with T as long as the items, and so the pieces, stay the same:
// the last T of each number of items is asked. With items * 6.5 >= sms * t one piece
// is the least for good (n pieces cost at least items / sms * (t + 5 n) + 4).
size_t paged_prompt_ws_bound(int R, int G, int H, int T, int cap, int window, int sinks) {
  if (R < 1 || G < 1 || H < 1 || H > 8 || T < 1) return 0;
  const int64_t per2 = 2 * (kRows / H), t = longest_item(H, cap, window, sinks), sms = sm_count();
  size_t most = 0;
  for (int64_t x = 1; x <= T; ++x) {
    if (x >= R) {
      const int64_t empty = R * (per2 - 1), blocks = (x + empty) / per2;
      x = std::min<int64_t>(T, (blocks + 1) * per2 - empty - 1);
    }
    most = std::max(most, paged_prompt_ws_bytes(R, G, H, static_cast<int>(x), cap, window, sinks));
    if (6.5 * most_items(R, G, H, static_cast<int>(x)) >= static_cast<double>(sms) * t) break;
  }
  return most;
}

kvs_status paged_prompt_launch(const kvs_paged_prompt_args* a, void* ws, int32_t* dev_status, cudaStream_t s,
                               int test_warp, int64_t wait_cycles) {
  PromptParams p{};
  p.kv = paged_view(a->kv);
  p.cu = a->cu;
  p.T = a->T;
  p.H = a->H;
  p.per = kRows / a->H;
  p.window = a->window;
  p.sinks = a->sinks;
  p.scale_log2 = (a->scale < 0.f ? -a->scale : a->scale) * 1.4426950408889634f;
  p.flip = a->scale < 0.f;
  p.out = a->out;
  p.out_ld = a->out_ld;
  p.lse = a->lse;
  p.dev_status = dev_status;
  const int box = a->kv->page < kTok ? a->kv->page : kTok;
  CUtensorMap mq, mk, mv;
  KVS_PROPAGATE(paged_tensor_map(&mk, a->kv->K, p.kv, box, 1, "paged_prompt_attn"));
  KVS_PROPAGATE(paged_tensor_map(&mv, a->kv->V, p.kv, box, 1, "paged_prompt_attn"));
  KVS_PROPAGATE(query_tensor_map(&mq, a, p.per));
  p.test_warp = test_warp;
  p.wait_cycles = wait_cycles;
  p.pieces = test_warp >= 0 ? 1
                            : pieces_of(p.kv.R, p.kv.G, p.H, p.T, static_cast<int64_t>(a->kv->max_pages) * a->kv->page,
                                        p.window, p.sinks);
  carve(&p, ws, p.kv.G, p.H, p.T, p.pieces);
  const int64_t items = most_items(p.kv.R, p.kv.G, p.H, p.T) * p.pieces;
  KVS_REQUIRE(items < (1ll << 31) - (1 << 20), KVS_EUNSUPPORTED, "paged_prompt_attn: T=%d queries of G=%d KV heads", a->T,
              p.kv.G);
  const auto go = [&](auto kernel) -> kvs_status {
    // the register split must fit what the kernel is launched with, or the softmax
    // warps would wait for registers that never come
    static const int regs = [&] {
      cudaFuncAttributes f{};
      return cudaFuncGetAttributes(&f, kernel.value) == cudaSuccess ? f.numRegs : 0;
    }();
    KVS_REQUIRE(regs * kThreads >= 32 * kSoftWarps * kSoftRegs + (kThreads - 32 * kSoftWarps) * kOtherRegs, KVS_ECUDA,
                "paged_prompt_attn: built with %d registers a thread", regs);
    const int sms = sm_count();
    allow_smem<kernel.value>(sizeof(PromptSmem));
    launch_chained(kernel.value, dim3(static_cast<unsigned>(items < sms ? items : sms)), dim3(kThreads),
                   sizeof(PromptSmem), s, p, mq, mk, mv);
    return KVS_OK;
  };
  if (test_warp >= 0)
    KVS_PROPAGATE(go(std::integral_constant<decltype(&paged_prompt_kernel<false, true>), paged_prompt_kernel<false, true>>()));
  else if (p.pieces > 1)
    KVS_PROPAGATE(go(std::integral_constant<decltype(&paged_prompt_kernel<true>), paged_prompt_kernel<true>>()));
  else
    KVS_PROPAGATE(go(std::integral_constant<decltype(&paged_prompt_kernel<false>), paged_prompt_kernel<false>>()));
  if (p.pieces > 1) {
    const int64_t rows = static_cast<int64_t>(p.T) * p.kv.G * p.H;
    launch_chained(paged_prompt_join_kernel, dim3(static_cast<unsigned>((rows + 7) / 8)), dim3(256), 0, s, p);
  }
  return check_launch("paged_prompt_attn");
}

}  // namespace kvs
