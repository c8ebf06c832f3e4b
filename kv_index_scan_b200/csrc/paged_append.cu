// paged_append.cu -- the newest tokens' K and V rows into the pages of their
// requests: packed row cu[r] + t of c = cu[r+1] - cu[r] new tokens goes to
// position n[r] - c + t, and its weight and place start at 0 and seen[r] - c + t.
//
// A copy: 512 bytes read and written per token and KV head. A warp takes up to
// kHeads heads of one token, sixteen lanes the K row and sixteen the V row in
// 16-byte pieces, all loads issued before the first store.
#include "paged.cuh"

namespace kvs {

namespace {

constexpr int kAppendWarps = 8;
constexpr int kHeads = 4;

// The request of packed row t: the last r with cu[r] <= t (cu[0] = 0), searched
// by the whole warp, 32 ways at a time. -1 for rows behind the last request.
__device__ __forceinline__ int request_of(const int32_t* cu, int R, int t, int lane) {
  if (t >= __ldg(cu + R)) return -1;
  int lo = 0, len = R;  // cu[lo] <= t < cu[lo + len]
  while (len > 1) {
    const int step = (len + 31) / 32;
    const int at = lo + lane * step;
    const unsigned le = __ballot_sync(0xFFFFFFFFu, lane * step < len && __ldg(cu + at) <= t);
    const int k = le ? 31 - __clz(le) : 0;
    len = min(step, len - k * step);
    lo += k * step;
  }
  return lo;
}

__global__ void __launch_bounds__(32 * kAppendWarps) paged_append_kernel(
    PagedView kv, const uint16_t* __restrict__ Knew, const uint16_t* __restrict__ Vnew, int64_t new_ld,
    const int32_t* __restrict__ cu, int T, float* __restrict__ mass, int32_t* __restrict__ pos,
    const int32_t* __restrict__ seen, int32_t* dev_status) {
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int groups = (kv.G + kHeads - 1) / kHeads;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kAppendWarps + (threadIdx.x >> 5);
  if (item >= static_cast<int64_t>(T) * groups) return;
  const int t = static_cast<int>(item / groups);
  const int g0 = static_cast<int>(item % groups) * kHeads, g1 = min(kv.G, g0 + kHeads);
  const bool isv = lane >= 16;
  const int c = 8 * (lane & 15);
  const uint16_t* from = (isv ? Vnew : Knew) + t * new_ld + c;
  uint4 v[kHeads];
#pragma unroll
  for (int h = 0; h < kHeads; ++h)
    if (g0 + h < g1) v[h] = __ldg(reinterpret_cast<const uint4*>(from + (g0 + h) * kD));
  int r = t, behind = 1;  // tokens of the request from this one on
  if (cu) {
    if (item == 0 && __ldg(cu + kv.R) > T) set_status(dev_status, KVS_EBOUNDS);  // rows that are not there
    r = request_of(cu, kv.R, t, lane);
    if (r < 0) return;
    const int first = __ldg(cu + r);
    behind = __ldg(cu + r + 1) - t;
    if (behind <= 0 || first > t) {  // offsets that do not begin at 0 or do not ascend: nobody's row
      set_status(dev_status, KVS_EBOUNDS);
      return;
    }
  }
  const int i = kv.n[r] - behind;
  if (i < 0 || i >= kv.cap()) {
    set_status(dev_status, KVS_EBOUNDS);
    return;
  }
  if (lane < g1 - g0) {
    const size_t at = (static_cast<size_t>(r) * kv.G + g0 + lane) * kv.cap() + i;
    if (mass) mass[at] = 0.f;
    if (pos) pos[at] = seen ? seen[r] - behind : i;
  }
  const int id = kv.page_of(r, i, dev_status);
  if (id < 0) return;
  uint16_t* to = (isv ? kv.V : kv.K) + kv.row(id, g0, i) + c;
#pragma unroll
  for (int h = 0; h < kHeads; ++h)
    if (g0 + h < g1) *reinterpret_cast<uint4*>(to + h * kv.head_stride) = v[h];
}

}  // namespace

kvs_status paged_append_launch(const PagedView& kv, const uint16_t* Knew, const uint16_t* Vnew, int64_t new_ld,
                               const int32_t* cu, int T, float* mass, int32_t* pos, const int32_t* seen,
                               int32_t* dev_status, cudaStream_t s) {
  const int64_t items = static_cast<int64_t>(T) * ((kv.G + kHeads - 1) / kHeads);
  const int64_t blocks = (items + kAppendWarps - 1) / kAppendWarps;
  KVS_REQUIRE(blocks < (1ll << 31), KVS_EUNSUPPORTED, "kvs_paged_append: T=%d tokens of G=%d heads", T, kv.G);
  launch_chained(paged_append_kernel, dim3(static_cast<unsigned>(blocks)), dim3(32 * kAppendWarps), 0, s, kv, Knew,
                 Vnew, new_ld, cu, T, mass, pos, seen, dev_status);
  return check_launch("kvs_paged_append");
}

}  // namespace kvs
