// paged_api.cu -- the extern "C" boundary of the paged K/V cache: argument
// checks on the host (nothing is launched or written when a check fails) and
// the launches, all on the caller's stream.
#include <cmath>

#include "paged.cuh"

namespace kvs {

PagedView paged_view(const kvs_paged_kv* kv) {
  PagedView v{};
  v.K = kv->K;
  v.V = kv->V;
  v.page_stride = kv->page_stride;
  v.head_stride = kv->head_stride;
  v.token_stride = kv->token_stride;
  v.table = kv->table;
  v.table_ld = kv->table_ld;
  v.n = kv->n;
  v.R = kv->R;
  v.G = kv->G;
  v.max_pages = kv->max_pages;
  v.num_pages = kv->num_pages;
  while ((1 << v.shift) < kv->page) ++v.shift;
  return v;
}

}  // namespace kvs

using namespace kvs;

namespace {

kvs_status check_paged(const char* who, const kvs_paged_kv* kv) {
  KVS_REQUIRE(kv != nullptr, KVS_EINVAL, "%s: the cache descriptor is null", who);
  KVS_REQUIRE(kv->K && kv->V && kv->table && kv->n, KVS_EINVAL, "%s: K/V/table/n must be non-null", who);
  KVS_REQUIRE(kv->D == kD, KVS_EUNSUPPORTED, "%s: D=%d (only 128 is built)", who, kv->D);
  KVS_REQUIRE(kv->R >= 1 && kv->G >= 1 && kv->G <= 65535 && kv->max_pages >= 1 && kv->num_pages >= 1, KVS_EINVAL,
              "%s: R=%d G=%d (1..65535) max_pages=%d num_pages=%d", who, kv->R, kv->G, kv->max_pages, kv->num_pages);
  KVS_REQUIRE(static_cast<int64_t>(kv->R) * kv->G < (1 << 24), KVS_EUNSUPPORTED, "%s: R*G=%lld (below 2^24)", who,
              static_cast<long long>(kv->R) * kv->G);
  KVS_REQUIRE(kv->page >= 16 && kv->page <= 1024 && (kv->page & (kv->page - 1)) == 0, KVS_EUNSUPPORTED,
              "%s: page=%d tokens (a power of two from 16 to 1024)", who, kv->page);
  KVS_REQUIRE(static_cast<int64_t>(kv->max_pages) * kv->page <= (1 << 30), KVS_EUNSUPPORTED,
              "%s: max_pages=%d pages of %d tokens (at most 2^30 tokens)", who, kv->max_pages, kv->page);
  KVS_REQUIRE(kv->table_ld >= kv->max_pages, KVS_EINVAL, "%s: table_ld=%lld < max_pages=%d", who,
              static_cast<long long>(kv->table_ld), kv->max_pages);
  for (int64_t st : {kv->page_stride, kv->head_stride, kv->token_stride})
    KVS_REQUIRE(st >= kD && st % 8 == 0 && st < (1ll << 38), KVS_EINVAL,
                "%s: strides must be multiples of 8 elements and at least 128, got %lld", who,
                static_cast<long long>(st));
  KVS_REQUIRE(aligned16(kv->K) && aligned16(kv->V), KVS_EINVAL, "%s: K and V must be 16-byte aligned", who);
  return KVS_OK;
}

kvs_status check_mask(const char* who, int window, int sinks, float scale) {
  // (the softmax is in base 2, so scale * log2(e) has to be finite too)
  KVS_REQUIRE(std::isfinite(scale * 1.4426950408889634f) && scale != 0.f, KVS_EINVAL,
              "%s: scale=%g must not be 0, and at most 2.3e38 in magnitude", who, static_cast<double>(scale));
  KVS_REQUIRE(window >= 0 && sinks >= 0, KVS_EINVAL, "%s: window=%d sinks=%d must not be negative", who, window,
              sinks);
  return KVS_OK;
}

kvs_status check_decode(const kvs_paged_decode_args* a, const void* ws, size_t ws_bytes) {
  KVS_REQUIRE(a != nullptr, KVS_EINVAL, "paged_decode_attn: args is null");
  KVS_PROPAGATE(check_paged("paged_decode_attn", a->kv));
  KVS_PROPAGATE(check_mask("paged_decode_attn", a->window, a->sinks, a->scale));
  KVS_REQUIRE(a->H >= 1 && a->H <= 8, KVS_EINVAL, "paged_decode_attn: H=%d query heads per KV head (1..8)", a->H);
  KVS_REQUIRE(a->q && a->out, KVS_EINVAL, "paged_decode_attn: q and out must be non-null");
  KVS_REQUIRE(a->q_dtype == KVS_F32 || a->q_dtype == KVS_BF16, KVS_EINVAL, "paged_decode_attn: q_dtype=%d", a->q_dtype);
  KVS_REQUIRE(aligned16(a->q) && aligned16(a->out), KVS_EINVAL, "paged_decode_attn: q and out must be 16-byte aligned");
  KVS_REQUIRE((a->mass == nullptr) == (a->mass_out == nullptr), KVS_EINVAL,
              "paged_decode_attn: mass and mass_out go together");
  const size_t need =
      paged_decode_ws_bytes(a->kv->R, a->kv->G, a->H, a->mass ? a->kv->max_pages * a->kv->page : 0);
  KVS_REQUIRE(need == 0 || (ws && ws_bytes >= need), KVS_EWORKSPACE, "paged_decode_attn: workspace %zu < %zu bytes",
              ws_bytes, need);
  KVS_REQUIRE(aligned16(ws), KVS_EINVAL, "paged_decode_attn: the workspace must be 16-byte aligned");
  return KVS_OK;
}

kvs_status check_prompt(const kvs_paged_prompt_args* a) {
  KVS_REQUIRE(a != nullptr, KVS_EINVAL, "paged_prompt_attn: args is null");
  KVS_PROPAGATE(check_paged("paged_prompt_attn", a->kv));
  KVS_PROPAGATE(check_mask("paged_prompt_attn", a->window, a->sinks, a->scale));
  KVS_REQUIRE(a->T >= 0, KVS_EINVAL, "paged_prompt_attn: T=%d", a->T);
  KVS_REQUIRE(a->H >= 1 && a->H <= 8, KVS_EINVAL, "paged_prompt_attn: H=%d query heads per KV head (1..8)", a->H);
  if (a->T == 0) return KVS_OK;
  KVS_REQUIRE(a->q && a->out && a->cu, KVS_EINVAL, "paged_prompt_attn: q, out and cu must be non-null");
  const int64_t width = static_cast<int64_t>(a->kv->G) * a->H * kD;
  KVS_REQUIRE(a->q_ld >= width && a->q_ld % 8 == 0 && a->out_ld >= width && a->out_ld % 8 == 0, KVS_EINVAL,
              "paged_prompt_attn: q_ld=%lld out_ld=%lld must be multiples of 8, at least G*H*128",
              static_cast<long long>(a->q_ld), static_cast<long long>(a->out_ld));
  KVS_REQUIRE(static_cast<int64_t>(a->T) * a->H < (1ll << 31) - 4096, KVS_EUNSUPPORTED,
              "paged_prompt_attn: T*H=%lld rows (below 2^31)", static_cast<long long>(a->T) * a->H);
  KVS_REQUIRE(aligned16(a->q) && aligned16(a->out), KVS_EINVAL, "paged_prompt_attn: q and out must be 16-byte aligned");
  return KVS_OK;
}

}  // namespace

extern "C" {

kvs_status kvs_paged_append(const kvs_paged_kv* kv, const uint16_t* Knew, const uint16_t* Vnew, int64_t new_ld,
                            const int32_t* cu, int32_t T, float* mass, int32_t* pos, const int32_t* seen,
                            int32_t* dev_status, void* stream) {
  KVS_PROPAGATE(check_paged("kvs_paged_append", kv));
  KVS_REQUIRE(T >= 0, KVS_EINVAL, "kvs_paged_append: T=%d", T);
  if (T == 0) return ok();
  KVS_REQUIRE(Knew && Vnew, KVS_EINVAL, "kvs_paged_append: Knew/Vnew must be non-null");
  KVS_REQUIRE(cu || T == kv->R, KVS_EINVAL, "kvs_paged_append: without cu there is one token a request, T=%d R=%d", T,
              kv->R);
  KVS_REQUIRE(new_ld >= static_cast<int64_t>(kv->G) * kD && new_ld % 8 == 0, KVS_EINVAL,
              "kvs_paged_append: new_ld=%lld must be a multiple of 8, at least G*128", static_cast<long long>(new_ld));
  KVS_REQUIRE(aligned16(Knew) && aligned16(Vnew), KVS_EINVAL, "kvs_paged_append: Knew and Vnew must be 16-byte aligned");
  KVS_REQUIRE(!seen || pos, KVS_EINVAL, "kvs_paged_append: seen without pos");
  KVS_PROPAGATE(paged_append_launch(paged_view(kv), Knew, Vnew, new_ld, cu, T, mass, pos, seen, dev_status,
                                    static_cast<cudaStream_t>(stream)));
  return ok();
}

size_t kvs_paged_decode_workspace_size(int32_t R, int32_t G, int32_t H, int32_t weight_cap) {
  return paged_decode_ws_bytes(R, G, H, weight_cap);
}

kvs_status paged_decode_attn(const kvs_paged_decode_args* a, void* ws, size_t ws_bytes, int32_t* dev_status,
                             void* stream) {
  KVS_PROPAGATE(check_decode(a, ws, ws_bytes));
  KVS_PROPAGATE(paged_decode_launch(a, ws, dev_status, static_cast<cudaStream_t>(stream)));
  return ok();
}

kvs_status kvs_selftest_paged_decode_timeout(const kvs_paged_decode_args* a, void* ws, size_t ws_bytes, int32_t warp,
                                             int64_t wait_cycles, int32_t* dev_status, void* stream) {
  KVS_PROPAGATE(check_decode(a, ws, ws_bytes));
  KVS_REQUIRE(dev_status && warp >= 0 && warp <= 4 && wait_cycles >= 1000 && wait_cycles <= 2000000000LL, KVS_EINVAL,
              "kvs_selftest_paged_decode_timeout: dev_status is required, warp=%d (0..4), wait_cycles=%lld (1e3 .. 2e9)",
              warp, static_cast<long long>(wait_cycles));
  KVS_REQUIRE(a->q_dtype == KVS_BF16 && !a->mass, KVS_EUNSUPPORTED,
              "kvs_selftest_paged_decode_timeout: bf16 queries without weights");
  KVS_PROPAGATE(paged_decode_launch(a, ws, dev_status, static_cast<cudaStream_t>(stream), warp, wait_cycles));
  return ok();
}

size_t kvs_paged_prompt_workspace_size(int32_t R, int32_t G, int32_t H, int32_t T, int32_t cap, int32_t window,
                                       int32_t sinks) {
  return paged_prompt_ws_bytes(R, G, H, T, cap, window, sinks);
}

size_t kvs_paged_prompt_workspace_bound(int32_t R, int32_t G, int32_t H, int32_t T, int32_t cap, int32_t window,
                                        int32_t sinks) {
  return paged_prompt_ws_bound(R, G, H, T, cap, window, sinks);
}

kvs_status paged_prompt_attn(const kvs_paged_prompt_args* a, void* ws, size_t ws_bytes, int32_t* dev_status,
                             void* stream) {
  KVS_PROPAGATE(check_prompt(a));
  if (a->T == 0) return ok();
  const size_t need = paged_prompt_ws_bytes(a->kv->R, a->kv->G, a->H, a->T, a->kv->max_pages * a->kv->page, a->window,
                                           a->sinks);
  KVS_REQUIRE(need == 0 || (ws && ws_bytes >= need), KVS_EWORKSPACE, "paged_prompt_attn: workspace %zu < %zu bytes",
              ws_bytes, need);
  KVS_REQUIRE(aligned16(ws), KVS_EINVAL, "paged_prompt_attn: the workspace must be 16-byte aligned");
  KVS_PROPAGATE(paged_prompt_launch(a, ws, dev_status, static_cast<cudaStream_t>(stream)));
  return ok();
}

kvs_status kvs_selftest_paged_prompt_timeout(const kvs_paged_prompt_args* a, int32_t warp, int64_t wait_cycles,
                                             int32_t* dev_status, void* stream) {
  KVS_PROPAGATE(check_prompt(a));
  KVS_REQUIRE(a->T > 0 && dev_status && warp >= 0 && warp <= 11 && wait_cycles >= 1000 && wait_cycles <= 2000000000LL,
              KVS_EINVAL,
              "kvs_selftest_paged_prompt_timeout: queries and dev_status are required, warp=%d (0..11), wait_cycles=%lld "
              "(1e3 .. 2e9)",
              warp, static_cast<long long>(wait_cycles));
  KVS_PROPAGATE(paged_prompt_launch(a, nullptr, dev_status, static_cast<cudaStream_t>(stream), warp, wait_cycles));
  return ok();
}

size_t kvs_paged_evict_workspace_size(int32_t R, int32_t G, int32_t budget) {
  return paged_evict_ws_bytes(R, G, budget);
}

kvs_status kvs_paged_evict(const kvs_paged_evict_args* a, void* ws, size_t ws_bytes, int32_t* dev_status,
                           void* stream) {
  KVS_REQUIRE(a != nullptr, KVS_EINVAL, "kvs_paged_evict: args is null");
  KVS_PROPAGATE(check_paged("kvs_paged_evict", a->kv));
  KVS_REQUIRE(a->mass && a->mass_out && a->n_out && a->src, KVS_EINVAL,
              "kvs_paged_evict: mass/mass_out/n_out/src must be non-null");
  KVS_REQUIRE((a->pos == nullptr) == (a->pos_out == nullptr), KVS_EINVAL,
              "kvs_paged_evict: pos and pos_out go together");
  KVS_REQUIRE(a->budget >= 1 && a->sinks >= 0 && a->recent >= 0 &&
                  static_cast<int64_t>(a->sinks) + a->recent <= a->budget,
              KVS_EINVAL, "kvs_paged_evict: budget=%d sinks=%d recent=%d (sinks + recent <= budget)", a->budget,
              a->sinks, a->recent);
  KVS_REQUIRE(a->budget <= (1 << 30), KVS_EUNSUPPORTED, "kvs_paged_evict: budget=%d (at most 2^30)", a->budget);
  const size_t need = paged_evict_ws_bytes(a->kv->R, a->kv->G, a->budget);
  KVS_REQUIRE(ws && ws_bytes >= need, KVS_EWORKSPACE, "kvs_paged_evict: workspace %zu < %zu bytes", ws_bytes, need);
  KVS_REQUIRE(aligned16(ws), KVS_EINVAL, "kvs_paged_evict: the workspace must be 16-byte aligned");
  KVS_PROPAGATE(paged_evict_launch(a, ws, dev_status, static_cast<cudaStream_t>(stream)));
  return ok();
}

}  // extern "C"
