// paged_api.cuh - the C ABI of the paged key-value cache (include/ra.h):
// argument validation and launches.  Included by api.cu, whose helpers it uses.
#pragma once

#include <stdlib.h>

#include "page_select.cuh"
#include "paged.cuh"
#include "paged_decode.cuh"

namespace {

using namespace ra;

inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

inline int cache_code(ra_dtype dt) { return dt == RA_BF16 ? kCacheBf16 : dt == RA_I8 ? kCacheI8 : kCacheE4M3; }

inline int page_shift_of(int page_size) {
  return page_size == 16 ? 4 : page_size == 32 ? 5 : page_size == 64 ? 6 : page_size == 128 ? 7 : -1;
}

// The batch half of a cache argument: table, lengths and their ranges.
ra_status check_batch(const ra_paged_cache* c) {
  if (!c) return RA_ERR_INVALID_ARG;
  if (c->B < 1 || c->max_pages < 1 || c->n_pages < 1 || c->Hkv < 1) return RA_ERR_INVALID_ARG;
  if (page_shift_of(c->page_size) < 0 || (c->D != 64 && c->D != 128)) return RA_ERR_UNSUPPORTED;
  if (static_cast<long long>(c->n_pages) * c->Hkv * c->page_size >= 0x7fffffffLL - 127) return RA_ERR_UNSUPPORTED;
  if (static_cast<long long>(c->max_pages) * c->page_size > kPgNone) return RA_ERR_UNSUPPORTED;  // see kPgNone
  if (!c->page_table || !c->seq_lens) return RA_ERR_INVALID_ARG;
  if (!aligned4(c->page_table) || !aligned4(c->seq_lens) || !aligned4(c->new_lens)) return RA_ERR_INVALID_ARG;
  return RA_OK;
}

// The whole argument: the batch, the pages and what belongs to their type.
ra_status check_cache(const ra_paged_cache* c) {
  const ra_status s = check_batch(c);
  if (s != RA_OK) return s;
  if (c->dtype != RA_BF16 && c->dtype != RA_I8 && c->dtype != RA_E4M3)
    return c->dtype == RA_F32 ? RA_ERR_UNSUPPORTED : RA_ERR_INVALID_ARG;
  if (!c->k_pages || !c->v_pages || !aligned16(c->k_pages) || !aligned16(c->v_pages)) return RA_ERR_INVALID_ARG;
  const bool scaled = c->dtype != RA_BF16;
  if (scaled != (c->k_scales != nullptr) || scaled != (c->v_scales != nullptr)) return RA_ERR_INVALID_ARG;
  if (!aligned16(c->k_scales) || !aligned16(c->v_scales) || !aligned16(c->key_bounds)) return RA_ERR_INVALID_ARG;
  return RA_OK;
}

PagedBatch batch_of(const ra_paged_cache* c, int T) {
  PagedBatch b;
  b.page_table = c->page_table;
  b.seq_lens = c->seq_lens;
  b.new_lens = c->new_lens;
  b.B = c->B;
  b.T = T;
  b.max_pages = c->max_pages;
  b.n_pages = c->n_pages;
  b.Hkv = c->Hkv;
  b.page_shift = page_shift_of(c->page_size);
#ifdef RA_DEBUG_BOUNDS
  // an offset that one check of each kernel adds to its index: the check fails, the access is left out
  const char* inject = getenv("RA_DEBUG_INJECT_PAGED");
  b.inject = inject ? atoll(inject) : 0;
#endif
  return b;
}

// Launch as a programmatic dependent of the stream's last kernel: see chain_launches.
template <typename... P, typename... A>
ra_status launch_chained(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st, const A&... args) {
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cuda_status(cudaLaunchKernelEx(&cfg, kernel, args...));
}

template <int D>
ra_status launch_append_d(const AppendArgs& a, int et, unsigned grid, cudaStream_t st) {
  if (et == kCacheBf16) return launch_chained(cache_append_kernel<D, kCacheBf16>, grid, kAppendThreads, 0, st, a);
  if (et == kCacheI8) return launch_chained(cache_append_kernel<D, kCacheI8>, grid, kAppendThreads, 0, st, a);
  return launch_chained(cache_append_kernel<D, kCacheE4M3>, grid, kAppendThreads, 0, st, a);
}

template <int D, typename Tout>
ra_status launch_read_t(const ReadArgs& a, int et, unsigned grid, cudaStream_t st) {
  if (et == kCacheBf16) return launch_chained(cache_read_kernel<D, kCacheBf16, Tout>, grid, kReadThreads, 0, st, a);
  if (et == kCacheI8) return launch_chained(cache_read_kernel<D, kCacheI8, Tout>, grid, kReadThreads, 0, st, a);
  return launch_chained(cache_read_kernel<D, kCacheE4M3, Tout>, grid, kReadThreads, 0, st, a);
}

constexpr int kPgMinRun = 1;  // shortest run of a team, in units of the line (5, two tiles: 17 us for 1,000 keys, against 12)

struct PagedPlan {
  int rows, R, teams;  // query rows per KV head, warps per team, teams of a full grid
  size_t part_o, part_ml, cut, total;
};

ra_status check_queries(int B, int Tq, int Hq, int Hkv, int D) {
  if (B < 1 || Tq < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0) return RA_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return RA_ERR_UNSUPPORTED;
  if (static_cast<long long>(Hq / Hkv) * Tq > kDecMaxRows) return RA_ERR_UNSUPPORTED;
  if (static_cast<long long>(B) * Tq * Hq > 0x7fffffffLL) return RA_ERR_UNSUPPORTED;
  return RA_OK;
}

PagedPlan paged_plan(int B, int Tq, int Hq, int Hkv, int D) {
  PagedPlan p;
  p.rows = (Hq / Hkv) * Tq;
  p.R = p.rows <= 16 ? 1 : p.rows <= 32 ? 2 : 4;
  p.teams = sm_count() * (p.R == 1 ? 15 : 11 / p.R);  // most consumer warps of any cache type
  p.part_o = 0;
  p.part_ml = align256(static_cast<size_t>(p.teams) * 2 * p.rows * D * 4);
  p.cut = align256(p.part_ml + static_cast<size_t>(p.teams) * 2 * p.rows * 8);
  p.total = align256(p.cut + static_cast<size_t>(B) * Hkv * 8);
  return p;
}

template <int D, int COLS, int WPR, int NW>
ra_status launch_paged_combine(const PagedArgs& a, int teams, cudaStream_t st) {
  const long long rows = static_cast<long long>(a.bt.B) * a.bt.Hkv * a.rows;
  const long long grid = (rows + NW / WPR - 1) / (NW / WPR) * (D / COLS);
  return launch_chained(paged_combine_kernel<D, COLS, WPR, NW>, static_cast<unsigned>(grid), 32 * NW, 0, st, a, teams);
}

template <int D, int ET, int NB, bool TEAMS>
ra_status launch_paged_t(const PagedArgs& a, cudaStream_t st) {
  using SL = PgSmem<D, ET, NB, TEAMS>;
  static int attr_set[64] = {0};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 64 || !attr_set[dev]) {
    if (cudaFuncSetAttribute(paged_partial_kernel<D, ET, NB, TEAMS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             SL::kBytes) != cudaSuccess)
      return RA_ERR_CUDA;
    if (dev < 64) attr_set[dev] = 1;
  }
  // the longest line that the table (or the selection) allows
  const long long pages = a.selected && a.n_sel < a.bt.max_pages ? a.n_sel : a.bt.max_pages;
  const long long tiles = ((pages << a.bt.page_shift) + kPgKeys - 1) / kPgKeys;
  const long long line = (tiles + kPgPairCost) * a.bt.B * a.bt.Hkv;
  const long long runs = (line + a.min_run - 1) / a.min_run;
  const int grid = static_cast<int>(runs < sm_count() ? runs : sm_count());
  const ra_status s = launch_chained(paged_partial_kernel<D, ET, NB, TEAMS>, grid, SL::kThreads, SL::kBytes, st, a);
  if (s != RA_OK) return s;
  // a row's parts: 32 warps where the rows are few, one where they alone fill the GPU
  const long long rows = static_cast<long long>(a.bt.B) * a.bt.Hkv * a.rows;
  const int teams = grid * (SL::kWarps / a.R);
  if (rows * (D / 32) <= sm_count()) return launch_paged_combine<D, 32, 32, 32>(a, teams, st);
  if (rows <= 16 * sm_count()) return launch_paged_combine<D, D, 8, 8>(a, teams, st);
  return launch_paged_combine<D, D, 1, 8>(a, teams, st);
}

template <int D, int ET>
ra_status launch_paged_e(const PagedArgs& a, cudaStream_t st) {
  if (a.rows <= 8) return launch_paged_t<D, ET, 1, false>(a, st);
  return a.R == 1 ? launch_paged_t<D, ET, 2, false>(a, st) : launch_paged_t<D, ET, 2, true>(a, st);
}

template <int D>
ra_status launch_paged_d(const PagedArgs& a, int et, cudaStream_t st) {
  if (et == kCacheBf16) return launch_paged_e<D, kCacheBf16>(a, st);
  if (et == kCacheI8) return launch_paged_e<D, kCacheI8>(a, st);
  return launch_paged_e<D, kCacheE4M3>(a, st);
}

// Slots of one (sequence, KV head) in the workspace of a selection.
long long slot_stride(int max_pages) { return (static_cast<long long>(max_pages) + 15) / 16 * 16; }

// Most pages that T consecutive tokens touch.
int page_span(int T, int page_size) {
  return static_cast<int>((static_cast<long long>(T) + page_size - 2) / page_size) + 1;
}

template <int D>
ra_status launch_select_d(const SelectArgs& a, cudaStream_t st) {
  const int per = 16 * (kScoreThreads / 32);  // pages of a block
  // blocks for the table's width, up to 32 an SM over all pairs: the sequences may be much shorter
  const long long pairs = static_cast<long long>(a.bt.B) * a.bt.Hkv;
  const long long need = (a.bt.max_pages + per - 1) / per, most = (32LL * sm_count() + pairs - 1) / pairs;
  const dim3 grid(static_cast<unsigned>(need < most ? need : most), a.bt.Hkv, a.bt.B);
  const ra_status s = launch_chained(page_score_kernel<D>, grid, kScoreThreads, 0, st, a);
  if (s != RA_OK) return s;
  return launch_chained(page_select_kernel<D>, static_cast<unsigned>(pairs), kSelThreads, 0, st, a);
}

}  // namespace

extern "C" {

ra_status ra_cache_append(const ra_paged_cache* cache, const void* k, const void* v, ra_dtype in_dtype, int T,
                          void* stream) {
  ra_status s = check_cache(cache);
  if (s != RA_OK) return s;
  if (in_dtype != RA_BF16) return in_dtype == RA_F32 ? RA_ERR_UNSUPPORTED : RA_ERR_INVALID_ARG;
  if (T < 1 || !k || !v || !aligned16(k) || !aligned16(v)) return RA_ERR_INVALID_ARG;
  AppendArgs a;
  memset(&a, 0, sizeof(a));
  a.bt = batch_of(cache, T);
  a.k = static_cast<const __nv_bfloat16*>(k);
  a.v = static_cast<const __nv_bfloat16*>(v);
  a.k_pages = cache->k_pages;
  a.v_pages = cache->v_pages;
  a.k_scales = cache->k_scales;
  a.v_scales = cache->v_scales;
  a.bounds = static_cast<__nv_bfloat16*>(cache->key_bounds);
  const int ps = cache->page_size;
  a.span = page_span(T, ps);
  a.wpu = 1;  // about 16 rows for each warp of a unit, a CTA's warps at most
  while (a.wpu * 16 < ps && a.wpu * 16 < T && a.wpu < kAppendThreads / 32) a.wpu *= 2;
  a.units = static_cast<long long>(cache->B) * a.span * cache->Hkv;
  const int upc = (kAppendThreads / 32) / a.wpu;
  const long long grid = (a.units + upc - 1) / upc;
  if (grid > 0x7fffffffLL) return RA_ERR_UNSUPPORTED;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int et = cache_code(cache->dtype);
  return cache->D == 128 ? launch_append_d<128>(a, et, static_cast<unsigned>(grid), st)
                         : launch_append_d<64>(a, et, static_cast<unsigned>(grid), st);
}

ra_status ra_cache_read(const ra_paged_cache* cache, int first, int T, void* k, void* v, ra_dtype out_dtype,
                        void* stream) {
  ra_status s = check_cache(cache);
  if (s != RA_OK) return s;
  if (out_dtype != RA_F32 && out_dtype != RA_BF16) return RA_ERR_INVALID_ARG;
  if (first < 0 || T < 1 || !aligned16(k) || !aligned16(v)) return RA_ERR_INVALID_ARG;
  if (!k && !v) return RA_OK;
  ReadArgs a;
  memset(&a, 0, sizeof(a));
  a.bt = batch_of(cache, T);
  a.bt.new_lens = nullptr;
  a.first = first;
  a.pages[0] = cache->k_pages;
  a.pages[1] = cache->v_pages;
  a.scales[0] = cache->k_scales;
  a.scales[1] = cache->v_scales;
  a.out[0] = k;
  a.out[1] = v;
  a.groups = (T - 1) / read_rows(cache->D) + 1;
  a.units = static_cast<long long>(cache->B) * a.groups * cache->Hkv;
  const long long grid = (a.units - 1) / (kReadThreads / 32) + 1;
  if (grid > 0x7fffffffLL) return RA_ERR_UNSUPPORTED;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int et = cache_code(cache->dtype);
  const unsigned g = static_cast<unsigned>(grid);
  if (out_dtype == RA_BF16)
    return cache->D == 128 ? launch_read_t<128, __nv_bfloat16>(a, et, g, st) : launch_read_t<64, __nv_bfloat16>(a, et, g, st);
  return cache->D == 128 ? launch_read_t<128, float>(a, et, g, st) : launch_read_t<64, float>(a, et, g, st);
}

size_t ra_paged_decode_workspace(int B, int Tq, int Hq, int Hkv, int D) {
  if (check_queries(B, Tq, Hq, Hkv, D) != RA_OK) return static_cast<size_t>(-1);
  return paged_plan(B, Tq, Hq, Hkv, D).total;
}

ra_status ra_paged_decode_attention(const void* q, ra_dtype in_dtype, const ra_paged_cache* cache, int Tq, int Hq,
                                    int causal, const int32_t* selected, int n_sel, void* out, ra_dtype out_dtype,
                                    float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  ra_status s = check_cache(cache);
  if (s != RA_OK) return s;
  s = check_queries(cache->B, Tq, Hq, cache->Hkv, cache->D);
  if (s != RA_OK) return s;
  if (in_dtype != RA_BF16) return in_dtype == RA_F32 ? RA_ERR_UNSUPPORTED : RA_ERR_INVALID_ARG;
  if (out_dtype != RA_F32 && out_dtype != RA_BF16) return RA_ERR_INVALID_ARG;
  if (!q || !out || !lse || !aligned16(q) || !aligned16(out) || !aligned4(lse)) return RA_ERR_INVALID_ARG;
  if (selected ? n_sel < 1 || !aligned4(selected) : n_sel != 0) return RA_ERR_INVALID_ARG;
  const PagedPlan p = paged_plan(cache->B, Tq, Hq, cache->Hkv, cache->D);
  if (!workspace || workspace_bytes < p.total) return RA_ERR_WORKSPACE;
  if (reinterpret_cast<uintptr_t>(workspace) & 255) return RA_ERR_INVALID_ARG;
  // a team's run of the line (see launch_paged_t) is counted in 32 bits
  const long long width = static_cast<long long>(cache->max_pages) * cache->page_size / kPgKeys + 1 + kPgPairCost;
  if (width * cache->B >= (1LL << 30) * sm_count() / cache->Hkv) return RA_ERR_UNSUPPORTED;
  PagedArgs a;
  memset(&a, 0, sizeof(a));
  a.bt = batch_of(cache, Tq);
  a.Hq = Hq;
  a.groups = Hq / cache->Hkv;
  a.rows = p.rows;
  a.causal = causal != 0;
  a.R = p.R;
  a.min_run = kPgMinRun;
  a.n_sel = n_sel;
  a.selected = selected;
  a.scale_log2 = static_cast<float>(1.4426950408889634 / sqrt(static_cast<double>(cache->D)));
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.k_pages = cache->k_pages;
  a.v_pages = cache->v_pages;
  a.k_scales = cache->k_scales;
  a.v_scales = cache->v_scales;
  char* ws = static_cast<char*>(workspace);
  a.part_o = reinterpret_cast<float*>(ws + p.part_o);
  a.part_ml = reinterpret_cast<float2*>(ws + p.part_ml);
  a.cut = reinterpret_cast<int2*>(ws + p.cut);
  a.out = out;
  a.out_bf16 = out_dtype == RA_BF16;
  a.lse = lse;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int et = cache_code(cache->dtype);
  return cache->D == 128 ? launch_paged_d<128>(a, et, st) : launch_paged_d<64>(a, et, st);
}

size_t ra_page_select_workspace(int B, int Hkv, int max_pages) {
  if (B < 1 || Hkv < 1 || max_pages < 1) return static_cast<size_t>(-1);
  return align256(static_cast<size_t>(B) * Hkv * slot_stride(max_pages) * 8);
}

ra_status ra_page_select(const void* q, ra_dtype in_dtype, const ra_paged_cache* cache, int Tq, int Hq, int n_sel,
                         int32_t* selected, void* workspace, size_t workspace_bytes, void* stream) {
  ra_status s = check_batch(cache);
  if (s != RA_OK) return s;
  s = check_queries(cache->B, Tq, Hq, cache->Hkv, cache->D);
  if (s != RA_OK) return s;
  if (cache->B > 65535 || cache->Hkv > 65535) return RA_ERR_UNSUPPORTED;
  if (in_dtype != RA_BF16) return in_dtype == RA_F32 ? RA_ERR_UNSUPPORTED : RA_ERR_INVALID_ARG;
  if (n_sel < page_span(Tq, cache->page_size)) return RA_ERR_INVALID_ARG;
  if (!q || !aligned16(q) || !cache->key_bounds || !aligned16(cache->key_bounds) || !selected || !aligned4(selected))
    return RA_ERR_INVALID_ARG;
  if (!workspace || workspace_bytes < ra_page_select_workspace(cache->B, cache->Hkv, cache->max_pages))
    return RA_ERR_WORKSPACE;
  if (reinterpret_cast<uintptr_t>(workspace) & 255) return RA_ERR_INVALID_ARG;
  SelectArgs a;
  memset(&a, 0, sizeof(a));
  a.bt = batch_of(cache, Tq);
  a.Hq = Hq;
  a.groups = Hq / cache->Hkv;
  a.rows = a.groups * Tq;
  a.n_sel = n_sel;
  a.stride = slot_stride(cache->max_pages);
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.bounds = static_cast<const __nv_bfloat16*>(cache->key_bounds);
  a.slots = static_cast<unsigned long long*>(workspace);
  a.selected = selected;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return cache->D == 128 ? launch_select_d<128>(a, st) : launch_select_d<64>(a, st);
}

}  // extern "C"
