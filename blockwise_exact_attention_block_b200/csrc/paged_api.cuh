// paged_api.cuh - the C ABI of the paged key-value cache (include/ra.h):
// argument validation and launches.  Included by api.cu, whose helpers it uses.
#pragma once

#include "paged.cuh"

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
  if (static_cast<long long>(c->max_pages) * c->page_size >= 0x7fffffffLL) return RA_ERR_UNSUPPORTED;
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
  return b;
}

template <int D>
ra_status launch_append_d(const AppendArgs& a, int et, unsigned grid, cudaStream_t st) {
  if (et == kCacheBf16) cache_append_kernel<D, kCacheBf16><<<grid, kAppendThreads, 0, st>>>(a);
  else if (et == kCacheI8) cache_append_kernel<D, kCacheI8><<<grid, kAppendThreads, 0, st>>>(a);
  else cache_append_kernel<D, kCacheE4M3><<<grid, kAppendThreads, 0, st>>>(a);
  return cuda_status(cudaGetLastError());
}

template <int D, typename Tout>
ra_status launch_read_t(const ReadArgs& a, int et, unsigned grid, cudaStream_t st) {
  if (et == kCacheBf16) cache_read_kernel<D, kCacheBf16, Tout><<<grid, 256, 0, st>>>(a);
  else if (et == kCacheI8) cache_read_kernel<D, kCacheI8, Tout><<<grid, 256, 0, st>>>(a);
  else cache_read_kernel<D, kCacheE4M3, Tout><<<grid, 256, 0, st>>>(a);
  return cuda_status(cudaGetLastError());
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
  a.span = static_cast<int>((static_cast<long long>(T) - 1 + ps - 1) / ps) + 1;
  a.wpu = 1;  // about 16 rows for each warp of a unit
  while (a.wpu * 16 < ps && a.wpu * 16 < T) a.wpu *= 2;
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
  a.groups = (T - 1) / kReadRows + 1;
  a.units = static_cast<long long>(cache->B) * a.groups * cache->Hkv;
  const long long grid = (a.units + 7) / 8;
  if (grid > 0x7fffffffLL) return RA_ERR_UNSUPPORTED;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int et = cache_code(cache->dtype);
  const unsigned g = static_cast<unsigned>(grid);
  if (out_dtype == RA_BF16)
    return cache->D == 128 ? launch_read_t<128, __nv_bfloat16>(a, et, g, st) : launch_read_t<64, __nv_bfloat16>(a, et, g, st);
  return cache->D == 128 ? launch_read_t<128, float>(a, et, g, st) : launch_read_t<64, float>(a, et, g, st);
}

}  // extern "C"
