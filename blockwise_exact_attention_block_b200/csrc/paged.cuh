// paged.cuh - the paged key-value cache's device side: lengths and page table
// entries with their checks, the 8-bit types, and the kernels that write new
// tokens into the pages and read a stretch of them back.
//
// Pages are head-major, [n_pages][Hkv][page_size][D]: a KV head's rows of a
// page are adjacent, so every reader of one head (attention, page selection,
// the read-back) touches whole runs of page_size * D values, and a sparse read
// of single pages costs no more per byte than a dense one.
#pragma once

#include "common.cuh"
#include "permute.cuh"

namespace ra {

constexpr int kCacheBf16 = 0, kCacheI8 = 1, kCacheE4M3 = 2;  // template codes of the cache types

struct PagedBatch {
  const int* page_table;  // [B][max_pages]
  const int* seq_lens;    // [B]
  const int* new_lens;    // [B] or null
  int B, T, max_pages, n_pages, Hkv;
  int page_shift;  // log2(page_size)
};

// Tokens of sequence b and how many of its T rows are real, held to their ranges.
struct SeqLen {
  int len, fresh;
};

__device__ __forceinline__ SeqLen seq_len_of(const PagedBatch& a, int b) {
  SeqLen s;
  s.len = a.seq_lens[b];
  const int cap = a.max_pages << a.page_shift;
  if (s.len < 0 || s.len > cap) {
    set_status(RA_ERR_DEVICE_BOUNDS);
    s.len = min(max(s.len, 0), cap);
  }
  const int most = min(a.T, s.len);
  s.fresh = a.new_lens ? a.new_lens[b] : most;
  if (s.fresh < 0 || s.fresh > most) {
    set_status(RA_ERR_DEVICE_BOUNDS);
    s.fresh = min(max(s.fresh, 0), most);
  }
  return s;
}

// Page `logical` (below the sequence's page count) of sequence b; -1, recorded,
// when the table holds no valid page there.
__device__ __forceinline__ int page_of(const PagedBatch& a, int b, int logical) {
  const int p = a.page_table[static_cast<long long>(b) * a.max_pages + logical];
  if (p >= 0 && p < a.n_pages) return p;
  set_status(RA_ERR_DEVICE_BOUNDS);
  return -1;
}

// ------------------------------------------------------------- 8-bit values

// The value of e4m3 magnitude code c (0 .. 126): exponent and mantissa moved
// into an fp32's fields and the bias difference 2^(127 - 7) multiplied in,
// which is exact and covers the subnormal codes.
__device__ __forceinline__ float e4m3_value(uint32_t c) {
  return __uint_as_float(c << 20) * 0x1p120f;
}

// Code of x (|x| <= m s up to rounding) in int8 with scale s: the integer
// nearest to the exact x / s, ties to even.  x * inv is within a few ulp of
// the quotient, so only a neighbour of the rounded product can be nearer; the
// remainder x - q s is exact in fp32 (x has 8 significant bits, |x - q s| is at
// most about s / 2 and a multiple of s's last bit), so the comparison with
// s / 2 decides every case as infinite precision would.
__device__ __forceinline__ int quant_i8(float x, float s, float inv) {
  float q = rintf(x * inv);
  const float r = fmaf(-q, s, x);
  const float half = 0.5f * s;
  if (fabsf(r) >= half) {  // past the border, or on it
    const float up = r > 0.f ? 1.f : -1.f;
    if (fabsf(r) > half || (static_cast<int>(q) & 1)) q += up;
  }
  return static_cast<int>(q);
}

// The same for e4m3; returns the 8-bit code.  The conversion of x * inv is the
// answer unless the product lies within a few ulp of a border between two
// values (the middle of a mantissa step: the low 20 bits of the fp32 are about
// 0x80000; all of the range below the smallest normal value, 2^-6, is checked);
// there the exact remainders of the two candidates decide, ties to the even code.
__device__ __forceinline__ uint32_t quant_e4m3(float x, float s, float inv) {
  const float t = fabsf(x) * inv;
  uint16_t pair;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(pair) : "f"(0.f), "f"(t));
  uint32_t c = pair & 0xffu;
  const uint32_t low = (__float_as_uint(t) - 0x80000u + 8u) & 0xfffffu;
  if (low <= 16u || t < 0x1p-6f) {
    const float ax = fabsf(x);
    const float r = fmaf(-e4m3_value(c), s, ax);
    const uint32_t other = r > 0.f ? min(c + 1u, 126u) : (c > 0u ? c - 1u : 0u);
    const float r2 = fabsf(fmaf(-e4m3_value(other), s, ax)), r1 = fabsf(r);
    if (r2 < r1 || (r2 == r1 && (c & 1u))) c = other;
  }
  return c | (x < 0.f ? 0x80u : 0u);
}

// Eight cached values (8 codes of one row, or 8 bf16) as fp32.
template <int ET>
__device__ __forceinline__ void cached_octet(const void* pages, long long index, float scale, float (&v)[8]) {
  if constexpr (ET == kCacheBf16) {
    const uint4 w = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(pages) + index);
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(u[i] << 16);
      v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  } else {
    const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(pages) + index);
    const uint32_t u[2] = {w.x, w.y};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t c = (u[i >> 2] >> (8 * (i & 3))) & 0xffu;
      if constexpr (ET == kCacheI8) v[i] = static_cast<float>(static_cast<int8_t>(c)) * scale;
      else v[i] = __uint_as_float(__float_as_uint(e4m3_value(c & 0x7fu)) | ((c & 0x80u) << 24)) * scale;
    }
  }
}

// ------------------------------------------------------------------- append

struct AppendArgs {
  PagedBatch bt;
  const __nv_bfloat16* k;  // [B][T][Hkv][D]
  const __nv_bfloat16* v;
  void* k_pages;
  void* v_pages;
  float* k_scales;
  float* v_scales;
  __nv_bfloat16* bounds;  // [n_pages][Hkv][2][D] or null
  int span;               // pages that T consecutive tokens can touch
  int wpu;                // warps per unit
  long long units;        // B * span * Hkv
};

constexpr int kAppendThreads = 256;
constexpr int kAppendBatch = 4;  // rows of K and V a lane holds in flight

// One row's octet of this lane into the cache: bits, or codes and the row's
// scale (largest magnitude over the LPR lanes of the row).  bf16 magnitudes
// compare as integers, a NaN or an infinity above every finite value.
template <int D, int ET>
__device__ __forceinline__ void append_row(const uint4& w, bool act, int lane_in_row, void* pages, float* scales,
                                           long long row) {
  constexpr int LPR = D / 8;
  if constexpr (ET == kCacheBf16) {
    if (act) *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(pages) + row * D + 8 * lane_in_row) = w;
  } else {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
    uint32_t am = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) am = __vmaxu2(am, u[i] & 0x7fff7fffu);
    am = max(am & 0xffffu, am >> 16);
#pragma unroll
    for (int o = 1; o < LPR; o <<= 1) am = max(am, __shfl_xor_sync(0xffffffffu, am, o));
    float s = 0.f, inv = 0.f;
    if (am >= 0x7f80u) {
      s = __uint_as_float(0x7fc00000u);  // NaN: the row reads back as NaN
    } else if (__uint_as_float(am << 16) >= 0x1p-100f) {
      s = __fdiv_rn(__uint_as_float(am << 16), ET == kCacheI8 ? 127.f : 448.f);
      inv = 1.f / s;
    }
    uint32_t code[2] = {0u, 0u};
    if (inv != 0.f) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float x = __uint_as_float((i & 1) ? (u[i >> 1] & 0xffff0000u) : (u[i >> 1] << 16));
        const uint32_t c = ET == kCacheI8 ? static_cast<uint32_t>(quant_i8(x, s, inv)) & 0xffu : quant_e4m3(x, s, inv);
        code[i >> 2] |= c << (8 * (i & 3));
      }
    }
    if (act) {
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(pages) + row * D + 8 * lane_in_row) = make_uint2(code[0], code[1]);
      if (lane_in_row == 0) scales[row] = s;
    }
  }
}

// A unit is (sequence, touched page, KV head), heads fastest, so that a CTA's
// units read whole token rows between them; wpu warps of the CTA share a unit's
// rows.  D / 8 lanes hold a row (16 bytes of input each), 32 / (D / 8) rows per
// warp and step, kAppendBatch steps' loads in flight.  The column minima and
// maxima of the keys stay in registers until the unit's end.
template <int D, int ET>
__global__ void __launch_bounds__(kAppendThreads) cache_append_kernel(const __grid_constant__ AppendArgs a) {
  constexpr int LPR = D / 8, RPW = 32 / LPR;
  __shared__ float s_lo[kAppendThreads / 32][D], s_hi[kAppendThreads / 32][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane / LPR, lr = lane % LPR;
  const int upc = (kAppendThreads / 32) / a.wpu, wi = warp % a.wpu;  // units per CTA, warp in the unit
  const long long unit = static_cast<long long>(blockIdx.x) * upc + warp / a.wpu;
  int page = -1, r0 = 0, r1 = 0, h = 0, b = 0, tok0 = 0;
  if (unit < a.units) {
    h = static_cast<int>(unit % a.bt.Hkv);
    const long long bj = unit / a.bt.Hkv;
    const int j = static_cast<int>(bj % a.span);
    b = static_cast<int>(bj / a.span);
    const SeqLen s = seq_len_of(a.bt, b);
    const int ps = 1 << a.bt.page_shift;
    const int begin = s.len - s.fresh;  // position of the first new token
    const int logical = (begin >> a.bt.page_shift) + j;
    const long long first = static_cast<long long>(logical) << a.bt.page_shift;  // position of the page's row 0
    if (s.fresh > 0 && first < s.len) {
      page = page_of(a.bt, b, logical);
      r0 = max(begin - static_cast<int>(first), 0);
      r1 = min(s.len - static_cast<int>(first), ps);
      tok0 = static_cast<int>(first) - begin;  // token of the page's row 0 (may be negative)
    }
  }
  float lo[8], hi[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    lo[i] = INFINITY;
    hi[i] = -INFINITY;
  }
  if (page >= 0) {
    const long long prow = (static_cast<long long>(page) * a.bt.Hkv + h) << a.bt.page_shift;
    const int step = a.wpu * RPW;
    for (int rb = r0 + wi * RPW; rb < r1; rb += step * kAppendBatch) {
      uint4 kw[kAppendBatch], vw[kAppendBatch];
#pragma unroll
      for (int u = 0; u < kAppendBatch; ++u) {
        const int r = rb + u * step + sub;
        kw[u] = vw[u] = make_uint4(0u, 0u, 0u, 0u);
        if (r < r1) {
          const long long src = ((static_cast<long long>(b) * a.bt.T + tok0 + r) * a.bt.Hkv + h) * D + 8 * lr;
          kw[u] = __ldcs(reinterpret_cast<const uint4*>(a.k + src));
          vw[u] = __ldcs(reinterpret_cast<const uint4*>(a.v + src));
        }
      }
#pragma unroll
      for (int u = 0; u < kAppendBatch; ++u) {
        if (rb + u * step >= r1) break;  // the same for the whole warp
        const int r = rb + u * step + sub;
        const bool act = r < r1;
        append_row<D, ET>(kw[u], act, lr, a.k_pages, a.k_scales, prow + r);
        append_row<D, ET>(vw[u], act, lr, a.v_pages, a.v_scales, prow + r);
        if (a.bounds && act) {
          const uint32_t w[4] = {kw[u].x, kw[u].y, kw[u].z, kw[u].w};
#pragma unroll
          for (int i = 0; i < 8; ++i) {  // fminf and fmaxf pass over a NaN
            const float x = __uint_as_float((i & 1) ? (w[i >> 1] & 0xffff0000u) : (w[i >> 1] << 16));
            lo[i] = fminf(lo[i], x);
            hi[i] = fmaxf(hi[i], x);
          }
        }
      }
    }
  }
  if (a.bounds == nullptr) return;
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int o = LPR; o < 32; o <<= 1) {
      lo[i] = fminf(lo[i], __shfl_xor_sync(0xffffffffu, lo[i], o));
      hi[i] = fmaxf(hi[i], __shfl_xor_sync(0xffffffffu, hi[i], o));
    }
  if (a.wpu > 1) {
    if (sub == 0)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        s_lo[warp][8 * lr + i] = lo[i];
        s_hi[warp][8 * lr + i] = hi[i];
      }
    __syncthreads();
    if (wi == 0)
      for (int w = 1; w < a.wpu; ++w)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          lo[i] = fminf(lo[i], s_lo[warp + w][8 * lr + i]);
          hi[i] = fmaxf(hi[i], s_hi[warp + w][8 * lr + i]);
        }
  }
  if (page < 0 || wi != 0 || sub != 0) return;
  __nv_bfloat16* bl = a.bounds + (static_cast<long long>(page) * a.bt.Hkv + h) * 2 * D + 8 * lr;
  if (r0 > 0) {  // earlier tokens' bounds stand in the page
    float old[8];
    cached_octet<kCacheBf16>(bl, 0, 1.f, old);
#pragma unroll
    for (int i = 0; i < 8; ++i) lo[i] = fminf(lo[i], old[i]);
    cached_octet<kCacheBf16>(bl, D, 1.f, old);
#pragma unroll
    for (int i = 0; i < 8; ++i) hi[i] = fmaxf(hi[i], old[i]);
  }
  // the bounds are bf16 values (or infinities) already: packing them is exact
  *reinterpret_cast<uint4*>(bl) = make_uint4(pack_bf16x2(lo[0], lo[1]), pack_bf16x2(lo[2], lo[3]),
                                             pack_bf16x2(lo[4], lo[5]), pack_bf16x2(lo[6], lo[7]));
  *reinterpret_cast<uint4*>(bl + D) = make_uint4(pack_bf16x2(hi[0], hi[1]), pack_bf16x2(hi[2], hi[3]),
                                                 pack_bf16x2(hi[4], hi[5]), pack_bf16x2(hi[6], hi[7]));
}

// --------------------------------------------------------------------- read

struct ReadArgs {
  PagedBatch bt;  // T = rows of the output
  int first;
  const void* pages[2];    // K, V
  const float* scales[2];
  void* out[2];            // null: not asked for
  int groups;              // 16-row groups of T
  long long units;         // B * groups * Hkv
};

constexpr int kReadRows = 16;  // output rows of a warp

// A warp takes 16 consecutive tokens of one KV head (runs of 16 rows of a page
// to read, heads side by side in the CTA to write); D / 8 lanes hold a row.
template <int D, int ET, typename Tout>
__global__ void __launch_bounds__(256) cache_read_kernel(const __grid_constant__ ReadArgs a) {
  constexpr int LPR = D / 8, RPW = 32 / LPR, N = kReadRows / RPW;
  const int lane = threadIdx.x & 31;
  const int sub = lane / LPR, lr = lane % LPR;
  const long long unit = static_cast<long long>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (unit >= a.units) return;
  const int h = static_cast<int>(unit % a.bt.Hkv);
  const long long bg = unit / a.bt.Hkv;
  const int g = static_cast<int>(bg % a.groups), b = static_cast<int>(bg / a.groups);
  const int t0 = g * kReadRows;
  const int len = seq_len_of(a.bt, b).len;
  // lane i < 16: the cache row of output row t0 + i, -1 where there is none
  long long mine = -1;
  const long long pos = static_cast<long long>(a.first) + t0 + lane;
  if (lane < kReadRows && pos < len) {
    const int page = page_of(a.bt, b, static_cast<int>(pos >> a.bt.page_shift));
    if (page >= 0)
      mine = ((static_cast<long long>(page) * a.bt.Hkv + h) << a.bt.page_shift) + (pos & ((1 << a.bt.page_shift) - 1));
  }
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    if (a.out[kv] == nullptr) continue;
    float v[N][8];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const long long row = __shfl_sync(0xffffffffu, mine, i * RPW + sub);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] = 0.f;
      if (row >= 0) {
        const float s = ET == kCacheBf16 ? 1.f : a.scales[kv][row];
        cached_octet<ET>(a.pages[kv], row * D + 8 * lr, s, v[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int t = t0 + i * RPW + sub;
      if (t >= a.bt.T) continue;
      Tout* dst = static_cast<Tout*>(a.out[kv]) + ((static_cast<long long>(b) * a.bt.T + t) * a.bt.Hkv + h) * D + 8 * lr;
      if constexpr (sizeof(Tout) == 2) {
        __stcs(reinterpret_cast<uint4*>(dst),
               make_uint4(pack_bf16x2(v[i][0], v[i][1]), pack_bf16x2(v[i][2], v[i][3]), pack_bf16x2(v[i][4], v[i][5]),
                          pack_bf16x2(v[i][6], v[i][7])));
      } else {
        __stcs(reinterpret_cast<float4*>(dst), make_float4(v[i][0], v[i][1], v[i][2], v[i][3]));
        __stcs(reinterpret_cast<float4*>(dst) + 1, make_float4(v[i][4], v[i][5], v[i][6], v[i][7]));
      }
    }
  }
}

}  // namespace ra
