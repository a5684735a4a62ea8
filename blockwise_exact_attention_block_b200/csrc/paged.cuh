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

// Every kernel of the paged cache is launched as a programmatic dependent of what
// precedes it on the stream and begins with this: the next one may be brought
// onto the SMs from here on, and nothing in global memory is read or written
// until all that precedes has completed and is visible.  Every thread of every
// CTA comes here, so a grid's completion implies that of the grids before it.
__device__ __forceinline__ void chain_launches() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

struct PagedBatch {
  const int* page_table;  // [B][max_pages]
  const int* seq_lens;    // [B]
  const int* new_lens;    // [B] or null
  int B, T, max_pages, n_pages, Hkv;
  int page_shift;  // log2(page_size)
#ifdef RA_DEBUG_BOUNDS
  long long inject;  // added to an index where it is checked, not where it is used (a test's)
#endif
};
#ifdef RA_DEBUG_BOUNDS
#define PG_INJECTED(bt) ((bt).inject)
#else
#define PG_INJECTED(bt) 0
#endif

// Extents of the arrays, for the checked build: table entries, cached rows of all heads.
__device__ __forceinline__ long long table_extent(const PagedBatch& a) { return static_cast<long long>(a.B) * a.max_pages; }
__device__ __forceinline__ long long row_extent(const PagedBatch& a) {
  return (static_cast<long long>(a.n_pages) * a.Hkv) << a.page_shift;
}

// Tokens of sequence b and how many of its T rows are real, held to their ranges.
struct SeqLen {
  int len, fresh;
};

__device__ __forceinline__ SeqLen seq_len_of(const PagedBatch& a, int b) {
  SeqLen s;
  if (!RA_IN_BOUNDS(b, a.B)) return {0, 0};
  s.len = a.seq_lens[b];
  const int given = a.new_lens ? a.new_lens[b] : 0;  // (both loads before the first check)
  const int cap = a.max_pages << a.page_shift;
  if (s.len < 0 || s.len > cap) {
    set_status(RA_ERR_DEVICE_BOUNDS);
    s.len = min(max(s.len, 0), cap);
  }
  const int most = min(a.T, s.len);
  s.fresh = a.new_lens ? given : most;
  if (s.fresh < 0 || s.fresh > most) {
    set_status(RA_ERR_DEVICE_BOUNDS);
    s.fresh = min(max(s.fresh, 0), most);
  }
  return s;
}

// Page `logical` (below the sequence's page count) of sequence b; -1, recorded,
// when the table holds no valid page there.
__device__ __forceinline__ int page_of(const PagedBatch& a, int b, int logical) {
  const long long at = static_cast<long long>(b) * a.max_pages + logical;
  if (!RA_IN_BOUNDS(logical, a.max_pages) || !RA_IN_BOUNDS(at, table_extent(a))) return -1;
  const int p = a.page_table[at];
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

__device__ __forceinline__ uint32_t e4m3_quad(uint64_t lo, uint64_t hi) {  // codes of two fp32 pairs
  float2 l, h;
  f2_unpack(lo, l.x, l.y);
  f2_unpack(hi, h.x, h.y);
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\tcvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n\t"
      "mov.b32 %0, {l, h};\n\t}"
      : "=r"(r)
      : "f"(l.x), "f"(l.y), "f"(h.x), "f"(h.y));
  return r;
}

// An 8-bit row's scale s = fp32(a / m), a its largest magnitude and m = 127 or 448,
// and the factor `inv` with which quant_octet finds the code nearest to x / s for
// every value x of the row, although s is rounded and so is x * inv.
//
// x and a have 8 significant bits.  x m / a, the quotient were s not rounded, is
// then either exactly on a border between two codes (k + 1/2 for int8, 5 bits for
// e4m3) or at least 2^-16 (int8: 254 |x| against an 8-bit odd number times a, both
// integers of at most 64770) or 2^-13 (e4m3) of itself away from any.  x / s differs
// from it by 2^-24 of itself, which way is the same for the whole row.  So:
//   s too small (x / s beyond x m / a): inv is 1 / s made larger by 2^-18, too large:
//   smaller.  That is more than the errors of inv and of the product, so a value on
//   a border goes to its side, and too little to carry any other over a border.
//   s exact, m = 127: then a's 8 bits are 254 and s is a power of two, and so is inv;
//   the product is exact and a border goes to the even code by itself.
//   s exact, m = 448 (a divisible by 7): inv is 1 / s to a few ulp and quant_octet
//   rounds the product to 16 bits, which a border's 5 survive (`snap`).
struct RowScale {
  float s, inv;
  bool snap;
};

// fp32(a / m) for a >= 2^-100 by the division with a divisor known in advance of
// Brisebarre, Muller and Raina (IEEE Trans. Computers 2004): the product with the
// rounded 1 / m, its exact remainder, and the remainder's product added back.  That it
// is the correctly rounded quotient for every such a is checked value by value in
// the tests, and so are the codes of every x for every a.
template <int ET>
__device__ __forceinline__ RowScale scale_of(float a) {
  constexpr float m = ET == kCacheI8 ? 127.f : 448.f, r = static_cast<float>(1.0 / m);
  RowScale o;
  const float q = a * r;
  o.s = fmaf(fmaf(-q, m, a), r, q);
  const float rest = fmaf(-o.s, m, a);  // exact: positive when s is too small
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(o.inv) : "f"(o.s));
  o.snap = rest == 0.f;
  if (!o.snap) o.inv *= rest > 0.f ? 1.f + 0x1p-18f : 1.f - 0x1p-18f;
  return o;
}

// An fp32 value's bits rounded to 16 significant ones.
__device__ __forceinline__ float to_16_bits(uint32_t x) { return __uint_as_float((x + 0x80u) & 0xffffff00u); }

// Eight bf16 values (pairs in u) of a row as codes: see RowScale.  int8: x * inv +
// 1.5 2^23 in one fma rounds the product to the integer in the sum's low bits (the
// conversion instructions run at a quarter of the fma rate).
template <int ET>
__device__ __forceinline__ uint2 quant_octet(const uint32_t (&u)[4], const RowScale& rs) {
  const uint64_t inv = f2_pack(rs.inv, rs.inv);
  uint64_t x[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = f2_pack(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xffff0000u));
  uint32_t c[2];
  if constexpr (ET == kCacheI8) {
    const uint64_t magic = f2_pack(12582912.f, 12582912.f);
    uint32_t y[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint64_t t = f2_fma(x[i], inv, magic);
      y[2 * i] = static_cast<uint32_t>(t);
      y[2 * i + 1] = static_cast<uint32_t>(t >> 32);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
      c[i] = __byte_perm(__byte_perm(y[4 * i], y[4 * i + 1], 0x0040), __byte_perm(y[4 * i + 2], y[4 * i + 3], 0x0040), 0x5410);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = f2_mul(x[i], inv);
    if (rs.snap)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        x[i] = f2_pack(to_16_bits(static_cast<uint32_t>(x[i])), to_16_bits(static_cast<uint32_t>(x[i] >> 32)));
#pragma unroll
    for (int i = 0; i < 2; ++i) c[i] = e4m3_quad(x[2 * i], x[2 * i + 1]);
  }
  return make_uint2(c[0], c[1]);
}

// Eight bf16 values as fp32.
__device__ __forceinline__ void bf16_octet(const __nv_bfloat16* p, float (&v)[8]) {
  const uint4 w = *reinterpret_cast<const uint4*>(p);
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(u[i] << 16);
    v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}

// Of pairs; a NaN yields to the other operand.
__device__ __forceinline__ uint32_t bf16x2_min(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t bf16x2_max(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
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

constexpr int kAppendThreads = 128;  // (256: 35.2 us for 24,000 int8 tokens of 8 heads, against 34)
constexpr int kAppendBatch = 2;  // rows of K and V a lane holds in flight

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
    const float largest = __uint_as_float(am << 16);
    const RowScale rs = scale_of<ET>(largest);
    uint2 code = quant_octet<ET>(u, rs);
    float s = rs.s;
    if (!(largest >= 0x1p-100f && largest < INFINITY)) {  // too small, or NaN: then the row reads back as NaN
      s = largest < 1.f ? 0.f : __uint_as_float(0x7fc00000u);
      code = make_uint2(0u, 0u);
    }
    if (act) {
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(pages) + row * D + 8 * lane_in_row) = code;
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
__global__ void __launch_bounds__(kAppendThreads, 8) cache_append_kernel(const __grid_constant__ AppendArgs a) {
  constexpr int LPR = D / 8, RPW = 32 / LPR;
  __shared__ uint32_t s_lo[kAppendThreads / 32][D / 2], s_hi[kAppendThreads / 32][D / 2];
  chain_launches();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane / LPR, lr = lane % LPR;
  const int upc = (kAppendThreads / 32) / a.wpu, wi = warp % a.wpu;  // units per CTA, warp in the unit
  const long long unit = static_cast<long long>(blockIdx.x) * upc + warp / a.wpu;
  int page = -1, r0 = 0, r1 = 0, h = 0, b = 0, tok0 = 0;
  bool good = false;  // rows to write, and a page for them
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
      // (not looked at before the first rows are on their way: the loads overlap)
      if (RA_IN_BOUNDS(logical, a.bt.max_pages)) page = a.bt.page_table[static_cast<long long>(b) * a.bt.max_pages + logical];
      r0 = max(begin - static_cast<int>(first), 0);
      r1 = min(s.len - static_cast<int>(first), ps);
      tok0 = static_cast<int>(first) - begin;  // token of the page's row 0 (may be negative)
    }
  }
  // pairs of columns; min and max of bf16 pass over a NaN
  uint32_t lo[4] = {0x7f807f80u, 0x7f807f80u, 0x7f807f80u, 0x7f807f80u};
  uint32_t hi[4] = {0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u};
  if (r0 < r1) {
    const int step = a.wpu * RPW;
    for (int rb = r0 + wi * RPW; rb < r1; rb += step * kAppendBatch) {
      uint4 kw[kAppendBatch], vw[kAppendBatch];
#pragma unroll
      for (int u = 0; u < kAppendBatch; ++u) {
        const int r = rb + u * step + sub;
        kw[u] = vw[u] = make_uint4(0u, 0u, 0u, 0u);
        if (r < r1 && RA_IN_BOUNDS(tok0 + r, a.bt.T) && RA_IN_BOUNDS(b, a.bt.B)) {
          const long long src = ((static_cast<long long>(b) * a.bt.T + tok0 + r) * a.bt.Hkv + h) * D + 8 * lr;
          kw[u] = __ldcs(reinterpret_cast<const uint4*>(a.k + src));
          vw[u] = __ldcs(reinterpret_cast<const uint4*>(a.v + src));
        }
      }
      good = page >= 0 && page < a.bt.n_pages;
      const long long prow = (static_cast<long long>(page) * a.bt.Hkv + h) << a.bt.page_shift;
#pragma unroll
      for (int u = 0; u < kAppendBatch; ++u) {
        if (rb + u * step >= r1) break;  // the same for the whole warp
        const int r = rb + u * step + sub;
        const bool act = r < r1 && good && RA_IN_BOUNDS(prow + r + PG_INJECTED(a.bt), row_extent(a.bt));
        append_row<D, ET>(kw[u], act, lr, a.k_pages, a.k_scales, prow + r);
        append_row<D, ET>(vw[u], act, lr, a.v_pages, a.v_scales, prow + r);
        if (a.bounds && act) {
          const uint32_t w[4] = {kw[u].x, kw[u].y, kw[u].z, kw[u].w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            lo[i] = bf16x2_min(lo[i], w[i]);
            hi[i] = bf16x2_max(hi[i], w[i]);
          }
        }
      }
    }
  }
  if (r0 < r1 && wi == 0 && lane == 0 && !good) set_status(RA_ERR_DEVICE_BOUNDS);
  if (a.bounds == nullptr) return;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int o = LPR; o < 32; o <<= 1) {
      lo[i] = bf16x2_min(lo[i], __shfl_xor_sync(0xffffffffu, lo[i], o));
      hi[i] = bf16x2_max(hi[i], __shfl_xor_sync(0xffffffffu, hi[i], o));
    }
  if (a.wpu > 1) {
    if (sub == 0)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s_lo[warp][4 * lr + i] = lo[i];
        s_hi[warp][4 * lr + i] = hi[i];
      }
    __syncthreads();
    if (wi == 0)
      for (int w = 1; w < a.wpu; ++w)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          lo[i] = bf16x2_min(lo[i], s_lo[warp + w][4 * lr + i]);
          hi[i] = bf16x2_max(hi[i], s_hi[warp + w][4 * lr + i]);
        }
  }
  if (!good || wi != 0 || sub != 0) return;
  if (!RA_IN_BOUNDS(static_cast<long long>(page) * a.bt.Hkv + h, static_cast<long long>(a.bt.n_pages) * a.bt.Hkv)) return;
  uint4* bl = reinterpret_cast<uint4*>(a.bounds + (static_cast<long long>(page) * a.bt.Hkv + h) * 2 * D) + lr;
  if (r0 > 0) {  // earlier tokens' bounds stand in the page
    const uint4 x = bl[0], y = bl[D / 8];
    const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      lo[i] = bf16x2_min(lo[i], xs[i]);
      hi[i] = bf16x2_max(hi[i], ys[i]);
    }
  }
  bl[0] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  bl[D / 8] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
}

// --------------------------------------------------------------------- read

struct ReadArgs {
  PagedBatch bt;  // T = rows of the output
  int first;
  const void* pages[2];    // K, V
  const float* scales[2];
  void* out[2];            // null: not asked for
  int groups;              // groups of read_rows(D) rows of T
  long long units;         // B * groups * Hkv
};

constexpr int kReadThreads = 128;
// Output rows of a warp: 1,024 values of K and of V.  Small CTAs of short warps keep
// loads and stores mixed on every SM (4 x 24,000 int8 tokens of 8 heads to bf16: 16 rows
// in CTAs of 256 threads 98 us, of 128 90; 8 rows in 128 87, 95 % of the copy rate).
__host__ __device__ constexpr int read_rows(int D) { return 1024 / D; }

// One row's octet of a lane as it is stored, with its scale, and as fp32 values.
template <int ET>
struct Octet {
  uint4 w;  // (8-bit codes: x and y)
  float scale;
};
template <int ET>
__device__ __forceinline__ Octet<ET> load_octet(const void* pages, const float* scales, long long row, int D, int col) {
  Octet<ET> o;
  o.w = make_uint4(0u, 0u, 0u, 0u);
  o.scale = 0.f;
  if (row < 0) return o;
  if constexpr (ET == kCacheBf16) {
    o.w = __ldcs(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(pages) + row * D + col));
  } else {
    const uint2 c = __ldcs(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(pages) + row * D + col));
    o.w.x = c.x;
    o.w.y = c.y;
    o.scale = scales[row];
  }
  return o;
}
template <int ET>
__device__ __forceinline__ void octet_values(const Octet<ET>& o, float (&v)[8]) {
  if constexpr (ET == kCacheBf16) {
    const uint32_t u[4] = {o.w.x, o.w.y, o.w.z, o.w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(u[i] << 16);
      v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  } else {
    const uint32_t u[2] = {o.w.x, o.w.y};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (ET == kCacheI8) {
        // 2^23 + 128 + code as an fp32's bits (the byte with its sign flipped), less 2^23 + 128
        const uint32_t c = __byte_perm(u[i >> 2] ^ 0x80808080u, 0x4b000000u, 0x7650 + (i & 3));
        v[i] = (__uint_as_float(c) - 8388736.f) * o.scale;
      } else {
        const uint32_t c = (u[i >> 2] >> (8 * (i & 3))) & 0xffu;
        v[i] = __uint_as_float(__float_as_uint(e4m3_value(c & 0x7fu)) | ((c & 0x80u) << 24)) * o.scale;
      }
    }
  }
}

// A warp takes consecutive tokens of one KV head (rows of a page side by side to
// read, heads side by side in the CTA to write); D / 8 lanes hold a row.  Keys and
// values of all its tokens are loaded before the first is written.
template <int D, int ET, typename Tout>
__global__ void __launch_bounds__(kReadThreads) cache_read_kernel(const __grid_constant__ ReadArgs a) {
  constexpr int LPR = D / 8, RPW = 32 / LPR, kRows = read_rows(D), N = kRows / RPW;
  chain_launches();
  const int lane = threadIdx.x & 31;
  const int sub = lane / LPR, lr = lane % LPR;
  const long long unit = static_cast<long long>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (unit >= a.units) return;
  const int h = static_cast<int>(unit % a.bt.Hkv);
  const long long bg = unit / a.bt.Hkv;
  const int g = static_cast<int>(bg % a.groups), b = static_cast<int>(bg / a.groups);
  const int t0 = g * kRows;
  // lane i < kRows: the cache row of output row t0 + i, -1 where there is none.  The
  // table entry is loaded beside the length that says whether it counts.
  const long long pos = static_cast<long long>(a.first) + t0 + (lane & (kRows - 1));
  const long long logical = min(pos >> a.bt.page_shift, static_cast<long long>(a.bt.max_pages - 1));
  const long long entry = static_cast<long long>(b) * a.bt.max_pages + logical;
  const int page = RA_IN_BOUNDS(entry, table_extent(a.bt)) ? a.bt.page_table[entry] : -1;
  const int len = seq_len_of(a.bt, b).len;
  long long mine = -1;
  if (lane < kRows && pos < len) {
    if (page >= 0 && page < a.bt.n_pages)
      mine = ((static_cast<long long>(page) * a.bt.Hkv + h) << a.bt.page_shift) + (pos & ((1 << a.bt.page_shift) - 1));
    else
      set_status(RA_ERR_DEVICE_BOUNDS);
    if (mine >= 0 && !RA_IN_BOUNDS(mine + PG_INJECTED(a.bt), row_extent(a.bt))) mine = -1;
  }
  Octet<ET> o[2][N];
#pragma unroll
  for (int kv = 0; kv < 2; ++kv)
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const long long row = __shfl_sync(0xffffffffu, mine, i * RPW + sub);
      o[kv][i] = load_octet<ET>(a.pages[kv], a.scales[kv], a.out[kv] ? row : -1, D, 8 * lr);
    }
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    if (a.out[kv] == nullptr) continue;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int t = t0 + i * RPW + sub;
      if (t >= a.bt.T || !RA_IN_BOUNDS(b, a.bt.B)) continue;
      Tout* dst = static_cast<Tout*>(a.out[kv]) + ((static_cast<long long>(b) * a.bt.T + t) * a.bt.Hkv + h) * D + 8 * lr;
      if constexpr (sizeof(Tout) == 2 && ET == kCacheBf16) {
        __stcs(reinterpret_cast<uint4*>(dst), o[kv][i].w);
      } else {
        float v[8];
        octet_values<ET>(o[kv][i], v);
        if constexpr (sizeof(Tout) == 2) {
          __stcs(reinterpret_cast<uint4*>(dst),
                 make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])));
        } else {
          __stcs(reinterpret_cast<float4*>(dst), make_float4(v[0], v[1], v[2], v[3]));
          __stcs(reinterpret_cast<float4*>(dst) + 1, make_float4(v[4], v[5], v[6], v[7]));
        }
      }
    }
  }
}

}  // namespace ra
