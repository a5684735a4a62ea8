// page_select.cuh - the pages of a paged cache worth attending to: a score for
// each (sequence, KV head, page) from the page's key bounds, and the n_sel best.
//
// Mathematics: with lo, hi the columnwise minimum and maximum of a page's keys,
//     q . k <= sum_d max(q_d lo_d, q_d hi_d) = sum_d (min(q_d, 0) lo_d + max(q_d, 0) hi_d)
// for every key k of the page, so the sum bounds every score in the page.  A KV
// head's pages are ranked by the largest bound over its query rows; ties go to
// the lower page.  The pages that hold the step's new tokens come first whatever
// their score.
//
// Which pages win is a comparison, so it must not depend on the order of a
// sum: it is that of the sums in 64 bits, where products of bf16 values (16
// bits) and their sums are exact unless the terms' exponents differ by more
// than 30.  But 64-bit sums of every page cost more than reading the bounds
// (25 us by themselves, where scores and selection take 17.5 together: eight
// sequences of 2k to 24k keys, pages of 16, 8 heads, 4 rows), and few pages are
// close to the border.  So: scores of all
// pages from the tensor core in fp32 with a bound on their error; the n_sel-th
// largest of them; and 64-bit sums for the pages within the error of it.
#pragma once

#include "paged.cuh"
#include "paged_decode.cuh"

namespace ra {

struct SelectArgs {
  PagedBatch bt;  // T = Tq
  int Hq, groups, rows, n_sel;
  long long stride;             // slots of one (sequence, KV head): max_pages rounded up to 16
  const __nv_bfloat16* q;       // [B][Tq][Hq][D]
  const __nv_bfloat16* bounds;  // [n_pages][Hkv][2][D]
  // [B * Hkv][stride]: fp32 scores of the pages, then of every 16 the largest and a bound on
  // their errors; or the pages' exact keys
  unsigned long long* slots;
  int* selected;                // [B][Hkv][n_sel]
};

// Order-preserving integers of a score; a NaN ranks as -infinity.
__device__ __forceinline__ unsigned long long score_key(double s) {
  if (!(s == s)) s = -INFINITY;
  const unsigned long long b = static_cast<unsigned long long>(__double_as_longlong(s));
  return (b >> 63) ? ~b : b | (1ull << 63);
}
__device__ __forceinline__ uint32_t score_key(float s) {
  if (!(s == s)) s = -INFINITY;
  const uint32_t b = __float_as_uint(s);
  return (b >> 31) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_score(uint32_t k) { return __uint_as_float((k >> 31) ? k & 0x7fffffffu : ~k); }

// First page that holds a new token, or the page count when there is none.
__device__ __forceinline__ int first_new_page(const SeqLen& s, int shift) {
  const int pages = (s.len + (1 << shift) - 1) >> shift;
  return s.fresh > 0 ? (s.len - s.fresh) >> shift : pages;
}

// Query row `row` (of the real ones) of sequence b and KV head h.
__device__ __forceinline__ const __nv_bfloat16* select_row(const SelectArgs& a, int b, int h, int row, int D) {
  return a.q + ((static_cast<long long>(b) * a.bt.T + row / a.groups) * a.Hq + h * a.groups + row % a.groups) * D;
}

constexpr int kScoreThreads = 128;
// Bound on the error of an fp32 score, relative to A = sum_d |q_d| max(|lo_d|,
// |hi_d|), which is at least the sum of its terms' magnitudes: 2 D <= 256 exact
// products, added by the tensor core in fp32 with additions that may cut instead
// of round, 2^-23 of A for each, is 2^-15 A; A itself comes from the same
// products and is short by no more than that part of it.
constexpr float kScoreError = 0x1.01p-15f;

// Grid (page blocks, Hkv, B), striding over the pages that there are; a warp takes
// 16 pages at a time, the M side of mma.m16n8k16,
// with up to 8 query rows at a time on the N side and the 2 D columns (lo, then
// hi) as K.  A lane reads its pages' bounds as whole 16-byte chunks qd + 4 j and
// uses them as the K columns of two steps, with the query in the same order.
// Bound by the bounds' bytes.
template <int D>
__global__ void __launch_bounds__(kScoreThreads) page_score_kernel(const __grid_constant__ SelectArgs a) {
  constexpr int J = D / 32;  // 16-byte chunks of a lane in lo, and in hi
  const int b = blockIdx.z, h = blockIdx.y, lane = threadIdx.x & 31;
  const int gr = lane >> 2, qd = lane & 3;
  chain_launches();
  for (int p0 = (blockIdx.x * (kScoreThreads / 32) + (threadIdx.x >> 5)) * 16; p0 < a.bt.max_pages;
       p0 += gridDim.x * (kScoreThreads / 32) * 16) {
    // lengths, table and queries are loaded side by side; the lengths say afterwards what counts
    const int raw = lane < 16 && p0 + lane < a.bt.max_pages
                        ? a.bt.page_table[static_cast<long long>(b) * a.bt.max_pages + p0 + lane]
                        : 0;
    uint4 q0[J];
#pragma unroll
    for (int j = 0; j < J; ++j)
      q0[j] = gr < a.rows ? *(reinterpret_cast<const uint4*>(select_row(a, b, h, gr, D)) + qd + 4 * j) : make_uint4(0u, 0u, 0u, 0u);
    const SeqLen s = seq_len_of(a.bt, b);
    const int count = first_new_page(s, a.bt.page_shift);  // the others need no score
    if (p0 >= count) return;
    const bool bad = lane < 16 && p0 + lane < count && (raw < 0 || raw >= a.bt.n_pages);
    if (bad) set_status(RA_ERR_DEVICE_BOUNDS);
    const int mine = bad || p0 + lane >= count ? -1 : raw;  // (a slot without a page has bounds of 0: nothing counts there)
    const int real = s.fresh * a.groups;                   // rows of real tokens come first
    if (gr >= real)
#pragma unroll
      for (int j = 0; j < J; ++j) q0[j] = make_uint4(0u, 0u, 0u, 0u);  // (padding may hold anything)
    if (!RA_IN_BOUNDS(b, a.bt.B) || !RA_IN_BOUNDS(p0 + 15, a.stride)) return;
    uint32_t lo[2][J][4], hi[2][J][4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {  // pages gr and gr + 8
      int page = __shfl_sync(0xffffffffu, mine, gr + 8 * i);
      if (page >= 0 && !RA_IN_BOUNDS(page + PG_INJECTED(a.bt), a.bt.n_pages)) page = -1;
      const uint4* src =
          reinterpret_cast<const uint4*>(a.bounds + (static_cast<long long>(max(page, 0)) * a.bt.Hkv + h) * 2 * D) + qd;
#pragma unroll
      for (int j = 0; j < J; ++j) {
        uint4 x = src[4 * j], y = src[D / 8 + 4 * j];
        if (page < 0) x = y = make_uint4(0u, 0u, 0u, 0u);
        lo[i][j][0] = x.x, lo[i][j][1] = x.y, lo[i][j][2] = x.z, lo[i][j][3] = x.w;
        hi[i][j][0] = y.x, hi[i][j][1] = y.y, hi[i][j][2] = y.z, hi[i][j][3] = y.w;
      }
    }
    uint32_t bmax = 0, qmax = 0;  // largest magnitudes, as pairs of bf16 bits
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          // the smaller and the larger of the two, whatever the caller's order
          const uint32_t x = lo[i][j][w], y = hi[i][j][w];
          lo[i][j][w] = bf16x2_min(x, y);
          hi[i][j][w] = bf16x2_max(x, y);
        }
    float best[2] = {-INFINITY, -INFINITY}, err[2] = {0.f, 0.f};
    for (int r0 = 0; r0 < real; r0 += 8) {
      if (r0 > 0)
#pragma unroll
        for (int j = 0; j < J; ++j)
          q0[j] = r0 + gr < real ? *(reinterpret_cast<const uint4*>(select_row(a, b, h, r0 + gr, D)) + qd + 4 * j)
                                 : make_uint4(0u, 0u, 0u, 0u);
      float c[4] = {0.f, 0.f, 0.f, 0.f}, m[4] = {0.f, 0.f, 0.f, 0.f};  // scores, and their terms' magnitudes
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const uint32_t w[4] = {q0[j].x, q0[j].y, q0[j].z, q0[j].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) qmax = __vmaxu2(qmax, w[i] & 0x7fff7fffu);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const uint32_t al[4] = {lo[0][j][2 * t], lo[1][j][2 * t], lo[0][j][2 * t + 1], lo[1][j][2 * t + 1]};
          const uint32_t ah[4] = {hi[0][j][2 * t], hi[1][j][2 * t], hi[0][j][2 * t + 1], hi[1][j][2 * t + 1]};
          uint32_t aa[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            aa[i] = bf16x2_max(al[i] & 0x7fff7fffu, ah[i] & 0x7fff7fffu);
            bmax = __vmaxu2(bmax, aa[i]);
          }
          pg_mma<kCacheBf16>(c, al, bf16x2_min(w[2 * t], 0u), bf16x2_min(w[2 * t + 1], 0u));
          pg_mma<kCacheBf16>(c, ah, bf16x2_max(w[2 * t], 0u), bf16x2_max(w[2 * t + 1], 0u));
          pg_mma<kCacheBf16>(m, aa, w[2 * t] & 0x7fff7fffu, w[2 * t + 1] & 0x7fff7fffu);
        }
      }
      // c[2 i + e], m[2 i + e]: page gr + 8 i, row r0 + 2 qd + e
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (r0 + 2 * qd + e < real) {
            best[i] = fmaxf(best[i], c[2 * i + e]);
            // magnitudes that are not finite (an overflow) leave the pages to the exact sums
            err[i] = m[2 * i + e] < 3e38f ? fmaxf(err[i], m[2 * i + e]) : INFINITY;
          }
    }
    uint32_t big = max(max(bmax & 0xffffu, bmax >> 16), max(qmax & 0xffffu, qmax >> 16));
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) big = max(big, __shfl_xor_sync(0xffffffffu, big, x));
    // Should the tensor core flush subnormal operands, products or sums: 256 terms
    // of at most 2^-126 times the largest operand, or 2^-126.  Infinite and NaN
    // operands leave the warp's pages to the exact sums.
    const float floor_err = big >= 0x7f80u ? INFINITY : 0x1p-110f * fmaxf(__uint_as_float(big << 16), 1.f);
    float* scores = reinterpret_cast<float*>(a.slots + (static_cast<long long>(b) * a.bt.Hkv + h) * a.stride);
    float e = fmaxf(err[0], err[1]), all = -INFINITY;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int x = 1; x < 4; x <<= 1) best[i] = fmaxf(best[i], __shfl_xor_sync(0xffffffffu, best[i], x));
      const int p = p0 + gr + 8 * i;
      if (__shfl_sync(0xffffffffu, static_cast<int>(bad), gr + 8 * i) || p >= count) best[i] = -INFINITY;
      if (qd == 0) scores[p] = best[i];  // (the stride is a multiple of 16)
      all = fmaxf(all, best[i]);
    }
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) {
      e = fmaxf(e, __shfl_xor_sync(0xffffffffu, e, x));
      all = fmaxf(all, __shfl_xor_sync(0xffffffffu, all, x));
    }
    if (lane == 0) {
      scores[a.stride + p0 / 16] = all;
      scores[a.stride + a.stride / 16 + p0 / 16] = real > 0 ? fmaf(kScoreError, e, floor_err) : 0.f;
    }
  }
}

// A bf16 bound as a double's high word: its 15 magnitude bits moved into the
// double's exponent and mantissa fields give the value times 2^-896 (also for
// subnormal bounds; an infinity becomes 2^128, so that 0 times it is 0), and the
// query, widened the ordinary way and multiplied by 2^896, carries the factor back.
__device__ __forceinline__ double bound_times(double q, float x) {
  const uint32_t b = __float_as_uint(x);
  return q * __hiloint2double(static_cast<int>(((b & 0x7fff0000u) >> 3) | (b & 0x80000000u)), 0);
}

// The exact key of a page: D / 8 lanes (`lr` of them this one) hold 8 columns
// each; every lane of the warp calls it, with the same number of rows.
template <int D>
__device__ __forceinline__ unsigned long long exact_key(const SelectArgs& a, int b, int h, int page, int real, int lr) {
  if (!RA_IN_BOUNDS(page, a.bt.n_pages)) page = 0;
  const __nv_bfloat16* bl = a.bounds + (static_cast<long long>(page) * a.bt.Hkv + h) * 2 * D + 8 * lr;
  float lo[8], hi[8];
  bf16_octet(bl, lo);
  bf16_octet(bl + D, hi);
  double best = -INFINITY;
#pragma unroll 4
  for (int r = 0; r < real; ++r) {
    float q[8];
    bf16_octet(select_row(a, b, h, r, D) + 8 * lr, q);
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      sum += bound_times(static_cast<double>(q[i]) * 0x1p896, q[i] < 0.f ? fminf(lo[i], hi[i]) : fmaxf(lo[i], hi[i]));
#pragma unroll
    for (int o = D / 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (sum > best) best = sum;  // a NaN does not count
  }
  return score_key(best);
}

constexpr int kSelThreads = 512;  // (1024: 42.2 us against 40.7 for selection and attention of 8 sequences of 2k - 24k keys; 256: 42.9)
constexpr int kSelBits = 11;
constexpr int kSelBins = 1 << kSelBits;
constexpr int kSelFew = 64;     // keys ranked outright
constexpr int kSelClose = 512;  // pages whose exact keys are compared in shared memory
constexpr int kSelList = 2816;   // pages that can be held there as candidates

// Exclusive sum over the block (whole block).
__device__ __forceinline__ unsigned long long block_scan(unsigned long long x, unsigned long long* s_warp) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  unsigned long long upto = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long y = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += y;
  }
  __syncthreads();
  if (lane == 31) s_warp[warp] = upto;
  __syncthreads();
  if (warp == 0) {
    unsigned long long w = lane < kSelThreads / 32 ? s_warp[lane] : 0ull, v = w;
#pragma unroll
    for (int o = 1; o < kSelThreads / 32; o <<= 1) {
      const unsigned long long y = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += y;
    }
    if (lane < kSelThreads / 32) s_warp[lane] = v - w;
  }
  __syncthreads();
  return s_warp[warp] + upto - x;
}

struct SelectShared {
  unsigned int hist[kSelBins];
  unsigned long long warp[32], lows[32], highs[32], found, few[kSelFew];
  int nfew, digit, above, at;
  int err;                          // an error bound's bits
  unsigned long long close[kSelClose];
  int close_at[kSelClose];
  uint32_t list_key[kSelList];
  int list_page[kSelList];
};

// The want-th largest of the keys that each(fn) passes to fn in every thread, 1 <=
// want <= their number: a histogram over 11 bits from the highest in which the
// keys differ at all, and the bin in which the count from the top reaches
// `want`; a bin of at most kSelFew keys is ranked outright, a larger one (close
// scores, ties) is split by its next 11 bits.  `above` becomes how many keys are
// larger.  Whole block.
template <typename Key, typename Each>
__device__ __forceinline__ Key kth_largest(SelectShared& sh, Each&& each, int want, int& above) {
  constexpr int kWidth = 8 * sizeof(Key);
  const int tid = threadIdx.x;
  Key lo = static_cast<Key>(~static_cast<Key>(0)), hi = 0;
  each([&](Key k) {
    lo = min(lo, k);
    hi = max(hi, k);
  });
  if constexpr (kWidth == 32) {
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
  } else {
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      lo = min(lo, __shfl_xor_sync(0xffffffffu, lo, o));
      hi = max(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
  }
  if ((tid & 31) == 0) {
    sh.lows[tid >> 5] = lo;
    sh.highs[tid >> 5] = hi;
  }
  for (int i = tid; i < kSelBins; i += kSelThreads) sh.hist[i] = 0u;
  __syncthreads();
  lo = static_cast<Key>(sh.lows[tid % (kSelThreads / 32)]);
  hi = static_cast<Key>(sh.highs[tid % (kSelThreads / 32)]);
  if constexpr (kWidth == 32) {
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
  } else {
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      lo = min(lo, __shfl_xor_sync(0xffffffffu, lo, o));
      hi = max(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
  }
  Key top = hi;
  // the same in all keys from bit `low` up
  int low = lo == hi ? 0 : 64 - __clzll(static_cast<long long>(static_cast<unsigned long long>(lo ^ hi)));
  above = 0;
  while (low > 0) {
    const int next = max(low - kSelBits, 0), width = low - next;
    each([&](Key k) {
      if (low == kWidth || (k >> low) == (top >> low)) atomicAdd(&sh.hist[(k >> next) & ((1u << width) - 1u)], 1u);
    });
    if (tid == 0) sh.nfew = 0;
    __syncthreads();
    // a few bins a thread, from the top: the digit in which the running count reaches `want`
    constexpr int kBins = kSelBins / kSelThreads;
    const int d0 = kSelBins - 1 - kBins * tid;
    unsigned int c[kBins], sum = 0;
#pragma unroll
    for (int i = 0; i < kBins; ++i) {
      c[i] = sh.hist[d0 - i];
      sh.hist[d0 - i] = 0u;  // (for the next pass)
      sum += c[i];
    }
    int before = above + static_cast<int>(block_scan(sum, sh.warp));
    if (before < want && before + static_cast<int>(sum) >= want) {
#pragma unroll
      for (int i = 0; i < kBins; ++i) {
        if (before < want && before + static_cast<int>(c[i]) >= want) {
          sh.digit = d0 - i;
          sh.above = before;
          sh.at = static_cast<int>(c[i]);
        }
        before += static_cast<int>(c[i]);
      }
    }
    __syncthreads();
    const Key keep = low == kWidth ? 0 : (top >> low) << low;
    top = keep | (static_cast<Key>(sh.digit) << next);
    above = sh.above;
    low = next;
    const int at = sh.at;
    if (low > 0 && at <= kSelFew) {
      each([&](Key k) {
        if ((k >> low) == (top >> low)) sh.few[atomicAdd(&sh.nfew, 1)] = k;
      });
      __syncthreads();
      if (tid < at) {
        const unsigned long long k = sh.few[tid];
        int more = 0, upto = 0;
        for (int j = 0; j < at; ++j) {
          more += sh.few[j] > k;
          upto += sh.few[j] >= k;
        }
        if (above + more < want && want <= above + upto) {  // (equal keys write the same)
          sh.found = k;
          sh.above = above + more;
        }
      }
      __syncthreads();
      top = static_cast<Key>(sh.found);
      above = sh.above;
      low = 0;
    }
    __syncthreads();  // the shared results have been read
  }
  return top;
}

// One CTA per (sequence, KV head).  The new tokens' pages are in; `want` of the n
// scored pages are chosen.
//  - Candidates, of many pages: the want-th largest of the maxima of 16 pages each
//    has at least `want` scores at or above it, so no page more than two errors
//    below it can win; the rest are listed in shared memory.
//  - With T the want-th largest fp32 score and err the largest error of any, a page
//    above T + 2 err is in and one below T - 2 err is out (the want-th largest exact
//    score lies within err of T); those between, usually a handful, are ranked by
//    their exact keys, ties to the lower page.
//  - The chosen indices come out in page order.
// Where the pages are few or the candidates too many for the list, the same passes
// read all scores from memory; where many are close (equal or infinite scores), every page gets
// its exact key and the search runs on those.
template <int D>
__global__ void __launch_bounds__(kSelThreads) page_select_kernel(const __grid_constant__ SelectArgs a) {
  __shared__ SelectShared sh;
  chain_launches();
  constexpr int L = D / 8, G = 32 / L;  // lanes of a page in an exact sum, pages side by side
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.x / a.bt.Hkv, h = blockIdx.x % a.bt.Hkv;
  int* out = a.selected + static_cast<long long>(blockIdx.x) * a.n_sel;
  const SeqLen s = seq_len_of(a.bt, b);
  const int shift = a.bt.page_shift;
  const int pages = (s.len + (1 << shift) - 1) >> shift;
  const int n = first_new_page(s, shift), real = s.fresh * a.groups;
  if (pages <= a.n_sel) {  // every page
    for (int i = tid; i < a.n_sel; i += kSelThreads) out[i] = i < pages ? i : -1;
    return;
  }
  const int want = a.n_sel - (pages - n);  // 0 <= want < n: the host checked n_sel against T
  for (int i = tid; i < a.n_sel - want; i += kSelThreads) out[want + i] = n + i;
  if (want == 0) return;
  unsigned long long* slots = a.slots + static_cast<long long>(blockIdx.x) * a.stride;
  const float* scores = reinterpret_cast<const float*>(slots);
  const float* tops = scores + a.stride;
  const int groups = (n + 15) / 16;
  float err = 0.f;
  for (int i = tid; i < groups; i += kSelThreads) err = fmaxf(err, tops[a.stride / 16 + i]);
  if (tid == 0) sh.err = 0;
  const int err_bits = __reduce_max_sync(0xffffffffu, __float_as_int(err));  // (not negative)
  __syncthreads();
  if (lane == 0) atomicMax(&sh.err, err_bits);
  __syncthreads();
  err = __int_as_float(sh.err);
  const float wide = 2.5f * err;  // a little more than 2 err, so that the rounding of sums with it does not matter
  bool many = !(err < 3e38f);     // infinite or NaN scores
  int above, N = n;               // items of the search: the list's, or all pages
  bool listed = false;
  if (!many && want <= groups && n > kSelList) {
    uint32_t least;  // key of the lowest score that can win
    {
      const uint32_t k = kth_largest<uint32_t>(
          sh,
          [&](auto&& fn) {
            for (int i = tid; i < groups; i += kSelThreads) fn(score_key(tops[i]));
          },
          want, above);
      least = score_key(key_score(k) - wide);
    }
    int have = 0;
    for (int p0 = 0; p0 < n && have <= kSelList; p0 += 16 * kSelThreads) {  // 16 pages a thread
      const int i0 = p0 + 16 * tid;
      uint32_t keys[16], picked = 0;
      if (i0 < n) {  // (the slots go on to a multiple of 16)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const float4 x = *reinterpret_cast<const float4*>(scores + i0 + 4 * v);
          keys[4 * v] = score_key(x.x);
          keys[4 * v + 1] = score_key(x.y);
          keys[4 * v + 2] = score_key(x.z);
          keys[4 * v + 3] = score_key(x.w);
        }
#pragma unroll
        for (int v = 0; v < 16; ++v) picked |= (i0 + v < n && keys[v] >= least ? 1u : 0u) << v;
      }
      const int mine = __popc(picked);
      int at = have + static_cast<int>(block_scan(mine, sh.warp));
      if (tid == kSelThreads - 1) sh.at = at + mine;
#pragma unroll
      for (int v = 0; v < 16; ++v)
        if ((picked >> v) & 1u) {
          if (at < kSelList) {
            sh.list_key[at] = keys[v];
            sh.list_page[at] = i0 + v;
          }
          ++at;
        }
      __syncthreads();
      have = sh.at;
    }
    listed = have <= kSelList;
    if (listed) N = have;
    __syncthreads();
  }
  auto key_of = [&](int i) { return listed ? sh.list_key[i] : score_key(scores[i]); };
  auto page_at = [&](int i) { return listed ? sh.list_page[i] : i; };
  // Items in page order: sort(item) says 1 or 2 for the two kinds that count, 0 for
  // others, and put(kind, item, ones before, twos before) is then called for
  // those (whole block).
  auto in_order = [&](auto&& sort, auto&& put) {
    const int per = (N + kSelThreads - 1) / kSelThreads, i0 = min(tid * per, N), i1 = min(i0 + per, N);
    unsigned long long count = 0;  // ones << 32 | twos
#pragma unroll 1
    for (int i = i0; i < i1; ++i) {
      const int kind = sort(i);
      count += kind == 1 ? 1ull << 32 : kind == 2 ? 1ull : 0ull;
    }
    count = block_scan(count, sh.warp);
    int ones = static_cast<int>(count >> 32), twos = static_cast<int>(count & 0xffffffffu);
#pragma unroll 1
    for (int i = i0; i < i1; ++i) {
      const int kind = sort(i);
      if (kind != 0) put(kind, i, ones, twos);
      ones += kind == 1;
      twos += kind == 2;
    }
    __syncthreads();
  };
  uint32_t klo = 0, khi = 0;  // keys of the border's two ends
  int close = 0, need = 0;
  auto kind_of = [&](int i) {  // above the border, on it
    const uint32_t k = key_of(i);
    return k > khi ? 1 : k >= klo ? 2 : 0;
  };
  if (!many) {
    const float T = key_score(kth_largest<uint32_t>(
        sh,
        [&](auto&& fn) {
          for (int i = tid; i < N; i += kSelThreads) fn(key_of(i));
        },
        want, above));
    klo = score_key(T - wide);
    khi = score_key(T + wide);
    unsigned int in = 0, mid = 0;
    for (int i = tid; i < N; i += kSelThreads) {
      const int kind = kind_of(i);
      in += kind == 1;
      mid += kind == 2;
    }
    in = __reduce_add_sync(0xffffffffu, in);
    mid = __reduce_add_sync(0xffffffffu, mid);
    if (tid == 0) sh.above = sh.at = 0;
    __syncthreads();
    if (lane == 0) {
      atomicAdd(&sh.above, static_cast<int>(in));
      atomicAdd(&sh.at, static_cast<int>(mid));
    }
    __syncthreads();
    need = want - sh.above;  // > 0: at most want - 1 scores lie above T
    close = sh.at;
    many = close > kSelClose && close > need;
  }
  const int sub = lane / L, lr = lane % L;
  if (many) {  // exact keys for every page, in the slots
    for (int i = warp * G; i < n; i += (kSelThreads / 32) * G) {
      const int p = min(i + sub, n - 1);
      const int page = page_of(a.bt, b, p);
      const unsigned long long k = exact_key<D>(a, b, h, max(page, 0), real, lr);
      if (lr == 0 && i + sub < n && RA_IN_BOUNDS(p, a.stride)) slots[p] = page < 0 ? 0ull : k;
    }
    N = n;
    __syncthreads();
    const unsigned long long T = kth_largest<unsigned long long>(
        sh,
        [&](auto&& fn) {
          for (int i = tid; i < n; i += kSelThreads) fn(slots[i]);
        },
        want, above);
    const int ties = want - above;  // of the pages whose key is T, the first in page order
    in_order([&](int i) { return slots[i] > T ? 1 : slots[i] == T ? 2 : 0; },
             [&](int kind, int i, int ones, int twos) {
               if ((kind == 1 || twos < ties) && RA_IN_BOUNDS(ones + min(twos, ties), want)) out[ones + min(twos, ties)] = i;
             });
    return;
  }
  if (close > need) {
    in_order(kind_of, [&](int kind, int i, int, int twos) {
      if (kind == 2 && RA_IN_BOUNDS(twos, kSelClose)) sh.close_at[twos] = page_at(i);
    });
    for (int j0 = warp * G; j0 < close; j0 += (kSelThreads / 32) * G) {
      const int j = min(j0 + sub, close - 1);
      const int page = page_of(a.bt, b, sh.close_at[j]);
      const unsigned long long k = exact_key<D>(a, b, h, max(page, 0), real, lr);
      if (lr == 0) sh.close[j] = page < 0 ? 0ull : k;
    }
    __syncthreads();
    // each one's rank (the list is in page order), then how many chosen ones come before it, and whether it is one
    constexpr int kEach = (kSelClose + kSelThreads - 1) / kSelThreads;
    int chosen[kEach], sum = 0;
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const int j = kEach * tid + e;
      chosen[e] = 0;
      if (j >= close) continue;
      const unsigned long long k = sh.close[j];
      int place = 0;
      for (int i = 0; i < close; ++i) place += sh.close[i] > k || (sh.close[i] == k && i < j);
      chosen[e] = place < need;
      sum += chosen[e];
    }
    int upto = static_cast<int>(block_scan(sum, sh.warp));  // (its barriers order close_at)
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const int j = kEach * tid + e;
      if (j < close) sh.close_at[j] = chosen[e] ? upto : -1 - upto;
      upto += chosen[e];
    }
    __syncthreads();
  }
  in_order(kind_of, [&](int kind, int i, int ones, int twos) {
    int before = twos;  // chosen ones of the border before this item
    if (close > need) {
      const int x = twos < close ? sh.close_at[twos] : need;
      if (kind == 2 && x < 0) return;
      before = x < 0 ? -1 - x : x;
    }
    if (RA_IN_BOUNDS(ones + before, want)) out[ones + before] = page_at(i);
  });
}

}  // namespace ra
