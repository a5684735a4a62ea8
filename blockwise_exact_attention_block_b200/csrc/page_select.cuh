// page_select.cuh - the pages of a paged cache worth attending to: a score for
// each (sequence, KV head, page) from the page's key bounds, and the n_sel best.
//
// Mathematics: with lo, hi the columnwise minimum and maximum of a page's keys,
//     q . k <= sum_d max(q_d lo_d, q_d hi_d)     for every key k of the page,
// so the sum bounds every score in the page.  A KV head's pages are ranked by
// the largest bound over its query rows; ties go to the lower page.  The pages
// that hold the step's new tokens come first whatever their score.
//
// Which pages win is a comparison, so it must not depend on the order of a
// sum: the bounds are summed in 64 bits, where products of bf16 values (16
// bits) and their sums are exact unless the terms' exponents differ by more
// than 30.
#pragma once

#include "paged.cuh"

namespace ra {

struct SelectArgs {
  PagedBatch bt;  // T = Tq
  int Hq, groups, rows, n_sel;
  const __nv_bfloat16* q;       // [B][Tq][Hq][D]
  const __nv_bfloat16* bounds;  // [n_pages][Hkv][2][D]
  unsigned long long* keys;     // [B * Hkv][max_pages]: scores as ordered integers
  int* selected;                // [B][Hkv][n_sel]
};

constexpr int kScoreThreads = 128;
constexpr int kScoreRows = 8;  // query rows of a sweep over the bounds

// Order-preserving integer of a score; a NaN ranks as -infinity.
__device__ __forceinline__ unsigned long long score_key(double s) {
  if (!(s == s)) s = -INFINITY;
  const unsigned long long b = static_cast<unsigned long long>(__double_as_longlong(s));
  return (b >> 63) ? ~b : b | (1ull << 63);
}

// First page that holds a new token, or the page count when there is none.
__device__ __forceinline__ int first_new_page(const SeqLen& s, int shift) {
  const int pages = (s.len + (1 << shift) - 1) >> shift;
  return s.fresh > 0 ? (s.len - s.fresh) >> shift : pages;
}

// One thread per page (of one sequence and KV head); grid (page blocks, Hkv, B).
// A bf16 bound becomes a double by moving its 15 magnitude bits into the
// double's exponent and mantissa fields, which is the value times 2^-896 (also
// for subnormal bounds; an infinity becomes 2^128, so that 0 times it is 0); the query, widened the ordinary way and multiplied by
// 2^896, carries the factor back.  That is a few integer instructions a bound,
// where a conversion instruction runs at an eighth of that rate.
template <int D>
__global__ void __launch_bounds__(kScoreThreads) page_score_kernel(const __grid_constant__ SelectArgs a) {
  __shared__ double s_q[kScoreRows][D];
  const int b = blockIdx.z, h = blockIdx.y;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const SeqLen s = seq_len_of(a.bt, b);
  const int count = first_new_page(s, a.bt.page_shift);  // the others need no score
  if (static_cast<int>(blockIdx.x) * kScoreThreads >= count) return;
  const int p = blockIdx.x * kScoreThreads + threadIdx.x;
  int page = -1;
  if (p < count) page = page_of(a.bt, b, p);
  const __nv_bfloat16* bl = a.bounds + (static_cast<long long>(max(page, 0)) * a.bt.Hkv + h) * 2 * D;
  const int real = s.fresh * a.groups;  // rows of real tokens come first
  double best = -INFINITY;
  for (int r0 = 0; r0 < real; r0 += kScoreRows) {
    __syncthreads();
    for (int i = threadIdx.x; i < kScoreRows * D; i += kScoreThreads) {
      const int r = r0 + i / D;
      double x = 0.0;
      if (r < real)
        x = static_cast<double>(__bfloat162float(
                a.q[((static_cast<long long>(b) * a.bt.T + r / a.groups) * a.Hq + h * a.groups + r % a.groups) * D + i % D])) *
            0x1p896;
      s_q[i / D][i % D] = x;
    }
    __syncthreads();
    if (page < 0) continue;
    double acc[kScoreRows];
#pragma unroll
    for (int r = 0; r < kScoreRows; ++r) acc[r] = 0.0;
    for (int c = 0; c < D; c += 8) {
      const uint4 lw = *reinterpret_cast<const uint4*>(bl + c), hw = *reinterpret_cast<const uint4*>(bl + D + c);
      const uint32_t lo[4] = {lw.x, lw.y, lw.z, lw.w}, hi[4] = {hw.x, hw.y, hw.z, hw.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        // the smaller and the larger of the two, whatever the caller's order
        const float x0 = __uint_as_float((i & 1) ? (lo[i >> 1] & 0xffff0000u) : (lo[i >> 1] << 16));
        const float x1 = __uint_as_float((i & 1) ? (hi[i >> 1] & 0xffff0000u) : (hi[i >> 1] << 16));
        const uint32_t lb = __float_as_uint(fminf(x0, x1)), hb = __float_as_uint(fmaxf(x0, x1));
        const int ld = static_cast<int>(((lb & 0x7fff0000u) >> 3) | (lb & 0x80000000u));
        const int hd = static_cast<int>(((hb & 0x7fff0000u) >> 3) | (hb & 0x80000000u));
#pragma unroll
        for (int r = 0; r < kScoreRows; ++r) {
          const double x = s_q[r][c + i];
          acc[r] = fma(x, __hiloint2double(__double2hiint(x) < 0 ? ld : hd, 0), acc[r]);
        }
      }
    }
#pragma unroll
    for (int r = 0; r < kScoreRows; ++r)
      if (r0 + r < real) best = fmax(best, acc[r]);
  }
  if (p < count)
    a.keys[(static_cast<long long>(b) * a.bt.Hkv + h) * a.bt.max_pages + p] = score_key(best);
}

constexpr int kSelThreads = 1024;
constexpr int kSelBits = 11;
constexpr int kSelBins = 1 << kSelBits;

// Exclusive sum over the block of a packed pair of counts (whole block).
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
    unsigned long long w = s_warp[lane], v = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long y = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += y;
    }
    s_warp[lane] = v - w;
  }
  __syncthreads();
  return s_warp[warp] + upto - x;
}

// One CTA per (sequence, KV head).  The new tokens' pages are in; of the `n`
// scored pages the `want` best are found digit by digit (11 bits a pass, from
// the highest bit in which the keys differ at all): a histogram of the keys
// that share the digits found so far, and the digit at which the count from the
// top reaches `want`.  It stops when a digit's keys are all wanted, or with
// equal keys, of which the first in page order are taken.  Then every thread
// counts its stretch of pages, one scan gives the places, and the indices come
// out ascending.
__global__ void __launch_bounds__(kSelThreads) page_select_kernel(const __grid_constant__ SelectArgs a) {
  __shared__ unsigned int s_hist[kSelBins];
  __shared__ unsigned long long s_warp[32], s_lo, s_hi;
  __shared__ int s_digit, s_above, s_at;
  const int tid = threadIdx.x, lane = tid & 31;
  const int b = blockIdx.x / a.bt.Hkv;
  int* out = a.selected + static_cast<long long>(blockIdx.x) * a.n_sel;
  const SeqLen s = seq_len_of(a.bt, b);
  const int shift = a.bt.page_shift;
  const int pages = (s.len + (1 << shift) - 1) >> shift;
  const int n = first_new_page(s, shift);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (pages <= a.n_sel) {  // every page
    for (int i = tid; i < a.n_sel; i += kSelThreads) out[i] = i < pages ? i : -1;
    return;
  }
  const int want = a.n_sel - (pages - n);  // >= 0: the host checked n_sel against T
  const unsigned long long* keys = a.keys + static_cast<long long>(blockIdx.x) * a.bt.max_pages;
  unsigned long long top = ~0ull;  // keys whose bits from `low` up exceed top's are in; equal ones compete
  int low = 0;
  int ties = 0;                    // of the competing keys, how many are taken, in page order
  if (want > 0) {
    unsigned long long lo = ~0ull, hi = 0ull;
    for (int i = tid; i < n; i += kSelThreads) {
      const unsigned long long k = keys[i];
      lo = min(lo, k);
      hi = max(hi, k);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      lo = min(lo, __shfl_xor_sync(0xffffffffu, lo, o));
      hi = max(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    if (tid == 0) {
      s_lo = ~0ull;
      s_hi = 0ull;
    }
    __syncthreads();
    if (lane == 0) {
      atomicMin(&s_lo, lo);
      atomicMax(&s_hi, hi);
    }
    __syncthreads();
    top = s_hi;
    ties = want;
    // bits above `bit` are the same in all keys
    int bit = s_lo == s_hi ? 0 : 64 - __clzll(static_cast<long long>(s_lo ^ s_hi));
    low = bit;
    while (low > 0) {
      const int next = max(low - kSelBits, 0), width = low - next;
      for (int i = tid; i < kSelBins; i += kSelThreads) s_hist[i] = 0u;
      __syncthreads();
      for (int i = tid; i < n; i += kSelThreads) {
        const unsigned long long k = keys[i];
        if (low == 64 || (k >> low) == (top >> low)) atomicAdd(&s_hist[(k >> next) & ((1u << width) - 1u)], 1u);
      }
      __syncthreads();
      // two bins a thread, from the top: the digit in which the running count reaches `ties`
      const int d1 = kSelBins - 1 - 2 * tid;
      const unsigned int c1 = s_hist[d1], c0 = s_hist[d1 - 1];
      const int before = static_cast<int>(block_scan(c1 + c0, s_warp));
      if (before < ties && before + static_cast<int>(c1 + c0) >= ties) {
        const bool first = before + static_cast<int>(c1) >= ties;
        s_digit = first ? d1 : d1 - 1;
        s_above = first ? before : before + static_cast<int>(c1);
        s_at = static_cast<int>(first ? c1 : c0);
      }
      __syncthreads();
      const unsigned long long keep = low == 64 ? 0ull : (top >> low) << low;
      top = keep | (static_cast<unsigned long long>(s_digit) << next);
      ties -= s_above;
      low = next;
      const bool all = s_at == ties;
      __syncthreads();
      if (all) break;  // every key with this digit is taken
    }
  }
  // each thread's stretch of pages, in order
  const int per = (n + kSelThreads - 1) / kSelThreads;
  const int i0 = min(tid * per, n), i1 = min(i0 + per, n);
  unsigned int above = 0, equal = 0;
  if (want > 0)
    for (int i = i0; i < i1; ++i) {
      const unsigned long long k = keys[i] >> low, t = top >> low;
      above += k > t;
      equal += k == t;
    }
  const unsigned long long at = block_scan((static_cast<unsigned long long>(above) << 32) | equal, s_warp);
  if (want > 0) {
    unsigned int na = static_cast<unsigned int>(at >> 32), ne = static_cast<unsigned int>(at);
    for (int i = i0; i < i1; ++i) {
      const unsigned long long k = keys[i] >> low, t = top >> low;
      const unsigned int place = na + min(ne, static_cast<unsigned int>(ties));
      if (k > t) {
        out[place] = i;
        ++na;
      } else if (k == t) {
        if (ne < static_cast<unsigned int>(ties)) out[place] = i;
        ++ne;
      }
    }
  }
  for (int i = tid; i < a.n_sel - want; i += kSelThreads) out[want + i] = n + i;
}

}  // namespace ra
