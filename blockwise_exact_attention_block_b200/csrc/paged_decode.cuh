// paged_decode.cuh - attention of a few new tokens over a paged key-value
// cache (bf16, int8 or e4m3), all of it or only selected pages.
//
// TokenRing review (pith.science, arXiv 2412.20501), "Reading between the
// lines": the decode phase as KV-cache chunking, partial results joined by
// their log-sum-exp.  Here a chunk is whatever run of the cache one team of
// warps walks, and it may begin and end anywhere in a sequence.
//
// Mathematics, per query row (c = log2(e) / sqrt(D), everything in fp32), of an
// 8-bit cache with key and value scales ks_j, vs_j (both 1 for bf16):
//     x_j = c ks_j (q . k_j),   w_j = vs_j 2^(x_j - E),
//     l = sum 2^(x_j - E),   o = sum w_j v_j,   out = o / l,   lse = ln 2 (E + log2 l)
// with k_j, v_j the codes as they are stored.  E is any reference for which no
// term overflows: out and lse do not depend on it.  It starts at the first
// tile's max (x_j + log2 vs_j) less kPgStart, which makes the largest w_j 2^kPgStart, and is
// raised to that of a later tile, with l and o rescaled, only when a w_j passes kPgLazy.
// So most tiles need no maximum across lanes at all: each lane looks at its own
// terms, and one vote says that none is too large.
//
// The weights w_j go to the tensor core as two 16-bit terms, the leading bits
// and the rounded remainder, or three for an fp32 output: with bf16 (cache in
// bf16) 2^-16 or 2^-24 relative, with f16 (8-bit cache) 2^-22 relative and
// 2^-24 / 2^kPgStart of the row's largest w.  (At kPgStart = 0 a run of 50,000 keys 2^-25
// below the largest was missing from o, 1.4e-3 of it, while l had them; at 12, eight times
// below kPgLazy, the reference moves often: 8 x 9k-24k int8 keys, 16 rows 83 us, at 5 to 10
// 81.5.)  One rounded term (2^-8 for bf16) would cost as much accuracy as the output's
// own rounding.  8-bit codes are turned into f16, which
// holds them exactly; the queries then go in as f16 too, scaled by a power of two
// that brings the warp's largest to 2^14 (bf16's 8 bits fit down to 2^-30 of it).  A
// warp whose rows differ by more than 2^16 scales each row by itself and brings
// the scores to the largest's scale.
//
// The tensor core cuts its fp32 sums off instead of rounding them, always towards
// zero.  So o never goes through it: a tile's products start from zero and are added
// to o by rounded additions, two to an instruction.  With o as the product's
// accumulator a run of 50,000 keys came out 3.7e-4 too small, 6e-7 this way.  It
// costs 5 to 7 % where instruction issue is the bound (8 x 9k-24k int8 keys, 16 rows:
// 77.5 us then, 82 now), up to 13 % for a bf16 team of several warps, nothing where HBM is.
//
// What bounds it: a cached element meets the groups * Tq (<= 64) query rows of its KV
// head and is used once, so HBM bounds bf16 caches up to 16 rows (1M keys 174 us, 94 % of
// the copy rate); instruction issue and its latency bound 8-bit ones (eight sequences of
// 9k to 24k int8 keys, 8 heads, 128 columns: 58 us for 4 rows, 766 instructions a tile, 82
// for 16 rows, 1,040 a tile at 40 % of the issue slots; HBM alone 42) and teams of several
// warps (32 rows 191, of a bf16 cache 229).  So the cache is streamed once, through
// rings of shared memory, by 16-byte asynchronous copies: a page of one head may be
// as small as 1 KB and the tile's scales are 128 bytes, and a TMA copy costs the
// same to issue whatever its size (with TMA, one token a sequence, 16-key pages of
// those took 97 us where 64-key ones took 75).  The products are mma.sync m16n8k16 with the keys
// (scores) or the columns (output) on the 16 side and the query rows on the 8
// side: up to 8 rows, the usual single token, cost half of what rows on the 16
// side would, in products, in exponentials and in accumulator registers.
// (tcgen05 takes 128 by at least 16 and would add a pass through tensor memory.)
//
// Work split: the cache of all (sequence, KV head) pairs, cut into tiles of 32
// keys, is one line of tiles (sequence-major, then head, then position) in
// which each pair also takes kPgPairCost units for its start and end.  The
// lengths are on the device, so the teams work out the line's length from them
// and take equal runs of it; runs cross pair borders, so a batch of one 100k
// and many short sequences is as even as a uniform one, with one grid shape
// for all lengths (a captured graph replays with new ones).  A team's run
// covers whole pairs, written out directly, and at most two cut ones (its first
// and last), left as (E, l, o) in the workspace for the combine kernel, which
// knows each cut pair from a record of its first and last team.
//
// A CTA has one walker warp, whose lane t walks the run of team t, looks up pages
// and queues the tiles in shared memory, and kWarps consumer warps, which copy
// and compute them.  A team is one consumer warp for up to 8 (NB = 1) or 16
// (NB = 2) query rows, 2 or 4 warps (NB = 2) for up to 32 or 64, each with 16 of
// the rows and all sharing the team's ring.  Teams never meet at a barrier.
#pragma once

#include <type_traits>

#include "decode.cuh"
#include "paged.cuh"

namespace ra {

constexpr int kPgKeys = 32;         // keys of a tile
constexpr int kPgQueue = 8;         // tiles queued for a team
constexpr int kPgSlots = 8;         // ring items per warp, at most
constexpr int kPgPairCost = 3;      // a pair's start and end, in tiles
// log2 of the largest weight when the reference E is set, and the weight above which
// E moves.  bf16 terms have fp32's range; f16 ones end at 65504 and at 2^-24.
template <int ET>
constexpr float kPgStart = ET == kCacheBf16 ? 0.f : 10.f;
template <int ET>
constexpr float kPgLazy = ET == kCacheBf16 ? 1024.f : 32768.f;
constexpr int kPgNone = 0x7fffff00; // position of a key that no row sees

struct PagedArgs {
  PagedBatch bt;  // T = Tq
  int Hq, groups, rows, causal;
  int R;         // warps per team
  int min_run;   // a team's run is at least this long
  int n_sel;
  const int* selected;  // [B][Hkv][n_sel] or null
  float scale_log2;
  const __nv_bfloat16* q;  // [B][Tq][Hq][D]
  const void* k_pages;
  const void* v_pages;
  const float* k_scales;
  const float* v_scales;
  float* part_o;    // [teams][2][rows][D]
  float2* part_ml;  // [teams][2][rows]: E (log2 units), l
  int2* cut;        // [B * Hkv]: first and last team of a cut pair; first < 0: not cut
  void* out;        // [B][Tq][Hq][D]
  int out_bf16;
  float* lse;
};

// Shared memory and the shape of a CTA, the walker's warp included a multiple of
// four warps where registers matter (the register file is shared out by four).
// bf16, D = 128: an item is 8 KB, and 8 consumer warps with rings of three keep
// the copies in flight that HBM needs; 16 rows each want 255 registers, so 7 there
// (99 us against 117 with 8 and spilled registers: 8 x 9k-24k keys, 16 rows), but 8
// for teams of several warps, which 7 would leave with one team of four.  Smaller
// items, and a conversion of 8-bit codes besides, make instruction issue what
// must be fed: 15 warps of 8 rows (128 registers), 11 of 16 rows (168: the output
// accumulators alone take 64).
template <int D, int ET, int NB, bool TEAMS>
struct PgSmem {
  static constexpr bool kWide = ET == kCacheBf16 && D == 128;  // items of 8 KB
  static constexpr int kWarps = kWide ? (NB == 1 || TEAMS ? 8 : 7) : NB == 1 ? 15 : 11;
  static constexpr int kThreads = 32 * (kWarps + 1);
  static constexpr int kRing = kWide ? 24576 : NB == 1 ? 12288 : 16384;  // bytes per warp
  static constexpr int kElem = ET == kCacheBf16 ? 2 : 1;
  static constexpr int kItem = kPgKeys * D * kElem;  // one tile of K or of V
  static constexpr int kSlots = kRing / kItem < kPgSlots ? kRing / kItem : kPgSlots;  // per warp
  static constexpr int kRow = D * kElem;  // bytes of a cached row
  static constexpr int kScale = kWarps * kRing;                          // fp32 [slots][32]
  static constexpr int kMeta = kScale + (ET == kCacheBf16 ? 0 : kWarps * kSlots * kPgKeys * 4);
  static constexpr int kFull = kMeta + kWarps * kPgQueue * 32;           // barriers of a team's ring items
  static constexpr int kEmpty = kFull + kWarps * kSlots * 8;
  static constexpr int kQFull = kEmpty + kWarps * kSlots * 8;            // and of the queue entries
  static constexpr int kQEmpty = kQFull + kWarps * kPgQueue * 8;
  static constexpr int kAbort = kQEmpty + kWarps * kPgQueue * 8;
  static constexpr int kBytes = kAbort + 16 + 256;  // + slack to align the base to 256
};

// Ring items of a team: the loads run ahead of the tile in work by this many,
// which the queue has to cover.
template <typename SL>
__device__ __forceinline__ int pg_slots(int R) {
  return min(SL::kSlots * R, 2 * (kPgQueue - 2));
}

// A queued tile: the cache rows and the positions of the first key of each 16,
// the pair, its lengths, and these flags.
enum { kPgFirst = 1, kPgLast = 2, kPgWhole = 4, kPgOwner = 8, kPgStop = 16 };
struct alignas(16) PgTile {
  int r0, r1, p0, p1;
  int b, h, len;
  int fresh_flags;  // new tokens << 8 | flags
};

// Byte offset of the 16-byte chunk c of key j in a tile of rows of ROW bytes:
// chunks permuted within 128 bytes so that eight keys' chunks lie in eight
// different bank groups.
template <int ROW>
__device__ __forceinline__ uint32_t pg_off(int j, int c) {
  return j * ROW + ((c ^ (ROW >= 128 ? j & 7 : (j >> 1) & 3)) << 4);
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16;" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(src))
               : "memory");
}

// Arrives on `bar` (once per thread) when this thread's copies so far have landed.
__device__ __forceinline__ void copies_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// Closes the group of this thread's copies since the last one (it may be empty), and
// waits for all groups but the last N.
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void copies_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// D (16x8 fp32) += A (16x16, row-major) * B (16x8, column-major), operands bf16
// for a bf16 cache, f16 for an 8-bit one.
template <int ET>
__device__ __forceinline__ void pg_mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (ET == kCacheBf16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Transposes an 8x8 matrix of 16-bit values held two to a lane (row lane / 4,
// columns 2 (lane % 4), + 1).
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// The codes in bytes 0 and 2 of w as two f16 values, exactly: 0x6400 | u is the
// f16 1024 + u, so with the sign bit flipped (u = code + 128) and 1152 taken
// away the signed code is left.
__device__ __forceinline__ uint32_t i8_to_f16(uint32_t w) {
  uint32_t r;  // lop3 0x6a: (w & 0x00ff00ff) ^ 0x64806480
  asm("lop3.b32 %0, %1, %2, %3, 0x6a;" : "=r"(r) : "r"(w), "r"(0x00ff00ffu), "r"(0x64806480u));
  asm("add.rn.f16x2 %0, %0, %1;" : "+r"(r) : "r"(0xe480e480u));
  return r;
}

// The e4m3 codes in bytes 0 and 1 (HALF = 0) or 2 and 3 of w as two f16 values.
template <int HALF>
__device__ __forceinline__ uint32_t e4m3_to_f16(uint32_t w) {
  uint32_t r;
  if constexpr (HALF == 0)
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(r) : "r"(w));
  else
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(w));
  return r;
}

// A pair of weights as 16-bit pairs of the operand type: the leading bits (cut
// off, so that the remainder is exact), then the rounded remainder, and for a
// bf16 operand and an fp32 output what that left (f16 has 22 bits by then).
template <int ET>
__device__ __forceinline__ void split_pair(float x, float y, bool three, uint32_t (&t)[3]) {
  constexpr uint32_t kCut = ET == kCacheBf16 ? 0xffff0000u : 0xffffe000u;  // 8 or 11 bits
  const float xh = __uint_as_float(__float_as_uint(x) & kCut), yh = __uint_as_float(__float_as_uint(y) & kCut);
  const float xr = x - xh, yr = y - yh;
  t[2] = 0u;
  if constexpr (ET == kCacheBf16) {
    t[0] = __byte_perm(__float_as_uint(x), __float_as_uint(y), 0x7632);
    t[1] = pack_bf16x2(xr, yr);
    if (three)
      t[2] = pack_bf16x2(xr - __uint_as_float(t[1] << 16), yr - __uint_as_float(t[1] & 0xffff0000u));
  } else {
    t[0] = pack_f16x2(xh, yh);
    t[1] = pack_f16x2(xr, yr);
  }
}

// Tiles of one (sequence, KV head) pair; none where no row is real.
__device__ __forceinline__ int pg_tiles(const PagedArgs& a, const SeqLen& s) {
  if (s.fresh == 0) return 0;
  if (a.selected == nullptr) return (s.len + kPgKeys - 1) / kPgKeys;
  const int pages = (s.len + (1 << a.bt.page_shift) - 1) >> a.bt.page_shift;
  return ((min(a.n_sel, pages) << a.bt.page_shift) + kPgKeys - 1) / kPgKeys;
}

// Units of the line that a sequence takes: its pairs' tiles and costs.
__device__ __forceinline__ long long pg_units(const PagedArgs& a, const SeqLen& s) {
  const int n = pg_tiles(a, s);
  return n > 0 ? static_cast<long long>(n + kPgPairCost) * a.bt.Hkv : 0;
}

// Element of the output at column d of a row.
__device__ __forceinline__ void pg_store1(const PagedArgs& a, long long row, int D, int d, float x) {
  if (a.out_bf16) static_cast<__nv_bfloat16*>(a.out)[row * D + d] = __float2bfloat16_rn(x);
  else static_cast<float*>(a.out)[row * D + d] = x;
}
__device__ __forceinline__ void pg_store2(const PagedArgs& a, long long row, int D, int d, float x, float y) {
  if (a.out_bf16)
    *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(a.out) + row * D + d) = pack_bf16x2(x, y);
  else
    *reinterpret_cast<float2*>(static_cast<float*>(a.out) + row * D + d) = make_float2(x, y);
}

// ------------------------------------------------------------------ walker

// x / y of values that are not negative; most fit 32 bits, where a division is much shorter.
__device__ __forceinline__ long long quotient(long long x, long long y) {
  if (((x | y) >> 32) == 0) return static_cast<unsigned>(x) / static_cast<unsigned>(y);
  return x / y;
}

// The walker warp: lane t < teams walks the run of team t.  In every round the
// lanes whose queue has room post one tile.  Page numbers are loaded when a
// tile is reached and used in the round that posts it, so their latency
// overlaps the rounds between.  own: the units of sequence `lane`.
template <int D, int ET, int NB, bool TEAMS>
__device__ __forceinline__ void pg_walk(const PagedArgs& a, uint8_t* smem, volatile int* abort_flag, long long own) {
  using SL = PgSmem<D, ET, NB, TEAMS>;
  const int lane = threadIdx.x & 31;
  const int teams = SL::kWarps / a.R;
  const uint32_t sb = smem_u32(smem);
  const uint32_t qfull = sb + SL::kQFull + 8u * kPgQueue * lane, qempty = sb + SL::kQEmpty + 8u * kPgQueue * lane;
  PgTile* queue = reinterpret_cast<PgTile*>(smem + SL::kMeta) + kPgQueue * lane;
  const int ps = 1 << a.bt.page_shift;

  // the line and this lane's run [f0, f0 + n) of it; lane i holds the units of sequence i of each 32
  long long total = own;
  for (int i = lane + 32; i < a.bt.B; i += 32) total += pg_units(a, seq_len_of(a.bt, i));
#pragma unroll
  for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  const long long U = static_cast<long long>(gridDim.x) * teams;
  const long long u = static_cast<long long>(lane) * gridDim.x + blockIdx.x;
  const int run = max(static_cast<int>(quotient(total + U - 1, U)), a.min_run);  // (below 2^30: the host bounds the line)
  const long long f0 = u * run;
  const int n = static_cast<int>(max(min(f0 + run, total) - f0, 0ll));
  bool work = lane < teams && n > 0;
  // its place: sequence b (starting at unit `start` of the line)
  int b = 0;
  long long start = 0;
  {
    long long before = 0;
    bool found = false;
    for (int b0 = 0; b0 < a.bt.B; b0 += 32) {
      if (b0 > 0) own = b0 + lane < a.bt.B ? pg_units(a, seq_len_of(a.bt, b0 + lane)) : 0;
      long long upto = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += x;
      }
      const long long end = before + __shfl_sync(0xffffffffu, upto, 31);
      const bool here = work && !found && f0 < end;
      if (__any_sync(0xffffffffu, here)) {  // the first sequence that ends behind f0
        int i = 0;
#pragma unroll
        for (int step = 16; step; step >>= 1) {
          const long long x = before + __shfl_sync(0xffffffffu, upto, i + step - 1);
          if (here && f0 >= x) i += step;
        }
        const long long x = before + __shfl_sync(0xffffffffu, upto - own, i);
        if (here) {
          found = true;
          b = b0 + i;
          start = x;
        }
      }
      before = end;
    }
  }
  SeqLen s = {0, 0};
  int nt = 0, h = 0, t = 0;
  int pair = 0;  // the pair's first unit, from f0 (negative where an earlier team began it)
  if (work) {
    s = seq_len_of(a.bt, b);
    nt = pg_tiles(a, s);
    const long long rel = f0 - start;
    h = static_cast<int>(quotient(rel, nt + kPgPairCost));
    pair = static_cast<int>(static_cast<long long>(h) * (nt + kPgPairCost) - rel);
    t = max(-pair - kPgPairCost, 0);
  }
  // the next tile with work at or behind (b, h, t); work = false behind the run's end
  auto settle = [&]() {
    while (work) {
      if (pair + kPgPairCost + t >= n) work = false;  // the rest of the line is other teams'
      else if (t < nt) break;
      else {
        pair += nt + kPgPairCost;
        t = 0;
        if (++h == a.bt.Hkv) {
          h = 0;
          do {
            ++b;
            s = b < a.bt.B ? seq_len_of(a.bt, b) : SeqLen{0, 0};
            nt = pg_tiles(a, s);
          } while (b < a.bt.B && nt == 0);
          if (b >= a.bt.B) work = false;
        }
      }
    }
  };
  // Table index of the 16 keys from 16 u of the pair; -1 for none.
  auto logical_of = [&](int unit) -> int {
    const long long key = 16LL * unit;
    if (a.selected == nullptr) return key < s.len ? static_cast<int>(key >> a.bt.page_shift) : -1;
    const int pages = (s.len + ps - 1) >> a.bt.page_shift;
    const int idx = static_cast<int>(key >> a.bt.page_shift);
    if (idx >= min(a.n_sel, pages)) return -1;
    if (!RA_IN_BOUNDS(b, a.bt.B) || !RA_IN_BOUNDS(h, a.bt.Hkv) || !RA_IN_BOUNDS(idx, a.n_sel)) return -1;
    const int* sel = a.selected + (static_cast<long long>(b) * a.bt.Hkv + h) * a.n_sel;
    const int x = sel[idx];
    int prev = idx > 0 ? sel[idx - 1] : -1;  // the entry in range before it: as a rule the last one
    if (x == -1) return -1;
    bool good = x >= 0 && x < pages;
    if (good) {
      if (prev >= pages) prev = -1;
      for (int i = idx - 2; prev < 0 && i >= 0; i -= 8) {  // over a gap, eight loads at a time
        int y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = i >= e ? sel[i - e] : -1;
#pragma unroll
        for (int e = 7; e >= 0; --e)
          if (y[e] >= 0 && y[e] < pages) prev = y[e];
      }
      good = x > prev;
    }
    if (!good) set_status(RA_ERR_DEVICE_BOUNDS);
    return good ? x : -1;
  };
  // the tile's one or two pages: table indices and what the table holds there
  int lg0 = -1, lg1 = -1, pg0 = 0, pg1 = 0;
  auto look_up = [&]() {
    const int* row = a.bt.page_table + static_cast<long long>(b) * a.bt.max_pages;
    lg0 = logical_of(2 * t);
    if (!RA_IN_BOUNDS(b, a.bt.B) || (lg0 >= 0 && !RA_IN_BOUNDS(lg0, a.bt.max_pages))) lg0 = -1;
    if (lg0 >= 0) pg0 = row[lg0];
    if (ps == 16) {
      lg1 = logical_of(2 * t + 1);
      if (!RA_IN_BOUNDS(b, a.bt.B) || (lg1 >= 0 && !RA_IN_BOUNDS(lg1, a.bt.max_pages))) lg1 = -1;
      if (lg1 >= 0) pg1 = row[lg1];
    }
  };
  settle();
  if (work) look_up();

  bool first = true, stopped = lane >= teams;
  int posted = 0, slot = 0;
  uint32_t phase = 0;
  long long t0 = clock64();
  while (true) {
    const bool go = !stopped && (posted < kPgQueue || mbar_test_wait(qempty + 8u * slot, phase ^ 1u));
    if (go) {
      PgTile m;
      m.r0 = m.r1 = 0;
      m.p0 = m.p1 = kPgNone;
      m.b = b;
      m.h = h;
      m.len = s.len;
      int flags = kPgStop;  // the run's end
      if (work) {
        auto place = [&](int lg, int pg, int key, int& r, int& p) {
          if (lg < 0) return;
          if (pg < 0 || pg >= a.bt.n_pages) {
            set_status(RA_ERR_DEVICE_BOUNDS);
            return;
          }
          // (the consumers copy 16 rows from r, or 32 of a page that holds as many)
          if (!RA_IN_BOUNDS((((static_cast<long long>(pg) * a.bt.Hkv + h) << a.bt.page_shift) + (key & (ps - 1))) +
                                min(ps, kPgKeys) - 1 + PG_INJECTED(a.bt),
                            row_extent(a.bt)))
            return;
          r = ((pg * a.bt.Hkv + h) << a.bt.page_shift) + (key & (ps - 1));
          p = (lg << a.bt.page_shift) + (key & (ps - 1));
        };
        place(lg0, pg0, 32 * t, m.r0, m.p0);
        if (ps == 16) {
          place(lg1, pg1, 32 * t + 16, m.r1, m.p1);
        } else if (m.p0 != kPgNone) {
          m.r1 = m.r0 + 16;
          m.p1 = m.p0 + 16;
        }
        const bool owner = pair + kPgPairCost >= 0;
        const bool last = t + 1 == nt || pair + kPgPairCost + t + 1 >= n;
        flags = (first ? kPgFirst : 0) | (last ? kPgLast : 0) | (owner && t + 1 == nt ? kPgWhole : 0) | (owner ? kPgOwner : 0);
      }
      m.fresh_flags = (s.fresh << 8) | flags;
      queue[slot] = m;
      mbar_arrive(qfull + 8u * slot);
      ++posted;
      if (++slot == kPgQueue) {
        slot = 0;
        phase ^= 1u;
      }
      // what nobody waits for: the pair's record (cut, if its last tile is another team's) and the next tile
      if (work) {
        if ((flags & (kPgFirst | kPgOwner)) == (kPgFirst | kPgOwner)) {
          const int on = static_cast<int>(static_cast<unsigned>(pair + kPgPairCost + nt - 1) / static_cast<unsigned>(run));
          if (RA_IN_BOUNDS(b, a.bt.B) && RA_IN_BOUNDS(h, a.bt.Hkv) && RA_IN_BOUNDS(u + on, U))
            a.cut[static_cast<long long>(b) * a.bt.Hkv + h] =
                on == 0 ? make_int2(-1, -1) : make_int2(static_cast<int>(u), static_cast<int>(u) + on);
        }
        first = flags & kPgLast;
        ++t;
        settle();
        if (work) look_up();
      } else {
        stopped = true;
      }
    }
    if (__all_sync(0xffffffffu, stopped)) return;
    if (__any_sync(0xffffffffu, go)) {
      t0 = clock64();
      continue;
    }
    if (*abort_flag || grid_timed_out()) return;
    if (clock64() - t0 > kWaitLimitCycles) {
      set_status(RA_ERR_TIMEOUT);
      *abort_flag = 1;
      return;
    }
    __nanosleep(500);
  }
}

// ---------------------------------------------------------------- consumers

template <int D, int ET, int NB, bool TEAMS>
__global__ void __launch_bounds__(PgSmem<D, ET, NB, TEAMS>::kThreads, 1)
    paged_partial_kernel(const __grid_constant__ PagedArgs a) {
  using SL = PgSmem<D, ET, NB, TEAMS>;
  constexpr int KS = D / 16;  // k16 steps of the score product, and 16-column blocks of the output
  constexpr int NR = 2 * NB;  // query rows of a lane: 8 nb + 2 (lane % 4), + 1
  constexpr int ROW = SL::kRow;
  extern __shared__ uint8_t pg_raw[];
  uint8_t* smem = pg_raw + ((256u - (smem_u32(pg_raw) & 255u)) & 255u);
  const uint32_t sb = smem_u32(smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + SL::kAbort);
  const int teams = SL::kWarps / a.R, slots = TEAMS ? pg_slots<SL>(a.R) : SL::kSlots;

  for (int i = tid; TEAMS && i < teams * slots; i += SL::kThreads) {
    mbar_init(sb + SL::kFull + 8u * i, 32 * a.R);  // every thread of the team
    mbar_init(sb + SL::kEmpty + 8u * i, a.R);
  }
  for (int i = tid; i < teams * kPgQueue; i += SL::kThreads) {
    mbar_init(sb + SL::kQFull + 8u * i, 1);
    mbar_init(sb + SL::kQEmpty + 8u * i, a.R);
  }
  fence_mbar_init();
  chain_launches();
  long long own = 0;  // the walker's first lengths, on their way while the barriers are set up
  if (warp == SL::kWarps && lane < a.bt.B) own = pg_units(a, seq_len_of(a.bt, lane));
  if (tid == 32 * SL::kWarps) *abort_flag = grid_timed_out() ? 1 : 0;
  __syncthreads();
  if (*abort_flag) return;
  if (warp == SL::kWarps) {
    pg_walk<D, ET, NB, TEAMS>(a, smem, abort_flag, own);
    return;
  }

  // sequences without a tile (empty or idle): their rows are empty
  for (int b = blockIdx.x * SL::kWarps + warp; b < a.bt.B; b += gridDim.x * SL::kWarps) {
    if (pg_tiles(a, seq_len_of(a.bt, b)) > 0) continue;
    const long long q0 = static_cast<long long>(b) * a.bt.T * a.Hq, n = static_cast<long long>(a.bt.T) * a.Hq;
    for (long long i = lane; i < n * (D / 2); i += 32)
      pg_store2(a, q0 + i / (D / 2), D, 2 * static_cast<int>(i % (D / 2)), 0.f, 0.f);
    for (long long i = lane; i < n; i += 32) a.lse[q0 + i] = -INFINITY;
    for (int h = lane; h < a.bt.Hkv; h += 32) a.cut[static_cast<long long>(b) * a.bt.Hkv + h] = make_int2(-1, -1);
  }

  const int gr = lane >> 2, qd = lane & 3;  // fragment row and column pair of this lane
  const int team = warp / a.R, rt = warp % a.R;
  if (team >= teams) return;  // 11 warps hold 5 teams of two, 2 of four
  const uint32_t ring = sb + team * a.R * SL::kRing;
  const int slot0 = team * slots;
  const uint32_t full = sb + SL::kFull + 8u * slot0, empty = sb + SL::kEmpty + 8u * slot0;
  const uint32_t qfull = sb + SL::kQFull + 8u * kPgQueue * team, qempty = sb + SL::kQEmpty + 8u * kPgQueue * team;
  const PgTile* queue = reinterpret_cast<const PgTile*>(smem + SL::kMeta) + kPgQueue * team;
  const float* scales = reinterpret_cast<const float*>(smem + SL::kScale) + slot0 * kPgKeys;
  const int row0 = 8 * NB * rt;  // this warp's first query row

  // ---- copies: items K, V, K, V ... of the queued tiles into the ring's slots.
  // A warp instruction copies 512 bytes: copy n holds the keys from 512 / ROW * n,
  // lane i their 16 bytes from 16 i.  The permutation of a key's chunks depends on
  // n through kFlips values, so that many addresses serve all copies; the team's
  // warps take the copies in turn.
  constexpr int kCopies = SL::kItem / 512;
  constexpr int kFlips = ROW == 256 ? 4 : ROW == 128 ? 2 : 1;
  const uint32_t lane_off = pg_off<ROW>(lane / (ROW / 16), lane % (ROW / 16));
  const uint8_t* const src_k = static_cast<const uint8_t*>(a.k_pages) + 16 * lane;
  const uint8_t* const src_v = static_cast<const uint8_t*>(a.v_pages) + 16 * lane;
  int lslot = 0, lq = 0, lr0 = 0, lr1 = 0;  // next slot and queue entry, rows of the tile being loaded
  uint32_t lphase = 0, lqphase = 0;
  bool lstop = false, wrapped = false, ok = true;
  int slot = 0;  // and the slot to be read
  uint32_t phase = 0;
  auto copy_item = [&](const uint8_t* src, const float* sc) {
    if (TEAMS && wrapped) ok &= mbar_wait(empty + 8u * lslot, lphase ^ 1u, abort_flag);  // (one warp: it has read the slot)
    const uint8_t* g0 = src + static_cast<long long>(lr0) * ROW;
    const uint8_t* g1 = src + static_cast<long long>(lr1) * ROW - SL::kItem / 2;
    const uint32_t dst = ring + lslot * SL::kItem;
    if (!TEAMS) {
      uint32_t d[kFlips];
#pragma unroll
      for (int i = 0; i < kFlips; ++i) d[i] = dst + (lane_off ^ (static_cast<uint32_t>(512 / ROW * i & 7) << 4));
#pragma unroll
      for (int n = 0; n < kCopies; ++n) copy16(d[n % kFlips] + 512 * n, (n < kCopies / 2 ? g0 : g1) + 512 * n);
    } else {
      for (int n = rt; n < kCopies; n += a.R)
        copy16(dst + 512 * n + (lane_off ^ (static_cast<uint32_t>(512 / ROW * (n % kFlips) & 7) << 4)),
               (n < kCopies / 2 ? g0 : g1) + 512 * n);
    }
    if constexpr (ET != kCacheBf16)
      if (rt == 0 && lane < 8)
        copy16(sb + SL::kScale + (slot0 + lslot) * kPgKeys * 4 + 16 * lane, sc + (lane < 4 ? lr0 : lr1 - 16) + 4 * lane);
    if (TEAMS) copies_arrive(full + 8u * lslot);
    if (++lslot == slots) {
      lslot = 0;
      lphase ^= 1u;
      wrapped = true;
    }
  };
  // A warp on its own counts groups of copies: one for each item, empty behind the
  // last tile, so that `slots` of them are always open and the oldest is the next to
  // be read.  A team's warps wait for one another's copies on barriers.
  auto landed = [&]() {
    if constexpr (TEAMS) {
      ok &= mbar_wait(full + 8u * slot, phase, abort_flag);
    } else {
      copies_wait<SL::kSlots - 1>();
      __syncwarp();
    }
  };
  auto next_k = [&]() {  // the next queued tile's keys, if there is a tile
    if (lstop) return;
    ok &= mbar_wait(qfull + 8u * lq, lqphase, abort_flag);
    const int4 rows = *reinterpret_cast<const int4*>(&queue[lq]);
    lstop = !__all_sync(0xffffffffu, ok) || (queue[lq].fresh_flags & kPgStop);
    if (lstop) return;
    lr0 = rows.x;
    lr1 = rows.y;
    if (++lq == kPgQueue) {
      lq = 0;
      lqphase ^= 1u;
    }
    copy_item(src_k, a.k_scales);
  };
  auto load_k = [&]() {
    next_k();
    if (!TEAMS) copies_commit();
  };
  auto load_v = [&]() {  // and its values
    if (!lstop) copy_item(src_v, a.v_scales);
    if (!TEAMS) copies_commit();
  };
  int cq = 0;
  auto release = [&]() {  // this warp has read the slot
    __syncwarp();
    if (TEAMS && lane == 0) mbar_arrive(empty + 8u * slot);
    if (++slot == slots) {
      slot = 0;
      phase ^= 1u;
    }
  };
  static_assert(SL::kSlots <= 2 * (kPgQueue - 2), "the queue covers a warp's ring");
  const bool odd = slots & 1;  // then a released K slot takes a V, and the other way round
  load_k();
  for (int i = 1; i < slots; ++i) {
    if (i & 1) load_v();
    else load_k();
  }

  uint32_t qb[KS][NB][2];
  float o[KS][NB][4], E[NR], l[NR], qscale = a.scale_log2;
  float rowscale[NR];  // (8-bit cache, `uneven`) this lane's rows' scales by the warp's
  bool uneven = false;
  bool unset = false;  // the warp has a real row without a reference: all its scores so far are -inf
  int lim[NR], minlim = 0;
  // lane parts of the shared-memory addresses; a chunk index goes in by exclusive or
  // (the slots begin at multiples of the 256 bytes that it can change)
  const uint32_t k_lane = ET == kCacheBf16 ? pg_off<ROW>(lane & 15, lane >> 4) : pg_off<ROW>(gr, qd);
  const uint32_t v_lane = ET == kCacheBf16 ? pg_off<ROW>((lane & 7) + 8 * (lane >> 4), (lane >> 3) & 1)
                                           : pg_off<ROW>(lane & 15, 0);
  while (true) {
    if (TEAMS && !__all_sync(0xffffffffu, ok)) break;  // (a warp on its own has looked when it loaded)
    if (lstop && cq == lq) break;  // every loaded tile is done
    const int4 t0 = reinterpret_cast<const int4*>(&queue[cq])[0], t1 = reinterpret_cast<const int4*>(&queue[cq])[1];
    const PgTile tile = {t0.x, t0.y, t0.z, t0.w, t1.x, t1.y, t1.z, t1.w};
    const int fresh = tile.fresh_flags >> 8, flags = tile.fresh_flags & 255;
    if (flags & kPgFirst) {  // the query rows of this (sequence, KV head)
      minlim = 0x7fffffff;
#pragma unroll
      for (int i = 0; i < NR; ++i) {
        const int r = row0 + 8 * (i >> 1) + 2 * qd + (i & 1), tk = r / a.groups;
        const bool real = r < a.rows && tk < fresh;
        lim[i] = real ? (a.causal ? tile.len - fresh + tk + 1 : tile.len) : 0;
        if (real) minlim = min(minlim, lim[i]);
        E[i] = -INFINITY;
        l[i] = 0.f;
      }
      uint32_t qmax[NB];  // largest magnitudes, as pairs of bf16 bits
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        qmax[nb] = 0u;
        const int r = row0 + 8 * nb + gr, tk = r / a.groups;
        const bool real = r < a.rows && tk < fresh && RA_IN_BOUNDS(tk, a.bt.T) && RA_IN_BOUNDS(tile.b, a.bt.B) &&
                          RA_IN_BOUNDS(tile.h, a.bt.Hkv);
        const __nv_bfloat16* qr =
            a.q + (real ? ((static_cast<long long>(tile.b) * a.bt.T + tk) * a.Hq + tile.h * a.groups + r % a.groups) * D : 0);
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          if constexpr (ET == kCacheBf16) {
            qb[ks][nb][0] = real ? *reinterpret_cast<const uint32_t*>(qr + 16 * ks + 2 * qd) : 0u;
            qb[ks][nb][1] = real ? *reinterpret_cast<const uint32_t*>(qr + 16 * ks + 8 + 2 * qd) : 0u;
          } else {
            // step ks = 4 half + i of the product takes columns 16 (qd + 4 half) + 4 i + {0 .. 3}
            const uint2 x = real ? *reinterpret_cast<const uint2*>(qr + 16 * (qd + 4 * (ks >> 2)) + 4 * (ks & 3))
                                 : make_uint2(0u, 0u);
            qb[ks][nb][0] = x.x;
            qb[ks][nb][1] = x.y;
            qmax[nb] = __vmaxu2(qmax[nb], __vmaxu2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu));
          }
        }
      }
#pragma unroll
      for (int x = 16; x; x >>= 1) minlim = min(minlim, __shfl_xor_sync(0xffffffffu, minlim, x));
      if constexpr (ET != kCacheBf16) {
        // exponent fields of the rows' largest values, and of the warp's; a row with an
        // infinity or a NaN, whose result is NaN, counts for neither
        int er[NB], ew = 0;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          uint32_t m = max(qmax[nb] & 0xffffu, qmax[nb] >> 16);
#pragma unroll
          for (int x = 1; x < 4; x <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, x));
          er[nb] = m < 0x7f80u ? static_cast<int>(m >> 7) : 0;
          ew = max(ew, er[nb]);
        }
        ew = __reduce_max_sync(0xffffffffu, ew);
        bool low = false;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) low |= er[nb] > 0 && er[nb] + 16 < ew;
        uneven = __any_sync(0xffffffffu, low);
        // 2^up brings the largest query to [2^14, 2^15), within what an fp32 factor can say
        const int up = min(127 + 14 - ew, 110);
        float mul[NB];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) mul[nb] = __uint_as_float(static_cast<uint32_t>(127 + up) << 23);
        qscale = a.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 - up) << 23);
        if (uneven) {
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            const int own = er[nb] > 0 ? min(127 + 14 - er[nb], 110) : up;
            mul[nb] = __uint_as_float(static_cast<uint32_t>(127 + own) << 23);
#pragma unroll
            for (int e = 0; e < 2; ++e)  // (2^-126 apart: as good as 0)
              rowscale[2 * nb + e] = __uint_as_float(
                  static_cast<uint32_t>(max(127 + up - __shfl_sync(0xffffffffu, own, 4 * (2 * qd + e)), 0)) << 23);
          }
        }
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            const uint32_t x = qb[ks][nb][0], y = qb[ks][nb][1];
            const uint32_t xf = pack_f16x2(__uint_as_float(x << 16) * mul[nb], __uint_as_float(x & 0xffff0000u) * mul[nb]);
            const uint32_t yf = pack_f16x2(__uint_as_float(y << 16) * mul[nb], __uint_as_float(y & 0xffff0000u) * mul[nb]);
            // int8 codes pair up as bytes 0, 2 and 1, 3; e4m3 ones as 0, 1 and 2, 3
            qb[ks][nb][0] = ET == kCacheI8 ? __byte_perm(xf, yf, 0x5410) : xf;
            qb[ks][nb][1] = ET == kCacheI8 ? __byte_perm(xf, yf, 0x7632) : yf;
          }
      }
#pragma unroll
      for (int c = 0; c < KS; ++c)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) o[c][nb][0] = o[c][nb][1] = o[c][nb][2] = o[c][nb][3] = 0.f;
    }

    // ---- scores: s[mb][nb] holds keys 16 mb + gr, + 8 and rows 8 nb + 2 qd, + 1
    landed();
    const uint32_t kt = ring + slot * SL::kItem + k_lane;
    float s[2][NB][4];
    float xc[4];  // factors of the scores of keys gr + 8 i
#pragma unroll
    for (int mb = 0; mb < 2; ++mb)
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) s[mb][nb][0] = s[mb][nb][1] = s[mb][nb][2] = s[mb][nb][3] = 0.f;
    if constexpr (ET == kCacheBf16) {
#pragma unroll
      for (int ks = 0; ks < KS; ++ks)
#pragma unroll
        for (int mb = 0; mb < 2; ++mb) {
          uint32_t ka[4];
          ldsm_x4((kt ^ (32u * ks)) + 16 * ROW * mb, ka);
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) pg_mma<ET>(s[mb][nb], ka, qb[ks][nb][0], qb[ks][nb][1]);
        }
#pragma unroll
      for (int i = 0; i < 4; ++i) xc[i] = a.scale_log2;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) xc[i] = scales[slot * kPgKeys + gr + 8 * i] * qscale;
#pragma unroll
      for (int half = 0; half < KS / 4; ++half)
#pragma unroll
        for (int mb = 0; mb < 2; ++mb) {
          uint32_t c[2][4];  // keys gr and gr + 8 of the 16
#pragma unroll
          for (int i = 0; i < 2; ++i)
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(c[i][0]), "=r"(c[i][1]), "=r"(c[i][2]), "=r"(c[i][3])
                         : "r"((kt ^ (64u * half)) + (16 * mb + 8 * i) * ROW));
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t ka[4];
            if constexpr (ET == kCacheI8) {
              ka[0] = i8_to_f16(c[0][i]);
              ka[1] = i8_to_f16(c[1][i]);
              ka[2] = i8_to_f16(c[0][i] >> 8);
              ka[3] = i8_to_f16(c[1][i] >> 8);
            } else {
              ka[0] = e4m3_to_f16<0>(c[0][i]);
              ka[1] = e4m3_to_f16<0>(c[1][i]);
              ka[2] = e4m3_to_f16<1>(c[0][i]);
              ka[3] = e4m3_to_f16<1>(c[1][i]);
            }
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) pg_mma<ET>(s[mb][nb], ka, qb[4 * half + i][nb][0], qb[4 * half + i][nb][1]);
          }
        }
    }
    if (ET != kCacheBf16 && uneven)
#pragma unroll
      for (int mb = 0; mb < 2; ++mb)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[mb][nb][e] *= rowscale[2 * nb + (e & 1)];
    release();
    if (odd) load_v();
    else load_k();
    landed();  // V, and its scales

    // ---- weights
    const uint32_t vt = ring + slot * SL::kItem;
    const bool masked = tile.p0 + 16 > minlim || tile.p1 + 16 > minlim;  // the same for the whole warp
    uint32_t seen = 0xffffffffu;  // bit 8 mb + 4 nb + e: this lane's s[mb][nb][e] is of a visible key
    if (masked) {
      seen = 0u;
#pragma unroll
      for (int mb = 0; mb < 2; ++mb)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if ((mb ? tile.p1 : tile.p0) + gr + 8 * (e >> 1) < lim[2 * nb + (e & 1)]) seen |= 1u << (8 * mb + 4 * nb + e);
    }
    float vs[4] = {1.f, 1.f, 1.f, 1.f};
    if constexpr (ET != kCacheBf16) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        vs[i] = scales[slot * kPgKeys + gr + 8 * i];
        // A row of zeros: its codes are 0 and its term counts in l alone.  It holds E near
        // its score, or l would overflow, but must not crowd out the other weights' bits.
        if (vs[i] == 0.f) vs[i] = 0x1p-80f;
      }
    }
    float w[2][NB][4], lt[NR], top;
    auto weigh = [&](auto with_mask) {  // w_j and their sums against E as it is
      constexpr bool kMask = decltype(with_mask)::value;
      top = 0.f;
#pragma unroll
      for (int i = 0; i < NR; ++i) lt[i] = 0.f;
#pragma unroll
      for (int mb = 0; mb < 2; ++mb)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const bool hide = kMask && !((seen >> (8 * mb + 4 * nb + e)) & 1u);
            // (without a reference 2^x stands for 2^(x - E): 0, as -inf is all that a row can have there, or NaN)
            const float ref = E[2 * nb + (e & 1)], r0 = kMask && ref == -INFINITY ? 0.f : ref;
            float p = fast_exp2(fmaf(s[mb][nb][e], xc[2 * mb + (e >> 1)], -r0));
            if (hide) p = 0.f;
            lt[2 * nb + (e & 1)] += p;
            if constexpr (ET != kCacheBf16) p *= vs[2 * mb + (e >> 1)];
            if (hide) p = 0.f;  // an unseen key's scale may be anything
            w[mb][nb][e] = p;
          }
          top = fmax3(fmax3(top, w[mb][nb][0], w[mb][nb][1]), w[mb][nb][2], w[mb][nb][3]);
        }
      // Values of tiny scales weigh little and count in l in full: its terms move E at
      // 2^104 too.  (An E just set leaves a lane's four at 2^102 at most, see below.)
      if constexpr (ET != kCacheBf16)
#pragma unroll
        for (int i = 0; i < NR; ++i) top = fmaxf(top, lt[i] * (kPgLazy<ET> * 0x1p-104f));
    };
    bool raise = (flags & kPgFirst) || unset;  // (E = -inf there)
    if (!raise) {
      if (masked) weigh(std::true_type{});
      else weigh(std::false_type{});
      raise = __any_sync(0xffffffffu, top > kPgLazy<ET>);
    }
    if (raise) {
      unset = false;
#pragma unroll
      for (int i = 0; i < NR; ++i) {
        float y = -INFINITY;  // largest x_j + log2 vs_j of the row's visible keys
#pragma unroll
        for (int mb = 0; mb < 2; ++mb)
#pragma unroll
          for (int k8 = 0; k8 < 2; ++k8) {
            const int e = 2 * k8 + (i & 1);
            float x = s[mb][i >> 1][e] * xc[2 * mb + k8];
            // (no term of l above 2^100, or l could overflow; an append's scales are 2^-109 or more)
            if constexpr (ET != kCacheBf16) x += fmaxf(__log2f(vs[2 * mb + k8]), kPgStart<ET> - 100.f);
            if ((seen >> (8 * mb + 4 * (i >> 1) + e)) & 1u) y = fmaxf(y, x);
          }
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, x));
        const float En = fmaxf(E[i], y - kPgStart<ET>);
        const float al = E[i] == -INFINITY ? 0.f : fast_exp2(E[i] - En);
        E[i] = En;
        unset |= lim[i] > 0 && En == -INFINITY;
        l[i] *= al;
#pragma unroll
        for (int c = 0; c < KS; ++c) {
          o[c][i >> 1][i & 1] *= al;
          o[c][i >> 1][2 + (i & 1)] *= al;
        }
      }
      unset = __any_sync(0xffffffffu, unset);
      weigh(std::true_type{});
    }
#pragma unroll
    for (int i = 0; i < NR; ++i) l[i] += lt[i];

    // ---- o += V^T W
    bool slow = false;
    if (ET == kCacheBf16 && masked) {
      // A key that a row does not see may hold anything (old tokens, memory never
      // written): 0 * NaN must not reach the sum.
      uint32_t big = 0;
#pragma unroll
      for (int c = 0; c < KS; ++c)
#pragma unroll
        for (int kh = 0; kh < 2; ++kh) {
          uint32_t r4[4];
          ldsm_x4(vt + pg_off<ROW>(16 * kh + (lane & 15), 2 * c + (lane >> 4)), r4);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            big |= (r4[j] & 0x7f80u) == 0x7f80u;
            big |= (r4[j] & 0x7f800000u) == 0x7f800000u;
          }
        }
      slow = __any_sync(0xffffffffu, big != 0);
    }
    if (ET == kCacheE4M3 && masked) {
      // The same of e4m3, whose one magnitude without a value a visible row does not
      // hold: it becomes 0 (a team's warps may all do so).  int8 codes are all finite.
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        const uint32_t at = vt + 16 * (lane + 32 * i);
        uint32_t x[4], any = 0;
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]) : "r"(at));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t nan = ((x[j] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;  // bit 7 of such bytes
          any |= nan;
          x[j] &= ~(nan | (nan - (nan >> 7)));
        }
        if (any)
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3])
                       : "memory");
      }
      __syncwarp();
    }
    if (!slow) {
      uint32_t pb[2][3][NB][2];
#pragma unroll
      for (int kh = 0; kh < 2; ++kh)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int k8 = 0; k8 < 2; ++k8) {
            uint32_t t[3];
            split_pair<ET>(w[kh][nb][2 * k8], w[kh][nb][2 * k8 + 1], !a.out_bf16, t);
            pb[kh][0][nb][k8] = transpose_8x8(t[0]);
            pb[kh][1][nb][k8] = transpose_8x8(t[1]);
            pb[kh][2][nb][k8] = ET == kCacheBf16 && !a.out_bf16 ? transpose_8x8(t[2]) : 0u;
          }
#pragma unroll
      for (int c = 0; c < KS; ++c) {  // 16 output columns
        float part[NB][4];  // the tile's sums
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) part[nb][0] = part[nb][1] = part[nb][2] = part[nb][3] = 0.f;
#pragma unroll
        for (int kh = 0; kh < 2; ++kh) {
          uint32_t va[4];
          if constexpr (ET == kCacheBf16) {
            ldsm_x4_t(((vt + v_lane) ^ (32u * c)) + 16 * ROW * kh, va);
          } else {
            // 16-bit units of a transposed 8x8 load are two neighbouring codes of a
            // key: the even columns of the 16 make rows 0 - 7, the odd ones rows 8 - 15
            uint32_t r2[2];
            asm volatile("ldmatrix.sync.aligned.m8n8.x2.trans.shared.b16 {%0, %1}, [%2];"
                         : "=r"(r2[0]), "=r"(r2[1])
                         : "r"(((vt + v_lane) ^ (16u * c)) + 16 * ROW * kh));
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              if constexpr (ET == kCacheI8) {
                va[2 * j] = i8_to_f16(r2[j]);
                va[2 * j + 1] = i8_to_f16(r2[j] >> 8);
              } else {
                const uint32_t eo = __byte_perm(r2[j], 0u, 0x3120);  // bytes 0, 2, 1, 3
                va[2 * j] = e4m3_to_f16<0>(eo);
                va[2 * j + 1] = e4m3_to_f16<1>(eo);
              }
            }
          }
#pragma unroll
          for (int term = 0; term < 2; ++term)
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) pg_mma<ET>(part[nb], va, pb[kh][term][nb][0], pb[kh][term][nb][1]);
          if (ET == kCacheBf16 && !a.out_bf16)
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) pg_mma<ET>(part[nb], va, pb[kh][2][nb][0], pb[kh][2][nb][1]);
        }
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int e = 0; e < 4; e += 2)
            f2_unpack(f2_add(f2_pack(o[c][nb][e], o[c][nb][e + 1]), f2_pack(part[nb][e], part[nb][e + 1])), o[c][nb][e],
                      o[c][nb][e + 1]);
      }
    } else {
      // key by key, each row taking only the keys that it sees
#pragma unroll
      for (int mb = 0; mb < 2; ++mb)
#pragma unroll
        for (int k8 = 0; k8 < 2; ++k8)
          for (int x = 0; x < 8; ++x) {
            const int src = 4 * x + qd, j = 16 * mb + 8 * k8 + x;
            const uint32_t sn = __shfl_sync(0xffffffffu, seen, src);
#pragma unroll
            for (int i = 0; i < NR; ++i) {
              const int e = 2 * k8 + (i & 1);
              const float p = __shfl_sync(0xffffffffu, w[mb][i >> 1][e], src);
              if (!((sn >> (8 * mb + 4 * (i >> 1) + e)) & 1u)) continue;
#pragma unroll
              for (int c = 0; c < KS; ++c)
#pragma unroll
                for (int d8 = 0; d8 < 2; ++d8) {
                  uint16_t v;
                  asm volatile("ld.shared.b16 %0, [%1];" : "=h"(v) : "r"(vt + pg_off<ROW>(j, 2 * c + d8) + 2 * gr));
                  o[c][i >> 1][2 * d8 + (i & 1)] = fmaf(p, __uint_as_float(static_cast<uint32_t>(v) << 16), o[c][i >> 1][2 * d8 + (i & 1)]);
                }
            }
          }
    }
    release();
    if (odd) load_k();
    else load_v();
    if (lane == 0) mbar_arrive(qempty + 8u * cq);  // (tile is in registers)
    if (++cq == kPgQueue) cq = 0;

    // ---- the end of the pair, or of this team's part of it
    if (flags & kPgLast) {
      const long long u = static_cast<long long>(team) * gridDim.x + blockIdx.x;
#pragma unroll
      for (int i = 0; i < NR; ++i) {
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], x);
        const int r = row0 + 8 * (i >> 1) + 2 * qd + (i & 1);
        if (r >= a.rows) continue;
        const bool has = lim[i] > 0 && !(l[i] == 0.f);  // a NaN sum stays
        const int nb = i >> 1, e = i & 1;
        if (flags & kPgWhole) {
          const long long row =
              (static_cast<long long>(tile.b) * a.bt.T + r / a.groups) * a.Hq + tile.h * a.groups + r % a.groups;
          if (!RA_IN_BOUNDS(row, static_cast<long long>(a.bt.B) * a.bt.T * a.Hq)) continue;
          const float inv = has ? 1.f / l[i] : 0.f;
#pragma unroll
          for (int c = 0; c < KS; ++c) {
            const float x = has ? o[c][nb][e] * inv : 0.f, y = has ? o[c][nb][2 + e] * inv : 0.f;
            if constexpr (ET == kCacheBf16) {
              pg_store1(a, row, D, 16 * c + gr, x);
              pg_store1(a, row, D, 16 * c + 8 + gr, y);
            } else {
              pg_store2(a, row, D, 16 * c + 2 * gr, x, y);
            }
          }
          if (gr == 0) a.lse[row] = has ? (E[i] + log2f(l[i])) * 0.6931471805599453f : -INFINITY;
        } else {
          const long long pr = (2 * u + (flags & kPgOwner ? 1 : 0)) * a.rows + r;
          if (!RA_IN_BOUNDS(pr, static_cast<long long>(gridDim.x) * teams * 2 * a.rows)) continue;
          float* dst = a.part_o + pr * D;
#pragma unroll
          for (int c = 0; c < KS; ++c) {
            if constexpr (ET == kCacheBf16) {
              dst[16 * c + gr] = o[c][nb][e];
              dst[16 * c + 8 + gr] = o[c][nb][2 + e];
            } else {
              *reinterpret_cast<float2*>(dst + 16 * c + 2 * gr) = make_float2(o[c][nb][e], o[c][nb][2 + e]);
            }
          }
          if (gr == 0) a.part_ml[pr] = has ? make_float2(E[i], l[i]) : make_float2(-INFINITY, 0.f);
        }
      }
    }
  }
  copies_wait_all();  // none is left in the normal course
}

// Joins the parts of the cut pairs: with M = max E_i over the parts,
// l = sum 2^(E_i - M) l_i, out = sum 2^(E_i - M) o_i / l.  A CTA of NW warps does
// `COLS` columns of NW / WPR rows, WPR warps to a row, each with every WPR-th part.
// Where rows are few and their parts many (592 for one token against 1M keys),
// 32 warps share a row and the row's columns are spread over CTAs, 32 to each: a
// warp's parts then fit one or two batches of loads.  Where the rows alone
// fill the GPU a warp does a whole one.  Every part is read once and in a fixed
// order: the result does not depend on scheduling.
template <int D, int COLS, int WPR, int NW>
__global__ void __launch_bounds__(32 * NW) paged_combine_kernel(const __grid_constant__ PagedArgs a, int max_teams) {
  constexpr int kPer = COLS / 32, kBatch = WPR == 32 ? 8 : 16 / kPer;
  __shared__ float s_acc[WPR == 1 ? 1 : NW][COLS], s_l[NW], s_m[NW];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = COLS * (blockIdx.x % (D / COLS)) + kPer * lane;
  const long long id = static_cast<long long>(blockIdx.x / (D / COLS)) * (NW / WPR) + warp / WPR;
  const int w0 = warp % WPR;
  chain_launches();
  const long long pairs = static_cast<long long>(a.bt.B) * a.bt.Hkv;
  if (id >= pairs * a.rows) return;
  const long long pair = id / a.rows;
  const int r = static_cast<int>(id % a.rows);
  const int2 cut = a.cut[pair];
  if (cut.x < 0 || cut.y <= cut.x || cut.y >= max_teams) return;  // the last: records of a call that timed out
  auto part = [&](int t) { return (2LL * t + (t == cut.x ? 1 : 0)) * a.rows + r; };
  // this warp's parts w0, w0 + WPR, ... against their own maximum
  float M = -INFINITY, L = 0.f, acc[kPer];
#pragma unroll
  for (int e = 0; e < kPer; ++e) acc[e] = 0.f;
  for (int t0 = cut.x + w0; t0 <= cut.y; t0 += WPR * kBatch) {
    float v[kBatch][kPer];
    float2 ml[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int t = t0 + WPR * k;
      ml[k] = make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int e = 0; e < kPer; ++e) v[k][e] = 0.f;
      if (t <= cut.y && RA_IN_BOUNDS(part(t), 2LL * max_teams * a.rows)) {
        ml[k] = a.part_ml[part(t)];
        const float* src = a.part_o + part(t) * D + col;
#pragma unroll
        for (int e = 0; e < kPer; ++e) v[k][e] = src[e];
      }
    }
    float mb = M;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) mb = fmaxf(mb, ml[k].x);
    const float old = M == -INFINITY ? 0.f : fast_exp2(M - mb);
    M = mb;
    L *= old;
#pragma unroll
    for (int e = 0; e < kPer; ++e) acc[e] *= old;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      if (ml[k].y == 0.f) continue;  // a part in which the row sees no key
      const float w = ml[k].x == -INFINITY ? 1.f : fast_exp2(ml[k].x - M);  // -inf with a sum: NaN scores
      L = fmaf(w, ml[k].y, L);
#pragma unroll
      for (int e = 0; e < kPer; ++e) acc[e] = fmaf(w, v[k][e], acc[e]);
    }
  }
  if constexpr (WPR > 1) {
#pragma unroll
    for (int e = 0; e < kPer; ++e) s_acc[warp][kPer * lane + e] = acc[e];
    if (lane == 0) {
      s_l[warp] = L;
      s_m[warp] = M;
    }
    __syncthreads();
    if (w0 != 0) return;
    // lane w: the factor of warp w's result
    const float mw = lane < WPR ? s_m[warp + lane] : -INFINITY;
    M = mw;
#pragma unroll
    for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    const float lw = lane < WPR ? s_l[warp + lane] : 0.f;
    const float fw = lw == 0.f ? 0.f : mw == -INFINITY ? 1.f : fast_exp2(mw - M);
    L = fw * lw;
#pragma unroll
    for (int o = 16; o; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
#pragma unroll
    for (int e = 0; e < kPer; ++e) acc[e] = 0.f;
#pragma unroll 8
    for (int w = 0; w < WPR; ++w) {
      const float f = __shfl_sync(0xffffffffu, fw, w);
      if (f != 0.f)
#pragma unroll
        for (int e = 0; e < kPer; ++e) acc[e] = fmaf(f, s_acc[warp + w][kPer * lane + e], acc[e]);
    }
  }
  const bool has = !(L == 0.f);
  const float inv = has ? 1.f / L : 0.f;
  const int b = static_cast<int>(pair / a.bt.Hkv), h = static_cast<int>(pair % a.bt.Hkv);
  const long long row = (static_cast<long long>(b) * a.bt.T + r / a.groups) * a.Hq + h * a.groups + r % a.groups;
  if (!RA_IN_BOUNDS(row, static_cast<long long>(a.bt.B) * a.bt.T * a.Hq)) return;
  if constexpr (kPer == 1)
    pg_store1(a, row, D, col, has ? acc[0] * inv : 0.f);
  else
#pragma unroll
    for (int e = 0; e < kPer; e += 2)
      pg_store2(a, row, D, col + e, has ? acc[e] * inv : 0.f, has ? acc[e + 1] * inv : 0.f);
  if (lane == 0 && col == 0) a.lse[row] = has ? (M + log2f(L)) * 0.6931471805599453f : -INFINITY;
}

}  // namespace ra
