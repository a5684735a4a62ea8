// paged_decode.cuh - attention of a few new tokens over a paged key-value
// cache (bf16, int8 or e4m3), all of it or only selected pages.
//
// TokenRing review (pith.science, arXiv 2412.20501), "Reading between the
// lines": the decode phase as KV-cache chunking, partial results joined by
// their log-sum-exp.  Here a chunk is whatever run of the cache one team of
// warps walks, and it may begin and end anywhere in a sequence.
//
// Mathematics, per query row (s = 1 / sqrt(D), everything in fp32):
//     x_j = s (q . k_j),  m = max x_j,  l = sum e^(x_j - m),  o = sum e^(x_j - m) v_j,
//     out = o / l,  lse = m + ln l,
// with the running (m, l, o) rescaled whenever m grows.  For an 8-bit cache the
// codes are turned into bf16 (exactly: 8 significant bits at most) and the
// scales enter as factors: x_j = (s ks_j) (q . code_j), and e^(x_j - m) vs_j is the
// weight of v's codes.  The weights go to the tensor core as two bf16 terms
// (their rounding and what it left: 16 bits, an error of at most 2^-17), or
// three for an fp32 output (24 bits): a single bf16 weight (2^-9) would cost
// as much accuracy as the output's own rounding.
//
// Bound by HBM: a cached element meets the groups * Tq (<= 64) query rows of its
// KV head and is used once.  So the cache is streamed once by TMA through
// rings of shared memory, and the products are mma.sync on tiles of 16 rows.
//
// Work split: the cache of all (sequence, KV head) pairs, cut into tiles of 32
// keys, is one line of tiles (sequence-major, then head, then position).  The
// lengths are on the device, so each team works out the line's length from
// them and takes an equal run of it; runs cross sequence borders, so a batch
// of one 100k and many short sequences is as even as a uniform one, with
// one grid shape for all lengths (a captured graph replays with new ones).
// A team's run covers whole (sequence, head) pairs, written out directly, and
// at most two cut ones (its first and last), left as (m, l, o) in the workspace
// for the combine kernel, which knows each cut pair from a record that the
// team holding its first tile writes.
//
// A team is one warp for up to 16 query rows, 2 or 4 warps for up to 32 or 64
// (each warp one 16-row tile; the team shares its ring).  The warps of a team
// never meet at a barrier with other teams: softmax statistics are per warp
// (four lanes to a row), P goes from the score accumulators to the next
// product's operand registers without touching shared memory.
#pragma once

#include "attn_fwd.cuh"
#include "decode.cuh"
#include "paged.cuh"

namespace ra {

constexpr int kPgWarps = 8;
constexpr int kPgThreads = 32 * kPgWarps;
constexpr int kPgKeys = 32;       // keys of a tile
constexpr int kPgRing = 24576;    // ring bytes per warp
constexpr int kPgSlots = 8;       // ring items per warp, at most
constexpr int kPgNone = 0x7fffff00;  // position of a key that no row sees

struct PagedArgs {
  PagedBatch bt;  // T = Tq
  int Hq, groups, rows, causal;
  int R;         // warps per team: 16-row tiles of the query rows of one KV head
  int slots;     // ring items per team
  int min_tiles; // a team's run is at least this long
  int n_sel;
  const int* selected;  // [B][Hkv][n_sel] or null
  float scale_log2;
  const __nv_bfloat16* q;  // [B][Tq][Hq][D]
  const float* k_scales;
  const float* v_scales;
  float* part_o;    // [teams][2][rows][D]
  float2* part_ml;  // [teams][2][rows]: m (log2 units), l
  int2* cut;        // [B * Hkv]: first and last team of a cut pair; first < 0: not cut
  void* out;        // [B][Tq][Hq][D]
  int out_bf16;
  float* lse;
};

template <int D, int ET>
struct PgSmem {
  static constexpr int kElem = ET == kCacheBf16 ? 2 : 1;
  static constexpr int kItem = kPgKeys * D * kElem;  // one tile of K or of V
  static constexpr int kRowBytes = D * kElem < 128 ? D * kElem : 128;
  static constexpr int kScale = kPgWarps * kPgRing;  // fp32 [64 slots][32]
  static constexpr int kMeta = kScale + kPgWarps * kPgSlots * kPgKeys * 4;
  static constexpr int kFull = kMeta + kPgWarps * kPgSlots * 8;
  static constexpr int kEmpty = kFull + kPgWarps * kPgSlots * 8;
  static constexpr int kAbort = kEmpty + kPgWarps * kPgSlots * 8;
  static constexpr int kBytes = kAbort + 16 + 1024;  // + slack to align the base to 1024
};

// Byte offset of the 16-byte chunk c of key j in a tile that TMA wrote with
// 128-byte swizzle (64-byte for rows of 64 bytes); a bf16 tile of D = 128 is two
// halves of 64 columns.
template <int D, int ET>
__device__ __forceinline__ uint32_t pg_off(int j, int c) {
  if constexpr (PgSmem<D, ET>::kRowBytes == 128)
    return (c >> 3) * (kPgKeys * 128) + j * 128 + (((c & 7) ^ (j & 7)) << 4);
  else
    return j * 64 + ((c ^ ((j >> 1) & 3)) << 4);
}

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* m, int c0, int c1, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(c0), "r"(c1), "r"(bar)
      : "memory");
}

// Untiled copy of a multiple of 16 bytes, both ends 16-byte aligned; no multicast.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
               : "memory");
}

__device__ __forceinline__ uint32_t bf16x2_sub(uint32_t a, uint32_t b) {
  __nv_bfloat162 r = __hsub2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
  return *reinterpret_cast<uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t bf16x2_mul(uint32_t a, uint32_t b) {
  __nv_bfloat162 r = __hmul2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
  return *reinterpret_cast<uint32_t*>(&r);
}

// The codes in bytes 0 and 2 of w as two bf16 values, exactly.
//   int8: 128 + (low 7 bits) and 128 + 128 (sign bit) are bf16 bit patterns
//   (0x4300 | bits); their difference is the signed value.
//   e4m3: sign, exponent and mantissa moved into bf16's fields, times
//   2^(127 - 7) (0x7b80), which covers the subnormal codes too.
template <int ET>
__device__ __forceinline__ uint32_t codes_to_bf16(uint32_t w) {
  if constexpr (ET == kCacheI8)
    return bf16x2_sub((w & 0x007f007fu) | 0x43004300u, (w & 0x00800080u) | 0x43004300u);
  else
    return bf16x2_mul(((w << 4) & 0x07f007f0u) | ((w << 8) & 0x80008000u), 0x7b807b80u);
}

// Tiles of one (sequence, KV head) pair.
__device__ __forceinline__ int pg_tiles(const PagedArgs& a, int len) {
  if (a.selected == nullptr) return (len + kPgKeys - 1) / kPgKeys;
  const int pages = (len + (1 << a.bt.page_shift) - 1) >> a.bt.page_shift;
  return ((min(a.n_sel, pages) << a.bt.page_shift) + kPgKeys - 1) / kPgKeys;
}

// A place on the line of tiles.
struct PgWalk {
  int b, h, t, nt;
  SeqLen s;
};

// First sequence at or behind b that has tiles (whole warp).
__device__ __forceinline__ void pg_seek(const PagedArgs& a, PgWalk& w, int b, int lane) {
  for (; b < a.bt.B; b += 32) {
    const int n = b + lane < a.bt.B ? a.bt.seq_lens[b + lane] : 0;
    const uint32_t some = __ballot_sync(0xffffffffu, n > 0);
    if (some) {
      b += __ffs(some) - 1;
      break;
    }
  }
  w.b = min(b, a.bt.B);
  w.h = w.t = 0;
  w.nt = 0;
  if (w.b < a.bt.B) {
    w.s = seq_len_of(a.bt, w.b);
    w.nt = pg_tiles(a, w.s.len);
  }
}

__device__ __forceinline__ void pg_next(const PagedArgs& a, PgWalk& w, int lane) {
  if (++w.t < w.nt) return;
  w.t = 0;
  if (++w.h < a.bt.Hkv) return;
  pg_seek(a, w, w.b + 1, lane);
}

// Tiles of the whole line (whole warp).
__device__ __forceinline__ long long pg_total(const PagedArgs& a, int lane) {
  long long n = 0;
  for (int b = lane; b < a.bt.B; b += 32) n += pg_tiles(a, seq_len_of(a.bt, b).len);
#pragma unroll
  for (int o = 16; o; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
  return n * a.bt.Hkv;
}

// The place of tile f of the line, f below pg_total (whole warp).
__device__ __forceinline__ void pg_locate(const PagedArgs& a, long long f, PgWalk& w, int lane) {
  long long before = 0;
  for (int b0 = 0; b0 < a.bt.B; b0 += 32) {
    const int b = b0 + lane;
    const long long mine = b < a.bt.B ? static_cast<long long>(pg_tiles(a, seq_len_of(a.bt, b).len)) * a.bt.Hkv : 0;
    long long upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += x;
    }
    const uint32_t past = __ballot_sync(0xffffffffu, before + upto > f);
    if (past) {
      const int l = __ffs(past) - 1;
      const long long rel = f - before - __shfl_sync(0xffffffffu, upto - mine, l);
      w.b = b0 + l;
      w.s = seq_len_of(a.bt, w.b);
      w.nt = pg_tiles(a, w.s.len);
      w.h = static_cast<int>(rel / w.nt);
      w.t = static_cast<int>(rel % w.nt);
      return;
    }
    before += __shfl_sync(0xffffffffu, upto, 31);
  }
}

// One output element pair or quad at columns d.. of a row.
__device__ __forceinline__ void pg_store2(const PagedArgs& a, long long row, int D, int d, float x, float y) {
  if (a.out_bf16)
    *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(a.out) + row * D + d) = pack_bf16x2(x, y);
  else
    *reinterpret_cast<float2*>(static_cast<float*>(a.out) + row * D + d) = make_float2(x, y);
}

template <int D, int ET>
__global__ void __launch_bounds__(kPgThreads, 1)
    paged_partial_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                         const __grid_constant__ PagedArgs a) {
  using SL = PgSmem<D, ET>;
  constexpr int NT = D / 8;    // n8 blocks of the output
  constexpr int KS = D / 16;   // k16 steps of the score product
  extern __shared__ uint8_t pg_raw[];
  uint8_t* smem = pg_raw + ((1024u - (smem_u32(pg_raw) & 1023u)) & 1023u);
  const uint32_t sb = smem_u32(smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int gr = lane >> 2, qd = lane & 3;  // fragment row and column pair of this lane
  const int teams = kPgWarps / a.R, team = warp / a.R, rt = warp % a.R;
  const bool leader = rt == 0;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + SL::kAbort);
  const int slots = a.slots;
  const uint32_t ring = sb + team * a.R * kPgRing;
  const int slot0 = team * slots;  // this team's first barrier, scale row and meta entry
  const uint32_t full = sb + SL::kFull + 8u * slot0, empty = sb + SL::kEmpty + 8u * slot0;
  int2* meta = reinterpret_cast<int2*>(smem + SL::kMeta) + slot0;

  // the combine kernel may be brought onto the SMs; it waits for this grid's end itself
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (tid == 0) {
    *abort_flag = grid_timed_out() ? 1 : 0;
    for (int i = 0; i < teams * slots; ++i) {
      mbar_init(sb + SL::kFull + 8u * i, 1);
      mbar_init(sb + SL::kEmpty + 8u * i, a.R);
    }
    fence_mbar_init();
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  __syncthreads();
  if (*abort_flag) return;

  // sequences without a tile: their rows are empty
  for (int b = blockIdx.x * kPgWarps + warp; b < a.bt.B; b += gridDim.x * kPgWarps) {
    if (pg_tiles(a, seq_len_of(a.bt, b).len) > 0) continue;
    const long long r0 = static_cast<long long>(b) * a.bt.T * a.Hq, n = static_cast<long long>(a.bt.T) * a.Hq;
    for (long long i = lane; i < n * (D / 2); i += 32) pg_store2(a, r0 + i / (D / 2), D, 2 * static_cast<int>(i % (D / 2)), 0.f, 0.f);
    for (long long i = lane; i < n; i += 32) a.lse[r0 + i] = -INFINITY;
    for (int h = lane; h < a.bt.Hkv; h += 32) a.cut[static_cast<long long>(b) * a.bt.Hkv + h] = make_int2(-1, -1);
  }

  // this team's run [f0, f1) of the line
  const long long total = pg_total(a, lane);
  const long long U = static_cast<long long>(gridDim.x) * teams;
  const long long u = static_cast<long long>(team) * gridDim.x + blockIdx.x;
  long long run = (total + U - 1) / U;
  if (run < a.min_tiles) run = a.min_tiles;
  const long long f0 = u * run, f1 = min(f0 + run, total);
  if (f0 >= f1) return;
  PgWalk cw;
  pg_locate(a, f0, cw, lane);

  // ------------------------------------------------ loads (the leader warp)
  // Lane i of the leader holds the cache row and the position of the 16-key
  // unit ubase + i of the producer's pair (32 units: 16 tiles).
  PgWalk pw = cw;
  long long pf = f0;
  int issued = 0, pslot = 0, ubase = 0, ent_row = 0, ent_pos = kPgNone;
  uint32_t pphase = 0;
  const int ps = 1 << a.bt.page_shift;
  auto load_entries = [&]() {
    ubase = 2 * pw.t;
    const long long key = 16LL * (ubase + lane);
    const int in_page = static_cast<int>(key & (ps - 1));
    int logical = -1;
    if (a.selected == nullptr) {
      if (key < pw.s.len) logical = static_cast<int>(key >> a.bt.page_shift);
    } else {
      const int pages = (pw.s.len + ps - 1) >> a.bt.page_shift;
      const int idx = static_cast<int>(key >> a.bt.page_shift);
      if (idx < min(a.n_sel, pages)) {
        const int* sel = a.selected + (static_cast<long long>(pw.b) * a.bt.Hkv + pw.h) * a.n_sel;
        logical = sel[idx];
        const int prev = idx > 0 ? sel[idx - 1] : -1;
        if (logical != -1 && (logical < 0 || logical >= pages || logical <= prev)) {
          set_status(RA_ERR_DEVICE_BOUNDS);
          logical = -1;
        }
      }
    }
    ent_row = 0;
    ent_pos = kPgNone;
    if (logical >= 0) {
      const int page = page_of(a.bt, pw.b, logical);
      if (page >= 0) {
        ent_row = ((page * a.bt.Hkv + pw.h) << a.bt.page_shift) + in_page;
        ent_pos = (logical << a.bt.page_shift) + in_page;
      }
    }
  };
  // Issues the next item (K, then V of each tile); false when the ring never freed up.
  auto issue = [&]() -> bool {
    if (pf >= f1) return true;
    const bool is_v = issued & 1;
    if (a.R > 1 && issued >= slots &&
        !__all_sync(0xffffffffu, mbar_wait(empty + 8u * pslot, pphase ^ 1u, abort_flag)))
      return false;
    const int l0 = 2 * pw.t - ubase;
    const int r0 = __shfl_sync(0xffffffffu, ent_row, l0), r1 = __shfl_sync(0xffffffffu, ent_row, l0 + 1);
    const int p0 = __shfl_sync(0xffffffffu, ent_pos, l0), p1 = __shfl_sync(0xffffffffu, ent_pos, l0 + 1);
    if (lane == 0) {
      const uint32_t bar = full + 8u * pslot, dst = ring + pslot * SL::kItem;
      const CUtensorMap* tm = is_v ? &tmV : &tmK;
      meta[pslot] = make_int2(p0, p1);
      fence_proxy_async_smem();  // the ring slot's earlier reads precede the copy into it
      mbar_expect_tx(bar, SL::kItem + (ET == kCacheBf16 ? 0 : kPgKeys * 4));
#pragma unroll
      for (int half = 0; half < SL::kItem / (kPgKeys * SL::kRowBytes); ++half) {
        const uint32_t d = dst + half * kPgKeys * SL::kRowBytes;
        tma_load_2d(d, tm, half * 64, r0, bar);
        if (ps == 16) tma_load_2d(d + 16 * SL::kRowBytes, tm, half * 64, r1, bar);
      }
      if constexpr (ET != kCacheBf16) {
        const float* sc = is_v ? a.v_scales : a.k_scales;
        const uint32_t sd = sb + SL::kScale + (slot0 + pslot) * kPgKeys * 4;
        if (ps == 16) {
          bulk_load(sd, sc + r0, 64, bar);
          bulk_load(sd + 64, sc + r1, 64, bar);
        } else {
          bulk_load(sd, sc + r0, 128, bar);
        }
      }
    }
    __syncwarp();
    ++issued;
    if (++pslot == slots) {
      pslot = 0;
      pphase ^= 1u;
    }
    if (is_v) {
      const int b = pw.b, h = pw.h;
      ++pf;
      if (pf < f1) {
        pg_next(a, pw, lane);
        if (pw.b != b || pw.h != h || 2 * pw.t >= ubase + 32) load_entries();
      }
    }
    return true;
  };

  bool ok = true;
  if (leader) {
    load_entries();
    for (int i = 0; i < slots; ++i) issue();  // the first round waits for nothing
  }

  // --------------------------------------------------------------- the walk
  int consumed = 0, cslot = 0;
  uint32_t cphase = 0;
  uint32_t qa[KS][4];
  float o[NT][4], m[2], l[2];
  int lim[2], tok[2], minlim = 0;
  auto release = [&]() {  // this warp has read the slot; the next load into it may go out
    __syncwarp();
    if (a.R > 1 && lane == 0) mbar_arrive(empty + 8u * cslot);
    ++consumed;
    if (++cslot == slots) {
      cslot = 0;
      cphase ^= 1u;
    }
    if (leader && ok) ok = issue();
  };
  bool fresh_pair = true;
  for (long long f = f0; f < f1; ++f) {
    if (fresh_pair) {  // the query rows of this (sequence, KV head)
      fresh_pair = false;
      minlim = 0x7fffffff;
#pragma unroll
      for (int hr = 0; hr < 2; ++hr) {
        const int r = 16 * rt + gr + 8 * hr;
        const int t = r / a.groups;
        tok[hr] = r < a.rows ? t : -1;
        const bool real = r < a.rows && t < cw.s.fresh;
        lim[hr] = real ? (a.causal ? cw.s.len - cw.s.fresh + t + 1 : cw.s.len) : 0;
        if (real) minlim = min(minlim, lim[hr]);
        m[hr] = -INFINITY;
        l[hr] = 0.f;
        const __nv_bfloat16* qr = a.q;
        if (r < a.rows)
          qr += ((static_cast<long long>(cw.b) * a.bt.T + t) * a.Hq + cw.h * a.groups + r % a.groups) * D;
        if constexpr (ET == kCacheBf16) {
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) {
            qa[ks][hr] = r < a.rows ? *reinterpret_cast<const uint32_t*>(qr + 16 * ks + 2 * qd) : 0u;
            qa[ks][2 + hr] = r < a.rows ? *reinterpret_cast<const uint32_t*>(qr + 16 * ks + 8 + 2 * qd) : 0u;
          }
        } else {
          // k index of the product: step ks = 4 half + i takes columns 16 (qd + 4 half) + 4 i + {0, 2 | 1, 3}
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) {
            const uint2 w = r < a.rows ? *reinterpret_cast<const uint2*>(qr + 16 * (qd + 4 * (ks >> 2)) + 4 * (ks & 3))
                                       : make_uint2(0u, 0u);
            qa[ks][hr] = __byte_perm(w.x, w.y, 0x5410);
            qa[ks][2 + hr] = __byte_perm(w.x, w.y, 0x7632);
          }
        }
      }
#pragma unroll
      for (int x = 16; x; x >>= 1) minlim = min(minlim, __shfl_xor_sync(0xffffffffu, minlim, x));
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) o[nt][0] = o[nt][1] = o[nt][2] = o[nt][3] = 0.f;
    }

    // ---- scores of the tile's 32 keys
    ok = ok && __all_sync(0xffffffffu, mbar_wait(full + 8u * cslot, cphase, abort_flag));
    if (!ok) break;
    const uint32_t kt = ring + cslot * SL::kItem;
    const int2 pos = meta[cslot];
    float s[4][4];
#pragma unroll
    for (int nb = 0; nb < 4; ++nb) s[nb][0] = s[nb][1] = s[nb][2] = s[nb][3] = 0.f;
    if constexpr (ET == kCacheBf16) {
#pragma unroll
      for (int kp = 0; kp < KS / 2; ++kp)
#pragma unroll
        for (int nb = 0; nb < 4; ++nb) {
          uint32_t kb[4];
          ldsm_x4(kt + pg_off<D, ET>(8 * nb + (lane & 7), 4 * kp + (lane >> 3)), kb);
          mma_16816(s[nb], qa[2 * kp], kb[0], kb[1]);
          mma_16816(s[nb], qa[2 * kp + 1], kb[2], kb[3]);
        }
#pragma unroll
      for (int nb = 0; nb < 4; ++nb)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[nb][e] *= a.scale_log2;
    } else {
#pragma unroll
      for (int half = 0; half < KS / 4; ++half)
#pragma unroll
        for (int nb = 0; nb < 4; ++nb) {
          uint4 w4;
          asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(w4.x), "=r"(w4.y), "=r"(w4.z), "=r"(w4.w)
                       : "r"(kt + pg_off<D, ET>(8 * nb + gr, qd + 4 * half)));
          const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
          for (int i = 0; i < 4; ++i)
            mma_16816(s[nb], qa[4 * half + i], codes_to_bf16<ET>(w[i]), codes_to_bf16<ET>(w[i] >> 8));
        }
      const float* ksc = reinterpret_cast<const float*>(smem + SL::kScale) + (slot0 + cslot) * kPgKeys;
#pragma unroll
      for (int nb = 0; nb < 4; ++nb) {
        const float2 sc = *reinterpret_cast<const float2*>(ksc + 8 * nb + 2 * qd);
        s[nb][0] *= sc.x * a.scale_log2;
        s[nb][1] *= sc.y * a.scale_log2;
        s[nb][2] *= sc.x * a.scale_log2;
        s[nb][3] *= sc.y * a.scale_log2;
      }
    }
    release();

    // ---- mask, running maximum, weights
    const bool masked = pos.x + 16 > minlim || pos.y + 16 > minlim;  // the same for the whole warp
    uint32_t seen = 0xffffu;  // bit 4 nb + e: this lane's score s[nb][e] is of a visible key
    if (masked) {
      seen = 0u;
#pragma unroll
      for (int nb = 0; nb < 4; ++nb)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int kp = (nb < 2 ? pos.x + 8 * nb : pos.y + 8 * (nb - 2)) + 2 * qd + (e & 1);
          if (kp < lim[e >> 1]) seen |= 1u << (4 * nb + e);
          else s[nb][e] = -INFINITY;
        }
    }
    float mx[2];
#pragma unroll
    for (int hr = 0; hr < 2; ++hr) {
      float x = fmaxf(fmaxf(fmaxf(s[0][2 * hr], s[0][2 * hr + 1]), fmaxf(s[1][2 * hr], s[1][2 * hr + 1])),
                      fmaxf(fmaxf(s[2][2 * hr], s[2][2 * hr + 1]), fmaxf(s[3][2 * hr], s[3][2 * hr + 1])));
      x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
      mx[hr] = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
    }
    if (__any_sync(0xffffffffu, mx[0] > m[0] || mx[1] > m[1])) {
#pragma unroll
      for (int hr = 0; hr < 2; ++hr) {
        const float mn = fmaxf(m[hr], mx[hr]);
        const float al = m[hr] == -INFINITY ? 0.f : fast_exp2(m[hr] - mn);  // mn >= m > -inf there
        m[hr] = mn;
        l[hr] *= al;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          o[nt][2 * hr] *= al;
          o[nt][2 * hr + 1] *= al;
        }
      }
    }
#pragma unroll
    for (int hr = 0; hr < 2; ++hr) {
      const float base = m[hr] == -INFINITY ? 0.f : m[hr];
#pragma unroll
      for (int nb = 0; nb < 4; ++nb)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float p = fast_exp2(s[nb][2 * hr + e] - base);
          s[nb][2 * hr + e] = p;
          l[hr] += p;
        }
    }

    // ---- o += P V
    ok = ok && __all_sync(0xffffffffu, mbar_wait(full + 8u * cslot, cphase, abort_flag));
    if (!ok) break;
    const uint32_t vt = ring + cslot * SL::kItem;
    if constexpr (ET != kCacheBf16) {
      const float* vsc = reinterpret_cast<const float*>(smem + SL::kScale) + (slot0 + cslot) * kPgKeys;
#pragma unroll
      for (int nb = 0; nb < 4; ++nb) {
        const float2 sc = *reinterpret_cast<const float2*>(vsc + 8 * nb + 2 * qd);
#pragma unroll
        for (int e = 0; e < 4; ++e)  // a masked key's scale may be anything
          s[nb][e] = (seen >> (4 * nb + e)) & 1u ? s[nb][e] * ((e & 1) ? sc.y : sc.x) : 0.f;
      }
    }
    bool slow = false;
    if (ET == kCacheBf16 && masked) {
      // A row that no query row sees may hold anything (old tokens, memory never
      // written): 0 * NaN must not reach the sum.  Codes of 8 bits are finite.
      uint32_t big = 0;
#pragma unroll
      for (int i = 0; i < NT; i += 2)
#pragma unroll
        for (int kh = 0; kh < 2; ++kh) {
          uint32_t r4[4];
          ldsm_x4_t(vt + pg_off<D, ET>(16 * kh + (lane & 15), i + (lane >> 4)), r4);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            big |= (r4[j] & 0x7f80u) == 0x7f80u;
            big |= (r4[j] & 0x7f800000u) == 0x7f800000u;
          }
        }
      slow = __any_sync(0xffffffffu, big != 0);
    }
    if (!slow) {
#pragma unroll
      for (int kh = 0; kh < 2; ++kh) {
        // the weights as bf16 terms: rounded, the remainder rounded, and once more for an fp32 output
        uint32_t pa[3][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float x = s[2 * kh + (i >> 1)][2 * (i & 1)], y = s[2 * kh + (i >> 1)][2 * (i & 1) + 1];
#pragma unroll
          for (int term = 0; term < 3; ++term) {
            pa[term][i] = pack_bf16x2(x, y);
            x -= __uint_as_float(pa[term][i] << 16);
            y -= __uint_as_float(pa[term][i] & 0xffff0000u);
          }
        }
#pragma unroll
        for (int c = 0; c < NT / 2; ++c) {  // 16 output columns
          uint32_t b[2][2];
          if constexpr (ET == kCacheBf16) {
            uint32_t r4[4];
            ldsm_x4_t(vt + pg_off<D, ET>(16 * kh + (lane & 15), 2 * c + (lane >> 4)), r4);
            b[0][0] = r4[0];
            b[0][1] = r4[1];
            b[1][0] = r4[2];
            b[1][1] = r4[3];
          } else {
            // 16-bit units of a transposed 8x8 load are two neighbouring codes of
            // a key: the even columns of the 16 make one n8 block, the odd ones another
            uint32_t r2[2];
            asm volatile("ldmatrix.sync.aligned.m8n8.x2.trans.shared.b16 {%0, %1}, [%2];"
                         : "=r"(r2[0]), "=r"(r2[1])
                         : "r"(vt + pg_off<D, ET>(16 * kh + (lane & 15), c)));
            b[0][0] = codes_to_bf16<ET>(r2[0]);
            b[0][1] = codes_to_bf16<ET>(r2[1]);
            b[1][0] = codes_to_bf16<ET>(r2[0] >> 8);
            b[1][1] = codes_to_bf16<ET>(r2[1] >> 8);
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            mma_16816(o[2 * c + e], pa[0], b[e][0], b[e][1]);
            mma_16816(o[2 * c + e], pa[1], b[e][0], b[e][1]);
            if (!a.out_bf16) mma_16816(o[2 * c + e], pa[2], b[e][0], b[e][1]);
          }
        }
      }
    } else {
      // key by key, each row taking only the keys that it sees
#pragma unroll
      for (int nb = 0; nb < 4; ++nb)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          for (int x = 0; x < 4; ++x) {
            const int src = (lane & ~3) | x, j = 8 * nb + 2 * x + e;
            const float p0 = __shfl_sync(0xffffffffu, s[nb][e], src), p1 = __shfl_sync(0xffffffffu, s[nb][2 + e], src);
            const uint32_t sn = __shfl_sync(0xffffffffu, seen, src);
            const bool see0 = (sn >> (4 * nb + e)) & 1u, see1 = (sn >> (4 * nb + 2 + e)) & 1u;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              uint32_t w;
              asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w) : "r"(vt + pg_off<D, ET>(j, nt) + 4 * qd));
              const float v0 = __uint_as_float(w << 16), v1 = __uint_as_float(w & 0xffff0000u);
              if (see0) {
                o[nt][0] = fmaf(p0, v0, o[nt][0]);
                o[nt][1] = fmaf(p0, v1, o[nt][1]);
              }
              if (see1) {
                o[nt][2] = fmaf(p1, v0, o[nt][2]);
                o[nt][3] = fmaf(p1, v1, o[nt][3]);
              }
            }
          }
    }
    release();

    // ---- the end of the pair, or of this team's part of it
    if (cw.t + 1 == cw.nt || f + 1 == f1) {
      const long long seg0 = f - cw.t;  // the pair's first tile
      const bool owner = seg0 >= f0, whole = owner && cw.t + 1 == cw.nt;
      if (leader && lane == 0 && owner)
        a.cut[static_cast<long long>(cw.b) * a.bt.Hkv + cw.h] =
            whole ? make_int2(-1, -1) : make_int2(static_cast<int>(u), static_cast<int>((seg0 + cw.nt - 1) / run));
#pragma unroll
      for (int hr = 0; hr < 2; ++hr) {
        l[hr] += __shfl_xor_sync(0xffffffffu, l[hr], 1);
        l[hr] += __shfl_xor_sync(0xffffffffu, l[hr], 2);
        if (tok[hr] < 0) continue;
        const int r = 16 * rt + gr + 8 * hr;
        const bool has = lim[hr] > 0 && !(l[hr] == 0.f);  // a NaN sum stays
        if (whole) {
          const long long row = (static_cast<long long>(cw.b) * a.bt.T + tok[hr]) * a.Hq + cw.h * a.groups + r % a.groups;
          const float inv = has ? 1.f / l[hr] : 0.f;
#pragma unroll
          for (int c = 0; c < NT / 2; ++c) {
            const float x0 = has ? o[2 * c][2 * hr] * inv : 0.f, x1 = has ? o[2 * c][2 * hr + 1] * inv : 0.f;
            const float y0 = has ? o[2 * c + 1][2 * hr] * inv : 0.f, y1 = has ? o[2 * c + 1][2 * hr + 1] * inv : 0.f;
            if constexpr (ET == kCacheBf16) {
              pg_store2(a, row, D, 16 * c + 2 * qd, x0, x1);
              pg_store2(a, row, D, 16 * c + 8 + 2 * qd, y0, y1);
            } else {
              pg_store2(a, row, D, 16 * c + 4 * qd, x0, y0);
              pg_store2(a, row, D, 16 * c + 4 * qd + 2, x1, y1);
            }
          }
          if (qd == 0) a.lse[row] = has ? (m[hr] + log2f(l[hr])) * 0.6931471805599453f : -INFINITY;
        } else {
          const long long pr = (2 * u + (owner ? 1 : 0)) * a.rows + r;
          float* dst = a.part_o + pr * D;
#pragma unroll
          for (int c = 0; c < NT / 2; ++c) {
            const float x0 = o[2 * c][2 * hr], x1 = o[2 * c][2 * hr + 1];
            const float y0 = o[2 * c + 1][2 * hr], y1 = o[2 * c + 1][2 * hr + 1];
            if constexpr (ET == kCacheBf16) {
              *reinterpret_cast<float2*>(dst + 16 * c + 2 * qd) = make_float2(x0, x1);
              *reinterpret_cast<float2*>(dst + 16 * c + 8 + 2 * qd) = make_float2(y0, y1);
            } else {
              *reinterpret_cast<float4*>(dst + 16 * c + 4 * qd) = make_float4(x0, y0, x1, y1);
            }
          }
          if (qd == 0) a.part_ml[pr] = has ? make_float2(m[hr], l[hr]) : make_float2(-INFINITY, 0.f);
        }
      }
      fresh_pair = true;
    }
    if (f + 1 < f1) pg_next(a, cw, lane);
  }
  if (!ok && leader && lane == 0)  // let every copy already issued land before shared memory is released
    for (int i = consumed; i < issued; ++i) mbar_drain(full + 8u * (i % slots), (i / slots) & 1);
}

// Joins the parts of the cut pairs: with M = max m_i over the parts,
// l = sum 2^(m_i - M) l_i, out = sum 2^(m_i - M) o_i / l.  WPR warps share a
// row (8 where rows are few and parts many, 1 otherwise); the lanes hold its D
// columns.  Every part is read once, in team order: the result does not depend
// on scheduling.
template <int D, int WPR>
__global__ void __launch_bounds__(256) paged_combine_kernel(const __grid_constant__ PagedArgs a, int max_teams) {
  constexpr int kPer = D / 32, kBatch = 4;
  __shared__ float s_acc[WPR == 1 ? 1 : 8][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long id = static_cast<long long>(blockIdx.x) * (8 / WPR) + warp / WPR;
  const int w0 = warp % WPR;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const long long pairs = static_cast<long long>(a.bt.B) * a.bt.Hkv;
  if (id >= pairs * a.rows) return;
  const long long pair = id / a.rows;
  const int r = static_cast<int>(id % a.rows);
  const int2 cut = a.cut[pair];
  if (cut.x < 0 || cut.y <= cut.x || cut.y >= max_teams) return;  // the last: records of a call that timed out
  auto part = [&](int t) { return (2LL * t + (t == cut.x ? 1 : 0)) * a.rows + r; };
  float M = -INFINITY;
  for (int t = cut.x + lane; t <= cut.y; t += 32) M = fmaxf(M, a.part_ml[part(t)].x);
#pragma unroll
  for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  const float base = M == -INFINITY ? 0.f : M;
  float L = 0.f;
  for (int t = cut.x + lane; t <= cut.y; t += 32) {
    const float2 ml = a.part_ml[part(t)];
    L += fast_exp2(ml.x - base) * ml.y;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
  float acc[kPer];
#pragma unroll
  for (int e = 0; e < kPer; ++e) acc[e] = 0.f;
  for (int t0 = cut.x + w0; t0 <= cut.y; t0 += WPR * kBatch) {
    float v[kBatch][kPer], mm[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int t = t0 + WPR * k;
      mm[k] = -INFINITY;
#pragma unroll
      for (int e = 0; e < kPer; ++e) v[k][e] = 0.f;
      if (t <= cut.y) {
        mm[k] = a.part_ml[part(t)].x;
        const float* src = a.part_o + part(t) * D + kPer * lane;
#pragma unroll
        for (int e = 0; e < kPer; ++e) v[k][e] = src[e];
      }
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      if (mm[k] == -INFINITY) continue;  // a part in which the row sees no key
      const float w = fast_exp2(mm[k] - base);
#pragma unroll
      for (int e = 0; e < kPer; ++e) acc[e] = fmaf(w, v[k][e], acc[e]);
    }
  }
  if constexpr (WPR > 1) {
#pragma unroll
    for (int e = 0; e < kPer; ++e) s_acc[warp][kPer * lane + e] = acc[e];
    __syncthreads();
    if (w0 != 0) return;
#pragma unroll
    for (int w = 1; w < WPR; ++w)
#pragma unroll
      for (int e = 0; e < kPer; ++e) acc[e] += s_acc[warp + w][kPer * lane + e];
  }
  const bool has = !(L == 0.f);
  const float inv = has ? 1.f / L : 0.f;
  const int b = static_cast<int>(pair / a.bt.Hkv), h = static_cast<int>(pair % a.bt.Hkv);
  const long long row = (static_cast<long long>(b) * a.bt.T + r / a.groups) * a.Hq + h * a.groups + r % a.groups;
#pragma unroll
  for (int e = 0; e < kPer; e += 2)
    pg_store2(a, row, D, kPer * lane + e, has ? acc[e] * inv : 0.f, has ? acc[e + 1] * inv : 0.f);
  if (lane == 0) a.lse[row] = has ? (M + log2f(L)) * 0.6931471805599453f : -INFINITY;
}

}  // namespace ra
