// cache_attn.cu -- attention over the paged 8-bit latent cache.
//
//   z_s = scale * s_p * (q . code_s),  s <= t, and s > t - window or s < n_sink
//   out = sum_s softmax(z)_s * s_p * code_s[:Dc],   lse = log sum_s exp(z_s)
//
// The (512, 64) shape runs on tcgen05 with the cache's own bytes as operands:
// a tile of 128 keys goes from the pages to swizzled shared memory by TMA and
// is never converted. kind::f8f6f4 multiplies e4m3 with e4m3, so the other
// operand is split instead: q = qs * (hi + lo/16) and p = hi + lo with hi, lo
// in e4m3. A bf16 q has 8 significant bits and e4m3 has 4, and the residual of
// rounding 8 bits to 4 is a signed 4-bit number: hi + lo is q itself (down to
// 2^-22 of the row's largest element, where lo leaves e4m3's range). For p the
// residual is rounded once more, to 4 significant bits of its own: 2^-8 of p
// at most, 7e-4 rms, where a bf16 p has 1.7e-3 rms.
// Work of a tile, for R query rows (token, head) of one sequence:
//   QK^T  S^T[key, (hi, lo) x row] = K . Q^T      M = 128 keys, N = 2R, K = 576
//   softmax, one thread per key lane              p'' = 2^(z log2e + e_p - m)
//   PV    O^T[dim, row] += V^T . P^T              M = 128 dims x 4, K = 128 keys
// V is the latent part of the K tile read MN-major. The page scales 2^e_p stay
// out of the MMAs: in the logits they multiply S, in the output they are added
// to p's exponent, and the row sum takes p'' 2^-e_p.
// m is a running maximum of z log2e + e_p, lowered by 6: p'' starts at 2^6 at
// most and m is raised only when a value passes 2^8 (e4m3 ends at 448); O is
// rescaled in tensor memory then, by a power of two. A tile whose values stay
// below needs no exchange between threads but one vote.
//
// Rows of a tile: R = 32 (P's hi and lo side by side as N = 64, O_hi and O_lo
// apart) when no sequence can be expected to have more rows, as in decode,
// where the bytes bound; R = 64 else (P's lo and hi passes onto one O, N = 64),
// which shares the loads between twice as many rows. Shared memory: Q 36 or
// 72 KB, two tiles of 72 KB, P 8 KB; at R = 64 P's hi takes the place of the
// tile's rope chunk, which is dead by then. Tiles are handed out chunk by
// chunk (four of 128 dims and the rope): PV releases each chunk as it goes, so
// the next but one tile loads under it.
//
// Work is split over SMs by tiles, not by sequences: the tiles of all items
// (R rows of one sequence) form one list, and CTA c of G takes its c-th part.
// An item that crosses CTAs leaves partial results in the workspace, which
// cache_attn_combine joins. The list's length comes from the batch arrays, so
// each CTA counts it for itself; nothing of it is needed on the host.
#include <cuda_bf16.h>

#include "cache.cuh"
#include "sm100_primitives.cuh"

namespace dsa {
namespace {

using namespace sm100;

constexpr int kMaxCtas = 148;  // SMs of a B200; the workspace is laid out for as many
constexpr int kDC = 512, kDR = 64;
constexpr int kKeys = 128;
constexpr int kChunkBytes = kKeys * 128;             // 128 dims of 128 keys
constexpr int kRopeOff = 4 * kChunkBytes;            // the tile's rope chunk, 64-byte rows
constexpr int kStageBytes = kRopeOff + kKeys * kDR;  // 72 KB
constexpr int kThreads = 384;  // producer, MMA, two spare warps (the softmax warps start at a
                               // multiple of four: a warp reads the TMEM lanes of its index mod 4)
constexpr int kSoftmaxWarp0 = 4;

// What a CTA leaves for the combine pass.
struct CtaMeta {
  unsigned int status, info;  // device status of this CTA
  int row;                    // first query row (token * n_heads + head) of the item it ends
  int n_rows;                 // its rows; 0: this CTA ends no item that began in another
  int first;                  // the CTA in which the item began
  int pad[3];
};

struct CacheAttnParams {
  CacheAttnArgs a;
  CtaMeta* meta;   // [kMaxCtas]
  float2* part_ml; // [kMaxCtas][2][R]: (m, l)
  float* part_o;   // [kMaxCtas][2][R][kDC]
};

// R consecutive query rows of one sequence and the key tiles that any of them
// sees: the first nst tiles, then those from wt0 on; nt in all.
struct Item {
  int b, row, n_rows;   // sequence, first row in the call's tensors
  int i0;               // first row within the sequence
  int first;            // position of the sequence's first new token
  int t_lo, t_hi;       // positions of the first and last row
  int win_lo, sink_hi;  // keys [win_lo, t_hi] and [0, sink_hi) are seen by some row
  int nst, wt0, nt;
  __device__ __forceinline__ int tile(int k) const { return k < nst ? k : wt0 + k - nst; }
  __device__ __forceinline__ bool seen(int s) const {
    return s <= t_hi && (s >= win_lo || s < sink_hi);
  }
};

template <int R>
__device__ __forceinline__ int64_t slots_of(const CacheAttnArgs& a) {
  return static_cast<int64_t>(a.batch.n_tok) * a.n_heads / R + a.batch.n_seq;
}

template <int R>
struct ItemWalk {
  // Slot `slot` of the sequences' slots (R rows each), sequence b.
  int64_t slot, start, stop;
  int b;
  SeqRange r;

  __device__ void load(const CacheAttnArgs& a) {
    start = slot_start(a.batch, b, a.n_heads, R, 1);
    stop = b + 1 < a.batch.n_seq ? slot_start(a.batch, b + 1, a.n_heads, R, 1) : INT64_MAX;
    r = seq_range(a.batch, a.cache.page_size, b);
  }
  __device__ void seek(const CacheAttnArgs& a, int64_t s) {
    slot = s;
    b = seq_of_slot(a.batch, s, a.n_heads, R, 1);
    load(a);
  }
  __device__ void next(const CacheAttnArgs& a) {
    ++slot;
    while (slot >= stop && b + 1 < a.batch.n_seq) {
      ++b;
      load(a);
    }
  }
  // Tiles of this slot's item, 0 when the sequence has no such rows.
  __device__ int item(const CacheAttnArgs& a, Item& it) const {
    const int64_t rb = slot - start;
    const int64_t rows = static_cast<int64_t>(r.n) * a.n_heads;
    if (rb < 0 || rb * R >= rows) return 0;
    it.b = b;
    it.i0 = static_cast<int>(rb * R);
    it.n_rows = static_cast<int>(min(static_cast<int64_t>(R), rows - it.i0));
    it.row = r.tok0 * a.n_heads + it.i0;
    it.first = r.len - r.n;
    it.t_lo = it.first + it.i0 / a.n_heads;
    it.t_hi = it.first + (it.i0 + it.n_rows - 1) / a.n_heads;
    it.win_lo = a.window > 0 ? max(0, it.t_lo - a.window + 1) : 0;
    it.sink_hi = a.window > 0 ? min(a.n_sink, it.win_lo) : 0;
    it.nst = (it.sink_hi + kKeys - 1) / kKeys;
    it.wt0 = max(it.win_lo / kKeys, it.nst);
    it.nt = it.nst + it.t_hi / kKeys - it.wt0 + 1;
    return it.nt;
  }
};

// A CTA's part of the tile list as segments: tiles [k0, k1) of one item after
// the other. Every role walks its own copy.
template <int R>
struct Segments {
  ItemWalk<R> w;
  Item it;
  int k0, k1;
  int64_t left;  // tiles after this segment
  int64_t slots;
  // From the item of `slot`, tile k, for n > 0 tiles.
  __device__ void begin(const CacheAttnArgs& a, int64_t slot, int k, int64_t n) {
    slots = slots_of<R>(a);
    w.seek(a, slot);
    w.item(a, it);
    k0 = k;
    k1 = static_cast<int>(min(static_cast<int64_t>(it.nt), k + n));
    left = n - (k1 - k0);
  }
  __device__ bool next(const CacheAttnArgs& a) {
    if (left <= 0) return false;
    do {
      w.next(a);
      if (w.slot >= slots) return false;
    } while (w.item(a, it) == 0);
    k0 = 0;
    k1 = static_cast<int>(min(static_cast<int64_t>(it.nt), left));
    left -= k1;
    return true;
  }
};

template <int R>
struct Cfg {
  static constexpr int HR = R / 2;                 // rows of a softmax warpgroup
  static constexpr bool kSplitO = R == 32;         // hi and lo of P onto their own columns of O
  static constexpr int kQChunk = 2 * R * 128;      // 128 dims of the hi and lo rows
  static constexpr int kQBytes = 2 * R * (kDC + kDR);
  static constexpr int kTmemS = 0, kTmemO = 4 * R;  // S^T [2 buffers][2R], O^T [4][64]
  static constexpr int kOffQ = 0;
  static constexpr int kOffStage = kQBytes;
  static constexpr int kOffP = kOffStage + 2 * kStageBytes;
  static constexpr int kOffM = kOffP + kKeys * 64;       // float [8 warps][32]
  static constexpr int kOffRow = kOffM + 8 * 32 * 4;     // float rowfac[64], int row_t[64]
  static constexpr int kOffBar = kOffRow + 2 * 64 * 4;
  static constexpr int kNumBars = 10 + 10 + 2 + 2 + 5;
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;
  static constexpr int kMiscBytes = 160;
  static constexpr int kSmemBytes = kOffMisc + kMiscBytes + 1024;
  static constexpr uint32_t kIdescQK = idesc_e4m3_f32(128, 2 * R);
  static constexpr uint32_t kIdescPV = idesc_e4m3_f32(128, 64, true, true);
  static_assert(kOffStage % 1024 == 0 && kOffP % 1024 == 0, "operand alignment");
  static_assert(kSmemBytes <= 232448, "shared memory");
  static_assert(kTmemO + 256 <= 512, "tensor memory");
};

// Shared words after the barriers.
struct Misc {
  unsigned int status, info;  // stands in for the header of a workspace in report()
  uint32_t tmem;
  int abort_flag;
  long long slot, n_tiles, total;
  long long scan[12];
  int k0;
};
static_assert(sizeof(Misc) <= 160, "misc");

enum Bars { kFull = 0, kEmpty = 10, kSFull = 20, kSFree = 22, kPFull = 24, kPvDone, kQFull, kOFree, kDrain };
enum Sites { kSiteEmpty = 40, kSiteFull, kSiteSFull, kSiteSFree, kSiteP, kSitePv, kSiteQ, kSiteO };

__device__ __forceinline__ void named_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

__device__ __forceinline__ bool named_or(int id, int threads, bool p) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, %2, %3, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(p ? 1u : 0u), "r"(id), "r"(threads)
      : "memory");
  return r != 0;
}

__device__ __forceinline__ float warp_max(float x) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}

// Sum of v[e] over the 32 lanes for every e; lane l gets that of e = l % NV.
template <int NV>
__device__ __forceinline__ float warp_transpose_sum(float (&v)[NV]) {
  const int lane = threadIdx.x & 31;
  if constexpr (NV == 16) {
#pragma unroll
    for (int e = 0; e < NV; ++e) v[e] += __shfl_xor_sync(0xffffffffu, v[e], 16);
  }
#pragma unroll
  for (int s = NV / 2; s >= 1; s >>= 1) {
    const bool upper = (lane & s) != 0;
#pragma unroll
    for (int e = 0; e < s; ++e) {
      const float send = upper ? v[e] : v[e + s];
      const float keep = upper ? v[e + s] : v[e];
      v[e] = keep + __shfl_xor_sync(0xffffffffu, send, s);
    }
  }
  return v[0];
}

template <int NC>
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, uint32_t (&r)[NC]) {
  if constexpr (NC == 32) tmem_ld_32x32b_x32(taddr, r);
  else tmem_ld_32x32b_x16(taddr, r);
}

template <int NC>
__device__ __forceinline__ void tmem_st_cols(uint32_t taddr, const uint32_t (&r)[NC]) {
  if constexpr (NC == 32) tmem_st_32x32b_x32(taddr, r);
  else tmem_st_32x32b_x16(taddr, r);
}

// ------------------------------------------------------------------ schedule

// Counts the tiles of all items and finds this CTA's part. All threads.
template <int R>
__device__ void schedule(const CacheAttnArgs& a, Misc* ms) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // the slots need cu_seqlens that ascend; if they do not, there is no work
  int bad = 0;
  for (int b = tid; b < a.batch.n_seq; b += kThreads) {
    const int c0 = __ldg(a.batch.cu_seqlens + b), c1 = __ldg(a.batch.cu_seqlens + b + 1);
    bad |= c0 < 0 || c1 < c0 || c1 > a.batch.n_tok;
  }
  const int64_t slots = __syncthreads_or(bad) ? 0 : slots_of<R>(a);
  const int64_t per = (slots + kThreads - 1) / kThreads;
  const int64_t s0 = min(slots, tid * per), s1 = min(slots, s0 + per);
  ItemWalk<R> w;
  Item it;
  long long sum = 0;
  if (s0 < s1) {
    w.seek(a, s0);
    for (int64_t s = s0; s < s1; ++s) {
      sum += w.item(a, it);
      if (s + 1 < s1) w.next(a);
    }
  }
  long long inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) ms->scan[warp] = inc;
  __syncthreads();
  long long before = 0, total = 0;
  for (int i = 0; i < kThreads / 32; ++i) {
    if (i < warp) before += ms->scan[i];
    total += ms->scan[i];
  }
  const long long g = min(static_cast<long long>(gridDim.x), total);  // CTAs with work
  long long begin = 0, end = 0;
  if (static_cast<long long>(blockIdx.x) < g) {
    begin = total * blockIdx.x / g;
    end = total * (blockIdx.x + 1) / g;
  }
  const long long lo = before + inc - sum;
  if (begin < end && lo <= begin && begin < lo + sum) {  // one thread
    long long at = lo;
    w.seek(a, s0);
    int n;
    while (at + (n = w.item(a, it)) <= begin) {
      at += n;
      w.next(a);
    }
    ms->slot = w.slot;
    ms->k0 = static_cast<int>(begin - at);
  }
  if (tid == 0) {
    ms->n_tiles = end - begin;
    ms->total = total;
  }
  __syncthreads();
}

// The CTA whose part of the list holds tile `at`.
__device__ __forceinline__ int cta_of_tile(long long at, long long total, int grid) {
  const long long g = min(static_cast<long long>(grid), total);
  long long c = at * g / total;
  while (c + 1 < g && total * (c + 1) / g <= at) ++c;
  while (c > 0 && total * c / g > at) --c;
  return static_cast<int>(c);
}

// ---------------------------------------------------------------- q operand

// The exponent e of the smallest 2^e with |x| <= 448 * 2^e.
__device__ __forceinline__ int q_exp(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int e = static_cast<int>(b >> 23) - 127 - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return min(max(e, -110), 110);
}

__device__ __forceinline__ float2 bf16x2(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

// Eight bf16 as e4m3 hi and lo codes: x * inv = hi + lo / 16.
__device__ __forceinline__ void split_q(const uint4& v, float inv, uint2& hi, uint2& lo) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t h[4], l[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float2 x = bf16x2(w[e]);
    x.x *= inv;
    x.y *= inv;
    h[e] = f32_to_e4m3x2(x.x, x.y);
    const float2 y = e4m3x2_to_f32(h[e]);
    l[e] = f32_to_e4m3x2((x.x - y.x) * 16.f, (x.y - y.y) * 16.f);
  }
  hi = make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
  lo = make_uint2(l[0] | l[1] << 16, l[2] | l[3] << 16);
}

// Byte offset of group g (8 codes) of operand row n within the Q buffer.
template <int R>
__device__ __forceinline__ uint32_t q_off(int n, int g) {
  if (g < kDC / 8) {
    const int c = g >> 4, u = (g & 15) >> 1;  // chunk, 16-byte unit
    return c * Cfg<R>::kQChunk + n * 128 + ((u ^ (n & 7)) << 4) + (g & 1) * 8;
  }
  const int u = (g - kDC / 8) >> 1;
  return 4 * Cfg<R>::kQChunk + n * 64 + ((u ^ ((n >> 1) & 3)) << 4) + (g & 1) * 8;
}

// The item's rows as operand rows (hi at r, lo at R + r), their factors and
// positions. The eight softmax warps, a row at a time each.
template <int R>
__device__ void convert_q(const CacheAttnArgs& a, const Item& it, unsigned char* sq, float* rowfac,
                          int* row_t) {
  const int warp = (threadIdx.x >> 5) - kSoftmaxWarp0, lane = threadIdx.x & 31;
  constexpr int kGroups = (kDC + kDR) / 8;  // 72
  constexpr int kAtOnce = 4;
#pragma unroll
  for (int j0 = 0; j0 < R / 8; j0 += kAtOnce) {
    uint4 v[kAtOnce][3];
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
      const int r = warp + 8 * (j0 + j);
      const uint4* src = reinterpret_cast<const uint4*>(
          a.q + (static_cast<int64_t>(it.row) + r) * (kDC + kDR));
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        v[j][i] = make_uint4(0u, 0u, 0u, 0u);
        if (r < it.n_rows && lane + 32 * i < kGroups) v[j][i] = __ldg(src + lane + 32 * i);
      }
    }
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
      const int r = warp + 8 * (j0 + j);
      float mx = 0.f;
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        const uint32_t w[4] = {v[j][i].x, v[j][i].y, v[j][i].z, v[j][i].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 x = bf16x2(w[e]);
          mx = fmaxf(mx, fmaxf(fabsf(x.x), fabsf(x.y)));
        }
      }
      const int e = q_exp(warp_max(mx));
      const float inv = pow2f(-e);
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        const int g = lane + 32 * i;
        if (g < kGroups) {
          uint2 hi, lo;
          split_q(v[j][i], inv, hi, lo);
          *reinterpret_cast<uint2*>(sq + q_off<R>(r, g)) = hi;
          *reinterpret_cast<uint2*>(sq + q_off<R>(R + r, g)) = lo;
        }
      }
      if (lane == 0) {
        rowfac[r] = pow2f(e) * a.scale_log2;
        row_t[r] = it.first + (it.i0 + min(r, it.n_rows - 1)) / a.n_heads;
      }
    }
  }
}

// -------------------------------------------------------------------- kernel

template <int R>
struct Ctx {
  const CacheAttnParams& p;
  unsigned char* s;
  uint64_t* bar;
  Misc* ms;
  uint32_t tmem;
  __device__ bool wait(int b, uint32_t parity, unsigned site) const {
    return mbar_wait(bar + b, parity, &ms->abort_flag, reinterpret_cast<WsHeader*>(&ms->status),
                     site);
  }
  __device__ void error(unsigned site) const {
    report(reinterpret_cast<WsHeader*>(&ms->status), kDevRange, site);
  }
};

__device__ __forceinline__ void drain_wait(uint64_t* bar, uint32_t parity) {
  const long long t0 = clock64();
  while (!mbar_try_wait(bar, parity))
    if (clock64() - t0 > kWaitLimitCycles) break;
}

// Producer warp: lane l < 128 / page_size loads the tile's l-th page.
template <int R>
__device__ void producer(const Ctx<R>& x, const CUtensorMap* ml, const CUtensorMap* mr) {
  const CacheAttnArgs& a = x.p.a;
  const int lane = threadIdx.x & 31, ps = a.cache.page_size, npt = kKeys / ps;
  Segments<R> sg;
  sg.begin(a, x.ms->slot, x.ms->k0, x.ms->n_tiles);
  int i = 0, c_failed = 0;
  bool ok = true;
  int page_next = -1;
  // this lane's page of tile k, or -1 when no row of the item sees any of it
  auto page_of = [&](int k) {
    if (lane >= npt) return -1;
    const int s0 = sg.it.tile(k) * kKeys + lane * ps, s1 = s0 + ps - 1;
    const bool any = s0 <= sg.it.t_hi && (s1 >= sg.it.win_lo || s0 < sg.it.sink_hi);
    if (!any) return -1;
    const int pg = __ldg(a.batch.page_table + static_cast<int64_t>(sg.it.b) * a.batch.max_pages +
                         s0 / ps);
    if (pg >= 0 && pg < a.cache.n_pages) return pg;
    x.error(kCacheSitePage);
    return -1;
  };
  do {
    page_next = page_of(sg.k0);
    for (int k = sg.k0; k < sg.k1 && ok; ++k, ++i) {
      const int page = page_next;
      if (k + 1 < sg.k1) page_next = page_of(k + 1);
      const int n = __popc(__ballot_sync(0xffffffffu, page >= 0));
      const int st = i & 1;
      unsigned char* dst = x.s + Cfg<R>::kOffStage + st * kStageBytes;
      for (int c = 0; c < 5; ++c) {
        if (i >= 2) ok = x.wait(kEmpty + 5 * st + c, ((i >> 1) - 1) & 1, kSiteEmpty);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) {
          c_failed = c;
          break;
        }
        uint64_t* full = x.bar + kFull + 5 * st + c;
        const int row_bytes = c < 4 ? 128 : kDR;
        if (lane == 0) mbar_arrive_expect_tx(full, n * ps * row_bytes);
        __syncwarp();
        if (page >= 0) {
          if (c < 4) tma_load_3d(dst + c * kChunkBytes + lane * ps * 128, ml, c * 128, 0, page, full);
          else tma_load_3d(dst + kRopeOff + lane * ps * kDR, mr, 0, 0, page, full);
        }
      }
    }
  } while (ok && sg.next(a));
  if (!ok && lane == 0) {
    // Let the copies in flight land before the block ends: tile i - 1 was
    // begun up to chunk c_failed, the one before it in full.
    for (int c = 0; c < 5; ++c)
      for (int j = max(i - 3, 0); j < i; ++j)
        if (j < i - 1 || c < c_failed) drain_wait(x.bar + kFull + 5 * (j & 1) + c, (j >> 1) & 1);
  }
}

// MMA warp (warp-collective issue).
template <int R>
__device__ void mma_issuer(const Ctx<R>& x) {
  using C = Cfg<R>;
  const CacheAttnArgs& a = x.p.a;
  const uint32_t sb = smem_u32(x.s);
  const uint64_t dq = smem_desc(sb + C::kOffQ, 16, 1024, 2);
  const uint64_t dqr = smem_desc(sb + C::kOffQ + 4 * C::kQChunk, 16, 512, 4);
  const uint64_t dk = smem_desc(sb + C::kOffStage, 16, 1024, 2);
  const uint64_t dkr = smem_desc(sb + C::kOffStage + kRopeOff, 16, 512, 4);
  const uint64_t dv = smem_desc(sb + C::kOffStage, 16384, 1024, 2);
  const uint64_t dp = smem_desc(sb + C::kOffP, 512, 512, 4);
  const uint64_t dph = smem_desc(sb + C::kOffStage + kRopeOff, 512, 512, 4);
  Segments<R> sg;
  sg.begin(a, x.ms->slot, x.ms->k0, x.ms->n_tiles);
  int i = 0, seg = 0;
  bool ok = true;
  bool pend_first = false;  // the tile whose PV is due is its segment's first
  int pend_seg = 0;
  // PV of tile j: every block's chunk is released by its own commit
  auto pv = [&](int j, bool first, int sgi) {
    ok = ok && x.wait(kPFull, j & 1, kSiteP);
    if (first && sgi > 0) ok = ok && x.wait(kOFree, (sgi - 1) & 1, kSiteO);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) return;
    tc_fence_after();
    const uint64_t so = static_cast<uint64_t>((j & 1) * kStageBytes) >> 4;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const uint32_t d = x.tmem + C::kTmemO + 64 * c;
      const uint64_t av = dv + so + ((c * kChunkBytes) >> 4);
      const uint64_t bh = C::kSplitO ? dp : dph + so;
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
        mma_f8_ss_warp(d, av + ((kk * 4096) >> 4), bh + ((kk * 2048) >> 4), C::kIdescPV,
                       kk > 0 || !first);
      if constexpr (!C::kSplitO) {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          mma_f8_ss_warp(d, av + ((kk * 4096) >> 4), dp + ((kk * 2048) >> 4), C::kIdescPV, 1u);
      }
      mma_commit_warp(x.bar + kEmpty + 5 * (j & 1) + c);
    }
    mma_commit_warp(x.bar + kEmpty + 5 * (j & 1) + 4);
    mma_commit_warp(x.bar + kPvDone);
  };
  do {
    for (int k = sg.k0; k < sg.k1 && ok; ++k, ++i) {
      if (k == sg.k0) {
        if (i > 0) pv(i - 1, pend_first, pend_seg);
        ok = ok && x.wait(kQFull, seg & 1, kSiteQ);
      }
      if (i >= 2) ok = ok && x.wait(kSFree + (i & 1), ((i >> 1) - 1) & 1, kSiteSFree);
      const uint64_t so = static_cast<uint64_t>((i & 1) * kStageBytes) >> 4;
      const uint32_t d = x.tmem + C::kTmemS + 2 * R * (i & 1);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        ok = ok && x.wait(kFull + 5 * (i & 1) + c, (i >> 1) & 1, kSiteFull);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
          mma_f8_ss_warp(d, dk + so + ((c * kChunkBytes + ks * 32) >> 4),
                         dq + ((c * C::kQChunk + ks * 32) >> 4), C::kIdescQK, c > 0 || ks > 0);
      }
      ok = ok && x.wait(kFull + 5 * (i & 1) + 4, (i >> 1) & 1, kSiteFull);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
#pragma unroll
      for (int ks = 0; ks < 2; ++ks)
        mma_f8_ss_warp(d, dkr + so + ((ks * 32) >> 4), dqr + ((ks * 32) >> 4), C::kIdescQK, 1u);
      mma_commit_warp(x.bar + kSFull + (i & 1));
      if (k > sg.k0) pv(i - 1, pend_first, pend_seg);
      pend_first = k == sg.k0;
      pend_seg = seg;
    }
    ++seg;
  } while (ok && sg.next(a));
  if (ok) pv(i - 1, pend_first, pend_seg);
  // every MMA has to be done before the tensor memory is released
  mma_commit_warp(x.bar + kDrain);
  drain_wait(x.bar + kDrain, 0);
}

// Softmax warps: warpgroup g takes the rows [g * HR, (g + 1) * HR), a thread
// one key lane (then one dim lane of O). After a timeout they go on through
// all tiles without waiting or storing (every wait returns at once then), so
// that no warp is left alone at a named barrier.
template <int R>
__device__ void softmax_warps(const Ctx<R>& x) {
  using C = Cfg<R>;
  constexpr int HR = C::HR;
  const CacheAttnArgs& a = x.p.a;
  const int warp = (threadIdx.x >> 5) - kSoftmaxWarp0, lane = threadIdx.x & 31;
  const int g = warp >> 2, quarter = warp & 3, key = 32 * quarter + lane;
  const uint32_t lanes = static_cast<uint32_t>(32 * quarter) << 16;
  const int ps = a.cache.page_size;
  float* s_m = reinterpret_cast<float*>(x.s + C::kOffM);      // [8][32]
  float* my_m = s_m + 32 * warp;
  float* rowfac = reinterpret_cast<float*>(x.s + C::kOffRow);
  int* row_t = reinterpret_cast<int*>(rowfac + 64);
  Segments<R> sg;
  sg.begin(a, x.ms->slot, x.ms->k0, x.ms->n_tiles);
  convert_q<R>(a, sg.it, x.s + C::kOffQ, rowfac, row_t);
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) mbar_arrive(x.bar + kQFull);
  named_sync(3, 256);
  int i = 0;
  bool ok = true;
  for (;;) {
    const Item it = sg.it;
    const int k0 = sg.k0, k1 = sg.k1;
    float l[HR];
#pragma unroll
    for (int r = 0; r < HR; ++r) l[r] = 0.f;
    float m = 0.f;  // lane r: the reference of row g * HR + r
    uint32_t unset = HR == 32 ? 0xffffffffu : (1u << HR) - 1u;  // rows that saw no key yet
    if (lane < HR) my_m[lane] = 0.f;
    __syncwarp();
    auto page_at = [&](int k) {
      const int s = it.tile(k) * kKeys + key;
      if (!it.seen(s)) return -1;
      const int pg =
          __ldg(a.batch.page_table + static_cast<int64_t>(it.b) * a.batch.max_pages + s / ps);
      return pg >= 0 && pg < a.cache.n_pages ? pg : -1;
    };
    int page = page_at(k0);
    float sc = page >= 0 ? __ldg(a.cache.scale + page) : 1.f;
    for (int k = k0; k < k1; ++k, ++i) {
      const int page_next = k + 1 < k1 ? page_at(k + 1) : -1;
      const int s = it.tile(k) * kKeys + key;
      const int e_key = scale_exp(sc);
      const float sk = pow2f(e_key), inv_sk = pow2f(-e_key), ek = static_cast<float>(e_key);
      // does every row see the whole tile?
      const int t0 = it.tile(k) * kKeys;
      const bool whole = t0 + kKeys - 1 <= it.t_lo &&
                         (a.window == 0 || t0 > it.t_hi - a.window || t0 + kKeys <= a.n_sink);
      const bool masked = !whole || __any_sync(0xffffffffu, page < 0);
      ok = ok && x.wait(kSFull + (i & 1), (i >> 1) & 1, kSiteSFull);
      __syncwarp();
      tc_fence_after();
      float z[HR];
      {
        uint32_t hi[HR], lo[HR];
        const uint32_t col = x.tmem + lanes + C::kTmemS + 2 * R * (i & 1) + g * HR;
        tmem_ld_cols<HR>(col, hi);
        tmem_ld_cols<HR>(col + R, lo);
        tmem_ld_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(x.bar + kSFree + (i & 1));
#pragma unroll
        for (int r = 0; r < HR; ++r)
          z[r] = fmaf(fmaf(__uint_as_float(lo[r]), 0.0625f, __uint_as_float(hi[r])),
                      rowfac[g * HR + r] * sk, ek);
      }
      if (masked) {
        // row at position t sees key s iff s <= t and (t < s + window or s < n_sink)
        const unsigned span = page < 0 ? 0u
                              : a.window == 0 || s < a.n_sink ? 0x7fffffffu
                                                              : static_cast<unsigned>(a.window);
#pragma unroll
        for (int r = 0; r < HR; ++r)
          if (static_cast<unsigned>(row_t[g * HR + r] - s) >= span) z[r] = -INFINITY;
      }
      float over = -INFINITY;
#pragma unroll
      for (int r = 0; r < HR; ++r) over = fmaxf(over, z[r] - my_m[r]);
      bool pv_waited = i == 0;
      if (named_or(1 + g, 128, over > 8.f) || unset != 0u) {
        // a new reference for the rows that need one
        float mx = -INFINITY;
#pragma unroll
        for (int r = 0; r < HR; ++r) {
          const float v = warp_max(z[r]);
          if (lane == r) mx = v;
        }
        __syncwarp();
        if (lane < HR) my_m[lane] = mx;
        named_sync(1 + g, 128);
        if (lane < HR) {
#pragma unroll
          for (int q = 0; q < 4; ++q) mx = fmaxf(mx, s_m[32 * (4 * g + q) + lane]);
        }
        named_sync(1 + g, 128);
        const bool fresh = (unset >> lane) & 1u;
        const bool up = lane < HR && (fresh ? mx > -INFINITY : mx - m > 8.f);
        const float m_new = up ? ceilf(mx) - 6.f : m;
        const float f = up && !fresh ? ex2_approx(m - m_new) : 1.f;
        unset &= ~__ballot_sync(0xffffffffu, up);
        m = m_new;
        if (lane < HR) my_m[lane] = m;
        __syncwarp();
        if (__any_sync(0xffffffffu, f != 1.f)) {
          if (i > 0) ok = ok && x.wait(kPvDone, (i - 1) & 1, kSitePv);
          __syncwarp();
          pv_waited = true;
          tc_fence_after();
          float fr[HR];
#pragma unroll
          for (int r = 0; r < HR; ++r) {
            fr[r] = __shfl_sync(0xffffffffu, f, r);
            l[r] *= fr[r];
          }
          if (k > k0) {
#pragma unroll
            for (int c = 0; c < (C::kSplitO ? 8 : 4); ++c) {
              const uint32_t col = x.tmem + lanes + C::kTmemO + (C::kSplitO ? 32 : 64) * c + g * HR;
              uint32_t o[HR];
              tmem_ld_cols<HR>(col, o);
              tmem_ld_wait();
#pragma unroll
              for (int r = 0; r < HR; ++r) o[r] = __float_as_uint(__uint_as_float(o[r]) * fr[r]);
              tmem_st_cols<HR>(col, o);
            }
            tmem_st_wait();
          }
        }
      }
      if (!pv_waited) {  // P's place is free once the previous PV is done
        ok = ok && x.wait(kPvDone, (i - 1) & 1, kSitePv);
      }
      unsigned char* stage = x.s + C::kOffStage + (i & 1) * kStageBytes;
      {
        uint32_t hi[HR / 4], lo[HR / 4];
#pragma unroll
        for (int r = 0; r < HR; r += 4) {
          float p[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            p[e] = ex2_approx(z[r + e] - my_m[r + e]);
            l[r + e] = fmaf(p[e], inv_sk, l[r + e]);
          }
          const uint32_t h0 = f32_to_e4m3x2(p[0], p[1]), h1 = f32_to_e4m3x2(p[2], p[3]);
          const float2 b0 = e4m3x2_to_f32(h0), b1 = e4m3x2_to_f32(h1);
          constexpr float kLo = C::kSplitO ? 16.f : 1.f;
          hi[r / 4] = h0 | h1 << 16;
          lo[r / 4] = f32_to_e4m3x2((p[0] - b0.x) * kLo, (p[1] - b0.y) * kLo) |
                      f32_to_e4m3x2((p[2] - b1.x) * kLo, (p[3] - b1.y) * kLo) << 16;
        }
        unsigned char* row_hi = (C::kSplitO ? x.s + C::kOffP : stage + kRopeOff) + key * 64;
        unsigned char* row_lo = x.s + C::kOffP + key * 64;
        const int sw = (key >> 1) & 3;
#pragma unroll
        for (int u = 0; u < HR / 16; ++u) {
          const int uh = g * (HR / 16) + u, ul = C::kSplitO ? 2 + g : uh;
          *reinterpret_cast<uint4*>(row_hi + ((uh ^ sw) << 4)) =
              make_uint4(hi[4 * u], hi[4 * u + 1], hi[4 * u + 2], hi[4 * u + 3]);
          *reinterpret_cast<uint4*>(row_lo + ((ul ^ sw) << 4)) =
              make_uint4(lo[4 * u], lo[4 * u + 1], lo[4 * u + 2], lo[4 * u + 3]);
        }
      }
      if (masked) {
        // A key that no row sees: its bytes may be anything, and 0 * NaN is
        // NaN, so its latent row is zeroed before the PV. The tile's chunks
        // have landed (QK^T read them); waiting on them orders the writes.
        for (int c = 0; c < 4; ++c) ok = ok && x.wait(kFull + 5 * (i & 1) + c, (i >> 1) & 1, kSiteFull);
        if (page < 0) {
#pragma unroll
          for (int c = 2 * g; c < 2 * g + 2; ++c)
#pragma unroll
            for (int u = 0; u < 8; ++u)
              *reinterpret_cast<uint4*>(stage + c * kChunkBytes + key * 128 + u * 16) =
                  make_uint4(0u, 0u, 0u, 0u);
        }
      }
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(x.bar + kPFull);
      page = page_next;
      sc = page >= 0 ? __ldg(a.cache.scale + page) : 1.f;
    }
    // the next segment's Q, while the last PV runs
    const bool more = sg.next(a);
    if (more) {
      named_sync(3, 256);  // every warp is done with this item's factors
      convert_q<R>(a, sg.it, x.s + C::kOffQ, rowfac, row_t);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(x.bar + kQFull);
      named_sync(3, 256);
    }
    ok = ok && x.wait(kPvDone, (i - 1) & 1, kSitePv);
    ok = __all_sync(0xffffffffu, ok);
    tc_fence_after();
    // row sums over the key lanes
    float sum = warp_transpose_sum<HR>(l);
    __syncwarp();
    if (lane < HR) my_m[lane] = sum;
    named_sync(1 + g, 128);
    sum = 0.f;
    if (lane < HR) {
#pragma unroll
      for (int q = 0; q < 4; ++q) sum += s_m[32 * (4 * g + q) + lane];
    }
    named_sync(1 + g, 128);
    const int r0 = g * HR;
    const bool whole_item = k0 == 0 && k1 == it.nt;
    const int64_t part = 2ll * blockIdx.x + (k0 == 0 ? 1 : 0);
    if (ok && quarter == 0 && lane < HR && r0 + lane < it.n_rows) {
      if (whole_item) {
        if (a.lse)
          a.lse[static_cast<int64_t>(it.row) + r0 + lane] =
              sum > 0.f ? (m + log2f(sum)) * 0.69314718055994531f : -INFINITY;
      } else {
        x.p.part_ml[part * R + r0 + lane] = make_float2(sum > 0.f ? m : -INFINITY, sum);
      }
    }
    if (lane < HR) my_m[lane] = whole_item ? (sum > 0.f ? 1.f / sum : 0.f) : 1.f;
    __syncwarp();
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      float o[HR];
      {
        uint32_t v[HR];
        const uint32_t col = x.tmem + lanes + C::kTmemO + 64 * c + g * HR;
        tmem_ld_cols<HR>(col, v);
        if constexpr (C::kSplitO) {
          uint32_t w[HR];
          tmem_ld_cols<HR>(col + 32, w);
          tmem_ld_wait();
#pragma unroll
          for (int r = 0; r < HR; ++r)
            o[r] = fmaf(__uint_as_float(w[r]), 0.0625f, __uint_as_float(v[r])) * my_m[r];
        } else {
          tmem_ld_wait();
#pragma unroll
          for (int r = 0; r < HR; ++r) o[r] = __uint_as_float(v[r]) * my_m[r];
        }
      }
      const int dim = c * 128 + 32 * quarter + lane;
      if (whole_item) {
        // lanes pair up: the even one stores row r, the odd one row r + 1
        uint16_t* out = a.out + (static_cast<int64_t>(it.row) + r0) * kDC + (dim & ~1);
        const bool odd = lane & 1;
#pragma unroll
        for (int r = 0; r < HR; r += 2) {
          const float other = __shfl_xor_sync(0xffffffffu, odd ? o[r] : o[r + 1], 1);
          const __nv_bfloat162 v = odd ? __floats2bfloat162_rn(other, o[r + 1])
                                       : __floats2bfloat162_rn(o[r], other);
          const int row = r + (odd ? 1 : 0);
          if (ok && r0 + row < it.n_rows)
            *reinterpret_cast<__nv_bfloat162*>(out + static_cast<int64_t>(row) * kDC) = v;
        }
      } else {
        float* out = x.p.part_o + (part * R + r0) * kDC + dim;
#pragma unroll
        for (int r = 0; r < HR; ++r)
          if (ok && r0 + r < it.n_rows) out[static_cast<int64_t>(r) * kDC] = o[r];
      }
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(x.bar + kOFree);
    if (!more) break;
  }
}

template <int R>
__global__ void __launch_bounds__(kThreads, 1)
    cache_attn_tc(const __grid_constant__ CacheAttnParams p, const __grid_constant__ CUtensorMap ml,
                  const __grid_constant__ CUtensorMap mr) {
  using C = Cfg<R>;
  extern __shared__ unsigned char smem_raw[];
  Ctx<R> x{p};
  x.s = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                         ~static_cast<uintptr_t>(1023));
  x.bar = reinterpret_cast<uint64_t*>(x.s + C::kOffBar);
  x.ms = reinterpret_cast<Misc*>(x.s + C::kOffMisc);
  const int tid = threadIdx.x, warp = tid >> 5;
  if (tid == 0) {
    x.ms->status = x.ms->info = 0u;
    x.ms->abort_flag = 0;
    for (int b = 0; b < C::kNumBars; ++b) {
      const bool by_warps = b == kSFree || b == kSFree + 1 || b == kPFull || b == kQFull || b == kOFree;
      mbar_init(x.bar + b, by_warps ? 8 : 1);
    }
    fence_barrier_init();
    prefetch_tmap(&ml);
    prefetch_tmap(&mr);
  }
  if (warp == 1) tmem_alloc(&x.ms->tmem, 512);
  schedule<R>(p.a, x.ms);  // ends with a barrier
  tc_fence_after();
  x.tmem = x.ms->tmem;
  if (blockIdx.x == 0)  // the batch arrays, once for all
    for (int b = tid; b < p.a.batch.n_seq; b += kThreads)
      if (!seq_range(p.a.batch, p.a.cache.page_size, b).ok) x.error(kCacheSiteSeq);
  const bool work = x.ms->n_tiles > 0;
  if (work) {
    if (warp == 0) producer<R>(x, &ml, &mr);
    else if (warp == 1) mma_issuer<R>(x);
    else if (warp >= kSoftmaxWarp0) softmax_warps<R>(x);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(x.tmem, 512);
  }
  if (tid == 0) {
    CtaMeta me;
    me.status = x.ms->status;
    me.info = x.ms->info;
    me.row = me.n_rows = me.first = 0;
    if (work && x.ms->k0 > 0) {
      // the first segment's item began in another CTA; does it end here?
      ItemWalk<R> w;
      Item it;
      w.seek(p.a, x.ms->slot);
      w.item(p.a, it);
      if (x.ms->k0 + x.ms->n_tiles >= it.nt) {
        const long long g = min(static_cast<long long>(gridDim.x), x.ms->total);
        const long long begin = x.ms->total * blockIdx.x / g;
        me.row = it.row;
        me.n_rows = it.n_rows;
        me.first = cta_of_tile(begin - x.ms->k0, x.ms->total, gridDim.x);
      }
    }
    p.meta[blockIdx.x] = me;
  }
}

// ------------------------------------------------------------------- combine

constexpr int kCombineThreads = 512;

// Joins the partial results of the items that cross CTAs, one query row at a
// time: out = sum_c 2^(m_c - M) O_c / sum_c 2^(m_c - M) l_c. Four groups of 128
// threads (four dims a thread) take every fourth part. Also collects the
// CTAs' status.
template <int R>
__global__ void __launch_bounds__(kCombineThreads)
    cache_attn_combine(const __grid_constant__ CacheAttnParams p, int n_ctas) {
  __shared__ int s_owner[kMaxCtas];
  __shared__ int s_count;
  __shared__ float s_w[kMaxCtas + 2];
  __shared__ float4 s_acc[3][128];
  const int tid = threadIdx.x;
  if (tid < 32) {  // the CTAs that end such an item, in order (the same list in every block)
    int n = 0;
    for (int c0 = 0; c0 < n_ctas; c0 += 32) {
      const bool has = c0 + tid < n_ctas && p.meta[c0 + tid].n_rows > 0;
      const uint32_t b = __ballot_sync(0xffffffffu, has);
      if (has) s_owner[n + __popc(b & ((1u << tid) - 1u))] = c0 + tid;
      n += __popc(b);
    }
    if (tid == 0) s_count = n;
  }
  if (blockIdx.x == 0 && tid == 0) {
    unsigned int status = 0, info = 0;
    for (int c = 0; c < n_ctas && status == 0u; ++c) {
      status = p.meta[c].status;
      info = p.meta[c].info;
    }
    p.a.ws->status_info = info;
    p.a.ws->status = status;
  }
  __syncthreads();
  const int work = s_count * R;
  for (int u = blockIdx.x; u < work; u += gridDim.x) {
    const int c1 = s_owner[u / R], r = u % R;
    const CtaMeta me = p.meta[c1];
    if (r >= me.n_rows) continue;
    const int c0 = me.first, n = c1 - c0 + 1;
    auto part = [&](int j) { return 2ll * (c0 + j) + (j == 0 ? 1 : 0); };
    // weights of the parts, in the first warp
    __syncthreads();
    if (tid < 32) {
      float mx = -INFINITY;
      for (int j = tid; j < n; j += 32) mx = fmaxf(mx, p.part_ml[part(j) * R + r].x);
      mx = warp_max(mx);
      float sum = 0.f;
      for (int j = tid; j < n; j += 32) {
        const float2 v = p.part_ml[part(j) * R + r];
        const float w = v.x == -INFINITY ? 0.f : exp2f(v.x - mx);
        s_w[j] = w;
        sum += w * v.y;
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (tid == 0) {
        s_w[kMaxCtas + 1] = sum > 0.f ? 1.f / sum : 0.f;
        if (p.a.lse)
          p.a.lse[static_cast<int64_t>(me.row) + r] =
              sum > 0.f ? (mx + log2f(sum)) * 0.69314718055994531f : -INFINITY;
      }
    }
    __syncthreads();
    const int group = tid >> 7, d4 = tid & 127;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int j = group; j < n; j += 4) {
      const float w = s_w[j];
      const float4 v = reinterpret_cast<const float4*>(p.part_o + (part(j) * R + r) * kDC)[d4];
      if (w > 0.f) {
        acc.x = fmaf(w, v.x, acc.x);
        acc.y = fmaf(w, v.y, acc.y);
        acc.z = fmaf(w, v.z, acc.z);
        acc.w = fmaf(w, v.w, acc.w);
      }
    }
    if (group > 0) s_acc[group - 1][d4] = acc;
    __syncthreads();
    if (group == 0) {
#pragma unroll
      for (int j = 0; j < 3; ++j) {
        const float4 v = s_acc[j][d4];
        acc.x += v.x;
        acc.y += v.y;
        acc.z += v.z;
        acc.w += v.w;
      }
      const float inv = s_w[kMaxCtas + 1];
      const __nv_bfloat162 lo = __floats2bfloat162_rn(acc.x * inv, acc.y * inv);
      const __nv_bfloat162 hi = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
      uint2 v;
      v.x = *reinterpret_cast<const uint32_t*>(&lo);
      v.y = *reinterpret_cast<const uint32_t*>(&hi);
      *reinterpret_cast<uint2*>(p.a.out + (static_cast<int64_t>(me.row) + r) * kDC + 4 * d4) = v;
    }
  }
}

// ----------------------------------------------------- the (64, 16) shape

constexpr int kRowWarps = 4;

// One warp per query row (token, head). 32 keys at a time: a lane forms the
// dot product of its key (q from shared memory), the warp updates the running
// maximum and sum, then the lanes take the latent's dims and add the 32
// weighted rows.
template <int DC, int DR>
__global__ void __launch_bounds__(32 * kRowWarps)
    cache_attn_rows(const __grid_constant__ CacheAttnArgs a) {
  constexpr int kPer = DC / 32;
  __shared__ float s_q[kRowWarps][DC + DR];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kRowWarps + warp;
  const int tok = static_cast<int>(row / a.n_heads);
  if (tok >= a.batch.n_tok) return;
  const int b = seq_of_token(a.batch, tok);
  if (b < 0) return;
  const int ps = a.cache.page_size;
  const SeqRange r = seq_range(a.batch, ps, b);
  if (r.n == 0) return;
  const int t = r.len - r.n + tok - r.tok0;
  const uint16_t* q = a.q + row * (DC + DR);
  for (int i = lane; i < DC + DR; i += 32) s_q[warp][i] = bf16_to_f32(q[i]) * a.scale_log2;
  __syncwarp();
  const int lo = a.window > 0 ? max(0, t - a.window + 1) : 0;
  const int sinks = a.window > 0 ? min(a.n_sink, lo) : 0;
  float m = -INFINITY, l = 0.f, acc[kPer];
#pragma unroll
  for (int e = 0; e < kPer; ++e) acc[e] = 0.f;
  const int n_keys = sinks + t + 1 - lo;
  for (int k0 = 0; k0 < n_keys; k0 += 32) {
    const int k = k0 + lane;
    const int s = k < sinks ? k : lo + k - sinks;
    float z = -INFINITY, sc = 0.f;
    int page = -1;
    if (k < n_keys) {
      page = __ldg(a.batch.page_table + static_cast<int64_t>(b) * a.batch.max_pages + s / ps);
      if (page < 0 || page >= a.cache.n_pages) {
        page = -1;
        report(a.ws, kDevRange, kCacheSitePage);
      } else {
        sc = pow2f(scale_exp(__ldg(a.cache.scale + page)));
        const uint8_t* lat = a.cache.latent + page * a.cache.latent_page_stride + (s % ps) * DC;
        const uint8_t* rope = a.cache.rope + page * a.cache.rope_page_stride + (s % ps) * DR;
        float d = 0.f;
        for (int u = 0; u < (DC + DR) / 16; ++u) {
          const uint4 v = __ldg(reinterpret_cast<const uint4*>(u < DC / 16 ? lat + u * 16
                                                                           : rope + u * 16 - DC));
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
          const float* qq = &s_q[warp][u * 16];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 x = e4m3x2_to_f32(w[e]), y = e4m3x2_to_f32(w[e] >> 16);
            d += x.x * qq[4 * e] + x.y * qq[4 * e + 1] + y.x * qq[4 * e + 2] + y.y * qq[4 * e + 3];
          }
        }
        z = d * sc;
      }
    }
    float mx = z;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    if (mx == -INFINITY) continue;
    const float m_new = fmaxf(m, mx), f = exp2f(m - m_new), p = exp2f(z - m_new);
    m = m_new;
    l = l * f + p;
#pragma unroll
    for (int e = 0; e < kPer; ++e) acc[e] *= f;
    for (int i = 0; i < 32; ++i) {
      const int pg = __shfl_sync(0xffffffffu, page, i);
      const int ss = __shfl_sync(0xffffffffu, s, i);
      const float w = __shfl_sync(0xffffffffu, p * sc, i);
      if (pg < 0) continue;
      const uint8_t* lat = a.cache.latent + pg * a.cache.latent_page_stride + (ss % ps) * DC;
#pragma unroll
      for (int e = 0; e < kPer; e += 2) {
        const float2 x = e4m3x2_to_f32(
            __ldg(reinterpret_cast<const uint16_t*>(lat + lane * 2 + e * 32)));
        acc[e] += w * x.x;
        acc[e + 1] += w * x.y;
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  const float inv = l > 0.f ? 1.f / l : 0.f;
  uint16_t* out = a.out + row * DC;
#pragma unroll
  for (int e = 0; e < kPer; e += 2) {
    out[lane * 2 + e * 32] = f32_to_bf16_rne(acc[e] * inv);
    out[lane * 2 + e * 32 + 1] = f32_to_bf16_rne(acc[e + 1] * inv);
  }
  if (a.lse && lane == 0) a.lse[row] = l > 0.f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

// Sequences that fail the checks of dsa_batch.
__global__ void cache_attn_check(const __grid_constant__ CacheAttnArgs a) {
  for (int b = threadIdx.x; b < a.batch.n_seq; b += blockDim.x)
    if (!seq_range(a.batch, a.cache.page_size, b).ok) report(a.ws, kDevRange, kCacheSiteSeq);
}

}  // namespace

size_t cache_attn_scratch_bytes(const dsa_cache& c, const dsa_batch&, int) {
  if (c.d_latent != kDC) return 0;
  // laid out for 64 rows an item, whichever form the lengths call for
  return kMaxCtas * (sizeof(CtaMeta) + 2 * 64 * (sizeof(float2) + kDC * sizeof(float)));
}

namespace {

cudaError_t launch_rows(const CacheAttnArgs& a, cudaStream_t st) {
  cudaError_t e = cudaMemsetAsync(a.ws, 0, kWsHeaderBytes, st);
  if (e != cudaSuccess) return e;
  cache_attn_check<<<1, 256, 0, st>>>(a);
  const int64_t rows = static_cast<int64_t>(a.batch.n_tok) * a.n_heads;
  const unsigned grid = static_cast<unsigned>((rows + kRowWarps - 1) / kRowWarps);
  cache_attn_rows<64, 16><<<grid, 32 * kRowWarps, 0, st>>>(a);
  return cudaGetLastError();
}

template <int R>
cudaError_t launch_tc(const CacheAttnArgs& a, void* scratch, cudaStream_t st) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(cache_attn_tc<R>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             Cfg<R>::kSmemBytes);
  if (e != cudaSuccess) return e;
  CUtensorMap ml, mr;
  const dsa_cache& c = a.cache;
  if (!make_tmap_u8_pages(&ml, c.latent, kDC, c.page_size, c.n_pages, c.latent_page_stride, 128,
                          CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_tmap_u8_pages(&mr, c.rope, kDR, c.page_size, c.n_pages, c.rope_page_stride, kDR,
                          CU_TENSOR_MAP_SWIZZLE_64B))
    return cudaErrorInvalidValue;
  const int grid = sms < kMaxCtas ? sms : kMaxCtas;
  CacheAttnParams p;
  p.a = a;
  char* w = static_cast<char*>(scratch);
  p.meta = reinterpret_cast<CtaMeta*>(w);
  w += kMaxCtas * sizeof(CtaMeta);
  p.part_ml = reinterpret_cast<float2*>(w);
  w += kMaxCtas * 2 * R * sizeof(float2);
  p.part_o = reinterpret_cast<float*>(w);
  cache_attn_tc<R><<<grid, kThreads, Cfg<R>::kSmemBytes, st>>>(p, ml, mr);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cache_attn_combine<R><<<grid, kCombineThreads, 0, st>>>(p, grid);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_attn(const CacheAttnArgs& a, void* scratch, cudaStream_t st) {
  if (a.cache.d_latent != kDC) return launch_rows(a, st);
  // R = 32 when the sequences have no more than 32 rows on average
  const int64_t rows = static_cast<int64_t>(a.batch.n_tok) * a.n_heads;
  return rows <= 32ll * a.batch.n_seq ? launch_tc<32>(a, scratch, st)
                                      : launch_tc<64>(a, scratch, st);
}

}  // namespace dsa
