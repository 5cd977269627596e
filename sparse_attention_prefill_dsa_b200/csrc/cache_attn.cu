// cache_attn.cu -- attention over the paged 8-bit latent cache.
//
//   z_s = scale * s_p * (q . code_s),  s <= t, and s > t - window or s < n_sink
//   out = sum_s softmax(z)_s * s_p * code_s[:Dc],   lse = log sum_s exp(z_s)
//
// The (512, 64) shape runs on tcgen05 with the cache's own bytes as operands:
// a tile of 128 keys goes from the pages to swizzled shared memory by TMA and
// is never converted. kind::f8f6f4 multiplies 8-bit types, so the other operand
// is split instead: q = qs * (hi + lo/16) and p = hi + lo in two 8-bit parts. A
// bf16 q has 8 significant bits and e4m3 has 4, and the residual of rounding 8
// bits to 4 is a signed 4-bit number: hi + lo is q itself (down to 2^-22 of the
// row's largest element, where lo leaves e4m3's range). For p the residual is
// rounded once more: apart from hi (R = 32 below) to e4m3, to 2^-9 of p, 6e-4
// rms; on hi's own accumulators (R = 64) to e5m2, to 2^-8 of p, 1.3e-3 rms, where
// a bf16 p has 2^-8 and 1.6e-3 rms. Those bounds end at 2^-15 (2^-14) of the
// row's reference, below.
// Work of a tile, for R query rows (token, head) of one sequence:
//   QK^T  S^T[key, (hi, lo) x row] = K . Q^T      M = 128 keys, N = 2R, K = 576
//   softmax, one thread per key lane              p'' = 2^(z log2e + e_p - m)
//   PV    O^T[dim, row] += V^T . P^T              M = 128 dims x 4, K = 128 keys
// V is the latent part of the K tile read MN-major. The page scales 2^e_p stay
// out of the MMAs: in the logits they multiply S, in the output they are added
// to p's exponent, and the row sum takes p'' 2^-e_p.
// m is a row's reference, an integer that keeps p'' where its parts are exact: it
// is set so that the row's largest p'' of a tile is 2^5 to 2^6, raised when a
// value passes 2^8 (e4m3 ends at 448), and lowered when all are below 1/8, so
// that the flat tail behind one large weight (a first token's, say) does not
// fall below the parts' last bits: with a reference that only rose, a row whose
// first key has 0.8 of the weight of 17,000 was off by 40 %. O and l are rescaled
// then, O in tensor memory, by a power of two. A tile whose values stay inside needs
// no exchange between threads but one vote. That a row has fallen is noticed a
// tile later (found before the tile's own products it cost 4.5 %, so 2 %), but
// for a tile after a weight far above others, which is looked at in any case. So
// a weight is off by 2^-8 of itself at most or, if that is more, by 2^-11
// (R = 64) or 2^-12 of the largest in its tile or the one before. Logits that
// differ more move it more often: 2,048 queries at 8,192 keys took 886 / 896 us
// with the former reference and now at a standard deviation of 1, 895 / 930 at
// 2, 894 / 1,029 at 3 (lowered below 1/2 already, 972 and 1,117).
// Rows of a tile: R = 32 (P's hi and lo side by side as N = 64, O_hi and O_lo
// apart) when no sequence can be expected to have more rows, as in decode,
// where the bytes bound; R = 64 else (P's lo and hi passes onto one O, N = 64),
// which shares the loads between twice as many rows. Shared memory: Q 36 or
// 72 KB, two tiles of 72 KB, P 8 KB; at R = 64 P's hi takes the place of the
// tile's rope chunk, which is dead by then. A tile's place is handed out in four
// chunks of 128 dims (the rope with the last): PV releases each as it goes, so
// the next but one tile loads under it.
//
// Work is split over SMs by tiles, not by sequences: the tiles of all items
// (R rows of one sequence) form one list, and CTA c of G takes its c-th part.
// An item that crosses CTAs leaves partial results in the workspace, which
// cache_attn_combine joins. The list's length comes from the batch arrays, so
// each CTA counts it for itself; nothing of it is needed on the host.
//
// What bounds it (B200, 1.9 GHz; times with the combine pass):
//  - R = 64: 2,048 queries x 32 heads at 8,192 keys 1.05 ms (972 TFLOP/s), 8,192
//    queries with a window of 2,048 + 16 keys 1.57 ms (748 TFLOP/s). The MMAs of
//    a tile read 344 KB of operands at 128 bytes a clock, 2,690 clocks, of which
//    their math is 2,180; a tile takes about 3,800. The difference is the
//    turnaround of a tile's place: PV done, seen by the producer (about 600
//    clocks), loaded (about 400), seen by the MMA warp. A third place would hide
//    it and does not fit beside 72 KB of Q. An item begins with 8,000 clocks for
//    its Q, partly under the last PV.
//  - R = 32: 64 sequences of 1 to 17,408 rows 108 us (3.1 TB/s of cache bytes;
//    about 5 TB/s between the first tile and the last). QK^T (1,000 clocks),
//    softmax (1,300) and PV (950) of a tile follow each other unless the next
//    tile has landed in time; the loads alone would take 3,300 clocks a tile at
//    6.5 TB/s. Skipping half of the loads changed the time by 2 %, L2 prefetches
//    of later tiles made it 10 % longer.
//  - one sequence of 17,408 rows 22.5 us: 16 us of the first kernel, most of it
//    the chain schedule - Q - first tile - epilogue of cold loads, then the
//    combine pass.
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
constexpr int HR = 16;  // query rows of a softmax warpgroup

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
  long long wait_cycles;  // limit of a wait
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
  __device__ __forceinline__ bool seen(int s) const {
    return s <= t_hi && (s >= win_lo || s < sink_hi);
  }
};

// The keys that the rows [i0, i1] of a sequence (token * n_heads + head, its
// first new token at position `first`) see, and the tiles with them.
struct KeyRange {
  int t_lo, t_hi, win_lo, sink_hi, nst, wt0, nt;
};

__device__ __forceinline__ KeyRange key_range(const CacheAttnArgs& a, int first, unsigned i0,
                                              unsigned i1) {
  KeyRange k;
  k.t_lo = first + static_cast<int>(i0 / static_cast<unsigned>(a.n_heads));
  k.t_hi = first + static_cast<int>(i1 / static_cast<unsigned>(a.n_heads));
  k.win_lo = a.window > 0 ? max(0, k.t_lo - a.window + 1) : 0;
  k.sink_hi = a.window > 0 ? min(a.n_sink, k.win_lo) : 0;
  k.nst = (k.sink_hi + kKeys - 1) / kKeys;
  k.wt0 = max(k.win_lo / kKeys, k.nst);
  k.nt = k.nst + k.t_hi / kKeys - k.wt0 + 1;
  return k;
}

__device__ __forceinline__ Item make_item(const CacheAttnArgs& a, int b, const SeqRange& r, int i0,
                                          int n_rows, const KeyRange& k) {
  Item it;
  it.b = b;
  it.i0 = i0;
  it.n_rows = n_rows;
  it.row = r.tok0 * a.n_heads + i0;
  it.first = r.len - r.n;
  it.t_lo = k.t_lo;
  it.t_hi = k.t_hi;
  it.win_lo = k.win_lo;
  it.sink_hi = k.sink_hi;
  it.nst = k.nst;
  it.wt0 = k.wt0;
  it.nt = k.nt;
  return it;
}

template <int R>
__device__ __forceinline__ int64_t slots_of(const CacheAttnArgs& a) {
  return static_cast<int64_t>(a.batch.n_tok) * a.n_heads / R + a.batch.n_seq;
}

template <int R>
struct ItemWalk {
  static constexpr int kShift = R == 32 ? 5 : 6;
  // Slot `slot` of the sequences' slots (R rows each), sequence b.
  int64_t slot, start, stop;
  int b;
  SeqRange r;

  // (not inlined: the walk is off the critical paths, and the kernel's
  // instructions have to stay within the instruction cache)
  __device__ __noinline__ void load(const CacheAttnArgs& a) {
    start = slot_start(a.batch, b, a.n_heads, kShift, 1);
    stop = b + 1 < a.batch.n_seq ? slot_start(a.batch, b + 1, a.n_heads, kShift, 1) : INT64_MAX;
    r = seq_range(a.batch, a.cache.page_size, b);
  }
  __device__ __noinline__ void seek(const CacheAttnArgs& a, int64_t s) {
    slot = s;
    b = seq_of_slot(a.batch, s, a.n_heads, kShift, 1);
    load(a);
  }
  __device__ __noinline__ void next(const CacheAttnArgs& a) {
    ++slot;
    while (slot >= stop && b + 1 < a.batch.n_seq) {
      ++b;
      load(a);
    }
  }
  // Tiles of this slot's item, 0 when the sequence has no such rows.
  __device__ __noinline__ int item(const CacheAttnArgs& a, Item& it) const {
    const int64_t rb = slot - start;
    const int64_t rows = static_cast<int64_t>(r.n) * a.n_heads;
    if (rb < 0 || rb * R >= rows) return 0;
    const int i0 = static_cast<int>(rb * R);
    const int n_rows = static_cast<int>(min(static_cast<int64_t>(R), rows - i0));
    it = make_item(a, b, r, i0, n_rows, key_range(a, r.len - r.n, i0, i0 + n_rows - 1));
    return it.nt;
  }
};

// Tiles [k0, k1) of an item, as the producer publishes them to the other
// warps; more: the CTA has another segment after it.
struct Segment {
  Item it;
  int k0, k1, more, pad;
};

// A CTA's part of the tile list as segments, one after the other.
template <int R>
struct SegmentWalk {
  ItemWalk<R> w;
  Item it;
  int k0, k1;
  int64_t left;  // tiles after this segment
  int64_t slots;
  bool at_first = true;  // the walk has not been set up yet
  int64_t slot0;
  // From the CTA's first segment, of the item of `slot`, for n > 0 tiles.
  __device__ void begin(const Segment& first, int64_t slot, int64_t n) {
    it = first.it;
    k0 = first.k0;
    k1 = first.k1;
    left = n - (k1 - k0);
    slot0 = slot;
  }
  __device__ bool next(const CacheAttnArgs& a) {
    if (left <= 0) return false;
    if (at_first) {
      slots = slots_of<R>(a);
      w.seek(a, slot0);
      at_first = false;
    }
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

// Published segments. The producer publishes a segment three tiles before it
// loads its first; a tile's place is loaded again once its PV is done, which
// every warp has taken part in. So the warp that is furthest behind is at most
// six tiles, and segments, behind.
constexpr int kSegSlots = 8;
static_assert(sizeof(Segment) <= 64, "segment slot");

// What the producer tells the softmax of a tile, in a ring of four, a tile
// before it loads it.
struct TileInfo {
  int exp[8];  // the scale exponents of its pages, kNoPage where nothing was loaded
  int t0;      // first key
  int masked;  // some row does not see some key
  int pad[2];
};
static_assert(sizeof(TileInfo) == 48, "tile info");

// Shared words after the barriers.
struct Misc {
  unsigned int status, info;  // stands in for the header of a workspace in report()
  uint32_t tmem;
  int abort_flag;
  long long slot, n_tiles, total, begin;
};
static_assert(sizeof(Misc) <= 48, "misc");

// mbarriers: what TMA and the tensor cores arrive on, and rare events.
enum Bars {
  kFull = 0,              // [2 stages][4 chunks] a chunk has landed (the last with the rope)
  kEmpty = 8,             // [2][4] the PV is done with it
  kSFull = 16,            // [2] QK^T of a tile is done
  kPvDone = 18,           // PV of a tile is done
  kQFull,                 // the segment's Q is written
  kOFree,                 // the segment's O has been read
  kPFull,                 // P of a tile is written (kPollP)
  kSeg,                   // [kSegSlots] a segment is published
  kInfo = kSeg + kSegSlots,  // [4] a tile's info is in place
  kDrain = kInfo + 4,
  kBarCount
};

// Hardware barriers. The MMAs read their operands from shared memory at its
// full 128 bytes a clock, and whatever else reads it then waits for a gap
// between two of them (a dependent load takes 114 clocks instead of 40, and
// warps that poll an mbarrier wait for each other). So two relay warps poll for
// all softmax warps, and the rest of the exchange between them and the MMA warp
// is on these, which take no shared memory. Those in pairs go by the tile's
// parity: one side may be a tile ahead of the other, never two (a tile's place
// in shared memory is loaded again only after its PV).
enum HwBars {
  kVote = 1,     // [groups] within a softmax warpgroup
  kAll = 5,      // all softmax warps
  kSReady = 6,   // [2] relay -> softmax: S of a tile, and the info of the next
  kPvReady = 8,  // [2] relay -> softmax: PV of a tile is done
  kSFree = 10,   // [2] softmax -> MMA: S has been read
  kPReady = 12   // softmax -> MMA: P is written (not kPollP)
};

template <int R>
struct Cfg {
  static constexpr int kGroups = R / HR;           // softmax warpgroups: warps 0 .. 4 kGroups - 1
  static constexpr int kWarps = 4 * kGroups;       // (a warp reads the TMEM lanes of its index mod 4)
  static constexpr int kThreads = 32 * (kWarps + 4);  // + producer, MMA, two relays
  static constexpr int kSync = 32 * (kWarps + 1);     // the softmax warps and one other
  static constexpr bool kSplitO = R == 32;         // hi and lo of P onto their own columns of O
  static constexpr bool kPollP = R == 32;          // the MMA warp takes what is ready first (below)
  static constexpr int kQChunk = 2 * R * 128;      // 128 dims of the hi and lo rows
  static constexpr int kQBytes = 2 * R * (kDC + kDR);
  static constexpr int kTmemS = 0, kTmemO = 4 * R;  // S^T [2 buffers][2R], O^T [4][64]
  static constexpr int kOffQ = 0;
  static constexpr int kOffStage = kQBytes;
  static constexpr int kOffP = kOffStage + 2 * kStageBytes;
  static constexpr int kOffM = kOffP + kKeys * 64;       // float [warps][HR]
  static constexpr int kOffRow = kOffM + 16 * HR * 4;    // float rowfac[64], uint8 row_dt[64]
  static constexpr int kOffSeg = kOffRow + 64 * 5;       // Segment [kSegSlots]
  static constexpr int kOffTile = kOffSeg + kSegSlots * 64;  // TileInfo [4]
  static constexpr int kOffBar = kOffTile + 4 * 48;
  static constexpr int kNumBars = kBarCount;
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;
  static constexpr int kMiscBytes = 48;
  static constexpr int kSmemBytes = kOffMisc + kMiscBytes;
  static constexpr uint32_t kIdescQK = idesc_e4m3_f32(128, 2 * R);
  static constexpr uint32_t kIdescPV = idesc_e4m3_f32(128, 64, true, true);
  static constexpr uint32_t kIdescPVLo = idesc_e4m3_f32(128, 64, true, true, !kSplitO);  // (e5m2)
  static_assert(kOffStage % 1024 == 0 && kOffP % 1024 == 0, "operand alignment");
  static_assert(kSmemBytes <= 232448, "shared memory");
  static_assert(kTmemO + 256 <= 512, "tensor memory");
};

enum Sites { kSiteEmpty = 40, kSiteFull, kSiteSFull, kSitePv, kSiteQ, kSiteO, kSiteSeg, kSiteInfo, kSiteP };

constexpr unsigned kPollPauseNs = 20;  // (0 to 100 measured alike)
constexpr long long kPollCheckCycles = 1 << 20;  // waits shorter than this look at every poll
// A steadfast wait (below) outlasts a chain of the MMA warp's own waits.
constexpr long long kSteadfastCycles = 8 * kWaitLimitCycles;
constexpr int kNoPage = 1 << 20;

// The kernel's shared memory: a symbol, so that operand addresses are
// constants (uniform registers of the MMA warp). Swizzled operands need a
// 1024-byte boundary, checked when the kernel starts.
extern __shared__ __align__(1024) unsigned char cache_attn_smem[];

// Hardware barriers by number. The warp has to be converged there; waits and
// single-lane blocks before them may leave it split.
__device__ __forceinline__ void named_sync(int id, int threads) {
  __syncwarp();
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

__device__ __forceinline__ void named_arrive(int id, int threads) {
  __syncwarp();
  asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

__device__ __forceinline__ bool named_or(int id, int threads, bool p) {
  uint32_t r;
  __syncwarp();
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

// log(2^m sum) for an integer m. The exponent of sum > 0 goes to m first: where
// the pages' scales are far from 1 the two are large and of opposite sign.
__device__ __forceinline__ float log_sum(float m, float sum) {
  const uint32_t b = __float_as_uint(sum);
  const float e = static_cast<float>(static_cast<int>(b >> 23) - 127);
  return (m + e + log2f(__uint_as_float((b & 0x7FFFFFu) | 0x3F800000u))) * 0.69314718055994531f;
}

// Sum of v[e] over the 32 lanes for every e; lane l gets that of e = l % 16.
__device__ __forceinline__ float warp_transpose_sum(float (&v)[16]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int e = 0; e < 16; ++e) v[e] += __shfl_xor_sync(0xffffffffu, v[e], 16);
#pragma unroll
  for (int s = 8; s >= 1; s >>= 1) {
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

// ------------------------------------------------------------------ schedule

// CTA c's part of `total` tiles on `grid` CTAs starts at this tile (CTAs past
// the number of tiles have none).
__device__ __noinline__ long long part_begin(long long total, int grid, int c) {
  const unsigned long long g = min(static_cast<long long>(grid), total);
  if (static_cast<unsigned long long>(c) >= g) return total;
  if (total < (1 << 24)) return static_cast<unsigned>(total) * c / static_cast<unsigned>(g);
  return static_cast<long long>(static_cast<unsigned long long>(total) * c / g);
}

// The CTA up to `last` whose part of the list holds tile `at`.
__device__ __noinline__ int cta_of_tile(long long at, long long total, int grid, int last) {
  int lo = 0;
  while (lo < last) {
    const int mid = (lo + last + 1) >> 1;
    if (part_begin(total, grid, mid) <= at) lo = mid;
    else last = mid - 1;
  }
  return lo;
}

// Counts the tiles of all items and finds this CTA's part and its first
// segment. All threads; `scan` is scratch for a long long of each warp.
template <int R>
__device__ void schedule(const CacheAttnArgs& a, Misc* ms, long long* scan, Segment* first) {
  constexpr int kThreads = Cfg<R>::kThreads;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // the slots need cu_seqlens that ascend; if they do not, there is no work
  int bad = 0;
  for (int b = tid; b < a.batch.n_seq; b += kThreads) {
    const SeqRange r = seq_range(a.batch, a.cache.page_size, b);
    const int c1 = __ldg(a.batch.cu_seqlens + b + 1);
    bad |= r.tok0 < 0 || c1 < r.tok0 || c1 > a.batch.n_tok;
    if (!r.ok && blockIdx.x == 0)
      report(reinterpret_cast<WsHeader*>(&ms->status), kDevRange, kCacheSiteSeq);
  }
  const int64_t slots = __syncthreads_or(bad) ? 0 : slots_of<R>(a);
  const int64_t per = (slots + kThreads - 1) / kThreads;
  const int64_t s0 = min(slots, tid * per), s1 = min(slots, s0 + per);
  // The slots [s0, s1) in order; `at` gets a slot's sequence, its first row
  // there and its keys, and tells whether to stop.
  auto walk = [&](auto at) {
    if (s0 >= s1) return;
    constexpr int kShift = ItemWalk<R>::kShift;
    int b = seq_of_slot(a.batch, s0, a.n_heads, kShift, 1);
    SeqRange r = seq_range(a.batch, a.cache.page_size, b);
    int64_t start = slot_start(a.batch, b, a.n_heads, kShift, 1);
    auto stop_of = [&] {
      return b + 1 < a.batch.n_seq ? slot_start(a.batch, b + 1, a.n_heads, kShift, 1) : INT64_MAX;
    };
    int64_t stop = stop_of();
#pragma unroll 1
    for (int64_t s = s0; s < s1; ++s) {
      while (s >= stop) {
        ++b;
        r = seq_range(a.batch, a.cache.page_size, b);
        start = stop;
        stop = stop_of();
      }
      const int64_t i0 = (s - start) * R, rows = static_cast<int64_t>(r.n) * a.n_heads;
      if (i0 < rows) {
        const int n_rows = static_cast<int>(min(static_cast<int64_t>(R), rows - i0));
        const KeyRange k = key_range(a, r.len - r.n, static_cast<unsigned>(i0),
                                     static_cast<unsigned>(i0) + n_rows - 1);
        if (at(s, b, r, static_cast<int>(i0), n_rows, k)) return;
      }
    }
  };
  long long sum = 0;
  walk([&](int64_t, int, const SeqRange&, int, int, const KeyRange& k) {
    sum += k.nt;
    return false;
  });
  long long inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) scan[warp] = inc;
  __syncthreads();
  long long before = 0, total = 0;
  for (int i = 0; i < kThreads / 32; ++i) {
    if (i < warp) before += scan[i];
    total += scan[i];
  }
  const long long begin = part_begin(total, gridDim.x, blockIdx.x);
  const long long end = part_begin(total, gridDim.x, blockIdx.x + 1);
  const long long lo = before + inc - sum;
  if (begin < end && lo <= begin && begin < lo + sum) {
    // this thread's: it publishes the CTA's first segment
    long long done = lo;
    walk([&](int64_t slot, int b, const SeqRange& r, int i0, int n_rows, const KeyRange& k) {
      if (done + k.nt <= begin) {
        done += k.nt;
        return false;
      }
      first->it = make_item(a, b, r, i0, n_rows, k);
      first->k0 = static_cast<int>(begin - done);
      first->k1 = static_cast<int>(min(static_cast<long long>(k.nt), first->k0 + end - begin));
      first->more = first->k1 - first->k0 < end - begin;
      ms->slot = slot;
      return true;
    });
  }
  if (tid == 0) {
    ms->n_tiles = end - begin;
    ms->total = total;
    ms->begin = begin;
  }
  __syncthreads();
}

// ---------------------------------------------------------------- q operand

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// The exponent e of the smallest 2^e with |x| <= 448 * 2^e.
__device__ __forceinline__ int q_exp(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int e = static_cast<int>(b >> 23) - 127 - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return min(max(e, -110), 110);
}

__device__ __forceinline__ float2 bf16x2(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

// Eight bf16 as e4m3 hi and lo codes: x * inv = hi + lo / 16. The steps in
// between are in float16: |x * inv| <= 448, and its 11 bits hold a bf16's 8.
__device__ __forceinline__ void split_q(const uint4& v, float inv, uint32_t (&hi)[2],
                                        uint32_t (&lo)[2]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t h[4], l[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 x = bf16x2(w[e]);
    const __half2 f = __floats2half2_rn(x.x * inv, x.y * inv);
    h[e] = __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(f), __NV_SATFINITE, __NV_E4M3);
    const __half2 b = __half2(
        __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(h[e]), __NV_E4M3));
    const __half2 r = __hmul2(__hsub2(f, b), __float2half2_rn(16.f));
    l[e] = __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(r), __NV_SATFINITE, __NV_E4M3);
  }
  hi[0] = h[0] | h[1] << 16;
  hi[1] = h[2] | h[3] << 16;
  lo[0] = l[0] | l[1] << 16;
  lo[1] = l[2] | l[3] << 16;
}

// Byte offset of 16-byte unit u (16 codes) of operand row n within the Q buffer.
template <int R>
__device__ __forceinline__ uint32_t q_off(int n, int u) {
  return u < kDC / 16 ? (u >> 3) * Cfg<R>::kQChunk + n * 128 + (((u & 7) ^ (n & 7)) << 4)
                      : 4 * Cfg<R>::kQChunk + n * 64 + (((u & 3) ^ ((n >> 1) & 3)) << 4);
}

// n rows from `row` on, or none where the checking build finds that they are not
// all rows of the call.
__device__ __forceinline__ int in_call(const CacheAttnArgs& a, int row, int n, WsHeader* ws,
                                       unsigned int site) {
  const int64_t rows = static_cast<int64_t>(a.batch.n_tok) * a.n_heads;
  (void)rows;
  return n <= 0 || (DSA_IN_BOUNDS(ws, row, rows, site) &&
                    DSA_IN_BOUNDS(ws, static_cast<int64_t>(row) + n - 1, rows, site))
             ? n
             : 0;
}

// The item's rows as operand rows (hi at r, lo at R + r), their factors and
// positions (less t_lo). Each softmax warp takes four rows: 144 units of 16
// elements, five for a lane.
template <int R>
__device__ void convert_q(const CacheAttnArgs& a, const Item& it, unsigned char* sq, float* rowfac,
                          uint8_t* row_dt, Misc* ms) {
  WsHeader* ws = reinterpret_cast<WsHeader*>(&ms->status);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kUnits = (kDC + kDR) / 16;  // 36 of a row
  constexpr int kRows = 4, kRounds = (kRows * kUnits + 31) / 32;
  static_assert(R == kRows * Cfg<R>::kWarps, "rows of a warp");
  const uint4* src = reinterpret_cast<const uint4*>(a.q + static_cast<int64_t>(it.row) * (kDC + kDR));
  const int r0 = warp * kRows, n_units = (min(in_call(a, it.row, it.n_rows, ws, 65), r0 + kRows) - r0) * kUnits;
  src += r0 * kUnits * 2;
  uint4 v[kRounds][2];
#pragma unroll
  for (int i = 0; i < kRounds; ++i) {
    const int x = lane + 32 * i;
    v[i][0] = v[i][1] = make_uint4(0u, 0u, 0u, 0u);
    if (x < n_units) {
      v[i][0] = __ldg(src + 2 * x);
      v[i][1] = __ldg(src + 2 * x + 1);
    }
  }
  // the rows' largest |x|: bf16 magnitudes order as integers
  uint32_t mx[kRows] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int i = 0; i < kRounds; ++i) {
    const uint32_t w[8] = {v[i][0].x, v[i][0].y, v[i][0].z, v[i][0].w,
                           v[i][1].x, v[i][1].y, v[i][1].z, v[i][1].w};
    uint32_t m = 0u;
#pragma unroll
    for (int e = 0; e < 8; ++e) m = max_u16x2(m, w[e] & 0x7FFF7FFFu);
    m = max(m & 0xFFFFu, m >> 16);
    const int j = (lane + 32 * i) / kUnits;
#pragma unroll
    for (int r = 0; r < kRows; ++r)
      if (32 * i < (r + 1) * kUnits && 32 * i + 31 >= r * kUnits) mx[r] = max(mx[r], j == r ? m : 0u);
  }
  int e_row[kRows];
#pragma unroll
  for (int r = 0; r < kRows; ++r)
    e_row[r] = q_exp(__uint_as_float(__reduce_max_sync(0xffffffffu, mx[r]) << 16));
#pragma unroll
  for (int i = 0; i < kRounds; ++i) {
    const int x = lane + 32 * i, j = x / kUnits, u = x - j * kUnits;
    if (j >= kRows) continue;
    int e = e_row[0];
#pragma unroll
    for (int r = 1; r < kRows; ++r) e = j == r ? e_row[r] : e;
    const float inv = pow2f(-e);
    uint32_t h0[2], l0[2], h1[2], l1[2];
    split_q(v[i][0], inv, h0, l0);
    split_q(v[i][1], inv, h1, l1);
    *reinterpret_cast<uint4*>(sq + q_off<R>(r0 + j, u)) = make_uint4(h0[0], h0[1], h1[0], h1[1]);
    *reinterpret_cast<uint4*>(sq + q_off<R>(R + r0 + j, u)) = make_uint4(l0[0], l0[1], l1[0], l1[1]);
  }
#pragma unroll
  for (int r = 0; r < kRows; ++r)
    if (lane == r) {
      rowfac[r0 + r] = pow2f(e_row[r]) * a.scale_log2;
      row_dt[r0 + r] = static_cast<uint8_t>(
          it.first + (it.i0 + min(r0 + r, it.n_rows - 1)) / a.n_heads - it.t_lo);
    }
}

// -------------------------------------------------------------------- kernel

// The polling loop of a wait, once for all waits. Polls read shared memory,
// which the MMAs keep busy: a warp that polls without a pause holds up the
// others' (a producer that shared it with three such warps took 570 clocks for
// each wait, barrier and load of a chunk). It gives up after `limit` clocks, or
// when another wait of the block has; a steadfast one only after its limit.
__device__ __noinline__ bool wait_on(uint64_t* bar, uint32_t parity, Misc* ms, unsigned site,
                                     long long limit, bool steadfast) {
  const long long t0 = clock64();
  for (uint32_t i = 1;; ++i) {
    __nanosleep(kPollPauseNs);
    if (mbar_test_wait(bar, parity)) return true;
    if ((i & 63u) == 0u || limit < kPollCheckCycles) {
      if (!steadfast && *reinterpret_cast<volatile int*>(&ms->abort_flag)) return false;
      if (clock64() - t0 > limit) {
        ms->abort_flag = 1;
        report(reinterpret_cast<WsHeader*>(&ms->status), kDevTimeout, site);
        return false;
      }
    }
  }
}

template <int R>
struct Ctx {
  const CacheAttnParams& p;
  __device__ __forceinline__ unsigned char* s() const { return cache_attn_smem; }
  __device__ __forceinline__ uint64_t* bar(int b) const {
    return reinterpret_cast<uint64_t*>(cache_attn_smem + Cfg<R>::kOffBar) + b;
  }
  __device__ __forceinline__ Misc* ms() const {
    return reinterpret_cast<Misc*>(cache_attn_smem + Cfg<R>::kOffMisc);
  }
  __device__ __forceinline__ Segment* segment(int seg) const {
    return reinterpret_cast<Segment*>(cache_attn_smem + Cfg<R>::kOffSeg) + seg % kSegSlots;
  }
  __device__ __forceinline__ TileInfo* info(int i) const {
    return reinterpret_cast<TileInfo*>(cache_attn_smem + Cfg<R>::kOffTile) + (i & 3);
  }
  __device__ __forceinline__ bool wait(int b, uint32_t parity, unsigned site) const {
    return mbar_test_wait(bar(b), parity) ||
           wait_on(bar(b), parity, ms(), site, p.wait_cycles, false);
  }
  // For what comes also after a timeout, and keeps the warps in step.
  __device__ __forceinline__ void wait_steadfast(int b, uint32_t parity, unsigned site) const {
    if (!mbar_test_wait(bar(b), parity))
      wait_on(bar(b), parity, ms(), site, kSteadfastCycles, true);
  }
  __device__ __forceinline__ bool wait_segment(int seg) const {
    return wait(kSeg + seg % kSegSlots, (seg / kSegSlots) & 1, kSiteSeg);
  }
  __device__ void error(unsigned site) const {
    report(reinterpret_cast<WsHeader*>(&ms()->status), kDevRange, site);
  }
};
static_assert(sizeof(Segment) == 64, "segments are an array of slots");

__device__ __forceinline__ void drain_wait(uint64_t* bar, uint32_t parity) {
  const long long t0 = clock64();
  while (!mbar_try_wait(bar, parity))
    if (clock64() - t0 > kWaitLimitCycles) break;
}

// How far the producer came: its last tile, and the chunks that it asked for of it.
struct Begun {
  int tile, chunks;
};

// Producer warp: lane l < 128 / page_size loads the tile's l-th page.
template <int R>
__device__ Begun producer(const Ctx<R>& x, const CUtensorMap* ml, const CUtensorMap* mr) {
  const CacheAttnArgs& a = x.p.a;
  const int lane = threadIdx.x & 31, ps = a.cache.page_size, npt = kKeys / ps;
  const int n = static_cast<int>(x.ms()->n_tiles);
  SegmentWalk<R> sg;
  sg.begin(*x.segment(0), x.ms()->slot, n);
  int seg = 1;
  auto publish = [&] {
    if (lane == 0) {
      Segment* out = x.segment(seg);
      out->it = sg.it;
      out->k0 = sg.k0;
      out->k1 = sg.k1;
      out->more = sg.left > 0;
      mbar_arrive(x.bar(kSeg + seg % kSegSlots));
    }
    ++seg;
  };
  if (lane == 0) {
    mbar_arrive(x.bar(kSeg));  // (the first is there)
    // an item that began in another CTA and ends here: this CTA's entry tells
    // the combine pass of it
    CtaMeta& me = x.p.meta[blockIdx.x];
    me.n_rows = 0;
    if (sg.k0 > 0 && sg.k1 == sg.it.nt) {
      me.row = sg.it.row;
      me.n_rows = sg.it.n_rows;
      me.first = cta_of_tile(x.ms()->begin - sg.k0, x.ms()->total, gridDim.x, blockIdx.x);
    }
  }
  // The segment that is being planned, in registers (the walk itself is in
  // local memory, and reading it for every tile took longer than the loads).
  const int32_t* table;
  int k, k1, nst, wt0, t_lo, t_hi, win_lo, sink_hi;
  auto enter = [&] {
    table = a.batch.page_table + static_cast<int64_t>(sg.it.b) * a.batch.max_pages;
    k = sg.k0;
    k1 = sg.k1;
    nst = sg.it.nst;
    wt0 = sg.it.wt0;
    t_lo = sg.it.t_lo;
    t_hi = sg.it.t_hi;
    win_lo = sg.it.win_lo;
    sink_hi = sg.it.sink_hi;
  };
  enter();
  // A tile's plan: whether some row of the item sees any of this lane's page,
  // the page as the table has it (any number), the tile's first key, whether all
  // rows see all of it.
  const int page_shift = 31 - __clz(ps);
  struct Plan {
    int page, t0;
    bool whole, wanted;
  };
  auto plan = [&] {
    Plan p;
    p.t0 = (k < nst ? k : wt0 + k - nst) * kKeys;
    p.whole = p.t0 + kKeys - 1 <= t_lo &&
              (a.window == 0 || p.t0 > t_hi - a.window || p.t0 + kKeys <= a.n_sink);
    const int s0 = p.t0 + lane * ps;
    p.wanted = lane < npt && s0 <= t_hi && (s0 + ps > win_lo || s0 < sink_hi);
    p.page = p.wanted ? __ldg(table + (s0 >> page_shift)) : -1;
    if (++k == k1 && sg.next(a)) {
      enter();
      publish();
    }
    return p;
  };
  auto in_pool = [&](int page) { return page >= 0 && page < a.cache.n_pages; };
  auto scale_of = [&](const Plan& p) { return in_pool(p.page) ? __ldg(a.cache.scale + p.page) : 0.f; };
  auto tell = [&](int i, const Plan& p, float sc) {
    const bool has = in_pool(p.page);
    if (p.wanted && !has) x.error(kCacheSitePage);
    const bool full = __all_sync(0xffffffffu, has || lane >= npt) && p.whole;
    TileInfo* out = x.info(i);
    if (lane < npt) out->exp[lane] = has ? scale_exp(sc) : kNoPage;
    if (lane == 0) {
      out->t0 = p.t0;
      out->masked = !full;
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(x.bar(kInfo + (i & 3)));
  };
  // Tile i is loaded, tile i + 1 has its pages and gets its scales, tile i + 2
  // gets its pages.
  Plan now = plan(), next = now, after = now;
  if (n > 1) next = plan();
  float sc0 = 0.f;
  bool ok = true;
  int c_failed = 0, i = 0;
#pragma unroll 1
  for (; i < n && ok; ++i) {
    if (i + 2 < n) after = plan();
    const int pg = in_pool(now.page) ? now.page : -1;
    const int bytes = __popc(__ballot_sync(0xffffffffu, pg >= 0)) << page_shift;
    const int st = i & 1;
    unsigned char* dst = x.s() + Cfg<R>::kOffStage + st * kStageBytes;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      if (i >= 2 && ok) ok = x.wait(kEmpty + 4 * st + c, ((i >> 1) - 1) & 1, kSiteEmpty);
      ok = __all_sync(0xffffffffu, ok);
      if (ok) {
        uint64_t* full = x.bar(kFull + 4 * st + c);
        if (c == 0) {
          // All four barriers are armed at once (each arrival costs a turn at
          // shared memory). Not before the first chunk is free: until QK^T of
          // the tile that was there is done they may still wait for its loads.
          if (lane < 4) mbar_arrive_expect_tx(full + lane, bytes * (lane < 3 ? 128 : 128 + kDR));
          __syncwarp();
        }
        if (pg >= 0) {
          tma_load_3d(dst + c * kChunkBytes + lane * ps * 128, ml, c * 128, 0, pg, full);
          if (c == 3) tma_load_3d(dst + kRopeOff + lane * ps * kDR, mr, 0, 0, pg, full);
        }
        c_failed = c + 1;  // chunks of this tile that were asked for
      } else if (c == 0) {
        c_failed = 0;
      }
    }
    if (i == 0) sc0 = scale_of(now);
    const float sc1 = i + 1 < n ? scale_of(next) : 0.f;
    if (i == 0) tell(0, now, sc0);
    if (i + 1 < n) tell(i + 1, next, sc1);
    now = next;
    next = after;
  }
  return {i - 1, c_failed};
}

// No copy may be in flight when the block ends, and after a timeout nobody else
// waits for the last ones. Tile b.tile was begun up to chunk b.chunks, the tile
// before it in full; the one before that landed if tile b.tile was begun.
template <int R>
__device__ __noinline__ void drain_copies(const Ctx<R>& x, const Begun b) {
  for (int c = 0; c < 4; ++c) {
    const int j0 = b.chunks == 0 ? max(b.tile - 2, 0) : max(b.tile - 1, 0);
    const int j1 = c < b.chunks ? b.tile : b.tile - 1;
    for (int j = j0; j <= j1; ++j) drain_wait(x.bar(kFull + 4 * (j & 1) + c), (j >> 1) & 1);
  }
}

// Waits until one of two phases is complete: 1 or 2 (the first if both are), 0
// after a timeout. The whole warp, one answer.
__device__ __noinline__ int wait_either(uint64_t* a, uint32_t pa, uint64_t* b, uint32_t pb, Misc* ms,
                                        unsigned site, long long limit) {
  const long long t0 = clock64();
  for (uint32_t i = 1;; ++i) {
    int r = mbar_test_wait(a, pa) ? 1 : mbar_test_wait(b, pb) ? 2 : 0;
    if (r == 0) __nanosleep(kPollPauseNs);
    if (r == 0 && ((i & 63u) == 0u || limit < kPollCheckCycles)) {
      if (*reinterpret_cast<volatile int*>(&ms->abort_flag)) r = 3;
      else if (clock64() - t0 > limit) {
        ms->abort_flag = 1;
        report(reinterpret_cast<WsHeader*>(&ms->status), kDevTimeout, site);
        r = 3;
      }
    }
    r = __shfl_sync(0xffffffffu, r, 0);
    if (r != 0) return r == 3 ? 0 : r;
  }
}

// MMA warp: one thread issues. A tile's products are QK^T and, once the softmax
// has turned S into P, PV; at R = 64 QK^T runs a tile ahead, so that the
// softmax of one tile overlaps the products of another. At R = 32 the bytes
// bound, and the warp takes whichever comes first, the next tile's landing or
// P: a PV that waits for the tile would hold back the place that it frees, and
// with it the load of the tile after, and a QK^T that waits for P would leave
// the softmax without work. A segment's first QK^T comes after the last PV of
// the one before, whose epilogue it overlaps.
// After a timeout the warp goes on through all tiles without issuing, in step
// with the softmax warps as before: it arrives itself where its commits would
// have, so that the relays still tell the softmax of every product, in turn. (A
// relay that went on by itself arrived twice at a hardware barrier before the
// softmax had been there once, and some of its warps then waited for good.)
template <int R>
__device__ void mma_issuer(const Ctx<R>& x) {
  using C = Cfg<R>;
  const uint32_t sb = smem_u32(cache_attn_smem);
  const uint64_t dq = smem_desc(sb + C::kOffQ, 16, 1024, 2);
  const uint64_t dqr = smem_desc(sb + C::kOffQ + 4 * C::kQChunk, 16, 512, 4);
  const uint64_t dk = smem_desc(sb + C::kOffStage, 16, 1024, 2);
  const uint64_t dkr = smem_desc(sb + C::kOffStage + kRopeOff, 16, 512, 4);
  const uint64_t dv = smem_desc(sb + C::kOffStage, 16384, 1024, 2);
  const uint64_t dp = smem_desc(sb + C::kOffP, 512, 512, 4);
  const uint64_t dph = smem_desc(sb + C::kOffStage + kRopeOff, 512, 512, 4);
  const int n = __shfl_sync(0xffffffffu, static_cast<int>(x.ms()->n_tiles), 0);
  const bool lead = elect_one();
  bool ok = true;
  int q = 0, v = 0;         // next tiles of QK^T and PV
  int seg = 0, left = 0;    // segment of tile q, its tiles from q on (0: not looked at yet)
  uint32_t first = 0;       // bit i & 1: tile i is its segment's first
  int v_seg = -1;           // segment of the last PV
#pragma unroll 1
  for (;;) {
    bool pv = v < q && (q == n || q - v == 2 || left == 0);
    if (C::kPollP && !pv && v < q) {
      const int r = ok ? wait_either(x.bar(kFull + 4 * (q & 1) + 3), (q >> 1) & 1, x.bar(kPFull),
                                     v & 1, x.ms(), kSiteP, x.p.wait_cycles) : 0;
      ok = ok && r != 0;
      pv = r == 2;
    }
    if (pv) {
      const int i = v;
      const bool fresh = (first >> (i & 1)) & 1u;
      if constexpr (C::kPollP) x.wait_steadfast(kPFull, i & 1, kSiteP);
      else named_sync(kPReady, C::kSync);
      if (fresh && ++v_seg > 0) ok = ok && x.wait(kOFree, (v_seg - 1) & 1, kSiteO);
      ok = __all_sync(0xffffffffu, ok);
      tc_fence_after();
      if (ok && lead) {
        const uint64_t so = static_cast<uint64_t>((i & 1) * kStageBytes) >> 4;
        const uint64_t bh = C::kSplitO ? dp : dph + so;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint32_t d = C::kTmemO + 64 * c;
          const uint64_t av = dv + so + ((c * kChunkBytes) >> 4);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_f8_ss(d, av + ((kk * 4096) >> 4), bh + ((kk * 2048) >> 4), C::kIdescPV,
                      kk > 0 ? 1u : fresh ? 0u : 1u);
          if (!C::kSplitO) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_f8_ss(d, av + ((kk * 4096) >> 4), dp + ((kk * 2048) >> 4), C::kIdescPVLo, 1u);
          }
          mma_commit(x.bar(kEmpty + 4 * (i & 1) + c));  // a chunk goes as its block is done
        }
        mma_commit(x.bar(kPvDone));
      }
      if (!ok && lead) mbar_arrive(x.bar(kPvDone));
      __syncwarp();
      if (++v == n) break;
    } else {
      const int i = q;
      const bool begins = left == 0;
      if (begins) {
        ok = ok && x.wait_segment(seg);
        ok = __all_sync(0xffffffffu, ok);
        left = ok ? x.segment(seg)->k1 - x.segment(seg)->k0 : n - q;
        ok = ok && x.wait(kQFull, seg & 1, kSiteQ);
      }
      first = (first & ~(1u << (i & 1))) | (begins ? 1u : 0u) << (i & 1);
      if (i >= 2) named_sync(kSFree + (i & 1), C::kSync);
      const uint64_t so = static_cast<uint64_t>((i & 1) * kStageBytes) >> 4;
      const uint32_t d = C::kTmemS + 2 * R * (i & 1);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        ok = ok && x.wait(kFull + 4 * (i & 1) + c, (i >> 1) & 1, kSiteFull);
        ok = __all_sync(0xffffffffu, ok);
        tc_fence_after();
        if (ok && lead) {
#pragma unroll
          for (int ks = 0; ks < 4; ++ks)
            mma_f8_ss(d, dk + so + ((c * kChunkBytes + ks * 32) >> 4),
                      dq + ((c * C::kQChunk + ks * 32) >> 4), C::kIdescQK, c > 0 || ks > 0);
        }
      }
      if (ok && lead) {
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
          mma_f8_ss(d, dkr + so + ((ks * 32) >> 4), dqr + ((ks * 32) >> 4), C::kIdescQK, 1u);
        mma_commit(x.bar(kSFull + (i & 1)));
      }
      if (!ok && lead) mbar_arrive(x.bar(kSFull + (i & 1)));
      __syncwarp();
      ++q;
      if (--left == 0) ++seg;
    }
  }
  // every MMA has to be done before the tensor memory is released
  if (lead) mma_commit(x.bar(kDrain));
  __syncwarp();
  drain_wait(x.bar(kDrain), 0);
}

// Relay warps: one sees S of every tile done, the other PV, and they tell the
// softmax warps. After a timeout the MMA warp still tells them of every tile.
template <int R>
__device__ void relay(const Ctx<R>& x, bool pv) {
  const int n = static_cast<int>(x.ms()->n_tiles);
  bool ok = true;
#pragma unroll 1
  for (int i = 0; i < n; ++i) {
    if (pv) {
      x.wait_steadfast(kPvDone, i & 1, kSitePv);
    } else {
      if (i == 0) ok = ok && x.wait(kInfo, 0, kSiteInfo);
      if (i + 1 < n) ok = ok && x.wait(kInfo + ((i + 1) & 3), ((i + 1) >> 2) & 1, kSiteInfo);
      x.wait_steadfast(kSFull + (i & 1), (i >> 1) & 1, kSiteSFull);
    }
    named_arrive((pv ? kPvReady : kSReady) + (i & 1), Cfg<R>::kSync);
  }
}

// Two float32 in one 64-bit register: the FMA pipe takes pairs.
__device__ __forceinline__ uint64_t pack2(float x, float y) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(x), "f"(y));
  return v;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
  return f;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// The range of p'': at most 2^kTop, so that hi ends at 256 and its residual at 8.
// A row's reference is raised when a weight of a tile would pass that, and
// lowered when all its weights in a tile are below 2^kLow. It never goes more
// than kReach below its highest: what comes later cannot matter then in float32,
// and O, which is scaled up, stays far from float32's end. A weight 2^kFar above
// another warp's largest, or above the reference, makes the next tile be looked at.
constexpr float kTop = 8.f;
constexpr float kLow = -3.f;
constexpr float kReach = 40.f;
constexpr float kFar = 10.f;
constexpr float kLoScale = 32.f;

// The codes of P's second part: residuals of hi. Apart from hi (R = 32) they are
// e4m3, scaled; on hi's own accumulators (R = 64) there is no scale, and e5m2
// reaches down to 2^-16, where e4m3 would end at 2^-9.
template <bool kApart>
__device__ __forceinline__ uint32_t p_low(float x, float y) {
  return kApart ? f32_to_e4m3x2(x * kLoScale, y * kLoScale)
                : __nv_cvt_float2_to_fp8x2(make_float2(x, y), __NV_SATFINITE, __NV_E5M2);
}

// Softmax warps: warpgroup g takes the rows [16 g, 16 g + 16), a thread one key
// lane (then one dim lane of O). Four groups at R = 64 rather than two with 32
// rows each: twice the warps to hide the latencies of a tile's chain (load,
// vote, exp2, conversions), in as many registers. The rows' references and
// factors are in lanes and come by shuffles, not from shared memory.
// These warps keep to the hardware barriers, which have no limit: the relays and
// the MMA warp reach every one of them in the same order after a timeout too.
// All then go through the barriers of every tile, and nothing is stored.
template <int R>
__device__ void softmax_warps(const Ctx<R>& x) {
  using C = Cfg<R>;
  const CacheAttnArgs& a = x.p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = warp >> 2, quarter = warp & 3, key = 32 * quarter + lane;
  const uint32_t lanes = static_cast<uint32_t>(32 * quarter) << 16;
  const int slot = key / a.cache.page_size;  // the key's page within a tile
  float* s_m = reinterpret_cast<float*>(x.s() + C::kOffM);  // exchange between the warps of a group
  float* my_m = s_m + HR * warp;
  float* rowfac = reinterpret_cast<float*>(x.s() + C::kOffRow);
  uint8_t* row_dt = reinterpret_cast<uint8_t*>(rowfac + 64);
  const int n = static_cast<int>(x.ms()->n_tiles);
  int i = 0;
  int e_page = 0, t0 = 0;
  bool masked = false;
  float l[HR];
  float m = 0.f;      // lane r: the reference of row 16 g + r, an integer
  float m_top = 0.f;  // and the highest it has been
#pragma unroll 1
  for (int seg = 0;; ++seg) {
    const bool more = seg == 0 || x.segment(seg - 1)->more != 0;
    bool lost = false;  // the segment was never published: a timeout
    if (more) {
      // the segment's Q, while the last PV of the one before runs (the first
      // barrier: every warp is done with that one's factors)
      lost = named_or(kAll, 32 * C::kWarps, !x.wait_segment(seg));
      if (!lost) {
        convert_q<R>(a, x.segment(seg)->it, x.s() + C::kOffQ, rowfac, row_dt, x.ms());
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(x.bar(kQFull));
        named_sync(kAll, 32 * C::kWarps);
      }
    }
    if (seg > 0) {
      const Segment& sg = *x.segment(seg - 1);
      const Item& it = sg.it;
      named_sync(kPvReady + ((i - 1) & 1), C::kSync);
      const bool ok = *reinterpret_cast<volatile int*>(&x.ms()->abort_flag) == 0;
      tc_fence_after();
      // row sums over the key lanes
      float sum = warp_transpose_sum(l);
      if (lane < HR) my_m[lane] = sum;
      named_sync(kVote + g, 128);
      sum = 0.f;
      if (lane < HR) {
#pragma unroll
        for (int q = 0; q < 4; ++q) sum += s_m[HR * (4 * g + q) + lane];
      }
      named_sync(kVote + g, 128);
      const int r0 = g * HR;
      const bool whole_item = sg.k0 == 0 && sg.k1 == it.nt;
      // rows to store
      const int n_rows = ok ? in_call(a, it.row + r0, min(it.n_rows - r0, HR),
                                      reinterpret_cast<WsHeader*>(&x.ms()->status), 66) : 0;
      const int64_t part = 2ll * blockIdx.x + (sg.k0 == 0 ? 1 : 0);
      if (quarter == 0 && lane < HR && lane < n_rows) {
        if (whole_item) {
          if (a.lse)
            a.lse[static_cast<int64_t>(it.row) + r0 + lane] =
                sum > 0.f ? log_sum(m, sum) : -INFINITY;
        } else {
          x.p.part_ml[part * R + r0 + lane] = make_float2(sum > 0.f ? m : -INFINITY, sum);
        }
      }
      const float inv = whole_item ? (sum > 0.f ? 1.f / sum : 0.f) : 1.f;
      const int row0 = it.row + r0;
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        float o[HR];
        {
          uint32_t v[HR];
          const uint32_t col = lanes + C::kTmemO + 64 * c + g * HR;
          tmem_ld_32x32b_x16(col, v);
          if constexpr (C::kSplitO) {
            uint32_t w[HR];
            tmem_ld_32x32b_x16(col + 32, w);
            tmem_ld_wait();
#pragma unroll
            for (int r = 0; r < HR; ++r)
              o[r] = fmaf(__uint_as_float(w[r]), 1.f / kLoScale, __uint_as_float(v[r])) *
                     __shfl_sync(0xffffffffu, inv, r);
          } else {
            tmem_ld_wait();
#pragma unroll
            for (int r = 0; r < HR; ++r)
              o[r] = __uint_as_float(v[r]) * __shfl_sync(0xffffffffu, inv, r);
          }
        }
        const int dim = c * 128 + 32 * quarter + lane;
        if (whole_item) {
          // lanes pair up: the even one stores row r, the odd one row r + 1
          const bool odd = lane & 1;
          uint16_t* out = a.out + (static_cast<int64_t>(row0) + (odd ? 1 : 0)) * kDC + (dim & ~1);
#pragma unroll
          for (int r = 0; r < HR; r += 2) {
            const float other = __shfl_xor_sync(0xffffffffu, odd ? o[r] : o[r + 1], 1);
            const __nv_bfloat162 v = odd ? __floats2bfloat162_rn(other, o[r + 1])
                                         : __floats2bfloat162_rn(o[r], other);
            if (r + (odd ? 1 : 0) < n_rows) *reinterpret_cast<__nv_bfloat162*>(out + r * kDC) = v;
          }
        } else {
          float* out = x.p.part_o + (part * R + r0) * kDC + dim;
#pragma unroll
          for (int r = 0; r < HR; ++r)
            if (r < n_rows) out[r * kDC] = o[r];
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(x.bar(kOFree));
    }
    if (!more) break;
    if (lost) {
      for (; i < n; ++i) {
        named_sync(kSReady + (i & 1), C::kSync);
        if (i + 2 < n) named_arrive(kSFree + (i & 1), C::kSync);
        if constexpr (C::kPollP) {
          __syncwarp();
          if (lane == 0) mbar_arrive(x.bar(kPFull));
        } else {
          named_arrive(kPReady, C::kSync);
        }
        named_sync(kPvReady + (i & 1), C::kSync);
      }
      break;
    }
    const int n_seg = x.segment(seg)->k1 - x.segment(seg)->k0;
#pragma unroll
    for (int r = 0; r < HR; ++r) l[r] = 0.f;
    m = 0.f;
    uint32_t unset = (1u << HR) - 1u;                      // rows that saw no key yet
    // the item's rows of this group, row r as bit 6 of a code, by the byte and the
    // register that its codes are in
    uint32_t mine = 0u;
#pragma unroll
    for (int r = 0; r < HR; ++r)
      mine |= r < x.segment(seg)->it.n_rows - g * HR ? 64u << 8 * (r & 3) >> (r >> 2) : 0u;
    bool small = false;  // some row's weights of the tile before were small
    bool look = false;
    const float fac = rowfac[g * HR + (lane & (HR - 1))];  // lane r: the factor of row 16 g + r
    if (i == 0) {
      named_sync(kSReady, C::kSync);  // (tile 0)
      e_page = x.info(0)->exp[slot];
      t0 = x.info(0)->t0;
      masked = x.info(0)->masked != 0;
    }
#pragma unroll 1
    for (int k = 0; k < n_seg; ++k, ++i) {
      if (i > 0) named_sync(kSReady + (i & 1), C::kSync);
      tc_fence_after();
      const int e_key = e_page == kNoPage ? 0 : e_page;
      // y = z log2e + e_key - m: the exponents of p''
      float y[HR];
      {
        uint32_t hi[HR], lo[HR];
        const uint32_t col = lanes + C::kTmemS + 2 * R * (i & 1) + g * HR;
        tmem_ld_32x32b_x16(col, hi);
        tmem_ld_32x32b_x16(col + R, lo);
        const float sk = pow2f(e_key), ek = static_cast<float>(e_key);
        const uint64_t sk2 = pack2(sk, sk), ek2 = pack2(ek, ek), lo2 = pack2(0.0625f, 0.0625f),
                       neg2 = pack2(-1.f, -1.f);
        tmem_ld_wait();
        tc_fence_before();
        __syncwarp();
        if (i + 2 < n) named_arrive(kSFree + (i & 1), C::kSync);
#pragma unroll
        for (int j = 0; j < HR; j += 2) {
          const uint64_t t = fma2(pack2(__uint_as_float(lo[j]), __uint_as_float(lo[j + 1])), lo2,
                                  pack2(__uint_as_float(hi[j]), __uint_as_float(hi[j + 1])));
          const uint64_t f = pack2(__shfl_sync(0xffffffffu, fac, j), __shfl_sync(0xffffffffu, fac, j + 1));
          const uint64_t mm = pack2(__shfl_sync(0xffffffffu, m, j), __shfl_sync(0xffffffffu, m, j + 1));
          const float2 v = unpack2(fma2(t, mul2(f, sk2), fma2(mm, neg2, ek2)));
          y[j] = v.x;
          y[j + 1] = v.y;
        }
      }
      bool gone = false;  // no row sees this lane's key, or it has no page
      if (masked) {
        const Item& it = x.segment(seg)->it;
        const int s = t0 + key;
        gone = e_page == kNoPage || !it.seen(s);
        // row at position t sees key s iff s <= t and (t < s + window or s < n_sink)
        const unsigned span = gone ? 0u
                              : a.window == 0 || s < a.n_sink ? 0x7fffffffu
                                                              : static_cast<unsigned>(a.window);
        const int dt = it.t_lo - s;
#pragma unroll
        for (int r = 0; r < HR; ++r)
          if (static_cast<unsigned>(dt + row_dt[g * HR + r]) >= span) y[r] = -INFINITY;
      }
      float over = y[0];
#pragma unroll
      for (int r = 1; r < HR; ++r) over = fmaxf(over, y[r]);
      // the previous PV has to be waited for (a segment's last one was)
      bool pv_due = k > 0;
      // A row's reference may have to move: one of its weights is above 2^kTop,
      // they may all have been small in the tile before, or the tile before
      // showed a weight far above others, so that they may be small now.
      const bool shift = named_or(kVote + g, 128, over > kTop || small) || unset != 0u || look;
      look = false;
      if (shift) {
        // a new reference for the rows that need one
        float mx = -INFINITY;
#pragma unroll
        for (int r = 0; r < HR; ++r) {
          const float v = warp_max(y[r]);
          if (lane == r) mx = v;
        }
        if (lane < HR) my_m[lane] = mx;
        named_sync(kVote + g, 128);
        float mn = INFINITY;  // the least of the four warps' maxima
        if (lane < HR) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float v = s_m[HR * (4 * g + q) + lane];
            mx = fmaxf(mx, v);
            mn = v == -INFINITY ? mn : fminf(mn, v);
          }
        }
        named_sync(kVote + g, 128);
        const bool fresh = (unset >> lane) & 1u;
        float d = 0.f;  // what the reference rises by
        if (lane < HR && mx > -INFINITY) {
          if (fresh) d = ceilf(mx) - 6.f;
          else if (mx > kTop) d = ceilf(mx) - 6.f;
          else if (mx < kLow) d = fminf(fmaxf(ceilf(mx) - 4.f, m_top - kReach - m), 0.f);
        }
        look = __any_sync(0xffffffffu, mx - mn > kFar || (!fresh && d > kFar));
        const float f = fresh ? 1.f : ex2_approx(-d);
        const bool seen = fresh && lane < HR && mx > -INFINITY;
        unset &= ~__ballot_sync(0xffffffffu, seen);
        m += d;
        m_top = seen ? m : fmaxf(m_top, m);
#pragma unroll
        for (int r = 0; r < HR; ++r) y[r] -= __shfl_sync(0xffffffffu, d, r);
        if (__any_sync(0xffffffffu, f != 1.f)) {
          if (pv_due) named_sync(kPvReady + ((i - 1) & 1), C::kSync);
          tc_fence_after();
          float fr[HR];
#pragma unroll
          for (int r = 0; r < HR; ++r) {
            fr[r] = __shfl_sync(0xffffffffu, f, r);
            l[r] *= fr[r];
          }
          if (k > 0) {
#pragma unroll 1
            for (int c = 0; c < (C::kSplitO ? 8 : 4); ++c) {
              const uint32_t col = lanes + C::kTmemO + (C::kSplitO ? 32 : 64) * c + g * HR;
              uint32_t o[HR];
              tmem_ld_32x32b_x16(col, o);
              tmem_ld_wait();
#pragma unroll
              for (int r = 0; r < HR; ++r) o[r] = __float_as_uint(__uint_as_float(o[r]) * fr[r]);
              tmem_st_32x32b_x16(col, o);
            }
            tmem_st_wait();
          }
          pv_due = false;
        }
      }
      uint32_t hi[HR / 4], lo[HR / 4];
      {
        const float inv_sk = pow2f(-e_key);
#pragma unroll
        for (int r = 0; r < HR; r += 4) {
          float p[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            p[e] = ex2_approx(y[r + e]);
            l[r + e] = fmaf(p[e], inv_sk, l[r + e]);
          }
          const uint32_t h0 = f32_to_e4m3x2(p[0], p[1]), h1 = f32_to_e4m3x2(p[2], p[3]);
          const float2 b0 = e4m3x2_to_f32(h0), b1 = e4m3x2_to_f32(h1);
          hi[r / 4] = h0 | h1 << 16;
          lo[r / 4] = p_low<C::kSplitO>(p[0] - b0.x, p[1] - b0.y) |
                      p_low<C::kSplitO>(p[2] - b1.x, p[3] - b1.y) << 16;
        }
      }
      if (pv_due) named_sync(kPvReady + ((i - 1) & 1), C::kSync);  // P's place is free
      unsigned char* stage = x.s() + C::kOffStage + (i & 1) * kStageBytes;
      {
        // 16 rows are one 16-byte unit of the key's 64-byte row, 64-byte swizzle
        unsigned char* row_hi = (C::kSplitO ? x.s() + C::kOffP : stage + kRopeOff) + key * 64;
        unsigned char* row_lo = x.s() + C::kOffP + key * 64;
        const int sw = (key >> 1) & 3, ul = C::kSplitO ? 2 + g : g;
        *reinterpret_cast<uint4*>(row_hi + ((g ^ sw) << 4)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4*>(row_lo + ((ul ^ sw) << 4)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      }
      if (__any_sync(0xffffffffu, gone)) {
        // A key that no row sees: its bytes may be anything, and 0 * NaN is
        // NaN, so its latent row is zeroed before the PV. The tile's chunks
        // have landed (QK^T read them); waiting on them orders the writes.
#pragma unroll 1
        for (int c = g; c < 4; c += C::kGroups) {
          const bool there = x.wait(kFull + 4 * (i & 1) + c, (i >> 1) & 1, kSiteFull);
          if (gone && there) {
            // (lanes start at different units, for different banks)
#pragma unroll
            for (int u = 0; u < 8; ++u)
              *reinterpret_cast<uint4*>(stage + c * kChunkBytes + key * 128 +
                                        (((u + lane) & 7) << 4)) = make_uint4(0u, 0u, 0u, 0u);
          }
        }
      }
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if constexpr (C::kPollP) {
        if (lane == 0) mbar_arrive(x.bar(kPFull));
      } else {
        named_arrive(kPReady, C::kSync);
      }
      if (i + 1 < n) {
        const TileInfo* next = x.info(i + 1);
        e_page = next->exp[slot];
        t0 = next->t0;
        masked = next->masked != 0;
      }
      if (quarter == 0 && k + 1 < n_seg) {
        // For the next tile's vote: does some row have no weight of 2^kLow here
        // (bits 5 and 6 of its codes)? Of the group's warps the first
        // speaks for all; a row that is small there only costs the vote.
        uint32_t some = 0u;
#pragma unroll
        for (int q = 0; q < HR / 4; ++q)
          some |= ((hi[q] | hi[q] << 1) & 0x40404040u) >> q;
        small = (~__reduce_or_sync(0xffffffffu, some) & mine) != 0u;
      }
    }
  }
}

template <int R>
__global__ void __launch_bounds__(Cfg<R>::kThreads, 1)
    cache_attn_tc(const __grid_constant__ CacheAttnParams p, const __grid_constant__ CUtensorMap ml,
                  const __grid_constant__ CUtensorMap mr) {
  using C = Cfg<R>;
  const Ctx<R> x{p};
  Misc* ms = x.ms();
  const int tid = threadIdx.x, warp = tid >> 5;
  if (tid == 0) {
    ms->status = ms->info = 0u;
    ms->abort_flag = 0;
    prefetch_tmap(&ml);
    prefetch_tmap(&mr);
  }
  if (tid >= 32 && tid < 32 + C::kNumBars) {
    const int b = tid - 32;
    mbar_init(x.bar(b), b == kQFull || b == kOFree || b == kPFull ? C::kWarps : 1);
    fence_barrier_init();
  }
  if (warp == C::kWarps + 1) tmem_alloc(&ms->tmem, 512);
  __syncthreads();  // the status word before schedule() may report
  schedule<R>(p.a, ms, reinterpret_cast<long long*>(x.s() + C::kOffM), x.segment(0));  // ends with a barrier
  tc_fence_after();
  // All 512 columns are this CTA's, so they begin at 0; operands are at
  // constant addresses on that account.
  bool work = ms->n_tiles > 0;
  if (ms->tmem != 0u || (smem_u32(x.s()) & 1023u) != 0u) {
    if (tid == 0) report(reinterpret_cast<WsHeader*>(&ms->status), kDevInternal, 0);
    work = false;
  }
  Begun begun = {-1, 0};
  if (work) {
    if (warp < C::kWarps) softmax_warps<R>(x);
    else if (warp == C::kWarps) begun = producer<R>(x, &ml, &mr);
    else if (warp == C::kWarps + 1) mma_issuer<R>(x);
    else relay<R>(x, warp == C::kWarps + 3);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == C::kWarps + 1) {
    tc_fence_after();
    tmem_dealloc(ms->tmem, 512);
  }
  if (begun.tile >= 0 && ms->abort_flag != 0 && (tid & 31) == 0) drain_copies<R>(x, begun);
  if (tid == 0) {
    CtaMeta& me = p.meta[blockIdx.x];
    me.status = ms->status;
    me.info = ms->info;
    if (!work) me.n_rows = 0;
  }
}

// ------------------------------------------------------------------- combine

constexpr int kCombineThreads = 128;
constexpr int kCombineBlocks = 8;  // per SM

// Parts of an item up to which a warp joins a whole row by itself.
constexpr int kFewParts = 4;

// The weights 2^(m_j - M) of one query row's parts (part 32 i + lane in w[i])
// and the sum of the weighted l. All loads at once: one latency.
template <int kRounds>
struct RowParts {
  float w[kRounds], mx, sum;
  template <class Part>
  __device__ __forceinline__ void load(const float2* part_ml, int n, Part part) {
    const int lane = threadIdx.x & 31;
    float2 ml[kRounds];
#pragma unroll
    for (int i = 0; i < kRounds; ++i)
      ml[i] = 32 * i + lane < n ? __ldcg(part_ml + part(32 * i + lane)) : make_float2(-INFINITY, 0.f);
    mx = ml[0].x;
#pragma unroll
    for (int i = 1; i < kRounds; ++i) mx = fmaxf(mx, ml[i].x);
    mx = warp_max(mx);
    sum = 0.f;
#pragma unroll
    for (int i = 0; i < kRounds; ++i) {
      w[i] = ml[i].x == -INFINITY ? 0.f : exp2f(ml[i].x - mx);
      sum += w[i] * ml[i].y;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  }
  __device__ __forceinline__ float inv() const { return sum > 0.f ? 1.f / sum : 0.f; }
  __device__ __forceinline__ float lse() const {
    return sum > 0.f ? log_sum(mx, sum) : -INFINITY;
  }
};

__device__ __forceinline__ void add_part(float4& acc, float f, const float4& v) {
  // (O of a part without keys is 0: its p were)
  acc.x = fmaf(f, v.x, acc.x);
  acc.y = fmaf(f, v.y, acc.y);
  acc.z = fmaf(f, v.z, acc.z);
  acc.w = fmaf(f, v.w, acc.w);
}

__device__ __forceinline__ void store_bf16x4(uint16_t* dst, const float4& v, float f) {
  const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x * f, v.y * f);
  const __nv_bfloat162 hi = __floats2bfloat162_rn(v.z * f, v.w * f);
  *reinterpret_cast<uint2*>(dst) = make_uint2(*reinterpret_cast<const uint32_t*>(&lo),
                                              *reinterpret_cast<const uint32_t*>(&hi));
}

// Rows of an item (last CTA, first CTA, row, rows) whose parts are to be joined;
// none where the checking build finds a part or a row out of bounds.
__device__ __forceinline__ int in_parts(const CacheAttnParams& p, const int4& me, unsigned int site) {
  return DSA_IN_BOUNDS(p.a.ws, me.y, me.x + 1, site) && DSA_IN_BOUNDS(p.a.ws, me.x, kMaxCtas, site)
             ? in_call(p.a, me.z, me.w, p.a.ws, site)
             : 0;
}

// Joins the partial results of the items that cross CTAs: out = sum_c
// 2^(m_c - M) O_c / sum_c 2^(m_c - M) l_c. An item in few parts (a batch: most
// are in two) takes a warp for each row; one in many (a long sequence is in up
// to 148) a block for 128 dims of a row, its warps every fourth part each.
// Also collects the CTAs' status.
template <int R>
__global__ void __launch_bounds__(kCombineThreads)
    cache_attn_combine(const __grid_constant__ CacheAttnParams p, int n_ctas) {
  constexpr int kRounds = (kMaxCtas + 31) / 32;
  __shared__ float s_w[4][kMaxCtas];  // a warp's own copy
  __shared__ int4 s_few[kMaxCtas], s_many[kMaxCtas];  // last CTA, first CTA, row, rows
  __shared__ uint32_t s_has[2][kRounds];
  __shared__ float4 s_acc[3][32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // the CTAs that end such an item, in order (the same lists in every block)
  unsigned int status = 0, info = 0;
  int4 mine[(kRounds + 3) / 4];
  int kind[(kRounds + 3) / 4];
#pragma unroll
  for (int k = 0; k < (kRounds + 3) / 4; ++k) {
    const int i = warp + 4 * k, c = 32 * i + lane;
    kind[k] = -1;
    if (i < kRounds && c < n_ctas) {
      const CtaMeta me = p.meta[c];
      mine[k] = make_int4(c, me.first, me.row, me.n_rows);
      if (me.n_rows > 0) kind[k] = c - me.first + 1 > kFewParts ? 1 : 0;
      if (me.status != 0u) {
        status = me.status;
        info = me.info;
      }
    }
    const uint32_t few = __ballot_sync(0xffffffffu, kind[k] == 0);
    const uint32_t many = __ballot_sync(0xffffffffu, kind[k] == 1);
    if (lane == 0 && i < kRounds) {
      s_has[0][i] = few;
      s_has[1][i] = many;
    }
  }
#if !(defined(DSA_CHECK) && DSA_CHECK)  // (there other blocks may report; the host clears it)
  if (blockIdx.x == 0 && tid == 0) {
    p.a.ws->status = 0u;
    p.a.ws->status_info = 0u;
  }
#endif
  __syncthreads();
  int n_few = 0, n_many = 0;
#pragma unroll
  for (int i = 0; i < kRounds; ++i) {
    const uint32_t few = s_has[0][i], many = s_has[1][i], below = (1u << lane) - 1u;
    if (warp == i % 4) {
      if (kind[i / 4] == 0) s_few[n_few + __popc(few & below)] = mine[i / 4];
      if (kind[i / 4] == 1) s_many[n_many + __popc(many & below)] = mine[i / 4];
    }
    n_few += __popc(few);
    n_many += __popc(many);
  }
  __syncthreads();
  if (blockIdx.x == 0 && status != 0u) report(p.a.ws, status, info);
  for (int u = blockIdx.x * 4 + warp; u < n_few * R; u += gridDim.x * 4) {
    const int4 me = s_few[u / R];
    const int r = u % R, c0 = me.y, n = me.x - c0 + 1;
    if (r >= in_parts(p, me, 67)) continue;
    // (the item's first part is its CTA's second slot)
    auto part = [&](int j) { return (2ll * (c0 + j) + (j == 0 ? 1 : 0)) * R + r; };
    float4 v[kFewParts][4];
#pragma unroll
    for (int j = 0; j < kFewParts; ++j)
      if (j < n) {
        const float4* src = reinterpret_cast<const float4*>(p.part_o + part(j) * kDC);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[j][e] = __ldcg(src + 32 * e + lane);
      }
    RowParts<1> rp;
    rp.load(p.part_ml, n, part);
    const int64_t row = static_cast<int64_t>(me.z) + r;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int j = 0; j < kFewParts; ++j) {
        const float f = __shfl_sync(0xffffffffu, rp.w[0], j);
        if (j < n) add_part(acc, f, v[j][e]);
      }
      store_bf16x4(p.a.out + row * kDC + 128 * e + 4 * lane, acc, rp.inv());
    }
    if (lane == 0 && p.a.lse) p.a.lse[row] = rp.lse();
  }
  for (int u = blockIdx.x; u < n_many * R * 4; u += gridDim.x) {
    const int4 me = s_many[u / (4 * R)];
    const int r = (u >> 2) % R, quarter = u & 3, c0 = me.y, n = me.x - c0 + 1;
    if (r >= in_parts(p, me, 67)) continue;
    auto part = [&](int j) { return (2ll * (c0 + j) + (j == 0 ? 1 : 0)) * R + r; };
    // eight parts ahead, the first eight before the weights are known
    auto fetch = [&](float4(&v)[8], int j0) {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        v[k] = j0 + 4 * k < n ? __ldcg(reinterpret_cast<const float4*>(
                                           p.part_o + part(j0 + 4 * k) * kDC + quarter * 128) + lane)
                              : make_float4(0.f, 0.f, 0.f, 0.f);
    };
    float4 v[8];
    fetch(v, warp);
    RowParts<kRounds> rp;
    rp.load(p.part_ml, n, part);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kRounds; ++i)
      if (32 * i + lane < n) s_w[warp][32 * i + lane] = rp.w[i];
    __syncwarp();
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int j0 = warp; j0 < n; j0 += 32) {
      float4 next[8];
      fetch(next, j0 + 32);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (j0 + 4 * k < n) add_part(acc, s_w[warp][j0 + 4 * k], v[k]);
        v[k] = next[k];
      }
    }
    if (warp > 0) s_acc[warp - 1][lane] = acc;
    __syncthreads();
    if (warp == 0) {
#pragma unroll
      for (int j = 0; j < 3; ++j) add_part(acc, 1.f, s_acc[j][lane]);
      const int64_t row = static_cast<int64_t>(me.z) + r;
      store_bf16x4(p.a.out + row * kDC + quarter * 128 + 4 * lane, acc, rp.inv());
      if (lane == 0 && quarter == 0 && p.a.lse) p.a.lse[row] = rp.lse();
    }
    __syncthreads();  // before s_acc is written again
  }
}

// ----------------------------------------------------- the (64, 16) shape

constexpr int kRowWarps = 4;

// One warp per query row (token, head). 32 keys at a time: a lane forms the
// dot product of its key (q from shared memory), the warp updates the running
// maximum and sum, then the lanes take the latent's dims and add the 32
// weighted rows. This is the small shape of the tests, kept simple: a row's keys
// are one chain on one warp (4 heads: 256 queries at 1,024 keys 0.23 ms, 2,048 at
// 8,192 4.4 ms, one token of 64 sequences of 1 to 17,408 rows 3.5 ms).
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
  if (!DSA_IN_BOUNDS(a.ws, row, static_cast<int64_t>(a.batch.n_tok) * a.n_heads, 68)) return;
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
cudaError_t launch_tc(const CacheAttnArgs& a, void* scratch, long long wait_cycles,
                      cudaStream_t st) {
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
#if defined(DSA_CHECK) && DSA_CHECK
  e = cudaMemsetAsync(a.ws, 0, kWsHeaderBytes, st);
  if (e != cudaSuccess) return e;
#endif
  CacheAttnParams p;
  p.a = a;
  char* w = static_cast<char*>(scratch);
  p.meta = reinterpret_cast<CtaMeta*>(w);
  w += kMaxCtas * sizeof(CtaMeta);
  p.part_ml = reinterpret_cast<float2*>(w);
  w += kMaxCtas * 2 * R * sizeof(float2);
  p.part_o = reinterpret_cast<float*>(w);
  p.wait_cycles = wait_cycles < 0 ? kWaitLimitCycles : wait_cycles;
  cache_attn_tc<R><<<grid, Cfg<R>::kThreads, Cfg<R>::kSmemBytes, st>>>(p, ml, mr);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cache_attn_combine<R><<<grid * kCombineBlocks, kCombineThreads, 0, st>>>(p, grid);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_attn(const CacheAttnArgs& a, void* scratch, cudaStream_t st,
                              long long wait_cycles) {
  if (a.cache.d_latent != kDC) return launch_rows(a, st);
  // R = 32 when the sequences have no more than 32 rows on average, as far as the
  // host knows (cu_seqlens is on the device). R = 32 / R = 64, in us, 64
  // sequences of 1 to 17,408 rows unless said: 1 token of 32 heads 122 / 145, 2
  // tokens 202 / 155, 64 heads 202 / 156, 128 heads 375 / 256, one of them with
  // 512 tokens 342 / 279; 3 tokens at 131,071 75 / 68; 2,048 tokens at 8,192 1,617
  // / 908. The average misleads beside many sequences without tokens (100 tokens
  // at 4,000 and 200 such: 75 / 64), and one sequence with 64 heads is short of
  // tiles either way (28 / 32).
  const int64_t rows = static_cast<int64_t>(a.batch.n_tok) * a.n_heads;
  return rows <= 32ll * a.batch.n_seq ? launch_tc<32>(a, scratch, wait_cycles, st)
                                      : launch_tc<64>(a, scratch, wait_cycles, st);
}

}  // namespace dsa
