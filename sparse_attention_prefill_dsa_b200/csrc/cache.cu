// cache.cu -- the paged 8-bit latent cache: appending rows with the position
// rotation, and reading rows back as bf16.
//
// Append. A page is the unit of work, because its rows share one scale: a CTA
// takes one page that gets new rows, keeps the new rows in registers (one
// read), reduces the exponent of the scale over them, and writes codes. The
// scale is a power of two, so "the smallest s with |x| <= 448 s" is an integer
// of the exponent and top mantissa bits (448 = 1.75 * 2^8): the reduction is a
// maximum of integers, exact and independent of its order. The rotation of
// the 64-wide rope is done in float64 (angles reach 10^5 radians, and a value
// next to a rounding border of e4m3 must fall on the same side everywhere);
// its 32 pairs a token are 1/18 of a row's elements.
// The queries' rope is rotated by CTAs of its own, a few tokens each: the
// angle in float64, once for each token and pair, cos and sin rounded to float32
// for the heads, whose outputs are bf16 (8 bits).
// Bound: the bytes of a prefill chunk, most of them the queries' rope (8,192
// tokens with 32 heads 22.6 us, 3.6 TB/s; the angles' chain between a CTA's
// loads and stores keeps it from the copy rate), the chain of dependent loads
// (batch arrays, page table, rows) of a decode step (7.2 us of kernel, alone).
//
// One more CTA checks the batch arrays and the page table entries that the
// call uses, and is the only one that writes the status word: the others skip
// what is wrong by the same tests. The word then needs no clearing launch.
#include <cuda_bf16.h>

#include "cache.cuh"

namespace dsa {
namespace {


// ------------------------------------------------------------------ status

// Writes the status word from the threads' findings (0, or a site).
__device__ void write_status(WsHeader* ws, unsigned int site) {
  const unsigned int bad = __reduce_max_sync(0xffffffffu, site);
  __shared__ unsigned int s_bad;
  if (threadIdx.x == 0) s_bad = 0;
  __syncthreads();
  if ((threadIdx.x & 31) == 0 && bad) atomicMax(&s_bad, bad);
  __syncthreads();
  if (threadIdx.x == 0) {
#if defined(DSA_CHECK) && DSA_CHECK
    if (s_bad) report(ws, kDevRange, s_bad);  // the word was cleared: others may have written it
#else
    ws->status_info = s_bad;
    ws->status = s_bad ? kDevRange : 0u;
#endif
  }
}

// Of the checking build, in which every block may report.
cudaError_t clear_status_for_checks(WsHeader* ws, cudaStream_t st) {
#if defined(DSA_CHECK) && DSA_CHECK
  return cudaMemsetAsync(ws, 0, kWsHeaderBytes, st);
#else
  (void)ws, (void)st;
  return cudaSuccess;
#endif
}

__device__ __forceinline__ int page_of(const dsa_batch& bt, int seq, int64_t j) {
  return __ldg(bt.page_table + static_cast<int64_t>(seq) * bt.max_pages + j);
}

__device__ __forceinline__ bool page_ok(const dsa_cache& c, int page) {
  return page >= 0 && page < c.n_pages;
}

// Slots of the page CTAs: a sequence of n tokens touches at most
// floor((n - 1) / page_size) + 2 pages.
__device__ void append_check(const AppendArgs& a) {
  unsigned int site = 0;
  const int ps = a.cache.page_size, shift = 31 - __clz(ps);
  for (int b = threadIdx.x; b < a.batch.n_seq; b += blockDim.x)
    if (!seq_range(a.batch, ps, b).ok) site = max(site, kCacheSiteSeq);
  const int64_t slots = a.batch.n_tok / ps + 2ll * a.batch.n_seq;
  for (int64_t s = threadIdx.x; s < slots; s += blockDim.x) {
    const int b = seq_of_slot(a.batch, s, 1, shift, 2);
    const SeqRange r = seq_range(a.batch, ps, b);
    const int64_t j = s - slot_start(a.batch, b, 1, shift, 2);
    if (r.n == 0 || j < 0) continue;
    const int64_t pg = (r.len - r.n) / ps + j;
    if (pg * ps < r.len && !page_ok(a.cache, page_of(a.batch, b, pg)))
      site = max(site, kCacheSitePage);
  }
  write_status(a.ws, site);
}

// ------------------------------------------------------------------ append

// The exponent e of the smallest 2^e with |x| <= 448 * 2^e (a large negative
// number for zero): |x| = 1.f * 2^E needs E - 8 when 1.f <= 1.75, else E - 7.
__device__ __forceinline__ int need_exp_f32(float x) {
  const uint32_t b = __float_as_uint(x) & 0x7FFFFFFFu;
  if (b == 0u) return -1000;
  return static_cast<int>(b >> 23) - 127 - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
}

__device__ __forceinline__ int need_exp_f64(double x) {
  const uint64_t b = static_cast<uint64_t>(__double_as_longlong(x)) & 0x7FFFFFFFFFFFFFFFull;
  if (b == 0ull) return -1000;
  return static_cast<int>(b >> 52) - 1023 - 8 +
         ((b & 0xFFFFFFFFFFFFFull) > 0xC000000000000ull ? 1 : 0);
}

// float64 -> float32 by round-to-odd, so that a following rounding to e4m3
// is that of the float64 value.
__device__ __forceinline__ float f64_to_f32_odd(double x) {
  const float f = __double2float_rz(x);
  return static_cast<double>(f) == x ? f : __uint_as_float(__float_as_uint(f) | 1u);
}

__device__ __forceinline__ float2 bf16x2(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

// Re-expresses `n16` 16-byte groups of codes by the factor 2^-k.
__device__ void rescale_codes(uint8_t* p, int n16, float f) {
  for (int i = threadIdx.x; i < n16; i += blockDim.x) {
    uint4 v = reinterpret_cast<uint4*>(p)[i];
    uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 lo = e4m3x2_to_f32(w[e]), hi = e4m3x2_to_f32(w[e] >> 16);
      w[e] = f32_to_e4m3x2(lo.x * f, lo.y * f) | f32_to_e4m3x2(hi.x * f, hi.y * f) << 16;
    }
    reinterpret_cast<uint4*>(p)[i] = v;
  }
}

// A page's rows are read twice, for the scale and for the codes (the second
// time from L2): the registers they would take are better given to more
// threads, which the queries' CTAs of the same launch, most of the bytes, need.
// The rotated rope stays in registers, four pairs of float64 a thread (with
// eight, on half the threads, a page took so long that a chunk of 8,192 tokens
// took 31 us instead of 24).
template <int DC, int DR, int PS>
struct AppendCfg {
  static constexpr int kThr = PS <= 32 ? 256 : 8 * PS;
  static constexpr int kMinBlocks = 1024 / kThr;
  static constexpr int kMaxQTokens = 16;      // tokens of a q CTA, at most
  static constexpr int kRowUnits = DC / 8;    // 16-byte units of a latent row
  static constexpr int kUnits = (PS * kRowUnits + kThr - 1) / kThr;
  static constexpr int kRowPairs = DR / 2;
  static constexpr int kPairs = (PS * kRowPairs + kThr - 1) / kThr;
};

// seq_of_slot by the whole block: every step loads one start a thread and
// counts those up to the slot, so that up to as many sequences as threads take
// one load instead of a chain of log2 of them.
__device__ int block_seq_of_slot(const dsa_batch& bt, int64_t slot, int shift, int extra) {
  int lo = 0, n = bt.n_seq;  // the answer is one of lo .. lo + n - 1
  while (n > 1) {
    const int step = (n + blockDim.x - 1) / blockDim.x;
    const int64_t k = static_cast<int64_t>(threadIdx.x) * step;
    const int count =
        __syncthreads_count(k < n && slot_start(bt, lo + static_cast<int>(k), 1, shift, extra) <= slot);
    const int at = max(count - 1, 0) * step;
    lo += at;
    n = min(step, n - at);
  }
  return lo;
}

template <int DC, int DR, int PS>
__device__ void append_page(const AppendArgs& a, int64_t slot) {
  using C = AppendCfg<DC, DR, PS>;
  __shared__ int s_exp;
  constexpr int kShift = PS == 16 ? 4 : PS == 32 ? 5 : PS == 64 ? 6 : 7;
  const int b = block_seq_of_slot(a.batch, slot, kShift, 2);
  const SeqRange r = seq_range(a.batch, PS, b);
  const int64_t j = slot - slot_start(a.batch, b, 1, kShift, 2);
  if (r.n == 0 || j < 0) return;
  const int p0 = r.len - r.n;            // the sequence's first new position
  const int64_t pg = p0 / PS + j;        // this CTA's page of the sequence
  if (pg * PS >= r.len) return;
  const int page = page_of(a.batch, b, pg);  // (looked at after the rows: the loads overlap)
  const int base = static_cast<int>(pg) * PS;
  const int r0 = max(p0 - base, 0), r1 = min(r.len - base, PS);  // new rows of the page
  const int64_t tok = static_cast<int64_t>(r.tok0) + base - p0;  // token of row 0 (row r0 on is real)
  if (threadIdx.x == 0) s_exp = kCacheMinExp;

  int need = kCacheMinExp;
  auto unit = [&](int u) {
    const int x = threadIdx.x + u * C::kThr, row = x / C::kRowUnits;
    return row >= r0 && row < r1 && DSA_IN_BOUNDS(a.ws, tok + row, a.batch.n_tok, 60)
               ? __ldg(reinterpret_cast<const uint4*>(a.latent + (tok + row) * a.ld_latent) +
                       x % C::kRowUnits)
               : make_uint4(0u, 0u, 0u, 0u);
  };
  {
    uint32_t top = 0u;  // the largest |x|: bf16 magnitudes order as integers
#pragma unroll 8
    for (int u = 0; u < C::kUnits; ++u) {
      const uint4 v = unit(u);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int e = 0; e < 4; ++e)
        top = max(top, max((w[e] & 0x7FFFu) << 16, w[e] & 0x7FFF0000u));
    }
    need = max(need, need_exp_f32(__uint_as_float(top)));
  }
  if (!page_ok(a.cache, page)) return;
  // (a plain load: thread 0 writes it below)
  const float old_scale = r0 > 0 ? a.cache.scale[page] : 0.f;
  double2 rot[C::kPairs];
#pragma unroll
  for (int u = 0; u < C::kPairs; ++u) {
    const int x = threadIdx.x + u * C::kThr, row = x / C::kRowPairs, i = x % C::kRowPairs;
    rot[u] = make_double2(0.0, 0.0);
    if (row >= r0 && row < r1 && DSA_IN_BOUNDS(a.ws, tok + row, a.batch.n_tok, 60)) {
      const uint16_t* src = a.rope + (tok + row) * a.ld_rope;
      const double v = bf16_to_f64(src[a.halves ? i : 2 * i]);
      const double w = bf16_to_f64(src[a.halves ? i + DR / 2 : 2 * i + 1]);
      double sn, cs;
      sincos(static_cast<double>(base + row) * static_cast<double>(__ldg(a.inv_freq + i)), &sn,
             &cs);
      rot[u] = make_double2(v * cs - w * sn, w * cs + v * sn);
      need = max(need, max(need_exp_f64(rot[u].x), need_exp_f64(rot[u].y)));
    }
  }
  need = __reduce_max_sync(0xffffffffu, need);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) atomicMax(&s_exp, need);
  __syncthreads();
  int e_new = min(s_exp, kCacheMaxExp);
  uint8_t* lat_page = a.cache.latent + static_cast<int64_t>(page) * a.cache.latent_page_stride;
  uint8_t* rope_page = a.cache.rope + static_cast<int64_t>(page) * a.cache.rope_page_stride;
  if (r0 > 0) {
    const int e_old = scale_exp(old_scale);
    e_new = max(e_new, e_old);
    if (e_new > e_old) {
      // at most 2^-126: a code is below 2^9, so every such factor gives 0
      const float f = pow2f(max(e_old - e_new, -126));
      rescale_codes(lat_page, r0 * DC / 16, f);
      rescale_codes(rope_page, r0 * DR / 16, f);
    }
  }
  const float inv = pow2f(-e_new);
  if (threadIdx.x == 0) a.cache.scale[page] = pow2f(e_new);
#pragma unroll 8
  for (int u = 0; u < C::kUnits; ++u) {
    const int x = threadIdx.x + u * C::kThr, row = x / C::kRowUnits;
    if (row < r0 || row >= r1) continue;
    const uint4 w = unit(u);
    const float2 f0 = bf16x2(w.x), f1 = bf16x2(w.y), f2 = bf16x2(w.z), f3 = bf16x2(w.w);
    uint2 v;
    v.x = f32_to_e4m3x2(f0.x * inv, f0.y * inv) | f32_to_e4m3x2(f1.x * inv, f1.y * inv) << 16;
    v.y = f32_to_e4m3x2(f2.x * inv, f2.y * inv) | f32_to_e4m3x2(f3.x * inv, f3.y * inv) << 16;
    if (DSA_IN_BOUNDS(a.ws, x * 8 + 7, PS * DC, 61)) *reinterpret_cast<uint2*>(lat_page + x * 8) = v;
  }
  const double inv_d = static_cast<double>(inv);
#pragma unroll
  for (int u = 0; u < C::kPairs; ++u) {
    const int x = threadIdx.x + u * C::kThr, row = x / C::kRowPairs, i = x % C::kRowPairs;
    if (row < r0 || row >= r1) continue;
    const uint32_t v =
        f32_to_e4m3x2(f64_to_f32_odd(rot[u].x * inv_d), f64_to_f32_odd(rot[u].y * inv_d));
    uint8_t* dst = rope_page + row * DR;
    if (!DSA_IN_BOUNDS(a.ws, row * DR + DR - 1, PS * DR, 62)) continue;
    if (a.halves) {
      dst[i] = static_cast<uint8_t>(v);
      dst[i + DR / 2] = static_cast<uint8_t>(v >> 8);
    } else {
      *reinterpret_cast<uint16_t*>(dst + 2 * i) = static_cast<uint16_t>(v);
    }
  }
}

__device__ __forceinline__ uint32_t pack_bf16x2(float x, float y) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Eight pairs of one head: two 16-byte groups, adjacent (interleaved) or
// d_rope/2 apart.
template <int DC, int DR>
struct QItem {
  uint4 v, w;
  const uint4* src;
  uint4* dst;
  const float2* cs;
  int other;  // groups between the two
  __device__ __forceinline__ bool load(const AppendArgs& a, int64_t tok0, int x, int items,
                                       const float2* s_cs) {
    if (x >= items) return false;
    constexpr int kPerHead = DR / 16;
    const int g = x % kPerHead, h = (x / kPerHead) % a.n_heads, k = x / kPerHead / a.n_heads;
    const int64_t tok = tok0 + k;
    if (tok >= a.batch.n_tok || !DSA_IN_BOUNDS(a.ws, tok * a.n_heads + h,
                                               static_cast<int64_t>(a.batch.n_tok) * a.n_heads, 63))
      return false;
    other = a.halves ? DR / 16 : 1;
    const int at = a.halves ? g : 2 * g;
    src = reinterpret_cast<const uint4*>(a.q_rope + tok * a.ld_q_tok + h * a.ld_q_head) + at;
    dst = reinterpret_cast<uint4*>(a.q + (tok * a.n_heads + h) * (DC + DR) + DC) + at;
    cs = s_cs + k * (DR / 2) + g * 8;
    v = __ldg(src);
    w = __ldg(src + other);
    return true;
  }
  __device__ __forceinline__ void store(bool halves) const {
    const uint32_t vi[4] = {v.x, v.y, v.z, v.w}, wi[4] = {w.x, w.y, w.z, w.w};
    uint32_t vo[4], wo[4];
    if (halves) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 p = bf16x2(vi[e]), q = bf16x2(wi[e]), c0 = cs[2 * e], c1 = cs[2 * e + 1];
        vo[e] = pack_bf16x2(p.x * c0.x - q.x * c0.y, p.y * c1.x - q.y * c1.y);
        wo[e] = pack_bf16x2(q.x * c0.x + p.x * c0.y, q.y * c1.x + p.y * c1.y);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 p = bf16x2(vi[e]), q = bf16x2(wi[e]), c0 = cs[e], c1 = cs[4 + e];
        vo[e] = pack_bf16x2(p.x * c0.x - p.y * c0.y, p.y * c0.x + p.x * c0.y);
        wo[e] = pack_bf16x2(q.x * c1.x - q.y * c1.y, q.y * c1.x + q.x * c1.y);
      }
    }
    dst[0] = make_uint4(vo[0], vo[1], vo[2], vo[3]);
    dst[other] = make_uint4(wo[0], wo[1], wo[2], wo[3]);
  }
};

// Rotates the queries' rope of n_tok tokens. A thread's first items are loaded
// before the angles are worked out.
template <int DC, int DR, int kMaxTokens>
__device__ void rotate_q(const AppendArgs& a, int64_t tok0, int n_tok) {
  __shared__ float2 s_cs[kMaxTokens * (DR / 2)];
  __shared__ int s_pos[kMaxTokens];
  constexpr int kPerHead = DR / 16, kAhead = 2;
  const int items = n_tok * a.n_heads * kPerHead;
  QItem<DC, DR> it[kAhead];
  bool has[kAhead];
#pragma unroll
  for (int i = 0; i < kAhead; ++i)
    has[i] = it[i].load(a, tok0, threadIdx.x + i * blockDim.x, items, s_cs);
  if (threadIdx.x < n_tok) {
    const int64_t tok = tok0 + threadIdx.x;
    int pos = -1;
    if (tok < a.batch.n_tok) {
      const int b = seq_of_token(a.batch, static_cast<int>(tok));
      if (b >= 0) {
        const SeqRange r = seq_range(a.batch, a.cache.page_size, b);
        if (r.n > 0) pos = r.len - r.n + static_cast<int>(tok) - r.tok0;
      }
    }
    s_pos[threadIdx.x] = pos;
  }
  __syncthreads();
  for (int x = threadIdx.x; x < n_tok * (DR / 2); x += blockDim.x) {
    double sn, cs;
    sincos(static_cast<double>(s_pos[x / (DR / 2)]) *
               static_cast<double>(__ldg(a.inv_freq + x % (DR / 2))), &sn, &cs);
    s_cs[x] = make_float2(static_cast<float>(cs), static_cast<float>(sn));
  }
  __syncthreads();
  for (int x = threadIdx.x; x < items; x += kAhead * blockDim.x) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (has[i] && s_pos[(x + i * blockDim.x) / (kPerHead * a.n_heads)] >= 0) it[i].store(a.halves);
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      has[i] = it[i].load(a, tok0, x + (kAhead + i) * blockDim.x, items, s_cs);
  }
}

template <int DC, int DR, int PS>
__global__ void __launch_bounds__(AppendCfg<DC, DR, PS>::kThr, AppendCfg<DC, DR, PS>::kMinBlocks)
    cache_append_kernel(const __grid_constant__ AppendArgs a, int64_t page_slots, int q_tokens) {
  const int64_t x = blockIdx.x;
  if (x < page_slots)
    append_page<DC, DR, PS>(a, x);
  else if (x == page_slots)
    append_check(a);
  else
    rotate_q<DC, DR, AppendCfg<DC, DR, PS>::kMaxQTokens>(a, (x - page_slots - 1) * q_tokens, q_tokens);
}

template <int DC, int DR, int PS>
cudaError_t launch_append_t(const AppendArgs& a, cudaStream_t st) {
  using C = AppendCfg<DC, DR, PS>;
  const int64_t pages = a.batch.n_tok / PS + 2ll * a.batch.n_seq;
  // two items a thread: the loads that are in flight while the angles are worked out
  int q_tokens = 1;
  while (q_tokens < C::kMaxQTokens && 2 * q_tokens * a.n_heads * (DR / 16) <= 2 * C::kThr) q_tokens *= 2;
  const int64_t q = a.q ? (static_cast<int64_t>(a.batch.n_tok) + q_tokens - 1) / q_tokens : 0;
  cache_append_kernel<DC, DR, PS><<<static_cast<unsigned>(pages + 1 + q), C::kThr, 0, st>>>(
      a, pages, q_tokens);
  return cudaGetLastError();
}

template <int DC, int DR>
cudaError_t launch_append_p(const AppendArgs& a, cudaStream_t st) {
  switch (a.cache.page_size) {
    case 16: return launch_append_t<DC, DR, 16>(a, st);
    case 32: return launch_append_t<DC, DR, 32>(a, st);
    case 64: return launch_append_t<DC, DR, 64>(a, st);
    default: return launch_append_t<DC, DR, 128>(a, st);
  }
}

// ------------------------------------------------------------------ gather

struct GatherArgs {
  dsa_cache cache;
  dsa_batch batch;
  uint16_t* latent;
  uint16_t* rope;
  int seq, pos0, n_rows;
  bool wide;  // both outputs on 32-byte boundaries
  WsHeader* ws;
};

// A thread turns 16 codes (one 16-byte load) into 32 bytes of bf16 (one
// 32-byte store), eight rows of the same column for eight loads in flight.
// Bound: bytes, 576 read and 1,152 written a row (17,408 rows 8.2 us, most of
// it the launch; 130,995 rows 43 us, 5.2 TB/s; with four loads in flight and
// 16-byte stores 50 us).
template <int DC, int DR>
struct GatherCfg {
  static constexpr int kCols = (DC + DR) / 16;                  // 36 (5)
  static constexpr int kLanes = DC == 512 ? 8 : 64;             // rows side by side (whole warps)
  static constexpr int kThr = kCols * kLanes;
  static constexpr int kDeep = 8;
  static constexpr int kRows = kLanes * kDeep;
};

template <int DC, int DR>
__global__ void __launch_bounds__(GatherCfg<DC, DR>::kThr)
    cache_gather_kernel(const __grid_constant__ GatherArgs a) {
  using C = GatherCfg<DC, DR>;
  const int ps = a.cache.page_size, shift = 31 - __clz(ps);
  const int len = __ldg(a.batch.seq_lens + a.seq);
  const int end = min(a.pos0 + a.n_rows, min(len, a.batch.max_pages << shift));
  if (blockIdx.x == gridDim.x - 1) {
    unsigned int site = end < a.pos0 + a.n_rows ? kCacheSiteSeq : 0u;
    for (int j = (a.pos0 >> shift) + static_cast<int>(threadIdx.x);
         (static_cast<int64_t>(j) << shift) < end; j += blockDim.x)
      if (!page_ok(a.cache, page_of(a.batch, a.seq, j))) site = max(site, kCacheSitePage);
    write_status(a.ws, site);
    return;
  }
  const int u = threadIdx.x % C::kCols;
  const int row0 = blockIdx.x * C::kRows + threadIdx.x / C::kCols;
  const bool lat = u < DC / 16;
  const uint8_t* pool = lat ? a.cache.latent + u * 16 : a.cache.rope + (u - DC / 16) * 16;
  const int64_t stride = lat ? a.cache.latent_page_stride : a.cache.rope_page_stride;
  const int width = lat ? DC : DR;
  int page[C::kDeep];
#pragma unroll
  for (int i = 0; i < C::kDeep; ++i) {
    const int pos = a.pos0 + row0 + i * C::kLanes;
    page[i] = pos < end ? page_of(a.batch, a.seq, pos >> shift) : -1;
  }
  uint4 v[C::kDeep];
  float s[C::kDeep];
#pragma unroll
  for (int i = 0; i < C::kDeep; ++i) {
    if (!page_ok(a.cache, page[i])) page[i] = -1;
    s[i] = 0.f;
    if (page[i] >= 0) {
      const int row = (a.pos0 + row0 + i * C::kLanes) & (ps - 1);
      v[i] = __ldg(reinterpret_cast<const uint4*>(pool + page[i] * stride + row * width));
      s[i] = __ldg(a.cache.scale + page[i]);
    }
  }
  uint16_t* out = lat ? a.latent + u * 16 : a.rope + (u - DC / 16) * 16;
#pragma unroll
  for (int i = 0; i < C::kDeep; ++i) {
    if (page[i] < 0 || !DSA_IN_BOUNDS(a.ws, row0 + i * C::kLanes, a.n_rows, 64)) continue;
    const float f = pow2f(scale_exp(s[i]));
    const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
    uint32_t o[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 lo = e4m3x2_to_f32(w[e]), hi = e4m3x2_to_f32(w[e] >> 16);
      o[2 * e] = pack_bf16x2(lo.x * f, lo.y * f);
      o[2 * e + 1] = pack_bf16x2(hi.x * f, hi.y * f);
    }
    uint16_t* dst = out + static_cast<int64_t>(row0 + i * C::kLanes) * width;
    if (a.wide)
      asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(o[0]),
                   "r"(o[1]), "r"(o[2]), "r"(o[3]), "r"(o[4]), "r"(o[5]), "r"(o[6]), "r"(o[7])
                   : "memory");
    else {
      reinterpret_cast<uint4*>(dst)[0] = make_uint4(o[0], o[1], o[2], o[3]);
      reinterpret_cast<uint4*>(dst)[1] = make_uint4(o[4], o[5], o[6], o[7]);
    }
  }
}

template <int DC, int DR>
void launch_gather_t(const GatherArgs& a, cudaStream_t st) {
  using C = GatherCfg<DC, DR>;
  const unsigned grid = static_cast<unsigned>((static_cast<int64_t>(a.n_rows) + C::kRows - 1) / C::kRows);
  cache_gather_kernel<DC, DR><<<grid + 1, C::kThr, 0, st>>>(a);
}

}  // namespace

cudaError_t launch_cache_append(const AppendArgs& a, cudaStream_t st) {
  const cudaError_t e = clear_status_for_checks(a.ws, st);
  if (e != cudaSuccess) return e;
  return a.cache.d_latent == 512 ? launch_append_p<512, 64>(a, st)
                                 : launch_append_p<64, 16>(a, st);
}

cudaError_t launch_cache_gather(const dsa_cache& c, const dsa_batch& b, int seq, int pos0,
                                int n_rows, uint16_t* latent, uint16_t* rope, WsHeader* ws,
                                cudaStream_t st) {
  const bool wide = ((reinterpret_cast<uintptr_t>(latent) | reinterpret_cast<uintptr_t>(rope)) & 31u) == 0;
  const cudaError_t e = clear_status_for_checks(ws, st);
  if (e != cudaSuccess) return e;
  const GatherArgs a{c, b, latent, rope, seq, pos0, n_rows, wide, ws};
  if (c.d_latent == 512) launch_gather_t<512, 64>(a, st);
  else launch_gather_t<64, 16>(a, st);
  return cudaGetLastError();
}

}  // namespace dsa
