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
// Bound: the bytes of a prefill chunk (most of them the queries' rope), the
// chain of dependent loads (batch arrays, page table, rows) of a decode step.
//
// One more CTA checks the batch arrays and the page table entries that the
// call uses, and is the only one that writes the status word: the others skip
// what is wrong by the same tests. The word then needs no clearing launch.
#include <cuda_bf16.h>

#include "cache.cuh"

namespace dsa {
namespace {

constexpr int kThreads = 256;
constexpr int kQTokens = 4;  // tokens of a q CTA

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
    ws->status_info = s_bad;
    ws->status = s_bad ? kDevRange : 0u;
  }
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

// Sixteen-byte units of a latent row (8 elements) and pairs of a rope row are
// dealt over the CTA so that each thread holds kUnits and kPairs of them.
template <int DC, int DR, int PS>
struct AppendCfg {
  static constexpr int kThr = PS == 128 ? 2 * kThreads : kThreads;
  static constexpr int kRowUnits = DC / 8;
  static constexpr int kUnits = (PS * kRowUnits + kThr - 1) / kThr;
  static constexpr int kRowPairs = DR / 2;
  static constexpr int kPairs = (PS * kRowPairs + kThr - 1) / kThr;
};

template <int DC, int DR, int PS>
__device__ void append_page(const AppendArgs& a, int64_t slot) {
  using C = AppendCfg<DC, DR, PS>;
  __shared__ int s_exp;
  constexpr int kShift = PS == 16 ? 4 : PS == 32 ? 5 : PS == 64 ? 6 : 7;
  const int b = seq_of_slot(a.batch, slot, 1, kShift, 2);
  const SeqRange r = seq_range(a.batch, PS, b);
  const int64_t j = slot - slot_start(a.batch, b, 1, kShift, 2);
  if (r.n == 0 || j < 0) return;
  const int p0 = r.len - r.n;            // the sequence's first new position
  const int64_t pg = p0 / PS + j;        // this CTA's page of the sequence
  if (pg * PS >= r.len) return;
  const int page = page_of(a.batch, b, pg);
  if (!page_ok(a.cache, page)) return;
  const int base = static_cast<int>(pg) * PS;
  const int r0 = max(p0 - base, 0), r1 = min(r.len - base, PS);  // new rows of the page
  const int64_t tok = static_cast<int64_t>(r.tok0) + base - p0;  // token of row 0 (row r0 on is real)
  const float old_scale = __ldg(a.cache.scale + page);
  if (threadIdx.x == 0) s_exp = kCacheMinExp;

  uint4 lat[C::kUnits];
  int need = kCacheMinExp;
#pragma unroll
  for (int u = 0; u < C::kUnits; ++u) {
    const int x = threadIdx.x + u * C::kThr, row = x / C::kRowUnits;
    lat[u] = make_uint4(0u, 0u, 0u, 0u);
    if (row >= r0 && row < r1)
      lat[u] = __ldg(reinterpret_cast<const uint4*>(a.latent + (tok + row) * a.ld_latent) +
                     x % C::kRowUnits);
  }
  double2 rot[C::kPairs];
#pragma unroll
  for (int u = 0; u < C::kPairs; ++u) {
    const int x = threadIdx.x + u * C::kThr, row = x / C::kRowPairs, i = x % C::kRowPairs;
    rot[u] = make_double2(0.0, 0.0);
    if (row >= r0 && row < r1) {
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
#pragma unroll
  for (int u = 0; u < C::kUnits; ++u) {
    const uint32_t w[4] = {lat[u].x, lat[u].y, lat[u].z, lat[u].w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 f = bf16x2(w[e]);
      need = max(need, max(need_exp_f32(f.x), need_exp_f32(f.y)));
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
#pragma unroll
  for (int u = 0; u < C::kUnits; ++u) {
    const int x = threadIdx.x + u * C::kThr, row = x / C::kRowUnits;
    if (row < r0 || row >= r1) continue;
    const float2 f0 = bf16x2(lat[u].x), f1 = bf16x2(lat[u].y), f2 = bf16x2(lat[u].z),
                 f3 = bf16x2(lat[u].w);
    uint2 v;
    v.x = f32_to_e4m3x2(f0.x * inv, f0.y * inv) | f32_to_e4m3x2(f1.x * inv, f1.y * inv) << 16;
    v.y = f32_to_e4m3x2(f2.x * inv, f2.y * inv) | f32_to_e4m3x2(f3.x * inv, f3.y * inv) << 16;
    *reinterpret_cast<uint2*>(lat_page + x * 8) = v;
  }
  const double inv_d = static_cast<double>(inv);
#pragma unroll
  for (int u = 0; u < C::kPairs; ++u) {
    const int x = threadIdx.x + u * C::kThr, row = x / C::kRowPairs, i = x % C::kRowPairs;
    if (row < r0 || row >= r1) continue;
    const uint32_t v =
        f32_to_e4m3x2(f64_to_f32_odd(rot[u].x * inv_d), f64_to_f32_odd(rot[u].y * inv_d));
    uint8_t* dst = rope_page + row * DR;
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

// Rotates the queries' rope of kQTokens tokens. A work item is eight pairs of
// one head: two 16-byte groups, adjacent (interleaved) or d_rope/2 apart.
template <int DC, int DR>
__device__ void rotate_q(const AppendArgs& a, int64_t tok0) {
  __shared__ float2 s_cs[kQTokens][DR / 2];
  __shared__ int s_pos[kQTokens];
  if (threadIdx.x < kQTokens) {
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
  for (int x = threadIdx.x; x < kQTokens * (DR / 2); x += blockDim.x) {
    const int k = x / (DR / 2), i = x % (DR / 2);
    double sn, cs;
    sincos(static_cast<double>(s_pos[k]) * static_cast<double>(__ldg(a.inv_freq + i)), &sn, &cs);
    s_cs[k][i] = make_float2(static_cast<float>(cs), static_cast<float>(sn));
  }
  __syncthreads();
  const int per_head = DR / 16, items = kQTokens * a.n_heads * per_head;
  for (int x = threadIdx.x; x < items; x += blockDim.x) {
    const int g = x % per_head, h = (x / per_head) % a.n_heads, k = x / per_head / a.n_heads;
    if (s_pos[k] < 0) continue;
    const int64_t tok = tok0 + k;
    const uint4* src = reinterpret_cast<const uint4*>(a.q_rope + tok * a.ld_q_tok + h * a.ld_q_head);
    uint4* dst = reinterpret_cast<uint4*>(a.q + (tok * a.n_heads + h) * (DC + DR) + DC);
    const float2* cs = &s_cs[k][g * 8];
    if (a.halves) {
      const uint4 v = __ldg(src + g), w = __ldg(src + g + DR / 16);
      const uint32_t vi[4] = {v.x, v.y, v.z, v.w}, wi[4] = {w.x, w.y, w.z, w.w};
      uint32_t vo[4], wo[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 p = bf16x2(vi[e]), q = bf16x2(wi[e]), c0 = cs[2 * e], c1 = cs[2 * e + 1];
        vo[e] = pack_bf16x2(p.x * c0.x - q.x * c0.y, p.y * c1.x - q.y * c1.y);
        wo[e] = pack_bf16x2(q.x * c0.x + p.x * c0.y, q.y * c1.x + p.y * c1.y);
      }
      dst[g] = make_uint4(vo[0], vo[1], vo[2], vo[3]);
      dst[g + DR / 16] = make_uint4(wo[0], wo[1], wo[2], wo[3]);
    } else {
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const uint4 v = __ldg(src + 2 * g + half);
        const uint32_t vi[4] = {v.x, v.y, v.z, v.w};
        uint32_t vo[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 p = bf16x2(vi[e]), c = cs[4 * half + e];
          vo[e] = pack_bf16x2(p.x * c.x - p.y * c.y, p.y * c.x + p.x * c.y);
        }
        dst[2 * g + half] = make_uint4(vo[0], vo[1], vo[2], vo[3]);
      }
    }
  }
}

template <int DC, int DR, int PS>
__global__ void __launch_bounds__(AppendCfg<DC, DR, PS>::kThr)
    cache_append_kernel(const __grid_constant__ AppendArgs a, int64_t page_slots) {
  const int64_t x = blockIdx.x;
  if (x < page_slots) append_page<DC, DR, PS>(a, x);
  else if (x == page_slots) append_check(a);
  else rotate_q<DC, DR>(a, (x - page_slots - 1) * kQTokens);
}

template <int DC, int DR, int PS>
cudaError_t launch_append_t(const AppendArgs& a, cudaStream_t st) {
  const int64_t pages = a.batch.n_tok / PS + 2ll * a.batch.n_seq;
  const int64_t q = a.q ? (static_cast<int64_t>(a.batch.n_tok) + kQTokens - 1) / kQTokens : 0;
  cache_append_kernel<DC, DR, PS><<<static_cast<unsigned>(pages + 1 + q),
                                    AppendCfg<DC, DR, PS>::kThr, 0, st>>>(a, pages);
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
  WsHeader* ws;
};

// A thread turns 16 codes (one 16-byte load) into 32 bytes of bf16; kGatherIlp
// of them at once keep enough loads in flight. Bound: bytes (576 read and
// 1,152 written a row).
constexpr int kGatherIlp = 4;

template <int DC, int DR>
__global__ void __launch_bounds__(kThreads) cache_gather_kernel(const __grid_constant__ GatherArgs a) {
  constexpr int kRow = (DC + DR) / 16;
  const int ps = a.cache.page_size;
  const int len = __ldg(a.batch.seq_lens + a.seq);
  const int end = min(a.pos0 + a.n_rows, min(len, a.batch.max_pages * ps));
  if (blockIdx.x == gridDim.x - 1) {
    unsigned int site = end < a.pos0 + a.n_rows ? kCacheSiteSeq : 0u;
    for (int j = a.pos0 / ps + static_cast<int>(threadIdx.x); static_cast<int64_t>(j) * ps < end;
         j += blockDim.x)
      if (!page_ok(a.cache, page_of(a.batch, a.seq, j))) site = max(site, kCacheSitePage);
    write_status(a.ws, site);
    return;
  }
  uint4 v[kGatherIlp];
  float s[kGatherIlp];
  const int64_t x0 = static_cast<int64_t>(blockIdx.x) * kThreads * kGatherIlp + threadIdx.x;
#pragma unroll
  for (int i = 0; i < kGatherIlp; ++i) {
    const int64_t x = x0 + i * kThreads;
    const int64_t pos = a.pos0 + x / kRow;
    const int u = static_cast<int>(x % kRow);
    s[i] = 0.f;
    if (pos >= end) continue;
    const int page = page_of(a.batch, a.seq, pos / ps), row = static_cast<int>(pos % ps);
    if (!page_ok(a.cache, page)) continue;
    s[i] = pow2f(scale_exp(__ldg(a.cache.scale + page)));
    const uint8_t* src = u < DC / 16
                             ? a.cache.latent + page * a.cache.latent_page_stride + row * DC + u * 16
                             : a.cache.rope + page * a.cache.rope_page_stride + row * DR +
                                   (u - DC / 16) * 16;
    v[i] = __ldg(reinterpret_cast<const uint4*>(src));
  }
#pragma unroll
  for (int i = 0; i < kGatherIlp; ++i) {
    if (s[i] == 0.f) continue;
    const int64_t x = x0 + i * kThreads, row = x / kRow;
    const int u = static_cast<int>(x % kRow);
    const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
    uint32_t o[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 lo = e4m3x2_to_f32(w[e]), hi = e4m3x2_to_f32(w[e] >> 16);
      o[2 * e] = pack_bf16x2(lo.x * s[i], lo.y * s[i]);
      o[2 * e + 1] = pack_bf16x2(hi.x * s[i], hi.y * s[i]);
    }
    uint4* dst = reinterpret_cast<uint4*>(u < DC / 16 ? a.latent + row * DC + u * 16
                                                      : a.rope + row * DR + (u - DC / 16) * 16);
    dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
    dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
  }
}

}  // namespace

cudaError_t launch_cache_append(const AppendArgs& a, cudaStream_t st) {
  return a.cache.d_latent == 512 ? launch_append_p<512, 64>(a, st)
                                 : launch_append_p<64, 16>(a, st);
}

cudaError_t launch_cache_gather(const dsa_cache& c, const dsa_batch& b, int seq, int pos0,
                                int n_rows, uint16_t* latent, uint16_t* rope, WsHeader* ws,
                                cudaStream_t st) {
  const GatherArgs a{c, b, latent, rope, seq, pos0, n_rows, ws};
  const int64_t per = static_cast<int64_t>(kThreads) * kGatherIlp;
  const int64_t units = static_cast<int64_t>(n_rows) * ((c.d_latent + c.d_rope) / 16);
  const unsigned grid = static_cast<unsigned>((units + per - 1) / per + 1);
  if (c.d_latent == 512) cache_gather_kernel<512, 64><<<grid, kThreads, 0, st>>>(a);
  else cache_gather_kernel<64, 16><<<grid, kThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace dsa
