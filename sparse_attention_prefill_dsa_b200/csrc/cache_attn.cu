// cache_attn.cu -- attention over the paged 8-bit latent cache.
#include "cache.cuh"

namespace dsa {
namespace {

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

size_t cache_attn_scratch_bytes(const dsa_cache&, const dsa_batch&, int) { return 0; }

cudaError_t launch_cache_attn(const CacheAttnArgs& a, void*, cudaStream_t st) {
  cudaError_t e = cudaMemsetAsync(a.ws, 0, kWsHeaderBytes, st);
  if (e != cudaSuccess) return e;
  cache_attn_check<<<1, 256, 0, st>>>(a);
  const int64_t rows = static_cast<int64_t>(a.batch.n_tok) * a.n_heads;
  const unsigned grid = static_cast<unsigned>((rows + kRowWarps - 1) / kRowWarps);
  if (a.cache.d_latent == 512) cache_attn_rows<512, 64><<<grid, 32 * kRowWarps, 0, st>>>(a);
  else cache_attn_rows<64, 16><<<grid, 32 * kRowWarps, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace dsa
