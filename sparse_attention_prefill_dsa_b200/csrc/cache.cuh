// cache.cuh -- shared definitions of the paged 8-bit latent cache (cache.cu,
// cache_attn.cu, cache_api.cu).
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "dsa.h"
#include "dsa_internal.cuh"

namespace dsa {

// Scales are 2^e with e in this range: e4m3 * 2^-32 and up is far above
// float32's subnormals, and 2^120 * 448 covers every finite bf16.
constexpr int kCacheMinExp = -32;
constexpr int kCacheMaxExp = 120;

// Where the status word's `info` points for errors of the batch arrays.
constexpr unsigned int kCacheSiteSeq = 1;   // cu_seqlens / seq_lens of a sequence
constexpr unsigned int kCacheSitePage = 2;  // a page table entry

// Sequence b of a batch on the device: its new tokens [tok0, tok0 + n) and
// its rows [0, len); n = 0 (and nothing else is to be used) when the arrays
// fail the checks of dsa_batch.
struct SeqRange {
  int tok0, n, len;
  bool ok;
};

__device__ __forceinline__ SeqRange seq_range(const dsa_batch& bt, int page_size, int b) {
  SeqRange r;
  const int c0 = __ldg(bt.cu_seqlens + b), c1 = __ldg(bt.cu_seqlens + b + 1);
  const int len = __ldg(bt.seq_lens + b);
  r.ok = c0 >= 0 && c1 >= c0 && c1 <= bt.n_tok && len >= c1 - c0 &&
         len <= static_cast<int64_t>(bt.max_pages) * page_size;
  r.tok0 = c0;
  r.n = r.ok ? c1 - c0 : 0;
  r.len = len;
  return r;
}

// The sequences' slots of a grid that is sized without knowing cu_seqlens:
// sequence b gets the slots [start(b), start(b + 1)), start(b) =
// floor(cu_seqlens[b] * mul / 2^shift) + extra * b, which is ascending in b. A
// sequence of n tokens then has at least floor(n * mul / 2^shift) + extra slots.
// Returns the b whose slots hold `slot` (0 <= slot, n_seq >= 1). For
// cu_seqlens that do not ascend it returns some b in range.
__device__ __forceinline__ int64_t slot_start(const dsa_batch& bt, int b, int mul, int shift,
                                              int extra) {
  const int64_t c = min(max(__ldg(bt.cu_seqlens + b), 0), bt.n_tok);
  return ((c * mul) >> shift) + static_cast<int64_t>(extra) * b;
}

__device__ __forceinline__ int seq_of_slot(const dsa_batch& bt, int64_t slot, int mul, int shift,
                                           int extra) {
  int lo = 0, hi = bt.n_seq - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (slot_start(bt, mid, mul, shift, extra) <= slot) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// The sequence a token belongs to, or -1 (a token of no sequence).
__device__ __forceinline__ int seq_of_token(const dsa_batch& bt, int tok) {
  int lo = 0, hi = bt.n_seq - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (__ldg(bt.cu_seqlens + mid) <= tok) lo = mid;
    else hi = mid - 1;
  }
  return __ldg(bt.cu_seqlens + lo) <= tok && tok < __ldg(bt.cu_seqlens + lo + 1) ? lo : -1;
}

// Two e4m3 codes (low byte first) as float32, exact.
__device__ __forceinline__ float2 e4m3x2_to_f32(uint32_t codes) {
  const __half2_raw h =
      __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(codes & 0xFFFFu), __NV_E4M3);
  return __half22float2(__half2(h));
}

// Two float32 as e4m3 codes (x in the low byte): nearest, ties to even.
__device__ __forceinline__ uint32_t f32_to_e4m3x2(float x, float y) {
  return __nv_cvt_float2_to_fp8x2(make_float2(x, y), __NV_SATFINITE, __NV_E4M3);
}

// 2^e as float32, -126 <= e <= 127.
__device__ __forceinline__ float pow2f(int e) {
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// Exponent of a page's scale (a power of two), kept in the scales' range.
__device__ __forceinline__ int scale_exp(float s) {
  const int e = static_cast<int>((__float_as_uint(s) >> 23) & 255u) - 127;
  return min(max(e, kCacheMinExp), kCacheMaxExp);
}

struct AppendArgs {
  dsa_cache cache;
  dsa_batch batch;
  const uint16_t* latent;
  const uint16_t* rope;
  const float* inv_freq;
  const uint16_t* q_rope;
  uint16_t* q;
  int64_t ld_latent, ld_rope, ld_q_tok, ld_q_head;
  int n_heads, halves;
  WsHeader* ws;
};

struct CacheAttnArgs {
  dsa_cache cache;
  dsa_batch batch;
  const uint16_t* q;
  uint16_t* out;
  float* lse;
  int n_heads, window, n_sink;
  float scale_log2;  // softmax_scale * log2(e)
  WsHeader* ws;
};

cudaError_t launch_cache_append(const AppendArgs& a, cudaStream_t st);
cudaError_t launch_cache_gather(const dsa_cache& c, const dsa_batch& b, int seq, int pos0,
                                int n_rows, uint16_t* latent, uint16_t* rope, WsHeader* ws,
                                cudaStream_t st);
// Workspace of the attention past the header.
size_t cache_attn_scratch_bytes(const dsa_cache& c, const dsa_batch& b, int n_heads);
// wait_cycles: the limit of the kernel's waits where it is not negative (a test's).
cudaError_t launch_cache_attn(const CacheAttnArgs& a, void* scratch, cudaStream_t st,
                              long long wait_cycles = -1);

}  // namespace dsa
