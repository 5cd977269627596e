// cache_api.cu -- the C ABI of the paged 8-bit latent cache: argument checks
// (complete before anything is launched) and launches.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "cache.cuh"

namespace {

constexpr int kMaxTok = 1 << 24;  // token rows x 128 heads stay below 2^31
constexpr int64_t kMaxLen = 1ll << 30;
constexpr int64_t kMaxPageStride = 1ll << 39;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Sizes of the structs (no pointer is looked at).
dsa_status check_sizes(const dsa_cache* c, const dsa_batch* b) {
  if (!c || !b) return DSA_ERR_NULL;
  if (!((c->d_latent == 512 && c->d_rope == 64) || (c->d_latent == 64 && c->d_rope == 16)))
    return DSA_ERR_DIMS;
  const int ps = c->page_size;
  if (ps != 16 && ps != 32 && ps != 64 && ps != 128) return DSA_ERR_DIMS;
  if (c->n_pages < 1) return DSA_ERR_DIMS;
  if (c->latent_page_stride < static_cast<int64_t>(ps) * c->d_latent ||
      c->rope_page_stride < static_cast<int64_t>(ps) * c->d_rope ||
      c->latent_page_stride > kMaxPageStride || c->rope_page_stride > kMaxPageStride)
    return DSA_ERR_DIMS;
  if (b->n_seq < 0 || b->n_seq > kMaxTok || b->max_pages < 1 || b->n_tok < 0 ||
      b->n_tok >= kMaxTok || b->reserved != 0 ||
      static_cast<int64_t>(b->max_pages) * ps > kMaxLen)
    return DSA_ERR_DIMS;
  if (c->latent_page_stride % 16 != 0 || c->rope_page_stride % 16 != 0) return DSA_ERR_ALIGN;
  return DSA_OK;
}

dsa_status check_batch(const dsa_cache* c, const dsa_batch* b) {
  const dsa_status s = check_sizes(c, b);
  if (s != DSA_OK) return s;
  if (!c->latent || !c->rope || !c->scale || !b->cu_seqlens) return DSA_ERR_NULL;
  if (b->n_seq > 0 && (!b->page_table || !b->seq_lens)) return DSA_ERR_NULL;
  if (!aligned16(c->latent) || !aligned16(c->rope) || !aligned16(c->scale) ||
      !aligned16(b->page_table) || !aligned16(b->cu_seqlens) || !aligned16(b->seq_lens))
    return DSA_ERR_ALIGN;
  return DSA_OK;
}

// Nothing to read or write: the token tensors may be NULL, as empty ones are.
bool nothing(const dsa_batch* b) { return b->n_seq == 0 || b->n_tok == 0; }

dsa_status check_ws(const dsa_cache* c, const dsa_batch* b, int32_t n_heads, bool header_only,
                    const void* ws, size_t bytes) {
  if (!ws) return DSA_ERR_WORKSPACE;
  if (!aligned16(ws)) return DSA_ERR_ALIGN;
  const size_t need =
      header_only ? dsa::kWsHeaderBytes : dsa_cache_workspace_size(c, b, n_heads);
  return bytes < need ? DSA_ERR_WORKSPACE : DSA_OK;
}

// The current device is a B200 and the one that holds the workspace (work on
// another device's memory would run over NVLink, or fault, as it would on the
// host's).
dsa_status check_device(const void* ws) {
  const dsa_status s = dsa::check_current_device();
  if (s != DSA_OK) return s;
  int dev = 0;
  cudaPointerAttributes at;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaPointerGetAttributes(&at, ws) != cudaSuccess) {
    cudaGetLastError();
    return DSA_ERR_CUDA;
  }
  if (at.type == cudaMemoryTypeManaged) return DSA_OK;
  return at.type == cudaMemoryTypeDevice && at.device == dev ? DSA_OK : DSA_ERR_DEVICE;
}

dsa_status from_cuda(cudaError_t e) { return e == cudaSuccess ? DSA_OK : DSA_ERR_CUDA; }

// A call with nothing to do still clears the status word.
dsa_status nothing_to_do(void* ws, void* stream) {
  return from_cuda(
      cudaMemsetAsync(ws, 0, dsa::kWsHeaderBytes, static_cast<cudaStream_t>(stream)));
}

dsa_status attend(const dsa_cache* cache, const dsa_batch* batch, const uint16_t* q,
                  int32_t n_heads, float softmax_scale, int32_t window, int32_t n_sink,
                  uint16_t* out, float* lse, long long wait_cycles, void* workspace,
                  size_t workspace_bytes, void* stream) {
  dsa_status s = check_batch(cache, batch);
  if (s != DSA_OK) return s;
  if (n_heads < 1 || n_heads > 128 || window < 0 || n_sink < 0) return DSA_ERR_DIMS;
  if (!(softmax_scale > 0.0f && softmax_scale < 1e30f)) return DSA_ERR_DIMS;
  if (!nothing(batch) && (!q || !out)) return DSA_ERR_NULL;
  if (!aligned16(q) || !aligned16(out) || !aligned16(lse)) return DSA_ERR_ALIGN;
  s = check_ws(cache, batch, n_heads, false, workspace, workspace_bytes);
  if (s != DSA_OK) return s;
  s = check_device(workspace);
  if (s != DSA_OK) return s;
  if (nothing(batch)) return nothing_to_do(workspace, stream);
  dsa::CacheAttnArgs a;
  a.cache = *cache;
  a.batch = *batch;
  a.q = q;
  a.out = out;
  a.lse = lse;
  a.n_heads = n_heads;
  a.window = window;
  a.n_sink = n_sink;
  a.scale_log2 = softmax_scale * 1.4426950408889634f;
  a.ws = static_cast<dsa::WsHeader*>(workspace);
  return from_cuda(dsa::launch_cache_attn(a, static_cast<char*>(workspace) + dsa::kWsHeaderBytes,
                                          static_cast<cudaStream_t>(stream), wait_cycles));
}

}  // namespace

extern "C" {

size_t dsa_cache_workspace_size(const dsa_cache* cache, const dsa_batch* batch, int32_t n_heads) {
  if (check_sizes(cache, batch) != DSA_OK || n_heads < 1 || n_heads > 128) return 0;
  return dsa::kWsHeaderBytes + dsa::cache_attn_scratch_bytes(*cache, *batch, n_heads);
}

dsa_status dsa_cache_append(const dsa_cache* cache, const dsa_batch* batch,
                            const uint16_t* latent, int64_t ld_latent, const uint16_t* rope,
                            int64_t ld_rope, const float* inv_freq, int32_t rope_style,
                            const uint16_t* q_rope, int64_t ld_q_tok, int64_t ld_q_head,
                            uint16_t* q, int32_t n_heads, void* workspace, size_t workspace_bytes,
                            void* stream) {
  dsa_status s = check_batch(cache, batch);
  if (s != DSA_OK) return s;
  if (rope_style != DSA_ROPE_INTERLEAVED && rope_style != DSA_ROPE_HALVES) return DSA_ERR_DIMS;
  if (!inv_freq || (!nothing(batch) && (!latent || !rope || !q_rope != !q))) return DSA_ERR_NULL;
  if (!aligned16(latent) || !aligned16(rope) || !aligned16(inv_freq) || !aligned16(q_rope) ||
      !aligned16(q))
    return DSA_ERR_ALIGN;
  if (ld_latent < cache->d_latent || ld_rope < cache->d_rope) return DSA_ERR_DIMS;
  if (ld_latent % 8 != 0 || ld_rope % 8 != 0) return DSA_ERR_ALIGN;
  if (q) {
    if (n_heads < 1 || n_heads > 128 || ld_q_tok < 0 || ld_q_head < 0) return DSA_ERR_DIMS;
    if (ld_q_tok % 8 != 0 || ld_q_head % 8 != 0) return DSA_ERR_ALIGN;
  }
  s = check_ws(cache, batch, n_heads, true, workspace, workspace_bytes);
  if (s != DSA_OK) return s;
  s = check_device(workspace);
  if (s != DSA_OK) return s;
  if (nothing(batch)) return nothing_to_do(workspace, stream);
  dsa::AppendArgs a;
  a.cache = *cache;
  a.batch = *batch;
  a.latent = latent;
  a.rope = rope;
  a.inv_freq = inv_freq;
  a.q_rope = q_rope;
  a.q = q;
  a.ld_latent = ld_latent;
  a.ld_rope = ld_rope;
  a.ld_q_tok = ld_q_tok;
  a.ld_q_head = ld_q_head;
  a.n_heads = n_heads;
  a.halves = rope_style == DSA_ROPE_HALVES;
  a.ws = static_cast<dsa::WsHeader*>(workspace);
  return from_cuda(dsa::launch_cache_append(a, static_cast<cudaStream_t>(stream)));
}

dsa_status dsa_cache_gather(const dsa_cache* cache, const dsa_batch* batch, int32_t seq,
                            int32_t pos0, int32_t n_rows, uint16_t* latent, uint16_t* rope,
                            void* workspace, size_t workspace_bytes, void* stream) {
  dsa_status s = check_batch(cache, batch);
  if (s != DSA_OK) return s;
  if (seq < 0 || seq >= batch->n_seq || pos0 < 0 || n_rows < 0 ||
      static_cast<int64_t>(pos0) + n_rows >
          static_cast<int64_t>(batch->max_pages) * cache->page_size)
    return DSA_ERR_DIMS;
  if (n_rows > 0 && (!latent || !rope)) return DSA_ERR_NULL;
  if (!aligned16(latent) || !aligned16(rope)) return DSA_ERR_ALIGN;
  s = check_ws(cache, batch, 1, true, workspace, workspace_bytes);
  if (s != DSA_OK) return s;
  s = check_device(workspace);
  if (s != DSA_OK) return s;
  if (n_rows == 0) return nothing_to_do(workspace, stream);
  return from_cuda(dsa::launch_cache_gather(*cache, *batch, seq, pos0, n_rows, latent, rope,
                                            static_cast<dsa::WsHeader*>(workspace),
                                            static_cast<cudaStream_t>(stream)));
}

dsa_status dsa_cache_attn(const dsa_cache* cache, const dsa_batch* batch, const uint16_t* q,
                          int32_t n_heads, float softmax_scale, int32_t window, int32_t n_sink,
                          uint16_t* out, float* lse, void* workspace, size_t workspace_bytes,
                          void* stream) {
  return attend(cache, batch, q, n_heads, softmax_scale, window, n_sink, out, lse, -1, workspace,
                workspace_bytes, stream);
}

dsa_status dsa_selftest_cache_wait(const dsa_cache* cache, const dsa_batch* batch,
                                   const uint16_t* q, int32_t n_heads, float softmax_scale,
                                   int32_t window, int32_t n_sink, uint16_t* out, float* lse,
                                   int64_t wait_cycles, void* workspace, size_t workspace_bytes,
                                   void* stream) {
  if (wait_cycles < 0 || (cache && cache->d_latent != 512)) return DSA_ERR_DIMS;
  return attend(cache, batch, q, n_heads, softmax_scale, window, n_sink, out, lse, wait_cycles,
                workspace, workspace_bytes, stream);
}

}  // extern "C"
