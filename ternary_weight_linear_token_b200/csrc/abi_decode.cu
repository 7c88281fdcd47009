// abi_decode.cu -- the C ABI of the decode step's other operators: the 8-bit
// paged key/value cache, products with 4-bit weights, token log
// probabilities.  As in abi.cu every argument check runs before any CUDA
// call.
#include <cuda_runtime.h>

#include <math.h>

#include "../../include/bitnet158.h"
#include "internal.h"

using namespace bitnet;

namespace {

constexpr int64_t kMaxCount = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxK = int64_t(1) << 24;

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool float_type(bitnet_dtype t) { return t == BITNET_F32 || t == BITNET_BF16; }
int64_t float_size(bitnet_dtype t) { return t == BITNET_F32 ? 4 : 2; }
bitnet_status from_cuda(cudaError_t e) { return e == cudaSuccess ? BITNET_OK : BITNET_ERR_CUDA; }
bool overlap(const void *a, uint64_t na, const void *b, uint64_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return na > 0 && nb > 0 && x < y + nb && y < x + na;
}

bitnet_status check_cache(const bitnet_kv_cache *c) {
  if (c == nullptr) return BITNET_ERR_INVALID_ARG;
  if (c->num_pages < 1 || c->num_pages > kMaxCount || c->heads < 1 || c->heads > 32767)
    return BITNET_ERR_INVALID_ARG;
  if (c->page_tokens != 16 && c->page_tokens != 32 && c->page_tokens != 64 && c->page_tokens != 128)
    return BITNET_ERR_UNSUPPORTED_SHAPE;
  if (c->head_dim != 64 && c->head_dim != 128) return BITNET_ERR_UNSUPPORTED_SHAPE;
  if (c->k_codes == nullptr || c->v_codes == nullptr || c->k_scales == nullptr || c->v_scales == nullptr)
    return BITNET_ERR_INVALID_ARG;
  if (!aligned(c->k_codes, 16) || !aligned(c->v_codes, 16) || !aligned(c->k_scales, 4) ||
      !aligned(c->v_scales, 4))
    return BITNET_ERR_MISALIGNED;
  return BITNET_OK;
}

// A window past every position is the same as one of 2^31 - 1 (and a sum with
// it must not overflow).
int64_t window_of(int64_t window) { return window < kMaxCount ? window : kMaxCount; }

// Sizes of a batch; then, where it has rows, its arrays.
bitnet_status check_batch_sizes(int64_t T, int64_t B, int64_t max_pages, const int32_t *offsets,
                                int64_t max_new, const bitnet_kv_cache *cache) {
  if (T < 0 || T > kMaxCount || B < 0 || B > kMaxCount || max_pages < 0 || max_new < 0)
    return BITNET_ERR_INVALID_ARG;
  if (max_pages > (int64_t(1) << 30) / cache->page_tokens || max_new > kMaxCount) return BITNET_ERR_INVALID_ARG;
  if (offsets == nullptr && T != B) return BITNET_ERR_INVALID_ARG;  // one row per sequence
  return BITNET_OK;
}
bitnet_status check_batch_arrays(const int32_t *pages, int64_t max_pages, const int32_t *lens,
                                 const int32_t *offsets) {
  if ((pages == nullptr && max_pages > 0) || lens == nullptr) return BITNET_ERR_INVALID_ARG;
  if (!aligned(pages, 4) || !aligned(lens, 4) || !aligned(offsets, 4)) return BITNET_ERR_MISALIGNED;
  return BITNET_OK;
}

KvCache cache_of(const bitnet_kv_cache *c) {
  return {c->k_codes, c->v_codes, c->k_scales, c->v_scales, c->num_pages, c->heads, c->page_tokens, c->head_dim};
}

bitnet_status check_attention(const bitnet_kv_cache *cache, bitnet_dtype dtype, int64_t T, int32_t q_heads,
                              int64_t B, int64_t max_pages, const int32_t *offsets, int64_t max_new,
                              int64_t window) {
  if (bitnet_status st = check_cache(cache)) return st;
  if (!float_type(dtype)) return BITNET_ERR_INVALID_ARG;
  if (bitnet_status st = check_batch_sizes(T, B, max_pages, offsets, max_new, cache)) return st;
  if (q_heads < 1 || q_heads % cache->heads != 0 || window < 0) return BITNET_ERR_INVALID_ARG;
  if (q_heads > 32767) return BITNET_ERR_UNSUPPORTED_SHAPE;
  return BITNET_OK;
}

}  // namespace

extern "C" {

bitnet_status bitnet_kv_append(const bitnet_kv_cache *cache, const void *K, int64_t k_stride, const void *V,
                               int64_t v_stride, bitnet_dtype dtype, int64_t T, const int32_t *pages,
                               int64_t max_pages, const int32_t *lens, const int32_t *offsets, int64_t B,
                               int64_t max_new, bitnet_stream_t stream) {
  if (bitnet_status st = check_cache(cache)) return st;
  if (!float_type(dtype)) return BITNET_ERR_INVALID_ARG;
  if (bitnet_status st = check_batch_sizes(T, B, max_pages, offsets, max_new, cache)) return st;
  if (T == 0 || B == 0) return BITNET_OK;
  if (K == nullptr || V == nullptr) return BITNET_ERR_INVALID_ARG;
  if (bitnet_status st = check_batch_arrays(pages, max_pages, lens, offsets)) return st;
  const int64_t row = static_cast<int64_t>(cache->heads) * cache->head_dim, size = float_size(dtype);
  if (T > 1 && (k_stride < row || v_stride < row)) return BITNET_ERR_INVALID_ARG;
  if (k_stride > (int64_t(1) << 40) || v_stride > (int64_t(1) << 40)) return BITNET_ERR_INVALID_ARG;
  if (!aligned(K, 16) || !aligned(V, 16) || (T > 1 && (k_stride * size % 16 != 0 || v_stride * size % 16 != 0)))
    return BITNET_ERR_MISALIGNED;
  const int64_t P = cache->page_tokens, tiles = max_new <= 1 ? 1 : (max_new + P - 2) / P + 1;
  if (tiles > kMaxCount / B) return BITNET_ERR_UNSUPPORTED_SHAPE;
  LaunchCtx ctx;
  if (const int st = launch_ctx_status(stream, &ctx)) return static_cast<bitnet_status>(st);
  const KvBatch batch = {pages, lens, offsets, max_pages, B, T};
  return from_cuda(launch_kv_append(cache_of(cache), K, V, dtype, k_stride, v_stride, batch, max_new, ctx));
}

size_t bitnet_kv_attention_workspace_size(const bitnet_kv_cache *cache, bitnet_dtype dtype, int64_t T,
                                          int32_t q_heads, int64_t B, int64_t max_pages, int64_t max_new,
                                          int64_t window) {
  int32_t some = 0;  // offsets or none: the workspace is the same
  if (check_attention(cache, dtype, T, q_heads, B, max_pages, &some, max_new, window) != BITNET_OK ||
      T == 0 || B == 0)
    return 0;
  const AttnArgs args = {nullptr, nullptr, dtype, q_heads, 1.0f, window_of(window), max_new};
  const KvBatch batch = {nullptr, nullptr, nullptr, max_pages, B, T};
  return kv_attention_fits(cache_of(cache), batch, args) ? kv_attention_workspace(cache_of(cache), batch, args) : 0;
}

bitnet_status bitnet_kv_attention(const bitnet_kv_cache *cache, const void *Q, void *O, bitnet_dtype dtype,
                                  int64_t T, int32_t q_heads, const int32_t *pages, int64_t max_pages,
                                  const int32_t *lens, const int32_t *offsets, int64_t B, int64_t max_new,
                                  float scale, int64_t window, void *workspace, size_t workspace_bytes,
                                  bitnet_stream_t stream) {
  if (bitnet_status st = check_attention(cache, dtype, T, q_heads, B, max_pages, offsets, max_new, window))
    return st;
  if (!isfinite(scale)) return BITNET_ERR_INVALID_ARG;
  if (T == 0 || B == 0) return BITNET_OK;
  if (Q == nullptr || O == nullptr) return BITNET_ERR_INVALID_ARG;
  if (bitnet_status st = check_batch_arrays(pages, max_pages, lens, offsets)) return st;
  if (!aligned(Q, 16) || !aligned(O, 16)) return BITNET_ERR_MISALIGNED;
  const uint64_t bytes = static_cast<uint64_t>(T) * q_heads * cache->head_dim * float_size(dtype);
  if (overlap(Q, bytes, O, bytes)) return BITNET_ERR_INVALID_ARG;
  const AttnArgs args = {Q, O, dtype, q_heads, scale, window_of(window), max_new};
  const KvBatch batch = {pages, lens, offsets, max_pages, B, T};
  const KvCache c = cache_of(cache);
  if (!kv_attention_fits(c, batch, args)) return BITNET_ERR_UNSUPPORTED_SHAPE;
  const size_t need = kv_attention_workspace(c, batch, args);
  if (need > 0) {
    if (workspace == nullptr || workspace_bytes < need) return BITNET_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return BITNET_ERR_MISALIGNED;
  }
  LaunchCtx ctx;
  if (const int st = launch_ctx_status(stream, &ctx)) return static_cast<bitnet_status>(st);
  return from_cuda(launch_kv_attention(c, batch, args, workspace, ctx));
}

bitnet_status bitnet_quantize_weights_w4(const void *W, bitnet_dtype w_dtype, int64_t N, int64_t K,
                                         int32_t group, uint8_t *packed, void *scales, bitnet_stream_t stream) {
  if (!float_type(w_dtype) || N < 0 || N > kMaxCount || K <= 0) return BITNET_ERR_INVALID_ARG;
  if ((group != 32 && group != 64 && group != 128) || K % group != 0 || K > kMaxK)
    return BITNET_ERR_UNSUPPORTED_SHAPE;
  if (N == 0) return BITNET_OK;
  if (W == nullptr || packed == nullptr || scales == nullptr) return BITNET_ERR_INVALID_ARG;
  if (!aligned(W, 16) || !aligned(packed, 16) || !aligned(scales, 16)) return BITNET_ERR_MISALIGNED;
  const uint64_t n = static_cast<uint64_t>(N) * K;
  if (overlap(W, n * float_size(w_dtype), packed, n / 2) ||
      overlap(W, n * float_size(w_dtype), scales, n / group * 2))
    return BITNET_ERR_INVALID_ARG;
  LaunchCtx ctx;
  if (const int st = launch_ctx_status(stream, &ctx)) return static_cast<bitnet_status>(st);
  return from_cuda(launch_quantize_weights_w4(W, w_dtype, N, K, group, packed, static_cast<uint16_t *>(scales), ctx));
}

bitnet_status bitnet_w4a16_matmul(const void *X, bitnet_dtype x_dtype, const uint8_t *packed,
                                  const void *scales, int64_t M, int64_t N, int64_t K, int32_t group, void *Y,
                                  bitnet_dtype y_dtype, uint32_t flags, bitnet_stream_t stream) {
  if (!float_type(x_dtype) || !float_type(y_dtype) || (flags & ~BITNET_FLAG_WEIGHTS_STATIC) != 0)
    return BITNET_ERR_INVALID_ARG;
  if (M < 0 || N < 0 || M > kMaxCount || N > kMaxCount || K <= 0) return BITNET_ERR_INVALID_ARG;
  if ((group != 32 && group != 64 && group != 128) || K % group != 0 || K > kMaxK)
    return BITNET_ERR_UNSUPPORTED_SHAPE;
  if (M == 0 || N == 0) return BITNET_OK;
  if (X == nullptr || packed == nullptr || scales == nullptr || Y == nullptr) return BITNET_ERR_INVALID_ARG;
  if (!aligned(X, 16) || !aligned(packed, 16) || !aligned(Y, 16) || !aligned(scales, 16))
    return BITNET_ERR_MISALIGNED;
  if (overlap(X, static_cast<uint64_t>(M) * K * float_size(x_dtype), Y,
              static_cast<uint64_t>(M) * N * float_size(y_dtype)))
    return BITNET_ERR_INVALID_ARG;
  if (M > 8 * 65535) return BITNET_ERR_UNSUPPORTED_SHAPE;
  LaunchCtx ctx;
  if (const int st = launch_ctx_status(stream, &ctx)) return static_cast<bitnet_status>(st);
  return from_cuda(launch_w4(X, x_dtype, packed, static_cast<const uint16_t *>(scales), M, N, K, group, Y, y_dtype,
                             (flags & BITNET_FLAG_WEIGHTS_STATIC) != 0, ctx));
}

bitnet_status bitnet_token_logprobs(const void *logits, bitnet_dtype dtype, int64_t M, int64_t V, int64_t stride,
                                    const int64_t *tokens, int32_t top, float *logprob, float *entropy,
                                    int64_t *top_ids, float *top_logprobs, bitnet_stream_t stream) {
  if (!float_type(dtype) || M < 0 || M > kMaxCount || V < 1 || V > kMaxCount || top < 0 || top > V)
    return BITNET_ERR_INVALID_ARG;
  if (top > BITNET_LOGPROBS_MAX_TOP || M > kMaxCount / 8) return BITNET_ERR_UNSUPPORTED_SHAPE;
  if (M == 0) return BITNET_OK;
  if (logits == nullptr || tokens == nullptr || logprob == nullptr || entropy == nullptr ||
      (top > 0 && (top_ids == nullptr || top_logprobs == nullptr)))
    return BITNET_ERR_INVALID_ARG;
  if ((M > 1 && stride < V) || stride > (int64_t(1) << 40)) return BITNET_ERR_INVALID_ARG;
  if (!aligned(logits, static_cast<uintptr_t>(float_size(dtype))) || !aligned(tokens, 8) || !aligned(logprob, 4) ||
      !aligned(entropy, 4) || !aligned(top_ids, 8) || !aligned(top_logprobs, 4))
    return BITNET_ERR_MISALIGNED;
  LaunchCtx ctx;
  if (const int st = launch_ctx_status(stream, &ctx)) return static_cast<bitnet_status>(st);
  return from_cuda(launch_token_logprobs(logits, dtype, M, V, stride, tokens, top, logprob, entropy, top_ids,
                                         top_logprobs, ctx));
}

}  // extern "C"
