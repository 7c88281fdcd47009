// kv_append.cu -- writes new keys and values into the 8-bit paged cache.
//
// For one page and head let a be the largest |x| over the rows that the call
// writes there and d_old the page's scale if it already holds older rows of
// the sequence (else 0).  Then, every operation one fp32 rounding,
//   d = max(d_old, a / 127), 0 if that is below 2^-60;  r = d > 0 ? 1 / d : 0,
//   code = clamp(round_half_away(x * r), -127, 127)        for the new rows,
//   code <- round_half_away(code * (d_old * r))            for the other rows
// of a page that holds older ones when d > d_old (they keep their codes
// otherwise).  |x| * r exceeds 127 by
// at most two roundings of 2^-24 each, far from 127.5, so the clamp never
// changes a code; |code| * (d_old * r) <= 127 likewise.
//
// One CTA owns one (page, head) of K or of V: the scale and the older codes
// have one writer, and the result does not depend on any order.  The new rows
// are read once, in 8-element chunks kept in registers between the maximum
// and the rounding.  Bound by latency: for single tokens by three dependent
// loads (length, page, scale): 64 bf16 tokens of 5 heads 2.7 us; for a page of
// a prompt by one load of its rows and the rounding of each value (8
// instructions): 3 prompts of up to 2011 tokens (22 MB) 13.0 us, 1.7 TB/s.
#include "common.cuh"
#include "internal.h"

namespace bitnet {
namespace {

constexpr int kMaxThreads = 256;
constexpr int kMaxChunks = 8;    // 8-element chunks per thread: 128 x 128 values / 256 threads

struct AppendParams {
  KvCache cache;
  KvBatch batch;
  const void *x[2];      // K, V
  int64_t stride[2];     // elements between tokens
  int tiles;             // CTAs per sequence (each strides over its pages)
  int *status;
};

template <int KIND>
__device__ __forceinline__ void load8(const void *base, int64_t at, float (&v)[8]) {
  if (KIND == kF32) {
    const float4 *p = reinterpret_cast<const float4 *>(static_cast<const float *>(base) + at);
    const float4 a = __ldcg(p), b = __ldcg(p + 1);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
    const uint4 u = __ldcg(reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(base) + at));
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
}

// The largest value over the CTA (all values >= 0), returned to every thread.
__device__ __forceinline__ float block_max(float v, float *red) {
  const unsigned m = __reduce_max_sync(0xffffffffu, __float_as_uint(v));
  const int warps = blockDim.x >> 5;
  if (warps == 1) return __uint_as_float(m);
  __syncthreads();  // the last use of red is over
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = __uint_as_float(m);
  __syncthreads();
  float r = red[0];
  for (int w = 1; w < warps; ++w) r = fmaxf(r, red[w]);
  return r;
}

template <int KIND>
__global__ void __launch_bounds__(kMaxThreads) kv_append_kernel(const AppendParams p) {
  __shared__ float red[kMaxThreads / 32];
  pdl_wait();
  pdl_launch_dependents();
  const int P = p.cache.page_tokens, D = p.cache.head_dim, H = p.cache.heads;
  const int page_shift = 31 - __clz(P), row_shift = 28 - __clz(D);  // D / 8 chunks per row
  const int b = blockIdx.x / static_cast<unsigned>(p.tiles);
  const int which = blockIdx.y & 1, h = blockIdx.y >> 1;
  // (positions and rows fit 32 bits)
  const int len = p.batch.lens[b];
  int r0 = b, r1 = b + 1;
  if (p.batch.offsets != nullptr) {
    r0 = p.batch.offsets[b];
    r1 = p.batch.offsets[b + 1];
  }
  const bool lead = threadIdx.x == 0 && blockIdx.y == 0 && blockIdx.x % p.tiles == 0;
  if (r0 < 0 || r1 > p.batch.T || r1 < r0 || len < r1 - r0 || len > p.batch.max_pages * P) {
    if (lead) record_status(p.status, kStatusRange);
    return;  // rows, or positions, that do not exist: nothing of the sequence is written
  }
  if (r1 == r0) return;
  const int first = len - (r1 - r0);  // position of row r0
  int8_t *codes = which ? p.cache.v_codes : p.cache.k_codes;
  float *scales = which ? p.cache.v_scales : p.cache.k_scales;
  const void *x = p.x[which];
  const int64_t stride = p.stride[which];
  const int *table = p.batch.pages + static_cast<int64_t>(b) * p.batch.max_pages;

  for (int i = (first >> page_shift) + static_cast<int>(blockIdx.x - b * static_cast<unsigned>(p.tiles)); i <= (len - 1) >> page_shift;
       i += p.tiles) {
    const int64_t page = table[i];
    if (page < 0 || page >= p.cache.pages) {
      if (threadIdx.x == 0) record_status(p.status, kStatusRange);
      continue;
    }
    const int lo = first > i * P ? first : i * P;             // the page's new positions
    const int hi = len - i * P < P ? len : (i + 1) * P;
    const int older = lo - i * P;
    const int chunks = (hi - lo) << row_shift;
    const float was = older > 0 ? scales[page * H + h] : 0.0f;
    const int64_t base = static_cast<int64_t>(r0 + (lo - first)) * stride + h * D;
    int8_t *out = codes + ((page * H + h) * P + older) * D;

    float v[kMaxChunks][8];
    float peak = 0.0f;
#pragma unroll
    for (int j = 0; j < kMaxChunks; ++j) {
      const int c = threadIdx.x + j * blockDim.x;
      if (c < chunks) {
        load8<KIND>(x, base + (c >> row_shift) * stride + ((c << 3) & (D - 1)), v[j]);
#pragma unroll
        for (int e = 0; e < 8; ++e) peak = fmaxf(peak, fabsf(v[j][e]));
      }
    }
    // a tile of more chunks than the CTA holds in registers (its launch was
    // told of fewer new tokens): the rest is read twice
    for (int c = threadIdx.x + kMaxChunks * blockDim.x; c < chunks; c += blockDim.x) {
      float w[8];
      load8<KIND>(x, base + (c >> row_shift) * stride + ((c << 3) & (D - 1)), w);
#pragma unroll
      for (int e = 0; e < 8; ++e) peak = fmaxf(peak, fabsf(w[e]));
    }
    peak = block_max(peak, red);
    float d = fmaxf(was, __fdiv_rn(peak, 127.0f));
    if (d < kKvMinScale) d = 0.0f;
    const float r = d > 0.0f ? __fdiv_rn(1.0f, d) : 0.0f;
    if (older > 0 && d > was) {
      const float f = __fmul_rn(was, r);
      uint32_t *w = reinterpret_cast<uint32_t *>(codes + (page * H + h) * P * D);
      const int skip = (hi - lo) * D / 4;  // the new rows
      for (int i = threadIdx.x; i < P * D / 4 - skip; i += blockDim.x) {
        const int c = i < older * D / 4 ? i : i + skip;
        const uint32_t u = w[c];
        int q[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          q[e] = quant_i8(static_cast<float>(static_cast<int8_t>(u >> (8 * e))), f);
        w[c] = pack4(q[0], q[1], q[2], q[3]);
      }
    }
    auto store = [&](int c, const float (&a)[8]) {
      int q[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) q[e] = quant_i8(a[e], r);
      *reinterpret_cast<uint2 *>(out + 8 * c) =
          make_uint2(pack4(q[0], q[1], q[2], q[3]), pack4(q[4], q[5], q[6], q[7]));
    };
#pragma unroll
    for (int j = 0; j < kMaxChunks; ++j) {
      const int c = threadIdx.x + j * blockDim.x;
      if (c < chunks) store(c, v[j]);
    }
    for (int c = threadIdx.x + kMaxChunks * blockDim.x; c < chunks; c += blockDim.x) {
      float w[8];
      load8<KIND>(x, base + (c >> row_shift) * stride + ((c << 3) & (D - 1)), w);
      store(c, w);
    }
    if (threadIdx.x == 0) scales[page * H + h] = d;
  }
}

}  // namespace

cudaError_t launch_kv_append(const KvCache &cache, const void *K, const void *V, int kind,
                             int64_t k_stride, int64_t v_stride, const KvBatch &batch,
                             int64_t max_new, const LaunchCtx &ctx) {
  const int64_t P = cache.page_tokens;
  // pages that max_new rows can touch; a sequence with more strides over them
  const int64_t tiles = max_new <= 1 ? 1 : (max_new + P - 2) / P + 1;
  const int64_t chunks = (max_new < P ? max_new : P) * cache.head_dim / 8;
  const int64_t threads = chunks <= 32 ? 32 : (chunks + kMaxChunks / 2 - 1) / (kMaxChunks / 2);
  const unsigned block = static_cast<unsigned>(threads > kMaxThreads ? kMaxThreads : ceil_div(threads, 32) * 32);
  AppendParams p = {cache, batch, {K, V}, {k_stride, v_stride}, static_cast<int>(tiles), ctx.status};
  const dim3 grid(static_cast<unsigned>(batch.B * tiles), static_cast<unsigned>(2 * cache.heads));
  return kind == kF32 ? launch_k(kv_append_kernel<kF32>, grid, dim3(block), 0, ctx, p)
                      : launch_k(kv_append_kernel<kBF16>, grid, dim3(block), 0, ctx, p);
}

}  // namespace bitnet
