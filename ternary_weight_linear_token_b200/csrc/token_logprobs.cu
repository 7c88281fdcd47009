// token_logprobs.cu -- log probability of a given token, entropy and the most
// probable tokens of each row of logits.
//
// With the row's maximum m: d_v = x_v - m, s = sum e^d, u = sum d e^d.  Then
//   log sum e^x = m + ln s,  logprob = (x_token - m) - ln s,
//   entropy = -sum p ln p = ln s - u / s.
// The maximum is taken away before anything is scaled, so rows of the type's
// lowest value lose nothing.
// One pass over the row: every thread keeps (m, s, u) of its chunks of 16
// bytes, following its own running maximum, and the chunk of its largest
// value.  The sums join over the CTA, then over the row's cluster of CTAs.
//
// The top k: a value's key is (its bits in an order that integers have,
// then the inverted index), so that keys are all different and equal values
// rank by the lower index.  The k-th largest of the threads' largest keys is
// a bound that at least k keys reach, and only the (at most k) threads whose
// largest key reaches it hold such keys: their chunks alone are read again
// (from L2), a lane per chunk.  Warps keep the best 32 keys sorted, one per
// lane, and join two such lists by a bitonic merge; CTAs of a cluster join
// theirs through distributed shared memory.
// 701 bf16 rows of 128256: 62 us with the top 5 (2.9 TB/s, 1.6 waves), 45 us
// without a selection, whose sorts and barriers have no loads in flight
// (counters: issue slots 58 %, ALU 42 %, exponentials 37 %, HBM 36 %); three
// CTAs per SM with batches of 2 chunks against two with batches of 4: 61
// against 69 us.  One fp32 row over 8 CTAs: 12.9 us with the top 20, 6.0
// without, latency.
#include "common.cuh"
#include "internal.h"
#include "pairs.cuh"

namespace bitnet {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;

struct LogprobParams {
  const void *x;
  int64_t M, V, stride;
  const int64_t *tokens;
  int top;
  float *logprob, *entropy;
  int64_t *top_ids;
  float *top_logprobs;
  int *status;
};

struct Sums {
  float m, s, u;
};
// x - m, at least -1e28 (e^d is 0 there, and so is d e^d, times any sum); NaN
// stays NaN.
__device__ __forceinline__ float below(float x, float m) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(__fsub_rn(x, m)), "f"(-1e28f));
  return y;
}
__device__ __forceinline__ float min3(float a, float b, float c) {
  float r;
  asm("min.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// The sums of two parts, at the larger maximum; the same whichever comes
// first.  (Equal maxima, infinite ones too, count as they are; a part without
// a maximum has s = 0, or NaN, which goes on.)
__device__ __forceinline__ Sums join(const Sums &a, const Sums &b) {
  const float m = fmaxf(a.m, b.m);
  const float da = a.m == m ? 0.0f : below(a.m, m), db = b.m == m ? 0.0f : below(b.m, m);
  const float fa = ex2(__fmul_rn(da, kLog2e)), fb = ex2(__fmul_rn(db, kLog2e));
  return {m, __fadd_rn(__fmul_rn(fa, a.s), __fmul_rn(fb, b.s)),
          __fadd_rn(__fmul_rn(fa, __fmaf_rn(da, a.s, a.u)), __fmul_rn(fb, __fmaf_rn(db, b.s, b.u)))};
}
// The sums of all lanes, in every lane.
__device__ __forceinline__ Sums join_lanes(Sums w) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const Sums b = {__shfl_xor_sync(0xffffffffu, w.m, o), __shfl_xor_sync(0xffffffffu, w.s, o),
                    __shfl_xor_sync(0xffffffffu, w.u, o)};
    w = join(w, b);
  }
  return w;
}

__device__ __forceinline__ uint64_t key_of(float x, uint32_t index) {
  if (x == 0.0f) x = 0.0f;  // -0 ranks as 0
  const uint32_t b = __float_as_uint(x);
  uint32_t o = (b & 0x80000000u) != 0 ? ~b : b | 0x80000000u;
  if (x != x) o = 0;  // NaN below everything
  return (static_cast<uint64_t>(o) << 32) | (0xFFFFFFFFu - index);
}
__device__ __forceinline__ float key_value(uint64_t key) {
  const uint32_t o = static_cast<uint32_t>(key >> 32);
  if (o == 0) return __uint_as_float(0x7FC00000u);
  return __uint_as_float((o & 0x80000000u) != 0 ? o & 0x7FFFFFFFu : ~o);
}

// One compare-exchange step of a sorting network over the lanes.
__device__ __forceinline__ uint64_t exchange(uint64_t a, int lane, int j, bool descending) {
  const uint64_t b = __shfl_xor_sync(0xffffffffu, a, j);
  const bool low = (lane & j) == 0;  // the lane that keeps the larger when descending
  return (a > b) == (low == descending) ? a : b;
}
__device__ __forceinline__ uint64_t sort32(uint64_t a, int lane) {
#pragma unroll
  for (int k = 2; k <= 32; k <<= 1)
#pragma unroll
    for (int j = k >> 1; j > 0; j >>= 1) a = exchange(a, lane, j, (lane & k) == 0);
  return a;
}
// The best 32 of two descending lists, descending.
__device__ __forceinline__ uint64_t merge32(uint64_t a, uint64_t b, int lane) {
  b = __shfl_sync(0xffffffffu, b, 31 - lane);
  a = a > b ? a : b;
#pragma unroll
  for (int j = 16; j > 0; j >>= 1) a = exchange(a, lane, j, true);
  return a;
}
// The best 32 of all warps' lists, in warp 0 (and in list[0..31]).
__device__ __forceinline__ uint64_t block_best(uint64_t a, uint64_t *list, int warp, int lane) {
#pragma unroll
  for (int half = kWarps / 2; half > 0; half >>= 1) {
    if (warp >= half && warp < 2 * half) list[(warp - half) * 32 + lane] = a;
    __syncthreads();
    if (warp < half) a = merge32(a, list[warp * 32 + lane], lane);
    __syncthreads();
  }
  if (warp == 0) list[lane] = a;
  __syncthreads();
  return a;
}

template <int KIND> struct Vec {
  static constexpr int kN = KIND == kF32 ? 4 : 8;
};
// The values of 16 bytes.
template <int KIND>
__device__ __forceinline__ void values_of(const uint4 &u, float *v) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (KIND == kF32) {
      v[e] = __uint_as_float(w[e]);
    } else {
      v[2 * e] = __uint_as_float(w[e] << 16);
      v[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
    }
  }
}
// Chunk c of the row: elements c * kN - skew + e, those outside [0, V) as
// -infinity.
template <int KIND>
__device__ __forceinline__ void load_chunk(const void *row, int64_t c, int skew, int64_t V,
                                           float (&v)[Vec<KIND>::kN]) {
  constexpr int N = Vec<KIND>::kN;
  const int64_t i0 = c * N - skew;
  if (i0 >= 0 && i0 + N <= V) {
    values_of<KIND>(__ldcg(reinterpret_cast<const uint4 *>(static_cast<const char *>(row) + i0 * (16 / N))), v);
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e) {
      v[e] = -INFINITY;
      if (i0 + e >= 0 && i0 + e < V)
        v[e] = KIND == kF32 ? static_cast<const float *>(row)[i0 + e]
                            : __bfloat162float(static_cast<const __nv_bfloat16 *>(row)[i0 + e]);
    }
  }
}

template <int KIND>
__global__ void __launch_bounds__(kThreads, 3) token_logprobs_kernel(const LogprobParams p) {
  constexpr int N = Vec<KIND>::kN;
  __shared__ Sums sums[kWarps];
  __shared__ uint64_t list[kWarps / 2 * 32];
  __shared__ int winners[32];
  __shared__ int n_winners;
  pdl_wait();
  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t ctas, rank;
  asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(ctas));
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  const int64_t m = blockIdx.x / ctas;
  const char *row = static_cast<const char *>(p.x) + m * p.stride * (KIND == kF32 ? 4 : 2);
  const int skew = static_cast<int>((reinterpret_cast<uintptr_t>(row) & 15) / (KIND == kF32 ? 4 : 2));
  const int64_t chunks = (p.V + skew + N - 1) / N;
  const int64_t c0 = chunks * rank / ctas, c1 = chunks * (rank + 1) / ctas;

  // ---- sums, and where the largest value is: kBatch chunks at a time,
  // kThreads apart, so that the maximum is looked at once for all of them
  Sums a = {-INFINITY, 0.0f, 0.0f};
  int64_t best_chunk = c0 + threadIdx.x;
  auto add = [&](const float *v, int count, int64_t c) {  // (count is a constant where it is called)
    float cm = fmaxf(v[0], v[1]), cl = fminf(v[0], v[1]);
#pragma unroll
    for (int e = 2; e < count; e += 2) {
      cm = max3(cm, v[e], v[e + 1]);
      cl = min3(cl, v[e], v[e + 1]);
    }
    if (cm > a.m) {
      best_chunk = c;
      if (a.m != -INFINITY) {
        const float d = below(a.m, cm), f = ex2(d * kLog2e);
        a.u = f * __fmaf_rn(d, a.s, a.u);
        a.s *= f;
      }
      a.m = cm;
    }
    // d = -infinity (a value of -infinity, or a finite one too far below the
    // maximum): d e^d counts as 0, by a lower limit for d
    if (cl - a.m == -INFINITY || a.m == -INFINITY) {
#pragma unroll
      for (int e = 0; e < count; ++e) {
        if (a.m == -INFINITY) {  // only -infinity so far, or NaN
          if (v[e] != v[e]) a.s = v[e];
        } else {
          const float d = below(v[e], a.m), x = ex2(__fmul_rn(d, kLog2e));
          a.s += x;
          a.u = __fmaf_rn(x, d, a.u);
        }
      }
      return;
    }
    const uint64_t minus_m = pair(-a.m, -a.m), log2e = pair(kLog2e, kLog2e);
    uint64_t s[2], u[2];
    s[0] = s[1] = u[0] = u[1] = pair(0.0f, 0.0f);
#pragma unroll
    for (int e = 0; e < count; e += 2) {
      const uint64_t d = add2(pair(v[e], v[e + 1]), minus_m);
      float t0, t1;
      unpair(mul2(d, log2e), t0, t1);
      const uint64_t x = pair(ex2(t0), ex2(t1));
      s[(e >> 1) & 1] = add2(s[(e >> 1) & 1], x);
      u[(e >> 1) & 1] = fma2(x, d, u[(e >> 1) & 1]);
    }
    float s0, s1;
    unpair(add2(s[0], s[1]), s0, s1);
    a.s += s0 + s1;
    unpair(add2(u[0], u[1]), s0, s1);
    a.u += s0 + s1;
  };
  constexpr int kBatch = 2;
  int64_t c = c0 + threadIdx.x;
  for (; c + (kBatch - 1) * kThreads < c1; c += kBatch * kThreads) {
    float v[kBatch * N];
    if (c > 0 && c + (kBatch - 1) * kThreads < chunks - 1) {  // whole chunks, all loads before the first use
      uint4 raw[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        raw[i] = __ldcg(reinterpret_cast<const uint4 *>(row - skew * (16 / N)) + c + i * kThreads);
#pragma unroll
      for (int i = 0; i < kBatch; ++i) values_of<KIND>(raw[i], &v[i * N]);
    } else {
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        load_chunk<KIND>(row, c + i * kThreads, skew, p.V, *reinterpret_cast<float(*)[N]>(&v[i * N]));
    }
    add(v, kBatch * N, c);
  }
  for (; c < c1; c += kThreads) {
    float v[N];
    load_chunk<KIND>(row, c, skew, p.V, v);
    add(v, N, c);
  }
  Sums w = a;
  w = join_lanes(w);
  if (lane == 0) sums[warp] = w;
  __syncthreads();
  if (warp == 0) {  // the CTA's
    w = lane < kWarps ? sums[lane] : Sums{-INFINITY, 0.0f, 0.0f};
    w = join_lanes(w);
    __syncwarp();
    if (lane == 0) sums[0] = w;
  }

  // ---- top k of this CTA's part
  uint64_t mine = 0;
  if (p.top > 0) {
    uint64_t key = 0;
    auto chunk_keys = [&](int64_t at, uint64_t (&k)[N]) {
      float v[N];
      load_chunk<KIND>(row, at, skew, p.V, v);
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const int64_t i = at * N - skew + e;
        k[e] = i >= 0 && i < p.V ? key_of(v[e], static_cast<uint32_t>(i)) : 0;
      }
    };
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int64_t at = best_chunk + i * kThreads;
      if (at < c1) {
        uint64_t k[N];
        chunk_keys(at, k);
#pragma unroll
        for (int e = 0; e < N; ++e) key = k[e] > key ? k[e] : key;
      }
    }
    if (threadIdx.x == 0) n_winners = 0;
    block_best(sort32(key, lane), list, warp, lane);
    const uint64_t bound = list[p.top - 1];
    if (key > 0 && key >= bound) winners[atomicAdd(&n_winners, 1)] = threadIdx.x;
    __syncthreads();
    const int n = n_winners;
    for (int i = warp; i < n; i += kWarps) {  // order does not matter: keys are all different
      const int64_t first = c0 + winners[i];
      for (int64_t at = first; at < c1; at += 32 * kThreads) {
        const int64_t at_lane = at + static_cast<int64_t>(lane) * kThreads;
        uint64_t k[N];
#pragma unroll
        for (int e = 0; e < N; ++e) k[e] = 0;
        if (at_lane < c1) chunk_keys(at_lane, k);
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const bool in = k[e] > 0 && k[e] >= bound;
          if (__any_sync(0xffffffffu, in)) mine = merge32(mine, sort32(in ? k[e] : 0, lane), lane);
        }
      }
    }
    mine = block_best(mine, list, warp, lane);
  }
  __syncthreads();
  if (ctas > 1) cluster_sync();
  if (rank != 0) {
    cluster_sync();  // rank 0 reads this CTA's lists and sums until here
    return;
  }
  if (warp == 0) {
    Sums all = {-INFINITY, 0.0f, 0.0f};
    if (lane < static_cast<int>(ctas)) {
      const uint32_t at = mapa_shared(sums, static_cast<uint32_t>(lane));
      asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(all.m) : "r"(at) : "memory");
      asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(all.s) : "r"(at + 4) : "memory");
      asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(all.u) : "r"(at + 8) : "memory");
    }
    all = join_lanes(all);
    if (p.top > 0) {
      for (uint32_t r = 1; r < ctas; ++r) {
        uint64_t b;
        asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(b) : "r"(mapa_shared(list, r) + lane * 8) : "memory");
        mine = merge32(mine, b, lane);
      }
    }
    const bool none = all.s == 0.0f;  // every logit is -infinity
    const float ln_s = none ? 0.0f : logf(all.s);
    const float from = none ? 0.0f : all.m;
    if (lane == 0) {
      p.entropy[m] = none ? 0.0f : ln_s - __fdiv_rn(all.u, all.s);
      const int64_t token = p.tokens[m];
      float lp = 0.0f;  // a negative token asks for none
      if (token >= p.V) {
        record_status(p.status, kStatusRange);
        lp = __uint_as_float(0x7FC00000u);
      } else if (token >= 0) {
        const float x = KIND == kF32 ? reinterpret_cast<const float *>(row)[token]
                                     : __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(row)[token]);
        lp = (x - from) - ln_s;
      }
      p.logprob[m] = lp;
    }
    if (lane < p.top) {
      p.top_ids[m * p.top + lane] = 0xFFFFFFFFu - static_cast<uint32_t>(mine);
      p.top_logprobs[m * p.top + lane] = (key_value(mine) - from) - ln_s;
    }
  }
  if (ctas > 1) cluster_sync();
}

}  // namespace

cudaError_t launch_token_logprobs(const void *X, int x_kind, int64_t M, int64_t V, int64_t stride,
                                  const int64_t *tokens, int top, float *logprob, float *entropy,
                                  int64_t *top_ids, float *top_logprobs, const LaunchCtx &ctx) {
  const LogprobParams p = {X, M, V, stride, tokens, top, logprob, entropy, top_ids, top_logprobs, ctx.status};
  // few rows: up to 8 CTAs each, while every thread has a chunk
  const int64_t per = kThreads * (x_kind == kF32 ? 4 : 8);
  unsigned ctas = 1;
  while (ctas < 8 && M * ctas * 2 <= 2 * ctx.num_sms && V >= 2 * ctas * per) ctas *= 2;
  const dim3 grid(static_cast<unsigned>(M * ctas));
  return x_kind == kF32 ? launch_k_cluster(token_logprobs_kernel<kF32>, grid, dim3(kThreads), 0, ctas, ctx, p)
                        : launch_k_cluster(token_logprobs_kernel<kBF16>, grid, dim3(kThreads), 0, ctas, ctx, p);
}

}  // namespace bitnet
