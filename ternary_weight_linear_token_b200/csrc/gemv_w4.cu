// gemv_w4.cu -- products with 4-bit weights and one scale per group of
// weights, for the layers that are not ternary (the output head), and their
// quantiser.
//
//   y[m][n] = sum over groups g of s[n][g] * sum_{k in g} x[m][k] * c[n][k]
// with codes c in -8..7 stored as c + 8 in four bits: a 32-bit word holds 8
// consecutive weights of a row, weight 2i + h at bits [16h + 4i, 16h + 4i + 4),
// so that (w >> 4i) & 0x000F000F are two neighbours in the halves of a
// register.  Under the bf16 exponent of 128 a nibble is 128 + (c + 8), one
// subtraction of 136 makes it c, exactly.
//
// The product is mma m16n8k16 with the weights as the A operand (16 output
// features) and the tokens as the N axis.  The order of the K axis is free,
// so a thread of a quad takes a quarter of the group: its words' halves are
// its A fragments, and the 8 matching activations, 16 contiguous bytes of
// the row, its B fragments.  Sums are fp32: inside a group by the tensor
// core, over groups after the scale.  fp32 activations are split beforehand
// into three bf16 terms that add up to 24 bits (a kernel of its own, into the
// workspace), each with its own product into the same sums.
#include "common.cuh"
#include "internal.h"

namespace bitnet {
namespace {

constexpr int kWarps = 8;
constexpr int kRows = 16;  // features per CTA

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Weights 2i and 2i + 1 of a word as two bf16.
__device__ __forceinline__ uint32_t two_codes(uint32_t w, int i) {
  const uint32_t x = ((w >> (4 * i)) & 0x000F000Fu) | 0x43004300u, bias = 0x43084308u;  // 136, twice
  const __nv_bfloat162 v = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&x),
                                   *reinterpret_cast<const __nv_bfloat162 *>(&bias));
  return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ float bf16_value(uint16_t b) { return __uint_as_float(static_cast<uint32_t>(b) << 16); }

// ------------------------------------------------------------ quantiser
// s = bf16(max |w| / 7) of the group (0 below 2^-60), r = 1 / s,
// c = clamp(round_half_away(w * r), -8, 7).  A thread takes the 8 weights of
// one word, group / 8 neighbouring threads a group.
__device__ __forceinline__ int quant_i4(float w, float r) {
  int c = quant_i8(w, r);
  return c < -8 ? -8 : (c > 7 ? 7 : c);
}
template <int KIND, int G>
__global__ void __launch_bounds__(256) quantize_w4_kernel(const void *W, int64_t words,
                                                          uint32_t *packed, uint16_t *scales) {
  pdl_wait();
  pdl_launch_dependents();
  // whole warps: the last one's spare threads shuffle zeros
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
       i - (threadIdx.x & 31) < words; i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    float v[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    if (i < words) {
      if (KIND == kF32) {
        const float4 *p = static_cast<const float4 *>(W) + 2 * i;
        const float4 a = __ldcs(p), b = __ldcs(p + 1);
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
      } else {
        const uint4 u = __ldcs(static_cast<const uint4 *>(W) + i);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          v[2 * e] = __uint_as_float(w[e] << 16);
          v[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
        }
      }
    }
    float peak = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) peak = fmaxf(peak, fabsf(v[e]));
#pragma unroll
    for (int o = 1; o < G / 8; o <<= 1) peak = fmaxf(peak, __shfl_xor_sync(0xffffffffu, peak, o));
    __nv_bfloat16 sb = __float2bfloat16_rn(__fdiv_rn(peak, 7.0f));
    if (__bfloat162float(sb) < kKvMinScale) sb = __float2bfloat16_rn(0.0f);
    const float s = __bfloat162float(sb), r = s > 0.0f ? __fdiv_rn(1.0f, s) : 0.0f;
    uint32_t word = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e)
      word |= static_cast<uint32_t>(quant_i4(v[e], r) + 8) << (16 * (e & 1) + 4 * (e >> 1));
    if (i < words) {
      packed[i] = word;
      if (i % (G / 8) == 0) scales[i / (G / 8)] = __bfloat16_as_ushort(sb);
    }
  }
}

// fp32 activations as three bf16 terms, [3][M * K]: each term is the nearest
// bf16 to what the ones before leave, so the three hold 24 bits.
__global__ void __launch_bounds__(256) split_terms_kernel(const float *X, __nv_bfloat16 *out, int64_t n) {
  pdl_wait();
  pdl_launch_dependents();
  for (int64_t i = 4 * (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x); i < n;
       i += 4 * static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const float4 v = *reinterpret_cast<const float4 *>(X + i);
    float x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int t = 0; t < 3; ++t) {
      __nv_bfloat16 h[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        h[e] = __float2bfloat16_rn(x[e]);
        const float left = __fsub_rn(x[e], __bfloat162float(h[e]));
        // an infinity (or a value that rounds to one) is its first term alone
        x[e] = isfinite(__bfloat162float(h[e])) ? left : 0.0f;
      }
      *reinterpret_cast<uint2 *>(out + t * n + i) = *reinterpret_cast<const uint2 *>(h);
    }
  }
}

// ------------------------------------------------------------ product
struct W4Params {
  const __nv_bfloat16 *x;  // [TERMS][M][K]
  const uint8_t *packed;
  const uint16_t *scales;
  void *y;
  int64_t M, N, K;
};

// A CTA: 16 features, 8 * NT tokens, every warp every 8th group.
template <int G, int NT, int TERMS, int YK>
__global__ void __launch_bounds__(kWarps * 32) w4_kernel(const W4Params p) {
  constexpr int kWords = G / 32;  // words per thread, row and group
  __shared__ float part[kWarps][kRows][8 * NT + 1];
  pdl_wait();
  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * kRows;
  const int64_t m0 = static_cast<int64_t>(blockIdx.y) * 8 * NT;
  const int groups = static_cast<int>(p.K / G);
  // rows and tokens past the end read the last one and are not stored
  const int64_t na = n0 + g < p.N ? n0 + g : p.N - 1, nb = n0 + g + 8 < p.N ? n0 + g + 8 : p.N - 1;
  const uint8_t *wa = p.packed + na * (p.K / 2) + t * (G / 8), *wb = p.packed + nb * (p.K / 2) + t * (G / 8);
  const __nv_bfloat16 *xr[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int64_t m = m0 + 8 * j + g < p.M ? m0 + 8 * j + g : p.M - 1;
    xr[j] = p.x + m * p.K + t * (G / 4);
  }
  float y[NT][4];
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) y[j][e] = 0.0f;
  for (int q = warp; q < groups; q += kWarps) {
    uint32_t a[kWords], b[kWords];
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      a[i] = __ldg(reinterpret_cast<const uint32_t *>(wa + static_cast<int64_t>(q) * (G / 2)) + i);
      b[i] = __ldg(reinterpret_cast<const uint32_t *>(wb + static_cast<int64_t>(q) * (G / 2)) + i);
    }
    const float sa = bf16_value(__ldg(p.scales + na * groups + q)), sb = bf16_value(__ldg(p.scales + nb * groups + q));
    float c[NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) c[j][e] = 0.0f;
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      uint32_t fa[4], fb[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        fa[e] = two_codes(a[i], e);
        fb[e] = two_codes(b[i], e);
      }
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int k = TERMS - 1; k >= 0; --k) {
          const uint4 x = __ldg(reinterpret_cast<const uint4 *>(xr[j] + k * p.M * p.K + static_cast<int64_t>(q) * G) + i);
          mma_bf16(c[j], fa[0], fb[0], fa[1], fb[1], x.x, x.y);
          mma_bf16(c[j], fa[2], fb[2], fa[3], fb[3], x.z, x.w);
        }
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      y[j][0] = __fmaf_rn(sa, c[j][0], y[j][0]);
      y[j][1] = __fmaf_rn(sa, c[j][1], y[j][1]);
      y[j][2] = __fmaf_rn(sb, c[j][2], y[j][2]);
      y[j][3] = __fmaf_rn(sb, c[j][3], y[j][3]);
    }
  }
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    part[warp][g][8 * j + 2 * t] = y[j][0];
    part[warp][g][8 * j + 2 * t + 1] = y[j][1];
    part[warp][g + 8][8 * j + 2 * t] = y[j][2];
    part[warp][g + 8][8 * j + 2 * t + 1] = y[j][3];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < kRows * 8 * NT; i += kWarps * 32) {
    const int row = i % kRows, col = i / kRows;
    if (n0 + row >= p.N || m0 + col >= p.M) continue;
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v = __fadd_rn(v, part[w][row][col]);
    const int64_t o = (m0 + col) * p.N + n0 + row;
    if (YK == kF32)
      static_cast<float *>(p.y)[o] = v;
    else
      static_cast<__nv_bfloat16 *>(p.y)[o] = __float2bfloat16_rn(v);
  }
}

template <int G, int NT, int TERMS>
cudaError_t launch_y(const W4Params &p, int y_kind, const LaunchCtx &ctx) {
  const dim3 grid(static_cast<unsigned>(ceil_div(p.N, kRows)), static_cast<unsigned>(ceil_div(p.M, 8 * NT)));
  return y_kind == kF32 ? launch_k(w4_kernel<G, NT, TERMS, kF32>, grid, dim3(kWarps * 32), 0, ctx, p)
                        : launch_k(w4_kernel<G, NT, TERMS, kBF16>, grid, dim3(kWarps * 32), 0, ctx, p);
}
template <int G, int TERMS>
cudaError_t launch_nt(const W4Params &p, int y_kind, const LaunchCtx &ctx) {
  if (p.M <= 8) return launch_y<G, 1, TERMS>(p, y_kind, ctx);
  if (p.M <= 16) return launch_y<G, 2, TERMS>(p, y_kind, ctx);
  return launch_y<G, 4, TERMS>(p, y_kind, ctx);
}
template <int TERMS>
cudaError_t launch_g(const W4Params &p, int group, int y_kind, const LaunchCtx &ctx) {
  if (group == 128) return launch_nt<128, TERMS>(p, y_kind, ctx);
  if (group == 64) return launch_nt<64, TERMS>(p, y_kind, ctx);
  return launch_nt<32, TERMS>(p, y_kind, ctx);
}

template <int KIND, int G>
cudaError_t quantize(const void *W, int64_t words, uint8_t *packed, uint16_t *scales, const LaunchCtx &ctx) {
  int64_t blocks = ceil_div(words, 256);
  if (blocks > ctx.num_sms * 16) blocks = ctx.num_sms * 16;
  return launch_k(quantize_w4_kernel<KIND, G>, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, ctx, W, words,
                  reinterpret_cast<uint32_t *>(packed), scales);
}
template <int KIND>
cudaError_t quantize_g(const void *W, int64_t words, int group, uint8_t *packed, uint16_t *scales,
                       const LaunchCtx &ctx) {
  if (group == 128) return quantize<KIND, 128>(W, words, packed, scales, ctx);
  if (group == 64) return quantize<KIND, 64>(W, words, packed, scales, ctx);
  return quantize<KIND, 32>(W, words, packed, scales, ctx);
}

}  // namespace

cudaError_t launch_quantize_weights_w4(const void *W, int w_kind, int64_t N, int64_t K, int group,
                                       uint8_t *packed, uint16_t *scales, const LaunchCtx &ctx) {
  const int64_t words = N * (K / 8);
  return w_kind == kF32 ? quantize_g<kF32>(W, words, group, packed, scales, ctx)
                        : quantize_g<kBF16>(W, words, group, packed, scales, ctx);
}

size_t w4_workspace(int64_t M, int64_t N, int64_t K, int x_kind) {
  (void)N;
  return x_kind == kF32 ? (static_cast<size_t>(M) * K * 6 + 255) & ~size_t(255) : 0;
}

cudaError_t launch_w4(const void *X, int x_kind, const uint8_t *packed, const uint16_t *scales,
                      int64_t M, int64_t N, int64_t K, int group, void *Y, int y_kind,
                      void *workspace, bool weights_static, const LaunchCtx &ctx) {
  (void)weights_static;
  W4Params p = {static_cast<const __nv_bfloat16 *>(X), packed, scales, Y, M, N, K};
  if (x_kind != kF32) return launch_g<1>(p, group, y_kind, ctx);
  int64_t blocks = ceil_div(M * K, 1024);
  if (blocks > ctx.num_sms * 8) blocks = ctx.num_sms * 8;
  __nv_bfloat16 *terms = static_cast<__nv_bfloat16 *>(workspace);
  const cudaError_t e = launch_k(split_terms_kernel, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, ctx,
                                 static_cast<const float *>(X), terms, M * K);
  if (e != cudaSuccess) return e;
  p.x = terms;
  return launch_g<3>(p, group, y_kind, ctx);
}

}  // namespace bitnet
