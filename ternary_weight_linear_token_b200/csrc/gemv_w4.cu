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
// The products are mma m16n8k16 with the weights as the A operand (16 output
// features) and the tokens as the N axis.  The order of the K axis is free,
// so a thread of a quad takes a quarter of the group: its words' halves are
// its A fragments, and the 8 matching activations, 16 contiguous bytes of
// the row, its B fragments.  Sums are fp32: inside a group by the tensor
// core, over groups after the scale.  fp32 activations are split into three
// bf16 terms that add up to 24 bits, each with its own product into the same
// sums.
//   few tokens (up to 8, activations in shared memory whole): w4_few_kernel;
//     128256 x 2560, one bf16 token: 48 us, 3.5 TB/s
//   more: w4_many_kernel; 23 fp32 tokens, 6912 -> 2560: 25 us, by its barriers
//     and shared-memory reads of three terms (counters: tensor pipe 28 %,
//     issue slots 26 %, 160 CTAs)
// The quantiser: 128256 x 2560 bf16 295 us (127 at the HBM rate), fp32 296 (227).
#include <atomic>

#include "common.cuh"
#include "internal.h"

namespace bitnet {
namespace {

constexpr int kRows = 16;  // features of an MMA tile

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

// ------------------------------------------------------------ products
struct W4Params {
  const void *x;           // [M][K] bf16 or fp32
  const uint8_t *packed;
  const uint16_t *scales;
  void *y;
  int64_t M, N, K;
  int tiles;               // of output features
  bool weights_static;
  int *status;
};

// 8 activations as they lie in memory, ...
template <int TERMS> struct Raw {
  uint4 v[TERMS == 1 ? 1 : 2];
  __device__ __forceinline__ void load(const void *x, int64_t at) {
    const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(x) + at * (TERMS == 1 ? 2 : 4));
    v[0] = __ldcg(p);
    if (TERMS != 1) v[TERMS == 1 ? 0 : 1] = __ldcg(p + 1);
  }
};
// ... and as TERMS rows of bf16: themselves, or 8 bits of the fp32 value each,
// cut off (rounding would take the largest ones to infinity).
template <int TERMS>
__device__ __forceinline__ void split(const Raw<TERMS> &raw, uint4 (&out)[TERMS]) {
  if (TERMS == 1) {
    out[0] = raw.v[0];
  } else {
    const uint4 a = raw.v[0], b = raw.v[TERMS == 1 ? 0 : 1];
    float v[8] = {__uint_as_float(a.x), __uint_as_float(a.y), __uint_as_float(a.z), __uint_as_float(a.w),
                  __uint_as_float(b.x), __uint_as_float(b.y), __uint_as_float(b.z), __uint_as_float(b.w)};
#pragma unroll
    for (int t = 0; t < TERMS; ++t) {
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t lo = __float_as_uint(v[2 * e]), hi = __float_as_uint(v[2 * e + 1]);
        w[e] = __byte_perm(lo, hi, 0x7632);
        v[2 * e] = __fsub_rn(v[2 * e], __uint_as_float(lo & 0xFFFF0000u));
        v[2 * e + 1] = __fsub_rn(v[2 * e + 1], __uint_as_float(hi & 0xFFFF0000u));
      }
      out[t] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

template <int YK> __device__ __forceinline__ void store_y(void *y, int64_t at, float v) {
  if (YK == kF32)
    static_cast<float *>(y)[at] = v;
  else
    static_cast<__nv_bfloat16 *>(y)[at] = __float2bfloat16_rn(v);
}

// A row's words of one group: thread t of a quad has a quarter.
template <int G> struct Words {
  static constexpr int kN = G / 32;
  uint32_t w[kN];
  __device__ __forceinline__ void load(const uint8_t *p) {
    if (kN == 4) {
      const uint4 v = *reinterpret_cast<const uint4 *>(p);
      w[0] = v.x; w[1 % kN] = v.y; w[2 % kN] = v.z; w[3 % kN] = v.w;
    } else if (kN == 2) {
      const uint2 v = *reinterpret_cast<const uint2 *>(p);
      w[0] = v.x; w[1 % kN] = v.y;
    } else {
      w[0] = *reinterpret_cast<const uint32_t *>(p);
    }
  }
};

// Few tokens.  A tile of 16 features is contiguous in memory,
// and so are its scales: a CTA of 4 warps goes over tiles whose bulk copies
// are a tile ahead in shared memory (two stages: a third costs a CTA per SM
// and time, 55 against 49 us for 128256 x 2560), each warp over every 4th
// group; the warps' sums meet in shared memory, one barrier per tile, which
// also hands the stage back.  No unit is full (counters: shared memory 64 %,
// ALU 60 %, issue slots 56 %, HBM 39 %, 10 warps an SM).  Codes are made exact
// before the products: leaving out that subtraction, 4 of 11 instructions per
// 8 weights, and taking 136 times the group's activation sum away afterwards
// gains nothing (49.5 against 48.3 us), and its error grows with the largest
// activation, whatever that one's code is.
constexpr int kFewWarps = 4, kFewStages = 2;
constexpr size_t kFewSmem = 112 * 1024;  // of a CTA, two per SM
struct FewPlan {
  int x_bytes, w_bytes, stage_bytes, stages;
  size_t smem;
};
// false: the tiles are too long
inline bool few_plan(int64_t M, int64_t K, int group, int terms, FewPlan *f) {
  const int64_t groups = K / group;
  const int64_t x = terms * (M + 1) * (K + 8) * 2, w = 8 * K, s = 32 * groups;
  const int64_t x16 = (x + 15) / 16 * 16, stage = w + s;
  if (x16 + kFewStages * stage + 64 > static_cast<int64_t>(kFewSmem)) return false;
  f->x_bytes = static_cast<int>(x16);
  f->w_bytes = static_cast<int>(w);
  f->stage_bytes = static_cast<int>(stage);
  f->stages = kFewStages;
  f->smem = static_cast<size_t>(x16 + kFewStages * stage + 64);
  return true;
}

template <int G, int TERMS, int YK>
__global__ void __launch_bounds__(kFewWarps * 32) w4_few_kernel(const W4Params p, const FewPlan f) {
  constexpr int kWords = G / 32;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float part[2][kFewWarps][kRows][9];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int K = static_cast<int>(p.K), groups = K / G, M = static_cast<int>(p.M), pitch = K + 8;
  __nv_bfloat16 *xs = reinterpret_cast<__nv_bfloat16 *>(smem);       // [TERMS][M + 1][pitch], the last row 0
  uint8_t *ring = smem + f.x_bytes;
  uint64_t *full = reinterpret_cast<uint64_t *>(ring + f.stages * f.stage_bytes);
  if (threadIdx.x < f.stages) mbar_init(&full[threadIdx.x], 1);
  fence_barrier_init();
  __syncthreads();
  // (thread 0) the tile's rows and scales; the last tile's may be fewer, and
  // then the scales' bytes no multiple of 16: everybody reads those itself
  auto copy = [&](int tile, int stage) {
    const int64_t n0 = static_cast<int64_t>(tile) * kRows;
    const int rows = p.N - n0 < kRows ? static_cast<int>(p.N - n0) : kRows;
    uint8_t *to = ring + stage * f.stage_bytes;
    const uint32_t w = rows * (K / 2), s = rows == kRows ? 32 * groups : 0;
    mbar_arrive_expect_tx(&full[stage], w + s);
    bulk_g2s(to, p.packed + n0 * (K / 2), w, &full[stage]);
    if (s > 0) bulk_g2s(to + f.w_bytes, p.scales + n0 * groups, s, &full[stage]);
  };
  auto start = [&]() {
    if (threadIdx.x == 0)
      for (int i = 0; i < f.stages; ++i) {
        const int64_t tile = blockIdx.x + static_cast<int64_t>(i) * gridDim.x;
        if (tile < p.tiles) copy(static_cast<int>(tile), i);
      }
  };
  if (p.weights_static) start();
  pdl_wait();
  pdl_launch_dependents();
  if (!p.weights_static) start();
  for (int i = threadIdx.x; i < TERMS * (K / 8); i += kFewWarps * 32) {
    const int k = i / (K / 8), c = i - k * (K / 8);
    *reinterpret_cast<uint4 *>(xs + (k * (M + 1) + M) * pitch + c * 8) = make_uint4(0, 0, 0, 0);
  }
  for (int i = threadIdx.x; i < M * (K / 8); i += kFewWarps * 32) {
    const int m = i / (K / 8), c = i - m * (K / 8);
    Raw<TERMS> raw;
    raw.load(p.x, static_cast<int64_t>(m) * K + c * 8);
    uint4 v[TERMS];
    split<TERMS>(raw, v);
#pragma unroll
    for (int k = 0; k < TERMS; ++k) *reinterpret_cast<uint4 *>(xs + (k * (M + 1) + m) * pitch + c * 8) = v[k];
  }
  __syncthreads();

  const __nv_bfloat16 *x_lane = xs + (g < M ? g : M) * pitch + t * (G / 4);
  int stage = 0, buffer = 0;
  uint32_t phase = 0;
  for (int tile = blockIdx.x; tile < p.tiles; tile += gridDim.x) {
    const bool ok = mbar_wait(&full[stage], phase, nullptr);  // (recorded below)
    if (!ok) record_status(p.status, kStatusTimeout);
    const uint8_t *w = ring + stage * f.stage_bytes + g * (K / 2) + t * (G / 8);
    const uint16_t *s = reinterpret_cast<const uint16_t *>(ring + stage * f.stage_bytes + f.w_bytes) + g * groups;
    int s8 = 8 * groups;  // to the scales of row g + 8
    if (p.N - static_cast<int64_t>(tile) * kRows < kRows) {
      const int64_t na = static_cast<int64_t>(tile) * kRows + g;
      s = p.scales + (na < p.N ? na : p.N - 1) * groups;
      s8 = static_cast<int>((na + 8 < p.N ? na + 8 : p.N - 1) - (na < p.N ? na : p.N - 1)) * groups;
    }
    float y[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
    for (int q = warp; q < groups; q += kFewWarps) {
      Words<G> wa, wb;
      wa.load(w + q * (G / 2));
      wb.load(w + q * (G / 2) + 4 * K);
      float c[2][4];  // two chains of sums
#pragma unroll
      for (int e = 0; e < 4; ++e) c[0][e] = c[1][e] = 0.0f;
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        uint32_t fa[4], fb[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          fa[e] = two_codes(wa.w[i], e);
          fb[e] = two_codes(wb.w[i], e);
        }
#pragma unroll
        for (int k = TERMS - 1; k >= 0; --k) {
          const uint4 x = *reinterpret_cast<const uint4 *>(x_lane + k * (M + 1) * pitch + q * G + i * 8);
          mma_bf16(c[0], fa[0], fb[0], fa[1], fb[1], x.x, x.y);
          mma_bf16(c[1], fa[2], fb[2], fa[3], fb[3], x.z, x.w);
        }
      }
      const float s0 = bf16_value(s[q]), s1 = bf16_value(s[q + s8]);
      y[0] = __fmaf_rn(s0, c[0][0] + c[1][0], y[0]);
      y[1] = __fmaf_rn(s0, c[0][1] + c[1][1], y[1]);
      y[2] = __fmaf_rn(s1, c[0][2] + c[1][2], y[2]);
      y[3] = __fmaf_rn(s1, c[0][3] + c[1][3], y[3]);
    }
    float (&mine)[kRows][9] = part[buffer][warp];
    mine[g][2 * t] = y[0];
    mine[g][2 * t + 1] = y[1];
    mine[g + 8][2 * t] = y[2];
    mine[g + 8][2 * t + 1] = y[3];
    if (__syncthreads_or(!ok)) {  // nothing that gave up is stored; the copies under way end first (with a limit)
      if (threadIdx.x == 0)
        for (int i = 0; i < f.stages && tile + static_cast<int64_t>(i) * gridDim.x < p.tiles; ++i)
          mbar_wait(&full[(stage + i) % f.stages], stage + i < f.stages ? phase : phase ^ 1u, nullptr);
      return;
    }
    if (threadIdx.x == 0 && tile + static_cast<int64_t>(f.stages) * gridDim.x < p.tiles)
      copy(tile + f.stages * static_cast<int>(gridDim.x), stage);
    const int row = threadIdx.x % kRows, col = threadIdx.x / kRows;
    const int64_t n = static_cast<int64_t>(tile) * kRows + row;
    if (n < p.N && col < M) {
      float v = 0.0f;
#pragma unroll
      for (int e = 0; e < kFewWarps; ++e) v += part[buffer][e][row][col];
      store_y<YK>(p.y, col * p.N + n, v);
    }
    buffer ^= 1;
    if (++stage == f.stages) {
      stage = 0;
      phase ^= 1u;
    }
  }
}

// More tokens.  A CTA of 8 warps takes 128 features (a warp 16) and 8 * NT
// tokens over a slice of K, in chunks of 128 weights: the chunk's activations
// (terms) in shared memory, two buffers, the next ones and the next weights on
// their way in registers.  The CTAs of a cluster take the slices of K and add
// their sums up through distributed shared memory, in slice order.
constexpr int kManyWarps = 8;
constexpr int kManyRows = kManyWarps * kRows;
constexpr int kChunkK = 128, kChunkPitch = kChunkK + 8;
template <int NT, int TERMS> constexpr size_t many_smem() {
  return 2 * static_cast<size_t>(TERMS) * 8 * NT * kChunkPitch * 2 > sizeof(float) * kManyRows * (8 * NT + 1)
             ? 2 * static_cast<size_t>(TERMS) * 8 * NT * kChunkPitch * 2
             : sizeof(float) * kManyRows * (8 * NT + 1);
}

template <int G, int NT, int TERMS, int YK>
__global__ void __launch_bounds__(kManyWarps * 32, 2) w4_many_kernel(const W4Params p) {
  constexpr int kWords = G / 32, kGroups = kChunkK / G;
  constexpr int kUnits = 8 * NT * (kChunkK / 8);                       // 8 activations each
  constexpr int kPer = (kUnits + kManyWarps * 32 - 1) / (kManyWarps * 32);
  extern __shared__ __align__(16) uint8_t smem[];
  __nv_bfloat16 *xs = reinterpret_cast<__nv_bfloat16 *>(smem);         // [2][TERMS][8 NT][pitch]
  constexpr int kBuffer = TERMS * 8 * NT * kChunkPitch;
  float *part = reinterpret_cast<float *>(smem);                       // [128][8 NT + 1], afterwards
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  uint32_t slices;
  asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(slices));
  const uint32_t slice = cluster_ctarank();
  const int64_t n0 = static_cast<int64_t>(blockIdx.x / slices) * kManyRows + warp * kRows;
  const int64_t m0 = static_cast<int64_t>(blockIdx.y) * 8 * NT;
  const int64_t K = p.K, groups = K / G;
  const int64_t chunks = (K + kChunkK - 1) / kChunkK;
  const int64_t c0 = chunks * slice / slices, c1 = chunks * (slice + 1) / slices;
  // rows and tokens past the end read the last one and are not stored
  const int64_t na = n0 + g < p.N ? n0 + g : p.N - 1, nb = n0 + g + 8 < p.N ? n0 + g + 8 : p.N - 1;

  Words<G> wa[kGroups], wb[kGroups];
  uint16_t sa[kGroups], sb[kGroups];
  Raw<TERMS> xr[kPer];
  Words<G> wa1[kGroups], wb1[kGroups];  // the next chunk's
  uint16_t sa1[kGroups], sb1[kGroups];
  auto fetch_weights = [&](int64_t c) {
#pragma unroll
    for (int q = 0; q < kGroups; ++q) {
      const int64_t at = c * kGroups + q;
      if (c < c1 && at < groups) {
        wa1[q].load(p.packed + na * (K / 2) + at * (G / 2) + t * (G / 8));
        wb1[q].load(p.packed + nb * (K / 2) + at * (G / 2) + t * (G / 8));
        sa1[q] = __ldcg(p.scales + na * groups + at);
        sb1[q] = __ldcg(p.scales + nb * groups + at);
      }
    }
  };
  auto fetch_x = [&](int64_t c) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int u = threadIdx.x + i * kManyWarps * 32;
      const int64_t k = c * kChunkK + u % (kChunkK / 8) * 8;
      if (u < kUnits && c < c1 && k < K) {
        const int64_t m = m0 + u / (kChunkK / 8) < p.M ? m0 + u / (kChunkK / 8) : p.M - 1;
        xr[i].load(p.x, m * K + k);
      }
    }
  };
  auto keep_x = [&](int buffer) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int u = threadIdx.x + i * kManyWarps * 32;
      if (u < kUnits) {
        uint4 v[TERMS];
        split<TERMS>(xr[i], v);
#pragma unroll
        for (int k = 0; k < TERMS; ++k)
          *reinterpret_cast<uint4 *>(xs + buffer * kBuffer + (k * 8 * NT + u / (kChunkK / 8)) * kChunkPitch +
                                     u % (kChunkK / 8) * 8) = v[k];
      }
    }
  };
  if (p.weights_static) fetch_weights(c0);
  pdl_wait();
  pdl_launch_dependents();
  if (!p.weights_static) fetch_weights(c0);
  fetch_x(c0);
  float y[NT][4];
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) y[j][e] = 0.0f;
  for (int64_t c = c0; c < c1; ++c) {
    const int buffer = static_cast<int>(c & 1);
#pragma unroll
    for (int q = 0; q < kGroups; ++q) {
      wa[q] = wa1[q];
      wb[q] = wb1[q];
      sa[q] = sa1[q];
      sb[q] = sb1[q];
    }
    keep_x(buffer);  // (last read two chunks ago, before the last barrier)
    fetch_weights(c + 1);
    fetch_x(c + 1);
    __syncthreads();
#pragma unroll
    for (int q = 0; q < kGroups; ++q) {
      if (c * kGroups + q >= groups) break;
      float acc[NT][4];
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[j][e] = 0.0f;
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        uint32_t fa[4], fb[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          fa[e] = two_codes(wa[q].w[i], e);
          fb[e] = two_codes(wb[q].w[i], e);
        }
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int k = TERMS - 1; k >= 0; --k) {
            const uint4 x = *reinterpret_cast<const uint4 *>(xs + buffer * kBuffer + (k * 8 * NT + 8 * j + g) * kChunkPitch +
                                                             q * G + t * (G / 4) + i * 8);
            mma_bf16(acc[j], fa[0], fb[0], fa[1], fb[1], x.x, x.y);
            mma_bf16(acc[j], fa[2], fb[2], fa[3], fb[3], x.z, x.w);
          }
      }
      const float s0 = bf16_value(sa[q]), s1 = bf16_value(sb[q]);
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        y[j][0] = __fmaf_rn(s0, acc[j][0], y[j][0]);
        y[j][1] = __fmaf_rn(s0, acc[j][1], y[j][1]);
        y[j][2] = __fmaf_rn(s1, acc[j][2], y[j][2]);
        y[j][3] = __fmaf_rn(s1, acc[j][3], y[j][3]);
      }
    }
  }
  __syncthreads();  // the activations are done with
  constexpr int kPitch = 8 * NT + 1;
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    float *at = part + (warp * kRows + g) * kPitch + 8 * j + 2 * t;
    at[0] = y[j][0];
    at[1] = y[j][1];
    at[8 * kPitch] = y[j][2];
    at[8 * kPitch + 1] = y[j][3];
  }
  if (slices > 1)
    cluster_sync();
  else
    __syncthreads();
  // each CTA adds up and stores its share of the rows
  const int rows = kManyRows / static_cast<int>(slices);
  const int64_t first = static_cast<int64_t>(blockIdx.x / slices) * kManyRows + slice * rows;
  for (int i = threadIdx.x; i < rows * 8 * NT; i += kManyWarps * 32) {
    const int row = i % rows, col = i / rows;
    if (first + row >= p.N || m0 + col >= p.M) continue;
    const float *at = part + (slice * rows + row) * kPitch + col;
    float v = 0.0f;
    for (uint32_t s = 0; s < slices; ++s) {
      float x;
      asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(mapa_shared(at, s)) : "memory");
      v += x;
    }
    store_y<YK>(p.y, (m0 + col) * p.N + first + row, v);
  }
  if (slices > 1) cluster_sync();  // the others have read this CTA's sums
}

template <int G, int TERMS, int YK>
cudaError_t launch_few(W4Params p, const FewPlan &f, const LaunchCtx &ctx) {
  static std::atomic<uint64_t> ready;
  if (const cudaError_t e = allow_smem(w4_few_kernel<G, TERMS, YK>, kFewSmem, ready, ctx)) return e;
  p.tiles = static_cast<int>(ceil_div(p.N, kRows));
  // resident CTAs only: each goes on to further tiles with its copies ahead
  int per_sm = static_cast<int>(size_t(224 * 1024) / (f.smem + 6 * 1024));
  per_sm = per_sm > 5 ? 5 : (per_sm < 1 ? 1 : per_sm);
  const int most = ctx.num_sms * per_sm;
  const dim3 grid(static_cast<unsigned>(p.tiles < most ? p.tiles : most));
  return launch_k(w4_few_kernel<G, TERMS, YK>, grid, dim3(kFewWarps * 32), f.smem, ctx, p, f);
}
template <int G, int NT, int TERMS, int YK>
cudaError_t launch_many(W4Params p, const LaunchCtx &ctx) {
  constexpr size_t smem = many_smem<NT, TERMS>();
  static std::atomic<uint64_t> ready;
  if (const cudaError_t e = allow_smem(w4_many_kernel<G, NT, TERMS, YK>, smem, ready, ctx)) return e;
  p.tiles = static_cast<int>(ceil_div(p.N, kManyRows));
  const int64_t blocks = p.tiles * ceil_div(p.M, 8 * NT), chunks = ceil_div(p.K, kChunkK);
  unsigned slices = 1;  // of K, until the CTAs fill the GPU
  while (slices < 8 && blocks * slices * 2 <= 2 * ctx.num_sms && slices * 2 <= chunks) slices *= 2;
  const dim3 grid(static_cast<unsigned>(p.tiles) * slices, static_cast<unsigned>(ceil_div(p.M, 8 * NT)));
  return launch_k_cluster(w4_many_kernel<G, NT, TERMS, YK>, grid, dim3(kManyWarps * 32), smem, slices, ctx, p);
}
template <int G, int TERMS, int YK>
cudaError_t launch_m(const W4Params &p, const LaunchCtx &ctx) {
  FewPlan f;
  if (p.M <= 8 && few_plan(p.M, p.K, G, TERMS, &f)) return launch_few<G, TERMS, YK>(p, f, ctx);
  if (p.M <= 8) return launch_many<G, 1, TERMS, YK>(p, ctx);
  if (p.M <= 16) return launch_many<G, 2, TERMS, YK>(p, ctx);
  if (p.M <= 24) return launch_many<G, 3, TERMS, YK>(p, ctx);
  return launch_many<G, 4, TERMS, YK>(p, ctx);
}
template <int TERMS, int YK>
cudaError_t launch_g(const W4Params &p, int group, const LaunchCtx &ctx) {
  if (group == 128) return launch_m<128, TERMS, YK>(p, ctx);
  if (group == 64) return launch_m<64, TERMS, YK>(p, ctx);
  return launch_m<32, TERMS, YK>(p, ctx);
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

cudaError_t launch_w4(const void *X, int x_kind, const uint8_t *packed, const uint16_t *scales,
                      int64_t M, int64_t N, int64_t K, int group, void *Y, int y_kind,
                      bool weights_static, const LaunchCtx &ctx) {
  const W4Params p = {X, packed, scales, Y, M, N, K, 0, weights_static, ctx.status};
  if (x_kind == kF32)
    return y_kind == kF32 ? launch_g<3, kF32>(p, group, ctx) : launch_g<3, kBF16>(p, group, ctx);
  return y_kind == kF32 ? launch_g<1, kF32>(p, group, ctx) : launch_g<1, kBF16>(p, group, ctx);
}

}  // namespace bitnet
