// kv_attention_prompt.cu -- attention of prompts over the 8-bit paged cache
// on the fifth-generation tensor cores (tcgen05, fp16 operands, fp32 sums in
// tensor memory).  bf16 queries; the formula and the treatment of the scales
// are those of kv_attention.cu.
//
// A CTA takes 256 query rows (query, head of the group) of one sequence and
// key head as two tiles of 128, and goes over the tokens 128 at a time:
//   S = Q K^T    Q from shared memory (fp16, scaled by a power of two per
//                row), K's codes from shared memory, both K-major
//   O += P V     P from tensor memory, where the softmax left it as fp16 over
//                the S it came from; V's codes transposed, K-major, from
//                shared memory
// warps 0-3, 4-7  softmax of tile 0, 1, a thread per row: maximum, weights,
//                 row sum; O is rescaled in tensor memory only when a maximum
//                 passes the one in use by 2^kLazy
// warps 8-11      convert the int8 codes of the next block to fp16 (byte
//                 permutes and one subtraction per two codes) into two
//                 shared-memory stages each for K and V, loads one block
//                 ahead, page numbers two
// warp 12         one lane issues the MMAs: P0 V, Q0 K' of the next block,
//                 P1 V, Q1 K', so each tile's softmax runs under the other
//                 tile's products
// Tensor memory: S0 S1 (128 columns each, P over their first 64), O0 O1.
// Bound by the exponentials (16 a clock and SM) and the tensor cores about
// equally at head_dim 128: 2,048 against 2,040 clocks per block of 128 tokens.
// Every wait is bounded (common.cuh).
#include <atomic>

#include "attention.cuh"
#include "common.cuh"
#include "internal.h"

namespace bitnet {
namespace {

constexpr int kTile = 128;    // query rows of a tile; tokens of a block
constexpr int kSegs = kTile / 16;
constexpr int kStages = 2;
constexpr int kConvWarp0 = 8;
constexpr int kMmaWarp = 12;
constexpr int kThreads = 13 * 32;
constexpr int kTmemCols = 512;

struct PromptParams {
  KvCache cache;
  KvBatch batch;
  const __nv_bfloat16 *q;
  __nv_bfloat16 *o;
  int q_heads, group;
  float scale_log2;     // >= 0; a negative scale turns q's sign
  bool negate;
  int64_t window;
  int row_blocks;       // of 256 rows, per sequence; a sequence with more strides over them
  int *status;
};

struct BlockScales {
  float ks[kSegs], lv[kSegs], iv[kSegs];  // ks < 0: no page
};

template <int D> struct Smem {
  static constexpr int kOperand = kTile * D * 2;       // one fp16 operand tile
  static constexpr int kQ = 0, kK = 2 * kOperand, kV = kK + kStages * kOperand;
  static constexpr int kScales = kV + kStages * kOperand;
  static constexpr int kBars = kScales + kStages * static_cast<int>(sizeof(BlockScales));
  static constexpr int kNumBars = 1 + 5 * kStages + 3 * 2;
  static constexpr size_t kBytes = 1024 + kBars + 8 * kNumBars + 16;
};

__device__ __forceinline__ void mma_smem(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// A from tensor memory: 128 lanes, two halves per column.
__device__ __forceinline__ void mma_tmem(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
#define BITNET_R8(r, i) "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3]), "=r"(r[i + 4]), \
                        "=r"(r[i + 5]), "=r"(r[i + 6]), "=r"(r[i + 7])
#define BITNET_U8(r, i) "r"(r[i]), "r"(r[i + 1]), "r"(r[i + 2]), "r"(r[i + 3]), "r"(r[i + 4]), \
                        "r"(r[i + 5]), "r"(r[i + 6]), "r"(r[i + 7])
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
      "%14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : BITNET_R8(r, 0), BITNET_R8(r, 8), BITNET_R8(r, 16), BITNET_R8(r, 24)
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, "
      "%13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::
          BITNET_U8(r, 0), BITNET_U8(r, 8), BITNET_U8(r, 16), BITNET_U8(r, 24), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, "
      "%13, %14, %15};" ::BITNET_U8(r, 0), BITNET_U8(r, 8), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Byte offset of 16-byte chunk `chunk` of row `row` of an operand tile of
// `rows` rows, stored as panels of 64 halves (128-byte rows, 128-byte swizzle).
__device__ __forceinline__ int operand_offset(int rows, int row, int chunk) {
  return (chunk >> 3) * rows * 128 + row * 128 + (((chunk & 7) ^ (row & 7)) << 4);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) kv_attention_prompt_kernel(const PromptParams p) {
  using S = Smem<D>;
  constexpr int kPanelsD = D / 64;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  BlockScales *scales = reinterpret_cast<BlockScales *>(smem + S::kScales);
  uint64_t *q_full = reinterpret_cast<uint64_t *>(smem + S::kBars);
  uint64_t *k_full = q_full + 1, *k_empty = k_full + kStages;
  uint64_t *v_full = k_empty + kStages, *v_empty = v_full + kStages;
  uint64_t *sc_full = v_empty + kStages;                       // [kStages]
  uint64_t *s_full = sc_full + kStages, *p_full = s_full + 2, *pv_done = p_full + 2;
  uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(pv_done + 2);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    mbar_init(q_full, 2 * kTile);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&k_full[s], 4 * 32);
      mbar_init(&k_empty[s], 1);
      mbar_init(&v_full[s], 4 * 32);
      mbar_init(&v_empty[s], 1);
      mbar_init(&sc_full[s], 32);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&s_full[t], 1);
      mbar_init(&p_full[t], kTile);
      mbar_init(&pv_done[t], 1);
    }
    fence_barrier_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(tmem_holder, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  pdl_wait();
  pdl_launch_dependents();

  // row block slowest and the last first (the longest under a causal mask)
  int64_t i = blockIdx.x;
  const int h = static_cast<int>(i % p.cache.heads);
  i /= p.cache.heads;
  const int64_t b = i % p.batch.B;
  const int block0 = p.row_blocks - 1 - static_cast<int>(i / p.batch.B);
  const int P = p.cache.page_tokens, G = p.group;
  int64_t r0, r1, len;
  const bool fine = kv_sequence(p.batch, P, b, &r0, &r1, &len);
  if (!fine && threadIdx.x == 0) record_status(p.status, kStatusRange);
  const int64_t n = r1 - r0, blocks = fine ? (n * G + 2 * kTile - 1) / (2 * kTile) : 0;

  uint32_t done = 0;        // KV blocks that this CTA has been through (stage and phase counters)
  uint32_t tiles_done[2] = {0, 0};  // of them, blocks of tile 0, 1
  uint32_t q_phase = 0;
  bool ok = true;
  for (int64_t rb = block0; rb < blocks && ok; rb += p.row_blocks) {
    const int64_t row0 = rb * 2 * kTile;
    // positions that rows of the block see: [lo, hi), lo on a block boundary;
    // hi of each tile, 0 blocks for a tile without rows
    int64_t lo = 0;
    int nb[2];
    int64_t hi = 0;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int64_t first = row0 + t * kTile, last = first + kTile < n * G ? first + kTile : n * G;
      nb[t] = 0;
      if (t == 0 && p.window > 0) {
        const int64_t from = len - n + row0 / G - p.window + 1;
        lo = (from > 0 ? from : 0) / kTile * kTile;
      }
      if (first < last) {
        const int64_t end = len - n + (last - 1) / G + 1;
        if (end > lo) nb[t] = static_cast<int>((end - lo + kTile - 1) / kTile);
        if (end > hi) hi = end;
      }
    }
    const int total = nb[0] > nb[1] ? nb[0] : nb[1];
    auto stage = [&](int j) { return static_cast<int>((done + j) % kStages); };
    auto use = [&](int j) { return (done + j) / kStages; };  // of that stage

    if (warp < kConvWarp0) {
      // ================================================ softmax
      const int t = warp >> 2, row = threadIdx.x & (kTile - 1);
      const int64_t gr = row0 + t * kTile + row;
      const bool have = gr < n * G;
      const int64_t query = (have ? gr : n * G - 1) / G;
      const int64_t at = (have ? (r0 + gr / G) * p.q_heads + static_cast<int64_t>(h) * G + gr % G : 0) * D;
      // q to shared memory, its largest value brought to [2^14, 2^15)
      float fac;
      {
        uint4 v[D / 8];
        uint32_t peak = 0;
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          v[c] = have ? __ldg(reinterpret_cast<const uint4 *>(p.q + at) + c) : make_uint4(0, 0, 0, 0);
          const uint32_t w[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t a = (w[e] << 16) & 0x7FFFFFFFu, c2 = w[e] & 0x7FFF0000u;
            peak = peak > a ? peak : a;
            peak = peak > c2 ? peak : c2;
          }
        }
        int k = 14 - (static_cast<int>(peak >> 23) - 127);
        k = k < -110 ? -110 : (k > 110 ? 110 : k);
        const float up = __uint_as_float((static_cast<uint32_t>(127 + k) << 23) | (p.negate ? 0x80000000u : 0u));
        fac = __fmul_rn(p.scale_log2, __uint_as_float(static_cast<uint32_t>(127 - k) << 23));
        uint8_t *tile = smem + S::kQ + t * S::kOperand;
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          const uint32_t w[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
          uint32_t o[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const __half2 x = __floats2half2_rn(__fmul_rn(__uint_as_float(w[e] << 16), up),
                                                __fmul_rn(__uint_as_float(w[e] & 0xFFFF0000u), up));
            o[e] = half2_bits(x);
          }
          *reinterpret_cast<uint4 *>(tile + operand_offset(kTile, row, c)) = make_uint4(o[0], o[1], o[2], o[3]);
        }
        fence_proxy_async_smem();
        mbar_arrive(q_full);
      }
      const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // 32 lanes per warp, bits 16 and up
      const uint32_t ts = tmem + lanes + t * kTile, to = tmem + lanes + 2 * kTile + t * D;
      const int64_t pos = len - n + query;
      float m = -INFINITY, l = 0.0f;
      for (int j = 0; j < nb[t] && ok; ++j) {
        const int st = stage(j);
        const uint32_t tj = tiles_done[t] + j;
        ok = mbar_wait(&sc_full[st], use(j) & 1, p.status) && mbar_wait(&s_full[t], tj & 1, p.status);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        const BlockScales &sc = scales[st];
        const int64_t base = lo + static_cast<int64_t>(j) * kTile;
        // visible columns of the block: [c_lo, c_hi)
        const int64_t end = pos + 1 - base, begin = p.window > 0 ? pos - p.window + 1 - base : 0;
        const int c_hi = static_cast<int>(end < 0 ? 0 : (end > kTile ? kTile : end));
        const int c_lo = static_cast<int>(begin < 0 ? 0 : (begin > kTile ? kTile : begin));
        bool part = c_hi < kTile || c_lo > 0;
#pragma unroll
        for (int s = 0; s < kSegs; ++s) part |= sc.ks[s] < 0.0f;
        const bool masked = __any_sync(0xffffffffu, part);
        auto hide = [&](uint32_t (&v)[32], int c0) {  // columns c0 .. c0 + 31
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const int c = c0 + e;
            if (c < c_lo || c >= c_hi || sc.ks[c / 16] < 0.0f) v[e] = 0xFF800000u;
          }
        };

        // ---- the row's maximum of score + log2 vs
        float top = -INFINITY;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t v[32];
          tmem_ld32(ts + 32 * q, v);
          tmem_wait_ld();
          if (masked) hide(v, 32 * q);
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            float x = __uint_as_float(v[16 * s]);
#pragma unroll
            for (int e = 1; e < 16; ++e) x = fmaxf(x, __uint_as_float(v[16 * s + e]));
            // (0 * -inf of a fully hidden segment would be NaN, which fmaxf drops)
            top = fmaxf(top, __fmaf_rn(x, fac * fabsf(sc.ks[2 * q + s]), sc.lv[2 * q + s]));
          }
        }
        // ---- follow it where it has grown by more than 2^kLazy
        if (__any_sync(0xffffffffu, top > m + kLazy)) {
          const float next = fmaxf(m, top);
          const float f = m == next ? 1.0f : ex2(m - next);
          m = next;
          l *= f;
          if (j > 0) {
            ok = mbar_wait(&pv_done[t], (tj - 1) & 1, p.status);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int q = 0; q < D / 32; ++q) {
              uint32_t v[32];
              tmem_ld32(to + 32 * q, v);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__fmul_rn(__uint_as_float(v[e]), f));
              tmem_st32(to + 32 * q, v);
            }
          }
        }
        const float from = m == -INFINITY ? 0.0f : m - kRaise;
        // ---- weights, over the scores they come from, and the row sum
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t v[32], w[16];
          tmem_ld32(ts + 32 * q, v);
          tmem_wait_ld();
          if (masked) hide(v, 32 * q);
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            const float c1 = fac * fabsf(sc.ks[2 * q + s]), c0 = sc.lv[2 * q + s] - from;
            float sum = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              float x0 = __fmaf_rn(__uint_as_float(v[16 * s + 2 * e]), c1, c0);
              float x1 = __fmaf_rn(__uint_as_float(v[16 * s + 2 * e + 1]), c1, c0);
              if (masked) {  // a factor of 0 turns what is hidden into NaN
                if (v[16 * s + 2 * e] == 0xFF800000u) x0 = -INFINITY;
                if (v[16 * s + 2 * e + 1] == 0xFF800000u) x1 = -INFINITY;
              }
              x0 = ex2(x0);
              x1 = ex2(x1);
              sum += x0 + x1;
              w[8 * s + e] = half2_bits(__floats2half2_rn(x0, x1));
            }
            l = __fmaf_rn(sum, sc.iv[2 * q + s], l);
          }
          tmem_st16(ts + 16 * q, w);
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&p_full[t]);
      }
      // ---- the tile's rows
      if (ok && nb[t] > 0) {
        ok = mbar_wait(&pv_done[t], (tiles_done[t] + nb[t] - 1) & 1, p.status);
        ok = __all_sync(0xffffffffu, ok);
        tc_fence_after();
      }
      if (ok) {
        const float inv = l == 0.0f ? 0.0f : __fdiv_rn(1.0f, l);  // nothing visible: zeros
#pragma unroll
        for (int q = 0; q < D / 32; ++q) {
          uint32_t v[32];
          if (nb[t] > 0) {
            tmem_ld32(to + 32 * q, v);
            tmem_wait_ld();
          }
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t x[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float a = nb[t] > 0 ? __uint_as_float(v[8 * c + 2 * e]) * inv : 0.0f;
              const float d = nb[t] > 0 ? __uint_as_float(v[8 * c + 2 * e + 1]) * inv : 0.0f;
              const __nv_bfloat162 y = __floats2bfloat162_rn(a, d);
              x[e] = *reinterpret_cast<const uint32_t *>(&y);
            }
            if (have)
              reinterpret_cast<uint4 *>(p.o + at)[4 * q + c] = make_uint4(x[0], x[1], x[2], x[3]);
          }
        }
      }
      tc_fence_before();
    } else if (warp < kMmaWarp) {
      // ================================================ int8 -> fp16
      const int cw = warp - kConvWarp0;
      const int *table = p.batch.pages + b * p.batch.max_pages;
      auto page_of = [&](int j) -> int {  // of segment `lane` of block j
        const int64_t tok = lo + static_cast<int64_t>(j) * kTile + 16 * lane;
        if (lane >= kSegs || j >= total || tok >= hi) return -1;
        const int page = __ldg(table + tok / P);
        return page;
      };
      auto checked = [&](int page, int j) -> int {
        if (page >= 0 && page < p.cache.pages) return page;
        const int64_t tok = lo + static_cast<int64_t>(j) * kTile + 16 * lane;
        if (lane < kSegs && j < total && tok < hi) record_status(p.status, kStatusRange);
        return -1;
      };
      constexpr int kLanesK = D / 16;            // lanes of a row's 16-byte chunks
      constexpr int kItK = D / 16;               // loads per thread: kTile rows / (128 / kLanesK)
      constexpr int kRowsIt = 128 / kLanesK;     // rows per round
      uint4 kr[kItK], vr[8];
      const int k_row = (cw * 32 + lane) / kLanesK, k_chunk = (cw * 32 + lane) % kLanesK;
      // V: 8 tokens (an octet) by 16 columns per thread
      const int v_octet = (lane & 7) + 8 * (cw & 1);
      const int v_chunk = (lane >> 3) + 4 * (cw >> 1);   // D = 64: 4 chunks, warps 0 and 1 only
      const bool v_mine = v_chunk < D / 16;
      auto load_k = [&](int page, int j) {
#pragma unroll
        for (int it = 0; it < kItK; ++it) {
          const int r = it * kRowsIt + k_row;
          const int pg = __shfl_sync(0xffffffffu, page, r / 16);
          kr[it] = make_uint4(0, 0, 0, 0);
          if (pg >= 0) {
            const int64_t row = (lo + static_cast<int64_t>(j) * kTile + r) % P;
            kr[it] = __ldg(reinterpret_cast<const uint4 *>(
                p.cache.k_codes + ((static_cast<int64_t>(pg) * p.cache.heads + h) * P + row) * D) + k_chunk);
          }
        }
      };
      auto load_v = [&](int page, int j) {
        const int pg = __shfl_sync(0xffffffffu, page, v_octet / 2);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          vr[e] = make_uint4(0, 0, 0, 0);
          if (pg >= 0 && v_mine) {
            const int64_t row = (lo + static_cast<int64_t>(j) * kTile + v_octet * 8 + e) % P;
            vr[e] = __ldg(reinterpret_cast<const uint4 *>(
                p.cache.v_codes + ((static_cast<int64_t>(pg) * p.cache.heads + h) * P + row) * D) + v_chunk);
          }
        }
      };
      float ks = -1.0f, vs = 0.0f;  // of segment `lane`, the first warp's
      auto load_scales = [&](int page) {
        ks = -1.0f;
        if (cw == 0 && page >= 0) {
          ks = __ldg(p.cache.k_scales + static_cast<int64_t>(page) * p.cache.heads + h);
          vs = __ldg(p.cache.v_scales + static_cast<int64_t>(page) * p.cache.heads + h);
        }
      };
      int page = checked(page_of(0), 0), next = page_of(1);
      load_k(page, 0);
      load_v(page, 0);
      load_scales(page);
      for (int j = 0; j < total && ok; ++j) {
        const int st = stage(j);
        const uint32_t u = use(j);
        if (u > 0) {  // the stage's last user has gone through
          ok = mbar_wait(&v_empty[st], (u - 1) & 1, p.status) && mbar_wait(&k_empty[st], (u - 1) & 1, p.status);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
        }
        if (cw == 0) {
          if (lane < kSegs) {
            const bool some = !(vs < kKvMinScale);
            scales[st].ks[lane] = ks;
            scales[st].lv[lane] = ks >= 0.0f && some ? log2f(vs) : -60.0f;
            scales[st].iv[lane] = ks >= 0.0f && some ? __fdiv_rn(1.0f, vs) : 1.152921504606846976e18f;  // 2^60
          }
          mbar_arrive(&sc_full[st]);
        }
        const int page1 = checked(next, j + 1);
        next = page_of(j + 2);
        uint8_t *kt = smem + S::kK + st * S::kOperand, *vt = smem + S::kV + st * S::kOperand;
#pragma unroll
        for (int it = 0; it < kItK; ++it) {
          const int r = it * kRowsIt + k_row;
          // the upper half's lanes store their second 16 bytes first: two
          // panels, other banks
          const bool swap = (k_chunk & 4) != 0;
          const uint32_t w[4] = {swap ? kr[it].z : kr[it].x, swap ? kr[it].w : kr[it].y,
                                 swap ? kr[it].x : kr[it].z, swap ? kr[it].y : kr[it].w};
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const uint32_t a = w[2 * half] ^ 0x80808080u, c = w[2 * half + 1] ^ 0x80808080u;
            const int chunk = 2 * k_chunk + (half ^ static_cast<int>(swap));
            *reinterpret_cast<uint4 *>(kt + operand_offset(kTile, r, chunk)) =
                make_uint4(codes01(a), codes23(a), codes01(c), codes23(c));
          }
        }
        fence_proxy_async_smem();
        mbar_arrive(&k_full[st]);
        load_k(page1, j + 1);
        if (v_mine) {
          // V^T: row = column of the head, 8 tokens per 16-byte chunk
#pragma unroll
          for (int i4 = 0; i4 < 4; ++i4) {
            uint32_t x[4][2];  // [token pair][columns 0 1 | 2 3]
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint4 &va = vr[2 * e], &vb = vr[2 * e + 1];
              const uint32_t a = (i4 == 0 ? va.x : i4 == 1 ? va.y : i4 == 2 ? va.z : va.w) ^ 0x80808080u;
              const uint32_t c = (i4 == 0 ? vb.x : i4 == 1 ? vb.y : i4 == 2 ? vb.z : vb.w) ^ 0x80808080u;
              x[e][0] = __byte_perm(a, c, 0x5140);
              x[e][1] = __byte_perm(a, c, 0x7362);
            }
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const int d = 16 * v_chunk + 4 * i4 + c;
              uint32_t o[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) o[e] = (c & 1) != 0 ? codes23(x[e][c >> 1]) : codes01(x[e][c >> 1]);
              *reinterpret_cast<uint4 *>(vt + operand_offset(D, d, v_octet)) = make_uint4(o[0], o[1], o[2], o[3]);
            }
          }
        }
        fence_proxy_async_smem();
        mbar_arrive(&v_full[st]);
        load_v(page1, j + 1);
        load_scales(page1);
        page = page1;
      }
    } else if (lane == 0) {
      // ================================================ MMAs
      constexpr uint32_t kIdescS = (1u << 4) | ((kTile >> 3) << 17) | ((kTile >> 4) << 24);
      constexpr uint32_t kIdescO = (1u << 4) | ((D >> 3) << 17) | ((kTile >> 4) << 24);
      const uint32_t base = smem_u32(smem);
      ok = mbar_wait(q_full, q_phase, p.status);
      tc_fence_after();
      auto scores = [&](int t, int j) {  // S_t = Q_t K_j^T
        const uint32_t a = base + S::kQ + t * S::kOperand, k = base + S::kK + stage(j) * S::kOperand;
#pragma unroll
        for (int q = 0; q < kPanelsD; ++q)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            mma_smem(tmem + t * kTile, smem_desc_sw128(a + q * kTile * 128 + 32 * e),
                     smem_desc_sw128(k + q * kTile * 128 + 32 * e), kIdescS, (q | e) != 0 ? 1u : 0u);
        mma_commit(&s_full[t]);
      };
      auto values = [&](int t, int j) {  // O_t += P_t V_j
        const uint32_t v = base + S::kV + stage(j) * S::kOperand;
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            mma_tmem(tmem + 2 * kTile + t * D, tmem + t * kTile + 32 * q + 8 * e,
                     smem_desc_sw128(v + q * D * 128 + 32 * e), kIdescO, j > 0 || (q | e) != 0 ? 1u : 0u);
        mma_commit(&pv_done[t]);
      };
      for (int j = 0; j <= total && ok; ++j) {  // values of block j - 1, then scores of block j
        bool k_ready = false;
        for (int t = 0; t < 2 && ok; ++t) {
          if (j > 0 && j - 1 < nb[t]) {
            ok = mbar_wait(&p_full[t], (tiles_done[t] + j - 1) & 1, p.status) &&
                 mbar_wait(&v_full[stage(j - 1)], use(j - 1) & 1, p.status);
            if (!ok) break;
            tc_fence_after();
            values(t, j - 1);
          }
          if (j < nb[t]) {
            if (!k_ready) {
              ok = k_ready = mbar_wait(&k_full[stage(j)], use(j) & 1, p.status);
              if (!ok) break;
              tc_fence_after();
            }
            scores(t, j);
          }
        }
        if (!ok) break;
        if (j > 0) mma_commit(&v_empty[stage(j - 1)]);
        if (j < total) mma_commit(&k_empty[stage(j)]);
      }
    }
    done += static_cast<uint32_t>(total);
    tiles_done[0] += static_cast<uint32_t>(nb[0]);
    tiles_done[1] += static_cast<uint32_t>(nb[1]);
    q_phase ^= 1u;
    // the next rows' q overwrites this one's: every product has been waited
    // for by the softmax warps
    __syncwarp();
    ok = __syncthreads_and(ok) != 0;
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) tmem_dealloc(tmem, kTmemCols);
}

}  // namespace

bool kv_attention_prompt_fits(const KvCache &cache, const KvBatch &batch, const AttnArgs &args) {
  const int64_t most = (int64_t(1) << 31) - 1;
  const int64_t row_blocks = ceil_div(args.max_new * (args.q_heads / cache.heads), 2 * kTile);
  return row_blocks <= most / cache.heads && batch.B <= most / (row_blocks * cache.heads);
}

cudaError_t launch_kv_attention_prompt(const KvCache &cache, const KvBatch &batch, const AttnArgs &args,
                                       const LaunchCtx &ctx) {
  PromptParams p = {};
  p.cache = cache;
  p.batch = batch;
  p.q = static_cast<const __nv_bfloat16 *>(args.Q);
  p.o = static_cast<__nv_bfloat16 *>(args.O);
  p.q_heads = args.q_heads;
  p.group = args.q_heads / cache.heads;
  p.negate = args.scale < 0.0f;
  p.scale_log2 = (p.negate ? -args.scale : args.scale) * kLog2e;
  p.window = args.window;
  p.row_blocks = static_cast<int>(ceil_div(args.max_new * p.group, 2 * kTile));
  p.status = ctx.status;
  const dim3 grid(static_cast<unsigned>(batch.B * p.row_blocks * cache.heads));
  static std::atomic<uint64_t> ready[2];
  const bool wide = cache.head_dim == 128;
  auto kernel = wide ? kv_attention_prompt_kernel<128> : kv_attention_prompt_kernel<64>;
  const size_t smem = wide ? Smem<128>::kBytes : Smem<64>::kBytes;
  if (const cudaError_t e = allow_smem(kernel, smem, ready[wide ? 1 : 0], ctx)) return e;
  return launch_k(kernel, grid, dim3(kThreads), smem, ctx, p);
}

}  // namespace bitnet
