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
// warps 8-11      convert K's int8 codes of the blocks ahead to fp16 (byte
// (12-15: V's)    permutes and one subtraction per two codes) into two
//                 shared-memory stages, loads one block ahead, page numbers
//                 two
// warp 16         (of four; the others give up their registers) one lane issues the MMAs: P0 V, Q0 K' of the next block,
//                 P1 V, Q1 K', so each tile's softmax runs under the other
//                 tile's products
// Tensor memory: S0 S1 (128 columns each, P over their first 64), O0 O1.
// At head_dim 128 a block of 128 tokens has 2,048 clocks of exponentials (16 a
// clock and SM) and 2,040 of tensor-core work.  Measured (clock64 in a copy):
// about 6,500, of which a tile's softmax takes 4,500 (its four warps are two
// per scheduler and wait on their own latencies; knocking out the exponentials
// saves a tenth) and the products behind it most of the rest: 224 us for
// prompts of 4096 and 1236 tokens and 118 GFLOP (527 TFLOP/s; counters: tensor
// pipe 28 %, exponentials 28 %, issue slots 41 %).  Two threads per row and smaller
// register sets (296 us) and weights before the maximum is known, redone
// where it grows (243 us at the time of 245), were measured and not kept.
// Every wait is bounded (common.cuh).
#include <atomic>
#include <type_traits>

#include "attention.cuh"
#include "common.cuh"
#include "internal.h"
#include "pairs.cuh"

namespace bitnet {
namespace {

constexpr int kTile = 128;    // query rows of a tile; tokens of a block
constexpr int kSegs = kTile / 16;
constexpr int kStages = 2, kSlots = 4;
constexpr int kConvWarp0 = 8;
constexpr int kValueWarp0 = 12;
constexpr int kMmaWarp = 16;
constexpr int kThreads = 20 * 32;
// Registers per thread, 96 at launch, by groups of four warps: softmax twice,
// conversion twice, and the MMA warp with three that are idle.
constexpr int kRegsSoftmax = 152, kRegsConvert = 64, kRegsMma = 48;
static_assert(2 * kRegsSoftmax + 2 * kRegsConvert + kRegsMma == 5 * 96, "register split");
constexpr int kTmemCols = 512;

struct PromptParams {
  KvCache cache;
  KvBatch batch;
  const __nv_bfloat16 *q;
  __nv_bfloat16 *o;
  int q_heads, group;
  float scale_log2;     // >= 0; a negative scale turns q's sign
  bool negate;
  int window;
  int row_blocks;       // of 256 rows, per sequence; a sequence with more strides over them
  int *status;
};

struct BlockScales {
  // ks < 0: no page, iv = 0; iv < 0: value scales far apart, here or before (attention.cuh)
  float ks[kSegs], lv[kSegs], iv[kSegs];
};

template <int D> struct Smem {
  static constexpr int kOperand = kTile * D * 2;       // one fp16 operand tile
  static constexpr int kQ = 0, kK = 2 * kOperand, kV = kK + kStages * kOperand;
  static constexpr int kScales = kV + kStages * kOperand;
  static constexpr int kBars = kScales + kSlots * static_cast<int>(sizeof(BlockScales));
  static constexpr int kNumBars = 1 + 4 * kStages + kSlots + 3 * 2 + 1;
  static constexpr size_t kBytes = 1024 + kBars + 8 * kNumBars + 16;
};

// The tensor cores take 64 clocks per MMA here, which the issuing lane must
// not exceed: descriptors are a low word that steps by constants under a
// constant high word (smem_desc_sw128), and everything is unrolled.
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_low(uint32_t saddr) { return ((saddr & 0x3FFFFu) >> 4) | (1u << 16); }
__device__ __forceinline__ void mma_smem(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "mov.b64 da, {%1, %5};\n\t"
      "mov.b64 db, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(acc), "r"(kDescHigh)
      : "memory");
}
// A from tensor memory: 128 lanes, two halves per column.
__device__ __forceinline__ void mma_tmem(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "mov.b64 db, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(acc), "r"(kDescHigh)
      : "memory");
}
#define BITNET_R8(r, i) "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3]), "=r"(r[i + 4]), \
                        "=r"(r[i + 5]), "=r"(r[i + 6]), "=r"(r[i + 7])
#define BITNET_U8(r, i) "r"(r[i]), "r"(r[i + 1]), "r"(r[i + 2]), "r"(r[i + 3]), "r"(r[i + 4]), \
                        "r"(r[i + 5]), "r"(r[i + 6]), "r"(r[i + 7])
#define BITNET_RW8(r, i) "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]), \
                         "+r"(r[i + 5]), "+r"(r[i + 6]), "+r"(r[i + 7])
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
      "%14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : BITNET_R8(r, 0), BITNET_R8(r, 8), BITNET_R8(r, 16), BITNET_R8(r, 24)
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, "
      "%13, %14, %15};" ::BITNET_U8(r, 0), BITNET_U8(r, 8), "r"(taddr)
      : "memory");
}
// Waits for this thread's loads from tensor memory; the registers that the
// caller goes on with are operands, so that no use moves ahead of the wait.
__device__ __forceinline__ void tmem_arrived(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" : BITNET_RW8(r, 0), BITNET_RW8(r, 8)::"memory");
}
__device__ __forceinline__ void tmem_arrived(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : BITNET_RW8(r, 0), BITNET_RW8(r, 8), BITNET_RW8(r, 16), BITNET_RW8(r, 24)::"memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Byte offset of 16-byte chunk `chunk` of row `row` of an operand tile of
// `rows` rows, stored as panels of 64 halves (128-byte rows, 128-byte swizzle).
__device__ __forceinline__ int operand_offset(int rows, int row, int chunk) {
  return (chunk >> 3) * rows * 128 + row * 128 + (((chunk & 7) ^ (row & 7)) << 4);
}

template <int N> __device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N> __device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// A block of the softmax below with value scales far apart: every score
// compared with the mask, shares of the row sum by themselves, rescaled in two
// steps (l may be 2^75, f 2^-181).  Its own function, so that the form for
// scales as they should be keeps its registers (236 against 224 us for prompts
// of 4096 tokens).
struct Row {
  float m, l;
  bool ok;
};
template <int D>
__device__ __noinline__ Row far_block(Row r, uint32_t ts, uint32_t to, float fac, const BlockScales &sc, int c_lo,
                                      int c_hi, uint64_t *pv_done, uint32_t parity, int *status) {
  // score + log2 vs of column c, -infinity where it is not seen
  auto score = [&](uint32_t v, int c, float plus) -> float {
    const float ks = sc.ks[c / 16];
    return c < c_lo || c >= c_hi || ks < 0.0f ? -INFINITY
                                              : __fmaf_rn(__uint_as_float(v), __fmul_rn(fac, fabsf(ks)), plus);
  };
  float top = -INFINITY;
#pragma unroll 1
  for (int c0 = 0; c0 < kTile; c0 += 16) {
    uint32_t v[16];
    tmem_ld16(ts + c0, v);
    tmem_arrived(v);
#pragma unroll
    for (int e = 0; e < 16; ++e) top = fmaxf(top, score(v[e], c0 + e, sc.lv[c0 / 16]));
  }
  const bool grow = top > r.m + kLazy;
  if (__any_sync(0xffffffffu, grow)) {
    const float next = grow ? ceilf(top) : r.m;
    const int steps = r.m == next ? 0 : static_cast<int>(fmaxf(r.m - next, -250.0f)), half = steps / 2;
    const float f0 = __uint_as_float(static_cast<uint32_t>(127 + half) << 23);
    const float f1 = __uint_as_float(static_cast<uint32_t>(127 + steps - half) << 23);
    r.m = next;
    r.l = __fmul_rn(__fmul_rn(r.l, f0), f1);
    if (pv_done != nullptr) {  // there is an O
      r.ok = wait_for(pv_done, parity, status);
      r.ok = __all_sync(0xffffffffu, r.ok);
      if (!r.ok) return r;
      tc_fence_after();
#pragma unroll 1
      for (int e = 0; e < D / 16; ++e) {
        uint32_t o[16];
        tmem_ld16(to + 16 * e, o);
        tmem_arrived(o);
#pragma unroll
        for (int z = 0; z < 16; ++z)
          o[z] = __float_as_uint(__fmul_rn(__fmul_rn(__uint_as_float(o[z]), f0), f1));
        tmem_st16(to + 16 * e, o);
      }
    }
  }
  const float from = r.m == -INFINITY ? 0.0f : kRaise - r.m;
#pragma unroll 1
  for (int c0 = 0; c0 < kTile; c0 += 32) {
    uint32_t v[32], w[16];
    tmem_ld32(ts + c0, v);
    tmem_arrived(v);
#pragma unroll
    for (int e = 0; e < 32; e += 2) {
      const int c = c0 + e;
      const float lv = sc.lv[c / 16];
      r.l += ex2_whole(score(v[e], c, from)) + ex2_whole(score(v[e + 1], c + 1, from));
      w[e / 2] = half2_bits(__floats2half2_rn(ex2(score(v[e], c, lv + from)), ex2(score(v[e + 1], c + 1, lv + from))));
    }
    tmem_st16(ts + c0 / 2, w);
  }
  return r;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) kv_attention_prompt_kernel(const PromptParams p) {
  using S = Smem<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  BlockScales *scales = reinterpret_cast<BlockScales *>(smem + S::kScales);
  uint64_t *q_full = reinterpret_cast<uint64_t *>(smem + S::kBars);
  uint64_t *k_full = q_full + 1, *k_empty = k_full + kStages;
  uint64_t *v_full = k_empty + kStages, *v_empty = v_full + kStages;
  uint64_t *sc_full = v_empty + kStages;                       // [kSlots]
  uint64_t *s_full = sc_full + kSlots, *p_full = s_full + 2, *pv_done = p_full + 2;
  uint64_t *drained = pv_done + 2;
  uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(drained + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    mbar_init(q_full, 2 * kTile);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&k_full[s], 4 * 32);
      mbar_init(&k_empty[s], 1);
      mbar_init(&v_full[s], 4 * 32);
      mbar_init(&v_empty[s], 1);
    }
    for (int s = 0; s < kSlots; ++s) mbar_init(&sc_full[s], 32);
    for (int t = 0; t < 2; ++t) {
      mbar_init(&s_full[t], 1);
      mbar_init(&p_full[t], kTile);
      mbar_init(&pv_done[t], 1);
    }
    mbar_init(drained, 1);
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

  // the last row block of every sequence first (the longest under a causal
  // mask), then the one before it, ...
  unsigned i = blockIdx.x;
  const int h = static_cast<int>(i % p.cache.heads);
  i /= p.cache.heads;
  const int b = static_cast<int>(i % p.batch.B);
  const int from_end = static_cast<int>(i / p.batch.B);
  const int P = p.cache.page_tokens, G = p.group;
  int r0, r1, len;
  const bool fine = kv_sequence(p.batch, P, b, &r0, &r1, &len);
  if (!fine && threadIdx.x == 0) record_status(p.status, kStatusRange);
  const int n = r1 - r0, blocks = fine ? (n * G + 2 * kTile - 1) / (2 * kTile) : 0;

  // KV blocks that this CTA has been through, all in all and of each tile: the
  // counters of the stages' and tiles' barriers
  uint32_t done = 0, tiles_done[2] = {0, 0};
  // Positions that rows of row block rb see: [lo, hi), lo on a block boundary;
  // KV blocks of each tile (0: no rows, or none that see anything).  (A table
  // holds less than 2^31 positions.)
  int lo, hi, nb[2], total, row0;
  auto enter = [&](int rb) {
    row0 = rb * 2 * kTile;
    hi = 0;
    lo = first_seen(len - n + row0 / G, p.window) / kTile * kTile;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int first = row0 + t * kTile, last = first + kTile < n * G ? first + kTile : n * G;
      nb[t] = 0;
      if (first < last) {
        const int end = len - n + (last - 1) / G + 1;
        if (end > lo) nb[t] = (end - lo + kTile - 1) / kTile;
        if (end > hi) hi = end;
      }
    }
    total = nb[0] > nb[1] ? nb[0] : nb[1];
  };
  // The next row block's q overwrites this one's: every product has been
  // waited for by the softmax warps.  True when all warps are still in step.
  auto leave = [&](bool ok) -> bool {
    done += static_cast<uint32_t>(total);
    tiles_done[0] += static_cast<uint32_t>(nb[0]);
    tiles_done[1] += static_cast<uint32_t>(nb[1]);
    __syncwarp();
    return __syncthreads_and(ok) != 0;
  };
  auto stage = [&](int j) { return static_cast<int>((done + j) % kStages); };
  auto use = [&](int j) { return (done + j) / kStages; };  // of that stage
  bool ok = true;

  if (warp < kConvWarp0) {
    more_registers<kRegsSoftmax>();
    for (int rb = blocks - 1 - from_end; rb >= 0 && ok; rb -= p.row_blocks) {
      enter(rb);
      // ================================================ softmax
      const int t = warp >> 2, row = threadIdx.x & (kTile - 1);
      const int mine = t ? nb[1] : nb[0];
      const uint32_t before = t ? tiles_done[1] : tiles_done[0];
      const int gr = row0 + t * kTile + row;
      const bool have = gr < n * G;
      const int query = (have ? gr : n * G - 1) / G;
      const int64_t at = have ? (static_cast<int64_t>(r0 + query) * p.q_heads + h * G + (gr - query * G)) * D : 0;
      // q to shared memory, its largest value brought to [2^14, 2^15)
      float fac;
      {
        uint4 v[D / 8];
#pragma unroll
        for (int c = 0; c < D / 8; ++c)
          v[c] = have ? __ldcg(reinterpret_cast<const uint4 *>(p.q + at) + c) : make_uint4(0, 0, 0, 0);
        uint32_t peak = 0;
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          const uint32_t w[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t a = (w[e] << 16) & 0x7FFFFFFFu, c2 = w[e] & 0x7FFF0000u;
            peak = peak > a ? peak : a;
            peak = peak > c2 ? peak : c2;
          }
        }
        int k = 14 - (static_cast<int>(peak >> 23) - 127);
        k = k < -113 ? -113 : (k > 110 ? 110 : k);  // (finite ones need -113 at least)
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
      const int pos = len - n + query, first = first_seen(pos, p.window);
      float m = -INFINITY, l = 0.0f;  // m is whole
      for (int j = 0; j < mine && ok; ++j) {
        const int slot = static_cast<int>((done + j) % kSlots);
        const uint32_t tj = before + j;
        ok = wait_for(&sc_full[slot], ((done + j) / kSlots) & 1, p.status) && wait_for(&s_full[t], tj & 1, p.status);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        const BlockScales &sc = scales[slot];
        // visible columns of the block: [c_lo, c_hi)
        const int c_hi = pos + 1 - (lo + j * kTile), c_lo = first - (lo + j * kTile);
        bool part = c_hi < kTile || c_lo > 0;
#pragma unroll
        for (int s = 0; s < kSegs; ++s) part |= !(sc.iv[s] > 0.0f);
        // Twice over the scores, 32 columns at a time with the next ones on
        // their way: the row's maximum; then weights, written over scores that
        // have been read, and their sum.  A block that every row of the warp
        // sees whole takes the form without comparisons.
        auto weights = [&](auto masked_form) -> bool {
          constexpr bool kMasked = decltype(masked_form)::value;
          uint32_t buf[2][32];
          tmem_ld32(ts, buf[0]);
          float top = -INFINITY;  // of score + log2 vs
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t(&v)[32] = buf[q & 1];
            tmem_arrived(v);
            tmem_ld32(ts + 32 * ((q + 1) & 3), buf[(q + 1) & 1]);  // (the first ones again at the end)
#pragma unroll
            for (int s = 0; s < 2; ++s) {
              const float ks = sc.ks[2 * q + s];
              if (kMasked) {
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                  const int c = 32 * q + 16 * s + e;
                  if (c < c_lo || c >= c_hi || ks < 0.0f) v[16 * s + e] = 0xFF800000u;
                }
              }
              float x0 = __uint_as_float(v[16 * s]), x1 = __uint_as_float(v[16 * s + 1]);
#pragma unroll
              for (int e = 2; e < 14; e += 4) {
                x0 = max3(x0, __uint_as_float(v[16 * s + e]), __uint_as_float(v[16 * s + e + 1]));
                x1 = max3(x1, __uint_as_float(v[16 * s + e + 2]), __uint_as_float(v[16 * s + e + 3]));
              }
              x0 = max3(x0, __uint_as_float(v[16 * s + 14]), __uint_as_float(v[16 * s + 15]));
              // (0 * -inf of a fully hidden segment would be NaN, which fmaxf drops)
              top = fmaxf(top, __fmaf_rn(fmaxf(x0, x1), fac * fabsf(ks), sc.lv[2 * q + s]));
            }
          }
          // m follows where a score passes it by 2^kLazy (or is the row's
          // first), in whole steps, so that the row's sum and O are scaled
          // exactly
          const bool grow = top > m + kLazy;
          if (__any_sync(0xffffffffu, grow)) {
            const float next = grow ? ceilf(top) : m;
            const float down = fmaxf(m - next, -127.0f);  // m = -inf: f = 0
            const float f = m == next ? 1.0f : __uint_as_float(static_cast<uint32_t>(127 + static_cast<int>(down)) << 23);
            m = next;
            l *= f;
            if (j > 0) {
              const bool waited = wait_for(&pv_done[t], (tj - 1) & 1, p.status);
              if (!__all_sync(0xffffffffu, waited)) return false;
              tc_fence_after();
#pragma unroll 1
              for (int e = 0; e < D / 16; ++e) {
                uint32_t o[16];
                tmem_ld16(to + 16 * e, o);
                tmem_arrived(o);
#pragma unroll
                for (int z = 0; z < 16; ++z) o[z] = __float_as_uint(__fmul_rn(__uint_as_float(o[z]), f));
                tmem_st16(to + 16 * e, o);
              }
            }
          }
          const float from = m == -INFINITY ? 0.0f : kRaise - m;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t(&v)[32] = buf[q & 1];
            tmem_arrived(v);
            if (q < 3) tmem_ld32(ts + 32 * (q + 1), buf[(q + 1) & 1]);
            uint32_t w[16];
#pragma unroll
            for (int s = 0; s < 2; ++s) {
              const float ks = sc.ks[2 * q + s];
              const float c1 = fac * fabsf(ks), c0 = sc.lv[2 * q + s] + from;
              const uint64_t c11 = pair(c1, c1), c00 = pair(c0, c0);
              uint64_t sum = pair(0.0f, 0.0f);
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const int at = 16 * s + 2 * e, c = 32 * q + at;
                float x0, x1;
                unpair(fma2(pair(__uint_as_float(v[at]), __uint_as_float(v[at + 1])), c11, c00), x0, x1);
                if (kMasked) {
                  if (c < c_lo || c >= c_hi || ks < 0.0f) x0 = -INFINITY;
                  if (c + 1 < c_lo || c + 1 >= c_hi || ks < 0.0f) x1 = -INFINITY;
                }
                x0 = ex2(x0);
                x1 = ex2(x1);
                sum = add2(sum, pair(x0, x1));
                w[8 * s + e] = half2_bits(__floats2half2_rn(x0, x1));
              }
              float s0, s1;
              unpair(sum, s0, s1);
              l = __fmaf_rn(__fadd_rn(s0, s1), sc.iv[2 * q + s], l);
            }
            tmem_st16(ts + 16 * q, w);
          }
          return true;
        };
        if (!__any_sync(0xffffffffu, part)) {
          ok = weights(std::false_type{});
        } else {
          bool apart = false;
#pragma unroll
          for (int s = 0; s < kSegs; ++s) apart |= sc.iv[s] < 0.0f;
          if (apart) {
            const Row r = far_block<D>({m, l, true}, ts, to, fac, sc, c_lo, c_hi, j > 0 ? &pv_done[t] : nullptr,
                                       (tj - 1) & 1, p.status);
            m = r.m;
            l = r.l;
            ok = r.ok;
          } else {
            ok = weights(std::true_type{});
          }
        }
        if (!ok) break;
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&p_full[t]);
      }
      // ---- the tile's rows
      if (ok && mine > 0) {
        ok = wait_for(&pv_done[t], (before + mine - 1) & 1, p.status);
        ok = __all_sync(0xffffffffu, ok);
        tc_fence_after();
      }
      if (ok) {
        const float inv = l == 0.0f ? 0.0f : __fdiv_rn(1.0f, l);  // nothing visible: zeros
#pragma unroll
        for (int q = 0; q < D / 32; ++q) {
          uint32_t v[32];
          if (mine > 0) {
            tmem_ld32(to + 32 * q, v);
            tmem_arrived(v);
          }
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t x[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float a = mine > 0 ? __uint_as_float(v[8 * c + 2 * e]) * inv : 0.0f;
              const float d = mine > 0 ? __uint_as_float(v[8 * c + 2 * e + 1]) * inv : 0.0f;
              const __nv_bfloat162 y = __floats2bfloat162_rn(a, d);
              x[e] = *reinterpret_cast<const uint32_t *>(&y);
            }
            if (have)
              reinterpret_cast<uint4 *>(p.o + at)[4 * q + c] = make_uint4(x[0], x[1], x[2], x[3]);
          }
        }
      }
      tc_fence_before();
      ok = leave(ok);
    }
  } else if (warp < kMmaWarp) {
    // ================================================== int8 -> fp16
    fewer_registers<kRegsConvert>();
    const bool keys = warp < kValueWarp0;
    const int id = (warp & 3) * 32 + lane;  // thread of the group
    const int *table = p.batch.pages + static_cast<int64_t>(b) * p.batch.max_pages;
    const int64_t page_bytes = static_cast<int64_t>(p.cache.heads) * P * D;
    const int8_t *head = (keys ? p.cache.k_codes : p.cache.v_codes) + static_cast<int64_t>(h) * P * D;
    const int page_shift = 31 - __clz(P);
    auto page_of = [&](int j) -> int {  // of segment `lane` of block j
      const int tok = lo + j * kTile + 16 * lane;
      return lane < kSegs && j < total && tok < hi ? __ldcg(table + (tok >> page_shift)) : -1;
    };
    auto checked = [&](int page, int j) -> int {
      if (page >= 0 && page < p.cache.pages) return page;
      if (lane < kSegs && j < total && lo + j * kTile + 16 * lane < hi) record_status(p.status, kStatusRange);
      return -1;
    };
    // the 16 codes of row `r` of block j at chunk `chunk`; zeros where there is no page
    auto load16 = [&](int page, int j, int r, int chunk) -> uint4 {
      if (page < 0) return make_uint4(0, 0, 0, 0);
      const int row = (j * kTile + r) & (P - 1);  // (lo is a multiple of every page size)
      return __ldcg(reinterpret_cast<const uint4 *>(head + page * page_bytes + row * D) + chunk);
    };
    for (int rb = blocks - 1 - from_end; rb >= 0 && ok; rb -= p.row_blocks) {
      enter(rb);
      int page = checked(page_of(0), 0), next = page_of(1);
      if (keys) {
        constexpr int kLanes = D / 16;             // lanes of a row's 16-byte chunks
        constexpr int kRounds = D / 16;            // kTile rows in rounds of 128 / kLanes
        const int row = id / kLanes, chunk = id % kLanes;
        uint4 kr[kRounds];
        auto load = [&](int from, int j) {
#pragma unroll
          for (int it = 0; it < kRounds; ++it) {
            const int r = it * (128 / kLanes) + row;
            kr[it] = load16(__shfl_sync(0xffffffffu, from, r / 16), j, r, chunk);
          }
        };
        float ks = -1.0f, vs = 0.0f;  // of segment `lane`, the first warp's
        bool apart = false;           // a value scale far from others so far
        auto load_scales = [&](int from) {
          ks = -1.0f;
          if (id < kSegs && from >= 0) {
            ks = __ldcg(p.cache.k_scales + static_cast<int64_t>(from) * p.cache.heads + h);
            vs = __ldcg(p.cache.v_scales + static_cast<int64_t>(from) * p.cache.heads + h);
          }
        };
        load(page, 0);
        load_scales(page);
        // (a page that no row sees must not count as a scale far from the others)
        if (lo + 16 * lane + 16 <= first_seen(len - n + row0 / G, p.window)) vs = 1.0f;
        for (int j = 0; j < total; ++j) {
          const int st = stage(j);
          if (use(j) > 0) {  // the stage's last user has gone through
            ok = wait_for(&k_empty[st], (use(j) - 1) & 1, p.status);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
          }
          if (id < 32) {
            // (slot j % kSlots was last read for block j - 4, whose products
            // come before those of block j - 2 that k_empty waits for)
            BlockScales &sc = scales[(done + j) % kSlots];
            if (lane < kSegs) {
              sc.ks[lane] = ks;
              sc.lv[lane] = vs < kKvMinScale ? -60.0f : log2f(vs);
              apart |= ks >= 0.0f && far_scale(vs);
              // (a weight of 0 must stay 0: no NaN where the page is masked)
              sc.iv[lane] = apart ? -1.0f : ks < 0.0f ? 0.0f : vs < INFINITY ? __fdiv_rn(1.0f, vs) : 1.0f;
            }
            mbar_arrive(&sc_full[(done + j) % kSlots]);
          }
          page = checked(next, j + 1);
          next = page_of(j + 2);
          uint8_t *kt = smem + S::kK + st * S::kOperand;
#pragma unroll
          for (int it = 0; it < kRounds; ++it) {
            const int r = it * (128 / kLanes) + row;
            // lanes of the second panel store their second 16 bytes first:
            // other banks
            const bool swap = (chunk & 4) != 0;
            const uint32_t w[4] = {swap ? kr[it].z : kr[it].x, swap ? kr[it].w : kr[it].y,
                                   swap ? kr[it].x : kr[it].z, swap ? kr[it].y : kr[it].w};
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              const uint32_t a = w[2 * half] ^ 0x80808080u, c = w[2 * half + 1] ^ 0x80808080u;
              const int to = 2 * chunk + (half ^ static_cast<int>(swap));
              *reinterpret_cast<uint4 *>(kt + operand_offset(kTile, r, to)) =
                  make_uint4(codes01(a), codes23(a), codes01(c), codes23(c));
            }
          }
          fence_proxy_async_smem();
          mbar_arrive(&k_full[st]);
          load(page, j + 1);
          load_scales(page);
        }
      } else {
        // 8 tokens (an octet) by 16 columns per thread; D = 64: two warps
        const int octet = (lane & 7) + 8 * (warp & 1), chunk = (lane >> 3) + 4 * ((warp & 3) >> 1);
        const bool mine = chunk < D / 16;
        uint4 vr[8];
        auto load = [&](int from, int j) {
          const int pg = __shfl_sync(0xffffffffu, from, octet / 2);
#pragma unroll
          for (int e = 0; e < 8; ++e) vr[e] = load16(mine ? pg : -1, j, octet * 8 + e, chunk);
        };
        load(page, 0);
        for (int j = 0; j < total; ++j) {
          const int st = stage(j);
          if (use(j) > 0) {
            ok = wait_for(&v_empty[st], (use(j) - 1) & 1, p.status);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
          }
          page = checked(next, j + 1);
          next = page_of(j + 2);
          uint8_t *vt = smem + S::kV + st * S::kOperand;
          if (mine) {
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
                const int d = 16 * chunk + 4 * i4 + c;
                uint32_t o[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) o[e] = (c & 1) != 0 ? codes23(x[e][c >> 1]) : codes01(x[e][c >> 1]);
                *reinterpret_cast<uint4 *>(vt + operand_offset(D, d, octet)) = make_uint4(o[0], o[1], o[2], o[3]);
              }
            }
          }
          fence_proxy_async_smem();
          mbar_arrive(&v_full[st]);
          load(page, j + 1);
        }
      }
      ok = leave(ok);
    }
  } else {
    fewer_registers<kRegsMma>();
    uint32_t q_phase = 0;
    for (int rb = blocks - 1 - from_end; rb >= 0 && ok; rb -= p.row_blocks) {
      enter(rb);
      if (warp == kMmaWarp && lane == 0) {
        // ================================================ MMAs
        constexpr uint32_t kIdescS = (1u << 4) | ((kTile >> 3) << 17) | ((kTile >> 4) << 24);
        constexpr uint32_t kIdescO = (1u << 4) | ((D >> 3) << 17) | ((kTile >> 4) << 24);
        const uint32_t base = smem_u32(smem);
        ok = wait_for(q_full, q_phase, p.status);
        tc_fence_after();
        const uint32_t q0 = desc_low(base + S::kQ), k0 = desc_low(base + S::kK), v0 = desc_low(base + S::kV);
        auto scores = [&](int t, int st) {  // S_t = Q_t K^T, K of stage st
          const uint32_t a = q0 + t * (S::kOperand >> 4), k = k0 + st * (S::kOperand >> 4), d = tmem + t * kTile;
#pragma unroll
          for (int e = 0; e < D / 16; ++e) {  // 32 bytes of a panel's row each
            const uint32_t step = (e >> 2) * (kTile * 128 >> 4) + (e & 3) * 2;
            mma_smem(d, a + step, k + step, kIdescS, e != 0 ? 1u : 0u);
          }
          mma_commit(&s_full[t]);
        };
        auto values = [&](int t, int st, bool more) {  // O_t (+)= P_t V, V of stage st
          const uint32_t v = v0 + st * (S::kOperand >> 4), a = tmem + t * kTile, d = tmem + 2 * kTile + t * D;
#pragma unroll
          for (int e = 0; e < kTile / 16; ++e)
            mma_tmem(d, a + 8 * e, v + (e >> 2) * (D * 128 >> 4) + (e & 3) * 2, kIdescO, more || e != 0 ? 1u : 0u);
          mma_commit(&pv_done[t]);
        };
        for (int j = 0; j <= total && ok; ++j) {  // values of block j - 1, then scores of block j
          bool k_ready = false;
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (!ok) break;
            if (j > 0 && j - 1 < (t ? nb[1] : nb[0])) {
              ok = wait_for(&p_full[t], ((t ? tiles_done[1] : tiles_done[0]) + j - 1) & 1, p.status) &&
                   wait_for(&v_full[stage(j - 1)], use(j - 1) & 1, p.status);
              if (!ok) break;
              tc_fence_after();
              values(t, stage(j - 1), j > 1);
            }
            if (t == 1 && j > 0) mma_commit(&v_empty[stage(j - 1)]);  // both tiles' products with it
            if (j < (t ? nb[1] : nb[0])) {
              if (!k_ready) {
                ok = k_ready = wait_for(&k_full[stage(j)], use(j) & 1, p.status);
                if (!ok) break;
                tc_fence_after();
              }
              scores(t, stage(j));
            }
          }
          if (!ok) break;
          if (j < total) mma_commit(&k_empty[stage(j)]);
        }
      }
      ok = leave(ok);
      q_phase ^= 1u;
    }
    if (!ok && warp == kMmaWarp && lane == 0) {  // a wait gave up: the products under way end first
      mma_commit(drained);
      wait_for(drained, 0, p.status);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) tmem_dealloc(tmem, kTmemCols);
}

}  // namespace

bool kv_attention_prompt_fits(const KvCache &cache, const KvBatch &batch, const AttnArgs &args) {
  const int64_t most = (int64_t(1) << 31) - 1;
  const int64_t row_blocks = ceil_div(args.max_new * (args.q_heads / cache.heads), 2 * kTile);
  return batch.T <= (most - 512) / args.q_heads && row_blocks <= most / cache.heads && batch.B <= most / (row_blocks * cache.heads);
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
  p.window = static_cast<int>(args.window);
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
