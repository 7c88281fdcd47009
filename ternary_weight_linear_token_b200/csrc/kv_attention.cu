// kv_attention.cu -- attention over the 8-bit paged key/value cache.
//
// For a query row q (one query token and head) at position pos of its
// sequence, over the visible positions j <= pos (and j > pos - window):
//   s_j = scale * (q . kc_j) * ks(j),  o = sum_j e^{s_j} vs(j) vc_j / sum_j e^{s_j}
// with int8 codes kc, vc and one scale ks, vs per page and head.
//
// The int8 codes are exact in fp16, so the tensor cores multiply them
// (mma m16n8k16, fp32 sums) after a byte permute and one subtraction per two
// codes: the permute puts (code + 128) under the fp16 exponent of 1024, the
// subtraction takes 1152 away.  The tokens are the M axis (16 at a time, all
// in one page) and the query rows the N axis, so a decode step of 4 to 8
// query heads per key head fills a tile of 8 rows:
//   S^T = Kc Q^T            the codes of a thread's 16-byte loads are its A
//                           fragments (the order of the K axis is free)
//   O^T += Vc^T P^T         S^T's accumulators become P^T's B fragments by
//                           one 8 x 8 transpose
// q is scaled by a power of two per row so that fp16 holds it: bf16 values
// exactly, fp32 ones as a sum of two halves (22 bits), which take two
// neighbouring columns of the tile; fp32 P is split the same way.
// vs enters as log2(vs) added to the score: p' = 2^(s + log2 vs - m) with the
// running maximum m of that sum, so O += p' vc needs no further scale, while
// the row sum adds p' / vs.  A page of zeros (vs = 0) counts with log2 vs =
// -60 (scales far apart: attention.cuh).  p' is held 2^kRaise higher, and m may
// lag behind by kLazy: p' stays below 2^15, and fp16 rounds it by at most 2^-11
// of itself or, below fp16's normal numbers, by 2^-25: 2^-32 of the largest
// weight.
//
// A CTA's 4 warps take every 4th chunk of 32 tokens of its piece of the
// sequence, each with its own ring of chunks filled by bulk copies (K and V
// of a chunk are contiguous in a page), page numbers and scales fetched
// ahead; they join their sums in shared memory.  Few rows over a long cache
// are cut into pieces, which a second kernel joins in piece order; a short one
// into the CTAs of a cluster, which join by themselves (one launch and no
// workspace: 10.5 against 14.8 us a call for one sequence of 700 tokens, 15.6
// against 20.9 for 8 of 4000, 15.6 against 23.5 for 5 drafts each of 16 within
// a window of 1024).
// 48 sequences of up to 4096 tokens (124 MB): 39 us, 3.2 TB/s.  No unit is
// full (counters: HBM 41 %, issue slots 43 %, ALU 37 %): 10 warps an SM (12 is
// what registers and rings allow) wait in turn for their own results, shared
// memory and copies, in 1.6 waves.  Converting the codes is some 380 of the 840
// instructions that a chunk costs with its share of a CTA's start and end.
// Three CTAs per SM with two stages against two with three: 44 against 48 us;
// pieces for 5 CTAs per SM against 8: 40 against 44 us.
#include <atomic>

#include "attention.cuh"
#include "common.cuh"
#include "internal.h"

namespace bitnet {
namespace {

constexpr int kWarps = 4;
constexpr int kChunk = 32;       // tokens per ring stage

struct AttnParams {
  KvCache cache;
  KvBatch batch;
  const void *q;
  void *o;
  int q_heads, group;
  float scale_log2;
  int window;
  int row_tiles, pieces;
  int piece;           // tokens per piece, a multiple of kChunk
  bool cluster;        // the pieces are the CTAs of a cluster, which join them
  float *part_o;       // else, for several: [pieces][T * q_heads][D] for the joining kernel
  float2 *part_ml;     // [pieces][T * q_heads] (max, sum)
  int *status;
};

template <int D> struct Ring {
  static constexpr int kStages = D == 128 ? 2 : 4;
  static constexpr int kBytes = kChunk * D;            // K, and V, of a chunk
  static constexpr int kStageBytes = 2 * kBytes;
};
// per warp and stage: ks, log2 vs, 1 / vs of the chunk's two 16-token tiles
struct ChunkScales {
  float ks[2], lv[2], iv[2];
};
template <int D> constexpr size_t attn_smem() {
  return static_cast<size_t>(kWarps) * Ring<D>::kStages *
         (Ring<D>::kStageBytes + sizeof(ChunkScales) + sizeof(uint64_t));
}

// Positions that some of the queries i0..i1 of a sequence sees: [lo, hi),
// lo rounded down to a chunk.
__device__ __forceinline__ void visible(int len, int n, int i0, int i1, int window, int *lo, int *hi) {
  *hi = len - n + i1 + 1;
  *lo = first_seen(len - n + i0, window) / kChunk * kChunk;
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Transpose of an 8 x 8 matrix of halves held two per lane.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// *p of CTA `rank` of the cluster.
__device__ __forceinline__ float2 peer(const float2 *p, int rank) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];"
               : "=f"(v.x), "=f"(v.y)
               : "r"(mapa_shared(p, static_cast<uint32_t>(rank)))
               : "memory");
  return v;
}

// sum + f ml.y of a part with maximum and row sum ml, f = 2^(ml.x - top) (0
// for a part without a maximum); f can be 0 where the product is not.
__device__ __forceinline__ float add_share(float sum, float2 ml, float top, float f) {
  sum = __fmaf_rn(f, ml.y, sum);
  if (f == 0.0f && ml.y > 0.0f) sum += times_ex2(ml.y, ml.x - top);
  return sum;
}

template <typename T> __device__ __forceinline__ T lds(const void *p) { return *static_cast<const T *>(p); }

// One row tile of one piece.  TERMS: columns per query row (1 bf16, 2 fp32);
// NT: column tiles of 8.  APART: for value scales far apart (attention.cuh);
// the other form returns true when it has met some, and has stored nothing.
template <int D, int TERMS, int NT, bool APART>
__device__ __forceinline__ bool attend(const AttnParams &p, uint8_t *smem, int b, int h, int row_tile,
                                       int piece_index, int r0, int n, int len, uint32_t &phase,
                                       int &stage) {
  using R = Ring<D>;
  constexpr int kRows = 8 * NT / TERMS;
  constexpr int kSteps = D / 16;     // K steps of S^T; M tiles of O^T
  constexpr int kPer = 2 / TERMS;    // query rows per lane and column tile
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int P = p.cache.page_tokens, G = p.group, page_shift = 31 - __clz(P);
  uint8_t *ring = smem + warp * R::kStages * R::kStageBytes;
  ChunkScales *scales = reinterpret_cast<ChunkScales *>(smem + kWarps * R::kStages * R::kStageBytes) +
                        warp * R::kStages;
  uint64_t *full = reinterpret_cast<uint64_t *>(
                       smem + kWarps * R::kStages * (R::kStageBytes + sizeof(ChunkScales))) +
                   warp * R::kStages;

  // query rows of the tile: row = query * G + head of the group
  const int row0 = row_tile * kRows;
  const int rows = n * G - row0 < kRows ? n * G - row0 : kRows;
  const int query0 = row0 / G, query1 = (row0 + rows - 1) / G;  // of the first and last row
  int lo, hi;
  visible(len, n, query0, query1, p.window, &lo, &hi);
  if (p.pieces > 1) {
    lo = hi - lo > piece_index * p.piece ? lo + piece_index * p.piece : hi;
    if (hi - lo > p.piece) hi = lo + p.piece;
  }
  const int chunks = hi > lo ? (hi - lo + kChunk - 1) / kChunk : 0;
  if (chunks == 0 && p.part_o != nullptr) return false;  // the joining kernel knows

  // Lanes 0-3 fetch the chunk of the warp's round i (tile = lane & 1, K or V =
  // lane >> 1): the page number (-1 where there is none), ...
  const int *table = p.batch.pages + static_cast<int64_t>(b) * p.batch.max_pages;
  const int64_t page_bytes = static_cast<int64_t>(p.cache.heads) * P * D;
  const int8_t *codes = (lane >> 1 ? p.cache.v_codes : p.cache.k_codes) + static_cast<int64_t>(h) * P * D;
  const float *page_scales = (lane >> 1 ? p.cache.v_scales : p.cache.k_scales) + h;
  const int tok_lane = lo + warp * kChunk + 16 * (lane & 1);
  const int rounds = (chunks - warp + kWarps - 1) / kWarps;
  auto page_of = [&](int i) -> int {
    const int tok = tok_lane + i * (kWarps * kChunk);
    return lane < 4 && i < rounds && tok < hi ? __ldcg(table + (tok >> page_shift)) : -1;
  };
  // ... then its bytes into stage st (pages of 32 tokens and more: the first
  // tile's lanes copy both tiles), and its scale, -1 where there is no page.
  const bool whole = P >= kChunk;
  const uint32_t bytes = whole ? R::kBytes : R::kBytes / 2;
  auto issue = [&](int i, int page, int st) -> float {
    const int tok = tok_lane + i * (kWarps * kChunk);
    const bool wanted = lane < 4 && tok < hi;
    const bool ok = wanted && page >= 0 && page < p.cache.pages;
    if (wanted && !ok) record_status(p.status, kStatusRange);
    const unsigned copies = __ballot_sync(0xffffffffu, ok) & (whole ? 5u : 15u);
    if (lane == 0) mbar_arrive_expect_tx(&full[st], bytes * __popc(copies));
    __syncwarp();
    float s = -1.0f;
    if (ok) {
      s = __ldcg(page_scales + static_cast<int64_t>(page) * p.cache.heads);
      if ((copies >> lane) & 1u)
        bulk_g2s(ring + st * R::kStageBytes + (lane >> 1) * R::kBytes + (lane & 1) * (R::kBytes / 2),
                 codes + page * page_bytes + (tok & (P - 1)) * D, bytes, &full[st]);
    }
    return s;
  };
  bool far = false;  // lanes 2, 3: a scale far from others
  auto keep_scale = [&](int st, float s) {
    ChunkScales &k = scales[st];
    if (lane < 2) k.ks[lane] = s;
    if (lane == 2 || lane == 3) {
      // s = 0: a page of zeros; s < 0: no page, its tokens are not seen
      const bool some = !(s < kKvMinScale);
      k.lv[lane & 1] = some ? log2f(s) : -60.0f;
      if (!APART) {
        far |= s >= 0.0f && far_scale(s);
        // (a weight of 0 must stay 0: no NaN where the page is masked)
        k.iv[lane & 1] = some && s < INFINITY ? __fdiv_rn(1.0f, s) : 1.0f;
      }
    }
  };

  // ring: the first kStages chunks of this warp
  int next_page;
  {
    int page[R::kStages];
    float s[R::kStages];
#pragma unroll
    for (int i = 0; i < R::kStages; ++i) page[i] = page_of(i);
    next_page = page_of(R::kStages);
#pragma unroll
    for (int i = 0; i < R::kStages; ++i)
      if (i < rounds) s[i] = issue(i, page[i], (stage + i) % R::kStages);
#pragma unroll
    for (int i = 0; i < R::kStages; ++i)
      if (i < rounds) {
        // (a first tile that no row sees must not count as a scale far from the others)
        const bool unseen = i == 0 && lane == 2 && tok_lane + 16 <= first_seen(len - n + query0, p.window);
        keep_scale((stage + i) % R::kStages, unseen ? 1.0f : s[i]);
      }
  }

  // q as B fragments: column g of column tile j is row j * 8 / TERMS + g / TERMS
  uint32_t qf[NT][kSteps][2];
  float fac[NT][kPer];     // score factor of the lane's rows (columns 2t, 2t + 1)
  int pos[NT][kPer], first[NT][kPer];  // the last and first positions they see; no such row: -1, 0
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int row = row0 + j * (8 / TERMS) + g / TERMS, query = row / G;
    const bool have = row < row0 + rows;
    const int64_t at = (static_cast<int64_t>(r0 + query) * p.q_heads + h * G + (row - query * G)) * D;
    const int place = have ? len - n + query : -1;
    float v[D / 4];
    float peak = 0.0f;
#pragma unroll
    for (int c = 0; c < D / 64; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if (have) {
          const int64_t e = at + 64 * c + 16 * t + 4 * i;
          if (TERMS == 2) {
            const float4 f = __ldcg(reinterpret_cast<const float4 *>(static_cast<const float *>(p.q) + e));
            x[0] = f.x; x[1] = f.y; x[2] = f.z; x[3] = f.w;
          } else {
            const uint2 u = __ldcg(reinterpret_cast<const uint2 *>(static_cast<const __nv_bfloat16 *>(p.q) + e));
            x[0] = __uint_as_float(u.x << 16); x[1] = __uint_as_float(u.x & 0xFFFF0000u);
            x[2] = __uint_as_float(u.y << 16); x[3] = __uint_as_float(u.y & 0xFFFF0000u);
          }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          v[(c * 4 + i) * 4 + e] = x[e];
          peak = fmaxf(peak, fabsf(x[e]));
        }
      }
    peak = fmaxf(peak, __shfl_xor_sync(0xffffffffu, peak, 1));
    peak = fmaxf(peak, __shfl_xor_sync(0xffffffffu, peak, 2));
    // 2^k brings the row's largest value into [2^14, 2^15)
    int k = 14 - (static_cast<int>(__float_as_uint(peak) >> 23) - 127);
    k = k < -113 ? -113 : (k > 110 ? 110 : k);  // (finite ones need -113 at least)
    const float up = __uint_as_float(static_cast<uint32_t>(127 + k) << 23);
    const float f = __fmul_rn(p.scale_log2, __uint_as_float(static_cast<uint32_t>(127 - k) << 23));
#pragma unroll
    for (int s = 0; s < kSteps; ++s)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float a = __fmul_rn(v[s * 4 + 2 * r], up), c = __fmul_rn(v[s * 4 + 2 * r + 1], up);
        __half2 x = __floats2half2_rn(a, c);
        if (TERMS == 2 && (g & 1) != 0) {
          const float2 hi2 = __half22float2(x);
          x = __floats2half2_rn(__fsub_rn(a, hi2.x), __fsub_rn(c, hi2.y));
        }
        qf[j][s][r] = half2_bits(x);
      }
#pragma unroll
    for (int r = 0; r < kPer; ++r) {
      const int col = 2 * t + r;
      fac[j][r] = __shfl_sync(0xffffffffu, f, col * 4);
      pos[j][r] = __shfl_sync(0xffffffffu, place, col * 4);
      first[j][r] = first_seen(pos[j][r], p.window);
    }
  }

  float acc[NT][kSteps][4];
  float m[NT][kPer], l[NT][kPer];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
#pragma unroll
    for (int s = 0; s < kSteps; ++s)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[j][s][e] = 0.0f;
#pragma unroll
    for (int r = 0; r < kPer; ++r) {
      m[j][r] = -INFINITY;
      l[j][r] = 0.0f;
    }
  }
  // positions that every row of the tile sees need no mask
  // (columns past the last row hold zeros and are not stored)
  const int all_hi = len - n + query0 + 1, all_lo = first_seen(len - n + query1, p.window);

  __syncwarp();
#pragma unroll 1
  for (int i = 0; i < rounds; ++i) {
    const int st = stage;
    stage = stage + 1 == R::kStages ? 0 : stage + 1;
    const bool ok = wait_for(&full[st], (phase >> st) & 1u, p.status);
    if (!__all_sync(0xffffffffu, ok)) {  // the copies under way end first (again with a limit); the rows are NaN
#pragma unroll 1
      for (int k = 0; k < R::kStages && i + k < rounds; ++k) {
        stage = (st + k) % R::kStages;
        wait_for(&full[stage], (phase >> stage) & 1u, p.status);
        phase ^= 1u << stage;
      }
      stage = (stage + 1) % R::kStages;
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int r = 0; r < kPer; ++r) l[j][r] = __uint_as_float(0x7FC00000u);
      break;
    }
    phase ^= 1u << st;
    const uint8_t *kt = ring + st * R::kStageBytes;
    const uint8_t *vt = kt + R::kBytes;
    const int tok0 = lo + (i * kWarps + warp) * kChunk;

    // ---- scores (log2) of the chunk's two tiles: [tile][j][row of lane][token g, g + 8]
    float s2[2][NT][kPer][2];
#pragma unroll
    for (int tile = 0; tile < 2; ++tile) {
      float sc[NT][4];
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[j][e] = 0.0f;
#pragma unroll
      for (int q = 0; q < D / 64; ++q) {
        const uint4 a = lds<uint4>(kt + (tile * 16 + g) * D + 64 * q + 16 * t);
        const uint4 a8 = lds<uint4>(kt + (tile * 16 + g + 8) * D + 64 * q + 16 * t);
        const uint32_t w[4] = {a.x, a.y, a.z, a.w}, w8[4] = {a8.x, a8.y, a8.z, a8.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t u = w[i] ^ 0x80808080u, u8 = w8[i] ^ 0x80808080u;
          const uint32_t a0 = codes01(u), a1 = codes01(u8), a2 = codes23(u), a3 = codes23(u8);
#pragma unroll
          for (int j = 0; j < NT; ++j)
            mma_f16(sc[j], a0, a1, a2, a3, qf[j][q * 4 + i][0], qf[j][q * 4 + i][1]);
        }
      }
      const float ks = scales[st].ks[tile], lv = scales[st].lv[tile];
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int r = 0; r < kPer; ++r)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float x = TERMS == 2 ? sc[j][2 * e] + sc[j][2 * e + 1] : sc[j][2 * e + r];
            s2[tile][j][r][e] = __fmaf_rn(x, ks * fac[j][r], lv);
          }
    }
    // not seen by all rows: compare (one branch for the chunk)
    if (tok0 + kChunk > all_hi || tok0 < all_lo || tok0 + kChunk > hi || scales[st].ks[0] < 0.0f ||
        scales[st].ks[1] < 0.0f) {
#pragma unroll 1
      for (int tile = 0; tile < 2; ++tile) {
        const int at = tok0 + 16 * tile + g;
        const bool there = !(scales[st].ks[tile] < 0.0f);
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int r = 0; r < kPer; ++r)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (!(there && at + 8 * e <= pos[j][r] && at + 8 * e >= first[j][r] && at + 8 * e < hi)) {
                if (tile == 0)
                  s2[0][j][r][e] = -INFINITY;
                else
                  s2[1][j][r][e] = -INFINITY;
              }
      }
    }

    // ---- running maximum
    bool grow = false;
    float top[NT][kPer];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int r = 0; r < kPer; ++r) {
        float x = fmaxf(fmaxf(s2[0][j][r][0], s2[0][j][r][1]), fmaxf(s2[1][j][r][0], s2[1][j][r][1]));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
        top[j][r] = x;
        grow |= x > m[j][r] + kLazy;  // also the first finite score (m = -inf)
      }
    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        float f[kPer];
#pragma unroll
        for (int r = 0; r < kPer; ++r) {
          const float to = fmaxf(m[j][r], top[j][r]);
          f[r] = m[j][r] == to ? 1.0f : ex2(m[j][r] - to);
          l[j][r] = APART && f[r] == 0.0f && l[j][r] > 0.0f ? times_ex2(l[j][r], m[j][r] - to) : l[j][r] * f[r];
          m[j][r] = to;
        }
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[j][s][e] *= f[(e & 1) % kPer];
      }
    }

    // ---- weights, row sums and O^T
    float from[NT][kPer];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int r = 0; r < kPer; ++r) from[j][r] = m[j][r] == -INFINITY ? 0.0f : m[j][r] - kRaise;
#pragma unroll
    for (int tile = 0; tile < 2; ++tile) {
      const float lv = APART ? scales[st].lv[tile] : 0.0f, iv = APART ? 0.0f : scales[st].iv[tile];
      auto share = [&](float weight, float score, float &sum) {
        if (APART)
          sum += ex2_whole(score - lv);
        else
          sum = __fmaf_rn(weight, iv, sum);
      };
      uint32_t pf[NT][2];
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          __half2 x;
          if (TERMS == 2) {
            const float a = ex2(s2[tile][j][0][e] - from[j][0]);
            share(a, s2[tile][j][0][e] - from[j][0], l[j][0]);
            const float hi_part = __half2float(__float2half_rn(a));
            x = __floats2half2_rn(hi_part, a - hi_part);
          } else {
            float a[2];
#pragma unroll
            for (int r = 0; r < kPer; ++r) {
              a[r] = ex2(s2[tile][j][r][e] - from[j][r]);
              share(a[r], s2[tile][j][r][e] - from[j][r], l[j][r]);
            }
            x = __floats2half2_rn(a[0], a[kPer - 1]);
          }
          pf[j][e] = transpose8(half2_bits(x));
        }
      constexpr int kWords = D / 32;  // 32-bit words of a lane's columns
      uint32_t w[4][kWords];          // tokens 2t, 2t + 1, 2t + 8, 2t + 9
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint8_t *src = vt + (tile * 16 + 2 * t + (k & 1) + 8 * (k >> 1)) * D + g * (D / 8);
        if (D == 128) {
          const uint4 x = lds<uint4>(src);
          w[k][0] = x.x; w[k][1] = x.y; w[k][kWords - 2] = x.z; w[k][kWords - 1] = x.w;
        } else {
          const uint2 x = lds<uint2>(src);
          w[k][0] = x.x; w[k][1] = x.y;
        }
      }
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        uint32_t x[2][2];  // [token pair][columns 0 1 | 2 3]: bytes col0 a, b, col1 a, b
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const uint32_t a = w[2 * q][i] ^ 0x80808080u, c2 = w[2 * q + 1][i] ^ 0x80808080u;
          x[q][0] = __byte_perm(a, c2, 0x5140);
          x[q][1] = __byte_perm(a, c2, 0x7362);
        }
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const uint32_t a0 = codes01(x[0][q]), a1 = codes23(x[0][q]);
          const uint32_t a2 = codes01(x[1][q]), a3 = codes23(x[1][q]);
#pragma unroll
          for (int j = 0; j < NT; ++j) mma_f16(acc[j][2 * i + q], a0, a1, a2, a3, pf[j][0], pf[j][1]);
        }
      }
    }

    // ---- refill this stage
    __syncwarp();  // every lane has read it
    const int ahead = i + R::kStages;
    if (ahead < rounds) {
      const int page = next_page;
      next_page = page_of(ahead + 1);
      keep_scale(st, issue(ahead, page, st));
      __syncwarp();
    }
  }

  // ---- join the warps: [warp][row][D] sums, [warp][row] (m, l)
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int r = 0; r < kPer; ++r) {
      l[j][r] += __shfl_xor_sync(0xffffffffu, l[j][r], 4);
      l[j][r] += __shfl_xor_sync(0xffffffffu, l[j][r], 8);
      l[j][r] += __shfl_xor_sync(0xffffffffu, l[j][r], 16);
    }
  if (__syncthreads_or(far)) return true;  // (the rings are idle)
  float *so = reinterpret_cast<float *>(smem);
  float2 *sml = reinterpret_cast<float2 *>(so + kWarps * kRows * D);
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int r = 0; r < kPer; ++r) {
      const int row = j * (8 / TERMS) + (2 * t + r) / TERMS;
      if (g == 0) sml[warp * kRows + row] = make_float2(m[j][r], l[j][r]);
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        // M tile s: columns d, d + 1 of the head
        const int d = g * (D / 8) + 2 * s;
        float2 x;
        if (TERMS == 2)
          x = make_float2(acc[j][s][0] + acc[j][s][1], acc[j][s][2] + acc[j][s][3]);
        else
          x = make_float2(acc[j][s][r], acc[j][s][2 + r]);
        *reinterpret_cast<float2 *>(so + (warp * kRows + row) * D + d) = x;
      }
    }
  __syncthreads();
  float *co = reinterpret_cast<float *>(sml + kWarps * kRows);  // the CTA's rows, for its cluster
  float2 *cml = reinterpret_cast<float2 *>(co + kRows * D);
  auto row_of = [&](int row) -> int64_t {
    const int query = (row0 + row) / G;
    return static_cast<int64_t>(r0 + query) * p.q_heads + h * G + (row0 + row - query * G);
  };
  auto store = [&](int64_t out_row, int d, float x, float y, float sum) {
    const float inv = sum == 0.0f ? 0.0f : __fdiv_rn(1.0f, sum);  // nothing visible: zeros
    if (TERMS == 2)
      *reinterpret_cast<float2 *>(static_cast<float *>(p.o) + out_row * D + d) = make_float2(x * inv, y * inv);
    else
      *reinterpret_cast<__nv_bfloat162 *>(static_cast<__nv_bfloat16 *>(p.o) + out_row * D + d) =
          __floats2bfloat162_rn(x * inv, y * inv);
  };
  for (int i = threadIdx.x; i < kRows * D / 2; i += kWarps * 32) {
    const int row = i / (D / 2), d = i % (D / 2) * 2;
    if (row >= rows) break;
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sml[w * kRows + row].x);
    float x = 0.0f, y = 0.0f, sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float2 ml = sml[w * kRows + row];
      const float f = ml.x == -INFINITY ? 0.0f : ex2(ml.x - top);
      const float2 v = *reinterpret_cast<const float2 *>(so + (w * kRows + row) * D + d);
      x = __fmaf_rn(f, v.x, x);
      y = __fmaf_rn(f, v.y, y);
      sum = APART ? add_share(sum, ml, top, f) : __fmaf_rn(f, ml.y, sum);
    }
    if (p.cluster) {
      *reinterpret_cast<float2 *>(co + row * D + d) = make_float2(x, y);
      if (d == 0) cml[row] = make_float2(top, sum);
      continue;
    }
    const int64_t out_row = row_of(row);
    if (p.part_o != nullptr) {
      const int64_t at = static_cast<int64_t>(piece_index) * p.batch.T * p.q_heads + out_row;
      *reinterpret_cast<float2 *>(p.part_o + at * D + d) = make_float2(x, y);
      if (d == 0) p.part_ml[at] = make_float2(top, sum);
    } else {
      store(out_row, d, x, y, sum);
    }
  }
  if (p.cluster) {  // this CTA's share of the rows, over the pieces in order
    cluster_sync();
    for (int i = static_cast<int>(threadIdx.x) + piece_index * kWarps * 32; i < rows * D / 2; i += p.pieces * kWarps * 32) {
      const int row = i / (D / 2), d = i % (D / 2) * 2;
      float top = -INFINITY;
      for (int s = 0; s < p.pieces; ++s) top = fmaxf(top, peer(cml + row, s).x);
      float x = 0.0f, y = 0.0f, sum = 0.0f;
      for (int s = 0; s < p.pieces; ++s) {
        const float2 ml = peer(cml + row, s), v = peer(reinterpret_cast<const float2 *>(co + row * D + d), s);
        const float f = ml.x == -INFINITY ? 0.0f : ex2(ml.x - top);
        x = __fmaf_rn(f, v.x, x);
        y = __fmaf_rn(f, v.y, y);
        sum = add_share(sum, ml, top, f);
      }
      store(row_of(row), d, x, y, sum);
    }
    cluster_sync();  // the others have read this CTA's
  }
  return false;
}

// The form for value scales far apart.  (A function of its own, so that the
// other form keeps its registers: 39.4 against 40.5 us for 48 sequences of up
// to 4096 tokens.)
struct RingState {
  uint32_t phase;
  int stage;
};
template <int D, int TERMS, int NT>
__device__ __noinline__ RingState attend_apart(const AttnParams &p, uint8_t *smem, int b, int h, int row_tile,
                                               int piece_index, int r0, int n, int len, RingState ring) {
  attend<D, TERMS, NT, true>(p, smem, b, h, row_tile, piece_index, r0, n, len, ring.phase, ring.stage);
  return ring;
}

template <int D, int TERMS, int NT>
__global__ void __launch_bounds__(kWarps * 32, 3) kv_attention_kernel(const __grid_constant__ AttnParams p) {
  extern __shared__ __align__(128) uint8_t smem[];
  using R = Ring<D>;
  uint64_t *full = reinterpret_cast<uint64_t *>(
      smem + kWarps * R::kStages * (R::kStageBytes + sizeof(ChunkScales)));
  if (threadIdx.x < kWarps * R::kStages) mbar_init(&full[threadIdx.x], 1);
  fence_barrier_init();
  __syncthreads();
  pdl_wait();
  pdl_launch_dependents();
  constexpr int kRows = 8 * NT / TERMS;
  // piece fastest, then head, row tile, sequence
  unsigned i = blockIdx.x;
  const int piece = static_cast<int>(i % p.pieces);
  i /= p.pieces;
  const int h = static_cast<int>(i % p.cache.heads);
  i /= p.cache.heads;
  const int first_tile = static_cast<int>(i % p.row_tiles);
  const int b = static_cast<int>(i / p.row_tiles);
  int r0, r1, len;
  if (!kv_sequence(p.batch, p.cache.page_tokens, b, &r0, &r1, &len)) {
    if (threadIdx.x == 0) record_status(p.status, kStatusRange);
    return;
  }
  const int n = r1 - r0, tiles = (n * p.group + kRows - 1) / kRows;
  uint32_t phase = 0;  // bit s: the parity of the warp's stage s to wait for next
  int stage = 0;       // its next stage
  for (int rt = first_tile; rt < tiles; rt += p.row_tiles) {
    if (attend<D, TERMS, NT, false>(p, smem, b, h, rt, piece, r0, n, len, phase, stage)) {
      const RingState ring = attend_apart<D, TERMS, NT>(p, smem, b, h, rt, piece, r0, n, len, {phase, stage});
      phase = ring.phase;
      stage = ring.stage;
    }
    fence_proxy_async_smem();  // the joined sums lie where the next bulk copies go
    __syncthreads();
  }
}

// Joins the pieces of one query row (a CTA each), in piece order.
template <int D, bool F32>
__global__ void __launch_bounds__(kWarps * 32) kv_join_kernel(const AttnParams p, int rows_per_tile) {
  __shared__ int seq;
  __shared__ float so[kWarps][D];
  __shared__ float weight[kWarps * 32], tops[kWarps], sums[kWarps];
  pdl_wait();
  pdl_launch_dependents();
  const int row = blockIdx.x;               // token * q_heads + head
  const int t = row / p.q_heads;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int b = t;
  if (p.batch.offsets != nullptr) {
    if (threadIdx.x == 0) seq = -1;
    __syncthreads();
    for (int i = threadIdx.x; i < p.batch.B; i += kWarps * 32)
      if (p.batch.offsets[i] <= t && t < p.batch.offsets[i + 1]) seq = i;
    __syncthreads();
    b = seq;
    if (b < 0) return;  // a row of no sequence: left as it is
  }
  int r0, r1, len;
  if (!kv_sequence(p.batch, p.cache.page_tokens, b, &r0, &r1, &len)) return;
  const int n = r1 - r0;
  const int in = (t - r0) * p.group + row % p.q_heads % p.group;
  const int row0 = in / rows_per_tile * rows_per_tile;
  const int last = row0 + rows_per_tile < n * p.group ? row0 + rows_per_tile : n * p.group;
  int lo, hi;
  visible(len, n, row0 / p.group, (last - 1) / p.group, p.window, &lo, &hi);
  int pieces = hi > lo ? (hi - lo + p.piece - 1) / p.piece : 0;
  if (pieces > p.pieces) pieces = p.pieces;

  // weights of 128 pieces at a time (their maxima and sums fetched together),
  // then their rows, a warp every 4th, several in flight
  constexpr int kPer = D / 32;
  const int64_t stride = p.batch.T * p.q_heads;
  float top = -INFINITY, sum = 0.0f, x[kPer];
#pragma unroll
  for (int e = 0; e < kPer; ++e) x[e] = 0.0f;
  for (int i0 = 0; i0 < pieces; i0 += kWarps * 32) {
    const int mine = i0 + threadIdx.x;
    const float2 ml = mine < pieces ? p.part_ml[mine * stride + row] : make_float2(-INFINITY, 0.0f);
    __syncthreads();  // the last round's weights have been read
    const unsigned key = __float_as_uint(ml.x);  // (order of floats as integers, NaN aside)
    const int ordered = static_cast<int>(key ^ ((key >> 31) != 0 ? 0x7FFFFFFFu : 0u));
    const int best = __reduce_max_sync(0xffffffffu, ordered);
    if (lane == 0) tops[warp] = __uint_as_float(static_cast<unsigned>(best) ^ (best < 0 ? 0x7FFFFFFFu : 0u));
    __syncthreads();
    float to = top;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) to = fmaxf(to, tops[w]);
    const float old = top == -INFINITY ? 0.0f : ex2(top - to);
    // (a piece without a maximum has a sum of 0, or of NaN, which goes on)
    const float f = ml.x == -INFINITY ? (ml.y == 0.0f ? 0.0f : ml.y) : ex2(ml.x - to);
    weight[threadIdx.x] = f;
    __syncthreads();
    float part = f == 0.0f && ml.y > 0.0f ? times_ex2(ml.y, ml.x - to) : f * ml.y;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) part += __shfl_xor_sync(0xffffffffu, part, o);
    sum = old == 0.0f && sum > 0.0f ? times_ex2(sum, top - to) + part : __fmaf_rn(sum, old, part);  // this warp's
    top = to;
#pragma unroll
    for (int e = 0; e < kPer; ++e) x[e] *= old;
    const int n_here = pieces - i0 < kWarps * 32 ? pieces - i0 : kWarps * 32;
#pragma unroll 4
    for (int i = warp; i < n_here; i += kWarps) {
      const float *src = p.part_o + ((i0 + i) * stride + row) * D + lane * kPer;
#pragma unroll
      for (int e = 0; e < kPer; ++e) x[e] = __fmaf_rn(weight[i], src[e], x[e]);
    }
  }
#pragma unroll
  for (int e = 0; e < kPer; ++e) so[warp][lane * kPer + e] = x[e];
  if (lane == 0) sums[warp] = sum;
  __syncthreads();
  for (int d = threadIdx.x; d < D; d += kWarps * 32) {
    float y = 0.0f, z = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      y += so[w][d];
      z += sums[w];
    }
    const float out = z == 0.0f ? 0.0f : __fdiv_rn(y, z);  // nothing visible: zeros
    const int64_t at = static_cast<int64_t>(row) * D + d;    // (rows fit 32 bits, values don't)
    if (F32)
      static_cast<float *>(p.o)[at] = out;
    else
      static_cast<__nv_bfloat16 *>(p.o)[at] = __float2bfloat16_rn(out);
  }
}

// How a call is cut: column tiles per CTA, row tiles per sequence, pieces.
struct AttnPlan {
  int nt, rows;
  int64_t row_tiles, piece, pieces;
  bool cluster;
};
constexpr int64_t kSms = 148;
// A cluster of 8 spares the second launch but has longer pieces.  bf16, 20/5
// heads of 128, cluster against pieces, us:
//   span       256         1024         4096         8192         16384
//   1 seq.   6.5 / 7.7   6.8 /  8.0  11.3 / 10.4  17.1 / 13.8  28.7 / 23.7
//   4 seq.   6.7 / 7.7   8.2 /  9.6  13.8 / 18.9  21.2 / 25.6  35.3 / 35.3
//   16 seq.  7.6 / 9.2  13.1 / 18.6  27.6 / 34.3  47.1 / 51.2  80.9 / 81.9
// So up to a span of 4096 (and a window's or a page's rounding), where the
// pieces are 512 tokens; with fewer CTAs a cluster, pieces of up to 1024.
constexpr int64_t kClusterSpan = 4096 + 128, kClusterPiece = 1024 + 32;
AttnPlan plan_of(const KvCache &cache, const KvBatch &batch, const AttnArgs &args) {
  AttnPlan a;
  const int terms = args.kind == kF32 ? 2 : 1;
  const int64_t G = args.q_heads / cache.heads;
  const int64_t need = G * (args.max_new < 1 ? 1 : args.max_new);
  a.nt = need * terms > 8 ? 2 : 1;
  a.rows = 8 * a.nt / terms;
  a.row_tiles = ceil_div(need, a.rows);
  int64_t span = batch.max_pages * cache.page_tokens;
  if (args.window > 0 && args.window + a.rows + kChunk < span) span = args.window + a.rows + kChunk;
  const int64_t units = batch.B * cache.heads * a.row_tiles;
  const int64_t target = kSms * 5;
  int64_t piece = ceil_div(ceil_div(span * units, target), 128) * 128;
  if (piece < 128) piece = 128;
  a.pieces = ceil_div(span, piece);
  if (a.pieces <= 1 || units >= target) {
    a.pieces = 1;
    piece = (int64_t(1) << 30);
  }
  // A short span for few rows: up to 8 pieces as a cluster, which join in the
  // same launch.  Only while all of them run at once: the CTAs of a cluster
  // wait for each other.
  a.cluster = false;
  if (a.pieces > 1 && span <= kClusterSpan) {
    int64_t size = 1;
    while (size < 8 && size * 128 < span && units * size * 2 <= kSms * 3) size *= 2;
    if (size > 1 && span <= size * kClusterPiece) {
      a.cluster = true;
      a.pieces = size;
      piece = ceil_div(ceil_div(span, size), 128) * 128;
    }
  }
  a.piece = piece;
  return a;
}
size_t align256(size_t n) { return (n + 255) & ~size_t(255); }

template <int D, int TERMS>
cudaError_t launch(const AttnParams &p, const AttnPlan &a, const LaunchCtx &ctx) {
  const int64_t blocks = p.batch.B * a.row_tiles * p.cache.heads * a.pieces;
  auto kernel = a.nt == 2 ? kv_attention_kernel<D, TERMS, 2> : kv_attention_kernel<D, TERMS, 1>;
  constexpr size_t smem = attn_smem<D>();
  static std::atomic<uint64_t> ready[2];  // bit d: device d allows the kernel its shared memory
  cudaError_t e = allow_smem(kernel, smem, ready[a.nt - 1], ctx);
  if (e != cudaSuccess) return e;
  if (a.cluster)
    return launch_k_cluster(kernel, dim3(static_cast<unsigned>(blocks)), dim3(kWarps * 32), smem,
                            static_cast<unsigned>(a.pieces), ctx, p);
  e = launch_k(kernel, dim3(static_cast<unsigned>(blocks)), dim3(kWarps * 32), smem, ctx, p);
  if (e != cudaSuccess || a.pieces == 1) return e;
  return launch_k(kv_join_kernel<D, TERMS == 2>, dim3(static_cast<unsigned>(p.batch.T * p.q_heads)),
                  dim3(kWarps * 32), 0, ctx, p, a.rows);
}

// Prompts of bf16 queries go to the tcgen05 kernel, by their rows alone.  One
// sequence, 20/5 heads of 128, that kernel against the one above, us:
//   new 32 of 2048      54 / 18      of 8192   178 /  43    of 60000  1261 /  148
//   new 128 of 128      19 / 11      of 2048    63 /  35    of 60000  1417 /  535
//   new 512 of 512      28 / 32      of 4096   110 / 197    of 60000  1417 / 2279
//   new 2048 of 2048    67 / 185     new 4096 of 4096   159 / 591
// It does not split the keys, so short prompts behind long prefixes, which leave
// most SMs without a CTA, are better served by the other one; the rule does not
// look at that.
bool use_prompt(const KvCache &cache, const AttnArgs &args) {
  return args.kind == kBF16 && args.max_new * (args.q_heads / cache.heads) >= 128;
}

}  // namespace

size_t kv_attention_workspace(const KvCache &cache, const KvBatch &batch, const AttnArgs &args) {
  if (use_prompt(cache, args)) return 0;
  const AttnPlan a = plan_of(cache, batch, args);
  if (a.pieces == 1 || a.cluster) return 0;
  const size_t rows = static_cast<size_t>(a.pieces) * batch.T * args.q_heads;
  return align256(rows * cache.head_dim * sizeof(float)) + align256(rows * sizeof(float2));
}

bool kv_attention_fits(const KvCache &cache, const KvBatch &batch, const AttnArgs &args) {
  if (use_prompt(cache, args)) return kv_attention_prompt_fits(cache, batch, args);
  const AttnPlan a = plan_of(cache, batch, args);
  const int64_t most = (int64_t(1) << 31) - 1;
  return a.row_tiles <= most && batch.B * a.row_tiles <= most / cache.heads &&
         batch.B * a.row_tiles * cache.heads <= most / a.pieces &&
         batch.T <= (most - 512) / args.q_heads;
}

cudaError_t launch_kv_attention(const KvCache &cache, const KvBatch &batch, const AttnArgs &args,
                                void *workspace, const LaunchCtx &ctx) {
  if (use_prompt(cache, args)) return launch_kv_attention_prompt(cache, batch, args, ctx);
  const AttnPlan a = plan_of(cache, batch, args);
  AttnParams p = {};
  p.cache = cache;
  p.batch = batch;
  p.q = args.Q;
  p.o = args.O;
  p.q_heads = args.q_heads;
  p.group = args.q_heads / cache.heads;
  p.scale_log2 = args.scale * kLog2e;
  p.window = static_cast<int>(args.window);
  p.row_tiles = static_cast<int>(a.row_tiles);
  p.pieces = static_cast<int>(a.pieces);
  p.piece = static_cast<int>(a.piece);
  p.status = ctx.status;
  p.cluster = a.cluster;
  if (a.pieces > 1 && !a.cluster) {
    const size_t rows = static_cast<size_t>(a.pieces) * batch.T * args.q_heads;
    p.part_o = static_cast<float *>(workspace);
    p.part_ml = reinterpret_cast<float2 *>(static_cast<uint8_t *>(workspace) +
                                           align256(rows * cache.head_dim * sizeof(float)));
  }
  if (args.kind == kF32)
    return cache.head_dim == 128 ? launch<128, 2>(p, a, ctx) : launch<64, 2>(p, a, ctx);
  return cache.head_dim == 128 ? launch<128, 1>(p, a, ctx) : launch<64, 1>(p, a, ctx);
}

}  // namespace bitnet
