// attention.cuh -- what the attention kernels over the 8-bit cache share.
//
// Here and in the other kernels of the decode step, what an earlier kernel may
// have written is read after griddepcontrol.wait (these kernels start before
// that one has ended), by plain loads, loads through L2 (__ldcg) or bulk
// copies, never through the read-only path.  The exception is weights that the
// caller calls static.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"
#include "internal.h"

namespace bitnet {

// Weights are 2^(score - m + kRaise); m follows the scores once they pass it
// by kLazy (both log2): weights stay below 2^15, and fp16 keeps them to 2^-11
// or to 2^-32 of the largest (2^-31 for prompts, whose m is whole).
constexpr float kLazy = 8.0f;
constexpr float kRaise = 7.0f;

// The rows r0 .. r1 - 1 of sequence b and its length; false for numbers that
// do not describe one.  (Rows of queries and positions fit 32 bits: T *
// q_heads and max_pages * page_tokens are below 2^31.)
__device__ __forceinline__ bool kv_sequence(const KvBatch &batch, int P, int b, int *r0, int *r1, int *len) {
  *len = __ldcg(batch.lens + b);
  *r0 = b;
  *r1 = b + 1;
  if (batch.offsets != nullptr) {
    *r0 = __ldcg(batch.offsets + b);
    *r1 = __ldcg(batch.offsets + b + 1);
  }
  return *r0 >= 0 && *r1 <= batch.T && *r0 <= *r1 && *len >= 0 && *len <= batch.max_pages * P;
}
// The first position that a query at `pos` sees.
__device__ __forceinline__ int first_seen(int pos, int window) {
  return window > 0 && pos >= window ? pos - window + 1 : 0;
}


// 2^x down to fp32's smallest number (2^-149).
__device__ __forceinline__ float ex2_whole(float x) {
  float y;
  asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Value scales far apart.  A weight p' = 2^(score + log2 vs - m + kRaise)
// counts for O only next to the largest p', but its share p' / vs of the row
// sum counts next to the other shares: with vs = 2^-59 (or a page of zeros,
// log2 vs = -60) beside vs = 2^60, p' can be below 2^-126 where p' / vs is the
// larger share.  As long as vs stays within 2^-30 and 2^30, such a share is
// below 2^-66 of the largest.  Where one does not, shares are taken as
// 2^(score - m + kRaise) by an exponential of their own.
__device__ __forceinline__ bool far_scale(float vs) {  // (infinite: what sees it is NaN anyway)
  return vs < 9.313225746154785e-10f || (vs > 1073741824.0f && vs < INFINITY);
}
// v * 2^d where 2^d alone is below 2^-126 (a share can be 2^75).
__device__ __forceinline__ float times_ex2(float v, float d) {
  const float half = ex2(__fmul_rn(d, 0.5f));
  return __fmul_rn(__fmul_rn(v, half), half);
}

__device__ __forceinline__ uint32_t half2_bits(__half2 h) {
  return *reinterpret_cast<uint32_t *>(&h);
}
// Two codes + 128, one in the low byte of each half, to two halves.
__device__ __forceinline__ uint32_t from_biased(uint32_t x) {
  const uint32_t bias = 0x64806480u;  // 1152, twice
  return half2_bits(__hsub2(*reinterpret_cast<__half2 *>(&x), *reinterpret_cast<const __half2 *>(&bias)));
}
// Bytes 0, 1 (2, 3) of w (codes + 128) as two halves.
__device__ __forceinline__ uint32_t codes01(uint32_t w) { return from_biased(__byte_perm(w, 0x64646464u, 0x4140)); }
__device__ __forceinline__ uint32_t codes23(uint32_t w) { return from_biased(__byte_perm(w, 0x64646464u, 0x4342)); }

// mbar_wait in few instructions (its retries unrolled would fill the
// instruction cache of kernels that wait in many places).
__device__ __forceinline__ bool wait_for(uint64_t *bar, uint32_t parity, int *status) {
  if (mbar_try_wait(bar, parity)) return true;
  const long long t0 = clock64();
#pragma unroll 1
  while (!mbar_try_wait(bar, parity)) {
    if (clock64() - t0 > kWaitLimitCycles) {
      record_status(status, kStatusTimeout);
      return false;
    }
  }
  return true;
}

}  // namespace bitnet
