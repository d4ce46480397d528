// pod_kv4.cuh -- device helpers of the 4-bit KV cache: row types, the order of
// the codes inside a record, and the request that a row belongs to.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <climits>
#include <cstdint>

#include "pod_kv4_params.h"
#include "pod_ptx.cuh"

namespace pod {

// Two adjacent channels of a bf16 or fp16 row, as fp32 and back (one rounding).
template <bool FP16>
__device__ __forceinline__ float2 row2_to_float(uint32_t v) {
  if constexpr (FP16)
    return __half22float2(*reinterpret_cast<__half2*>(&v));
  else
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}

template <bool FP16>
__device__ __forceinline__ uint32_t float_to_row2(float a, float b) {
  if constexpr (FP16) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}

// Least or largest (NaN if either is) of two values each.
template <bool FP16>
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
  uint32_t r;
  if constexpr (FP16)
    asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
template <bool FP16>
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  uint32_t r;
  if constexpr (FP16)
    asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{.reg .b64 a, b, c, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mov.b64 c, {%6, %7};\n"
      "fma.rn.f32x2 d, a, b, c;\n mov.b64 {%0, %1}, d;}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{.reg .b64 a, b, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n"
      "mul.rn.f32x2 d, a, b;\n mov.b64 {%0, %1}, d;}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{.reg .b64 a, b, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n"
      "add.rn.f32x2 d, a, b;\n mov.b64 {%0, %1}, d;}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
// The two fp16 of a word.
__device__ __forceinline__ float2 pair(uint32_t v) {
  return __half22float2(*reinterpret_cast<__half2*>(&v));
}

// Byte offsets inside a record (the orders stated in pod_kv4.h). Eight
// channels 8 g .. 8 g + 7 of a K token are one word; four channels 4 g ..
// 4 g + 3 of a V token are one half word.
template <int D>
__device__ __forceinline__ int k_code_byte(int token, int g8) {
  return token * (D / 2) + 4 * ((g8 & 3) * (D / 32) + (g8 >> 2));
}
template <int D>
__device__ __forceinline__ int v_code_byte(int token, int g4) {
  return 8 * D + 4 * ((32 * (token >> 3) + 4 * (g4 & 7) + ((token & 7) >> 1)) * (D / 32) + (g4 >> 3)) +
         2 * (token & 1);
}
// The pair (s, m) of a token's channel group, K (kv = 0) or V (kv = 1).
template <int D>
__device__ __forceinline__ int pair_byte(int kv, int token, int grp, int ngrp) {
  return kKv4Page * D + ((kv * kKv4Page + token) * ngrp + grp) * 4;
}

// The largest r < n with cu[r] <= i (0 if there is none), by the whole warp: each
// round divides the range by 33. cu is read within its n + 1 entries whatever
// it holds.
__device__ __forceinline__ int warp_request(const int* __restrict__ cu, int n, int i, int lane) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int probe = lo + (int)((long long)(hi - lo) * (lane + 1) / 33);
    const uint32_t below = __ballot_sync(0xffffffffu, __ldg(cu + probe) <= i);
    // the probes that are not above i, counted from the first: cu is sorted
    const int k = below == 0xffffffffu ? 32 : __ffs(~below) - 1;
    const int next_lo = lo + (int)((long long)(hi - lo) * k / 33);
    hi = k == 32 ? hi : max(lo + (int)((long long)(hi - lo) * (k + 1) / 33), next_lo + 1);
    lo = next_lo;
  }
  return lo;
}

}  // namespace pod
