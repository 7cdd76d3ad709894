// Shared device code of the e4m3 quantisers (fp8_quantize.cu, and fp8_matmul_few.cu for the
// tokens of a small batch): eight values of a row at a time, magnitudes, scales and codes.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <stdint.h>

#include "common.cuh"
#include "tc_common.cuh"

namespace gptq {

constexpr float kFp8Max = 448.0f;  // the largest finite e4m3 value

// ------------------------------------------------------------------ eight values of a row
//
// Kept as they were loaded (bf16 pairs stay packed: half the registers, twice the tiles in
// flight); pair(j) gives values 2 j and 2 j + 1.
template <typename T>
struct Eight;

template <>
struct Eight<__nv_bfloat16> {
  static constexpr int W = 4;  // 32-bit words
  uint32_t w[W];
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    const uint4 u = __ldcs(reinterpret_cast<const uint4*>(p));
    w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
  }
  __device__ __forceinline__ void load_some(const __nv_bfloat16* p, int n) {
    const uint16_t* e = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      w[j] = (2 * j < n ? e[2 * j] : 0u) | (2 * j + 1 < n ? static_cast<uint32_t>(e[2 * j + 1]) << 16 : 0u);
  }
  __device__ __forceinline__ float2 pair(int j) const {
    return make_float2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xffff0000u));
  }
};
template <>
struct Eight<float> {
  static constexpr int W = 8;
  uint32_t w[W];
  __device__ __forceinline__ void load(const float* p) {
    const uint4 a = __ldcs(reinterpret_cast<const uint4*>(p));
    const uint4 b = __ldcs(reinterpret_cast<const uint4*>(p) + 1);
    w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
    w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
  }
  __device__ __forceinline__ void load_some(const float* p, int n) {
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = j < n ? __float_as_uint(p[j]) : 0u;
  }
  __device__ __forceinline__ float2 pair(int j) const {
    return make_float2(__uint_as_float(w[2 * j]), __uint_as_float(w[2 * j + 1]));
  }
};

// A row that does not start on a 16-byte boundary: `e` holds the aligned 16-byte pieces from the
// boundary before the lane's eight values on, `next` the piece after them (lane 15 of the row
// has read its own, the other lanes take the neighbour's first).  Moves the eight values,
// `mis` bytes in, to the front.
template <typename T>
__device__ __forceinline__ void realign(Eight<T>& e, uint4 next, int mis) {
  constexpr int W = Eight<T>::W;
  const bool last = threadIdx.x % 16 == 15;
  uint32_t w[W + 4];
#pragma unroll
  for (int i = 0; i < W; ++i) w[i] = e.w[i];
  const uint32_t own[4] = {next.x, next.y, next.z, next.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t theirs = __shfl_down_sync(0xffffffffu, e.w[i], 1, 16);
    w[W + i] = last ? own[i] : theirs;
  }
  if (mis & 8) {
#pragma unroll
    for (int i = 0; i < W + 2; ++i) w[i] = w[i + 2];
  }
  if (mis & 4) {
#pragma unroll
    for (int i = 0; i < W + 1; ++i) w[i] = w[i + 1];
  }
#pragma unroll
  for (int i = 0; i < W; ++i)
    e.w[i] = sizeof(T) == 2 ? __funnelshift_r(w[i], w[i + 1], (mis & 2) * 8) : w[i];
}

// only the first n values exist
template <typename T>
__device__ __forceinline__ void keep_first(Eight<T>& e, int n) {
  constexpr int W = Eight<T>::W;
#pragma unroll
  for (int i = 0; i < W; ++i) {
    if (sizeof(T) == 4) e.w[i] = i < n ? e.w[i] : 0u;
    else e.w[i] &= 2 * i + 1 < n ? 0xffffffffu : (2 * i < n ? 0xffffu : 0u);
  }
}

// ------------------------------------------------------------------ magnitudes
//
// Magnitudes compare as bit patterns, and a NaN's pattern is above infinity's, so that the
// integer maximum keeps a NaN.  Of bf16 pairs both halves are compared at once.
template <typename T>
struct MaxPair;  // the running magnitudes of the even and the odd values
template <>
struct MaxPair<__nv_bfloat16> {
  uint32_t m;
  __device__ __forceinline__ void add(const Eight<__nv_bfloat16>& e, int j) {
    m = __vmaxu2(m, e.w[j] & 0x7fff7fffu);
  }
  __device__ __forceinline__ void join(const MaxPair& o) { m = __vmaxu2(m, o.m); }
  __device__ __forceinline__ void join_lane16() { m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 16)); }
  __device__ __forceinline__ uint32_t even() const { return m << 16; }
  __device__ __forceinline__ uint32_t odd() const { return m & 0xffff0000u; }
};
template <>
struct MaxPair<float> {
  uint32_t a, b;
  __device__ __forceinline__ void add(const Eight<float>& e, int j) {
    a = max(a, e.w[2 * j] & 0x7fffffffu);
    b = max(b, e.w[2 * j + 1] & 0x7fffffffu);
  }
  __device__ __forceinline__ void join(const MaxPair& o) { a = max(a, o.a); b = max(b, o.b); }
  __device__ __forceinline__ void join_lane16() {
    a = max(a, __shfl_xor_sync(0xffffffffu, a, 16));
    b = max(b, __shfl_xor_sync(0xffffffffu, b, 16));
  }
  __device__ __forceinline__ uint32_t even() const { return a; }
  __device__ __forceinline__ uint32_t odd() const { return b; }
};
__device__ __forceinline__ float scale_of(uint32_t amax) {
  const float s = __fdiv_rn(__uint_as_float(amax), kFp8Max);
  return s < 0x1p-126f ? 0x1p-126f : s;  // a NaN stays
}

// ------------------------------------------------------------------ codes
//
// x / s rounded to nearest.  With y the correctly rounded reciprocal of s, q = x y is within
// one ulp of the quotient and q + (x - q s) y rounds it correctly (Markstein's theorem), as
// long as nothing under- or overflows.  Scales outside [2^-80, 2^100] take the division itself;
// y = 0 marks them.  In an all-zero group (padding, masked tokens) any y will do.
//
// What is computed is -x / s, with -y in y's place, and the codes' signs are turned back (an
// operation for four): for x = -0 the corrected quotient adds +0 to -0 and would lose the sign,
// the negated one adds two zeros of the sign that it needs, for either x.
__device__ __forceinline__ float minus_reciprocal_of(uint32_t amax, float s) {
  if (amax == 0) return -1.0f;
  return s >= 0x1p-80f && s <= 0x1p100f ? -__frcp_rn(s) : 0.0f;
}
constexpr uint32_t kTurnSigns = 0x80808080u;  // of four codes
static __device__ __noinline__ float2 divide_pair(float2 x, float s) {
  return make_float2(__fdiv_rn(x.x, s), __fdiv_rn(x.y, s));
}
// -x / s, y as minus_reciprocal_of gives it
__device__ __forceinline__ float2 minus_quotient(float2 x, float2 s, float2 y) {
  const float2 q = tc::mul2(x, y);
  return tc::fma2(tc::fma2(q, s, x), y, q);
}
__device__ __forceinline__ uint32_t codes2(float2 q) {
  return __nv_cvt_float2_to_fp8x2(q, __NV_SATFINITE, __NV_E4M3);
}

// the codes of a thread's eight values of a row, all with scale s (y: minus_reciprocal_of)
template <typename T>
__device__ __forceinline__ uint2 codes8(const Eight<T>& e, float s, float y) {
  uint32_t c[4], turn = 0;
  if (y != 0.0f) {
    turn = kTurnSigns;
#pragma unroll
    for (int j = 0; j < 4; ++j) c[j] = codes2(minus_quotient(e.pair(j), make_float2(s, s), make_float2(y, y)));
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) c[j] = codes2(divide_pair(e.pair(j), s));
  }
  return make_uint2((c[0] | (c[1] << 16)) ^ turn, (c[2] | (c[3] << 16)) ^ turn);
}

}  // namespace gptq
