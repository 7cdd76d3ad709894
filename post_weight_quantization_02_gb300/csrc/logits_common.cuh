// Shared device helpers of the kernels that stream rows of logits (top_logits.cu,
// distill.cu): 16-byte reads of a row from any alignment, and running log-sum-exp pairs.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "common.cuh"
#include "tc_common.cuh"

namespace gptq {

// Most entries of a row's top logits (teacher entries of the loss, k of the selection).
constexpr int kMaxTop = 256;

constexpr float kLog2e = 1.4426950408889634f;

// Whether a row is short, so that the latencies at its ends count: it gets 256 threads, a long one
// 512, and an SM about twice as many short rows at a time as long ones (top logits six and three,
// gradient alone four and two, loss and gradient two and one).
inline bool small_rows(int64_t row_bytes) { return row_bytes <= 96 * 1024; }

template <typename T>
struct LogitVec;
template <>
struct LogitVec<__nv_bfloat16> {
  static constexpr int N = 8;  // elements of one 16-byte access
  __device__ static __forceinline__ void unpack(uint4 u, float (&v)[N]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = __uint_as_float(w[j] << 16);
      v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
    }
  }
  __device__ static __forceinline__ float get(__nv_bfloat16 v) { return __bfloat162float(v); }
  __device__ static __forceinline__ __nv_bfloat16 put(float v) { return __float2bfloat16(v); }
};
template <>
struct LogitVec<float> {
  static constexpr int N = 4;
  __device__ static __forceinline__ void unpack(uint4 u, float (&v)[N]) {
    v[0] = __uint_as_float(u.x); v[1] = __uint_as_float(u.y);
    v[2] = __uint_as_float(u.z); v[3] = __uint_as_float(u.w);
  }
  __device__ static __forceinline__ float get(float v) { return v; }
  __device__ static __forceinline__ float put(float v) { return v; }
};

// A stretch of a row, [beg, end), cut into `head` single elements up to the first 16-byte
// boundary, `nvec` 16-byte pieces and the elements after them.
template <typename T>
struct RowSpan {
  int beg, head, nvec, tail0, end;
  __device__ __forceinline__ RowSpan(const T* row, int b, int e) : beg(b), end(e) {
    constexpr int N = LogitVec<T>::N;
    const uint32_t off = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(row + b) / sizeof(T)) % N;
    head = min((N - static_cast<int>(off)) % N, e - b);
    nvec = (e - b - head) / N;
    tail0 = b + head + nvec * N;
  }
};

// exp2(x) for any x (one instruction, within 2^-22 of the value; -inf gives 0)
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// the larger; NaN if either is
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

// A running maximum m and sum s of exp2((v - m) c) over values v; (-inf, 0) when empty.  The
// difference is formed before the product, so that the largest value's term is exactly 1
// however large the values are.  A NaN among them makes m NaN; with a maximum that is not
// finite s means nothing.
struct MaxSum {
  float m, s;
};
__device__ __forceinline__ MaxSum max_sum_of(float v) { return {v, v == -INFINITY ? 0.0f : 1.0f}; }
// differences are taken from the maximum, or from 0 where there is none yet
__device__ __forceinline__ float base_of(float m) { return m == -INFINITY ? 0.0f : m; }
__device__ __forceinline__ MaxSum join(MaxSum a, MaxSum b, float c) {
  const float m = max_nan(a.m, b.m), base = base_of(m);
  return {m, a.s * ex2((a.m - base) * c) + b.s * ex2((b.m - base) * c)};
}
// natural log-sum-exp of the values times `scale` (c = scale log2(e))
__device__ __forceinline__ float lse_of(MaxSum z, float scale) {
  return fabsf(z.m) < INFINITY ? z.m * scale + logf(z.s) : z.m;
}

__device__ __forceinline__ MaxSum warp_join(MaxSum v, float c, int width = 32) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    if (o < width)
      v = join(v, MaxSum{__shfl_xor_sync(0xffffffffu, v.m, o), __shfl_xor_sync(0xffffffffu, v.s, o)}, c);
  return v;
}

// The two halves of a block's join: every warp leaves its pair, and, behind a barrier, every
// thread gets the same result, joined in a fixed order.
__device__ __forceinline__ void leave_pair(MaxSum v, float c, MaxSum* scratch) {
  v = warp_join(v, c);
  if (threadIdx.x % 32 == 0) scratch[threadIdx.x / 32] = v;
}
template <int NT>
__device__ __forceinline__ MaxSum take_pair(float c, const MaxSum* scratch) {
  constexpr int W = NT / 32;
  return warp_join(scratch[threadIdx.x % W], c, W);
}

// ------------------------------------------------------------------ one pass over a row
//
// Pieces in flight per thread and batch.
constexpr int kBatch = 4;

// The largest of the elements of n pieces, NaN if one is (bf16: two at a time).
template <typename T, int n>
__device__ __forceinline__ float max_of(const uint4 (&u)[n]) {
  if constexpr (sizeof(T) == 2) {
    const auto pair = [](uint32_t w) { return *reinterpret_cast<const __nv_bfloat162*>(&w); };
    __nv_bfloat162 m = __hmax2_nan(__hmax2_nan(pair(u[0].x), pair(u[0].y)),
                                   __hmax2_nan(pair(u[0].z), pair(u[0].w)));
#pragma unroll
    for (int i = 1; i < n; ++i)
      m = __hmax2_nan(m, __hmax2_nan(__hmax2_nan(pair(u[i].x), pair(u[i].y)),
                                     __hmax2_nan(pair(u[i].z), pair(u[i].w))));
    return max_nan(__low2float(m), __high2float(m));
  } else {
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < n; ++i)
      m = max_nan(m, max_nan(max_nan(__uint_as_float(u[i].x), __uint_as_float(u[i].y)),
                             max_nan(__uint_as_float(u[i].z), __uint_as_float(u[i].w))));
    return m;
  }
}

// elements 2 j and 2 j + 1 of a piece
template <typename T>
__device__ __forceinline__ float2 pair_of(const uint4& u, int j) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  if constexpr (sizeof(T) == 2)
    return make_float2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xffff0000u));
  else
    return make_float2(__uint_as_float(w[2 * j]), __uint_as_float(w[2 * j + 1]));
}

// Joins the elements of n pieces to z; `top` is their largest.
template <typename T, int n>
__device__ __forceinline__ void accumulate(MaxSum& z, const uint4 (&u)[n], float top, float c) {
  const float m = max_nan(z.m, top), base = base_of(m);
  const float2 c2 = make_float2(c, c), b2 = make_float2(-base, -base);
  float2 s = make_float2(z.s * ex2((z.m - base) * c), 0.0f);
#pragma unroll
  for (int i = 0; i < n; ++i)
#pragma unroll
    for (int j = 0; j < LogitVec<T>::N / 2; ++j) {
      const float2 e = tc::mul2(tc::add2(pair_of<T>(u[i], j), b2), c2);
      s = tc::add2(s, make_float2(ex2(e.x), ex2(e.y)));
    }
  z = {m, s.x + s.y};
}

// The running maximum and sum over a thread's share of the pieces [p0, p1) of a row.
template <typename T, int NT>
__device__ __forceinline__ MaxSum stream_pieces(const uint4* xv, int p0, int p1, float c) {
  MaxSum z{-INFINITY, 0.0f};
  int p = p0 + threadIdx.x;
  for (; p + (kBatch - 1) * NT < p1; p += kBatch * NT) {
    uint4 u[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) u[i] = xv[p + i * NT];
    accumulate<T, kBatch>(z, u, max_of<T, kBatch>(u), c);
  }
  for (; p < p1; p += NT) {
    const uint4 u[1] = {xv[p]};
    accumulate<T, 1>(z, u, max_of<T, 1>(u), c);
  }
  return z;
}

}  // namespace gptq
