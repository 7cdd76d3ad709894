// The k largest logits of each row, in descending order (equal values by ascending index; a
// NaN counts as larger than any number), and the row's log-sum-exp.
//
// Bound by memory: every logit is read once.  One CTA takes a row.  While it streams the row
// each thread keeps the largest element of each quarter of its share and the running
// log-sum-exp.  The k-th largest of the thread maxima is a bound that at least k elements reach,
// and few more do, all of them in the quarters whose maximum reaches it: only those (about 70 of
// 2048 for k = 64) are read again, from L2, by whole warps, and the elements that reach the bound
// are ranked by counting.  Where too many reach it (long runs of equal values), it is refined to
// the exact k-th element by a radix selection over (key, index) pairs, which are all distinct.  (So
// it is in a row of fewer pieces than k, which has no bound, and more than 1024 elements: top 256 of
// 2048 x 2000 bf16 255 us, top 128 of them 61.)
#include <cuda_bf16.h>

#include "common.cuh"
#include "kernels.cuh"
#include "logits_common.cuh"

namespace gptq {

namespace {

constexpr int kCap = 1024;  // candidates held

// order-preserving key: larger float, larger key; -0 and +0 alike, every NaN the largest
__device__ __forceinline__ uint32_t key_of(float v) {
  const uint32_t u = __float_as_uint(v + 0.0f);
  return v == v ? u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u) : 0xffffffffu;
}
__device__ __forceinline__ float value_of(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
}
// (key, index) as one number: larger key first, then the smaller index
__device__ __forceinline__ uint64_t entry_of(float v, int i) {
  return static_cast<uint64_t>(key_of(v)) << 32 | static_cast<uint32_t>(~i);
}

// f(value, index) for the elements of piece p
template <typename T, typename F>
__device__ __forceinline__ void visit_piece(const uint4& u, const RowSpan<T>& sp, int p, F&& f) {
  using V = LogitVec<T>;
  float v[V::N];
  V::unpack(u, v);
#pragma unroll
  for (int j = 0; j < V::N; ++j) f(v[j], sp.beg + sp.head + p * V::N + j);
}
// for the elements outside the pieces
template <typename T, int NT, typename F>
__device__ __forceinline__ void visit_edges(const T* x, const RowSpan<T>& sp, F&& f) {
  for (int p = threadIdx.x; p < sp.head + (sp.end - sp.tail0); p += NT) {
    const int at = p < sp.head ? sp.beg + p : sp.tail0 + p - sp.head;
    f(LogitVec<T>::get(x[at]), at);
  }
}
// for the whole row
template <typename T, int NT, typename F>
__device__ __forceinline__ void visit(const T* x, const RowSpan<T>& sp, F&& f) {
  const uint4* xv = reinterpret_cast<const uint4*>(x + sp.beg + sp.head);
  for (int p = threadIdx.x; p < sp.nvec; p += NT) visit_piece<T>(xv[p], sp, p, f);
  visit_edges<T, NT>(x, sp, f);
}

// The largest key, or one close below it, that k of the block's keys reach.  Bits that all keys
// share are not searched, and a key that a few more than k reach will do.
template <int NT>
__device__ __forceinline__ uint32_t bound_of(uint32_t mine, int k, uint32_t (&common)[2]) {
  const uint32_t all = __reduce_and_sync(0xffffffffu, mine), any = __reduce_or_sync(0xffffffffu, mine);
  if (threadIdx.x % 32 == 0) {
    atomicAnd(&common[0], all);
    atomicOr(&common[1], any);
  }
  __syncthreads();
  const uint32_t differ = common[0] ^ common[1];
  if (differ == 0) return mine;
  const int top = 31 - __clz(differ);
  uint32_t bound = common[1] >> top >> 1 << top << 1;
  for (int b = top; b >= 0; --b) {
    const uint32_t t = bound | (1u << b);
    const int n = __syncthreads_count(mine >= t);
    if (n >= k) bound = t;
    if (n >= k && n <= k + k / 8) break;
  }
  return bound;
}

// Blocks an SM: three of 512 threads, six of 256 (2048 x 131072 bf16: 102 us; with two and four 111,
// with four and eight, in 32 registers, 112).
template <typename T, int NT>
__global__ void __launch_bounds__(NT, 1536 / NT) top_logits_kernel(const TopArgs a) {
  __shared__ MaxSum scratch[NT / 32];
  __shared__ uint64_t cand[kCap];
  __shared__ int count;
  __shared__ uint32_t common[2];
  __shared__ uint8_t ask[NT / 32][4 * 32];  // a warp's quarters to read again: 32 * quarter + lane
  __shared__ int hist[256];
  __shared__ uint64_t found;
  __shared__ int left;

  const int64_t row = blockIdx.x;
  const int tid = threadIdx.x, lane = tid % 32;
  const T* x = static_cast<const T*>(a.logits) + row * a.ld;
  const RowSpan<T> sp(x, 0, a.vocab);
  const uint4* xv = reinterpret_cast<const uint4*>(x + sp.head);
  if (tid == 0) {
    count = 0;
    common[0] = 0xffffffffu;
    common[1] = 0;
  }
  __syncthreads();

  // ---- the row, once, a quarter after the other
  const int quarter = max((sp.nvec + 3) / 4, kBatch * NT);  // short rows: whole batches, fewer of them
  uint32_t key[4];  // of an empty share: -inf's
  MaxSum z{-INFINITY, 0.0f};
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    const MaxSum part = stream_pieces<T, NT>(xv, h * quarter, min((h + 1) * quarter, sp.nvec), kLog2e);
    key[h] = key_of(part.m);
    z = join(z, part, kLog2e);
  }
  const int edges = sp.head + (sp.end - sp.tail0);
  const int edge = tid < sp.head ? tid : sp.tail0 + tid - sp.head;
  const float edge_value = tid < edges ? LogitVec<T>::get(x[edge]) : -INFINITY;
  z = join(z, max_sum_of(edge_value), kLog2e);
  leave_pair(z, kLog2e, scratch);
  const uint32_t mine = max(max(key[0], key[1]), max(key[2], key[3]));
  const uint32_t bound = bound_of<NT>(mine, a.k, common);
  if (tid < 32 && a.lse != nullptr) {
    const float lse = lse_of(take_pair<NT>(kLog2e, scratch), 1.0f);
    if (tid == 0) a.lse[row] = lse;
  }

  // ---- the elements that reach the bound
  uint64_t low = static_cast<uint64_t>(bound) << 32;
  const auto take = [&](float v, int i) {
    const uint64_t e = entry_of(v, i);
    if (e >= low) {
      const int at = atomicAdd(&count, 1);
      if (at < kCap) cand[at] = e;
    }
  };
  // the warp's quarters that reach it, listed, then eight lanes to one, eight in flight
  int asked = 0;
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    const uint32_t mask = __ballot_sync(0xffffffffu, key[h] >= bound);
    if (mask >> lane & 1)
      ask[tid / 32][asked + __popc(mask & ((1u << lane) - 1))] = static_cast<uint8_t>(32 * h + lane);
    asked += __popc(mask);
  }
  __syncwarp();
  for (int i = lane / 8; i < asked; i += 8) {
    int p[2], end[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int code = ask[tid / 32][min(i + 4 * j, asked - 1)], h = code / 32;
      p[j] = h * quarter + tid - lane + code % 32 + lane % 8 * NT;
      end[j] = i + 4 * j < asked ? min((h + 1) * quarter, sp.nvec) : 0;
    }
    for (; p[0] < end[0] || p[1] < end[1]; p[0] += 8 * NT, p[1] += 8 * NT) {
      uint4 u[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) u[j] = xv[min(p[j], sp.nvec - 1)];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint4 one[1] = {u[j]};
        if (p[j] < end[j] && key_of(max_of<T, 1>(one)) >= bound) visit_piece<T>(u[j], sp, p[j], take);
      }
    }
  }
  if (tid < edges) take(edge_value, edge);
  __syncthreads();

  if (count > kCap) {
    // too many: the exact k-th entry, eight bits at a time from the top
    uint64_t prefix = 0;
    if (tid == 0) left = a.k;
    for (int shift = 56; shift >= 0; shift -= 8) {
      for (int i = tid; i < 256; i += NT) hist[i] = 0;
      __syncthreads();
      visit<T, NT>(x, sp, [&](float v, int i) {
        const uint64_t e = entry_of(v, i);
        if (shift == 56 || (e >> (shift + 8)) == (prefix >> (shift + 8)))
          atomicAdd(&hist[(e >> shift) & 255], 1);
      });
      __syncthreads();
      if (tid == 0) {
        int n = left, d = 255;
        for (; d > 0 && hist[d] < n; --d) n -= hist[d];
        left = n;
        found = prefix | static_cast<uint64_t>(d) << shift;
        count = 0;
      }
      __syncthreads();
      prefix = found;
    }
    low = prefix;
    visit<T, NT>(x, sp, take);  // exactly k
    __syncthreads();
  }

  // ---- ranks: four threads count for one candidate
  const int n = min(count, kCap);
  for (int i = tid / 4; i < (n + 7) / 8 * 8; i += NT / 4) {
    const uint64_t e = i < n ? cand[i] : 0;
    int rank = 0;
#pragma unroll 8
    for (int j = tid % 4; j < n; j += 4) rank += cand[j] > e;
    const uint32_t mask = 0xffffffffu;
    rank += __shfl_xor_sync(mask, rank, 1);
    rank += __shfl_xor_sync(mask, rank, 2);
    if (tid % 4 == 0 && i < n && rank < a.k) {
      a.values[row * a.k + rank] = value_of(static_cast<uint32_t>(e >> 32));
      a.indices[row * a.k + rank] = static_cast<int32_t>(~static_cast<uint32_t>(e));
    }
  }
}

template <typename T, int NT>
void launch_nt(const TopArgs& a, cudaStream_t s) {
  GPTQ_LAUNCH(GPTQ_K_TOP_LOGITS, s, (top_logits_kernel<T, NT>), static_cast<unsigned>(a.rows), NT, 0, a);
}

template <typename T>
void launch_typed(const TopArgs& a, cudaStream_t s) {
  if (small_rows(static_cast<int64_t>(a.vocab) * sizeof(T)) && a.k <= 64) launch_nt<T, 256>(a, s);
  else launch_nt<T, 512>(a, s);
}

}  // namespace

void launch_top_logits(const TopArgs& a, bool bf16, cudaStream_t s) {
  if (a.rows == 0) return;
  if (bf16) launch_typed<__nv_bfloat16>(a, s);
  else launch_typed<float>(a, s);
}

}  // namespace gptq
