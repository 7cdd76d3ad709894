// Distillation from a teacher's top logits: the loss of each row and its gradient.
//
// Row n has student logits s[0 .. V) and k teacher entries (t_j, i_j); an entry with a
// negative index is padding.  With temperature T and weight w,
//     q_j = softmax(t / T) over the row's entries       Z = log sum_v exp(s_v / T)
//     loss = w sum_j q_j (log q_j - s_{i_j} / T + Z)
//     dloss/ds_v = g w (exp(s_v / T - Z) - Q_v) / T     Q_v = sum of the q_j with i_j = v
// A row of weight 0, or without an entry of non-zero q, does not count: its loss, log-sum-exp
// and gradient are 0 whatever its logits are (those of a row of weight 0 are not read).
//
// Bound by memory: a logit is read once from HBM and its gradient written once.  The loss
// streams rows through a ring in shared memory (row_ring.cuh) and keeps a running maximum and
// sum.  For the gradient the last chunks of the row are still in the ring; they are worked off
// first, the others are fetched again behind them (from L2, where the long rows in flight, one an
// SM, stay), so that the copies for this row's gradient and for the next row never wait for the
// row's end.  The entries' columns are written once more with their q.
#include <cuda_bf16.h>

#include "common.cuh"
#include "kernels.cuh"
#include "logits_common.cuh"
#include "row_ring.cuh"

namespace gptq {

namespace {

// Slots that the next loads may use while the end of a row stays in the ring.
constexpr int kAhead = 2;

// values 2 j, 2 j + 1 of the piece that is written
template <typename T>
__device__ __forceinline__ uint4 pack(const float2 (&v)[LogitVec<T>::N / 2]) {
  if constexpr (sizeof(T) == 2) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(v[j].x, v[j].y);
      w[j] = *reinterpret_cast<const uint32_t*>(&b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    return make_uint4(__float_as_uint(v[0].x), __float_as_uint(v[0].y), __float_as_uint(v[1].x),
                      __float_as_uint(v[1].y));
  }
}

// f exp2((v a - b) c): the gradient of a logit v that is no entry's
struct Gradient {
  float a, b, c, f;
  __device__ __forceinline__ float exponential(float v) const { return ex2(fmaf(v, a, -b) * c); }
  __device__ __forceinline__ float operator()(float v) const { return f * exponential(v); }
  template <typename T>
  __device__ __forceinline__ uint4 piece(const uint4& u) const {
    float2 v[LogitVec<T>::N / 2];
#pragma unroll
    for (int j = 0; j < LogitVec<T>::N / 2; ++j) {
      const float2 d = tc::fma2(pair_of<T>(u, j), make_float2(a, a), make_float2(-b, -b));
      const float2 e = tc::mul2(d, make_float2(c, c));
      v[j] = tc::mul2(make_float2(f, f), make_float2(ex2(e.x), ex2(e.y)));
    }
    return pack<T>(v);
  }
};

// a piece to its place among the row's (dx + head need not be aligned like the logits)
template <typename T>
__device__ __forceinline__ void store_piece(T* dst, const uint4& u, bool aligned16) {
  if (aligned16) {
    __stcs(reinterpret_cast<uint4*>(dst), u);
  } else {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < LogitVec<T>::N; ++j) {
      if constexpr (sizeof(T) == 2) {
        reinterpret_cast<uint16_t*>(dst)[j] = static_cast<uint16_t>(w[j / 2] >> (16 * (j % 2)));
      } else {
        reinterpret_cast<uint32_t*>(dst)[j] = w[j];
      }
    }
  }
}

template <typename T>
__device__ __forceinline__ void write_zeros(T* dx, int vocab, int nthreads) {
  const RowSpan<T> sp(dx, 0, vocab);
  uint4* dv = reinterpret_cast<uint4*>(dx + sp.head);
  for (int p = threadIdx.x; p < sp.nvec; p += nthreads) __stcs(dv + p, make_uint4(0, 0, 0, 0));
  for (int p = threadIdx.x; p < sp.head + (sp.end - sp.tail0); p += nthreads)
    dx[p < sp.head ? p : sp.tail0 + p - sp.head] = LogitVec<T>::put(0.0f);
}

// a row's entry of this thread: index (-1: none) and value (-inf where there is none)
struct Entry {
  int idx;
  float t;
};
__device__ __forceinline__ float weight_of(const DistillArgs& a, int64_t row) {
  return a.weights != nullptr ? a.weights[row] : 1.0f;
}
__device__ __forceinline__ Entry load_entry(const DistillArgs& a, int64_t row, bool counts) {
  Entry e{-1, -INFINITY};
  if (counts && static_cast<int>(threadIdx.x) < a.k) {
    e.idx = a.t_indices[row * a.k + threadIdx.x];
    e.t = a.t_values[row * a.k + threadIdx.x];
  }
  return e;
}
__device__ __forceinline__ void check_entry(const DistillArgs& a, Entry& e) {
  if (e.idx >= a.vocab) {
    dev_fail(a.st, GPTQ_ERR_INVALID_ARG, e.idx);
    e.idx = -1;
  }
  if (e.idx < 0) e.t = -INFINITY;
}

// A row's entries, for the columns that are written again.
template <typename T>
struct Entries {
  float q[kMaxTop];  // q_j
  int i[kMaxTop];    // index, -1: no entry
  T s[kMaxTop];      // the logit at the index
};
// Lanes that share the work on one entry: a power of two, at most 32.
__device__ __forceinline__ int lanes_per_entry(int k, int nthreads) {
  int lanes = 1;
  while (lanes < 32 && 2 * lanes * k <= nthreads) lanes *= 2;
  return lanes;
}
// dx at the entries' columns: g (scale p - Q), Q the sum of the q at that index; the first entry
// with an index writes it.  `lanes` threads compare one entry with all others.
template <typename T, typename F>
__device__ __forceinline__ void write_entries(T* dx, const Entries<T>& t, int k, int lanes, float g, F&& p) {
  const int self = static_cast<int>(threadIdx.x) / lanes, part = static_cast<int>(threadIdx.x) % lanes;
  if (static_cast<int>(threadIdx.x) / 32 * 32 / lanes >= k) return;  // the warp has no entry
  const int idx = self < k ? t.i[self] : -1;
  float sum = 0.0f;
  int before = 0;
#pragma unroll 4
  for (int j = part; j < k; j += lanes) {
    const bool same = t.i[j] == idx;
    sum += same ? t.q[j] : 0.0f;
    before |= same && j < self;
  }
  for (int o = lanes / 2; o > 0; o >>= 1) {
    sum += __shfl_xor_sync(0xffffffffu, sum, o);
    before |= __shfl_xor_sync(0xffffffffu, before, o);
  }
  if (idx >= 0 && part == 0 && before == 0) dx[idx] = LogitVec<T>::put(g * (p(LogitVec<T>::get(t.s[self])) - sum));
}

// ------------------------------------------------------------------ the loss (and gradient)

// s/T is handled in base 2: (s - m) c with c = log2(e) / T
template <typename T, typename S, bool GRAD>
__global__ void __launch_bounds__(S::kBlock, S::kPerSm) distill_kernel(const DistillArgs a) {
  using V = LogitVec<T>;
  constexpr int NW = S::kWarps, kThreads = S::kThreads, kSlots = S::kSlots, kChunk = S::kChunk;
  extern __shared__ __align__(128) uint4 slots[];
  __shared__ uint64_t full[kSlots], empty[kSlots];
  __shared__ int abort_word, counts[2];
  __shared__ MaxSum zpairs[NW], tpairs[NW];
  __shared__ Entries<T> entries;
  __shared__ float terms[NW];

  const int tid = threadIdx.x;
  const Ring<S> ring{slots, full, empty, &abort_word, a.wait_ns};
  if (tid == 0) {
    ring.init();
    counts[0] = counts[1] = 0;
  }
  __syncthreads();
  const float c = a.inv_temp * kLog2e;
  bool ok = true;
  RingAt<S> at;

  if (tid >= kThreads) {
    if (tid == kThreads) {
      int issued = 0;
      for (int64_t row = blockIdx.x; row < a.rows && ok; row += gridDim.x) {
        if (a.weights != nullptr && a.weights[row] == 0.0f) continue;
        const T* x = static_cast<const T*>(a.logits) + row * a.ld;
        const RowSpan<T> sp(x, 0, a.vocab);
        const uint4* xv = reinterpret_cast<const uint4*>(x + sp.head);
        const int chunks = (sp.nvec + kChunk - 1) / kChunk;
        ok = ring_fill(ring, at, xv, sp.nvec, chunks, issued);
        // the chunks that did not stay in the ring
        if (GRAD && ok) ok = ring_fill(ring, at, xv, sp.nvec, chunks - min(chunks, kSlots - kAhead), issued);
      }
      counts[0] = issued;
    }
  } else {
    int seen = 0;
    const int lanes = lanes_per_entry(a.k, kThreads);
    // a row's weight and entries are requested a row ahead
    float w_next = weight_of(a, blockIdx.x);
    Entry e_next = load_entry(a, blockIdx.x, true);
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
      const T* x = static_cast<const T*>(a.logits) + row * a.ld;
      T* dx = GRAD ? static_cast<T*>(a.dlogits) + row * a.ldd : nullptr;
      const float w = w_next;
      Entry e = e_next;
      if (row + gridDim.x < a.rows) {
        w_next = weight_of(a, row + gridDim.x);
        e_next = load_entry(a, row + gridDim.x, true);
      }
      if (w == 0.0f) {
        if (GRAD) write_zeros(dx, a.vocab, kThreads);
        if (tid == 0) {
          a.loss[row] = 0.0f;
          if (a.lse != nullptr) a.lse[row] = 0.0f;
        }
        continue;
      }
      check_entry(a, e);
      const RowSpan<T> sp(x, 0, a.vocab);
      const int chunks = (sp.nvec + kChunk - 1) / kChunk;
      const int kept = GRAD ? min(chunks, kSlots - kAhead) : 0;  // the row's last chunks stay
      // before the gradient may replace them; used after the row
      const float at_idx = e.idx >= 0 ? V::get(x[e.idx]) : 0.0f;
      const int edges = sp.head + (sp.end - sp.tail0);
      const int edge = tid < sp.head ? tid : sp.tail0 + tid - sp.head;
      const float edge_value = tid < edges ? V::get(x[edge]) : -INFINITY;

      leave_pair(max_sum_of(e.t), c, tpairs);

      // ---- log-sum-exp
      MaxSum z{-INFINITY, 0.0f};
      RingAt<S> first_kept = at;
      for (int ch = 0; ch < chunks; ++ch) {
        if (ch == chunks - kept) first_kept = at;
        ring_wait(ring, at, ok, seen);
        uint4 u[4];
        take_chunk<T, S>(ring, at, sp.nvec - ch * kChunk, u);
        if (ch < chunks - kept) ring_release(ring, at, ok);
        accumulate<T, 4>(z, u, max_of<T, 4>(u), c);
        at.next();
      }
      z = join(z, max_sum_of(edge_value), c);
      leave_pair(z, c, zpairs);
      consumer_sync<S>();
      z = take_pair<kThreads>(c, zpairs);

      // ---- the gradient: p = exp2((s - m) c) / sum; where no logit is above -inf, p is 0
      const MaxSum tm = take_pair<kThreads>(c, tpairs);
      const bool counted = tm.m != -INFINITY;
      const float g = w * a.inv_temp;
      const float scale = z.m == -INFINITY ? 0.0f : 1.0f / z.s;
      const Gradient grad{1.0f, base_of(z.m), c, g * scale};
      if (GRAD) {
        T* dv = dx + sp.head;
        const bool aligned16 = reinterpret_cast<uintptr_t>(dv) % 16 == 0;
        RingAt<S> from = first_kept;
        for (int i = 0; i < chunks; ++i) {
          const int ch = i < kept ? chunks - kept + i : i - kept;
          if (i >= kept) {
            from = at;
            ring_wait(ring, at, ok, seen);
            at.next();
          }
          const int n = sp.nvec - ch * kChunk;
          const uint4* piece = slots + from.slot * kChunk;
          T* dst = dv + static_cast<int64_t>(ch) * kChunk * V::N;
          if (n >= kChunk && counted && aligned16) {  // a whole chunk without a branch
            uint4 u[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) u[j] = piece[tid + j * kThreads];
#pragma unroll
            for (int j = 0; j < 4; ++j)
              __stcs(reinterpret_cast<uint4*>(dst) + tid + j * kThreads, grad.template piece<T>(u[j]));
          } else {
            for (int p = tid; p < min(n, kChunk); p += kThreads)
              store_piece<T>(dst + p * V::N,
                             counted ? grad.template piece<T>(piece[p]) : make_uint4(0, 0, 0, 0), aligned16);
          }
          ring_release(ring, from, ok);
          from.next();
        }
        if (tid < edges) dx[edge] = V::put(counted ? grad(edge_value) : 0.0f);
      }

      // ---- the loss: log q = (t - max) / T - log sum, and log p alike
      const float logq = (e.t - tm.m) * a.inv_temp - logf(tm.s);
      const float q = e.idx >= 0 && counted ? expf(logq) : 0.0f;
      float term = 0.0f;
      if (q != 0.0f) term = q * (logq - ((at_idx - z.m) * a.inv_temp - logf(z.s)));
      if (counted && z.m == -INFINITY) term = tid == 0 ? INFINITY : 0.0f;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) term += __shfl_xor_sync(0xffffffffu, term, o);
      if (tid % 32 == 0) terms[tid / 32] = term;
      if (tid == 0 && a.lse != nullptr) a.lse[row] = counted ? lse_of(z, a.inv_temp) : 0.0f;
      if (GRAD && tid < a.k) {
        entries.q[tid] = q;
        entries.s[tid] = V::put(at_idx);
        entries.i[tid] = e.idx;
      }
      consumer_sync<S>();
      if (tid < 32) {
        float l = tid < NW ? terms[tid] : 0.0f;
#pragma unroll
        for (int o = NW / 2; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
        if (tid == 0) a.loss[row] = w * l;
      }
      // the entries' columns again, with their q (`entries` is written again behind the next
      // row's first barrier)
      if (GRAD && counted)
        write_entries(dx, entries, a.k, lanes, g, [&](float v) { return scale * grad.exponential(v); });
    }
    if (tid == 0) counts[1] = seen;
  }
  if (!ok) {
    abort_word = 1;
    dev_fail(a.st, GPTQ_ERR_TIMEOUT, 0);
    atomicAdd(&a.st->timeouts, 1);
  }
  __syncthreads();
  // every copy that was issued has landed before the shared memory goes away
  if (tid == 0)
    for (int q = counts[1]; q < counts[0]; ++q)
      tc::mbar_wait_for(&full[q % kSlots], static_cast<uint32_t>(q / kSlots) & 1u, kWaitLimitNs);
}

// ------------------------------------------------------------------ the gradient alone

// The log-sum-exp Z comes rounded to float32, and the rounding is a relative error of p.  Up to
// this size it is at most 2^-15; rows beyond it (masked throughout by the type's lowest value, or far
// from zero), whose Z may even be infinite, are summed up again (2048 x 131072 bf16 165 us, 215 where
// all rows are).
constexpr float kLseKept = 1024.0f;

template <typename T, int NT>
__global__ void __launch_bounds__(NT, 1024 / NT) distill_backward_kernel(const DistillArgs a) {
  using V = LogitVec<T>;
  __shared__ MaxSum tpairs[NT / 32], zpairs[NT / 32];
  __shared__ Entries<T> entries;

  const int64_t row = blockIdx.x;
  const int tid = threadIdx.x;
  const T* x = static_cast<const T*>(a.logits) + row * a.ld;
  T* dx = static_cast<T*>(a.dlogits) + row * a.ldd;
  const float w = weight_of(a, row);
  const float c = a.inv_temp * kLog2e;
  Entry e = load_entry(a, row, w != 0.0f);
  check_entry(a, e);
  const float at_idx = e.idx >= 0 ? V::get(x[e.idx]) : 0.0f;  // before the gradient may replace it
  leave_pair(max_sum_of(e.t), c, tpairs);
  __syncthreads();
  const MaxSum tm = take_pair<NT>(c, tpairs);
  if (w == 0.0f || tm.m == -INFINITY) {
    write_zeros(dx, a.vocab, NT);
    return;
  }
  const float q = e.idx >= 0 ? expf((e.t - tm.m) * a.inv_temp - logf(tm.s)) : 0.0f;
  if (tid < a.k) {
    entries.q[tid] = q;
    entries.s[tid] = V::put(at_idx);
    entries.i[tid] = e.idx;
  }
  // p = exp2((s / T - Z) log2 e), or exp2((s - m) c) / sum; where no logit is above -inf, p is 0
  const float g = w * a.inv_temp * (a.grad_loss != nullptr ? a.grad_loss[row] : 1.0f);
  const float lse = a.lse[row];
  float scale = 1.0f;
  Gradient grad{a.inv_temp, lse, kLog2e, g};
  const RowSpan<T> sp(x, 0, a.vocab);
  const uint4* xv = reinterpret_cast<const uint4*>(x + sp.head);
  if (!(fabsf(lse) <= kLseKept)) {  // as the loss does; the row is read before any of it is written
    MaxSum z = stream_pieces<T, NT>(xv, 0, sp.nvec, c);
    const int edge = tid < sp.head ? tid : sp.tail0 + tid - sp.head;
    if (tid < sp.head + (sp.end - sp.tail0)) z = join(z, max_sum_of(V::get(x[edge])), c);
    leave_pair(z, c, zpairs);
    __syncthreads();
    z = take_pair<NT>(c, zpairs);
    scale = z.m == -INFINITY ? 0.0f : 1.0f / z.s;
    grad = Gradient{1.0f, base_of(z.m), c, g * scale};
  }
  T* dv = dx + sp.head;
  const bool aligned16 = reinterpret_cast<uintptr_t>(dv) % 16 == 0;
  int p = tid;
  for (; p + (kBatch - 1) * NT < sp.nvec; p += kBatch * NT) {
    uint4 u[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) u[i] = __ldcs(xv + p + i * NT);
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      store_piece<T>(dv + (p + i * NT) * V::N, grad.template piece<T>(u[i]), aligned16);
  }
  for (; p < sp.nvec; p += NT) store_piece<T>(dv + p * V::N, grad.template piece<T>(__ldcs(xv + p)), aligned16);
  for (p = tid; p < sp.head + (sp.end - sp.tail0); p += NT) {
    const int edge = p < sp.head ? p : sp.tail0 + p - sp.head;
    dx[edge] = V::put(grad(V::get(x[edge])));
  }
  __syncthreads();
  write_entries(dx, entries, a.k, lanes_per_entry(a.k, NT), g,
                [&](float v) { return scale * grad.exponential(v); });
}

template <typename T, typename S, bool GRAD>
void launch_ring(const DistillArgs& a, cudaStream_t s) {
  const int64_t most = S::kPerSm * static_cast<int64_t>(sm_count());
  const unsigned grid = static_cast<unsigned>(a.rows < most ? a.rows : most);
  auto kernel = distill_kernel<T, S, GRAD>;
  ensure_dynamic_smem(kernel, S::kBytes);
  GPTQ_LAUNCH(GPTQ_K_DISTILL, s, kernel, grid, S::kBlock, S::kBytes, a);
}

template <typename T>
void launch_typed(const DistillArgs& a, bool loss, bool grad, cudaStream_t s) {
  if (loss) {
    // the loss alone reads a row once: two CTAs an SM whatever its length (2048 x 131072 bf16:
    // 86 us, 97 with one)
    if (!grad) launch_ring<T, ShortRows, false>(a, s);
    else if (small_rows(static_cast<int64_t>(a.vocab) * sizeof(T))) launch_ring<T, ShortRows, true>(a, s);
    else launch_ring<T, LongRows<sizeof(T) == 2 ? 7 : 6>, true>(a, s);
    return;
  }
  const unsigned grid = static_cast<unsigned>(a.rows);
  if (small_rows(static_cast<int64_t>(a.vocab) * sizeof(T)))
    GPTQ_LAUNCH(GPTQ_K_DISTILL, s, (distill_backward_kernel<T, 256>), grid, 256, 0, a);
  else
    GPTQ_LAUNCH(GPTQ_K_DISTILL, s, (distill_backward_kernel<T, 512>), grid, 512, 0, a);
}

}  // namespace

void launch_distill(const DistillArgs& a, bool bf16, bool loss, bool grad, cudaStream_t s) {
  if (a.rows == 0) return;
  if (bf16) launch_typed<__nv_bfloat16>(a, loss, grad, s);
  else launch_typed<float>(a, loss, grad, s);
}

}  // namespace gptq
