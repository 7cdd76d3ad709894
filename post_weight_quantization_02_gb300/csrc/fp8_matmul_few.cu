// The products of fp8_matmul.cu for few rows of C (single tokens, small batches) and for
// results too small to fill the GPU with 256 x 256 tiles.
//
// The operands trade places: 128 rows of B (the weight) are the M side of a one-SM MMA and NT
// rows of A (the tokens) its N side, so that a single token costs an MMA of 16 columns and not
// of 256.  The contraction is split over the CTAs of a cluster, whose sums are joined through
// distributed shared memory in a fixed order.
//
// Bound by streaming the weight (an N x K byte matrix for 2 N K T flops): every SM keeps
// 160 to 200 KB of it in flight.  The weight's first stages are requested before the wait for
// the kernel before this one (the quantiser of the tokens, which does not write the weight),
// so that they travel while the tokens are quantised.  Where there are more CTAs than SMs, a CTA
// takes half of one, so that one CTA starts up while the other streams: 9 x 28672 x 8192 42 us, 48
// with one CTA an SM; 64 tokens 46 us, 64.  Where there are not, it takes a whole one, for the
// longer ring: 16 x 8192 x 28672 in two shares 46.7 us, 48.3 in half an SM.
//   warp 0      TMA producer       warp 1      TMEM owner, MMA issuer
//   warps 2..9  epilogue: warp = 32 rows of B, half of the tokens; a lane holds 4 rows by an eighth of
//               the tokens, whose scales it reads (a row by half of the tokens, all of whose scales
//               every lane has to read: 0.50 us a block
//               of 128 tokens, 0.43 so)
//   warps 10..17  with at most 8 tokens and a small weight: the tokens' quantiser
//               (fp8_quantize.cu's arithmetic).  Each CTA turns its share of every token into
//               codes in the operand's shared-memory layout, so that a step of decoding is one
//               launch and needs no workspace; such a CTA has an SM to itself, as the quantiser
//               takes 0.3 us a block and lives on a long ring
// NACC accumulators of NT columns rotate, so the round trip from an MMA through the epilogue
// back to the issuer (about a microsecond) is hidden behind the blocks in between.
#include <cuda_bf16.h>

#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "fp8_common.cuh"
#include "kernels.cuh"
#include "tc_common.cuh"

namespace gptq {

namespace {

constexpr int BJ = 128;   // rows of B per CTA
constexpr int BK = 128;   // one scale block
constexpr int EPI_WARPS = 8;
constexpr int EPI_WARP0 = 2;
constexpr int THREADS = 32 * (EPI_WARP0 + EPI_WARPS);
constexpr int QUANT_WARPS = 4, QUANT_WARP0 = EPI_WARP0 + EPI_WARPS;
// A quantiser warp takes this many blocks at once: its fence towards the tensor core also waits
// for its outstanding loads, so the loads of several blocks share one wait (a block at a time with
// the next ones' loads under way took 1600 cycles each).  Two sets of warps take turns.
constexpr int GROUP = 4, QUANT_SETS = 2;
constexpr int W_BYTES = BJ * BK;
constexpr int PART_LD = BJ + 4;
constexpr int NSCALE = 32;  // token scale slots: at least NSTAGE + NACC + 1 (see fp8_matmul.cu)

template <int NT, int PER_SM>  // PER_SM: CTAs an SM, 1 or 2
struct Few {
  static constexpr int X_BYTES = NT * BK;
  static constexpr int STAGE_BYTES = W_BYTES + X_BYTES;
  static constexpr int NSTAGE = (PER_SM == 2 ? 99000 : 204800) / STAGE_BYTES;  // 11, 10, 8, 6; two an SM: 5, 4, 4
  static constexpr int NACC = PER_SM == 2 || NT == 128 ? 4 : 8;  // PER_SM NACC NT <= 512 TMEM columns
  static constexpr int SLOT = NT < 32 ? 32 : NT;               // floats of a scale slot (128 bytes at least)
  static constexpr int SMEM_BYTES = NSTAGE * STAGE_BYTES + NSCALE * SLOT * 4 + 1024 + 1024;
  static_assert(NSCALE >= NSTAGE + NACC + 1 && PER_SM * (SMEM_BYTES + 1024) <= 233472, "");
  // a stage's barrier completes again only after its block's accumulator was handed back
  static_assert(NSTAGE >= NACC && NSTAGE <= 32 && NSCALE == 32, "");
  static_assert(PART_LD * NT * 4 <= NSTAGE * STAGE_BYTES, "the joined sums reuse the ring");
};

struct FewArgs {
  const void* x;      // the tokens, where the kernel quantises them
  int64_t ldx, k;
  bool vec;           // their rows start on 16-byte boundaries
  const float* sb;
  int64_t sb_n, sb_k;
  int64_t m, n;       // rows of A (tokens), rows of B
  int nk;             // blocks of the contraction
  int per;            // blocks of each CTA of the cluster
  int jt;             // tiles of B's rows
  void* c;
  bool c_bf16;
  int64_t ldc;
  DevStatus* st;
  uint64_t wait_ns;
};

__device__ __forceinline__ void store_c(const FewArgs& a, int64_t t, int64_t j, float v) {
  if (a.c_bf16) static_cast<__nv_bfloat16*>(a.c)[t * a.ldc + j] = __float2bfloat16(v);
  else static_cast<float*>(a.c)[t * a.ldc + j] = v;
}

// W_MN: B is stored with its row axis contiguous; TX: the tokens' type where they come as they
// are, void where they come as codes
template <int NT, bool W_MN, typename TX, int PER_SM>
__global__ void __launch_bounds__(THREADS + (std::is_void_v<TX> ? 0 : 32 * QUANT_SETS * QUANT_WARPS),
                                  PER_SM)
    fp8_few_kernel(const __grid_constant__ CUtensorMap tw, const __grid_constant__ CUtensorMap tx,
                   const __grid_constant__ CUtensorMap tsx, const FewArgs a) {
  constexpr bool QUANT = !std::is_void_v<TX>;
  using F = Few<NT, PER_SM>;
  constexpr int NSTAGE = F::NSTAGE, NACC = F::NACC, STAGE_BYTES = F::STAGE_BYTES;
  constexpr uint32_t TX_BYTES = QUANT ? W_BYTES : STAGE_BYTES + NT * 4;
  constexpr uint32_t IDESC = tc::idesc_e4m3_f32(BJ, NT, W_MN, false);
  constexpr int TMEM_COLS = NACC * NT;
  constexpr int HALF = NT / 2;  // tokens of an epilogue thread
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  float* xscales = reinterpret_cast<float*>(smem + NSTAGE * STAGE_BYTES);
  uint64_t* full = reinterpret_cast<uint64_t*>(xscales + NSCALE * F::SLOT);
  // A stage's MMAs have completed: its operands may be replaced and its accumulator read.  The
  // issuer arrives too: it has seen the block's token scales land, and passes that on to the
  // epilogue (a completed MMA alone makes what copies or other warps wrote visible to no thread).
  uint64_t* done = full + NSTAGE;
  uint64_t* accempty = done + NSTAGE;
  uint64_t* mma_drain = accempty + NACC;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  // [0] stages issued, [1] stages seen to land, [2 + w] groups that quantiser warp w made
  int* counts = const_cast<int*>(abort_flag) + 1;

  const int warp = threadIdx.x / 32;
  const int lane = threadIdx.x % 32;
  const int split = static_cast<int>(tc::cluster_ctarank());
  const int nsplit = static_cast<int>(tc::cluster_nctarank());
  const int64_t tile = blockIdx.x / nsplit;
  const int64_t j0 = (tile % a.jt) * BJ;
  const int64_t t0 = (tile / a.jt) * NT;
  const int kb0 = split * a.per;
  const int nb = max(0, min(a.per, a.nk - kb0));

  if (warp == 0) {  // a barrier a lane
    if (lane < NSTAGE) {
      tc::mbar_init(&full[lane], QUANT ? 1 + QUANT_WARPS : 1);
      tc::mbar_init(&done[lane], 2);
    }
    if (lane < NACC) tc::mbar_init(&accempty[lane], EPI_WARPS);
    if (lane == 0) {
      tc::mbar_init(mma_drain, 1);
      *abort_flag = 0;
      counts[0] = counts[1] = 0;
    }
    tc::fence_mbar_init();
  }
  if (warp == 1) {
    tc::tmem_alloc(tmem_slot, TMEM_COLS);
    tc::tmem_relinquish();
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem_base = *tmem_slot;
  bool ok = true;
  float2 sum[HALF / 2];
#pragma unroll
  for (int k = 0; k < HALF / 2; ++k) sum[k] = make_float2(0.0f, 0.0f);
  const int q = warp % 4;            // TMEM lane quarter this warp may access
  const int half = (warp - EPI_WARP0) / 4;   // which half of the tokens

  if (warp == 0 && lane == 0) {
    // ---------------------------------------------------------------- producer
    const auto load_w = [&](int i, int stage) {
      uint8_t* dst = smem + stage * STAGE_BYTES;
      if (W_MN) tc::tma_load_2d(dst, &tw, &full[stage], static_cast<int>(j0), (kb0 + i) * BK);
      else tc::tma_load_2d(dst, &tw, &full[stage], (kb0 + i) * BK, static_cast<int>(j0));
    };
    const auto load_x = [&](int i, int stage) {
      tc::tma_load_2d(smem + stage * STAGE_BYTES + W_BYTES, &tx, &full[stage], (kb0 + i) * BK,
                      static_cast<int>(t0));
      tc::tma_load_2d(xscales + (i % NSCALE) * F::SLOT, &tsx, &full[stage], static_cast<int>(t0), kb0 + i);
    };
    const int head = min(nb, NSTAGE);
    for (int i = 0; i < head; ++i) {
      tc::mbar_arrive_expect_tx(&full[i], TX_BYTES);
      load_w(i, i);
    }
    if (!QUANT) {
      griddep_wait();
      for (int i = 0; i < head; ++i) load_x(i, i);
    }
    int issued = head, stage = 0;
    uint32_t phase = 0;
    for (int i = head; i < nb; ++i) {
      if (!tc::mbar_wait_short(&done[stage], phase, abort_flag, a.wait_ns)) { ok = false; break; }
      tc::mbar_arrive_expect_tx(&full[stage], TX_BYTES);
      load_w(i, stage);
      if (!QUANT) load_x(i, stage);
      ++issued;
      if (++stage == NSTAGE) { stage = 0; phase ^= 1u; }
    }
    counts[0] = issued;
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer
    const uint32_t ring = tc::smem_u32(smem);
    int stage = 0, acc = 0, seen = 0;
    uint32_t phase = 0, accphase = 0;
    for (int i = 0; i < nb; ++i) {
      const uint64_t at = (ring >> 4) + static_cast<uint32_t>(stage) * (STAGE_BYTES >> 4);
      const uint64_t wd = (W_MN ? tc::desc128(W_BYTES) : tc::desc128(16)) + at;
      const uint64_t xd = tc::desc128(16) + at + (W_BYTES >> 4);
      const uint32_t d = tmem_base + static_cast<uint32_t>(acc * NT);
      if (!tc::mbar_wait_short(&full[stage], phase, abort_flag, a.wait_ns)) { ok = false; break; }
      ++seen;
      if (!tc::mbar_wait_short(&accempty[acc], accphase ^ 1u, abort_flag, a.wait_ns)) { ok = false; break; }
      __syncwarp();
      if (tc::elect_one()) {
        tc::fence_after();
#pragma unroll
        for (int kk = 0; kk < BK / 32; ++kk)  // N-major: 32 rows of k are four 8-row groups
          tc::mma_f8(d, wd + (W_MN ? 256 : 2) * kk, xd + 2 * kk, IDESC, kk != 0 ? 1u : 0u);
        tc::mma_commit(&done[stage]);
        tc::mbar_arrive(&done[stage]);
      }
      __syncwarp();
      if (++stage == NSTAGE) { stage = 0; phase ^= 1u; }
      if (++acc == NACC) { acc = 0; accphase ^= 1u; }
    }
    if (lane == 0) counts[1] = seen;
  } else if (QUANT && warp >= QUANT_WARP0) {
    // ---------------------------------------------------------------- the tokens' quantiser
    if constexpr (QUANT) {
      // half a warp takes a token: kFewTokens half-warps
      static_assert(kFewTokens == 2 * QUANT_WARPS, "");
      const int qw = warp - QUANT_WARP0, set = qw / QUANT_WARPS, w = qw % QUANT_WARPS;
      const int c8 = lane % 16, token = w + QUANT_WARPS * (lane / 16);
      const bool idle = t0 + w >= a.m;  // neither half has a token
      const TX* x = static_cast<const TX*>(a.x) + (t0 + token) * a.ldx;
      int made = 0;
      for (int i0 = GROUP * set; i0 < nb && ok; i0 += GROUP * QUANT_SETS) {
        Eight<TX> v[GROUP];
#pragma unroll
        for (int j = 0; j < GROUP; ++j) {
          const int64_t k0 = static_cast<int64_t>(kb0 + i0 + j) * BK + 8 * c8;
          const int64_t left = i0 + j < nb && t0 + token < a.m ? a.k - k0 : 0;
          if (left >= 8 && a.vec) v[j].load(x + k0);
          else v[j].load_some(x + k0, static_cast<int>(max(static_cast<int64_t>(0), min(static_cast<int64_t>(8), left))));
        }
#pragma unroll
        for (int j = 0; j < GROUP; ++j) {
          const int i = i0 + j, stage = i % NSTAGE;
          if (ok && i < nb && i >= NSTAGE)
            ok = tc::mbar_wait_short(&done[stage], static_cast<uint32_t>(i / NSTAGE - 1) & 1u, abort_flag, a.wait_ns);
        }
        if (!ok) break;
        if (!idle) {
#pragma unroll
          for (int j = 0; j < GROUP; ++j) {
            const int i = i0 + j;
            MaxPair<TX> p = {};
#pragma unroll
            for (int q4 = 0; q4 < 4; ++q4) p.add(v[j], q4);
            uint32_t m = max(p.even(), p.odd());
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
            const float s = scale_of(m);
            // the 128-byte swizzle: 16-byte pieces of a row exchanged by its number mod 8
            const uint2 c = codes8(v[j], s, minus_reciprocal_of(m, s));
            if (i < nb) {
              uint8_t* dst = smem + i % NSTAGE * STAGE_BYTES + W_BYTES + token * BK;
              *reinterpret_cast<uint2*>(dst + (((c8 >> 1) ^ (token & 7)) << 4) + (c8 & 1) * 8) = c;
              if (c8 == 0) xscales[(i % NSCALE) * F::SLOT + token] = s;
            }
          }
          tc::fence_proxy_async_shared();  // the tensor core reads what was written
        }
        __syncwarp();
        if (lane < GROUP && i0 + lane < nb) tc::mbar_arrive(&full[(i0 + lane) % NSTAGE]);
        ++made;
      }
      if (lane == 0) counts[2 + qw] = made;
    }
  } else if (warp >= EPI_WARP0) {
    // ---------------------------------------------------------------- epilogue
    const float* psb = a.sb + j0 / 128 * a.sb_n;
    int acc = 0, stage = 0;
    uint32_t phase = 0;
    float sw = 0.0f, sw_next = nb > 0 ? psb[min(kb0 + lane, a.nk - 1) * a.sb_k] : 0.0f;
    for (int i = 0; i < nb; ++i) {
      if (i % 32 == 0) {
        sw = sw_next;
        sw_next = psb[min(kb0 + i + 32 + lane, a.nk - 1) * a.sb_k];
      }
      const float s = __shfl_sync(0xffffffffu, sw, i % 32);
      if (!tc::mbar_wait_short(&done[stage], phase, abort_flag, a.wait_ns)) { ok = false; break; }
      tc::fence_after();
      const uint32_t tbase = tmem_base + (static_cast<uint32_t>(32 * q) << 16) +
                             static_cast<uint32_t>(acc * NT + half * HALF);
      const float2* xs = reinterpret_cast<const float2*>(xscales + (i % NSCALE) * F::SLOT + half * HALF) + lane % 4;
      const float2 s2 = make_float2(s, s);
      constexpr int CH = HALF < 32 ? HALF : 32;  // columns of one TMEM read
      uint32_t r[2][HALF / CH][CH / 2];          // of 16 rows
#pragma unroll
      for (int c = 0; c < HALF / CH; ++c)
#pragma unroll
        for (int h = 0; h < 2; ++h) tc::tmem_ld_16x256b(tbase + (h * 16 << 16) + c * CH, r[h][c]);
      float2 f[HALF / 8];
#pragma unroll
      for (int k = 0; k < HALF / 8; ++k) f[k] = tc::mul2(s2, xs[4 * k]);
      tc::tmem_ld_wait();
      tc::fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive_relaxed(&accempty[acc]);
#pragma unroll
      for (int k = 0; k < HALF / 8; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t* u = &r[e / 2][k / (CH / 8)][4 * (k % (CH / 8)) + 2 * (e % 2)];
          float2& to = sum[e * (HALF / 8) + k];
          to = tc::fma2(make_float2(__uint_as_float(u[0]), __uint_as_float(u[1])), f[k], to);
        }
      if (++stage == NSTAGE) { stage = 0; phase ^= 1u; }
      if (++acc == NACC) acc = 0;
    }
  }

  if (!ok) {
    *abort_flag = 1;
    if (lane == 0 || warp >= EPI_WARP0) {
      dev_fail(a.st, GPTQ_ERR_TIMEOUT, 0);
      atomicAdd(&a.st->timeouts, 1);
    }
  }
  // Drain on every exit: the MMAs by one more commit, then every copy that was issued.
  bool drained = true;
  if (warp == 1 && tc::elect_one()) {  // the lane that issued the MMAs
    tc::mma_commit(mma_drain);
    drained = tc::mbar_wait_for(mma_drain, 0, kWaitLimitNs);
  }
  __syncwarp();
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int k = counts[1]; k < counts[0]; ++k) {
      // the arrivals of quantiser warps that gave up before this block
      if (QUANT)
        for (int w = 0; w < QUANT_WARPS; ++w)
          if (counts[2 + k / GROUP % QUANT_SETS * QUANT_WARPS + w] <= k / GROUP / QUANT_SETS)
            tc::mbar_arrive(&full[k % NSTAGE]);
      if (!tc::mbar_wait_for(&full[k % NSTAGE], static_cast<uint32_t>(k / NSTAGE) & 1u, kWaitLimitNs))
        drained = false;
    }
  }
  if (!drained) {
    dev_fail(a.st, GPTQ_ERR_TIMEOUT, 1);
    atomicAdd(&a.st->timeouts, 1);
    tc::linger();
  }
  __syncthreads();
  griddep_wait();  // every thread, before C is written: the work before may still read it
  griddep_launch_dependents();

  // ------------------------------------------------------------------ the result
  // each CTA's sums, [token][row of B], where the ring was (rows of 132: the 4 tokens and 8 rows
  // that a warp writes at once lie in 32 banks); then every CTA of the cluster joins its share
  const int tokens = static_cast<int>(min(static_cast<int64_t>(NT), a.m - t0));
  const int rows = static_cast<int>(min(static_cast<int64_t>(BJ), a.n - j0));
  float* part = reinterpret_cast<float*>(smem);
  if (warp >= EPI_WARP0 && warp < EPI_WARP0 + EPI_WARPS) {
#pragma unroll
    for (int k = 0; k < HALF / 8; ++k) {
      const int t = half * HALF + 8 * k + 2 * (lane % 4);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float* p = part + t * PART_LD + 32 * q + 8 * e + lane / 4;
        if (t < tokens) p[0] = sum[e * (HALF / 8) + k].x;
        if (t + 1 < tokens) p[PART_LD] = sum[e * (HALF / 8) + k].y;
      }
    }
  }
  if (nsplit == 1) __syncthreads();
  else tc::cluster_sync();
  const uint32_t base = tc::smem_u32(part);
  const int threads = static_cast<int>(blockDim.x);
  for (int e = split * threads + threadIdx.x; e < tokens * BJ; e += nsplit * threads) {
    const int t = e / BJ, j = e % BJ;
    float v = 0.0f;
    if (nsplit == 1) v = part[t * PART_LD + j];
    else
      for (int r = 0; r < nsplit; ++r)
        v += __uint_as_float(tc::ld_shared_cluster_u32(
            tc::mapa_shared(base + 4 * (t * PART_LD + j), static_cast<uint32_t>(r))));
    if (j < rows) store_c(a, t0 + t, j0 + j, v);
  }
  if (nsplit > 1) tc::cluster_sync();  // no CTA leaves while its sums are read
  if (warp == 1) {
    __syncwarp();
    tc::fence_after();
    tc::tmem_dealloc(tmem_base, TMEM_COLS);
  }
}

template <int NT, bool W_MN, typename TX, int PER_SM>
void launch_nt(const Fp8Matmul& p, FewArgs a, int splits, cudaStream_t s) {
  constexpr bool QUANT = !std::is_void_v<TX>;
  using F = Few<NT, PER_SM>;
  auto kernel = fp8_few_kernel<NT, W_MN, TX, PER_SM>;
  ensure_dynamic_smem(kernel, F::SMEM_BYTES);
  CUtensorMap tw, tx, tsx;
  if (W_MN)
    make_tmap_2d(&tw, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.b, static_cast<uint64_t>(p.n),
                 static_cast<uint64_t>(p.k), static_cast<uint64_t>(p.ldb), BJ, BK, CU_TENSOR_MAP_SWIZZLE_128B);
  else
    make_tmap_2d(&tw, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.b, static_cast<uint64_t>(p.k),
                 static_cast<uint64_t>(p.n), static_cast<uint64_t>(p.ldb), BK, BJ, CU_TENSOR_MAP_SWIZZLE_128B);
  if (QUANT) {
    tx = tsx = tw;  // not used
  } else {
    make_tmap_2d(&tx, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.a, static_cast<uint64_t>(p.k),
                 static_cast<uint64_t>(p.m), static_cast<uint64_t>(p.lda), BK, NT, CU_TENSOR_MAP_SWIZZLE_128B);
    make_tmap_2d(&tsx, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, p.sa, static_cast<uint64_t>(p.m),
                 static_cast<uint64_t>(a.nk), static_cast<uint64_t>(p.sa_k) * 4, NT, 1, CU_TENSOR_MAP_SWIZZLE_NONE);
  }
  const int64_t tiles = a.jt * ceil_div(p.m, NT);
  trace_begin(GPTQ_K_FP8_MATMUL, s);
  // behind the quantiser the weight may be requested early; a kernel that quantises the tokens
  // itself follows whatever wrote them and the weight
  launch_cluster("fp8_few_kernel", kernel, dim3(static_cast<unsigned>(tiles * splits)),
                 dim3(THREADS + (QUANT ? 32 * QUANT_SETS * QUANT_WARPS : 0)), static_cast<unsigned>(splits),
                 F::SMEM_BYTES, s, !QUANT, tw, tx, tsx, a);
  trace_end(GPTQ_K_FP8_MATMUL, s);
}

}  // namespace

void launch_fp8_matmul_few(const Fp8Matmul& p, int tokens_per_tile, int splits, const void* x,
                           bool x_bf16, int64_t ldx, DevStatus* st, cudaStream_t s) {
  FewArgs a = {};
  a.sb = p.sb;
  a.sb_n = p.sb_n;
  a.sb_k = p.sb_k;
  a.m = p.m;
  a.n = p.n;
  a.nk = static_cast<int>(ceil_div(p.k, BK));
  a.per = static_cast<int>(ceil_div(a.nk, splits));
  a.jt = static_cast<int>(ceil_div(p.n, BJ));
  a.c = p.c;
  a.c_bf16 = p.c_bf16;
  a.ldc = p.ldc;
  a.st = st;
  a.wait_ns = wait_limit_ns();
  if (x != nullptr) {
    a.x = x;
    a.ldx = ldx;
    a.k = p.k;
    const size_t es = x_bf16 ? 2 : 4;
    a.vec = reinterpret_cast<uintptr_t>(x) % 16 == 0 && (static_cast<size_t>(ldx) * es) % 16 == 0;
    return x_bf16 ? launch_nt<16, false, __nv_bfloat16, 1>(p, a, splits, s)
                  : launch_nt<16, false, float, 1>(p, a, splits, s);
  }
  const bool two = fp8_few_two_per_sm(a.jt * ceil_div(p.m, tokens_per_tile) * splits, splits, tokens_per_tile);
  const auto launch = [&](auto nt) {
    constexpr int NT = decltype(nt)::value, TWO = NT <= 64 ? 2 : 1;
    if (p.b_mn) two ? launch_nt<NT, true, void, TWO>(p, a, splits, s) : launch_nt<NT, true, void, 1>(p, a, splits, s);
    else two ? launch_nt<NT, false, void, TWO>(p, a, splits, s) : launch_nt<NT, false, void, 1>(p, a, splits, s);
  };
  switch (tokens_per_tile) {
    case 16: return launch(std::integral_constant<int, 16>());
    case 32: return launch(std::integral_constant<int, 32>());
    case 64: return launch(std::integral_constant<int, 64>());
    default: return launch(std::integral_constant<int, 128>());
  }
}

}  // namespace gptq
