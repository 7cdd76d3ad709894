// Products of e4m3 operands with a float32 scale for every 128 values of the contraction, on
// the 5th-generation tensor cores:
//     C[i][j] = sum_b sa[b][i] sb[j][b] sum_{k in block b} A[i][k] B[j][k]
// for the 8-bit linear layer's output (A activations, B weight), its input gradient (B the
// weight read along its other axis: N-major) and its weight gradient (both operands quantised
// along the tokens, a scale for each column of C).
//
// The tensor core sums one 128-block at a time (four 32-deep MMAs into a fresh TMEM
// accumulator); the epilogue warps read the accumulator, multiply it by the block's two scales
// and add it to float32 registers.  Products of two e4m3 values are exact in float32 and a
// chain is only 128 long, so the truncation of the tensor core's sums stays near 2^-24.
//
// fp8_matmul_kernel: persistent, one CTA per SM, the CTAs in pairs.  A pair computes a
// 256 x 256 tile of C (each CTA's TMEM 128 rows; each CTA's shared memory its own 128 rows of
// A and half of B), unit by unit:
//   warp 0      TMA producer (every CTA): a ring of 32 KB stages, one 128-block each, and the
//               block's row scales and, where every column of C has its own, column scales
//   warp 1      TMEM owner (every CTA); in the even CTA the MMA issuer
//   warp 2      sees a block's scales land in this CTA and passes that on to the epilogue (every
//               CTA): a completed MMA says that copies have landed, but makes what they wrote
//               visible to no thread (a wait of the epilogue's own for them cost about 7 %)
//   warps 4..11 epilogue (every CTA): thread = one row of C, 128 columns in registers (or 4 rows,
//               32 columns: below)
// Two 256-column accumulators alternate, so the MMAs of one block overlap the scaling of the
// block before.  A block takes 700 to 800 cycles at 8192 x 8192 x 28672, 512 of them MMAs (1.37 ms,
// 2.8 PFLOP/s).  Neither a multicast B over two pairs (1.44 ms), nor halves of 128 columns with a
// completion and a hand-back of their own (1.45 ms), nor 16 epilogue warps of 64 columns (1.50 ms)
// bring it nearer; TMEM has no room for a third accumulator of 256 columns.  At a tile's end the sums
// are stored while the tensor cores wait: 4 us a tile, 5.5 with column scales (4864 x 4096 results
// over contractions of 1024 to 8192).
//
// Where the last wave of tiles, or the only one, leaves half of the pairs idle, a cluster of 2 or 4
// pairs shares a tile of it (a launch of its own after the full waves): each pair takes
// its share of the contraction and leaves its sums where its ring was, and every CTA joins a share
// of the rows over the pairs' shared memory, in order.  512 x 4096 x 14336: 55 us with one pair a
// tile, 36 with two.
//
// Where every column of C has its own scale, a warp reads the accumulator 16 rows x 32 columns at
// a time, so that a lane has 32 columns of 4 rows instead of 128 columns of one: 32 column scales
// a lane and block come from shared memory instead of 128 (a broadcast still delivers 16 bytes to
// each of 32 lanes).  Weight gradient of 8192 x 8192 x 8192: 617 us, 695 with a row a lane.
#include <cuda_bf16.h>

#include <algorithm>

#include "common.cuh"
#include "kernels.cuh"
#include "tc_common.cuh"

namespace gptq {

namespace {

constexpr int BM = 128;   // rows of C per CTA
constexpr int BN = 256;   // columns of C per pair
constexpr int BK = 128;   // one scale block
constexpr int NSTAGE = 6;
constexpr int A_BYTES = BM * BK;
constexpr int B_BYTES = (BN / 2) * BK;
constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
// Scales of a block, a slot each: 128 of the CTA's rows and, where every column of C has its
// own, 256 of the tile's columns.  A slot is refilled NSCALE blocks later, when the MMAs of
// block b - NSTAGE have completed; those began after every epilogue warp had read the
// accumulator of block b - NSTAGE - 2, so was done with the slot of b - NSTAGE - 3: 9 slots
// would do.
constexpr int NSCALE = 16;
constexpr int ROW_SCALE_BYTES = BM * 4;
constexpr int COL_SCALE_BYTES = BN * 4;
constexpr int SMEM_BYTES =
    NSTAGE * STAGE_BYTES + NSCALE * (ROW_SCALE_BYTES + COL_SCALE_BYTES) + 1024 + 384;
constexpr int PART_LD = BN + 4;  // floats of a row of shared sums
static_assert(BM * PART_LD * 4 <= NSTAGE * STAGE_BYTES, "the shared sums reuse the ring");
constexpr int EPI_WARPS = 8;
constexpr int EPI_WARP0 = 4;
constexpr int THREADS = 32 * (EPI_WARP0 + EPI_WARPS);
// 168 registers a thread at launch; the control warpgroup keeps 56 of them and each epilogue
// thread, with its 128 sums and two 32-column reads of TMEM, gets 224 (56 + 2 x 224 = 3 x 168)
constexpr int CONTROL_REGS = 56, EPI_REGS = 224;
constexpr int kBand = 8;  // tile rows of C walked together

struct MatmulArgs {
  const float* sb;
  int64_t sb_n, sb_k;   // one scale for 128 columns: sb[(j / 128) sb_n + b sb_k]
  int64_t m, n;
  int nk;               // blocks of the contraction
  int per;              // of them, each pair's of a cluster
  int64_t mt, nt;       // tiles of 256 x 256
  int64_t first, end;   // those of this launch
  void* c;
  int64_t ldc;
  bool vec;             // C's rows start on 32-byte boundaries
  DevStatus* st;
  uint64_t wait_ns;
};

// Unit u -> tile (row, column): bands of kBand tile rows, walked column by column, so that the
// units in flight share both operands' strips in L2.
__device__ __forceinline__ void decode_unit(int64_t u, const MatmulArgs& a, int64_t& im, int64_t& in) {
  const int64_t per_band = kBand * a.nt;
  const int64_t band = u / per_band, rem = u % per_band;
  const int64_t rows = min(static_cast<int64_t>(kBand), a.mt - band * kBand);
  im = band * kBand + rem % rows;
  in = rem / rows;
}

// On every exit of a producer: the scales that it asked for have landed (the last of each slot)
__device__ __forceinline__ bool drain_scales(uint64_t* scaled, int issued) {
  bool landed = true;
  for (int k = max(0, issued - NSCALE); k < issued; ++k)
    if (!tc::mbar_wait_for(&scaled[k % NSCALE], static_cast<uint32_t>(k / NSCALE) & 1u, kWaitLimitNs))
      landed = false;
  if (!landed) tc::linger();
  return landed;
}

// 32 bytes, a whole sector, in one store (p 32-byte aligned)
__device__ __forceinline__ void store32(void* p, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]),
               "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}
__device__ __forceinline__ uint32_t bf16_pair(float2 v) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(v.x, v.y);
  return *reinterpret_cast<const uint32_t*>(&b);
}

// 16 consecutive elements of a row of C, ncol of which exist
__device__ __forceinline__ void store16(__nv_bfloat16* p, const float2* v, int ncol, bool vec) {
  if (vec && ncol >= 16) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = bf16_pair(v[i]);
    store32(p, w);
  } else {
#pragma unroll
    for (int j = 0; j < 16; ++j)
      if (j < ncol) p[j] = __float2bfloat16(j % 2 == 0 ? v[j / 2].x : v[j / 2].y);
  }
}
__device__ __forceinline__ void store16(float* p, const float2* v, int ncol, bool vec) {
  if (vec && ncol >= 16) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t w[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        w[2 * i] = __float_as_uint(v[4 * h + i].x);
        w[2 * i + 1] = __float_as_uint(v[4 * h + i].y);
      }
      store32(p + 8 * h, w);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 16; ++j)
      if (j < ncol) p[j] = j % 2 == 0 ? v[j / 2].x : v[j / 2].y;
  }
}

// 2 consecutive elements of a row of C, ncol of which exist (p: an even element of the row)
__device__ __forceinline__ void store2(__nv_bfloat16* p, float2 v, int64_t ncol, bool vec) {
  if (vec && ncol >= 2) {
    *reinterpret_cast<uint32_t*>(p) = bf16_pair(v);
  } else {
    if (ncol > 0) p[0] = __float2bfloat16(v.x);
    if (ncol > 1) p[1] = __float2bfloat16(v.y);
  }
}
__device__ __forceinline__ void store2(float* p, float2 v, int64_t ncol, bool vec) {
  if (vec && ncol >= 2) {
    *reinterpret_cast<float2*>(p) = v;
  } else {
    if (ncol > 0) p[0] = v.x;
    if (ncol > 1) p[1] = v.y;
  }
}

// Four consecutive elements of a row of C, ncol of which exist
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 v, int64_t ncol, bool vec) {
  if (vec && ncol >= 4) {
    *reinterpret_cast<uint2*>(p) = make_uint2(bf16_pair(make_float2(v.x, v.y)), bf16_pair(make_float2(v.z, v.w)));
  } else {
    store2(p, make_float2(v.x, v.y), ncol, false);
    store2(p + 2, make_float2(v.z, v.w), ncol - 2, false);
  }
}
__device__ __forceinline__ void store4(float* p, float4 v, int64_t ncol, bool vec) {
  if (vec && ncol >= 4) {
    *reinterpret_cast<float4*>(p) = v;
  } else {
    store2(p, make_float2(v.x, v.y), ncol, false);
    store2(p + 2, make_float2(v.z, v.w), ncol - 2, false);
  }
}

// B_MN: B is stored with its n axis contiguous; COL: a scale for each column of C; SPLIT: the
// cluster's pairs share one tile's contraction (see below), otherwise a cluster is one pair
template <bool B_MN, bool COL, typename TC, bool SPLIT>
__global__ void __launch_bounds__(THREADS, 1)
    fp8_matmul_kernel(const __grid_constant__ CUtensorMap ta, const __grid_constant__ CUtensorMap tb,
                      const __grid_constant__ CUtensorMap tsa,
                      const __grid_constant__ CUtensorMap tsb, const MatmulArgs a) {
  constexpr uint32_t IDESC = tc::idesc_e4m3_f32(2 * BM, BN, false, B_MN);
  constexpr uint32_t SCALE_BYTES = ROW_SCALE_BYTES + (COL ? COL_SCALE_BYTES : 0);  // of a block
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  float* row_scales = reinterpret_cast<float*>(smem + NSTAGE * STAGE_BYTES);
  float* col_scales = row_scales + NSCALE * BM;
  uint64_t* full = reinterpret_cast<uint64_t*>(col_scales + NSCALE * BN);
  uint64_t* done = full + NSTAGE;     // a stage's MMAs have completed and its block's scales are
                                      // there: its operands may be replaced, its accumulator read
  uint64_t* accempty = done + NSTAGE;
  uint64_t* scaled = accempty + 2;    // a block's scales are in their slot of this CTA
  uint64_t* mma_drain = scaled + NSCALE;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* counts = const_cast<int*>(abort_flag) + 1;  // [0] stages issued here, [1] stages seen to land

  const int warp = threadIdx.x / 32;
  const int lane = threadIdx.x % 32;
  // the CTA's number in its pair, the pair's even CTA, and the pair's blocks
  const uint32_t crank = SPLIT ? tc::cluster_ctarank() % 2 : tc::cluster_ctarank();
  const uint32_t lead = SPLIT ? tc::cluster_ctarank() - crank : 0;
  const int nsplit = SPLIT ? static_cast<int>(tc::cluster_nctarank()) / 2 : 1;
  const int kb0 = SPLIT ? static_cast<int>(lead / 2) * a.per : 0;
  const int nb = SPLIT ? max(0, min(a.per, a.nk - kb0)) : a.nk;
  const int64_t units = a.end;
  const int64_t unit0 = a.first + blockIdx.x / (2 * nsplit), unit_step = gridDim.x / (2 * nsplit);

  if (threadIdx.x == 0) {
    for (int s = 0; s < NSTAGE; ++s) {
      tc::mbar_init(&full[s], 1);
      tc::mbar_init(&done[s], 2);
    }
    for (int b = 0; b < 2; ++b) {
      tc::mbar_init(&accempty[b], 2 * EPI_WARPS);
    }
    for (int s = 0; s < NSCALE; ++s) tc::mbar_init(&scaled[s], 1);
    tc::mbar_init(mma_drain, 1);
    *abort_flag = 0;
    counts[0] = counts[1] = 0;
    tc::fence_mbar_init();
    tc::prefetch_tmap(&ta);
    tc::prefetch_tmap(&tb);
    tc::prefetch_tmap(&tsa);
    if (COL) tc::prefetch_tmap(&tsb);
  }
  if (warp == 1) {
    tc::tmem_alloc_pair(tmem_slot, 512);
    tc::tmem_relinquish_pair();
  }
  tc::fence_before();
  __syncwarp();
  tc::cluster_sync();
  tc::fence_after();
  const uint32_t tmem_base = *tmem_slot;
  bool ok = true;
  griddep_wait();  // the quantiser before this kernel has written the operands

  if (warp >= EPI_WARP0) {
    tc::regs_grow<EPI_REGS>();
    // ---------------------------------------------------------------- epilogue
    const int q = warp % 4;            // TMEM lane quarter this warp may access
    const int half = (warp - EPI_WARP0) / 4;   // which 128 of the 256 columns
    int acc = 0, stage = 0;
    uint32_t phase = 0;
    int blocks = 0;
    for (int64_t u = unit0; u < units && ok; u += unit_step) {
      int64_t im, in;
      decode_unit(u, a, im, in);
      const int64_t row0 = im * 2 * BM + crank * BM + 32 * q;
      const int64_t col = in * BN + half * 128;
      const float* psb = COL ? nullptr : a.sb + min(col, a.n - 1) / 128 * a.sb_n;
      float2 sum[64];
#pragma unroll
      for (int k = 0; k < 64; ++k) sum[k] = make_float2(0.0f, 0.0f);
      // the scales that all of a warp's columns share: lane l reads block kb + l, 32 ahead
      float sb = 1.0f, sb_next = 1.0f;
      if (!COL) sb_next = psb[min(kb0 + lane, a.nk - 1) * a.sb_k];
      for (int kb = 0; kb < nb; ++kb) {
        if (!COL && kb % 32 == 0) {
          sb = sb_next;
          sb_next = psb[min(kb0 + kb + 32 + lane, a.nk - 1) * a.sb_k];
        }
        if (!tc::mbar_wait_short(&done[stage], phase, abort_flag, a.wait_ns)) { ok = false; break; }
        tc::fence_after();
        const uint32_t tbase = tmem_base + (static_cast<uint32_t>(32 * q) << 16) +
                               static_cast<uint32_t>(acc * BN + half * 128);
        const auto hand_back = [&]() {  // the accumulator has been read: before the last sums
          tc::fence_before();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive_cluster_relaxed(tc::mapa_shared(tc::smem_u32(&accempty[acc]), lead));
        };
        if constexpr (COL) {
          // 16 rows x 32 columns at a time, the next 16 x 32 being read
          const float2* cs = reinterpret_cast<const float2*>(col_scales + (blocks % NSCALE) * BN + half * 128) + lane % 4;
          const float* rs = row_scales + (blocks % NSCALE) * BM + 32 * q + lane / 4;
          const float s[4] = {rs[0], rs[8], rs[16], rs[24]};
          float2 f[4];
          uint32_t r[2][16];
          tc::tmem_ld_16x256b(tbase, r[0]);
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            if (c % 2 == 0) {
#pragma unroll
              for (int i = 0; i < 4; ++i) f[i] = cs[4 * (4 * (c / 2) + i)];
            }
            tc::tmem_ld_wait();
            if (c < 7) tc::tmem_ld_16x256b(tbase + ((c + 1) % 2 * 16 << 16) + (c + 1) / 2 * 32, r[(c + 1) & 1]);
            else hand_back();
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const float se = s[2 * (c % 2) + e];
                float2& to = sum[16 * (2 * (c % 2) + e) + 4 * (c / 2) + i];
                to = tc::fma2(make_float2(__uint_as_float(r[c & 1][4 * i + 2 * e]),
                                          __uint_as_float(r[c & 1][4 * i + 2 * e + 1])),
                              tc::mul2(make_float2(se, se), f[i]), to);
              }
          }
        } else {
          // 32 columns (two reads of 16: 2 % faster than one of 32) are scaled while the next 32 are read
          const float s = row_scales[(blocks % NSCALE) * BM + 32 * q + lane] * __shfl_sync(0xffffffffu, sb, kb % 32);
          uint32_t r[2][2][16];
          tc::tmem_ld_32x32b_x16(tbase, r[0][0]);
          tc::tmem_ld_32x32b_x16(tbase + 16, r[0][1]);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            tc::tmem_ld_wait();
            if (c < 3) {
              tc::tmem_ld_32x32b_x16(tbase + 32 * (c + 1), r[(c + 1) & 1][0]);
              tc::tmem_ld_32x32b_x16(tbase + 32 * (c + 1) + 16, r[(c + 1) & 1][1]);
            } else {
              hand_back();
            }
#pragma unroll
            for (int k = 0; k < 16; ++k)
              sum[c * 16 + k] = tc::fma2(make_float2(__uint_as_float(r[c & 1][k / 8][2 * k % 16]),
                                                     __uint_as_float(r[c & 1][k / 8][2 * k % 16 + 1])),
                                         make_float2(s, s), sum[c * 16 + k]);
          }
        }
        ++blocks;
        acc ^= 1;
        if (++stage == NSTAGE) { stage = 0; phase ^= 1u; }
      }
      if (!ok) break;
      if constexpr (SPLIT) {
        // where the ring was: all of this CTA's MMAs have completed
        float4* p = reinterpret_cast<float4*>(smem) + (32 * q + lane) * (PART_LD / 4) + half * 32;
#pragma unroll
        for (int k = 0; k < 32; ++k)
          p[k] = make_float4(sum[2 * k].x, sum[2 * k].y, sum[2 * k + 1].x, sum[2 * k + 1].y);
      } else if constexpr (COL) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int64_t row = row0 + 8 * e + lane / 4;
          if (row < a.m) {
            TC* prow = static_cast<TC*>(a.c) + row * a.ldc;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int64_t j = col + 8 * i + 2 * (lane % 4);
              store2(prow + j, sum[e * 16 + i], a.n - j, a.vec);
            }
          }
        }
      } else if (const int64_t row = row0 + lane; row < a.m) {
        TC* prow = static_cast<TC*>(a.c) + row * a.ldc + col;
        const int left = static_cast<int>(max(static_cast<int64_t>(0), min(static_cast<int64_t>(128), a.n - col)));
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (16 * k < left) store16(prow + 16 * k, &sum[8 * k], left - 16 * k, a.vec);
      }
    }
  } else {
    tc::regs_shrink<CONTROL_REGS>();
    if (warp == 0 && lane == 0) {
      // ---------------------------------------------------------------- producer
      int stage = 0;
      uint32_t phase = 0;
      int issued = 0;
      for (int64_t u = unit0; u < units && ok; u += unit_step) {
        int64_t im, in;
        decode_unit(u, a, im, in);
        const int row = static_cast<int>(im * 2 * BM + crank * BM);
        const int col = static_cast<int>(in * BN + crank * (BN / 2));
        for (int kb = kb0; kb < kb0 + nb; ++kb) {
          if (!tc::mbar_wait_short(&done[stage], phase ^ 1u, abort_flag, a.wait_ns)) { ok = false; break; }
          uint8_t* sa = smem + stage * STAGE_BYTES;
          const uint32_t bar = tc::mapa_shared(tc::smem_u32(&full[stage]), lead);
          if (crank == 0) tc::mbar_arrive_expect_tx(&full[stage], 2 * STAGE_BYTES);
          tc::tma_load_2d_pair(sa, &ta, bar, kb * BK, row);
          if (B_MN) tc::tma_load_2d_pair(sa + A_BYTES, &tb, bar, col, kb * BK);
          else tc::tma_load_2d_pair(sa + A_BYTES, &tb, bar, kb * BK, col);
          const int slot = issued % NSCALE;
          tc::mbar_arrive_expect_tx(&scaled[slot], SCALE_BYTES);
          tc::tma_load_2d(row_scales + slot * BM, &tsa, &scaled[slot], row, kb);
          if (COL) tc::tma_load_2d(col_scales + slot * BN, &tsb, &scaled[slot], static_cast<int>(in * BN), kb);
          ++issued;
          if (++stage == NSTAGE) { stage = 0; phase ^= 1u; }
        }
      }
      counts[0] = issued;
      if (!drain_scales(scaled, issued)) ok = false;
    } else if (crank == 0 && warp == 1) {
      // ---------------------------------------------------------------- MMA issuer
      const uint32_t ring = tc::smem_u32(smem);
      int stage = 0;
      uint32_t phase = 0;
      int acc = 0;
      uint32_t accphase = 0;
      int seen = 0;
      for (int64_t u = unit0; u < units && ok; u += unit_step) {
        for (int kb = 0; kb < nb; ++kb) {
          const uint64_t at = (ring >> 4) + static_cast<uint32_t>(stage) * (STAGE_BYTES >> 4);
          const uint64_t ad = tc::desc128(16) + at;
          const uint64_t bd = (B_MN ? tc::desc128(B_BYTES) : tc::desc128(16)) + at + (A_BYTES >> 4);
          const uint32_t d = tmem_base + static_cast<uint32_t>(acc * BN);
          if (!tc::mbar_wait_short(&full[stage], phase, abort_flag, a.wait_ns)) { ok = false; break; }
          ++seen;
          if (!tc::mbar_wait_short(&accempty[acc], accphase ^ 1u, abort_flag, a.wait_ns)) { ok = false; break; }
          __syncwarp();
          if (tc::elect_one()) {
            tc::fence_after();
#pragma unroll
            for (int kk = 0; kk < BK / 32; ++kk)  // N-major: 32 rows of k are four 8-row groups
              tc::mma_f8_pair(d, ad + 2 * kk, bd + (B_MN ? 256 : 2) * kk, IDESC, kk != 0 ? 1u : 0u);
            tc::mma_commit_pair(&done[stage], static_cast<uint16_t>(0x3u << lead));
          }
          __syncwarp();
          if (++stage == NSTAGE) { stage = 0; phase ^= 1u; }
          acc ^= 1;
          if (acc == 0) accphase ^= 1u;
        }
      }
      if (lane == 0) counts[1] = seen;
    } else if (warp == 2 && lane == 0) {
      // ---------------------------------------------------------------- the scales' landing
      int i = 0;  // the producer fills a slot again only behind `done` of six blocks before
      for (int64_t u = unit0; u < units && ok; u += unit_step) {
        for (int kb = 0; kb < nb; ++kb, ++i) {
          if (!tc::mbar_wait(&scaled[i % NSCALE], static_cast<uint32_t>(i / NSCALE) & 1u, abort_flag, a.wait_ns)) {
            ok = false;
            break;
          }
          tc::mbar_arrive(&done[i % NSTAGE]);
        }
      }
    }
  }
  griddep_launch_dependents();

  if (!ok) {
    *abort_flag = 1;
    if (lane == 0 || warp >= EPI_WARP0) {
      dev_fail(a.st, GPTQ_ERR_TIMEOUT, 0);
      atomicAdd(&a.st->timeouts, 1);
    }
  }
  // Drain on every exit: the MMAs by one more commit, then every operand copy that was issued.
  bool drained = true;
  if (crank == 0 && warp == 1 && tc::elect_one()) {  // the lane that issued the MMAs
    tc::mma_commit_pair(mma_drain, static_cast<uint16_t>(0x1u << lead));
    drained = tc::mbar_wait_for(mma_drain, 0, kWaitLimitNs);
  }
  tc::fence_before();
  __syncwarp();
  tc::cluster_sync();  // both producers have stopped; their counts are visible
  if (crank == 0 && threadIdx.x == 0) {
    const int other = static_cast<int>(tc::ld_shared_cluster_u32(tc::mapa_shared(tc::smem_u32(counts), lead + 1)));
    if (!tc::drain_pair_stages(full, NSTAGE, counts[1], counts[0], other, STAGE_BYTES)) drained = false;
  }
  if (!drained) {
    dev_fail(a.st, GPTQ_ERR_TIMEOUT, 1);
    atomicAdd(&a.st->timeouts, 1);
    tc::linger();
  }
  if constexpr (SPLIT) {
    // every CTA joins its share of its 128 rows, over the pairs in order
    int64_t im, in;
    decode_unit(unit0, a, im, in);
    const int rows = BM / nsplit, first = static_cast<int>(lead / 2) * rows;
    const uint32_t base = tc::smem_u32(smem);
    for (int e = threadIdx.x; e < rows * (BN / 4); e += THREADS) {
      const int i = first + e / (BN / 4), j = e % (BN / 4) * 4;
      float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      for (int p = 0; p < nsplit; ++p) {
        const float4 u = tc::ld_shared_cluster_f4(
            tc::mapa_shared(base + 4 * (i * PART_LD + j), 2 * p + crank));
        v.x += u.x; v.y += u.y; v.z += u.z; v.w += u.w;
      }
      const int64_t row = im * 2 * BM + crank * BM + i, col = in * BN + j;
      if (row < a.m && col < a.n) store4(static_cast<TC*>(a.c) + row * a.ldc + col, v, a.n - col, a.vec);
    }
  }
  tc::fence_before();
  __syncwarp();
  tc::cluster_sync();
  if (warp == 1) {
    __syncwarp();
    tc::fence_after();
    tc::tmem_dealloc_pair(tmem_base, 512);
  }
}

template <bool B_MN, bool COL, typename TC, bool SPLIT>
void launch_pair(const CUtensorMap& ta, const CUtensorMap& tb, const CUtensorMap& tsa,
                 const CUtensorMap& tsb, const MatmulArgs& a, int splits, cudaStream_t s) {
  auto kernel = fp8_matmul_kernel<B_MN, COL, TC, SPLIT>;
  ensure_dynamic_smem(kernel, SMEM_BYTES);
  const int64_t units = a.end - a.first;
  const int64_t pairs = SPLIT ? units * splits : std::min<int64_t>(units, sm_count() / 2);
  trace_begin(GPTQ_K_FP8_MATMUL, s);
  launch_cluster("fp8_matmul_kernel", kernel, dim3(static_cast<unsigned>(2 * pairs)), dim3(THREADS),
                 static_cast<unsigned>(2 * splits), SMEM_BYTES, s, true, ta, tb, tsa, tsb, a);
  trace_end(GPTQ_K_FP8_MATMUL, s);
}

// The tiles are taken in waves of a tile a pair.  How many pairs share a tile of the last wave,
// where that one is less than half full: a join, 5 us, and after other waves a launch, 5 us, for
// half or three quarters of a tile's time.  With and without: 8192 x 8192 x 28672 1550 and 1580 us,
// dx of 4096 x 14336 x 4096 190 and 205, 700 x 8192 x 28672 180 and 214, 2048 x 2560 x 4096 39 and
// 41; where it would save 7 us after another wave, 4096 x 4096 x 4096 95 and 91.
int tail_splits(int64_t units, int64_t nk) {
  const int64_t pairs = sm_count() / 2, rest = units % pairs;
  const double cost = units < pairs ? 5.0 : 10.0;
  for (int splits = 4; splits > 1; splits /= 2)
    if (rest > 0 && 2 * rest * splits <= fp8_few_slots(2 * splits) &&
        0.45 * static_cast<double>(nk - ceil_div(nk, splits)) > cost)
      return splits;
  return 1;
}

// Which kernel, and with which tile and split: the least of the times that a model gives, in us.
// A CTA of the few-rows kernel takes 4.5 + tb a block of its share of the contraction, times the
// waves where each has an SM to itself; all of them take what the weight's blocks need at 5.9 TB/s;
// the shorter of the two hides to three quarters behind the longer, and a CTA costs 0.013 to 0.03 to start
// (and 1 to 2.2 to join).  A wave of the paired kernel costs 3 + 0.45 a block, and 3 to join.  Both
// sides at the crossings, measured: 512 x 4096 x 4096 21.4 us in tiles of 128 tokens, 18.5 in pairs
// with two shares; 256 x 8192 x 28672 101 us in tiles, 62 in pairs with two shares; 128 x 8192 x
// 28672 56 and 59; 333 x 1111 x 5003 18.6 in tiles, 59 in pairs with one share; 16 x 8192 x 28672 45 us with four shares, 47 with two or
// eight, 66 with one, 108 in pairs; 9 x 28672 x 8192 42 us with one share, 46 with two;
// 16 x 1024 x 8192 10.4 us with eight, 12.5 with four; 64 x 14336 x 4096 15.4 us with one share
// and a whole SM, 18.6 with two and half an SM, 64 x 4096 x 14336 17.3 us with four and a whole
// SM, 16.7 with eight and half an SM.
struct Choice {
  int tokens, splits;  // tokens 0: the paired kernel, `splits` shares of a tile of the last wave
};
Choice choose_few(const Fp8Matmul& p, bool only_few) {
  Choice best = {0, 1};
  if (p.sb_group != 128) return best;  // scales of single columns: the paired kernel only
  const int64_t nsm = sm_count(), nk = ceil_div(p.k, BK), jt = ceil_div(p.n, 128);
  const int64_t units = ceil_div(p.m, 2 * BM) * ceil_div(p.n, BN);
  double least = 1e30;
  if (!only_few) {
    const int tail = tail_splits(units, nk);
    const int64_t waves = units / (nsm / 2), rest = units % (nsm / 2);
    least = 6.0 + static_cast<double>(waves) * (3.0 + 0.45 * static_cast<double>(nk)) +
            (rest == 0 ? 0.0 : 3.0 + 0.45 * static_cast<double>(ceil_div(nk, tail)) + (tail > 1 ? 3.0 : 0.0)) +
            (tail > 1 && waves > 0 ? 5.0 : 0.0);
    best = {0, tail};
  }
  const int tokens[4] = {16, 32, 64, 128};
  const double tb[2][4] = {{0.25, 0.26, 0.33, 0.36}, {0.25, 0.30, 0.50, 0.36}};  // one, two an SM
  for (int i = 0; i < (only_few ? 1 : 4); ++i) {
    if (i > 0 && p.m <= tokens[i - 1]) break;  // no tile wider than the tokens need
    for (int splits = 1; splits <= 8; splits *= 2) {
      const int64_t per = ceil_div(nk, splits), ctas = jt * ceil_div(p.m, tokens[i]) * splits;
      const bool two = !only_few && fp8_few_two_per_sm(ctas, splits, tokens[i]);
      const double chain = static_cast<double>(two ? 1 : ceil_div(ctas, fp8_few_slots(splits))) * (4.5 + tb[two][i] * static_cast<double>(per));
      const double stream = static_cast<double>(ctas * per) * (BK * BK / 5.9e6);
      const double t = std::max(chain, stream) + 0.25 * std::min(chain, stream) +
                       0.0102 * (1.0 + tokens[i] / 64.0) * static_cast<double>(ctas) + (splits > 1 ? 0.6 + 0.025 * std::min(tokens[i], 64) : 0.0);
      if (t < least) {
        least = t;
        best = {tokens[i], splits};
      }
    }
  }
  return best;
}

}  // namespace

void launch_fp8_matmul_tokens(const Fp8Matmul& p, const void* x, bool x_bf16, int64_t ldx,
                              DevStatus* st, cudaStream_t s) {
  if (p.m == 0 || p.n == 0) return;
  launch_fp8_matmul_few(p, 16, choose_few(p, true).splits, x, x_bf16, ldx, st, s);
}

void launch_fp8_matmul(const Fp8Matmul& p, DevStatus* st, cudaStream_t s) {
  if (p.m == 0 || p.n == 0) return;
  const Choice few = choose_few(p, false);
  if (few.tokens != 0)
    return launch_fp8_matmul_few(p, few.tokens, few.splits, nullptr, false, 0, st, s);
  MatmulArgs a = {};
  a.sb = p.sb;
  a.sb_n = p.sb_n;
  a.sb_k = p.sb_k;
  a.m = p.m;
  a.n = p.n;
  a.nk = static_cast<int>(ceil_div(p.k, BK));
  a.per = a.nk;
  a.mt = ceil_div(p.m, 2 * BM);
  a.nt = ceil_div(p.n, BN);
  a.c = p.c;
  a.ldc = p.ldc;
  const size_t es = p.c_bf16 ? 2 : 4;
  a.vec = reinterpret_cast<uintptr_t>(p.c) % 32 == 0 && (static_cast<size_t>(p.ldc) * es) % 32 == 0;
  a.st = st;
  a.wait_ns = wait_limit_ns();
  CUtensorMap ta, tb, tsa, tsb;
  make_tmap_2d(&ta, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.a, static_cast<uint64_t>(p.k),
               static_cast<uint64_t>(p.m), static_cast<uint64_t>(p.lda), BK, BM,
               CU_TENSOR_MAP_SWIZZLE_128B);
  if (p.b_mn)
    make_tmap_2d(&tb, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.b, static_cast<uint64_t>(p.n),
                 static_cast<uint64_t>(p.k), static_cast<uint64_t>(p.ldb), BN / 2, BK,
                 CU_TENSOR_MAP_SWIZZLE_128B);
  else
    make_tmap_2d(&tb, CU_TENSOR_MAP_DATA_TYPE_UINT8, p.b, static_cast<uint64_t>(p.k),
                 static_cast<uint64_t>(p.n), static_cast<uint64_t>(p.ldb), BK, BN / 2,
                 CU_TENSOR_MAP_SWIZZLE_128B);
  make_tmap_2d(&tsa, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, p.sa, static_cast<uint64_t>(p.m),
               static_cast<uint64_t>(a.nk), static_cast<uint64_t>(p.sa_k) * 4, BM, 1,
               CU_TENSOR_MAP_SWIZZLE_NONE);
  if (p.sb_group == 1)
    make_tmap_2d(&tsb, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, p.sb, static_cast<uint64_t>(p.n),
                 static_cast<uint64_t>(a.nk), static_cast<uint64_t>(p.sb_k) * 4, BN, 1,
                 CU_TENSOR_MAP_SWIZZLE_NONE);
  else
    tsb = tb;
  a.end = a.mt * a.nt;
  if (p.sb_group == 1) {
    if (p.c_bf16) launch_pair<false, true, __nv_bfloat16, false>(ta, tb, tsa, tsb, a, 1, s);
    else launch_pair<false, true, float, false>(ta, tb, tsa, tsb, a, 1, s);
    return;
  }
  if (few.splits > 1) a.end -= a.end % (sm_count() / 2);
  if (a.end > 0) {
    if (p.b_mn) p.c_bf16 ? launch_pair<true, false, __nv_bfloat16, false>(ta, tb, tsa, tsb, a, 1, s)
                         : launch_pair<true, false, float, false>(ta, tb, tsa, tsb, a, 1, s);
    else p.c_bf16 ? launch_pair<false, false, __nv_bfloat16, false>(ta, tb, tsa, tsb, a, 1, s)
                  : launch_pair<false, false, float, false>(ta, tb, tsa, tsb, a, 1, s);
  }
  if (few.splits > 1) {
    const int n = few.splits;
    a.first = a.end;
    a.end = a.mt * a.nt;
    a.per = static_cast<int>(ceil_div(a.nk, n));
    if (p.b_mn) p.c_bf16 ? launch_pair<true, false, __nv_bfloat16, true>(ta, tb, tsa, tsb, a, n, s)
                         : launch_pair<true, false, float, true>(ta, tb, tsa, tsb, a, n, s);
    else p.c_bf16 ? launch_pair<false, false, __nv_bfloat16, true>(ta, tb, tsa, tsb, a, n, s)
                  : launch_pair<false, false, float, true>(ta, tb, tsa, tsb, a, n, s);
  }
}

}  // namespace gptq
