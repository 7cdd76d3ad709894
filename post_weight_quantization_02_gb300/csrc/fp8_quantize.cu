// e4m3 codes with one float32 scale for every 128 values: the operands of the 8-bit linear
// layer (fp8_matmul.cu).
//
// A group is 128 consecutive columns of a row (rows form), 128 consecutive rows of a column
// (columns form, codes written transposed) or a 128 x 128 block (blocks form); the last group
// of an axis may be short.  For a group with largest magnitude amax
//     scale = max(amax / 448, 2^-126)          code = e4m3(x / scale)
// with both quotients in float32, rounded to nearest, and the code rounded to nearest even
// (448 is the largest e4m3 value).  A NaN or an infinity makes its group's scale non-finite,
// so that whatever reads the group comes out non-finite too.
//
// Bound by memory: an element is read once (2 or 4 bytes) and its code written once.  One CTA
// takes one 128 x 128 tile whatever the form, so a tile's amax in either direction, or both,
// comes from one read: thread (rg, c8) of 256 holds rows 8 rg .. 8 rg + 7 of columns
// 8 c8 .. 8 c8 + 7, loaded 16 bytes at a time with all of a thread's loads in flight together.
#include "common.cuh"
#include "fp8_common.cuh"
#include "kernels.cuh"

namespace gptq {

namespace {

constexpr int kThreads = 256;

struct Fp8QuantArgs {
  const void* x;
  int64_t ldx;
  int64_t rows;
  int cols;
  int col_tiles;
  uint8_t* codes;      // rows / blocks: [rows][ldc]
  int64_t ldc;
  float* scales;       // rows: [col_tiles][lds], the first rows of it; blocks: [row tiles][col_tiles]
  int64_t lds;
  uint8_t* codes_t;    // columns: [cols][ldt]
  int64_t ldt;
  float* scales_t;     // columns: [row tiles][lds_t], the first cols of a row
  int64_t lds_t;
};

// eight codes to p (8-byte aligned); only the first n exist
__device__ __forceinline__ void store8(uint8_t* p, uint2 c, int n) {
  if (n >= 8) {
    *reinterpret_cast<uint2*>(p) = c;
    return;
  }
  const uint64_t w = static_cast<uint64_t>(c.y) << 32 | c.x;
  for (int j = 0; j < n; ++j) p[j] = static_cast<uint8_t>(w >> (8 * j));
}

// VEC: every row of x starts on a 16-byte boundary
template <typename T, int FORMS, bool VEC>
__global__ void __launch_bounds__(kThreads) fp8_quantize_kernel(const Fp8QuantArgs a) {
  constexpr bool ROWS = (FORMS & GPTQ_FP8_ROWS) != 0, COLUMNS = (FORMS & GPTQ_FP8_COLUMNS) != 0,
                 BLOCKS = (FORMS & GPTQ_FP8_BLOCKS) != 0;
  __shared__ MaxPair<T> colmax[COLUMNS ? kThreads / 32 : 1][64];  // of each warp's 16 rows
  __shared__ float2 colscale[COLUMNS ? 128 : 1];                  // scale, minus its reciprocal
  __shared__ uint32_t warpmax[kThreads / 32];
  __shared__ uint2 tile[COLUMNS ? 128 * 16 : 1];  // [column][8-row chunk ^ c8]

  // a product launched behind this kernel may begin to set up (it waits before it reads)
  griddep_launch_dependents();
  const int tid = threadIdx.x, lane = tid % 32;
  const int c8 = tid % 16, rg = tid / 16;
  const int64_t rt = blockIdx.x / static_cast<unsigned>(a.col_tiles);
  const int ct = static_cast<int>(blockIdx.x % static_cast<unsigned>(a.col_tiles));
  const int64_t row0 = rt * 128 + 8 * rg;
  const int col = ct * 128 + 8 * c8;
  const int nrow = static_cast<int>(min(static_cast<int64_t>(8), a.rows - row0));  // may be <= 0
  const int ncol = min(8, a.cols - col);

  Eight<T> v[8];
  const T* px = static_cast<const T*>(a.x) + row0 * a.ldx + col;
  // Whole tiles are loaded without a branch between the loads, so that all are in flight
  // together; only threads at the matrix's edges go element by element.
  bool loaded = false;
  if constexpr (VEC) {
    if (nrow == 8 && ncol == 8) {
      loaded = true;
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i].load(px + i * a.ldx);
    }
  } else {
    // aligned pieces from the boundary before each row's 128 values on, where all of them lie
    // between the matrix's first and last element
    constexpr int kSpan = 128 * sizeof(T) + 16;
    const char* lo = static_cast<const char*>(a.x);
    const char* hi = lo + ((a.rows - 1) * a.ldx + a.cols) * sizeof(T);
    const char* r0 = reinterpret_cast<const char*>(px - 8 * c8);
    const char* r7 = r0 + 7 * a.ldx * sizeof(T);
    loaded = __all_sync(0xffffffffu, nrow == 8 && r0 - 15 >= lo && r7 + kSpan <= hi);
    if (loaded) {
      uint4 next[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const char* first = r0 + i * a.ldx * sizeof(T);
        const T* mine = reinterpret_cast<const T*>(first - reinterpret_cast<uintptr_t>(first) % 16) + 8 * c8;
        v[i].load(mine);
        // float32: lane 15 alone reads on (columns of 4099 x 5003 32 us, 40 where all lanes read);
        // bf16: every lane reads, without a predicate (rows of 4099 x 5003 22.8 us, 23.7 with one)
        if (sizeof(T) == 2) next[i] = __ldcs(reinterpret_cast<const uint4*>(mine + (c8 == 15 ? 8 : 0)));
        else next[i] = c8 == 15 ? __ldcs(reinterpret_cast<const uint4*>(mine + 8)) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        realign(v[i], next[i], static_cast<int>(reinterpret_cast<uintptr_t>(r0 + i * a.ldx * sizeof(T)) % 16));
        if (ncol < 8) keep_first(v[i], max(ncol, 0));
      }
    }
  }
  if (!loaded) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i].load_some(px + i * a.ldx, i < nrow ? ncol : 0);
  }

  if constexpr (ROWS) {
    // each row's magnitude over its 16 lanes: at every step a lane passes on half of its rows
    // and keeps the other half, until lane c8 holds row c8 / 2
    uint32_t m[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      MaxPair<T> p = {};
#pragma unroll
      for (int j = 0; j < 4; ++j) p.add(v[i], j);
      m[i] = max(p.even(), p.odd());
    }
#pragma unroll
    for (int o = 8, n = 4; n > 0; o >>= 1, n >>= 1) {
      const bool up = (lane & o) != 0;
#pragma unroll
      for (int i = 0; i < n; ++i) {
        const uint32_t give = up ? m[i] : m[i + n], keep = up ? m[i + n] : m[i];
        m[i] = max(keep, __shfl_xor_sync(0xffffffffu, give, o));
      }
    }
    m[0] = max(m[0], __shfl_xor_sync(0xffffffffu, m[0], 1));
    const float mine = scale_of(m[0]), inverse = minus_reciprocal_of(m[0], mine);
    if ((c8 & 1) == 0 && c8 / 2 < nrow) a.scales[static_cast<int64_t>(ct) * a.lds + row0 + c8 / 2] = mine;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float s = __shfl_sync(0xffffffffu, mine, (lane & 16) + 2 * i);
      const float y = __shfl_sync(0xffffffffu, inverse, (lane & 16) + 2 * i);
      if (i < nrow && ncol > 0) store8(a.codes + (row0 + i) * a.ldc + col, codes8(v[i], s, y), ncol);
    }
  }
  if constexpr (BLOCKS) {
    MaxPair<T> p = {};
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) p.add(v[i], j);
    uint32_t m = __reduce_max_sync(0xffffffffu, max(p.even(), p.odd()));
    if (lane == 0) warpmax[tid / 32] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) m = max(m, warpmax[w]);
    const float s = scale_of(m), y = minus_reciprocal_of(m, s);
    if (tid == 0) a.scales[rt * a.col_tiles + ct] = s;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < nrow && ncol > 0) store8(a.codes + (row0 + i) * a.ldc + col, codes8(v[i], s, y), ncol);
  }
  if constexpr (COLUMNS) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      MaxPair<T> p = {};
#pragma unroll
      for (int i = 0; i < 8; ++i) p.add(v[i], j);
      p.join_lane16();
      if (lane < 16) colmax[tid / 32][4 * c8 + j] = p;
    }
    __syncthreads();
    if (tid < 128) {
      MaxPair<T> p = colmax[0][tid / 2];
#pragma unroll
      for (int w = 1; w < kThreads / 32; ++w) p.join(colmax[w][tid / 2]);
      const uint32_t m = tid % 2 == 0 ? p.even() : p.odd();
      const float s = scale_of(m);
      colscale[tid] = make_float2(s, minus_reciprocal_of(m, s));
      if (ct * 128 + tid < a.cols) a.scales_t[rt * a.lds_t + ct * 128 + tid] = s;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 se = colscale[8 * c8 + 2 * j], so = colscale[8 * c8 + 2 * j + 1];
      const float2 s = make_float2(se.x, so.x), y = make_float2(se.y, so.y);
      uint32_t c[8], turn = 0;  // the even column's code in the low byte, the odd one's above
      if (y.x != 0.0f && y.y != 0.0f) {
        turn = kTurnSigns;
#pragma unroll
        for (int i = 0; i < 8; ++i) c[i] = codes2(minus_quotient(v[i].pair(j), s, y));
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 x = v[i].pair(j);
          c[i] = codes2(make_float2(divide_pair(x, s.x).x, divide_pair(x, s.y).y));
        }
      }
      // a column's chunks of 8 rows are permuted by its c8, so that the 16 lanes that store
      // one row group hit 16 different bank pairs
      const uint32_t a0 = __byte_perm(c[0], c[1], 0x5140) ^ turn, a1 = __byte_perm(c[2], c[3], 0x5140) ^ turn;
      const uint32_t a2 = __byte_perm(c[4], c[5], 0x5140) ^ turn, a3 = __byte_perm(c[6], c[7], 0x5140) ^ turn;
      tile[(8 * c8 + 2 * j) * 16 + (rg ^ c8)] =
          make_uint2(__byte_perm(a0, a1, 0x5410), __byte_perm(a2, a3, 0x5410));
      tile[(8 * c8 + 2 * j + 1) * 16 + (rg ^ c8)] =
          make_uint2(__byte_perm(a0, a1, 0x7632), __byte_perm(a2, a3, 0x7632));
    }
    __syncthreads();
    // thread (g, m): column 16 i + g, rows 8 m .. 8 m + 7
    const int m = tid % 16, g = tid / 16;
    const int n = static_cast<int>(min(static_cast<int64_t>(8), a.rows - rt * 128 - 8 * m));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int cc = 16 * i + g;
      if (ct * 128 + cc < a.cols && n > 0)
        store8(a.codes_t + static_cast<int64_t>(ct * 128 + cc) * a.ldt + rt * 128 + 8 * m,
               tile[cc * 16 + (m ^ (cc / 8))], n);
    }
  }
}

template <typename T, int FORMS>
void launch_form(const Fp8QuantArgs& a, bool vec, unsigned grid, cudaStream_t s) {
  if (vec) GPTQ_LAUNCH(GPTQ_K_FP8_QUANTIZE, s, (fp8_quantize_kernel<T, FORMS, true>), grid, kThreads, 0, a);
  else GPTQ_LAUNCH(GPTQ_K_FP8_QUANTIZE, s, (fp8_quantize_kernel<T, FORMS, false>), grid, kThreads, 0, a);
}

template <typename T>
void launch_typed(int forms, const Fp8QuantArgs& a, bool vec, unsigned grid, cudaStream_t s) {
  switch (forms) {
    case GPTQ_FP8_ROWS: return launch_form<T, GPTQ_FP8_ROWS>(a, vec, grid, s);
    case GPTQ_FP8_COLUMNS: return launch_form<T, GPTQ_FP8_COLUMNS>(a, vec, grid, s);
    case GPTQ_FP8_BLOCKS: return launch_form<T, GPTQ_FP8_BLOCKS>(a, vec, grid, s);
    case GPTQ_FP8_ROWS | GPTQ_FP8_COLUMNS:
      return launch_form<T, (GPTQ_FP8_ROWS | GPTQ_FP8_COLUMNS)>(a, vec, grid, s);
    default: fail(GPTQ_ERR_INVALID_ARG, "fp8 quantiser: unknown form %d", forms);
  }
}

}  // namespace

void launch_fp8_quantize(const void* x, bool bf16, int64_t rows, int cols, int64_t ldx, int forms,
                         uint8_t* codes, int64_t ldc, float* scales, int64_t lds, uint8_t* codes_t,
                         int64_t ldt, float* scales_t, int64_t lds_t, cudaStream_t s) {
  Fp8QuantArgs a;
  a.x = x;
  a.ldx = ldx;
  a.rows = rows;
  a.cols = cols;
  a.col_tiles = static_cast<int>(ceil_div(cols, 128));
  a.codes = codes;
  a.ldc = ldc;
  a.scales = scales;
  a.lds = lds;
  a.codes_t = codes_t;
  a.ldt = ldt;
  a.scales_t = scales_t;
  a.lds_t = lds_t;
  const int64_t tiles = ceil_div(rows, 128) * a.col_tiles;
  if (tiles == 0) return;
  if (tiles > 0x7fffffff) fail(GPTQ_ERR_UNSUPPORTED, "fp8 quantiser: more than 2^31 tiles of 128 x 128");
  const size_t es = bf16 ? 2 : 4;
  // 16-byte loads where every row starts on a 16-byte boundary; element loads otherwise
  const bool vec = reinterpret_cast<uintptr_t>(x) % 16 == 0 && (static_cast<size_t>(ldx) * es) % 16 == 0;
  if (bf16) launch_typed<__nv_bfloat16>(forms, a, vec, static_cast<unsigned>(tiles), s);
  else launch_typed<float>(forms, a, vec, static_cast<unsigned>(tiles), s);
}

}  // namespace gptq
