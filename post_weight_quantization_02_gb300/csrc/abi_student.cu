// The C ABI of what an 8-bit student needs: the fp8 quantiser and linear layer, the teacher's
// top logits and the distillation loss.  These entry points check their arguments, enqueue
// and return; device-side failures collect in one status word per device (include/gptq.h).
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <limits>
#include <mutex>

#include "abi_common.cuh"
#include "common.cuh"
#include "kernels.cuh"
#include "logits_common.cuh"

namespace gptq {
namespace {

__device__ __align__(256) DevStatus g_async_status;  // zero when the module loads
__device__ __align__(256) DevStatus g_async_taken;   // what a report took of it

// Takes the status and clears it in one go: a failure that another stream's kernel records
// meanwhile is in this report or in the next.
__global__ void take_status_kernel() {
  g_async_taken.timeouts = atomicExch(&g_async_status.timeouts, 0);
  g_async_taken.code = atomicExch(&g_async_status.code, 0);
  g_async_taken.info = g_async_status.info;
}

// Address of the status word on the current device, asked from the runtime once per host
// thread and device.
DevStatus* async_status() {
  int dev = 0;
  GPTQ_CUDA(cudaGetDevice(&dev));
  thread_local int cached_dev = -1;
  thread_local DevStatus* cached = nullptr;
  if (dev != cached_dev) {
    void* p = nullptr;
    GPTQ_CUDA(cudaGetSymbolAddress(&p, g_async_status));
    cached = static_cast<DevStatus*>(p);
    cached_dev = dev;
  }
  return cached;
}

bool known_dtype(int t) { return t == GPTQ_F32 || t == GPTQ_BF16; }
size_t elt(int t) { return t == GPTQ_BF16 ? 2 : 4; }
// a row of codes in the workspace starts on a 128-byte line
int64_t code_ld(int64_t n) { return (n + 127) / 128 * 128; }

void check_codes(const void* codes, int64_t ld, int64_t cols, const char* null_msg,
                 const char* align_msg) {
  require(codes != nullptr && ld >= cols, GPTQ_ERR_INVALID_ARG, null_msg);
  require(aligned(codes, 16) && ld % 16 == 0, GPTQ_ERR_UNSUPPORTED, align_msg);
}

struct Fp8Operand {
  uint8_t* codes;
  float* scales;
};

// a row of scales in the workspace: TMA reads it from 16-byte boundaries
int64_t scale_ld(int64_t n) { return (n + 3) / 4 * 4; }

// Codes of `rows` rows of `cols` and scales of ceil(cols / 128) rows of scale_ld(rows).
Fp8Operand take_operand(WsCarver& w, int64_t rows, int64_t cols) {
  Fp8Operand o;
  o.codes = w.take<uint8_t>(static_cast<size_t>(rows) * code_ld(cols));
  o.scales = w.take<float>(static_cast<size_t>(ceil_div(cols, 128)) * scale_ld(rows));
  return o;
}
void plan_operand(WsPlan& w, int64_t rows, int64_t cols) {
  w.add<uint8_t>(static_cast<size_t>(rows) * code_ld(cols));
  w.add<float>(static_cast<size_t>(ceil_div(cols, 128)) * scale_ld(rows));
}

// pointers to 32-bit numbers, null or not
template <typename... P>
void check_words(const char* msg, const P*... p) {
  require((aligned(p, 4) && ...), GPTQ_ERR_INVALID_ARG, msg);
}

void check_logits(const void* logits, int dtype, int64_t rows, int32_t vocab, int64_t ld,
                  int32_t k) {
  require(rows >= 0 && vocab > 0 && ld >= vocab, GPTQ_ERR_INVALID_ARG,
          "logits: need rows >= 0, vocab > 0 and a row stride of at least vocab");
  require(known_dtype(dtype), GPTQ_ERR_INVALID_ARG, "logits: dtype must be GPTQ_F32 or GPTQ_BF16");
  require(k >= 1, GPTQ_ERR_INVALID_ARG, "logits: k must be at least 1");
  require(k <= kMaxTop, GPTQ_ERR_UNSUPPORTED, "logits: k must be at most 256");
  require(vocab <= std::numeric_limits<int32_t>::max() - 65536 &&
              rows <= std::numeric_limits<int32_t>::max(),
          GPTQ_ERR_UNSUPPORTED, "logits: rows and vocab must be below 2^31 - 65536");
  require(rows == 0 || (logits != nullptr && aligned(logits, elt(dtype))), GPTQ_ERR_INVALID_ARG,
          "logits: null or misaligned pointer");
}

void check_teacher(int64_t rows, const float* t_values, const int32_t* t_indices,
                   const float* weights, float temperature) {
  require(rows == 0 || (t_values != nullptr && t_indices != nullptr), GPTQ_ERR_INVALID_ARG,
          "distillation: null teacher values or indices");
  check_words("distillation: misaligned teacher values, indices or weights", t_values, t_indices, weights);
  // the kernels work with log2(e) / T
  require(std::isfinite(temperature) && temperature > 0.0f && std::isfinite(kLog2e / temperature),
          GPTQ_ERR_INVALID_ARG, "distillation: temperature must be finite and > 0");
}

DistillArgs distill_args(const void* logits, int64_t rows, int32_t vocab, int64_t ld,
                         const float* t_values, const int32_t* t_indices, int32_t k,
                         float temperature, const float* weights) {
  DistillArgs a = {};
  a.logits = logits;
  a.ld = ld;
  a.rows = rows;
  a.vocab = vocab;
  a.t_values = t_values;
  a.t_indices = t_indices;
  a.k = k;
  a.inv_temp = 1.0f / temperature;
  a.weights = weights;
  a.wait_ns = wait_limit_ns();
  return a;
}

void check_gradient(const void* logits, int dtype, int64_t rows, int32_t vocab, int64_t ld,
                    const void* dlogits, int64_t ldd) {
  require(rows == 0 || (dlogits != nullptr && aligned(dlogits, elt(dtype))), GPTQ_ERR_INVALID_ARG,
          "distillation: null or misaligned dlogits");
  require(ldd >= vocab && (dlogits != logits || ldd == ld), GPTQ_ERR_INVALID_ARG,
          "distillation: dlogits needs a row stride of at least vocab, and the logits' own in place");
}

}  // namespace

size_t fp8_linear_ws_bytes(int64_t ntok, int d_out, int d_in) {
  WsPlan w;
  if (!fp8_quantises_tokens(ntok, d_out, d_in)) plan_operand(w, ntok, d_in);
  return std::max<size_t>(w.bytes, 256);
}

size_t fp8_backward_ws_bytes(int64_t ntok, int d_out, int d_in) {
  WsPlan w;
  plan_operand(w, ntok, d_out);  // dy along d_out
  plan_operand(w, d_out, ntok);  // dy along the tokens
  plan_operand(w, d_in, ntok);   // x along the tokens
  return std::max<size_t>(w.bytes, 256);
}

}  // namespace gptq

using namespace gptq;

extern "C" {

gptq_status gptq_fp8_quantize(const void* x, int xdtype, int64_t rows, int32_t cols, int64_t ldx,
                              int form, uint8_t* codes, int64_t ldc, float* scales, void* stream) {
  return guarded([&] {
    require(rows >= 0 && cols >= 0 && ldx >= cols, GPTQ_ERR_INVALID_ARG,
            "gptq_fp8_quantize: need rows, cols >= 0 and a row stride of at least cols");
    require(known_dtype(xdtype), GPTQ_ERR_INVALID_ARG,
            "gptq_fp8_quantize: xdtype must be GPTQ_F32 or GPTQ_BF16");
    require(form == GPTQ_FP8_ROWS || form == GPTQ_FP8_COLUMNS || form == GPTQ_FP8_BLOCKS,
            GPTQ_ERR_INVALID_ARG, "gptq_fp8_quantize: unknown form");
    if (rows == 0 || cols == 0) return;
    require(x != nullptr && scales != nullptr && aligned(x, elt(xdtype)), GPTQ_ERR_INVALID_ARG,
            "gptq_fp8_quantize: null or misaligned x or scales");
    check_words("gptq_fp8_quantize: misaligned scales", scales);
    const bool t = form == GPTQ_FP8_COLUMNS;
    check_codes(codes, ldc, t ? rows : cols, "gptq_fp8_quantize: null codes or too short rows",
                "gptq_fp8_quantize: codes must be 16-byte aligned, ldc a multiple of 16");
    launch_fp8_quantize(x, xdtype == GPTQ_BF16, rows, cols, ldx, form, t ? nullptr : codes, ldc,
                        t ? nullptr : scales, rows, t ? codes : nullptr, ldc, t ? scales : nullptr, cols,
                        static_cast<cudaStream_t>(stream));
  });
}

gptq_status gptq_fp8_linear(const void* x, int xdtype, int64_t ntok, int64_t ldx,
                            const uint8_t* w_codes, int64_t ldw, const float* w_scales,
                            int32_t d_out, int32_t d_in, void* y, int ydtype, int64_t ldy,
                            void* ws, size_t ws_bytes, void* stream) {
  return guarded([&] {
    require(ntok >= 0 && d_out >= 0 && d_in > 0 && ldx >= d_in && ldy >= d_out,
            GPTQ_ERR_INVALID_ARG,
            "gptq_fp8_linear: need ntok, d_out >= 0, d_in > 0 and row strides of at least a row");
    require(known_dtype(xdtype) && known_dtype(ydtype), GPTQ_ERR_INVALID_ARG,
            "gptq_fp8_linear: element types must be GPTQ_F32 or GPTQ_BF16");
    if (ntok == 0 || d_out == 0) return;
    require(x != nullptr && w_scales != nullptr && y != nullptr && aligned(x, elt(xdtype)) &&
                aligned(y, elt(ydtype)) && aligned(w_scales, 4),
            GPTQ_ERR_INVALID_ARG, "gptq_fp8_linear: null or misaligned x, w_scales or y");
    check_codes(w_codes, ldw, d_in, "gptq_fp8_linear: null w_codes or too short rows",
                "gptq_fp8_linear: w_codes must be 16-byte aligned, ldw a multiple of 16");
    require(ntok <= std::numeric_limits<int32_t>::max(), GPTQ_ERR_UNSUPPORTED,
            "gptq_fp8_linear: ntok must be below 2^31");
    const bool few = fp8_quantises_tokens(ntok, d_out, d_in);
    require(few || (ws != nullptr && aligned(ws, 256)), GPTQ_ERR_INVALID_ARG,
            "gptq_fp8_linear: null or unaligned ws");
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    Fp8Matmul p = {};
    p.b = w_codes;
    p.ldb = ldw;
    p.sb = w_scales;
    p.sb_group = 128;
    p.sb_n = ceil_div(d_in, 128);
    p.sb_k = 1;
    p.m = ntok;
    p.n = d_out;
    p.k = d_in;
    p.c = y;
    p.c_bf16 = ydtype == GPTQ_BF16;
    p.ldc = ldy;
    if (few) return launch_fp8_matmul_tokens(p, x, xdtype == GPTQ_BF16, ldx, async_status(), s);
    WsCarver wc(ws, ws_bytes);
    const Fp8Operand qx = take_operand(wc, ntok, d_in);
    DevStatus* st = async_status();
    p.a = qx.codes;
    p.lda = code_ld(d_in);
    p.sa = qx.scales;
    p.sa_k = scale_ld(ntok);
    launch_fp8_quantize(x, xdtype == GPTQ_BF16, ntok, d_in, ldx, GPTQ_FP8_ROWS, qx.codes,
                        code_ld(d_in), qx.scales, scale_ld(ntok), nullptr, 0, nullptr, 0, s);
    launch_fp8_matmul(p, st, s);
  });
}

gptq_status gptq_fp8_linear_backward(const void* dy, int dydtype, int64_t lddy, const void* x,
                                     int xdtype, int64_t ldx, int64_t ntok,
                                     const uint8_t* w_codes, int64_t ldw, const float* w_scales,
                                     int32_t d_out, int32_t d_in, void* dx, int dxdtype,
                                     int64_t lddx, void* dw, int dwdtype, int64_t lddw, void* ws,
                                     size_t ws_bytes, void* stream) {
  return guarded([&] {
    require(ntok >= 0 && d_out > 0 && d_in > 0 && lddy >= d_out, GPTQ_ERR_INVALID_ARG,
            "gptq_fp8_linear_backward: need ntok >= 0, d_out, d_in > 0 and row strides of at least a row");
    require(known_dtype(dydtype), GPTQ_ERR_INVALID_ARG,
            "gptq_fp8_linear_backward: element types must be GPTQ_F32 or GPTQ_BF16");
    if (dx == nullptr && dw == nullptr) return;
    require(ntok <= std::numeric_limits<int32_t>::max(), GPTQ_ERR_UNSUPPORTED,
            "gptq_fp8_linear_backward: ntok must be below 2^31");
    require(ntok == 0 || (dy != nullptr && aligned(dy, elt(dydtype))), GPTQ_ERR_INVALID_ARG,
            "gptq_fp8_linear_backward: null or misaligned dy");
    require(ws != nullptr && aligned(ws, 256), GPTQ_ERR_INVALID_ARG,
            "gptq_fp8_linear_backward: null or unaligned ws");
    if (dx != nullptr) {
      require(known_dtype(dxdtype) && aligned(dx, elt(dxdtype)) && lddx >= d_in, GPTQ_ERR_INVALID_ARG,
              "gptq_fp8_linear_backward: dx needs a known type, alignment and a row stride of at least d_in");
      require(w_scales != nullptr && aligned(w_scales, 4), GPTQ_ERR_INVALID_ARG,
              "gptq_fp8_linear_backward: null or misaligned w_scales");
      check_codes(w_codes, ldw, d_in, "gptq_fp8_linear_backward: null w_codes or too short rows",
                  "gptq_fp8_linear_backward: w_codes must be 16-byte aligned, ldw a multiple of 16");
    }
    if (dw != nullptr) {
      require(known_dtype(dwdtype) && aligned(dw, elt(dwdtype)) && lddw >= d_in, GPTQ_ERR_INVALID_ARG,
              "gptq_fp8_linear_backward: dw needs a known type, alignment and a row stride of at least d_in");
      require(known_dtype(xdtype) && ldx >= d_in &&
                  (ntok == 0 || (x != nullptr && aligned(x, elt(xdtype)))),
              GPTQ_ERR_INVALID_ARG, "gptq_fp8_linear_backward: dw needs x [ntok, d_in]");
    }
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (ntok == 0) {
      if (dw != nullptr)
        GPTQ_CUDA(cudaMemset2DAsync(dw, lddw * elt(dwdtype), 0, d_in * elt(dwdtype), d_out, s));
      return;
    }
    WsCarver wc(ws, ws_bytes);
    const Fp8Operand qy = take_operand(wc, ntok, d_out);
    const Fp8Operand qyt = take_operand(wc, d_out, ntok);
    const Fp8Operand qxt = take_operand(wc, d_in, ntok);
    DevStatus* st = async_status();
    const int64_t ldt = code_ld(ntok);
    launch_fp8_quantize(dy, dydtype == GPTQ_BF16, ntok, d_out, lddy,
                        (dx != nullptr ? GPTQ_FP8_ROWS : 0) | (dw != nullptr ? GPTQ_FP8_COLUMNS : 0),
                        qy.codes, code_ld(d_out), qy.scales, scale_ld(ntok), qyt.codes, ldt, qyt.scales, scale_ld(d_out), s);
    if (dw != nullptr)
      launch_fp8_quantize(x, xdtype == GPTQ_BF16, ntok, d_in, ldx, GPTQ_FP8_COLUMNS, nullptr, 0,
                          nullptr, 0, qxt.codes, ldt, qxt.scales, scale_ld(d_in), s);
    if (dx != nullptr) {
      Fp8Matmul p = {};
      p.a = qy.codes;
      p.lda = code_ld(d_out);
      p.b = w_codes;
      p.ldb = ldw;
      p.b_mn = true;
      p.sa = qy.scales;
      p.sa_k = scale_ld(ntok);
      p.sb = w_scales;
      p.sb_group = 128;
      p.sb_n = 1;
      p.sb_k = ceil_div(d_in, 128);
      p.m = ntok;
      p.n = d_in;
      p.k = d_out;
      p.c = dx;
      p.c_bf16 = dxdtype == GPTQ_BF16;
      p.ldc = lddx;
      launch_fp8_matmul(p, st, s);
    }
    if (dw != nullptr) {
      Fp8Matmul p = {};
      p.a = qyt.codes;
      p.lda = ldt;
      p.b = qxt.codes;
      p.ldb = ldt;
      p.sa = qyt.scales;
      p.sa_k = scale_ld(d_out);
      p.sb = qxt.scales;
      p.sb_group = 1;
      p.sb_n = 1;
      p.sb_k = scale_ld(d_in);
      p.m = d_out;
      p.n = d_in;
      p.k = ntok;
      p.c = dw;
      p.c_bf16 = dwdtype == GPTQ_BF16;
      p.ldc = lddw;
      launch_fp8_matmul(p, st, s);
    }
  });
}

gptq_status gptq_top_logits(const void* logits, int dtype, int64_t rows, int32_t vocab,
                            int64_t ld, int32_t k, float* values, int32_t* indices, float* lse,
                            void* stream) {
  return guarded([&] {
    check_logits(logits, dtype, rows, vocab, ld, k);
    require(k <= vocab, GPTQ_ERR_INVALID_ARG, "gptq_top_logits: k must be at most vocab");
    require(rows == 0 || (values != nullptr && indices != nullptr), GPTQ_ERR_INVALID_ARG,
            "gptq_top_logits: null values or indices");
    check_words("gptq_top_logits: misaligned values, indices or lse", values, indices, lse);
    TopArgs a = {};
    a.logits = logits;
    a.ld = ld;
    a.rows = rows;
    a.vocab = vocab;
    a.k = k;
    a.values = values;
    a.indices = indices;
    a.lse = lse;
    launch_top_logits(a, dtype == GPTQ_BF16, static_cast<cudaStream_t>(stream));
  });
}

gptq_status gptq_distill_loss(const void* logits, int dtype, int64_t rows, int32_t vocab,
                              int64_t ld, const float* t_values, const int32_t* t_indices,
                              int32_t k, float temperature, const float* weights, float* loss,
                              float* lse, void* stream) {
  return guarded([&] {
    check_logits(logits, dtype, rows, vocab, ld, k);
    check_teacher(rows, t_values, t_indices, weights, temperature);
    require(rows == 0 || loss != nullptr, GPTQ_ERR_INVALID_ARG, "gptq_distill_loss: null loss");
    check_words("gptq_distill_loss: misaligned loss or lse", loss, lse);
    DistillArgs a = distill_args(logits, rows, vocab, ld, t_values, t_indices, k, temperature, weights);
    a.loss = loss;
    a.lse = lse;
    a.st = async_status();
    launch_distill(a, dtype == GPTQ_BF16, true, false, static_cast<cudaStream_t>(stream));
  });
}

gptq_status gptq_distill_backward(const void* logits, int dtype, int64_t rows, int32_t vocab,
                                  int64_t ld, const float* lse, const float* t_values,
                                  const int32_t* t_indices, int32_t k, float temperature,
                                  const float* weights, const float* grad_loss, void* dlogits,
                                  int64_t ldd, void* stream) {
  return guarded([&] {
    check_logits(logits, dtype, rows, vocab, ld, k);
    check_teacher(rows, t_values, t_indices, weights, temperature);
    require(rows == 0 || lse != nullptr, GPTQ_ERR_INVALID_ARG, "gptq_distill_backward: null lse");
    check_words("gptq_distill_backward: misaligned lse or grad_loss", lse, grad_loss);
    check_gradient(logits, dtype, rows, vocab, ld, dlogits, ldd);
    DistillArgs a = distill_args(logits, rows, vocab, ld, t_values, t_indices, k, temperature, weights);
    a.lse = const_cast<float*>(lse);
    a.grad_loss = grad_loss;
    a.dlogits = dlogits;
    a.ldd = ldd;
    a.st = async_status();
    launch_distill(a, dtype == GPTQ_BF16, false, true, static_cast<cudaStream_t>(stream));
  });
}

gptq_status gptq_distill_loss_grad(const void* logits, int dtype, int64_t rows, int32_t vocab,
                                   int64_t ld, const float* t_values, const int32_t* t_indices,
                                   int32_t k, float temperature, const float* weights,
                                   float* loss, void* dlogits, int64_t ldd, void* stream) {
  return guarded([&] {
    check_logits(logits, dtype, rows, vocab, ld, k);
    check_teacher(rows, t_values, t_indices, weights, temperature);
    require(rows == 0 || loss != nullptr, GPTQ_ERR_INVALID_ARG, "gptq_distill_loss_grad: null loss");
    check_words("gptq_distill_loss_grad: misaligned loss", loss);
    check_gradient(logits, dtype, rows, vocab, ld, dlogits, ldd);
    DistillArgs a = distill_args(logits, rows, vocab, ld, t_values, t_indices, k, temperature, weights);
    a.loss = loss;
    a.dlogits = dlogits;
    a.ldd = ldd;
    a.st = async_status();
    launch_distill(a, dtype == GPTQ_BF16, true, true, static_cast<cudaStream_t>(stream));
  });
}

gptq_status gptq_async_status(void* stream) {
  return guarded([&] {
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    DevStatus h;
    std::memset(&h, 0, sizeof(h));
    {
      static std::mutex mu;  // of g_async_taken
      std::lock_guard<std::mutex> lock(mu);
      take_status_kernel<<<1, 1, 0, s>>>();
      GPTQ_CUDA(cudaGetLastError());
      GPTQ_CUDA(cudaMemcpyFromSymbolAsync(&h, g_async_taken, 3 * sizeof(int), 0, cudaMemcpyDeviceToHost, s));
      GPTQ_CUDA(cudaStreamSynchronize(s));
    }
    trace_flush();
    // a wait that ran out leaves outputs unset: it comes before whatever else was recorded
    if (h.timeouts != 0 || h.code == GPTQ_ERR_TIMEOUT)
      fail(GPTQ_ERR_TIMEOUT, "%d device-side wait(s) of an enqueued call ran out", h.timeouts);
    if (h.code == 0) return;
    if (h.code == GPTQ_ERR_INVALID_ARG)
      fail(GPTQ_ERR_INVALID_ARG, "a teacher index (%d) is not below the vocabulary's size", h.info);
    fail(static_cast<gptq_status>(h.code), "an enqueued call reported status %d", h.code);
  });
}

}  // extern "C"
