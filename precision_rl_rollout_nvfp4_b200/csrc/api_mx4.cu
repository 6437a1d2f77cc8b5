// C ABI of the MXFP4 and gated feed-forward operators (declared in
// include/nvfp4rac.h): argument checks, workspace carving, launches.  No call
// allocates or synchronizes; every check comes before any CUDA work.
#include "mx4.h"
#include "nvfp4rac.h"

using namespace nvfp4;

namespace {

#define NV_CHECK(cond, code)    \
  do {                          \
    if (!(cond)) return (code); \
  } while (0)
#define NV_TRY(expr)                                       \
  do {                                                     \
    if ((expr) != cudaSuccess) return NVFP4_ERR_CUDA;      \
  } while (0)
#define NV_DEVICE()                                                    \
  do {                                                                 \
    const int dc_ = device_check();                                    \
    if (dc_ != 0) return dc_ == 1 ? NVFP4_ERR_DEVICE : NVFP4_ERR_CUDA; \
  } while (0)

// Largest extent of a dimension: row and byte coordinates are 32-bit.
constexpr int64_t kMaxDim = (int64_t(1) << 31) - 1024;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
size_t round256(size_t n) { return (n + 255) & ~size_t(255); }
bool dim_ok(int64_t n, int64_t least) { return n >= least && n <= kMaxDim; }

// Codes and scales given, aligned, with a known layout.
bool filled(const mxfp4_tensor* t) {
  return t && t->codes && t->scales && (t->scale_layout == 0 || t->scale_layout == 1);
}
bool tensor_aligned(const mxfp4_tensor* t) { return aligned16(t->codes) && aligned16(t->scales); }
bool shape_ok(const mxfp4_tensor* t) { return dim_ok(t->rows, 0) && dim_ok(t->cols, 32) && t->cols % 32 == 0; }

// Longest reduction of a product (offsets into a scale row are 32-bit).
constexpr int64_t kMaxK = int64_t(1) << 28;

// An operand of a product (a weight or a quantized activation of at least one row).
nvfp4_status operand(const mxfp4_tensor* t, int64_t cols) {
  NV_CHECK(filled(t) && t->scale_layout == 1, NVFP4_ERR_INVALID_ARG);
  NV_CHECK(shape_ok(t) && t->rows >= 1 && t->cols == cols && cols <= kMaxK, NVFP4_ERR_UNSUPPORTED_SHAPE);
  NV_CHECK(tensor_aligned(t), NVFP4_ERR_MISALIGNED);
  return NVFP4_OK;
}

bool out_aligned(const void* y, int32_t y_dtype) {
  return (reinterpret_cast<uintptr_t>(y) & (y_dtype == 0 ? 3u : 1u)) == 0;
}

bool overlap(const void* a, int64_t a_bytes, const void* b, int64_t b_bytes) {
  const uintptr_t p = reinterpret_cast<uintptr_t>(a), q = reinterpret_cast<uintptr_t>(b);
  return p < q + static_cast<uintptr_t>(b_bytes) && q < p + static_cast<uintptr_t>(a_bytes);
}

mxfp4_tensor carve(uint8_t*& at, int64_t rows, int64_t cols) {
  mxfp4_tensor t{};
  t.codes = at;
  at += round256(static_cast<size_t>(rows) * (cols / 2));
  t.scales = at;
  at += round256(mxfp4_scale_bytes(rows, cols, 1));
  t.rows = rows;
  t.cols = cols;
  t.scale_layout = 1;
  return t;
}
size_t carve_bytes(int64_t rows, int64_t cols) {
  return round256(static_cast<size_t>(rows) * (cols / 2)) + round256(mxfp4_scale_bytes(rows, cols, 1));
}

// X quantized (x.codes), or bf16 rows (x_bf16) that the product quantizes.
cudaError_t product(const mxfp4_tensor& x, const uint16_t* x_bf16, int64_t ldx, const mxfp4_tensor& w,
                    const mxfp4_tensor* up, int act, void* y, int y_dtype, int64_t ldy, const mxfp4_tensor* qy,
                    cudaStream_t s) {
  Mx4Gemm g{};
  g.x = {x.codes, x.scales};
  g.x_bf16 = x_bf16;
  g.ldx = ldx;
  g.w = {w.codes, w.scales};
  if (up != nullptr) g.up = {up->codes, up->scales};
  g.M = x.rows;
  g.N = w.rows;
  g.K = x.cols;
  g.act = act;
  g.y_dtype = qy != nullptr ? 2 : y_dtype;
  g.y = y;
  g.ldy = ldy;
  if (qy != nullptr) {
    g.q_codes = qy->codes;
    g.q_scales = qy->scales;
  }
  g.err = error_word();
  return g.err == nullptr ? cudaErrorInvalidValue : launch_mx4_gemm(g, s);
}

}  // namespace

size_t nvfp4::gated_backward_ws(int64_t M, int64_t F, bool recompute) {
  return 2 * round256(static_cast<size_t>(M) * F * 2) + (recompute ? round256(gated_saved_bytes(M, F)) : 0) + 256;
}

size_t nvfp4::mx4_linear_ws(int64_t M, int64_t K) { return carve_bytes(M, K) + 256; }
size_t nvfp4::mx4_mlp_ws(int64_t M, int64_t F, int64_t K) { return carve_bytes(M, K) + carve_bytes(M, F) + 256; }

extern "C" {

size_t mxfp4_scale_bytes(int64_t rows, int64_t cols, int32_t layout) {
  if (rows < 0 || cols < 0 || (layout != 0 && layout != 1)) return 0;
  if (layout == 0) return static_cast<size_t>(rows * (cols / 32));
  return static_cast<size_t>((rows + 127) / 128 * 128 * ((cols + 127) / 128) * 4);
}

nvfp4_status mxfp4_quantize(const uint16_t* x, int64_t M, int64_t K, int64_t ldx, mxfp4_tensor* q_or_null,
                            uint16_t* qdq_or_null, int64_t ldo, void* stream) {
  NV_CHECK(q_or_null != nullptr || qdq_or_null != nullptr, NVFP4_ERR_INVALID_ARG);
  NV_CHECK(dim_ok(M, 0) && dim_ok(K, 32) && K % 32 == 0 && ldx >= K, NVFP4_ERR_UNSUPPORTED_SHAPE);
  if (q_or_null != nullptr)
    NV_CHECK(q_or_null->rows == M && q_or_null->cols == K, NVFP4_ERR_UNSUPPORTED_SHAPE);
  if (qdq_or_null != nullptr) NV_CHECK(ldo >= K, NVFP4_ERR_UNSUPPORTED_SHAPE);
  if (M == 0) return NVFP4_OK;
  NV_CHECK(x != nullptr && (q_or_null == nullptr || filled(q_or_null)), NVFP4_ERR_INVALID_ARG);
  NV_CHECK(aligned16(x) && ldx % 8 == 0, NVFP4_ERR_MISALIGNED);
  if (q_or_null != nullptr) NV_CHECK(tensor_aligned(q_or_null), NVFP4_ERR_MISALIGNED);
  if (qdq_or_null != nullptr) NV_CHECK(aligned16(qdq_or_null) && ldo % 8 == 0, NVFP4_ERR_MISALIGNED);
  NV_DEVICE();
  NV_TRY(launch_mx4_quant(x, M, K, ldx, q_or_null ? q_or_null->codes : nullptr,
                          q_or_null ? q_or_null->scales : nullptr, q_or_null ? q_or_null->scale_layout : 0,
                          qdq_or_null, ldo, static_cast<cudaStream_t>(stream)));
  return NVFP4_OK;
}

nvfp4_status mxfp4_dequantize(const mxfp4_tensor* q, void* y, int32_t y_dtype, int64_t ldy, void* stream) {
  NV_CHECK(q != nullptr && (y_dtype == 0 || y_dtype == 1), NVFP4_ERR_INVALID_ARG);
  NV_CHECK(shape_ok(q) && ldy >= q->cols, NVFP4_ERR_UNSUPPORTED_SHAPE);
  if (q->rows == 0) return NVFP4_OK;
  NV_CHECK(filled(q) && y != nullptr, NVFP4_ERR_INVALID_ARG);
  NV_CHECK(tensor_aligned(q) && aligned16(y) && ldy % (y_dtype == 0 ? 4 : 8) == 0, NVFP4_ERR_MISALIGNED);
  NV_DEVICE();
  NV_TRY(launch_mx4_dequant(q->codes, q->scales, q->scale_layout, q->rows, q->cols, y, y_dtype, ldy,
                            static_cast<cudaStream_t>(stream)));
  return NVFP4_OK;
}

nvfp4_status mxfp4_gemm_quantized(const mxfp4_tensor* qa, const mxfp4_tensor* qb, void* y, int32_t y_dtype,
                                  int64_t ldy, void* stream) {
  NV_CHECK(qa != nullptr && qb != nullptr && (y_dtype == 0 || y_dtype == 1), NVFP4_ERR_INVALID_ARG);
  NV_CHECK(shape_ok(qa), NVFP4_ERR_UNSUPPORTED_SHAPE);
  const nvfp4_status b = operand(qb, qa->cols);
  if (b != NVFP4_OK) return b;
  NV_CHECK(ldy >= qb->rows, NVFP4_ERR_UNSUPPORTED_SHAPE);
  if (qa->rows == 0) return NVFP4_OK;
  const nvfp4_status a = operand(qa, qa->cols);
  if (a != NVFP4_OK) return a;
  NV_CHECK(y != nullptr, NVFP4_ERR_INVALID_ARG);
  NV_CHECK(out_aligned(y, y_dtype), NVFP4_ERR_MISALIGNED);
  NV_DEVICE();
  NV_TRY(product(*qa, nullptr, 0, *qb, nullptr, 0, y, y_dtype, ldy, nullptr, static_cast<cudaStream_t>(stream)));
  return NVFP4_OK;
}

nvfp4_status mxfp4_gated_gemm(const mxfp4_tensor* qx, const mxfp4_tensor* q_gate, const mxfp4_tensor* q_up,
                              int32_t act, void* y_or_null, int32_t y_dtype, int64_t ldy, mxfp4_tensor* qy_or_null,
                              void* stream) {
  NV_CHECK(qx != nullptr && q_gate != nullptr && q_up != nullptr, NVFP4_ERR_INVALID_ARG);
  NV_CHECK(act == NVFP4_ACT_SILU || act == NVFP4_ACT_GELU_TANH, NVFP4_ERR_INVALID_ARG);
  NV_CHECK(qy_or_null != nullptr ? y_or_null == nullptr : (y_dtype == 0 || y_dtype == 1), NVFP4_ERR_INVALID_ARG);
  NV_CHECK(shape_ok(qx), NVFP4_ERR_UNSUPPORTED_SHAPE);
  const int64_t M = qx->rows, K = qx->cols, F = q_gate->rows;
  nvfp4_status st = operand(q_gate, K);
  if (st == NVFP4_OK) st = operand(q_up, K);
  if (st != NVFP4_OK) return st;
  NV_CHECK(q_up->rows == F, NVFP4_ERR_UNSUPPORTED_SHAPE);
  if (qy_or_null != nullptr)
    NV_CHECK(qy_or_null->rows == M && qy_or_null->cols == F && F % 32 == 0, NVFP4_ERR_UNSUPPORTED_SHAPE);
  else
    NV_CHECK(ldy >= F, NVFP4_ERR_UNSUPPORTED_SHAPE);
  if (M == 0) return NVFP4_OK;
  st = operand(qx, K);
  if (st == NVFP4_OK && qy_or_null != nullptr) st = operand(qy_or_null, F);
  if (st != NVFP4_OK) return st;
  if (qy_or_null == nullptr) {
    NV_CHECK(y_or_null != nullptr, NVFP4_ERR_INVALID_ARG);
    NV_CHECK(out_aligned(y_or_null, y_dtype), NVFP4_ERR_MISALIGNED);
  }
  NV_DEVICE();
  NV_TRY(product(*qx, nullptr, 0, *q_gate, q_up, act, y_or_null, y_dtype, ldy, qy_or_null,
                 static_cast<cudaStream_t>(stream)));
  return NVFP4_OK;
}

nvfp4_status mxfp4_linear(const uint16_t* x, int64_t M, int64_t K, int64_t ldx, const mxfp4_tensor* qw, void* y,
                          int32_t y_dtype, int64_t ldy, void* ws, size_t ws_bytes, void* stream) {
  NV_CHECK(qw != nullptr && (y_dtype == 0 || y_dtype == 1), NVFP4_ERR_INVALID_ARG);
  NV_CHECK(dim_ok(M, 0) && dim_ok(K, 32) && K % 32 == 0 && ldx >= K, NVFP4_ERR_UNSUPPORTED_SHAPE);
  const nvfp4_status b = operand(qw, K);
  if (b != NVFP4_OK) return b;
  NV_CHECK(ldy >= qw->rows, NVFP4_ERR_UNSUPPORTED_SHAPE);
  if (M == 0) return NVFP4_OK;
  NV_CHECK(x != nullptr && y != nullptr, NVFP4_ERR_INVALID_ARG);
  NV_CHECK(aligned16(x) && ldx % 8 == 0 && out_aligned(y, y_dtype) && aligned16(ws), NVFP4_ERR_MISALIGNED);
  NV_CHECK(ws != nullptr && ws_bytes >= carve_bytes(M, K), NVFP4_ERR_WORKSPACE);
  NV_DEVICE();
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint8_t* at = static_cast<uint8_t*>(ws);
  const mxfp4_tensor qx = carve(at, M, K);
  // (a product that quantizes X itself reads it while Y is being written)
  const bool fused = mx4_takes_bf16(M) && !overlap(x, ((M - 1) * ldx + K) * 2, y,
                                                   ((M - 1) * ldy + qw->rows) * (y_dtype == 0 ? 4 : 2));
  if (!fused) NV_TRY(launch_mx4_quant(x, M, K, ldx, qx.codes, qx.scales, 1, nullptr, 0, s));
  NV_TRY(product(qx, fused ? x : nullptr, ldx, *qw, nullptr, 0, y, y_dtype, ldy, nullptr, s));
  return NVFP4_OK;
}

nvfp4_status mxfp4_gated_mlp(const uint16_t* x, int64_t M, int64_t K, int64_t ldx, const mxfp4_tensor* q_gate,
                             const mxfp4_tensor* q_up, const mxfp4_tensor* q_down, int32_t act, void* y,
                             int32_t y_dtype, int64_t ldy, void* ws, size_t ws_bytes, void* stream) {
  NV_CHECK(q_gate != nullptr && q_up != nullptr && q_down != nullptr, NVFP4_ERR_INVALID_ARG);
  NV_CHECK(act == NVFP4_ACT_SILU || act == NVFP4_ACT_GELU_TANH, NVFP4_ERR_INVALID_ARG);
  NV_CHECK(y_dtype == 0 || y_dtype == 1, NVFP4_ERR_INVALID_ARG);
  NV_CHECK(dim_ok(M, 0) && dim_ok(K, 32) && K % 32 == 0 && ldx >= K, NVFP4_ERR_UNSUPPORTED_SHAPE);
  const int64_t F = q_gate->rows;
  nvfp4_status st = operand(q_gate, K);
  if (st == NVFP4_OK) st = operand(q_up, K);
  if (st != NVFP4_OK) return st;
  NV_CHECK(q_up->rows == F && F % 32 == 0, NVFP4_ERR_UNSUPPORTED_SHAPE);
  st = operand(q_down, F);
  if (st != NVFP4_OK) return st;
  NV_CHECK(ldy >= q_down->rows, NVFP4_ERR_UNSUPPORTED_SHAPE);
  if (M == 0) return NVFP4_OK;
  NV_CHECK(x != nullptr && y != nullptr, NVFP4_ERR_INVALID_ARG);
  NV_CHECK(aligned16(x) && ldx % 8 == 0 && out_aligned(y, y_dtype) && aligned16(ws), NVFP4_ERR_MISALIGNED);
  NV_CHECK(ws != nullptr && ws_bytes >= carve_bytes(M, K) + carve_bytes(M, F), NVFP4_ERR_WORKSPACE);
  NV_DEVICE();
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint8_t* at = static_cast<uint8_t*>(ws);
  const mxfp4_tensor qx = carve(at, M, K), qh = carve(at, M, F);
  NV_TRY(launch_mx4_quant(x, M, K, ldx, qx.codes, qx.scales, 1, nullptr, 0, s));
  NV_TRY(product(qx, nullptr, 0, *q_gate, q_up, act, nullptr, 0, 0, &qh, s));
  NV_TRY(product(qh, nullptr, 0, *q_down, nullptr, 0, y, y_dtype, ldy, nullptr, s));
  return NVFP4_OK;
}

// Longest reduction of a gated bf16 product, in K steps of 64: a CTA pair runs
// it serially at 0.4 us a step, 0.6 at the lowest clock seen under load (1.3
// GHz), and its epilogue waits for all of it in one wait of at most a second.
constexpr int64_t kMaxGatedSteps = int64_t(1) << 20;
static bool gated_reduction_ok(int64_t n, int segments) { return segments * ((n + 63) / 64) <= kMaxGatedSteps; }

// The checks both directions share; the matrices' addresses only when there
// are rows to read.
static nvfp4_status gated_ok(const uint16_t* x, int64_t M, int64_t K, int64_t ldx, const uint16_t* w_gate,
                             const uint16_t* w_up, int64_t F, int64_t ldw, int32_t act) {
  NV_CHECK(act == NVFP4_ACT_SILU || act == NVFP4_ACT_GELU_TANH, NVFP4_ERR_INVALID_ARG);
  NV_CHECK(dim_ok(M, 0) && dim_ok(K, 8) && K % 8 == 0 && dim_ok(F, 8) && F % 8 == 0 && ldx >= K && ldw >= K &&
               gated_reduction_ok(K, 1) && 2 * F <= kMaxDim,
           NVFP4_ERR_UNSUPPORTED_SHAPE);
  if (M == 0) return NVFP4_OK;
  NV_CHECK(x != nullptr && w_gate != nullptr && w_up != nullptr, NVFP4_ERR_INVALID_ARG);
  NV_CHECK(aligned16(x) && aligned16(w_gate) && aligned16(w_up) && ldx % 8 == 0 && ldw % 8 == 0,
           NVFP4_ERR_MISALIGNED);
  return NVFP4_OK;
}

size_t gated_linear_saved_bytes(int64_t M, int64_t F) { return M < 0 || F < 0 ? 0 : gated_saved_bytes(M, F); }

nvfp4_status gated_linear_forward(const uint16_t* x, int64_t M, int64_t K, int64_t ldx, const uint16_t* w_gate,
                                  const uint16_t* w_up, int64_t F, int64_t ldw, int32_t act, uint16_t* h, int64_t ldh,
                                  float* saved_or_null, void* stream) {
  const nvfp4_status st = gated_ok(x, M, K, ldx, w_gate, w_up, F, ldw, act);
  if (st != NVFP4_OK) return st;
  NV_CHECK(ldh >= F, NVFP4_ERR_UNSUPPORTED_SHAPE);
  if (M == 0) return NVFP4_OK;
  NV_CHECK(h != nullptr, NVFP4_ERR_INVALID_ARG);
  NV_CHECK(aligned16(h) && ldh % 8 == 0 && aligned16(saved_or_null), NVFP4_ERR_MISALIGNED);
  NV_DEVICE();
  GatedArgs a{x, w_gate, w_up, M, K, F, ldx, ldw, act, error_word()};
  NV_CHECK(a.err != nullptr, NVFP4_ERR_CUDA);
  NV_TRY(launch_gated_forward(a, h, ldh, saved_or_null, static_cast<cudaStream_t>(stream)));
  return NVFP4_OK;
}

nvfp4_status gated_linear_backward(const uint16_t* x, int64_t M, int64_t K, int64_t ldx, const uint16_t* w_gate,
                                   const uint16_t* w_up, int64_t F, int64_t ldw, int32_t act, const uint16_t* dh,
                                   int64_t ld_dh, const float* saved_or_null, uint16_t* dx_or_null, int64_t ld_dx,
                                   uint16_t* dw_gate_or_null, uint16_t* dw_up_or_null, void* ws, size_t ws_bytes,
                                   void* stream) {
  const nvfp4_status st = gated_ok(x, M, K, ldx, w_gate, w_up, F, ldw, act);
  if (st != NVFP4_OK) return st;
  NV_CHECK(ld_dh >= F && (dx_or_null == nullptr || ld_dx >= K), NVFP4_ERR_UNSUPPORTED_SHAPE);
  // dX reduces over F twice, dW over the tokens
  NV_CHECK((dx_or_null == nullptr || gated_reduction_ok(F, 2)) &&
               ((dw_gate_or_null == nullptr && dw_up_or_null == nullptr) || gated_reduction_ok(M, 1)),
           NVFP4_ERR_UNSUPPORTED_SHAPE);
  NV_CHECK(aligned16(dx_or_null) && aligned16(dw_gate_or_null) && aligned16(dw_up_or_null) &&
               (dx_or_null == nullptr || ld_dx % 8 == 0) && ld_dh % 8 == 0,
           NVFP4_ERR_MISALIGNED);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (M == 0) {
    // no tokens: the weights' gradients are zero
    const size_t bytes = static_cast<size_t>(F) * K * 2;
    NV_DEVICE();
    if (dw_gate_or_null != nullptr) NV_TRY(cudaMemsetAsync(dw_gate_or_null, 0, bytes, s));
    if (dw_up_or_null != nullptr) NV_TRY(cudaMemsetAsync(dw_up_or_null, 0, bytes, s));
    return NVFP4_OK;
  }
  if (dx_or_null == nullptr && dw_gate_or_null == nullptr && dw_up_or_null == nullptr) return NVFP4_OK;
  NV_CHECK(dh != nullptr, NVFP4_ERR_INVALID_ARG);
  NV_CHECK(aligned16(dh) && aligned16(saved_or_null) && aligned16(ws), NVFP4_ERR_MISALIGNED);
  NV_CHECK(ws != nullptr && ws_bytes >= gated_backward_ws(M, F, saved_or_null == nullptr) - 256, NVFP4_ERR_WORKSPACE);
  NV_DEVICE();
  GatedArgs a{x, w_gate, w_up, M, K, F, ldx, ldw, act, error_word()};
  NV_CHECK(a.err != nullptr, NVFP4_ERR_CUDA);
  uint8_t* at = static_cast<uint8_t*>(ws);
  uint16_t* dg = reinterpret_cast<uint16_t*>(at);
  at += round256(static_cast<size_t>(M) * F * 2);
  uint16_t* du = reinterpret_cast<uint16_t*>(at);
  at += round256(static_cast<size_t>(M) * F * 2);
  const float* saved = saved_or_null;
  if (saved == nullptr) {
    // the projections again; H lands where dG will be written after it
    NV_TRY(launch_gated_forward(a, dg, F, reinterpret_cast<float*>(at), s));
    saved = reinterpret_cast<const float*>(at);
  }
  NV_TRY(launch_gated_slope(a, saved, dh, ld_dh, dg, du, s));
  if (dx_or_null != nullptr) NV_TRY(launch_gated_grad_x(a, dg, du, dx_or_null, ld_dx, s));
  if (dw_gate_or_null != nullptr || dw_up_or_null != nullptr)
    NV_TRY(launch_gated_grad_w(a, dg, du, dw_gate_or_null, dw_up_or_null, s));
  return NVFP4_OK;
}

}  // extern "C"
