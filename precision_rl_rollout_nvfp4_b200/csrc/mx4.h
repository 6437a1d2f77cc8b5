// Host-side launchers of the MXFP4 and gated feed-forward kernels.  Internal
// to the library: the C ABI (api_mx4.cu) validates arguments and calls these.
#pragma once

#include "kernels.h"

namespace nvfp4 {

unsigned bounds_flags_mx4(unsigned* line);
unsigned bounds_flags_mx4_gemm(unsigned* line);
unsigned bounds_flags_mx4_pair(unsigned* line);
unsigned bounds_flags_gated(unsigned* line);

// Workspace bytes of mxfp4_linear and mxfp4_gated_mlp.
size_t mx4_linear_ws(int64_t M, int64_t K);
size_t mx4_mlp_ws(int64_t M, int64_t F, int64_t K);

// The device error word on the current device, null if it cannot be had.
unsigned* error_word();

// MXFP4 of bf16 x [rows, K] (K % 32 == 0): codes [rows, K/2], UE8M0 scales
// per 32 elements in `layout`, and / or the values the codes stand for as
// bf16 [rows, K] with row stride ldo (codes and qdq may each be null).
cudaError_t launch_mx4_quant(const uint16_t* x, int64_t rows, int64_t K, int64_t ldx, uint8_t* codes,
                             uint8_t* scales, int layout, uint16_t* qdq, int64_t ldo, cudaStream_t s);

// Values of an MXFP4 tensor as fp32 (y_dtype 0) or bf16 (1), row stride ldy.
cudaError_t launch_mx4_dequant(const uint8_t* codes, const uint8_t* scales, int layout, int64_t rows, int64_t K,
                               void* y, int y_dtype, int64_t ldy, cudaStream_t s);

// An MXFP4 operand: codes [rows, K/2], tiled scales.
struct Mx4Operand {
  const uint8_t* codes;
  const uint8_t* scales;
};

// Y = X W^T, or with `up` Y = act(X W^T) * (X Up^T): X [M, K], W and Up [N, K].
// y_dtype 0 fp32, 1 bf16 (row stride ldy), 2 MXFP4 (q_codes [M, N/2], tiled
// q_scales; N % 32 == 0).
struct Mx4Gemm {
  Mx4Operand x, w, up;      // up.codes null: a plain product
  const uint16_t* x_bf16;   // instead of x, for a plain product of mx4_takes_bf16 rows: quantized in the kernel
  int64_t ldx;
  int64_t M, N, K;
  int act;                  // kActSilu, kActGeluTanh
  int y_dtype;
  void* y;
  int64_t ldy;
  uint8_t* q_codes;
  uint8_t* q_scales;
  unsigned* err;
};
cudaError_t launch_mx4_gemm(const Mx4Gemm& g, cudaStream_t s);
// Whether the product of M rows quantizes bf16 rows itself.
bool mx4_takes_bf16(int64_t M);
// The CTA-pair kernel alone (chosen by launch_mx4_gemm).
cudaError_t launch_mx4_pair(const Mx4Gemm& g, cudaStream_t s);

// The trainer's gated projection in bf16: x [M, K] (row stride ldx), w_gate
// and w_up [F, K] (row stride ldw), K % 8 == F % 8 == 0.
struct GatedArgs {
  const uint16_t *x, *w_gate, *w_up;
  int64_t M, K, F, ldx, ldw;
  int act;
  unsigned* err;
};
// Bytes of the saved fp32 projections G and U.
size_t gated_saved_bytes(int64_t M, int64_t F);
// H [M, F], and G and U into `saved` unless it is null.
cudaError_t launch_gated_forward(const GatedArgs& a, uint16_t* h, int64_t ldh, float* saved, cudaStream_t s);
// dG and dU (bf16 [M, F]) from the saved projections and dH.
cudaError_t launch_gated_slope(const GatedArgs& a, const float* saved, const uint16_t* dh, int64_t ld_dh,
                               uint16_t* dg, uint16_t* du, cudaStream_t s);
// dX [M, K], and dWg / dWu [F, K] (either may be null).
cudaError_t launch_gated_grad_x(const GatedArgs& a, const uint16_t* dg, const uint16_t* du, uint16_t* dx,
                                int64_t ld_dx, cudaStream_t s);
cudaError_t launch_gated_grad_w(const GatedArgs& a, const uint16_t* dg, const uint16_t* du, uint16_t* dw_gate,
                                uint16_t* dw_up, cudaStream_t s);
// Workspace bytes of gated_linear_backward.
size_t gated_backward_ws(int64_t M, int64_t F, bool recompute);

enum { kActSilu = 0, kActGeluTanh = 1 };

}  // namespace nvfp4
