// ffn_internal.cuh -- host-side interfaces of the dense gated feed-forward
// block (ffn.cu) and of the microscaled 4-bit operators (mx4.cu), shared with
// the entry points in api.cu.
#pragma once

#include "bimoe_internal.cuh"

namespace bimoe {

// 1 / (1 + exp(-g)) by the hardware's approximate exponential and reciprocal,
// with subnormals flushed: as C++ intrinsics without flushing each takes
// several instructions more, and the epilogues that need a sigmoid for every
// element were bound by them.  Each is within 2 ulp or so of its argument's
// value; the argument's own rounding, half an ulp of 1.44 |g|, makes the
// exponential off by up to |g| 2^-24 more (5e-6 at g = -80), still far below
// the bf16 rounding that follows.  For g below about -87 the result is 0, its
// limit.
__device__ __forceinline__ float sigmoid_approx(float g) {
  float e, s;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(__fmul_rn(g, -1.4426950408889634f)));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(__fadd_rn(1.0f, e)));
  return s;
}

// silu(g) * u: one fixed fp32 sequence.
__device__ __forceinline__ float silu_mul(float g, float u) {
  return __fmul_rn(__fmul_rn(g, sigmoid_approx(g)), u);
}

// A row-major bf16 matrix [rows, cols] with row stride ld (elements).
struct Mat {
  const __nv_bfloat16 *p;
  int64_t ld;
};

enum GradMode { kGradBf16 = 0, kGradF32 = 1, kGradF32Accumulate = 2 };

// act [M, I] = silu(x Wg^T) * (x Wu^T); gu [M, 2I] fp32 (may be null) keeps the two projections.
bi_status launch_ffn_gate_up(Mat x, const __nv_bfloat16 *w13, __nv_bfloat16 *act, float *gu, int64_t M, int64_t H,
                             int64_t I, cudaStream_t s);
// out [M, H] = act W2^T (+ addend)
bi_status launch_ffn_down(const __nv_bfloat16 *act, const __nv_bfloat16 *w2, Mat addend, __nv_bfloat16 *out,
                          int64_t ldo, int64_t M, int64_t H, int64_t I, cudaStream_t s);
// dgu [M, 2I] = the gradient of the two projections, from dact = dout W2
bi_status launch_ffn_dact(Mat dout, const __nv_bfloat16 *w2, const float *gu, __nv_bfloat16 *dgu, int64_t M, int64_t H,
                          int64_t I, cudaStream_t s);
// dx [M, H] = dgu W13, dw13 [2I, H] = dgu^T x, dw2 [H, I] = dout^T act; what is null is not computed
struct FfnGrads {
  Mat dout, x;
  const __nv_bfloat16 *dgu, *act, *w13;
  __nv_bfloat16 *dx;
  int64_t lddx;
  void *dw13, *dw2;
  int grad_mode;
};
bi_status launch_ffn_grads(const FfnGrads &d, int64_t M, int64_t H, int64_t I, cudaStream_t s);

int set_ffn_schedule(int mode);  // bi_ffn_schedule; returns the old mode

constexpr int kMxBlock = 32;       // values that share a scale
constexpr int kMxTileRows = 128;   // a scale tile: 128 rows x 4 scales, 512 bytes
constexpr int kMxTileScales = 4;
constexpr int kMxTileBytes = 512;

bi_status launch_mx4_quantize(const void *x, bool f32, int64_t ldx, uint8_t *q, uint8_t *scales, int64_t R, int64_t K,
                              cudaStream_t s);
bi_status launch_mx4_dequantize(const uint8_t *q, const uint8_t *scales, void *y, bool f32, int64_t ldy, int64_t R,
                                int64_t K, cudaStream_t s);
bi_status launch_mx4_gemm(const uint8_t *xq, const uint8_t *xs, const uint8_t *wq, const uint8_t *ws, Mat addend,
                          __nv_bfloat16 *y, int64_t ldy, bool gated, int64_t M, int64_t N, int64_t K, cudaStream_t s);

int set_mx4_form(int mode);  // bi_mx4_form; returns the old mode

}  // namespace bimoe
