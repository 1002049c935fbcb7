// ffn.cu -- the dense gated feed-forward block (a shared expert), forward and
// backward.
//
//   forward   [g u] = x W13^T,  act = silu(g) u,  out = act W2^T (+ addend)
//   backward  dact = dout W2,  s = 1 / (1 + exp(-g)),
//             dg = dact u s (1 + g (1 - s)),  du = dact g s,
//             dx = [dg du] W13,  dW13 = [dg du]^T x,  dW2 = dout^T act
//
// One tile kernel over fp32 FMAs: 64 x 64 outputs per CTA, 4 x 4 per thread,
// operands read through their two strides, every output one chain of fused
// multiply-adds over increasing k.  The chain depends on the reduction length
// alone, so a token's row has the same bits whatever M is.
#include "ffn_internal.cuh"

namespace bimoe {

constexpr int kT = 64;   // outputs per tile side
constexpr int kTK = 16;  // reduction step

struct Strided {
  const __nv_bfloat16 *p;
  int64_t s_row, s_k;
};

enum Epi { kEpiGateUp, kEpiStore, kEpiDact, kEpiWgrad };

struct FfnParams {
  Strided a, b, b2;  // D[m, n] = sum_k a[m, k] b[n, k]; b2: the up rows (gate/up)
  int64_t M, N, K;
  void *out;
  int64_t ldo;
  const __nv_bfloat16 *addend;
  int64_t ld_add;
  float *gu;
  int mode;
};

template <Epi EPI>
__global__ void __launch_bounds__(256) ffn_tile_kernel(const FfnParams p) {
  constexpr bool kTwo = EPI == kEpiGateUp;
  __shared__ float as[kTK][kT + 1], bs[kTwo ? 2 : 1][kTK][kT + 1];
  griddep_wait();
  const int64_t m0 = static_cast<int64_t>(blockIdx.x) * kT, n0 = static_cast<int64_t>(blockIdx.y) * kT;
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
  float acc[kTwo ? 2 : 1][4][4] = {};
  for (int64_t k0 = 0; k0 < p.K; k0 += kTK) {
    for (int i = threadIdx.x; i < kT * kTK; i += 256) {
      // consecutive threads along whichever index is contiguous in memory
      const int ra = p.a.s_k == 1 ? i / kTK : i % kT, ka = p.a.s_k == 1 ? i % kTK : i / kT;
      const int rb = p.b.s_k == 1 ? i / kTK : i % kT, kb = p.b.s_k == 1 ? i % kTK : i / kT;
      const bool oka = m0 + ra < p.M && k0 + ka < p.K, okb = n0 + rb < p.N && k0 + kb < p.K;
      as[ka][ra] = oka ? __bfloat162float(p.a.p[(m0 + ra) * p.a.s_row + (k0 + ka) * p.a.s_k]) : 0.0f;
      bs[0][kb][rb] = okb ? __bfloat162float(p.b.p[(n0 + rb) * p.b.s_row + (k0 + kb) * p.b.s_k]) : 0.0f;
      if (kTwo) bs[1][kb][rb] = okb ? __bfloat162float(p.b2.p[(n0 + rb) * p.b2.s_row + (k0 + kb) * p.b2.s_k]) : 0.0f;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kTK; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          acc[0][i][j] = fmaf(as[k][ty * 4 + i], bs[0][k][tx * 4 + j], acc[0][i][j]);
          if (kTwo) acc[1][i][j] = fmaf(as[k][ty * 4 + i], bs[1][k][tx * 4 + j], acc[1][i][j]);
        }
    __syncthreads();
  }
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int64_t m = m0 + ty * 4 + i, n = n0 + tx * 4 + j;
      if (m >= p.M || n >= p.N) continue;
      const float v = acc[0][i][j];
      if (EPI == kEpiGateUp) {
        const float u = acc[kTwo ? 1 : 0][i][j];
        if (p.gu) {
          p.gu[m * 2 * p.N + n] = v;
          p.gu[m * 2 * p.N + p.N + n] = u;
        }
        static_cast<__nv_bfloat16 *>(p.out)[m * p.ldo + n] = __float2bfloat16_rn(v / (1.0f + __expf(-v)) * u);
      } else if (EPI == kEpiStore) {
        const float a = p.addend ? __bfloat162float(p.addend[m * p.ld_add + n]) : 0.0f;
        static_cast<__nv_bfloat16 *>(p.out)[m * p.ldo + n] = __float2bfloat16_rn(v + a);
      } else if (EPI == kEpiDact) {
        const float g = p.gu[m * 2 * p.N + n], u = p.gu[m * 2 * p.N + p.N + n];
        const float s = 1.0f / (1.0f + __expf(-g));
        __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(p.out) + m * p.ldo + n;
        o[0] = __float2bfloat16_rn(v * u * s * (1.0f + g * (1.0f - s)));
        o[p.N] = __float2bfloat16_rn(v * g * s);
      } else if (p.mode == kGradBf16) {
        static_cast<__nv_bfloat16 *>(p.out)[m * p.ldo + n] = __float2bfloat16_rn(v);
      } else {
        float *o = static_cast<float *>(p.out) + m * p.ldo + n;
        *o = p.mode == kGradF32Accumulate ? *o + v : v;
      }
    }
}

template <Epi EPI>
static bi_status launch_tile(const FfnParams &p, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>((p.M + kT - 1) / kT), static_cast<unsigned>((p.N + kT - 1) / kT));
  return launch_chained(ffn_tile_kernel<EPI>, grid, dim3(256), 0, s, 1, p);
}

bi_status launch_ffn_gate_up(Mat x, const __nv_bfloat16 *w13, __nv_bfloat16 *act, float *gu, int64_t M, int64_t H,
                             int64_t I, cudaStream_t s) {
  FfnParams p{{x.p, x.ld, 1}, {w13, H, 1}, {w13 + I * H, H, 1}, M, I, H, act, I, nullptr, 0, gu, 0};
  return launch_tile<kEpiGateUp>(p, s);
}

bi_status launch_ffn_down(const __nv_bfloat16 *act, const __nv_bfloat16 *w2, Mat addend, __nv_bfloat16 *out,
                          int64_t ldo, int64_t M, int64_t H, int64_t I, cudaStream_t s) {
  FfnParams p{{act, I, 1}, {w2, I, 1}, {}, M, H, I, out, ldo, addend.p, addend.ld, nullptr, 0};
  return launch_tile<kEpiStore>(p, s);
}

bi_status launch_ffn_dact(Mat dout, const __nv_bfloat16 *w2, const float *gu, __nv_bfloat16 *dgu, int64_t M, int64_t H,
                          int64_t I, cudaStream_t s) {
  FfnParams p{{dout.p, dout.ld, 1}, {w2, 1, I}, {}, M, I, H, dgu, 2 * I, nullptr, 0, const_cast<float *>(gu), 0};
  return launch_tile<kEpiDact>(p, s);
}

bi_status launch_ffn_dx(const __nv_bfloat16 *dgu, const __nv_bfloat16 *w13, __nv_bfloat16 *dx, int64_t lddx, int64_t M,
                        int64_t H, int64_t I, cudaStream_t s) {
  FfnParams p{{dgu, 2 * I, 1}, {w13, 1, H}, {}, M, H, 2 * I, dx, lddx, nullptr, 0, nullptr, 0};
  return launch_tile<kEpiStore>(p, s);
}

bi_status launch_ffn_wgrad(Mat a, Mat b, void *dw, int grad_mode, int64_t M, int64_t rows, int64_t cols,
                           cudaStream_t s) {
  FfnParams p{{a.p, 1, a.ld}, {b.p, 1, b.ld}, {}, rows, cols, M, dw, cols, nullptr, 0, nullptr, grad_mode};
  return launch_tile<kEpiWgrad>(p, s);
}

}  // namespace bimoe
