// mx4.cu -- microscaled 4-bit floating point: quantisation, its inverse and
// the product of two quantised matrices.
//
// The format is the Open Compute Project's MXFP4: 32 consecutive values of a
// row share a power of two s (8 bits, E8M0: 2^(byte - 127), 255 = NaN), and
// each is one of E2M1's values 0, .5, 1, 1.5, 2, 3, 4, 6 with a sign, times s.
// s is the power of two below the block's largest magnitude over the one
// below E2M1's largest value: with amax = m 2^e, 1 <= m < 2, s = 2^(e - 2), at
// least 2^-127; dividing by s is exact, the rounding is to nearest (ties to
// the even code), and magnitudes above 6 s become 6 s.  A block that holds a
// NaN or an infinity gets the NaN scale and zero codes: the whole block stands
// for NaN.
#include <cuda_fp4.h>

#include "ffn_internal.cuh"

namespace bimoe {

// 2^(byte - 127) as fp32; byte 0 is the subnormal 2^-127, 255 stands for NaN.
__device__ __forceinline__ float mx_scale(uint32_t byte) {
  return __uint_as_float(byte == 0 ? 0x00400000u : byte == 255 ? 0x7fc00000u : byte << 23);
}

// Value of a 4-bit code (sign, two exponent bits, one mantissa bit).
__device__ __forceinline__ float e2m1_value(uint32_t c) {
  const uint32_t e = (c >> 1) & 3u, m = c & 1u;
  const float v = e == 0 ? 0.5f * m : __uint_as_float(((e + 126u) << 23) | (m << 22));
  return (c & 8u) ? -v : v;
}

// Byte of the scale of (row, block of 32) in the tiled scale array: tiles of
// 128 rows x 4 blocks, 512 bytes each, in row-tile major order.
__device__ __forceinline__ int64_t mx_scale_at(int64_t r, int64_t b, int64_t ktiles) {
  return ((r / kMxTileRows) * ktiles + b / kMxTileScales) * kMxTileBytes + (r % 32) * 16 + (r / 32 % 4) * 4 +
         b % kMxTileScales;
}

__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ void from_f32(float v, float &o) { o = v; }
__device__ __forceinline__ void from_f32(float v, __nv_bfloat16 &o) { o = __float2bfloat16_rn(v); }

// One thread per block of 32 values of the padded scale tiles: rows up to a
// multiple of 128 and blocks up to a multiple of 4 get scale byte 0.
template <typename T>
__global__ void __launch_bounds__(256) mx4_quantize_kernel(const T *x, int64_t ldx, uint8_t *q, uint8_t *scales,
                                                           int64_t R, int64_t K, int64_t rows_p, int64_t ktiles) {
  griddep_wait();
  const int64_t nb = ktiles * kMxTileScales;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= rows_p * nb) return;
  const int64_t r = i / nb, b = i % nb;
  uint8_t *sp = scales + mx_scale_at(r, b, ktiles);
  if (r >= R || b >= K / kMxBlock) {
    *sp = 0;
    return;
  }
  const T *src = x + r * ldx + b * kMxBlock;
  uint32_t amax = 0;
  for (int j = 0; j < kMxBlock; ++j) amax = max(amax, __float_as_uint(to_f32(src[j])) & 0x7fffffffu);
  const uint32_t e = amax >> 23;
  const uint32_t s = e == 255 ? 255u : (e > 2 ? e - 2 : 0u);
  *sp = static_cast<uint8_t>(s);
  const float inv = __uint_as_float((254u - min(s, 253u)) << 23);
  uint8_t *dst = q + r * (K / 2) + b * (kMxBlock / 2);
  for (int j = 0; j < kMxBlock; j += 2) {
    const float2 v = make_float2(to_f32(src[j]) * inv, to_f32(src[j + 1]) * inv);
    dst[j / 2] = s == 255 ? 0 : static_cast<uint8_t>(__nv_cvt_float2_to_fp4x2(v, __NV_E2M1, cudaRoundNearest));
  }
}

template <typename T>
__global__ void __launch_bounds__(256) mx4_dequantize_kernel(const uint8_t *q, const uint8_t *scales, T *y, int64_t ldy,
                                                             int64_t R, int64_t K, int64_t ktiles) {
  griddep_wait();
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= R * (K / 2)) return;
  const int64_t r = i / (K / 2), j = i % (K / 2);
  const float s = mx_scale(scales[mx_scale_at(r, j / 16, ktiles)]);
  from_f32(e2m1_value(q[i] & 15u) * s, y[r * ldy + 2 * j]);
  from_f32(e2m1_value(q[i] >> 4) * s, y[r * ldy + 2 * j + 1]);
}

// Product: 64 tokens x 64 features per CTA, 4 x 4 per thread, one chain of
// fused multiply-adds over increasing k.  GATED: features pair up with the
// ones 16 rows further (16 gate rows, their 16 up rows, ...).
template <bool GATED>
__global__ void __launch_bounds__(256) mx4_tile_kernel(const uint8_t *xq, const uint8_t *xs, const uint8_t *wq,
                                                       const uint8_t *ws, const __nv_bfloat16 *addend, int64_t ld_add,
                                                       __nv_bfloat16 *y, int64_t ldy, int64_t M, int64_t N, int64_t K,
                                                       int64_t ktiles) {
  __shared__ float as[32][65], bs[32][65];
  __shared__ float tile[GATED ? 64 : 1][65];
  griddep_wait();
  const int64_t m0 = static_cast<int64_t>(blockIdx.x) * 64, n0 = static_cast<int64_t>(blockIdx.y) * 64;
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
  float acc[4][4] = {};
  for (int64_t k0 = 0; k0 < K; k0 += 32) {
    for (int i = threadIdx.x; i < 64 * 16; i += 256) {
      const int r = i / 16, j = i % 16;
      uint32_t ca = 0, cb = 0;
      float sa = 0.0f, sb = 0.0f;
      if (m0 + r < M) {
        ca = xq[(m0 + r) * (K / 2) + k0 / 2 + j];
        sa = mx_scale(xs[mx_scale_at(m0 + r, k0 / 32, ktiles)]);
      }
      if (n0 + r < N) {
        cb = wq[(n0 + r) * (K / 2) + k0 / 2 + j];
        sb = mx_scale(ws[mx_scale_at(n0 + r, k0 / 32, ktiles)]);
      }
      as[2 * j][r] = e2m1_value(ca & 15u) * sa;
      as[2 * j + 1][r] = e2m1_value(ca >> 4) * sa;
      bs[2 * j][r] = e2m1_value(cb & 15u) * sb;
      bs[2 * j + 1][r] = e2m1_value(cb >> 4) * sb;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 32; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(as[k][ty * 4 + i], bs[k][tx * 4 + j], acc[i][j]);
    __syncthreads();
  }
  if (GATED) {
    for (int i = 0; i < 4; ++i)
      for (int j = 0; j < 4; ++j) tile[ty * 4 + i][tx * 4 + j] = acc[i][j];
    __syncthreads();
    for (int i = threadIdx.x; i < 64 * 32; i += 256) {
      const int r = i / 32, f = i % 32, c = f / 16 * 32 + f % 16;
      if (m0 + r >= M || n0 + c >= N) continue;
      const float g = tile[r][c], u = tile[r][c + 16];
      y[(m0 + r) * ldy + n0 / 2 + f] = __float2bfloat16_rn(g / (1.0f + __expf(-g)) * u);
    }
  } else {
    for (int i = 0; i < 4; ++i)
      for (int j = 0; j < 4; ++j) {
        const int64_t m = m0 + ty * 4 + i, n = n0 + tx * 4 + j;
        if (m >= M || n >= N) continue;
        const float a = addend ? __bfloat162float(addend[m * ld_add + n]) : 0.0f;
        y[m * ldy + n] = __float2bfloat16_rn(acc[i][j] + a);
      }
  }
}

static unsigned blocks_of(int64_t n) { return static_cast<unsigned>((n + 255) / 256); }

bi_status launch_mx4_quantize(const void *x, bool f32, int64_t ldx, uint8_t *q, uint8_t *scales, int64_t R, int64_t K,
                              cudaStream_t s) {
  const int64_t rows_p = (R + kMxTileRows - 1) / kMxTileRows * kMxTileRows, ktiles = (K + 127) / 128;
  const dim3 grid(blocks_of(rows_p * ktiles * kMxTileScales));
  if (f32)
    return launch_chained(mx4_quantize_kernel<float>, grid, dim3(256), 0, s, 1, static_cast<const float *>(x), ldx, q,
                          scales, R, K, rows_p, ktiles);
  return launch_chained(mx4_quantize_kernel<__nv_bfloat16>, grid, dim3(256), 0, s, 1,
                        static_cast<const __nv_bfloat16 *>(x), ldx, q, scales, R, K, rows_p, ktiles);
}

bi_status launch_mx4_dequantize(const uint8_t *q, const uint8_t *scales, void *y, bool f32, int64_t ldy, int64_t R,
                                int64_t K, cudaStream_t s) {
  const int64_t ktiles = (K + 127) / 128;
  const dim3 grid(blocks_of(R * (K / 2)));
  if (f32)
    return launch_chained(mx4_dequantize_kernel<float>, grid, dim3(256), 0, s, 1, q, scales, static_cast<float *>(y),
                          ldy, R, K, ktiles);
  return launch_chained(mx4_dequantize_kernel<__nv_bfloat16>, grid, dim3(256), 0, s, 1, q, scales,
                        static_cast<__nv_bfloat16 *>(y), ldy, R, K, ktiles);
}

bi_status launch_mx4_gemm(const uint8_t *xq, const uint8_t *xs, const uint8_t *wq, const uint8_t *ws, Mat addend,
                          __nv_bfloat16 *y, int64_t ldy, bool gated, int64_t M, int64_t N, int64_t K, cudaStream_t s) {
  const int64_t ktiles = (K + 127) / 128;
  const dim3 grid(static_cast<unsigned>((M + 63) / 64), static_cast<unsigned>((N + 63) / 64));
  return launch_chained(gated ? mx4_tile_kernel<true> : mx4_tile_kernel<false>, grid, dim3(256), 0, s, 1, xq, xs, wq,
                        ws, addend.p, addend.ld, y, ldy, M, N, K, ktiles);
}

}  // namespace bimoe
