// mx4.cu -- microscaled 4-bit floating point: quantisation and its inverse.
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

// Eight consecutive values in fp32.
__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float (&v)[8]) {
  const uint4 w = __ldcs(reinterpret_cast<const uint4 *>(p));
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = __uint_as_float(u[j] << 16);
    v[2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u);
  }
}
__device__ __forceinline__ void load8(const float *p, float (&v)[8]) {
  const float4 a = __ldcs(reinterpret_cast<const float4 *>(p)), b = __ldcs(reinterpret_cast<const float4 *>(p) + 1);
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&v)[8]) {
  uint32_t u[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
    u[j] = *reinterpret_cast<const uint32_t *>(&h);
  }
  *reinterpret_cast<uint4 *>(p) = make_uint4(u[0], u[1], u[2], u[3]);
}
__device__ __forceinline__ void store8(float *p, const float (&v)[8]) {
  *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
  *(reinterpret_cast<float4 *>(p) + 1) = make_float4(v[4], v[5], v[6], v[7]);
}

// Quantisation and its inverse move bytes and little else.  One warp takes 256
// consecutive values (8 per lane, a block per 4 lanes) of the rows r, r + 32,
// r + 64 and r + 96 of a scale tile: their scale words are 16 consecutive bytes
// of it, so scales move as 16-byte words too, and four rows' loads are in
// flight per lane.
constexpr int kQWarps = 8;
constexpr int kQCols = 256;

struct Mx4Task {
  int64_t row, col;  // first row (of the four) and this lane's first value
  int64_t sword;     // byte offset of the 16 scale bytes of this half warp
};

// Warp `w` of all: row tile, row within 32, 256-value chunk (fastest).
__device__ __forceinline__ bool mx4_task(int64_t R, int64_t ktiles, int lane, Mx4Task &t) {
  // (fewer than 2^32 warps: 2^32 * 1024 values exceed any memory)
  const uint32_t w = blockIdx.x * kQWarps + (threadIdx.x >> 5);
  const uint32_t chunks = static_cast<uint32_t>(ktiles + 1) / 2;
  const uint32_t r = w / chunks, c = w % chunks;
  if (r >= (R + kMxTileRows - 1) / kMxTileRows * 32) return false;
  t.row = static_cast<int64_t>(r / 32) * kMxTileRows + r % 32;
  t.col = c * kQCols + lane * 8;
  t.sword = ((r / 32) * ktiles + 2 * c + lane / 16) * kMxTileBytes + r % 32 * 16;
  return true;
}

template <typename T>
__global__ void __launch_bounds__(kQWarps * 32) mx4_quantize_kernel(const T *x, int64_t ldx, uint8_t *q,
                                                                    uint8_t *scales, int64_t R, int64_t K,
                                                                    int64_t ktiles) {
  griddep_wait();
  const int lane = threadIdx.x & 31;
  Mx4Task t;
  if (!mx4_task(R, ktiles, lane, t)) return;
  float v[4][8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // rows past R and blocks past K hold zeros: scale byte 0
    if (t.row + 32 * i < R && t.col < K) {
      load8(x + (t.row + 32 * i) * ldx + t.col, v[i]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = 0.0f;
    }
  }
  uint32_t words[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t amax = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) amax = max(amax, __float_as_uint(v[i][j]) & 0x7fffffffu);
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    // the biased exponent of amax less E2M1's largest exponent
    const uint32_t e = amax >> 23;
    const uint32_t s = e == 255 ? 255u : (e > 2 ? e - 2 : 0u);
    const float inv = __uint_as_float((254u - min(s, 253u)) << 23);
    uint32_t code = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 p = make_float2(v[i][2 * j] * inv, v[i][2 * j + 1] * inv);
      code |= static_cast<uint32_t>(__nv_cvt_float2_to_fp4x2(p, __NV_E2M1, cudaRoundNearest)) << (8 * j);
    }
    if (s == 255) code = 0;
    if (t.row + 32 * i < R && t.col < K)
      *reinterpret_cast<uint32_t *>(q + (t.row + 32 * i) * (K / 2) + t.col / 2) = code;
    // the four scales of 128 values as one word on each of their 16 lanes
    uint32_t w = s << (8 * ((lane >> 2) & 3));
    w |= __shfl_xor_sync(0xffffffffu, w, 4);
    w |= __shfl_xor_sync(0xffffffffu, w, 8);
    words[i] = w;
  }
  if ((lane & 15) == 0 && t.col / 128 < ktiles)
    *reinterpret_cast<uint4 *>(scales + t.sword) = make_uint4(words[0], words[1], words[2], words[3]);
}

template <typename T>
__global__ void __launch_bounds__(kQWarps * 32) mx4_dequantize_kernel(const uint8_t *q, const uint8_t *scales, T *y,
                                                                      int64_t ldy, int64_t R, int64_t K,
                                                                      int64_t ktiles) {
  griddep_wait();
  const int lane = threadIdx.x & 31;
  Mx4Task t;
  if (!mx4_task(R, ktiles, lane, t) || t.col >= K) return;
  const uint4 w4 = *reinterpret_cast<const uint4 *>(scales + t.sword);
  const uint32_t words[4] = {w4.x, w4.y, w4.z, w4.w};
  uint32_t code[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    code[i] = t.row + 32 * i < R
                  ? __ldcs(reinterpret_cast<const uint32_t *>(q + (t.row + 32 * i) * (K / 2) + t.col / 2))
                  : 0u;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (t.row + 32 * i >= R) break;
    const float s = mx_scale((words[i] >> (8 * ((lane >> 2) & 3))) & 255u);
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = e2m1_value((code[i] >> (4 * j)) & 15u) * s;
    store8(y + (t.row + 32 * i) * ldy + t.col, v);
  }
}

static dim3 quant_grid(int64_t R, int64_t K) {
  const int64_t warps = (R + kMxTileRows - 1) / kMxTileRows * 32 * ((K + kQCols - 1) / kQCols);
  return dim3(static_cast<unsigned>((warps + kQWarps - 1) / kQWarps));
}

bi_status launch_mx4_quantize(const void *x, bool f32, int64_t ldx, uint8_t *q, uint8_t *scales, int64_t R, int64_t K,
                              cudaStream_t s) {
  const int64_t ktiles = (K + 127) / 128;
  const dim3 block(kQWarps * 32);
  if (f32)
    return launch_chained(mx4_quantize_kernel<float>, quant_grid(R, K), block, 0, s, 1, static_cast<const float *>(x),
                          ldx, q, scales, R, K, ktiles);
  return launch_chained(mx4_quantize_kernel<__nv_bfloat16>, quant_grid(R, K), block, 0, s, 1,
                        static_cast<const __nv_bfloat16 *>(x), ldx, q, scales, R, K, ktiles);
}

bi_status launch_mx4_dequantize(const uint8_t *q, const uint8_t *scales, void *y, bool f32, int64_t ldy, int64_t R,
                                int64_t K, cudaStream_t s) {
  const int64_t ktiles = (K + 127) / 128;
  const dim3 block(kQWarps * 32);
  if (f32)
    return launch_chained(mx4_dequantize_kernel<float>, quant_grid(R, K), block, 0, s, 1, q, scales,
                          static_cast<float *>(y), ldy, R, K, ktiles);
  return launch_chained(mx4_dequantize_kernel<__nv_bfloat16>, quant_grid(R, K), block, 0, s, 1, q, scales,
                        static_cast<__nv_bfloat16 *>(y), ldy, R, K, ktiles);
}

}  // namespace bimoe
