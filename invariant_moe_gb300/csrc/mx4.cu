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

// Eight 4-bit codes to bf16 pairs (element 2p in the low half of word p): the
// bf16 patterns of 0, .5, 1, 1.5, 2, 3, 4, 6 are 0000, 3f00, 3f80, 3fc0, 4000,
// 4040, 4080, 40c0, so byte permutes look their bytes up, four codes at a time.
__device__ __forceinline__ void e2m1_to_bf16x2(uint32_t code, uint32_t (&v)[4]) {
  const uint32_t sel = code & 0x77777777u;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t hi = __byte_perm(0x3f3f3f00u, 0x40404040u, sel >> (16 * h));
    const uint32_t lo = __byte_perm(0xc0800000u, 0xc0804000u, sel >> (16 * h));
    v[2 * h] = __byte_perm(lo, hi, 0x5140);
    v[2 * h + 1] = __byte_perm(lo, hi, 0x7362);
  }
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    // byte p of the codes holds both signs, bits 3 and 7: to bits 15 and 31
    const uint32_t t = __byte_perm(code, 0, p << 12 | 4 << 8 | p << 4 | 4);
    v[p] |= (t << 4 & 0x8000u) | (t & 0x80000000u);
  }
}

// Eight consecutive values as they lie in memory; their largest magnitude's
// biased exponent (shared by the 4 lanes of a block) and their fp32 values.
struct RawBf16 {
  uint4 w;
  __device__ __forceinline__ void load(const __nv_bfloat16 *p) { w = __ldcs(reinterpret_cast<const uint4 *>(p)); }
  __device__ __forceinline__ void zero() { w = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ uint32_t exponent() const {
    constexpr uint32_t kAbs = 0x7fff7fffu;  // two magnitudes, ordered as integers
    uint32_t m = __vmaxu2(__vmaxu2(w.x & kAbs, w.y & kAbs), __vmaxu2(w.z & kAbs, w.w & kAbs));
    m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 2));
    return max(m & 0xffffu, m >> 16) >> 7;
  }
  __device__ __forceinline__ void values(float (&v)[8]) const {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = __uint_as_float(u[j] << 16);
      v[2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u);
    }
  }
};
struct RawF32 {
  float4 a, b;
  __device__ __forceinline__ void load(const float *p) {
    a = __ldcs(reinterpret_cast<const float4 *>(p));
    b = __ldcs(reinterpret_cast<const float4 *>(p) + 1);
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.0f, 0.0f, 0.0f, 0.0f); }
  __device__ __forceinline__ uint32_t exponent() const {
    float v[8];
    values(v);
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(v[j]) & 0x7fffffffu);
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    return m >> 23;
  }
  __device__ __forceinline__ void values(float (&v)[8]) const {
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
};

// Eight code values (bf16 pairs) times the scale 2^(byte - 127), to memory.  Both
// products are exact: a code has two significant bits.
__device__ __forceinline__ void store_scaled(__nv_bfloat16 *p, const uint32_t (&v)[4], uint32_t byte) {
  const uint32_t s = byte == 0 ? 0x00400040u : byte == 255 ? 0x7fc07fc0u : byte << 7 | byte << 23;
  uint32_t r[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const __nv_bfloat162 m = __hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&v[j]),
                                     *reinterpret_cast<const __nv_bfloat162 *>(&s));
    r[j] = *reinterpret_cast<const uint32_t *>(&m);
  }
  __stcs(reinterpret_cast<uint4 *>(p), make_uint4(r[0], r[1], r[2], r[3]));
}
__device__ __forceinline__ void store_scaled(float *p, const uint32_t (&v)[4], uint32_t byte) {
  const float s = mx_scale(byte);
  float r[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    r[2 * j] = __uint_as_float(v[j] << 16) * s;
    r[2 * j + 1] = __uint_as_float(v[j] & 0xffff0000u) * s;
  }
  __stcs(reinterpret_cast<float4 *>(p), make_float4(r[0], r[1], r[2], r[3]));
  __stcs(reinterpret_cast<float4 *>(p) + 1, make_float4(r[4], r[5], r[6], r[7]));
}

// Quantisation and its inverse move bytes and little else.  One warp takes 256
// consecutive values (8 per lane, a block per 4 lanes) of the rows r, r + 32,
// r + 64 and r + 96 of a scale tile: their scale words are 16 consecutive bytes
// of it, so scales move as 16-byte words too, and four rows' loads are in
// flight per lane.  Bound by memory: 32768 x 4096 bf16 values take
// 57 us quantised (5.93 TB/s; a GB300 copies at 6.78) and 52 us dequantised
// (6.54 TB/s).  A warp per task and as many blocks as that takes: blocks that
// stay and loop were 4 to 15 % slower, five blocks a SM instead of eight 5 %.
constexpr int kQWarps = 8;
constexpr int kQCols = 256;

struct Mx4Task {
  int64_t row, col;  // first row (of the four) and this lane's first value
  int64_t sword;     // byte offset of the 16 scale bytes of this half warp
};

// This warp's task: row tile, row within 32, 256-value chunk (fastest).
__device__ __forceinline__ bool mx4_task(int64_t R, int64_t ktiles, int lane, Mx4Task &t) {
  // (fewer than 2^32 tasks: 2^32 * 1024 values exceed any memory)
  const uint32_t w = blockIdx.x * kQWarps + (threadIdx.x >> 5);
  const uint32_t chunks = static_cast<uint32_t>(ktiles + 1) / 2;
  const uint32_t r = w / chunks, c = w % chunks;
  if (r >= (R + kMxTileRows - 1) / kMxTileRows * 32) return false;
  t.row = static_cast<int64_t>(r / 32) * kMxTileRows + r % 32;
  t.col = c * kQCols + lane * 8;
  t.sword = ((r / 32) * ktiles + 2 * c + lane / 16) * kMxTileBytes + r % 32 * 16;
  return true;
}

template <typename T, typename Raw>
__global__ void __launch_bounds__(kQWarps * 32, sizeof(T) == 2 ? 8 : 4)
    mx4_quantize_kernel(const T *x, int64_t ldx, uint8_t *q, uint8_t *scales, int64_t R, int64_t K, int64_t ktiles) {
  griddep_wait();
  const int lane = threadIdx.x & 31;
  Mx4Task t;
  if (!mx4_task(R, ktiles, lane, t)) return;
  Raw raw[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // rows past R and blocks past K hold zeros: scale byte 0
    if (t.row + 32 * i < R && t.col < K) raw[i].load(x + (t.row + 32 * i) * ldx + t.col);
    else raw[i].zero();
  }
  uint32_t words[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // the biased exponent of the largest magnitude less E2M1's largest exponent
    const uint32_t e = raw[i].exponent();
    const uint32_t s = e == 255 ? 255u : (e > 2 ? e - 2 : 0u);
    const float inv = __uint_as_float((254u - min(s, 253u)) << 23);
    float v[8];
    raw[i].values(v);
    uint32_t code = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 p = make_float2(v[2 * j] * inv, v[2 * j + 1] * inv);
      code |= static_cast<uint32_t>(__nv_cvt_float2_to_fp4x2(p, __NV_E2M1, cudaRoundNearest)) << (8 * j);
    }
    if (s == 255) code = 0;
    if (t.row + 32 * i < R && t.col < K)
      *reinterpret_cast<uint32_t *>(q + (t.row + 32 * i) * (K / 2) + t.col / 2) = code;
    // the four scales of 128 values as one word on each of their 16 lanes
    uint32_t b = s << (8 * ((lane >> 2) & 3));
    b |= __shfl_xor_sync(0xffffffffu, b, 4);
    b |= __shfl_xor_sync(0xffffffffu, b, 8);
    words[i] = b;
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
  const uint4 w4 = __ldcs(reinterpret_cast<const uint4 *>(scales + t.sword));
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
    uint32_t v[4];
    e2m1_to_bf16x2(code[i], v);
    store_scaled(y + (t.row + 32 * i) * ldy + t.col, v, (words[i] >> (8 * ((lane >> 2) & 3))) & 255u);
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
    return launch_chained(mx4_quantize_kernel<float, RawF32>, quant_grid(R, K), block, 0, s, 1,
                          static_cast<const float *>(x), ldx, q, scales, R, K, ktiles);
  return launch_chained(mx4_quantize_kernel<__nv_bfloat16, RawBf16>, quant_grid(R, K), block, 0, s, 1,
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
