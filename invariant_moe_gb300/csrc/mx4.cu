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

#include <mutex>

#include "ffn_internal.cuh"

namespace bimoe {

// 2^(byte - 127) as fp32; byte 0 is the subnormal 2^-127, 255 stands for NaN.
__device__ __forceinline__ float mx_scale(uint32_t byte) {
  return __uint_as_float(byte == 0 ? 0x00400000u : byte == 255 ? 0x7fc00000u : byte << 23);
}

__device__ __forceinline__ float silu_mul(float g, float u) {
  return __fmul_rn(__fdividef(g, __fadd_rn(1.0f, __expf(-g))), u);
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

// ---------------------------------------------------------------- product --
//
// y = X W^T on the block-scaled tensor-core path: tcgen05.mma kind::mxf4 takes
// both operands as 4-bit codes and applies the scales itself, 64 k per MMA.
//   * Weight rows are the MMA's 128 rows, tokens its up to 192 columns; a stage
//     is 256 k: 16 KB of weight codes, up to 24 KB of token codes by TMA
//     (128-byte swizzle, as 128-byte rows), and the scale tiles by untiled
//     copies, which tcgen05.cp spreads into tensor memory before the MMAs that
//     use them.
//   * One chain of MMAs over increasing k per output, whatever the tile: a
//     token's row has the same bits in every batch.
//   * Two accumulators of 192 columns and the scales fill tensor memory's 512
//     columns; eight epilogue warps take the tile to registers and free it.
//   * Few tokens: the tile takes only 64 or 32 of the 128 rows (at their places
//     in the scale tile), so that more CTAs stream the weights.
constexpr int kXThreads = 320;       // TMA, MMA, 8 epilogue warps
constexpr int kXRows = 128;          // MMA rows
constexpr int kXMaxN = 192;          // largest token tile
constexpr int kXStageK = 256;        // values of k per stage
constexpr int kXABytes = kXRows * kXStageK / 2;
constexpr int kXMaxStages = 16;
constexpr int kXSfA = 2 * kXMaxN;    // tensor-memory columns: accumulators, A's scales, B's scales
constexpr int kXSfB = kXSfA + 8;
constexpr int kXMaxRowTiles = 2;     // scale tiles that a token tile (192 from a multiple of 64) touches

struct Mx4Gemm {
  const uint8_t *xs, *ws;
  int M, N;             // tokens, weight rows
  int nkb;              // stages (256 k) of the reduction
  int n64;              // K / 64 rounded up: MMAs of the reduction
  int ktiles;           // scale tiles per row tile
  int w_row_tiles, x_row_tiles;
  int rows;             // weight rows per tile: 128, 64 or 32
  int n;                // tokens per tile (the MMA's N)
  int m_tiles, n_tiles;
  int stages, stage_bytes;
  __nv_bfloat16 *y;
  int64_t ldy;
  const __nv_bfloat16 *addend;
  int64_t ld_add;
  int *err;
};

template <bool GATED>
__global__ void __launch_bounds__(kXThreads, 1)
    mx4_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                    const __grid_constant__ Mx4Gemm prm) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *aux = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint64_t *full = reinterpret_cast<uint64_t *>(aux);
  uint64_t *empty = full + kXMaxStages;
  uint64_t *tfull = empty + kXMaxStages;  // [2]
  uint64_t *tempty = tfull + 2;           // [2]
  uint64_t *drain = tempty + 2;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  uint8_t *tiles = aux + 1024;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int total = prm.m_tiles * prm.n_tiles;
  const int unit0 = static_cast<int>(blockIdx.x), nunits = static_cast<int>(gridDim.x);
  const int b_off = kXABytes, sfa_off = b_off + (prm.n * 128 + 1023) / 1024 * 1024, sfb_off = sfa_off + 1024;

  if (threadIdx.x == 0) {
    for (int s = 0; s < prm.stages; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(smem_u32(&tfull[a]), 1);
      mbar_init(smem_u32(&tempty[a]), 8);
    }
    mbar_init(smem_u32(drain), 1);
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
  }
  if (warp == 2) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  griddep_wait();

  auto row_of = [&](int tile) { return tile / prm.n_tiles * prm.rows; };
  auto col_of = [&](int tile) { return tile % prm.n_tiles * prm.n; };
  // scale tiles of the tokens col .. col + n - 1 that exist
  auto row_tiles = [&](int col) { return min(prm.x_row_tiles, (col + prm.n + 127) / 128) - col / 128; };

  // the TMA and the MMA thread are alone in their warps: branches and barrier
  // waits of a lane that others wait for are several times slower
  if (warp == 0) {
    // ---------------------------------------------------- TMA producer --
    if (elect_one()) {
      int stage = 0;
      uint32_t phase = 0, issued_mask = 0, issued_parity = 0;
      bool ok = true;
      for (int tile = unit0; tile < total && ok; tile += nunits) {
        const int row = row_of(tile), col = col_of(tile);
        const int rt = row_tiles(col);
        const uint8_t *sa = prm.ws + static_cast<int64_t>(row / 128) * prm.ktiles * kMxTileBytes;
        const uint8_t *sb = prm.xs + static_cast<int64_t>(col / 128) * prm.ktiles * kMxTileBytes;
        for (int kb = 0; kb < prm.nkb; ++kb) {
          if (!mbar_wait(smem_u32(&empty[stage]), phase ^ 1u, abort_flag, prm.err)) {
            ok = false;
            break;
          }
          const uint32_t st = smem_u32(tiles + stage * prm.stage_bytes), fb = smem_u32(&full[stage]);
          const uint32_t sf = static_cast<uint32_t>(min(2, prm.ktiles - 2 * kb)) * kMxTileBytes;
          mbar_arrive_expect_tx(fb, static_cast<uint32_t>((prm.rows + prm.n) * 128) + (1 + rt) * sf);
          // the rows at their places in the 128-row scale tile
          tma_load_2d(st + (row % 128) * 128, &tmA, fb, kb * 128, row);
          tma_load_2d(st + b_off, &tmB, fb, kb * 128, col);
          bulk_load(st + sfa_off, sa + kb * 2 * kMxTileBytes, sf, fb);
          for (int t = 0; t < rt; ++t)
            bulk_load(st + sfb_off + t * 1024, sb + (static_cast<int64_t>(t) * prm.ktiles + kb * 2) * kMxTileBytes, sf,
                      fb);
          issued_mask |= 1u << stage;
          issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
          if (++stage == prm.stages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (*abort_flag) {  // every copy this CTA started lands before it exits
        for (int s = 0; s < prm.stages; ++s)
          if ((issued_mask >> s) & 1u) mbar_wait(smem_u32(&full[s]), (issued_parity >> s) & 1u, nullptr, prm.err);
      }
    } else {
      return;
    }
  } else if (warp == 1) {
    // ------------------------------------------------------ MMA issuer --
    if (elect_one()) {
      const uint32_t idesc[2] = {idesc_mxf4(kXRows, prm.n, 0), idesc_mxf4(kXRows, prm.n, 1)};
      int stage = 0, buf = 0;
      uint32_t phase = 0, buf_phase = 0;
      bool ok = true, issued = false;
      for (int tile = unit0; tile < total && ok && !*abort_flag; tile += nunits) {
        if (!mbar_wait(smem_u32(&tempty[buf]), buf_phase ^ 1u, abort_flag, prm.err)) break;
        tc_fence_after();
        const int col = col_of(tile);
        const int rt = row_tiles(col);
        const uint32_t d = tmem_base + static_cast<uint32_t>(buf * kXMaxN);
        const uint32_t sfa = tmem_base + kXSfA;
        const uint32_t sfb = tmem_base + kXSfB;
        const uint32_t sfb_at = static_cast<uint32_t>(col % 128 / 32);  // the tile's first tokens' column
        for (int kb = 0; kb < prm.nkb; ++kb) {
          if (!mbar_wait(smem_u32(&full[stage]), phase, abort_flag, prm.err)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t st = smem_u32(tiles + stage * prm.stage_bytes);
          const int chunks = min(2, prm.ktiles - 2 * kb), mmas = min(4, prm.n64 - 4 * kb);
          for (int c = 0; c < chunks; ++c) {
            tmem_copy_scales(sfa + 4 * c, sdesc_scales(st + sfa_off + c * kMxTileBytes));
            for (int t = 0; t < rt; ++t)
              tmem_copy_scales(sfb + 4 * (c * kXMaxRowTiles + t), sdesc_scales(st + sfb_off + t * 1024 + c * kMxTileBytes));
          }
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (k < mmas)
              umma_mxf4(d, sdesc_sw128(st + k * 32), sdesc_sw128(st + b_off + k * 32), idesc[k & 1], sfa + 4 * (k / 2),
                        sfb + 4 * kXMaxRowTiles * (k / 2) + sfb_at, (kb | k) ? 1u : 0u);
          umma_commit(smem_u32(&empty[stage]));
          issued = true;
          if (++stage == prm.stages) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        umma_commit(smem_u32(&tfull[buf]));
        if (++buf == 2) {
          buf = 0;
          buf_phase ^= 1u;
        }
      }
      if (*abort_flag && issued) {
        umma_commit(smem_u32(drain));
        mbar_wait(smem_u32(drain), 0, nullptr, prm.err);
      }
    } else {
      return;
    }
  } else {
    // -------------------------------------------------------- epilogue --
    const int q = warp & 3, h = (warp - 2) >> 2;
    const int ncols = prm.n > 64 ? prm.n / 2 : (h == 0 ? prm.n : 0);  // columns of this warp
    int buf = 0;
    uint32_t buf_phase = 0;
    for (int tile = unit0; tile < total; tile += nunits) {
      // one lane polls: 256 polling threads slow the MMA thread's own waits
      int landed = 1;
      if (lane == 0) landed = mbar_wait(smem_u32(&tfull[buf]), buf_phase, abort_flag, prm.err) ? 1 : 0;
      if (!__shfl_sync(0xffffffffu, landed, 0)) break;
      tc_fence_after();
      const int row = row_of(tile), col0 = col_of(tile) + h * ncols;
      // a tile of 32 or 64 rows sits at its place among the 128
      const bool mine = q * 32 >= row % 128 && q * 32 < row % 128 + prm.rows;
      const uint32_t t = tmem_base + (static_cast<uint32_t>(q * 32) << 16) +
                         static_cast<uint32_t>(buf * kXMaxN + h * ncols);
      float acc[kXMaxN / 2];
#pragma unroll
      for (int c = 0; c < kXMaxN / 2; c += 16) {
        if (mine && c < ncols) {
          uint32_t d[16];
          tmem_ld16(t + c, d);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 16; ++j) acc[c + j] = __uint_as_float(d[j]);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_relaxed(smem_u32(&tempty[buf]));
      if (++buf == 2) {
        buf = 0;
        buf_phase ^= 1u;
      }
      if (!mine || ncols == 0) continue;
      const int limit = min(ncols, prm.M - col0);
      if (GATED) {
        // lanes 0-15 hold the gate values of 16 features, lanes 16-31 their up values
        const int f = (row / 128 * 128 + q * 32) / 2 + (lane & 15);
        const bool is_gate = lane < 16, okf = 2 * f < prm.N;
        __nv_bfloat16 *y = prm.y + static_cast<int64_t>(col0) * prm.ldy + f;
#pragma unroll
        for (int c = 0; c < kXMaxN / 2; c += 16) {
          if (c >= limit) break;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            // the gate lane finishes columns c..c+7, the up lane c+8..c+15
            const float keep = is_gate ? acc[c + j] : acc[c + 8 + j];
            const float other = __shfl_xor_sync(0xffffffffu, is_gate ? acc[c + 8 + j] : acc[c + j], 16);
            const int n = c + (is_gate ? j : 8 + j);
            const float g = is_gate ? keep : other, u = is_gate ? other : keep;
            if (okf && n < limit) y[n * prm.ldy] = __float2bfloat16_rn(silu_mul(g, u));
          }
        }
      } else {
        const int f = row / 128 * 128 + q * 32 + lane;
        if (f < prm.N) {
          __nv_bfloat16 *y = prm.y + static_cast<int64_t>(col0) * prm.ldy + f;
          const __nv_bfloat16 *a = prm.addend ? prm.addend + static_cast<int64_t>(col0) * prm.ld_add + f : nullptr;
#pragma unroll
          for (int c = 0; c < kXMaxN / 2; c += 16) {
            if (c >= limit) break;
            float add[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) add[j] = a && c + j < limit ? __bfloat162float(a[(c + j) * prm.ld_add]) : 0.0f;
#pragma unroll
            for (int j = 0; j < 16; ++j)
              if (c + j < limit) y[(c + j) * prm.ldy] = __float2bfloat16_rn(__fadd_rn(acc[c + j], add[j]));
          }
        }
        __syncwarp();
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 512);
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

bi_status launch_mx4_gemm(const uint8_t *xq, const uint8_t *xs, const uint8_t *wq, const uint8_t *ws, Mat addend,
                          __nv_bfloat16 *y, int64_t ldy, bool gated, int64_t M, int64_t N, int64_t K, cudaStream_t s) {
  constexpr int kSmem = 227 * 1024;
  static std::mutex mu;
  static ContextSetup setup;  // the shared-memory attribute is per context
  int dev = 0;
  cudaGetDevice(&dev);
  {
    std::lock_guard<std::mutex> lk(mu);
    if (setup.pending(dev)) {
      cudaError_t e = cudaFuncSetAttribute(mx4_gemm_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
      if (e == cudaSuccess)
        e = cudaFuncSetAttribute(mx4_gemm_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
      if (e != cudaSuccess) {
        cudaGetLastError();
        set_error("cudaFuncSetAttribute: %s", cudaGetErrorString(e));
        return BI_ERR_CUDA;
      }
      setup.done(dev);
    }
  }
  Mx4Gemm p{};
  p.xs = xs;
  p.ws = ws;
  p.M = static_cast<int>(M);
  p.N = static_cast<int>(N);
  p.nkb = static_cast<int>((K + kXStageK - 1) / kXStageK);
  p.n64 = static_cast<int>((K + 63) / 64);
  p.ktiles = static_cast<int>((K + 127) / 128);
  p.w_row_tiles = static_cast<int>((N + 127) / 128);
  p.x_row_tiles = static_cast<int>((M + 127) / 128);
  // tokens in tiles of up to 192; fewer in one tile, rounded up to 16
  p.n = M <= kXMaxN ? static_cast<int>((M + 15) / 16 * 16) : kXMaxN;
  if (M <= kXMaxN && p.n > 64) p.n = (p.n + 31) / 32 * 32;  // two halves of whole 16-column chunks
  p.n_tiles = static_cast<int>((M + p.n - 1) / p.n);
  // rows per tile: the most that still gives every SM a tile
  p.rows = kXRows;
  while (p.rows > 32 && (N + p.rows - 1) / p.rows * p.n_tiles < num_sms()) p.rows /= 2;
  p.m_tiles = static_cast<int>((N + p.rows - 1) / p.rows);
  const int sfb_tiles = M <= 128 ? 1 : kXMaxRowTiles;
  p.stage_bytes = kXABytes + (p.n * 128 + 1023) / 1024 * 1024 + 1024 + sfb_tiles * 1024;
  p.stages = std::min(kXMaxStages, (kSmem - 2048) / p.stage_bytes);
  p.y = y;
  p.ldy = ldy;
  p.addend = addend.p;
  p.ld_add = addend.ld;
  p.err = device_error_word();
  const int64_t tiles = static_cast<int64_t>(p.m_tiles) * p.n_tiles;
  if (tiles > (int64_t(1) << 30)) {
    set_error("4-bit product with %lld tiles", (long long)tiles);
    return BI_ERR_UNSUPPORTED;
  }
  CUtensorMap a, b;
  if (!make_tma_2d_u8(&a, wq, N, K / 2, p.rows) || !make_tma_2d_u8(&b, xq, M, K / 2, p.n)) return BI_ERR_CUDA;
  const int units = static_cast<int>(std::min<int64_t>(num_sms(), tiles));
  const size_t smem = 2048 + static_cast<size_t>(p.stages) * p.stage_bytes;
  return launch_chained(gated ? mx4_gemm_kernel<true> : mx4_gemm_kernel<false>, dim3(units), dim3(kXThreads), smem, s,
                        1, a, b, p);
}

}  // namespace bimoe
