// tile_epilogue.cuh -- epilogue pieces shared by the tensor-core products whose
// accumulators hold features on tensor-memory lanes and tokens on columns, while
// the result is token-major.
//
// A warp reads 16 lanes x 16 columns with tcgen05.ld.16x256b.x2: thread t then
// holds features t/4 and t/4 + 8 of tokens 2(t%4), 2(t%4)+1 (and the same 8
// tokens further), two neighbouring tokens in neighbouring registers.  Packed to
// bf16 pairs these are the fragments of 8 x 8 matrices that stmatrix.trans
// writes token-major into shared memory, from where a token's features leave as
// 16-byte words: for 32 features x 16 tokens two stores a lane instead of
// sixteen 2-byte ones.
#pragma once

#include "ffn_internal.cuh"

namespace bimoe {

// A warp's staging buffer: 16 tokens x 32 features bf16, rows 80 bytes apart (a
// multiple of 16 whose 8 consecutive rows fall into different banks).
constexpr int kStagePitch = 80;
constexpr int kStageBytes = 16 * kStagePitch;

// 16 lanes x 16 columns: r[0..3] the first 8 columns, r[4..7] the others; of
// each four: (t/4, 2(t%4)), (t/4, 2(t%4)+1), (t/4+8, ..), (t/4+8, ..).
// (fp32 bits; not to be touched before tmem_ld_wait.)
__device__ __forceinline__ void tmem_ld_16x16(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
__device__ __forceinline__ void stmatrix4_trans(uint32_t addr, const uint32_t (&r)[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3])
               : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&v);
}

// Where a warp's part of a token-major bf16 matrix lies: element (token t,
// feature f) of the warp at p[t * ld + f], t < tokens, f < feats.  vec: rows
// are 16-byte aligned.
struct RowsOut {
  __nv_bfloat16 *p;
  int64_t ld;
  int tokens, feats;
  bool vec;
};

// 8 features of a 16-byte aligned row, n of them valid.
__device__ __forceinline__ uint4 load_part(const __nv_bfloat16 *p, int n) {
  if (n >= 8) return *reinterpret_cast<const uint4 *>(p);
  uint32_t w[4] = {0, 0, 0, 0};
  const uint16_t *q = reinterpret_cast<const uint16_t *>(p);
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j < n) w[j / 2] |= static_cast<uint32_t>(q[j]) << (16 * (j & 1));
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store_part(__nv_bfloat16 *p, uint4 v, int n) {
  if (n >= 8) {
    *reinterpret_cast<uint4 *>(p) = v;
    return;
  }
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint16_t *q = reinterpret_cast<uint16_t *>(p);
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j < n) q[j] = static_cast<uint16_t>(w[j / 2] >> (16 * (j & 1)));
}
__device__ __forceinline__ uint16_t lds16(uint32_t addr) {
  uint16_t v;
  asm volatile("ld.shared.b16 %0, [%1];" : "=h"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void sts16(uint32_t addr, uint16_t v) {
  asm volatile("st.shared.b16 [%0], %1;" ::"r"(addr), "h"(v) : "memory");
}

// The part of 16 tokens x 32 features that a lane of store_rows32 loads of rows
// to be added (16-byte aligned ones; others are loaded there).
__device__ __forceinline__ void load_rows32(const RowsOut &add, int t0, int lane, uint4 (&w)[2]) {
  const int f = (lane & 3) * 8, nf = add.feats - f;
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    const int t = t0 + b * 8 + (lane >> 2);
    w[b] = make_uint4(0, 0, 0, 0);
    if (add.vec && t < add.tokens && nf > 0) w[b] = load_part(add.p + t * add.ld + f, nf);
  }
}

// 16 tokens (t0..) x 32 features: v[g] holds features 16g..16g+15 as
// tmem_ld_16x16 leaves them.  `stage`: this warp's buffer.  add (may be null):
// rows added in fp32 before the rounding, same shape and place as out, `w` what
// load_rows32 loaded of them.
__device__ __forceinline__ void store_rows32(uint32_t stage, const uint32_t (&v)[2][8], int t0, const RowsOut &out,
                                             const RowsOut *add, const uint4 (&aw)[2], int lane) {
  // lane's row of the four 8 x 8 matrices of a stmatrix / ldmatrix: token lane % 8, features 8 (lane / 8) ..
  const uint32_t mat = stage + static_cast<uint32_t>((lane & 7) * kStagePitch + (lane >> 3) * 16);
  // lane's 16-byte part of the row-wise accesses: token lane / 4 (and 8 further), features 8 (lane % 4) ..
  const uint32_t rowp = stage + static_cast<uint32_t>((lane >> 2) * kStagePitch + (lane & 3) * 16);
  const int f = (lane & 3) * 8, nf = out.feats - f;
  uint32_t a[2][4];
  if (add) {
    if (add->vec) {
#pragma unroll
      for (int b = 0; b < 2; ++b)
        asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(rowp + b * 8 * kStagePitch), "r"(aw[b].x),
                     "r"(aw[b].y), "r"(aw[b].z), "r"(aw[b].w)
                     : "memory");
    } else {  // a lane per feature, a token at a time
      uint16_t w[16];
      const uint16_t *q = reinterpret_cast<const uint16_t *>(add->p) + static_cast<int64_t>(t0) * add->ld + lane;
#pragma unroll
      for (int t = 0; t < 16; ++t)
        w[t] = t0 + t < add->tokens && lane < add->feats ? q[t * add->ld] : static_cast<uint16_t>(0);
#pragma unroll
      for (int t = 0; t < 16; ++t) sts16(stage + static_cast<uint32_t>(t * kStagePitch + lane * 2), w[t]);
    }
    __syncwarp();
#pragma unroll
    for (int b = 0; b < 2; ++b) ldmatrix4_trans(mat + b * 8 * kStagePitch, a[b]);
    __syncwarp();
  }
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    uint32_t r[4];
#pragma unroll
    for (int m = 0; m < 4; ++m) {  // features 8m .. 8m+7
      float lo = __uint_as_float(v[m / 2][b * 4 + (m & 1) * 2]);
      float hi = __uint_as_float(v[m / 2][b * 4 + (m & 1) * 2 + 1]);
      if (add) {
        lo = __fadd_rn(lo, __uint_as_float(a[b][m] << 16));
        hi = __fadd_rn(hi, __uint_as_float(a[b][m] & 0xffff0000u));
      }
      r[m] = pack_bf16(lo, hi);
    }
    stmatrix4_trans(mat + b * 8 * kStagePitch, r);
  }
  __syncwarp();
  if (out.vec) {
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const int t = t0 + b * 8 + (lane >> 2);
      uint4 w;
      asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                   : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
                   : "r"(rowp + b * 8 * kStagePitch)
                   : "memory");
      if (t < out.tokens && nf > 0) store_part(out.p + t * out.ld + f, w, nf);
    }
  } else {  // a lane per feature, a token at a time (all read first: read and stored in turn took a latency each)
    uint16_t *q = reinterpret_cast<uint16_t *>(out.p) + static_cast<int64_t>(t0) * out.ld + lane;
    uint16_t w[16];
#pragma unroll
    for (int t = 0; t < 16; ++t) w[t] = lds16(stage + static_cast<uint32_t>(t * kStagePitch + lane * 2));
#pragma unroll
    for (int t = 0; t < 16; ++t)
      if (t0 + t < out.tokens && lane < out.feats) q[t * out.ld] = w[t];
  }
  __syncwarp();
}

// 16 tokens x 16 features, one fragment (gated products).
__device__ __forceinline__ void store_rows16(uint32_t stage, const float (&v)[8], int t0, const RowsOut &out,
                                             int lane) {
  constexpr int kPitch = 48;
  // matrices: features 0-7 and 8-15 of the first 8 tokens, then of the others
  const uint32_t mat =
      stage + static_cast<uint32_t>(((lane >> 4) * 8 + (lane & 7)) * kPitch + ((lane >> 3) & 1) * 16);
  const uint32_t r[4] = {pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])};
  stmatrix4_trans(mat, r);
  __syncwarp();
  if (out.vec) {
    const int t = t0 + (lane >> 1), f = (lane & 1) * 8, nf = out.feats - f;
    uint4 w;
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
                 : "r"(stage + static_cast<uint32_t>((lane >> 1) * kPitch + (lane & 1) * 16))
                 : "memory");
    if (t < out.tokens && nf > 0) store_part(out.p + t * out.ld + f, w, nf);
  } else {  // a lane per feature, two tokens at a time
    const int f = lane & 15;
    uint16_t *q = reinterpret_cast<uint16_t *>(out.p) + static_cast<int64_t>(t0) * out.ld + f;
    uint16_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = lds16(stage + static_cast<uint32_t>((2 * i + (lane >> 4)) * kPitch + f * 2));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int t = 2 * i + (lane >> 4);
      if (t0 + t < out.tokens && f < out.feats) q[t * out.ld] = w[i];
    }
  }
  __syncwarp();
}

__device__ __forceinline__ bool rows_aligned(const void *p, int64_t ld) {
  return ((reinterpret_cast<uintptr_t>(p) | static_cast<uintptr_t>(ld * 2)) & 15) == 0;
}

}  // namespace bimoe
