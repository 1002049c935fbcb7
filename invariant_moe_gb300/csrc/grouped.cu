// grouped.cu -- products of rows grouped by expert with each group's own matrix,
// and their gradients, on 5th-generation tensor cores: the plain products, and
// the routed experts' training step.
//
//   rows      y[p] = W[e] x[p]                 (or with W[e] transposed: the rows' gradient)
//   gate/up   [g u] = W13[e] x[p],  act = silu(g) u w
//   dact      dact = W2[e]^T dout[p],  s = 1 / (1 + exp(-g)),  dw = sum(dact silu(g) u),
//             dg = dact w u s (1 + g (1 - s)),  du = dact w g s
//   dx        contrib[pair] = W13[e]^T [dg du]
//   dw        dW[e] = sum over the group's p of dy[p] x[p]^T
// for the positions offsets[e] <= p < offsets[e+1] of group e.
//
// One kernel template over CTA pairs (cta_group::2), the tiles of all groups
// behind one another: 256 rows of A by up to 256 columns of B.
//   * rows, gate/up, dact, dx: A is the group's matrix, B its rows (columns of the
//     accumulator), so a group with few rows costs its weight bytes and no more
//     MMA columns than its rows rounded up to 32.  The tiles of a group are equally
//     wide.  A matrix that is reduced over its row index (W[e] transposed) is read
//     as it lies, as an MN-major operand.
//   * dw: A and B are dy and x, both MN-major, reduced over the group's rows in
//     steps of 64.  A step that runs past the group's end has the rows of the next
//     group in it: only the K=16 MMAs that the group reaches into are issued, and
//     of the last one's rows those past the end are set to zero in shared memory
//     first, in both operands, by a warp of each CTA between the copies' barrier
//     and the MMA thread's (the next group's rows may hold NaN).
//   * Recipe: the reduction in slices of 1024, each one chain of K=16 MMAs, the
//     slices added in fp32 in increasing order by the epilogue warps while the next
//     one runs (the tensor cores' additions truncate; slices bound what that costs
//     over long reductions: a chain of n leaves its sum about 1.1e-9 n too small).
//     gate/up is one chain over H up to 2048, as in the inference kernel, whose bits
//     it then has; beyond, slices (32768 rows, 32 groups, H=4096, I=2048, forward:
//     one chain 1111 us, slices 1119).  dact is cut into slices of 4096, as its long
//     epilogue holds one of the two accumulators meanwhile and a shorter slice ends
//     before it does (the same sizes, gather, dact and the parts' sum: slices of 4096
//     478 us, of 2048 530, of 1024 567).  dwts, an fp32 result with the errors of g,
//     u and dact in it, is 2.9e-6 too small in the 2-norm at H=1024, 6.4e-6 at 2048,
//     6.3e-6 at 4096 and no more beyond (dact uncut: 2.1e-5 at 16384, 3.8e-5 at
//     32768).  The down product of one slot a token is one chain over I, like the
//     inference kernel's: it is rounded to bf16 at once.
#include <mutex>

#include "tile_epilogue.cuh"
#include "train_internal.cuh"

namespace bimoe {

constexpr int kTM = 128;                 // rows of A per CTA
constexpr int kTK = 64;                  // reduction step of a stage
constexpr int kTABytes = kTM * kTK * 2;  // 16 KB
constexpr int kTSlab = 64 * kTK * 2;     // an MN-major slab: 64 rows or columns x 64 k
constexpr int kTAccCols = 256;
constexpr int kTMaxStages = 12;
constexpr int kTThreads = 384;           // TMA, MMA and end-of-group warps, one idle, 8 epilogue warps
// registers a thread: 168 at launch (384 x 168 = 64512); the first four warps
// hand some of theirs to the epilogue's, 128 x 56 + 256 x 224 = 64512
constexpr int kTRegsFew = 56, kTRegsMany = 224;
constexpr int kTBarBytes = 512;
constexpr int kTSmemMax = 227 * 1024;
constexpr int kTSliceK = 1024;
constexpr int kTOneChain = 2048;         // gate/up: one chain up to this H
constexpr int kTDactSlice = 4096;        // dact: slices of this length
static_assert((3 * kTMaxStages + 5) * 8 + 12 <= kTBarBytes, "barriers");

// kGateUpLong, kDactLong: those whose reduction has more than one slice.
enum GroupedOp { kRows, kGateUp, kGateUpLong, kDact, kDactLong, kWgrad };
constexpr bool is_gate_up(GroupedOp op) { return op == kGateUp || op == kGateUpLong; }
constexpr bool is_dact(GroupedOp op) { return op == kDact || op == kDactLong; }

// Staging buffer of an epilogue warp (kWgrad: 32 rows x 128 bytes).
__host__ __device__ constexpr int staging_bytes(GroupedOp op) { return op == kWgrad ? 4096 : kFStaging; }

// kWgrad: one of the gradients of a launch, its tiles of every group behind one another.
struct WgradPart {
  int rows, m_tiles;  // rows of dW, and tiles of 256 of them
  int cols, n_tiles;  // columns of dW, and tiles of n of them
  int first;          // its first tile
  void *out;
};

struct GroupedArgs {
  Groups g;
  int rows, m_tiles;   // rows of A and the result's features per group, and tiles of them (256; gate/up: 128 features)
  WgradPart part[2];   // kWgrad
  int nparts, tiles;   // kWgrad: how many, and their tiles together
  int early;           // the offsets and A may be read before the predecessor has finished
  int n;               // columns of a tile at most: a multiple of 32
  int nkb, slice_kb;   // steps of 64 (not kWgrad: by the group's rows), and how many make a slice
  int stages, stage_bytes;
  void *out;
  int64_t ldo;
  int out_f32;         // kRows: fp32, else bf16
  int mode;            // kWgrad: a GradMode
  const int32_t *perm; // kRows: rows go to row perm[p] (may be null: row p); gate/up, dact: index of wts
  const float *wts;
  float *gu;           // gate/up: written; dact: read
  float *parts;        // dact: sums over 32 features of dact silu(g) u, or null
  int *err;
};

// The two projections' gradients and the weight's from dact = d: one fixed fp32 sequence.  (Its sigmoid is not
// the one of swiglu_p_f32, which has the inference kernel's bits: both are within a few units of the last place, far
// below the bf16 rounding of act, dg and du.)
struct GateGradsW {
  float dg, du, dw;
};
__device__ __forceinline__ GateGradsW gate_grads_w(float d, float g, float u, float w) {
  const float s = sigmoid_approx(g), sg = __fmul_rn(g, s), dww = __fmul_rn(d, w);
  return {__fmul_rn(__fmul_rn(__fmul_rn(dww, s), u), __fmaf_rn(g, __fsub_rn(1.0f, s), 1.0f)), __fmul_rn(dww, sg),
          __fmul_rn(__fmul_rn(d, sg), u)};
}

__device__ __forceinline__ void prefetch_l2(const void *p) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(p) : "memory");
}

// Tensor maps of A, B and (kWgrad) dW, of each part.
template <bool WGRAD>
struct GroupedMaps {
  CUtensorMap a[1], b[1];
};
template <>
struct GroupedMaps<true> {
  CUtensorMap a[2], b[2], c[2];
};

// What an epilogue warp holds of its (up to 128) columns besides the accumulator: lane l has columns 32 i + l.
struct ColumnInfo {
  int pair[4];
  float w[4];
};

// Where a lane's projections lie, for its first column and feature: a row's 2I are
// kept as the tiles hold them, for each 16 features 8 lanes' quads (g, g + 8
// features on, u, u + 8 features on), so that both passes move whole lines without
// passing them through shared memory.
__device__ __forceinline__ float *quads_of(float *gu, int64_t pos0, int row0, int64_t two, int lane) {
  return gu + (pos0 + (lane & 3) * 2) * two + row0 * 2 + (lane >> 2) * 4;
}

// Epilogue of one warp of a rows product: acc[chunk][half] holds 16 columns from 16 chunk of 16 features from row0
// (+ 16); column c is position pos0 + c, c < limit.
__device__ __forceinline__ void rows_epilogue(const GroupedArgs &p, const float (&acc)[8][2][8], int row0, int64_t pos0,
                                              int limit, const ColumnInfo &col, uint32_t stage, int lane) {
  if (limit <= 0 || row0 >= p.rows) return;
  const int feats = p.rows - row0;
  const uint4 none[2] = {};
  if (!p.out_f32) {
    const RowsOut out{static_cast<__nv_bfloat16 *>(p.out) + (p.perm ? 0 : pos0 * p.ldo) + row0, p.ldo, limit, feats,
                      true};
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      if (c * 16 >= limit) break;
      uint32_t v[2][8];
#pragma unroll
      for (int j = 0; j < 16; ++j) v[j / 8][j % 8] = __float_as_uint(acc[c][j / 8][j % 8]);
      if (!p.perm) {
        store_rows32(stage, v, c * 16, out, nullptr, none, lane);
        continue;
      }
      stage_rows32(stage, v, lane);
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int t = b * 8 + (lane >> 2), f = (lane & 3) * 8;
        const int row = __shfl_sync(0xffffffffu, col.pair[c / 2], (c & 1) * 16 + t);
        const uint4 w = staged_part(stage, t, lane & 3);
        if (c * 16 + t < limit && static_cast<unsigned>(row) < static_cast<unsigned>(p.g.P) && f < feats)
          store_part(out.p + row * out.ld + f, w, feats - f);
      }
      __syncwarp();
    }
    return;
  }
  float *o = static_cast<float *>(p.out) + row0 + (lane & 7) * 4;
  const bool in = (lane & 7) * 4 < feats;  // feats is a multiple of 16
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    if (c * 16 >= limit) break;
    frag_to_rows(stage, acc[c], lane);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = i * 4 + (lane >> 3);
      float4 w;
      asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];"
                   : "=f"(w.x), "=f"(w.y), "=f"(w.z), "=f"(w.w)
                   : "r"(stage + static_cast<uint32_t>(t * kFPitch + (lane & 7) * 16))
                   : "memory");
      int64_t row = pos0 + c * 16 + t;
      bool ok = c * 16 + t < limit;
      if (p.perm) {
        const int pair = __shfl_sync(0xffffffffu, col.pair[c / 2], (c & 1) * 16 + t);
        ok = ok && static_cast<unsigned>(pair) < static_cast<unsigned>(p.g.P);
        row = pair;
      }
      if (ok && in) __stcs(reinterpret_cast<float4 *>(o + row * p.ldo), w);
    }
    __syncwarp();
  }
}

// Epilogues of one warp of gate/up and of dact, from tensor memory at t: a chunk of
// 16 columns at a time in a loop that is not unrolled (eight chunks' code behind
// one another does not fit the instruction cache: gather, dact and the parts' sum
// of 32768 rows, 32 groups, H=4096, I=2048 516 us, so 478).
__device__ __forceinline__ void chunk_weights(const ColumnInfo &col, int c, int lane, float (&w)[4]) {
  const float v = c < 2 ? col.w[0] : c < 4 ? col.w[1] : c < 6 ? col.w[2] : col.w[3];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    w[j] = __shfl_sync(0xffffffffu, v, (c & 1) * 16 + (lane & 3) * 2 + (j & 1) + (j >> 1) * 8);
}

__device__ __forceinline__ void gate_up_epilogue(const GroupedArgs &p, uint32_t t, int row0, int64_t pos0, int limit,
                                                 const ColumnInfo &col, uint32_t stage, int lane) {
  if (limit <= 0 || row0 >= p.rows) return;
  // half 0: gate values of the warp's 16 features from row0, half 1: their up values
  const RowsOut act{static_cast<__nv_bfloat16 *>(p.out) + pos0 * p.ldo + row0, p.ldo, limit, p.rows - row0, true};
  const int64_t two = 2 * static_cast<int64_t>(p.rows);
  float *gu = quads_of(p.gu, pos0, row0, two, lane);
#pragma unroll 1
  for (int c = 0; c * 16 < limit; ++c) {
    uint32_t d[2][8];
    tmem_ld_16x16(t + c * 16, d[0]);
    tmem_ld_16x16(t + (16u << 16) + c * 16, d[1]);
    float a[8], w[4];
    chunk_weights(col, c, lane, w);
    tmem_ld_wait();
#pragma unroll
    for (int j = 0; j < 8; ++j)
      a[j] = swiglu_p_f32(__uint_as_float(d[0][j]), __uint_as_float(d[1][j]), w[(j & 1) + (j >> 2) * 2]);
    store_rows16(stage, a, c * 16, act, lane);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int j = (i & 1) + (i >> 1) * 4, at = c * 16 + (i & 1) + (i >> 1) * 8;
      if (at + (lane & 3) * 2 < limit)
        __stcs(reinterpret_cast<uint4 *>(gu + at * two), make_uint4(d[0][j], d[0][j + 2], d[1][j], d[1][j + 2]));
    }
  }
}

__device__ __forceinline__ void dact_epilogue(const GroupedArgs &p, uint32_t t, int row0, int64_t pos0, int limit,
                                              const ColumnInfo &col, uint32_t stage, int lane) {
  if (limit <= 0 || row0 >= p.rows) return;
  const int feats = p.rows - row0;
  const uint4 none[2] = {};
  const int64_t two = 2 * static_cast<int64_t>(p.rows);
  __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(p.out) + pos0 * two + row0;
  const RowsOut dg{o, two, limit, feats, true}, du{o + p.rows, two, limit, feats, true};
  const float *gu = quads_of(p.gu, pos0, row0, two, lane);
  float *parts = p.parts ? p.parts + static_cast<int64_t>(row0 / 32) * p.g.P + pos0 : nullptr;
  // the next chunk's projections are loaded while this one's gradients are stored
  float4 next[4][2];
  const auto load = [&](int c) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int at = c * 16 + (i & 1) + (i >> 1) * 8;
      const bool in = at + (lane & 3) * 2 < limit;
#pragma unroll
      for (int h = 0; h < 2; ++h)
        next[i][h] = in ? __ldcs(reinterpret_cast<const float4 *>(gu + at * two + h * 32))
                        : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
  };
  load(0);
#pragma unroll 1
  for (int c = 0; c * 16 < limit; ++c) {
    uint32_t d[2][8];
    tmem_ld_16x16(t + c * 16, d[0]);
    tmem_ld_16x16(t + (16u << 16) + c * 16, d[1]);
    float4 q[4][2];
    float w[4], dw[4] = {};
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i / 2][i % 2] = next[i / 2][i % 2];
    load(c + 1);  // (past the last chunk: nothing)
    chunk_weights(col, c, lane, w);
    tmem_ld_wait();
    uint32_t a[2][8], b[2][8];
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const int h = j / 8, i = j % 8, u = (i & 1) + (i >> 2) * 2;
      const bool second = (i >> 1) & 1;
      const GateGradsW r =
          gate_grads_w(__uint_as_float(d[h][i]), second ? q[u][h].y : q[u][h].x, second ? q[u][h].w : q[u][h].z, w[u]);
      a[h][i] = __float_as_uint(r.dg);
      b[h][i] = __float_as_uint(r.du);
      dw[u] = __fadd_rn(dw[u], r.dw);
    }
    store_rows32(stage, a, c * 16, dg, nullptr, none, lane);
    store_rows32(stage, b, c * 16, du, nullptr, none, lane);
    if (parts) {  // the sums over the warp's 32 features of each column
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) dw[i] = __fadd_rn(dw[i], __shfl_xor_sync(0xffffffffu, dw[i], x));
      if (lane < 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int at = c * 16 + lane * 2 + (i & 1) + (i >> 1) * 8;
          if (at < limit) parts[at] = dw[i];
        }
      }
    }
  }
}

// Epilogue of one warp of dW: acc = row row0 + lane, columns col0 ..  Parts of 32
// rows x 128 bytes go through the warp's staging buffer, in the copies' swizzle
// (16-byte part j of row r at j ^ (r & 7): eight lanes' stores fall into different
// banks), and leave as tiled stores, whole lines at a time and without holding the
// warp (a lane storing 32-byte pieces of its own row: 4.0 TB/s, so 5.2).  Rows and columns past
// dW's are not stored.
__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ void wgrad_epilogue(const WgradPart &p, int mode, const CUtensorMap *tmC,
                                               const float (&acc)[128], int e, int row0, int col0, int ncols, uint32_t stage, int lane) {
  if (row0 >= p.rows) return;
  const uint32_t row = stage + static_cast<uint32_t>(lane * 128);
  const uint32_t x = static_cast<uint32_t>(lane & 7);
#pragma unroll
  for (int c = 0; c < 128; c += 32) {
    if (c >= ncols || col0 + c >= p.cols) break;
    const bool f32 = mode != kGradBf16;
    if (!f32 && (c & 32)) continue;  // bf16: 64 columns at once
    if (lane == 0) bulk_wait_read();
    __syncwarp();
    if (f32) {
#pragma unroll
      for (uint32_t j = 0; j < 8; ++j)
        sts128(row + ((j ^ x) << 4), __float_as_uint(acc[c + 4 * j]), __float_as_uint(acc[c + 4 * j + 1]),
               __float_as_uint(acc[c + 4 * j + 2]), __float_as_uint(acc[c + 4 * j + 3]));
    } else if ((c & 32) == 0) {
#pragma unroll
      for (uint32_t j = 0; j < 8; ++j)
        sts128(row + ((j ^ x) << 4), pack_bf16(acc[c + 8 * j], acc[c + 8 * j + 1]),
               pack_bf16(acc[c + 8 * j + 2], acc[c + 8 * j + 3]), pack_bf16(acc[c + 8 * j + 4], acc[c + 8 * j + 5]),
               pack_bf16(acc[c + 8 * j + 6], acc[c + 8 * j + 7]));
    }
    fence_proxy_async_shared();
    __syncwarp();
    if (lane == 0) {
      if (mode == kGradF32Accumulate) tma_store_3d<true>(tmC, stage, col0 + c, row0, e);
      else tma_store_3d<false>(tmC, stage, col0 + c, row0, e);
      bulk_commit();
    }
  }
}

template <GroupedOp OP, bool A_MN>
__global__ void __launch_bounds__(kTThreads, 1)
    grouped_kernel(const __grid_constant__ GroupedMaps<OP == kWgrad> maps, const __grid_constant__ GroupedArgs prm) {
  static_assert(OP != kWgrad || A_MN, "dW's operands are MN-major");
  extern __shared__ uint8_t smem_raw[];
  uint8_t *tiles = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
  const int stages = prm.stages, stage_bytes = prm.stage_bytes;
  uint8_t *stagings = tiles + stages * stage_bytes;  // of the epilogue warps
  uint8_t *aux = stagings + 8 * staging_bytes(OP);
  uint64_t *full = reinterpret_cast<uint64_t *>(aux);
  uint64_t *empty = full + kTMaxStages;
  uint64_t *tail = empty + kTMaxStages;  // kWgrad: this CTA's copies of a step that runs past its group
  uint64_t *tfull = tail + kTMaxStages;  // [2]
  uint64_t *tempty = tfull + 2;          // [2]
  uint64_t *drain = tempty + 2;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  int *total_slot = const_cast<int *>(abort_flag) + 1;
  int *offs = reinterpret_cast<int *>(aux + kTBarBytes);  // [E + 1]
  int *first = offs + prm.g.E + 1;                        // [E + 1] first tile of each group (not kWgrad: all alike)

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int unit0 = static_cast<int>(cluster_id_x()), nunits = static_cast<int>(num_clusters_x());
  const int E = prm.g.E;

  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      // kWgrad: two arrivals, the even CTA's copy thread's, or one of each CTA's end-of-group warp
      mbar_init(smem_u32(&full[s]), OP == kWgrad ? 2 : 1);
      mbar_init(smem_u32(&empty[s]), 1);
      mbar_init(smem_u32(&tail[s]), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(smem_u32(&tfull[a]), 1);
      mbar_init(smem_u32(&tempty[a]), 16);  // the epilogue warps of both CTAs, on the even CTA's barrier
    }
    mbar_init(smem_u32(drain), 1);
    *abort_flag = 0;
    fence_barrier_init();
    for (int i = 0; i < (OP == kWgrad ? prm.nparts : 1); ++i) {
      tma_prefetch_desc(&maps.a[i]);
      tma_prefetch_desc(&maps.b[i]);
    }
  }
  if (warp == 2) {
    if (lane == 0) *tmem_slot = 0u;
    __syncwarp();
    tmem_alloc_pair(smem_u32(tmem_slot), 2 * kTAccCols);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  if (!prm.early) griddep_wait();
  for (int i = threadIdx.x; i <= E; i += kTThreads) offs[i] = __ldcg(prm.g.offsets + i);
  __syncthreads();
  if (warp == 3) {
    // first[e] = tiles of the groups before e; each lane scans a contiguous chunk.  Offsets that do not rise within
    // 0..P would put tiles outside the operands: then there is no tile, and the error is recorded.
    const auto tiles_of = [&](int e) { return prm.m_tiles * ((max(offs[e + 1] - offs[e], 0) + prm.n - 1) / prm.n); };
    const int per = (E + 31) / 32, e0 = min(lane * per, E), e1 = min(e0 + per, E);
    bool bad = lane == 0 && (offs[0] < 0 || offs[E] > prm.g.P);
    int local = 0;
    for (int e = e0; e < e1; ++e) {
      bad = bad || offs[e + 1] < offs[e];
      if (OP != kWgrad) local += tiles_of(e);
    }
    bad = __any_sync(0xffffffffu, bad);
    int incl = local;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += v;
    }
    int run = incl - local;
    for (int e = e0; e < e1; ++e) {
      if (OP == kWgrad) break;  // (all groups alike)
      first[e] = run;
      run += tiles_of(e);
    }
    if (lane == 31) {
      if (OP != kWgrad) first[E] = incl;
      *total_slot = bad ? 0 : OP == kWgrad ? prm.tiles : incl;
    }
    if (bad && lane == 0) report_error(prm.err, BI_DEVERR_BAD_PERMUTATION);
  }
  __syncthreads();
  const int total = *total_slot;

  auto wait = [&](uint32_t bar, uint32_t parity, volatile int *ab) { return mbar_wait_cl(bar, parity, ab, prm.err); };
  // A tile: its group, first row of A (gate/up: feature), first column (position, kWgrad: column of dW), columns (of
  // the group, and of the MMA), and reduction steps.  The groups' tiles rise, so a role's search for the group goes
  // on from the one before.  Columns fastest: the tiles of a row block follow one another and share its A in L2.
  struct Tile {
    int e, row, col, cols, n, nkb, part;
  };
  auto tile_at = [&](int tile, int e) {
    Tile t;
    if (OP == kWgrad) {
      t.part = prm.nparts > 1 && tile >= prm.part[1].first;
      const WgradPart &w = prm.part[t.part];
      const int all = w.m_tiles * w.n_tiles;
      t.e = (tile - w.first) / all;
      const int local = tile - w.first - t.e * all, r = local / w.n_tiles;
      t.row = r * 2 * kTM;
      t.col = (local - r * w.n_tiles) * prm.n;
      t.cols = offs[t.e + 1] - offs[t.e];  // rows of the group
      t.n = prm.n;
      t.nkb = (t.cols + kTK - 1) / kTK;
    } else {
      if (first[e + 1] <= tile) {  // often the next group; the last whose first tile is not past this one
        int hi = E - 1;
        ++e;
        while (first[e + 1] <= tile) {
          const int mid = (e + hi + 1) >> 1;
          if (first[mid] <= tile) e = mid;
          else hi = mid - 1;
        }
      }
      t.e = e;
      t.part = 0;
      const int local = tile - first[e], beg = offs[e], cnt = offs[e + 1] - beg;
      const int ntt = (cnt + prm.n - 1) / prm.n, r = local / ntt, c = local - r * ntt;
      const int width = ((cnt + ntt - 1) / ntt + 31) & ~31;  // of the group's tiles
      t.row = r * (is_gate_up(OP) ? kTM : 2 * kTM);
      t.col = beg + c * width;
      t.cols = min(width, cnt - c * width);
      t.n = (max(t.cols, 1) + 31) & ~31;
      t.nkb = prm.nkb;
    }
    return t;
  };
  // kWgrad: rows of the group in step kb, and whether the last K=16 MMA of the step reaches past them
  auto rows_in = [](int cnt, int kb) { return min(kTK, cnt - kb * kTK); };

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kTRegsFew));
    if (warp == 0) {
      // ---------------------------------------------------- TMA producer --
      // (alone in its warp, as the MMA thread: lanes waiting beside it slow its branches and waits)
      if (elect_one()) {
        int stage = 0, e = 0;
        uint32_t phase = 0;
        bool ok = true;
        const int b_rows = prm.n / 2;  // of the box
        const uint32_t b_bytes = OP == kWgrad ? static_cast<uint32_t>((b_rows + 63) / 64 * kTSlab)
                                              : static_cast<uint32_t>(b_rows * kTK * 2);
        // (early: A's copies of the first steps are under way before the wait, B's follow)
        int ahead = 0;
        const auto load_a = [&](const Tile &ti, uint32_t st, uint32_t fb, int k, int row) {
          const CUtensorMap *tmA = &maps.a[ti.part];
          if (OP == kWgrad) {
            tma_load_2d_pair(st, tmA, fb, row, offs[ti.e] + k);
            tma_load_2d_pair(st + kTSlab, tmA, fb, row + 64, offs[ti.e] + k);
          } else if (is_gate_up(OP)) {
            tma_load_4d_pair(st, tmA, fb, k, 0, 0, (ti.e * 2 * prm.rows + row) / 16);
          } else if (A_MN) {
            tma_load_3d_pair(st, tmA, fb, row, k, ti.e);
            tma_load_3d_pair(st + kTSlab, tmA, fb, row + 64, k, ti.e);
          } else {
            tma_load_2d_pair(st, tmA, fb, k, ti.e * prm.rows + row);
          }
        };
        const int row_of_rank = static_cast<int>(rank) * (is_gate_up(OP) ? kTM / 2 : kTM);
        if (prm.early) {
          if (OP != kWgrad && unit0 < total) {
            const Tile ti = tile_at(unit0, 0);
            for (; ahead < min(stages, ti.nkb); ++ahead) {
              if (rank == 0) mbar_arrive_expect_tx(smem_u32(&full[ahead]), 2 * (kTABytes + b_bytes));
              load_a(ti, smem_u32(tiles + ahead * stage_bytes), mapa_shared(smem_u32(&full[ahead]), 0), ahead * kTK,
                     ti.row + row_of_rank);
            }
          }
          griddep_wait();
        }
        griddep_launch_dependents();  // (a dependent's CTAs need an SM of their own: this one's shared memory is full)
        for (int tile = unit0; tile < total && ok; tile += nunits) {
          const Tile ti = tile_at(tile, e);
          e = ti.e;
          const CUtensorMap *tmB = &maps.b[ti.part];
          const int half = OP == kWgrad ? b_rows : ti.n / 2;
          const int row = ti.row + row_of_rank, col = ti.col + static_cast<int>(rank) * half;
          for (int kb = 0; kb < ti.nkb; ++kb) {
            const uint32_t st = smem_u32(tiles + stage * stage_bytes);
            uint32_t fb = mapa_shared(smem_u32(&full[stage]), 0);
            const int k = kb * kTK;
            if (ahead > 0) {
              --ahead;  // armed, and A's copies issued
            } else {
              if (!wait(smem_u32(&empty[stage]), phase ^ 1u, abort_flag)) {
                ok = false;
                break;
              }
              if (OP == kWgrad && (rows_in(ti.cols, kb) & 15)) {
                mbar_arrive_expect_tx(smem_u32(&tail[stage]), kTABytes + b_bytes);
                fb = mapa_shared(smem_u32(&tail[stage]), rank);
              } else if (rank == 0) {
                mbar_arrive_expect_tx(smem_u32(&full[stage]), 2 * (kTABytes + b_bytes));
                if (OP == kWgrad) mbar_arrive(smem_u32(&full[stage]));
              }
              load_a(ti, st, fb, k, row);
            }
            if (OP == kWgrad) {
              tma_load_2d_pair(st + kTABytes, tmB, fb, col, offs[e] + k);
              if (half > 64) tma_load_2d_pair(st + kTABytes + kTSlab, tmB, fb, col + 64, offs[e] + k);
            } else {
              tma_load_2d_pair(st + kTABytes, tmB, fb, k, col);
            }
            if (++stage == stages) {
              stage = 0;
              phase ^= 1u;
            }
          }
        }
        if (*abort_flag) {
          // copies take microseconds: every one that was started has landed after this
          const unsigned long long t0 = globaltimer_ns();
          while (globaltimer_ns() - t0 < 1000000ull) {
          }
        }
      } else {
        return;
      }
    } else if (warp == 1) {
      // ------------------------------------------------------ MMA issuer --
      if (rank == 0 && elect_one()) {
        int stage = 0, buf = 0, e = 0;
        uint32_t phase = 0, buf_phase = 0;
        bool ok = true;
        for (int tile = unit0; tile < total && ok && !*abort_flag; tile += nunits) {
          const Tile ti = tile_at(tile, e);
          e = ti.e;
          const uint32_t idesc =
              idesc_bf16_f32(2 * kTM, ti.n) | (A_MN ? kIdescAMn : 0u) | (OP == kWgrad ? kIdescBMn : 0u);
          for (int kb0 = 0; kb0 < ti.nkb && ok; kb0 += prm.slice_kb) {
            const int kb1 = min(ti.nkb, kb0 + prm.slice_kb);
            if (!wait(smem_u32(&tempty[buf]), buf_phase ^ 1u, abort_flag)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t d = tmem_base + static_cast<uint32_t>(buf * kTAccCols);
            for (int kb = kb0; kb < kb1; ++kb) {
              if (!wait(smem_u32(&full[stage]), phase, abort_flag)) {
                ok = false;
                break;
              }
              tc_fence_after();
              const uint32_t a0 = smem_u32(tiles + stage * stage_bytes), b0 = a0 + kTABytes;
              const int steps = OP == kWgrad ? (rows_in(ti.cols, kb) + 15) / 16 : kTK / 16;
#pragma unroll
              for (int k = 0; k < kTK / 16; ++k) {
                const uint64_t ad = A_MN ? sdesc_sw128_mn(a0 + k * 2048, kTSlab) : sdesc_sw128(a0 + k * 32);
                const uint64_t bd = OP == kWgrad ? sdesc_sw128_mn(b0 + k * 2048, kTSlab) : sdesc_sw128(b0 + k * 32);
                if (OP != kWgrad || k < steps) umma_f16_pair(d, ad, bd, idesc, (kb > kb0 || k) ? 1u : 0u);
              }
              umma_commit_pair(smem_u32(&empty[stage]), 0x3);
              if (++stage == stages) {
                stage = 0;
                phase ^= 1u;
              }
            }
            if (!ok) break;
            umma_commit_pair(smem_u32(&tfull[buf]), 0x3);
            if (++buf == 2) {
              buf = 0;
              buf_phase ^= 1u;
            }
          }
        }
        // every MMA into both CTAs' tensor memory has completed
        umma_commit_pair(smem_u32(drain), 0x3);
        wait(smem_u32(drain), 0, nullptr);
      } else {
        return;
      }
    } else if (OP == kWgrad && warp == 2) {
      // ------------------------------------------------ ends of the groups --
      int stage = 0, e = 0;
      uint32_t parity = 0;  // bit s: of the next phase of tail[s]
      const int b_slabs = (prm.n / 2 + 63) / 64;
      for (int tile = unit0; tile < total; tile += nunits) {
        const Tile ti = tile_at(tile, e);
        e = ti.e;
        if (ti.nkb == 0) continue;
        stage = (stage + ti.nkb - 1) % stages;
        const int n = rows_in(ti.cols, ti.nkb - 1);
        if (n & 15) {
          if (!__all_sync(0xffffffffu, wait(smem_u32(&tail[stage]), (parity >> stage) & 1u, abort_flag) ? 1 : 0)) break;
          parity ^= 1u << stage;
          // rows n .. of the 16 that the last MMA takes, 128 bytes each in every slab (a row's 16-byte parts change
          // places within the row)
          const uint32_t st = smem_u32(tiles + stage * stage_bytes);
          if ((lane >> 3) < 2 + b_slabs) {  // eight lanes a slab
            const uint32_t at = st + static_cast<uint32_t>((lane >> 3) * kTSlab + (lane & 7) * 16);
            for (int r = n; r & 15; ++r) sts128(at + static_cast<uint32_t>(r * 128), 0, 0, 0, 0);
          }
          fence_proxy_async_shared();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(&full[stage]), 0));
        }
        if (++stage == stages) stage = 0;
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kTRegsMany));
    // -------------------------------------------------------- epilogue --
    const int q = warp & 3, h = (warp - 4) >> 2;
    const uint32_t staging = smem_u32(stagings + (warp - 4) * staging_bytes(OP));
    if (prm.early) griddep_wait();
    int buf = 0, e = 0;
    uint32_t buf_phase = 0;
    bool ok = true;
    for (int tile = unit0; tile < total && ok; tile += nunits) {
      const Tile ti = tile_at(tile, e);
      e = ti.e;
      const int ncols = ti.n / 2;  // columns of this warp: half h of the tile
      const int limit = min(ncols, ti.cols - h * ncols);
      ColumnInfo col = {};
      if (OP != kWgrad && prm.perm) {
        bool bad = false;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int c = 32 * i + lane;
          if (c < limit) {
            col.pair[i] = __ldg(prm.perm + ti.col + h * ncols + c);
            const bool in = static_cast<unsigned>(col.pair[i]) < static_cast<unsigned>(prm.g.P);
            bad = bad || !in;
            if (OP != kRows && in) col.w[i] = __ldg(prm.wts + col.pair[i]);
          }
        }
        if (bad) report_error(prm.err, BI_DEVERR_BAD_PERMUTATION);
      }
      if (is_dact(OP)) {
        // the projections that the epilogue reads, on their way to L2 while the tile is computed: 256 bytes for each
        // of the warp's columns
        const int row0 = ti.row + static_cast<int>(rank) * kTM + q * 32;
        const float *gu = prm.gu + (static_cast<int64_t>(ti.col) + h * ncols) * 2 * prm.rows + row0 * 2;
        for (int c = lane; c < limit && row0 < prm.rows; c += 32) {
          prefetch_l2(gu + static_cast<int64_t>(c) * 2 * prm.rows);
          prefetch_l2(gu + static_cast<int64_t>(c) * 2 * prm.rows + 32);
        }
      }
      const int row0 =
          ti.row + static_cast<int>(rank) * (is_gate_up(OP) ? kTM / 2 : kTM) + q * (is_gate_up(OP) ? 16 : 32);
      const auto tfull_wait = [&] {
        ok = __all_sync(0xffffffffu, wait(smem_u32(&tfull[buf]), buf_phase, abort_flag) ? 1 : 0) != 0;
        tc_fence_after();
        return ok;
      };
      const auto release = [&] {  // the accumulator has been read
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster_relaxed(mapa_shared(smem_u32(&tempty[buf]), 0));
        if (++buf == 2) {
          buf = 0;
          buf_phase ^= 1u;
        }
      };
      const auto accumulator = [&] {
        return tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(buf * kTAccCols + h * ncols);
      };
      if constexpr (is_gate_up(OP) || is_dact(OP)) {
        const uint32_t halves = 16u << 16;  // from a warp's first 16 lanes to the others
        if constexpr (OP == kGateUpLong || OP == kDactLong) {
          // the sums of all slices into the last one's accumulator
          float acc[8][2][8];
#pragma unroll
          for (int c = 0; c < 128; ++c) acc[c / 16][c / 8 % 2][c % 8] = 0.0f;
          for (int kb0 = 0; kb0 < ti.nkb; kb0 += prm.slice_kb) {
            if (!tfull_wait()) break;
            const uint32_t t = accumulator();
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              if (c * 16 < ncols) {
                uint32_t d[2][8];
                tmem_ld_16x16(t + c * 16, d[0]);
                tmem_ld_16x16(t + halves + c * 16, d[1]);
                tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 16; ++j)
                  acc[c][j / 8][j % 8] = __fadd_rn(acc[c][j / 8][j % 8], __uint_as_float(d[j / 8][j % 8]));
              }
            }
            if (kb0 + prm.slice_kb < ti.nkb) release();
          }
          if (!ok) break;
          const uint32_t t = accumulator();
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            if (c * 16 < ncols) {
              tmem_st_16x16(t + c * 16, acc[c][0]);
              tmem_st_16x16(t + halves + c * 16, acc[c][1]);
            }
          }
          tmem_st_wait();
        } else {
          if (!tfull_wait()) break;
        }
        const int64_t pos0 = static_cast<int64_t>(ti.col) + h * ncols;
        if (is_gate_up(OP)) gate_up_epilogue(prm, accumulator(), row0, pos0, limit, col, staging, lane);
        else dact_epilogue(prm, accumulator(), row0, pos0, limit, col, staging, lane);
        release();
      } else {
        // the sums of the slices, in the order that the epilogue wants them
        float acc[8][2][8];
#pragma unroll
        for (int c = 0; c < 128; ++c)  // (-0 + d is d, whatever d: one slice is taken as it is)
          acc[c / 16][c / 8 % 2][c % 8] = OP == kWgrad ? 0.0f : -0.0f;
        for (int kb0 = 0; kb0 < ti.nkb; kb0 += prm.slice_kb) {
          if (!tfull_wait()) break;
          const uint32_t t = accumulator();
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            if (c * 16 < ncols) {
              uint32_t d[2][8];
              if (OP == kWgrad) {
                uint32_t w[16];
                tmem_ld16(t + c * 16, w);
                tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 16; ++j) d[j / 8][j % 8] = w[j];
              } else {
                tmem_ld_16x16(t + c * 16, d[0]);
                tmem_ld_16x16(t + (16u << 16) + c * 16, d[1]);
                tmem_ld_wait();
              }
#pragma unroll
              for (int j = 0; j < 16; ++j)
                acc[c][j / 8][j % 8] = __fadd_rn(acc[c][j / 8][j % 8], __uint_as_float(d[j / 8][j % 8]));
            }
          }
          release();
        }
        if (!ok) break;
        if constexpr (OP == kWgrad) {
          float flat[128];
#pragma unroll
          for (int c = 0; c < 128; ++c) flat[c] = acc[c / 16][c / 8 % 2][c % 8];
          wgrad_epilogue(prm.part[ti.part], prm.mode, &maps.c[ti.part], flat, e, row0, ti.col + h * ncols, ncols, staging,
                         lane);
        } else {
          rows_epilogue(prm, acc, row0, static_cast<int64_t>(ti.col) + h * ncols, limit, col, staging, lane);
        }
      }
    }
    if (OP == kWgrad && lane == 0) bulk_wait();
  }

  tc_fence_before();
  __syncthreads();
  // the even CTA's final commit: its last MMAs have left this CTA's memory too
  if (rank != 0 && threadIdx.x == 96) wait(smem_u32(drain), 0, nullptr);
  cluster_sync_rest();  // neither CTA leaves while the other may still signal its barriers
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, 2 * kTAccCols);
  }
}

// ------------------------------------------------------------------- host --
static int div_up(int64_t a, int64_t b) { return static_cast<int>((a + b - 1) / b); }

template <GroupedOp OP, bool A_MN>
static bi_status launch_grouped(const GroupedMaps<OP == kWgrad> &maps, GroupedArgs p, cudaStream_t s) {
  static std::mutex mu;
  static int max_units[64] = {};  // CTA pairs resident at once, per device
  static ContextSetup setup;      // the shared-memory attribute is per context
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64) {
    set_error("device ordinal %d out of range", dev);
    return BI_ERR_CUDA;
  }
  auto kern = grouped_kernel<OP, A_MN>;
  {
    std::lock_guard<std::mutex> lk(mu);
    if (max_units[dev] == 0 || setup.pending(dev)) {
      cudaLaunchConfig_t cfg = {};
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = 2;
      attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
      cfg.gridDim = dim3(2 * (num_sms() / 2));
      cfg.blockDim = dim3(kTThreads);
      cfg.dynamicSmemBytes = kTSmemMax;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      int clusters = 0;
      cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kTSmemMax);
      if (e == cudaSuccess) e = cudaOccupancyMaxActiveClusters(&clusters, kern, &cfg);
      if (e != cudaSuccess || clusters <= 0) {
        cudaGetLastError();
        set_error("grouped kernel set-up: %s (%d clusters)", cudaGetErrorString(e), clusters);
        return BI_ERR_CUDA;
      }
      max_units[dev] = clusters;
      setup.done(dev);
    }
  }
  p.err = device_error_word();
  const int fixed = 1024 + kTBarBytes + 8 * staging_bytes(OP) +
                    (OP == kWgrad ? 1 : 2) * (p.g.E + 1) * static_cast<int>(sizeof(int));
  p.stage_bytes = kTABytes + (OP == kWgrad ? div_up(p.n / 2, 64) * kTSlab : p.n / 2 * kTK * 2);
  p.stages = std::min(kTMaxStages, (kTSmemMax - fixed) / p.stage_bytes);
  int64_t most = static_cast<int64_t>(p.m_tiles) * (static_cast<int64_t>(p.g.P) / p.n + p.g.E);
  if (OP == kWgrad) {
    most = 0;
    for (int i = 0; i < p.nparts; ++i) {
      p.part[i].first = static_cast<int>(std::min<int64_t>(most, INT32_MAX));
      most += static_cast<int64_t>(p.g.E) * p.part[i].m_tiles * p.part[i].n_tiles;
    }
    p.tiles = static_cast<int>(std::min<int64_t>(most, INT32_MAX));
  }
  if (most > (int64_t(1) << 30)) {
    set_error("grouped product with more than 2^30 tiles");
    return BI_ERR_UNSUPPORTED;
  }
  const int units = static_cast<int>(std::min<int64_t>(max_units[dev], most));
  return launch_chained(kern, dim3(2 * units), dim3(kTThreads), static_cast<size_t>(fixed + p.stages * p.stage_bytes), s,
                        2, maps, p);
}

// Cycles of a reduction step of a tile of `cols` columns, up to n of them copied:
// bound by its MMAs (2 cols cycles) or by its copies (64 bytes a cycle and SM: 16 KB
// of A and 64 n bytes of B).
static int64_t step_cycles(int cols, int n) { return std::max(2 * cols, 256 + n); }

// Estimated cycles of a launch over the groups' rows with tiles of up to n columns:
// the waves of tiles over the CTA pairs, each as long as its reduction or its
// epilogue (`chunk` cycles for each 16 columns of its warps), whichever is longer,
// the other once, at the end.
static int64_t rows_cycles(const Groups &g, int m_tiles, int nkb, int n, int chunk) {
  const int64_t groups = std::min(g.E, g.P), mean = (g.P + groups - 1) / groups, per = (mean + n - 1) / n;
  const int64_t tiles = groups * m_tiles * per, pairs = std::max(1, num_sms() / 2), waves = (tiles + pairs - 1) / pairs;
  const int cols = static_cast<int>(((mean + per - 1) / per + 31) / 32 * 32);
  const int64_t reduce = nkb * step_cycles(cols, n) + 800, epilogue = static_cast<int64_t>(cols / 32) * chunk + 1500;
  return waves * std::max(reduce, epilogue) + std::min(reduce, epilogue);
}

static GroupedArgs problem(const Groups &g, int64_t rows, int64_t K, int64_t slice, int tile_rows, int chunk) {
  GroupedArgs p{};
  p.g = g;
  p.rows = static_cast<int>(rows);
  p.m_tiles = div_up(rows, tile_rows);
  p.nkb = div_up(K, kTK);
  p.slice_kb = std::max(1, static_cast<int>(slice / kTK));
  int64_t best = INT64_MAX;
  for (int n = 256; n >= 32; n /= 2) {
    const int64_t cost = rows_cycles(g, p.m_tiles, p.nkb, n, chunk);
    if (cost < best) best = cost, p.n = n;
  }
  return p;
}

// Rows x [P, K] (row stride ld) times w, `rows` features of the result; K-major w [E, rows, K] or MN-major [E, K, rows].
template <GroupedOp OP, bool A_MN>
static bi_status launch_over_rows(GroupedArgs p, Mat x, const __nv_bfloat16 *w, int64_t K, cudaStream_t s) {
  GroupedMaps<false> m;
  const uint64_t rows = static_cast<uint64_t>(p.rows), E = static_cast<uint64_t>(p.g.E);
  const bool ok = is_gate_up(OP) ? make_tma_inter_bf16(m.a, w, E * 2 * rows, rows, K)
                  : A_MN        ? make_tma_3d(m.a, w, false, E, K, rows, kTK)
                                : make_tma_2d_bf16(m.a, w, E * rows, K, kTM);
  if (!ok || !make_tma_2d_bf16_ld(m.b, x.p, p.g.P, K, x.ld, p.n / 2)) return BI_ERR_CUDA;
  return launch_grouped<OP, A_MN>(m, p, s);
}

bi_status launch_grouped_rows(Mat x, const __nv_bfloat16 *w, bool mn, Groups g, void *out, bool out_f32, int64_t ldo,
                              int64_t N, int64_t K, cudaStream_t s) {
  GroupedArgs p = problem(g, N, K, kTSliceK, 2 * kTM, 500);
  p.out = out;
  p.ldo = ldo;
  p.out_f32 = out_f32;
  return mn ? launch_over_rows<kRows, true>(p, x, w, K, s) : launch_over_rows<kRows, false>(p, x, w, K, s);
}

bi_status launch_grouped_dw(const GroupedDw *d, int count, Groups g, int mode, cudaStream_t s) {
  GroupedArgs p{};
  p.g = g;
  p.slice_kb = kTSliceK / kTK;
  p.mode = mode;
  p.n = 128;
  for (int i = 0; i < count; ++i)
    if (d[i].K > 128) p.n = 256;
  GroupedMaps<true> m;
  for (int i = 0; i < count; ++i) {
    p.part[p.nparts++] = WgradPart{static_cast<int>(d[i].N), div_up(d[i].N, 2 * kTM), static_cast<int>(d[i].K),
                                   div_up(d[i].K, p.n), 0, d[i].dw};
    if (!make_tma_2d_bf16_ld(&m.a[i], d[i].dy.p, g.P, d[i].N, d[i].dy.ld, kTK) ||
        !make_tma_2d_bf16_ld(&m.b[i], d[i].x.p, g.P, d[i].K, d[i].x.ld, kTK) ||
        !make_tma_3d(&m.c[i], d[i].dw, mode != kGradBf16, g.E, d[i].N, d[i].K, 32))
      return BI_ERR_CUDA;
  }
  return launch_grouped<kWgrad, true>(m, p, s);
}

// The training step's products follow a launch of this library that writes neither the weights nor the offsets, and
// whose own wait covers everything before it: both may be read before that launch has finished.
bi_status launch_train_gate_up(const __nv_bfloat16 *x, Groups g, const int32_t *perm, const float *wts,
                               const __nv_bfloat16 *w13, __nv_bfloat16 *act, float *gu, int64_t H, int64_t I,
                               cudaStream_t s) {
  const bool slices = H > kTOneChain;
  GroupedArgs p = problem(g, I, H, slices ? kTSliceK : H, kTM, 1000);
  p.out = act;
  p.ldo = I;
  p.perm = perm;
  p.wts = wts;
  p.gu = gu;
  p.early = 1;
  return slices ? launch_over_rows<kGateUpLong, false>(p, Mat{x, H}, w13, H, s)
                : launch_over_rows<kGateUp, false>(p, Mat{x, H}, w13, H, s);
}

bi_status launch_train_dact(const __nv_bfloat16 *dout, Groups g, const int32_t *perm, const float *wts,
                            const __nv_bfloat16 *w2, const float *gu, __nv_bfloat16 *dgu, float *dw_parts, int64_t H,
                            int64_t I, cudaStream_t s) {
  const bool slices = H > kTDactSlice;
  GroupedArgs p = problem(g, I, H, slices ? kTDactSlice : H, 2 * kTM, 2000);
  p.out = dgu;
  p.ldo = 2 * I;
  p.perm = perm;
  p.wts = wts;
  p.gu = const_cast<float *>(gu);
  p.parts = dw_parts;
  p.early = 1;
  return slices ? launch_over_rows<kDactLong, true>(p, Mat{dout, H}, w2, H, s)
                : launch_over_rows<kDact, true>(p, Mat{dout, H}, w2, H, s);
}

bi_status launch_train_dx(const __nv_bfloat16 *dgu, Groups g, const int32_t *perm, const __nv_bfloat16 *w13, void *out,
                          bool out_f32, int64_t H, int64_t I, cudaStream_t s) {
  GroupedArgs p = problem(g, H, 2 * I, kTSliceK, 2 * kTM, 700);
  p.out = out;
  p.ldo = H;
  p.out_f32 = out_f32;
  p.perm = perm;
  p.early = 1;
  return launch_over_rows<kRows, true>(p, Mat{dgu, 2 * I}, w13, 2 * I, s);
}

bi_status launch_train_down(const __nv_bfloat16 *act, Groups g, const int32_t *perm, const __nv_bfloat16 *w2,
                            __nv_bfloat16 *out, int64_t H, int64_t I, cudaStream_t s) {
  GroupedArgs p = problem(g, H, I, I, 2 * kTM, 700);
  p.out = out;
  p.ldo = H;
  p.perm = perm;
  p.early = 1;
  return launch_over_rows<kRows, false>(p, Mat{act, I}, w2, I, s);
}

}  // namespace bimoe
