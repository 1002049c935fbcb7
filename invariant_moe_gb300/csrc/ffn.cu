// ffn.cu -- the dense gated feed-forward block (a shared expert), forward and
// backward, on 5th-generation tensor cores.
//
//   forward   [g u] = x W13^T,  act = silu(g) u,  out = act W2^T (+ addend)
//   backward  dact = dout W2,  s = 1 / (1 + exp(-g)),
//             dg = dact u s (1 + g (1 - s)),  du = dact g s,
//             dx = [dg du] W13,  dW13 = [dg du]^T x,  dW2 = dout^T act
//
// Six products, one kernel template.  The left operand A (weights; for the
// weight gradients the token matrix whose columns become dW's rows) gives the
// 256 rows of a tile, the right operand B (tokens; for the weight gradients the
// other matrix' columns) its up to 256 columns.
//   * Operands come as they lie in memory.  Where the reduction index is the
//     contiguous one they are K-major tiles, where it is the row index (W2 in
//     dact, W13 in dx, all operands of the weight gradients) MN-major ones:
//     nothing is transposed in memory.
//   * CTA pairs (cta_group::2): each CTA stages its own 128 rows of A and half
//     of B's, one thread of the even CTA issues M=256 MMAs over both.  A K step
//     of 64 is 32 KB per SM, six of them in flight.
//   * Recipe.  The reduction is cut into slices of 1024; a slice is one chain of
//     K=16 MMAs in tensor memory and the slices are added in fp32 in increasing
//     order, from +0, by the epilogue warps in registers while the next slice
//     runs.  The recipe depends on the reduction length alone, so a token's row
//     of out and dx has the same bits in every batch.  The weight gradients
//     reduce over the tokens by the same slices: the tensor cores' additions
//     truncate, and one chain over 2^20 tokens of one sign ended 0.7 % low, past
//     a bf16 rounding, in slices within 2e-4 (backward, one chain and slices: 8191
//     tokens, H=4096, I=2048 542, 545 us; 65536, H=1024, I=512 413, 418).
//   * Eight epilogue warps, 32 rows x half of the columns each, keep the tile in
//     registers, so tensor memory is free again before anything is stored.
//     gate/up: each CTA holds 64 gate rows and the matching 64 up rows in
//     16-row groups, so a warp's two 16-lane reads give a thread both
//     projections of a feature.
//   * Rounded to bf16: act, dg and du, because the tensor cores take bf16
//     operands (one rounding between two products, 2^-9 on average), and each
//     result once.  g and u stay fp32 from forward to backward: rounded to bf16
//     as well they would add as much error again to every gradient.
//
// What bounds it, measured on a GB300 (cuBLAS bf16: 1.90 PFLOP/s in a burst,
// 1.70 held for seconds at the power cap):
//   4096 tokens, H=4096, I=2048: forward 112 us, 1.84 PFLOP/s, with an addend 119
//     (tensor cores; 4 waves of tiles of 224 tokens on 76 pairs);
//   8191 tokens: forward 238-256 us, backward 545 us, 1.6-1.7 and 1.5 PFLOP/s
//     (power: the SM clock falls to 1.5-1.6 GHz, where the tensor peak is 1.9);
//   4096 tokens, H=2048, I=768: forward 36 us, backward 63 us (1.1 and 1.2
//     PFLOP/s: one to two waves of tiles, and the last tile's epilogue, 9 us in
//     dact, which reads 8 bytes and writes 4 for each element);
//   fp32 weight gradients instead of bf16 ones: 65.7 us for that backward, added
//     to what is there 82.8 (a lane adds 32-byte pieces of its own row: the reads
//     come late and apart);
//   257 tokens, H=1040, I=720: step 29 us (six times a launch's fixed cost: set-up,
//     first copies, the last tile).
#include <atomic>
#include <mutex>

#include "tile_epilogue.cuh"

namespace bimoe {

constexpr int kFM = 128;                       // rows of A per CTA
constexpr int kFK = 64;                        // reduction step of a stage
constexpr int kFStages = 6;
constexpr int kFABytes = kFM * kFK * 2;        // 16 KB
constexpr int kFBBytes = 128 * kFK * 2;        // 16 KB: at most 128 rows of B per CTA
constexpr int kFStageBytes = kFABytes + kFBBytes;
constexpr int kFSlab = 64 * kFK * 2;           // an MN-major slab: 64 rows or columns x 64 k
constexpr int kFAccCols = 256;
constexpr int kFThreads = 384;                 // TMA and MMA warps (two idle), 8 epilogue warps
// registers a thread: 168 at launch (384 x 168 = 64512); the first four warps
// hand some of theirs to the epilogue's, 128 x 56 + 256 x 224 = 64512
constexpr int kFRegsFew = 56, kFRegsMany = 224;
constexpr int kFSmem = 1024 + kFStages * kFStageBytes + 256 + 8 * 16 * 144;  // ring, barriers, epilogue staging
constexpr int kSliceK = 1024;                  // reduction slice of the recipe
static_assert(kFSmem <= 227 * 1024, "shared memory");

// kGrads: up to three problems in one launch, each as kStore (dx) or a weight gradient.
enum FfnEpi { kGateUp, kStore, kDact, kGrads };

struct FfnGemm {
  int rows, cols;       // valid rows (A side; features) and columns (B side; tokens) of the result
  int m_tiles, n_tiles; // tiles of 256 rows (gate/up: 128 features) and n columns
  int n;                // columns of a tile: the MMA's N, a multiple of 32
  int nkb, slice_kb;    // K steps of 64, and how many make a slice
  void *out;
  int64_t ldo;
  const __nv_bfloat16 *addend;  // kStore
  int64_t ld_add;
  float *gu;            // kGateUp: written (may be null); kDact: read
  int wgrad;            // kGrads: a weight gradient (B is MN-major too), else dx
  int mode;             // a weight gradient's GradMode
};

// The problems of a launch and the tile numbers at which they begin.
template <int N>
struct FfnBatch {
  FfnGemm g[N];
  int first[N + 1];
  int *err;
};
template <int N>
struct FfnMaps {
  CUtensorMap a[N], b[N];
};

// The two projections' gradients from dact = d: one fixed fp32 sequence.
struct GateGrads {
  float dg, du;
};
__device__ __forceinline__ GateGrads gate_grads(float d, float g, float u) {
  const float s = sigmoid_approx(g), ds = __fmul_rn(d, s);
  return {__fmul_rn(__fmul_rn(ds, u), __fmaf_rn(g, __fsub_rn(1.0f, s), 1.0f)), __fmul_rn(ds, g)};
}

// 32 bytes to global memory: a whole sector per lane.
__device__ __forceinline__ void store_32b(void *p, const uint32_t (&v)[8], bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
  } else {
    uint4 *q = static_cast<uint4 *>(p);
    q[0] = make_uint4(v[0], v[1], v[2], v[3]);
    q[1] = make_uint4(v[4], v[5], v[6], v[7]);
  }
}

// Staging buffer of an epilogue warp: 16 tokens x 32 features, fp32 rows 144
// bytes apart (or bf16 ones, kStagePitch).
constexpr int kFPitch = 144;
constexpr int kFStaging = 16 * kFPitch;

// 16 tokens x 32 features of an fp32 matrix, rows 2I apart: 16-byte loads (lane:
// token lane / 8 and every 4th further, features 4 (lane % 8) ..).
__device__ __forceinline__ void load_rows_f32(const float *p, int64_t ld, int t0, int tokens, int feats, int lane,
                                              float4 (&w)[4]) {
  const float *q = p + (lane & 7) * 4;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = t0 + i * 4 + (lane >> 3);
    // feats is a multiple of 16: a part is inside or outside
    w[i] = t < tokens && (lane & 7) * 4 < feats ? __ldcs(reinterpret_cast<const float4 *>(q + t * ld))
                                                : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  }
}
// Through the staging buffer to the accumulator's order (tmem_ld_16x16, both halves).
__device__ __forceinline__ void rows_to_frag(uint32_t stage, const float4 (&w)[4], int lane, float (&v)[2][8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm volatile("st.shared.v4.f32 [%0], {%1,%2,%3,%4};" ::"r"(
                     stage + static_cast<uint32_t>((i * 4 + (lane >> 3)) * kFPitch + (lane & 7) * 16)),
                 "f"(w[i].x), "f"(w[i].y), "f"(w[i].z), "f"(w[i].w)
                 : "memory");
  __syncwarp();
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int t = (lane & 3) * 2 + (j & 1) + (j >> 2) * 8, f = h * 16 + (lane >> 2) + ((j >> 1) & 1) * 8;
      asm volatile("ld.shared.f32 %0, [%1];"
                   : "=f"(v[h][j])
                   : "r"(stage + static_cast<uint32_t>(t * kFPitch + f * 4))
                   : "memory");
    }
  __syncwarp();
}

// Epilogue of one warp over tokens (not the weight gradients): acc[chunk][half]
// holds 16 columns from col0 + 16 chunk of 16 rows from row0 (+ 16).
template <FfnEpi EPI>
__device__ __forceinline__ void ffn_epilogue(const FfnGemm &p, const float (&acc)[8][2][8], int row0, int col0,
                                             int ncols, uint32_t stage, int lane) {
  const int limit = min(ncols, p.cols - col0);  // valid columns
  if (limit <= 0 || row0 >= p.rows) return;
  if constexpr (EPI == kGateUp) {
    // half 0: gate values of the warp's 16 features from row0, half 1: their up values
    const RowsOut act{static_cast<__nv_bfloat16 *>(p.out) + static_cast<int64_t>(col0) * p.ldo + row0, p.ldo, limit,
                      p.rows - row0, true};
    const int64_t two = 2 * static_cast<int64_t>(p.rows);
    // the projections as 16-byte parts: part lane % 8 of a token's 16 gate and 16 up values
    float *gu = p.gu ? p.gu + col0 * two + row0 + (lane & 3) * 4 + (lane & 4 ? p.rows : 0) : nullptr;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      if (c * 16 >= limit) break;
      float a[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) a[j] = silu_mul(acc[c][0][j], acc[c][1][j]);
      store_rows16(stage, a, c * 16, act, lane);
      if (gu) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int t = (lane & 3) * 2 + (j & 1) + (j >> 2) * 8, f = h * 16 + (lane >> 2) + ((j >> 1) & 1) * 8;
            asm volatile("st.shared.f32 [%0], %1;" ::"r"(stage + static_cast<uint32_t>(t * kFPitch + f * 4)),
                         "f"(acc[c][h][j])
                         : "memory");
          }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int t = i * 4 + (lane >> 3);
          float4 w;
          asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];"
                       : "=f"(w.x), "=f"(w.y), "=f"(w.z), "=f"(w.w)
                       : "r"(stage + static_cast<uint32_t>(t * kFPitch + (lane & 7) * 16))
                       : "memory");
          if (c * 16 + t < limit) __stcs(reinterpret_cast<float4 *>(gu + (c * 16 + t) * two), w);
        }
        __syncwarp();
      }
    }
  } else if constexpr (EPI == kStore) {
    const RowsOut out{static_cast<__nv_bfloat16 *>(p.out) + static_cast<int64_t>(col0) * p.ldo + row0, p.ldo, limit,
                      p.rows - row0, true};
    const RowsOut add{const_cast<__nv_bfloat16 *>(p.addend) + static_cast<int64_t>(col0) * p.ld_add + row0, p.ld_add,
                      limit, p.rows - row0, true};
    uint4 aw[2][2] = {};  // the addend of a chunk, loaded while the one before is stored
    if (p.addend) load_rows32(add, 0, lane, aw[0]);
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      if (c * 16 >= limit) break;
      if (p.addend && (c + 1) * 16 < limit) load_rows32(add, (c + 1) * 16, lane, aw[(c + 1) & 1]);
      uint32_t v[2][8];
#pragma unroll
      for (int j = 0; j < 16; ++j) v[j / 8][j % 8] = __float_as_uint(acc[c][j / 8][j % 8]);
      store_rows32(stage, v, c * 16, out, p.addend ? &add : nullptr, aw[c & 1], lane);
    }
  } else if constexpr (EPI == kDact) {
    const int64_t two = 2 * static_cast<int64_t>(p.rows);
    const int feats = p.rows - row0;
    __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(p.out) + col0 * two + row0;
    const RowsOut dg{o, two, limit, feats, true}, du{o + p.rows, two, limit, feats, true};
    const float *gu = p.gu + col0 * two + row0;
    // the next chunk's projections are loaded while this one's gradients are stored
    float4 gw[4], uw[4];
    load_rows_f32(gu, two, 0, limit, feats, lane, gw);
    load_rows_f32(gu + p.rows, two, 0, limit, feats, lane, uw);
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      if (c * 16 >= limit) break;
      float g[2][8], u[2][8];
      rows_to_frag(stage, gw, lane, g);
      rows_to_frag(stage, uw, lane, u);
      if ((c + 1) * 16 < limit) {
        load_rows_f32(gu, two, (c + 1) * 16, limit, feats, lane, gw);
        load_rows_f32(gu + p.rows, two, (c + 1) * 16, limit, feats, lane, uw);
      }
      uint32_t a[2][8], b[2][8];
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const int h = j / 8, i = j % 8;
        const GateGrads r = gate_grads(acc[c][h][i], g[h][i], u[h][i]);
        a[h][i] = __float_as_uint(r.dg);
        b[h][i] = __float_as_uint(r.du);
      }
      const uint4 none[2] = {};
      store_rows32(stage, a, c * 16, dg, nullptr, none, lane);
      store_rows32(stage, b, c * 16, du, nullptr, none, lane);
    }
  }
}

// Epilogue of one warp of a weight gradient: acc[c] = D[row, col0 + c], row = row0 + lane.
template <int COLS>
__device__ __forceinline__ void ffn_wgrad_epilogue(const FfnGemm &p, const float (&acc)[COLS], int row0, int col0,
                                                   int ncols, int lane) {
  const int limit = min(ncols, p.cols - col0), r = row0 + lane;
  if (r >= p.rows) return;
  const int64_t at = static_cast<int64_t>(r) * p.ldo + col0;
  const bool wide = (reinterpret_cast<uintptr_t>(p.out) & 31) == 0;
#pragma unroll
  for (int c = 0; c < COLS; c += 16) {  // result columns come in multiples of 16
    if (c >= limit) break;
    if (p.mode == kGradBf16) {
      uint32_t v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = pack_bf16(acc[c + 2 * j], acc[c + 2 * j + 1]);
      store_32b(static_cast<__nv_bfloat16 *>(p.out) + at + c, v, wide);
    } else {
#pragma unroll
      for (int h = 0; h < 16; h += 8) {
        float *o = static_cast<float *>(p.out) + at + c + h;
        uint32_t v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
          v[j] = __float_as_uint(p.mode == kGradF32Accumulate ? __fadd_rn(o[j], acc[c + h + j]) : acc[c + h + j]);
        store_32b(o, v, wide);
      }
    }
  }
}

template <FfnEpi EPI, bool A_MN>
__global__ void __launch_bounds__(kFThreads, 1)
    ffn_gemm_kernel(const __grid_constant__ FfnMaps<EPI == kGrads ? 3 : 1> maps,
                    const __grid_constant__ FfnBatch<EPI == kGrads ? 3 : 1> batch) {
  constexpr int kProblems = EPI == kGrads ? 3 : 1;
  const FfnGemm &one = batch.g[0];  // the only problem, where there is one
  extern __shared__ uint8_t smem_raw[];
  uint8_t *tiles = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
  uint64_t *full = reinterpret_cast<uint64_t *>(tiles + kFStages * kFStageBytes);
  uint64_t *empty = full + kFStages;
  uint64_t *tfull = empty + kFStages;  // [2]
  uint64_t *tempty = tfull + 2;        // [2]
  uint64_t *drain = tempty + 2;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int unit0 = static_cast<int>(cluster_id_x()), nunits = static_cast<int>(num_clusters_x());
  const int total = batch.first[kProblems];

  if (threadIdx.x == 0) {
    for (int s = 0; s < kFStages; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(smem_u32(&tfull[a]), 1);
      mbar_init(smem_u32(&tempty[a]), 16);  // the epilogue warps of both CTAs, on the even CTA's barrier
    }
    mbar_init(smem_u32(drain), 1);
    *abort_flag = 0;
    fence_barrier_init();
    for (int i = 0; i < kProblems; ++i) {
      if (i > 0 && batch.first[i + 1] == batch.first[i]) continue;
      tma_prefetch_desc(&maps.a[i]);
      tma_prefetch_desc(&maps.b[i]);
    }
  }
  if (warp == 2) {
    if (lane == 0) *tmem_slot = 0u;
    __syncwarp();
    tmem_alloc_pair(smem_u32(tmem_slot), 2 * kFAccCols);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  griddep_wait();
  // The dependent grid may start: its CTAs need an SM of their own (this one's
  // shared memory is full), so they set up on SMs that are or become idle (a
  // training step of 257 tokens, H=1040, I=720: 32.8 -> 29.2 us).  Not behind
  // dact with wide tiles, whose long epilogue gets slower with CTAs parked beside
  // it.  The backward pass over six (H, I) from (1024, 512) to (4096, 2048),
  // without and with the trigger: tiles of up to 64 columns (200 to 1000 tokens)
  // 0.1 to 1.3 us less with it (H=1024, I=512, 200 tokens 13.7, 13.1); wider ones
  // between 1.1 us less and 4 us more (H=1040, I=720, 2000 tokens 35.7, 34.6;
  // H=2048, I=2048, 2000 tokens 80.3, 82.7; H=4096, I=2048, 3500 216, 220).
  if (EPI != kDact || one.n <= 64) griddep_launch_dependents();

  auto wait = [&](uint32_t bar, uint32_t parity, volatile int *ab) { return mbar_wait_cl(bar, parity, ab, batch.err); };
  // A tile: its problem, first row and column (of the pair).
  // Columns fastest: the tiles of a row block follow one another and share its A in L2.
  struct Tile {
    int i, row, col;
  };
  auto tile_at = [&](int tile) {
    Tile t;
    t.i = kProblems > 1 ? (tile >= batch.first[1]) + (tile >= batch.first[2]) : 0;
    const FfnGemm &g = batch.g[t.i];
    const int local = tile - batch.first[t.i];
    t.row = local / g.n_tiles * (EPI == kGateUp ? kFM : 2 * kFM);
    t.col = local % g.n_tiles * g.n;
    return t;
  };

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFRegsFew));
    // The TMA and the MMA thread are alone in their warps: while other lanes
    // wait for it at a warp or block barrier, every branch of a single lane
    // takes some 70 cycles and a wait on an mbarrier 280 instead of 46
    // (four M=128 x N=16 MMAs with a wait: 288 cycles, alone 194).
    if (warp == 0) {
      // ---------------------------------------------------- TMA producer --
      if (elect_one()) {
        int stage = 0;
        uint32_t phase = 0, issued_mask = 0, issued_parity = 0;
        bool ok = true;
        for (int tile = unit0; tile < total && ok; tile += nunits) {
          const Tile ti = tile_at(tile);
          const CUtensorMap *tmA = &maps.a[ti.i], *tmB = &maps.b[ti.i];
          const bool b_mn = EPI == kGrads && batch.g[ti.i].wgrad != 0;
          const int half = batch.g[ti.i].n / 2;
          const uint32_t b_bytes =
              b_mn ? static_cast<uint32_t>((half + 63) / 64 * kFSlab) : static_cast<uint32_t>(half * kFK * 2);
          const int row = ti.row + static_cast<int>(rank) * (EPI == kGateUp ? kFM / 2 : kFM);
          const int col = ti.col + static_cast<int>(rank) * half;
          for (int kb = 0; kb < batch.g[ti.i].nkb; ++kb) {
            if (!wait(smem_u32(&empty[stage]), phase ^ 1u, abort_flag)) {
              ok = false;
              break;
            }
            const uint32_t st = smem_u32(tiles + stage * kFStageBytes);
            const uint32_t fb = mapa_shared(smem_u32(&full[stage]), 0);
            if (rank == 0) mbar_arrive_expect_tx(smem_u32(&full[stage]), 2 * (kFABytes + b_bytes));
            const int k = kb * kFK;
            if (EPI == kGateUp) {
              tma_load_4d_pair(st, tmA, fb, k, 0, 0, row / 16);
            } else if (A_MN) {
              tma_load_2d_pair(st, tmA, fb, row, k);
              tma_load_2d_pair(st + kFSlab, tmA, fb, row + 64, k);
            } else {
              tma_load_2d_pair(st, tmA, fb, k, row);
            }
            if (b_mn) {
              tma_load_2d_pair(st + kFABytes, tmB, fb, col, k);
              if (half > 64) tma_load_2d_pair(st + kFABytes + kFSlab, tmB, fb, col + 64, k);
            } else {
              tma_load_2d_pair(st + kFABytes, tmB, fb, k, col);
            }
            issued_mask |= 1u << stage;
            issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
            if (++stage == kFStages) {
              stage = 0;
              phase ^= 1u;
            }
          }
        }
        if (*abort_flag) {
          // every copy this CTA started lands before it exits
          if (rank == 0) {
            for (int s = 0; s < kFStages; ++s)
              if ((issued_mask >> s) & 1u) wait(smem_u32(&full[s]), (issued_parity >> s) & 1u, nullptr);
          }
          // the odd CTA's copies complete on the even CTA's barriers: give them time to land
          const unsigned long long t0 = globaltimer_ns();
          while (globaltimer_ns() - t0 < 200000ull) {
          }
        }
      } else {
        return;
      }
    } else if (warp == 1) {
      // ------------------------------------------------------ MMA issuer --
      if (rank == 0 && elect_one()) {
        int stage = 0, buf = 0;
        uint32_t phase = 0, buf_phase = 0;
        bool ok = true;
        for (int tile = unit0; tile < total && ok && !*abort_flag; tile += nunits) {
          const Tile ti = tile_at(tile);
          const bool b_mn = EPI == kGrads && batch.g[ti.i].wgrad != 0;
          const uint32_t idesc =
              idesc_bf16_f32(2 * kFM, batch.g[ti.i].n) | (A_MN ? kIdescAMn : 0u) | (b_mn ? kIdescBMn : 0u);
          const int nkb = batch.g[ti.i].nkb, slice_kb = batch.g[ti.i].slice_kb;
          for (int kb0 = 0; kb0 < nkb && ok; kb0 += slice_kb) {
            const int kb1 = min(nkb, kb0 + slice_kb);
            if (!wait(smem_u32(&tempty[buf]), buf_phase ^ 1u, abort_flag)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t d = tmem_base + static_cast<uint32_t>(buf * kFAccCols);
            for (int kb = kb0; kb < kb1; ++kb) {
              if (!wait(smem_u32(&full[stage]), phase, abort_flag)) {
                ok = false;
                break;
              }
              tc_fence_after();
              const uint32_t a0 = smem_u32(tiles + stage * kFStageBytes), b0 = a0 + kFABytes;
#pragma unroll
              for (int k = 0; k < kFK / 16; ++k) {
                const uint64_t ad = A_MN ? sdesc_sw128_mn(a0 + k * 2048, kFSlab) : sdesc_sw128(a0 + k * 32);
                const uint64_t bd = b_mn ? sdesc_sw128_mn(b0 + k * 2048, kFSlab) : sdesc_sw128(b0 + k * 32);
                umma_f16_pair(d, ad, bd, idesc, (kb > kb0 || k) ? 1u : 0u);
              }
              umma_commit_pair(smem_u32(&empty[stage]), 0x3);
              if (++stage == kFStages) {
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
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kFRegsMany));
    // -------------------------------------------------------- epilogue --
    const int q = warp & 3, h = (warp - 4) >> 2;
    const uint32_t staging = smem_u32(tiles + kFStages * kFStageBytes + 256 + (warp - 4) * kFStaging);
    int buf = 0;
    uint32_t buf_phase = 0;
    bool ok = true;
    for (int tile = unit0; tile < total && ok; tile += nunits) {
      const Tile ti = tile_at(tile);
      const FfnGemm &prm = batch.g[ti.i];
      const bool wgrad = EPI == kGrads && prm.wgrad != 0;
      const int ncols = prm.n / 2;  // columns of this warp: half h of the tile
      // the sums of the slices, in the order that the epilogue wants them
      float acc[8][2][8];
#pragma unroll
      for (int c = 0; c < 128; ++c) acc[c / 16][c / 8 % 2][c % 8] = 0.0f;
      for (int kb0 = 0; kb0 < prm.nkb; kb0 += prm.slice_kb) {
        ok = __all_sync(0xffffffffu, wait(smem_u32(&tfull[buf]), buf_phase, abort_flag) ? 1 : 0) != 0;
        if (!ok) break;
        tc_fence_after();
        const uint32_t t = tmem_base + (static_cast<uint32_t>(q * 32) << 16) +
                           static_cast<uint32_t>(buf * kFAccCols + h * ncols);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          if (c * 16 < ncols) {
            uint32_t d[2][8];
            if (wgrad) {
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
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster_relaxed(mapa_shared(smem_u32(&tempty[buf]), 0));
        if (++buf == 2) {
          buf = 0;
          buf_phase ^= 1u;
        }
      }
      if (!ok) break;
      const int row0 = ti.row + static_cast<int>(rank) * (EPI == kGateUp ? kFM / 2 : kFM) +
                       q * (EPI == kGateUp ? 16 : 32);
      const int col0 = ti.col + h * ncols;
      if constexpr (EPI == kGrads) {
        if (wgrad) {
          float flat[128];
#pragma unroll
          for (int c = 0; c < 128; ++c) flat[c] = acc[c / 16][c / 8 % 2][c % 8];
          ffn_wgrad_epilogue(prm, flat, row0, col0, ncols, lane);
        }
      }
      if (!wgrad) ffn_epilogue<EPI == kGrads ? kStore : EPI>(prm, acc, row0, col0, ncols, staging, lane);
    }
  }

  tc_fence_before();
  __syncthreads();
  // the even CTA's final commit: its last MMAs have left this CTA's memory too
  if (rank != 0 && threadIdx.x == 96) wait(smem_u32(drain), 0, nullptr);
  cluster_sync_rest();  // neither CTA leaves while the other may still signal its barriers
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, 2 * kFAccCols);
  }
}

// ------------------------------------------------- few tokens: split kernel --
//
// With few tokens the weights are the whole cost and the pair tiles above are
// too few to stream them.  Here every slice of a row tile has a CTA of its own:
// the CTAs of a cluster take one slice each (same K=16 chains into tensor
// memory), leave their partial tiles in shared memory and, after a cluster
// barrier, each adds its share of the elements through distributed shared
// memory in slice order from +0 -- the recipe of the pair kernel, so the bits
// are the same.  (Sending the partials instead, one 32-bit store each, took
// 5 us for 32 rows x 48 tokens; reading them takes 0.7 us.)
//   * A row tile is 128, 64 or 32 rows, so that there are more CTAs than SMs (two
//     fit on one); up to 64 rows the MMA is an M=64 one (24 cycles each at N=16
//     instead of 40).  Rows past the tile's read whatever shared memory holds,
//     in accumulator rows that nothing reads.
//   * A CTA keeps to half of an SM's shared memory, so that the down kernel's
//     CTAs start beside the gate/up ones and load W2 (which no kernel between
//     writes) while those still run.
//   * Weights and tokens have a TMA thread each: one thread takes some 300
//     cycles to arm a stage and issue both copies, longer than a K step's MMAs.
//     A stage is two K steps, so that the MMA thread waits half as often.
//
// Measured (weights not in L2): one token at H=4096, I=2048 14.8 us, of which the
// 50 MB of weights take 7.4 at the copy bandwidth, two kernels' first copies 2,
// their joins and stores 3, the boundary between them 1; 64 tokens 19.5 us.  At
// H=2048, I=768: 8.0 us for one token, 9.1 for 33 (latency).
constexpr int kPThreads = 224;      // weight TMA, MMA, token TMA, 4 epilogue warps
constexpr int kPMaxSlices = 8;      // CTAs of a cluster
constexpr int kPK = 2 * kFK;        // reduction step of a stage
constexpr int kPMaxStages = kSliceK / kPK;
constexpr int kPMaxN = 64;          // tokens per tile
constexpr int kPSmem = 112 * 1024;
constexpr int kPBatch = 4;          // elements that an epilogue thread handles at once

struct FfnSplit {
  FfnGemm g;
  int tile_rows;          // rows of A per tile
  int mma_rows;           // M of the MMA: 128, or 64 for tiles of up to 64 rows
  int stages, stage_bytes, b_off;
  int share;              // elements that a CTA of the cluster finishes
  int early;              // A may be read before the predecessor has finished
  int *err;
};

// What an element's epilogue reads besides its sums, loaded apart from its use.
struct Extra {
  float a, b;
};

template <FfnEpi EPI>
__device__ __forceinline__ Extra ffn_extra(const FfnGemm &p, int f, int t) {
  Extra x = {0.0f, 0.0f};
  if constexpr (EPI == kStore) {
    if (p.addend) x.a = __bfloat162float(p.addend[t * p.ld_add + f]);
  } else if constexpr (EPI == kDact) {
    const float *gu = p.gu + static_cast<int64_t>(t) * 2 * p.rows + f;
    x.a = gu[0];
    x.b = gu[p.rows];
  }
  return x;
}

// One finished element of the result: D[f, t] (gate/up: the gate value and `up`).
template <FfnEpi EPI>
__device__ __forceinline__ void ffn_store_one(const FfnGemm &p, int f, int t, float d, float up, Extra x) {
  if constexpr (EPI == kGateUp) {
    static_cast<__nv_bfloat16 *>(p.out)[t * p.ldo + f] = __float2bfloat16_rn(silu_mul(d, up));
    if (p.gu) {
      float *gu = p.gu + static_cast<int64_t>(t) * 2 * p.rows + f;
      gu[0] = d;
      gu[p.rows] = up;
    }
  } else if constexpr (EPI == kStore) {
    if (p.addend) d = __fadd_rn(d, x.a);
    static_cast<__nv_bfloat16 *>(p.out)[t * p.ldo + f] = __float2bfloat16_rn(d);
  } else {
    __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(p.out) + static_cast<int64_t>(t) * 2 * p.rows + f;
    const GateGrads r = gate_grads(d, x.a, x.b);
    o[0] = __float2bfloat16_rn(r.dg);
    o[p.rows] = __float2bfloat16_rn(r.du);
  }
}

template <FfnEpi EPI, bool A_MN>
__global__ void __launch_bounds__(kPThreads)
    ffn_split_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                     const __grid_constant__ FfnSplit sp) {
  constexpr int kHalves = EPI == kGateUp ? 2 : 1;  // accumulators of an element: gate and up, or one
  const FfnGemm &prm = sp.g;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *aux = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint64_t *full = reinterpret_cast<uint64_t *>(aux);
  uint64_t *empty = full + kPMaxStages;
  uint64_t *done = empty + kPMaxStages;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(done + 1);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  uint8_t *tiles = aux + 1024;
  float *part = reinterpret_cast<float *>(tiles);  // [token][tile_rows], over the stages once the MMAs are done

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int slices = (prm.nkb + prm.slice_kb - 1) / prm.slice_kb;
  const int rank = static_cast<int>(cluster_ctarank());
  const int row = static_cast<int>(blockIdx.x) / slices * sp.tile_rows;  // first row of A (interleaved rows)
  const int col = static_cast<int>(blockIdx.y) * prm.n;
  const int k0 = rank * kSliceK;
  const int steps = (min(prm.nkb - rank * prm.slice_kb, prm.slice_kb) + 1) / 2;  // stages of this slice
  const uint32_t full0 = smem_u32(full), empty0 = smem_u32(empty), tiles0 = smem_u32(tiles);
  const uint32_t tmem_cols = prm.n <= 32 ? 32 : 64;

  if (threadIdx.x == 0) {
    for (int s = 0; s < sp.stages; ++s) {
      mbar_init(full0 + s * 8, 1);
      mbar_init(empty0 + s * 8, 1);
    }
    mbar_init(smem_u32(done), 1);
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
  }
  if (warp == 3) {
    tmem_alloc(smem_u32(tmem_slot), tmem_cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  // Elements of the tile, features fastest; this CTA finishes `share` of them,
  // this thread every 128th from `first` (the TMA and MMA threads none), in
  // batches whose loads are in flight together.
  const int feats_log = 31 - __clz(sp.tile_rows / kHalves), feats = 1 << feats_log;
  const int f0 = row / kHalves, ncols = min(prm.n, prm.cols - col);
  const int end = min((rank + 1) * sp.share, feats * ncols);
  const int first = warp >= 3 ? rank * sp.share + static_cast<int>(threadIdx.x) - 96 : end;
  auto valid = [&](int e) { return e < end && f0 + (e & (feats - 1)) < prm.rows; };
  auto extra_of = [&](int e) { return ffn_extra<EPI>(prm, f0 + (e & (feats - 1)), col + (e >> feats_log)); };
  // an element's place in the partial tile (gate/up: its gate row's; the up row is 16 further)
  auto place = [&](int e) {
    const int f = e & (feats - 1);
    return (e >> feats_log) * sp.tile_rows + (EPI == kGateUp ? f / 16 * 32 + f % 16 : f);
  };
  Extra extra[kPBatch];  // of the first batch

  if (warp == 0) {
    // ----------------------------------------------------- weight copies --
    if (elect_one()) {
      if (!sp.early) griddep_wait();
      const uint32_t bytes = static_cast<uint32_t>((sp.tile_rows + prm.n) * kPK * 2);  // with the tokens'
      const uint32_t sub = static_cast<uint32_t>(sp.tile_rows * kFK * 2);  // a K step's rows
      int s = 0, i = 0;
      uint32_t phase = 1;
      for (; i < steps; ++i) {
        if (i >= sp.stages && !mbar_wait(empty0 + s * 8, phase, abort_flag, sp.err)) break;
        const uint32_t st = tiles0 + static_cast<uint32_t>(s * sp.stage_bytes), fb = full0 + s * 8;
        mbar_arrive_expect_tx(fb, bytes);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int k = k0 + i * kPK + h * kFK;
          if (EPI == kGateUp) {
            tma_load_4d(st + h * sub, &tmA, fb, k, 0, 0, row / 32);
          } else if (A_MN) {
            tma_load_2d(st + h * sub, &tmA, fb, row, k);
            if (sp.tile_rows > 64) tma_load_2d(st + h * sub + kFSlab, &tmA, fb, row + 64, k);
          } else {
            tma_load_2d(st + h * sub, &tmA, fb, k, row);
          }
        }
        if (++s == sp.stages) {
          s = 0;
          phase ^= 1u;
        }
      }
      if (*abort_flag) {  // every copy this CTA started lands before it exits
        for (int j = max(0, i - sp.stages); j < i; ++j)
          mbar_wait(full0 + j % sp.stages * 8, j / sp.stages & 1, nullptr, sp.err);
      }
      if (sp.early) griddep_wait();
    } else {
      return;  // see the pair kernel: a thread alone in its warp
    }
  } else if (warp == 1) {
    // ------------------------------------------------------- MMA issuer --
    if (elect_one()) {
      const uint32_t idesc = idesc_bf16_f32(sp.mma_rows, prm.n) | (A_MN ? kIdescAMn : 0u);
      // Descriptors advance by additions to their address field (16-byte units).
      const uint64_t a_first = A_MN ? sdesc_sw128_mn(tiles0, kFSlab) : sdesc_sw128(tiles0);
      const uint64_t b_first = sdesc_sw128(tiles0 + sp.b_off);
      const uint32_t a_sub = static_cast<uint32_t>(sp.tile_rows * kFK * 2) / 16;
      const uint32_t b_sub = static_cast<uint32_t>(prm.n * kFK * 2) / 16;
      uint32_t at = 0, stage = 0, phase = 0;
      for (int i = 0; i < steps; ++i) {
        if (!mbar_wait(full0 + stage * 8, phase, abort_flag, sp.err)) break;
        tc_fence_after();
#pragma unroll
        for (int k = 0; k < kPK / 16; ++k)
          umma_f16(tmem_base, a_first + (at + k / 4 * a_sub + k % 4 * (A_MN ? 2048 : 32) / 16),
                   b_first + (at + k / 4 * b_sub + k % 4 * 2), idesc, (i | k) ? 1u : 0u);
        umma_commit(empty0 + stage * 8);
        at += static_cast<uint32_t>(sp.stage_bytes) / 16;
        if (++stage == static_cast<uint32_t>(sp.stages)) {
          stage = 0;
          phase ^= 1u;
          at = 0;
        }
      }
      umma_commit(smem_u32(done));
      // Only this thread polls for the accumulator; the rest of the CTA sleeps
      // at the block barrier below.  After an abort the MMAs that were issued
      // still complete.
      if (!mbar_wait(smem_u32(done), 0, nullptr, sp.err)) *abort_flag = 1;
      tc_fence_before();
      griddep_wait();
    } else {
      return;
    }
  } else if (warp == 2) {
    // ------------------------------------------------------ token copies --
    if (elect_one()) {
      griddep_wait();
      int s = 0;
      uint32_t phase = 1;
      for (int i = 0; i < steps; ++i) {
        if (i >= sp.stages && !mbar_wait(empty0 + s * 8, phase, abort_flag, sp.err)) break;
        const uint32_t st = tiles0 + static_cast<uint32_t>(s * sp.stage_bytes + sp.b_off);
        tma_load_2d(st, &tmB, full0 + s * 8, k0 + i * kPK, col);
        tma_load_2d(st + static_cast<uint32_t>(prm.n * kFK * 2), &tmB, full0 + s * 8, k0 + i * kPK + kFK, col);
        if (++s == sp.stages) {
          s = 0;
          phase ^= 1u;
        }
      }
    } else {
      return;
    }
  } else {
    griddep_wait();
#pragma unroll
    for (int u = 0; u < kPBatch; ++u)
      if (valid(first + u * 128)) extra[u] = extra_of(first + u * 128);
  }
  // the dependent kernel may start: everything before this one has finished
  griddep_launch_dependents();
  // ---------------------------------------------------------- epilogue --
  __syncthreads();
  const bool ok = *abort_flag == 0;
  tc_fence_after();
  if (warp >= 3 && ok) {
    // this warp's accumulator rows: 32, or 16 of an M=64 MMA (on lanes 0-15)
    const int q = warp & 3, per_warp = sp.mma_rows / 4;
    if (q * per_warp < sp.tile_rows) {
      const uint32_t t = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
      float *to = part + q * per_warp + lane;
      for (int c = 0; c < ncols; c += 16) {
        uint32_t d[16];
        tmem_ld16(t + c, d);
        tmem_ld_wait();
        if (lane < per_warp) {
#pragma unroll
          for (int j = 0; j < 16; ++j) to[(c + j) * sp.tile_rows] = __uint_as_float(d[j]);
        }
      }
    }
  }
  tc_fence_before();
  if (slices > 1) cluster_sync_rest();
  else __syncthreads();
  if (warp == 3) {
    tc_fence_after();
    tmem_dealloc(tmem_base, tmem_cols);
  }
  if (slices > 1) {
    // this CTA's share: sums into its own partial tile, in whose share no other CTA reads
    for (int e0 = first; ok && e0 < end; e0 += kPBatch * 128) {
      float v[kPBatch][kPMaxSlices], w[kPBatch][kPMaxSlices];
#pragma unroll
      for (int s = 0; s < kPMaxSlices; ++s) {
        if (s >= slices) break;
        const uint32_t tile = mapa_shared(smem_u32(part), s);
#pragma unroll
        for (int u = 0; u < kPBatch; ++u) {
          if (e0 + u * 128 >= end) break;
          const uint32_t at = tile + static_cast<uint32_t>(place(e0 + u * 128)) * 4;
          v[u][s] = ld_cluster_f32(at);
          if (EPI == kGateUp) w[u][s] = ld_cluster_f32(at + 64);
        }
      }
#pragma unroll
      for (int u = 0; u < kPBatch; ++u) {
        if (e0 + u * 128 >= end) break;
        float d = 0.0f, up = 0.0f;
#pragma unroll
        for (int s = 0; s < kPMaxSlices; ++s) {
          if (s >= slices) break;
          d = __fadd_rn(d, v[u][s]);
          if (EPI == kGateUp) up = __fadd_rn(up, w[u][s]);
        }
        float *to = part + place(e0 + u * 128);
        to[0] = d;
        if (EPI == kGateUp) to[16] = up;
      }
    }
    cluster_arrive();  // done with the others' tiles; the stores below overlap the barrier
  }
  for (int e0 = first; ok && e0 < end; e0 += kPBatch * 128) {
    if (e0 != first) {
#pragma unroll
      for (int u = 0; u < kPBatch; ++u)
        if (valid(e0 + u * 128)) extra[u] = extra_of(e0 + u * 128);
    }
#pragma unroll
    for (int u = 0; u < kPBatch; ++u) {
      const int e = e0 + u * 128;
      const float *v = part + place(e);
      if (valid(e))
        ffn_store_one<EPI>(prm, f0 + (e & (feats - 1)), col + (e >> feats_log), __fadd_rn(0.0f, v[0]),
                           EPI == kGateUp ? __fadd_rn(0.0f, v[16]) : 0.0f, extra[u]);
    }
  }
  if (slices > 1) cluster_wait();  // no CTA leaves while another reads its partials
}

// ------------------------------------------------------------------- host --
template <FfnEpi EPI, bool A_MN, int N>
static bi_status launch_ffn(const FfnMaps<N> &maps, FfnBatch<N> p, cudaStream_t s) {
  static std::mutex mu;
  static int max_units[64] = {};  // CTA pairs resident at once, per device
  static ContextSetup setup;      // the shared-memory attribute is per context
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64) {
    set_error("device ordinal %d out of range", dev);
    return BI_ERR_CUDA;
  }
  auto kern = ffn_gemm_kernel<EPI, A_MN>;
  {
    std::lock_guard<std::mutex> lk(mu);
    if (max_units[dev] == 0 || setup.pending(dev)) {
      cudaLaunchConfig_t cfg = {};
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = 2;
      attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
      cfg.gridDim = dim3(2 * (num_sms() / 2));
      cfg.blockDim = dim3(kFThreads);
      cfg.dynamicSmemBytes = kFSmem;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      int clusters = 0;
      cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kFSmem);
      if (e == cudaSuccess) e = cudaOccupancyMaxActiveClusters(&clusters, kern, &cfg);
      if (e != cudaSuccess || clusters <= 0) {
        cudaGetLastError();
        set_error("feed-forward kernel set-up: %s (%d clusters)", cudaGetErrorString(e), clusters);
        return BI_ERR_CUDA;
      }
      max_units[dev] = clusters;
      setup.done(dev);
    }
  }
  p.err = device_error_word();
  int64_t tiles = 0;
  p.first[0] = 0;
  for (int i = 0; i < N; ++i) {
    tiles += static_cast<int64_t>(p.g[i].m_tiles) * p.g[i].n_tiles;
    if (tiles > (int64_t(1) << 30)) {
      set_error("feed-forward product with more than 2^30 tiles");
      return BI_ERR_UNSUPPORTED;
    }
    p.first[i + 1] = static_cast<int>(tiles);
  }
  const int units = static_cast<int>(std::min<int64_t>(max_units[dev], tiles));
  return launch_chained(kern, dim3(2 * units), dim3(kFThreads), kFSmem, s, 2, maps, p);
}

static int div_up(int64_t a, int64_t b) { return static_cast<int>((a + b - 1) / b); }

// What a tile of n columns costs a CTA pair, in MMA columns per K step (256
// columns take 512 cycles): its MMAs or its copies, whichever is longer (an SM
// takes 64 bytes a cycle: 16 KB of A and 64 n bytes of B per K step), and a
// constant for the tile.
static int64_t tile_cost(int n, int nkb) { return static_cast<int64_t>(nkb) * std::max(n, 128 + n / 2) + 2000; }

// rows x cols result, reduction length K in slices of `slice`; n columns a tile.
static FfnGemm problem(int64_t rows, int64_t cols, int64_t K, int64_t slice, int tile_rows, int n) {
  FfnGemm p{};
  p.rows = static_cast<int>(rows);
  p.cols = static_cast<int>(cols);
  p.m_tiles = div_up(rows, tile_rows);
  p.n = n;
  p.n_tiles = div_up(cols, n);
  p.nkb = div_up(K, kFK);
  p.slice_kb = std::max(1, static_cast<int>(slice / kFK));
  return p;
}

// The same with the columns a tile (a multiple of 32 up to 256) whose waves over
// the CTA pairs take the least time by tile_cost.  n_step 128 for an MN-major B:
// only whole slabs per CTA, as a part of a slab costs a whole one's copy (dW2 of
// 8191 tokens, H=4096, I=2048: 104 us with 160 columns, 85 us with 256).
static FfnGemm plan(int64_t rows, int64_t cols, int64_t K, int64_t slice, int tile_rows, int n_step) {
  const int64_t pairs = std::max(1, num_sms() / 2);
  int64_t best = INT64_MAX;
  FfnGemm p{};
  for (int n = 256; n >= n_step; n -= n_step) {
    const FfnGemm q = problem(rows, cols, K, slice, tile_rows, n);
    const int64_t cost = (static_cast<int64_t>(q.m_tiles) * q.n_tiles + pairs - 1) / pairs * tile_cost(n, q.nkb);
    if (cost < best) {
      best = cost;
      p = q;
    }
  }
  return p;
}

// 0: automatic, 1: always the pair kernel, 2: the split kernel wherever the
// reduction has at most kPMaxSlices slices.
static std::atomic<int> g_ffn_schedule{0};

int set_ffn_schedule(int mode) { return g_ffn_schedule.exchange(mode); }

static int slices_of(int64_t K) { return static_cast<int>(std::min<int64_t>((K + kSliceK - 1) / kSliceK, 1 << 20)); }

// Whether a product of `rows` result rows, reduction K and M tokens goes to the
// split kernel; `limit` is the number of tokens up to which it is the faster
// one, by the reduction's slices (which it runs side by side, a pair one after
// another) and by the product:
//   gate/up and down  32 a slice of the longer reduction, as they go together
//                     (forward, split and pairs in us: H=512, I=256 32 tokens
//                     6.0, 7.6 and 64 8.4, 7.7; H=2048, I=768 64 tokens 10.4,
//                     11.9 and 96 12.5, 12.0; H=4096, I=1024 128 tokens 16.9, 21.8)
//   dact              32 up to two slices, then 32 a slice (with the weight
//                     gradients: H=2048, I=768 32 tokens 12.8, 14.1 and 64 16.3,
//                     14.8; H=2560, I=1024 96 tokens 20.9, 21.2; H=4096, I=2048
//                     128 tokens 32.6, 37.4)
//   dx                32 for each slice past the third: beside the weight
//                     gradients, in their launch, it costs pairs little (what it
//                     adds to the backward: H=4096, I=1024 one token 8.1, 5.2;
//                     H=4096, I=2048 32 tokens 11.9, 15.1 and 64 14.3, 14.2)
// and in one wave of two CTAs an SM, up to 32 tokens in two (forward, H=8192,
// I=4096, two waves: one token 37.7, 46.0, 32 tokens 44.9, 48.2, 64 tokens 52.7,
// 49.2; H=8192, I=2048, 80 tokens in two tiles, two waves: 44.7, 38.7; H=4096,
// I=14336, three waves: one token 85.0, 83.0, 32 tokens 97.1, 86.2), for the
// forward's two products together.
constexpr int64_t kSplitMaxM = 128;

static bool split_fits(int64_t M, int64_t rows, int64_t K) {
  return slices_of(K) <= kPMaxSlices &&
         (rows + kFM - 1) / kFM * slices_of(K) * ((M + kPMaxN - 1) / kPMaxN) <= (M <= 32 ? 4 : 2) * num_sms();
}
static bool use_split(int64_t M, int64_t rows, int64_t K, int64_t limit) {
  const int mode = g_ffn_schedule.load();
  if (mode == 2) return slices_of(K) <= kPMaxSlices;
  return mode == 0 && M <= std::min(limit, kSplitMaxM) && split_fits(M, rows, K);
}
static int64_t forward_limit(int64_t M, int64_t H, int64_t I) {
  return split_fits(M, 2 * I, H) && split_fits(M, H, I) ? 32 * std::max(slices_of(H), slices_of(I)) : 0;
}
static bool split_gate_up(int64_t M, int64_t H, int64_t I) { return use_split(M, 2 * I, H, forward_limit(M, H, I)); }
static bool split_down(int64_t M, int64_t H, int64_t I) { return use_split(M, H, I, forward_limit(M, H, I)); }
static bool split_dact(int64_t M, int64_t H, int64_t I) {
  return use_split(M, I, H, slices_of(H) <= 2 ? 32 : 32 * slices_of(H));
}
static bool split_dx(int64_t M, int64_t H, int64_t I) { return use_split(M, H, 2 * I, 32 * (slices_of(2 * I) - 3)); }

// The split kernel over `rows` rows of A (gate/up: 2I interleaved ones) and M
// tokens.  map_a encodes A's tensor map for a given tile height.
template <FfnEpi EPI, bool A_MN, typename MapA>
static bi_status launch_split(FfnGemm g, int64_t rows, int64_t M, int64_t K, bool early, MapA map_a,
                              const void *tokens, int64_t ld_tokens, cudaStream_t s) {
  FfnSplit p{};
  g.nkb = div_up(K, kFK);
  g.slice_kb = kSliceK / kFK;
  g.cols = static_cast<int>(M);
  g.n = static_cast<int>(std::min<int64_t>(kPMaxN, (M + 15) / 16 * 16));
  p.g = g;
  p.err = device_error_word();
  const int slices = div_up(K, kSliceK), token_tiles = div_up(M, g.n);
  // the tallest tiles that still give three CTAs to two SMs, but not more than two
  // to one.  Against tiles of 128 rows everywhere, the forward over seven (H, I)
  // from (1024, 512) to (5120, 1408): one token 0 to 1.6 us less (H=4096, I=2048
  // 15.7, 14.9), 16 tokens 1.8 to 3.1 (H=2048, I=2048 14.6, 11.5), 48 tokens 0 to
  // 8.4 (22.3, 13.9), 96 tokens 0 to 7 (H=4096, I=1024 23.3, 16.3); as low as two
  // to one allows them everywhere: level.
  p.tile_rows = kFM;
  const auto ctas = [&](int tile) { return static_cast<int64_t>(div_up(rows, tile)) * slices * token_tiles; };
  while (p.tile_rows > (A_MN ? 64 : 32) && ctas(p.tile_rows) * 2 < num_sms() * 3 &&
         ctas(p.tile_rows / 2) <= num_sms() * 2)
    p.tile_rows /= 2;
  p.mma_rows = p.tile_rows > 64 ? 128 : 64;
  p.b_off = p.tile_rows * kPK * 2;
  p.stage_bytes = p.b_off + g.n * kPK * 2;
  p.share = div_up(p.tile_rows / (EPI == kGateUp ? 2 : 1) * g.n, slices * 32) * 32;
  p.early = early;
  // the MMA reads mma_rows rows from every K step's start, for a lower tile past its end
  const int pad = (p.mma_rows - p.tile_rows) * kFK * 2;
  p.stages = std::min({kPMaxStages, div_up(g.nkb, 2), (kPSmem - 2048 - pad) / p.stage_bytes});
  const int smem = 2048 + std::max(p.stages * p.stage_bytes + pad, g.n * p.tile_rows * 4);
  if (token_tiles > 65535) {
    set_error("feed-forward product with %d token tiles", token_tiles);
    return BI_ERR_UNSUPPORTED;
  }
  static std::mutex mu;
  static ContextSetup setup;  // the shared-memory attribute is per context
  int dev = 0;
  cudaGetDevice(&dev);
  auto kern = ffn_split_kernel<EPI, A_MN>;
  {
    std::lock_guard<std::mutex> lk(mu);
    if (setup.pending(dev)) {
      const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kPSmem);
      if (e != cudaSuccess) {
        cudaGetLastError();
        set_error("cudaFuncSetAttribute: %s", cudaGetErrorString(e));
        return BI_ERR_CUDA;
      }
      setup.done(dev);
    }
  }
  CUtensorMap a, b;
  if (!map_a(&a, p.tile_rows) || !make_tma_2d_bf16_ld(&b, tokens, M, K, ld_tokens, g.n)) return BI_ERR_CUDA;
  return launch_chained(kern, dim3(div_up(rows, p.tile_rows) * slices, token_tiles), dim3(kPThreads), smem, s, slices,
                        a, b, p);
}

bi_status launch_ffn_gate_up(Mat x, const __nv_bfloat16 *w13, __nv_bfloat16 *act, float *gu, int64_t M, int64_t H,
                             int64_t I, cudaStream_t s) {
  FfnGemm p = plan(I, M, H, kSliceK, kFM, 32);
  p.out = act;
  p.ldo = I;
  p.gu = gu;
  if (split_gate_up(M, H, I))
    return launch_split<kGateUp, false>(
        p, 2 * I, M, H, false,
        [&](CUtensorMap *a, int r) { return make_tma_inter_bf16(a, w13, I, I, H, r / 32); }, x.p, x.ld, s);
  FfnMaps<1> m;
  if (!make_tma_inter_bf16(m.a, w13, I, I, H) || !make_tma_2d_bf16_ld(m.b, x.p, M, H, x.ld, p.n / 2))
    return BI_ERR_CUDA;
  return launch_ffn<kGateUp, false>(m, FfnBatch<1>{{p}, {}, nullptr}, s);
}

bi_status launch_ffn_down(const __nv_bfloat16 *act, const __nv_bfloat16 *w2, Mat addend, __nv_bfloat16 *out,
                          int64_t ldo, int64_t M, int64_t H, int64_t I, cudaStream_t s) {
  FfnGemm p = plan(H, M, I, kSliceK, 2 * kFM, 32);
  p.out = out;
  p.ldo = ldo;
  p.addend = addend.p;
  p.ld_add = addend.ld;
  if (split_down(M, H, I))  // launched behind launch_ffn_gate_up, which writes no weights: W2 may be read early
    return launch_split<kStore, false>(
        p, H, M, I, true, [&](CUtensorMap *a, int r) { return make_tma_2d_bf16(a, w2, H, I, r); }, act, I, s);
  FfnMaps<1> m;
  if (!make_tma_2d_bf16(m.a, w2, H, I, kFM) || !make_tma_2d_bf16(m.b, act, M, I, p.n / 2)) return BI_ERR_CUDA;
  return launch_ffn<kStore, false>(m, FfnBatch<1>{{p}, {}, nullptr}, s);
}

bi_status launch_ffn_dact(Mat dout, const __nv_bfloat16 *w2, const float *gu, __nv_bfloat16 *dgu, int64_t M, int64_t H,
                          int64_t I, cudaStream_t s) {
  FfnGemm p = plan(I, M, H, kSliceK, 2 * kFM, 32);
  p.out = dgu;
  p.ldo = 2 * I;
  p.gu = const_cast<float *>(gu);
  if (split_dact(M, H, I))
    return launch_split<kDact, true>(
        p, I, M, H, false, [&](CUtensorMap *a, int) { return make_tma_2d_bf16(a, w2, H, I, kFK); }, dout.p, dout.ld, s);
  FfnMaps<1> m;
  if (!make_tma_2d_bf16(m.a, w2, H, I, kFK) || !make_tma_2d_bf16_ld(m.b, dout.p, M, H, dout.ld, p.n / 2))
    return BI_ERR_CUDA;
  return launch_ffn<kDact, true>(m, FfnBatch<1>{{p}, {}, nullptr}, s);
}

// dx alone, for few tokens (the split kernel).
static bi_status launch_dx_split(const FfnGrads &d, int64_t M, int64_t H, int64_t I, cudaStream_t s) {
  FfnGemm p = problem(H, M, 2 * I, kSliceK, 2 * kFM, 256);
  p.out = d.dx;
  p.ldo = d.lddx;
  return launch_split<kStore, true>(
      p, H, M, 2 * I, false, [&](CUtensorMap *a, int) { return make_tma_2d_bf16(a, d.w13, 2 * I, H, kFK); }, d.dgu,
      2 * I, s);
}

// The products that need no more than dgu: dW13, dW2 and dx, as asked for.  In
// one launch, longest tiles first: their tiles fill the CTA pairs together
// (4096 tokens, H=2048, I=768: 48 + 24 + 128 tiles on 76 pairs; the backward
// pass 65 us, with a launch each 91 us). 
// (Clusters of pairs sharing a weight-gradient tile's tokens, in a launch before dx,
// were slower in all but the smallest: 8191 tokens, H=I=512 53.3 us by two pairs,
// 53.9 in one launch; 4096 tokens 36.1, 32.3; 2048 tokens, H=512, I=256 22.5, 14.6.)
bi_status launch_ffn_grads(const FfnGrads &d, int64_t M, int64_t H, int64_t I, cudaStream_t s) {
  const int64_t pairs = std::max(1, num_sms() / 2);
  const int nkb = div_up(M, kFK);
  auto wgrad = [&](int64_t rows, int64_t cols, int n, void *out) {
    FfnGemm p = problem(rows, cols, M, kSliceK, 2 * kFM, n);
    p.out = out;
    p.ldo = cols;
    p.mode = d.grad_mode;
    p.wgrad = 1;
    return p;
  };
  auto tiles_of = [](const FfnGemm &p) { return static_cast<int64_t>(p.m_tiles) * p.n_tiles; };
  FfnGemm dx = plan(H, M, 2 * I, kSliceK, 2 * kFM, 32);
  dx.out = d.dx;
  dx.ldo = d.lddx;
  // The width of the weight gradients' tiles, as if all three were asked for, so
  // that a gradient's bits do not depend on that.
  const bool dx_fits = split_dx(M, H, I);  // dx by the split kernel
  int n_w = 256;
  int64_t best = INT64_MAX;
  for (int n = 256; n >= 128; n -= 128) {
    const int64_t t13 = tiles_of(wgrad(2 * I, H, n, nullptr)), t2 = tiles_of(wgrad(H, I, n, nullptr));
    const int64_t tdx = dx_fits ? 0 : tiles_of(dx), c_dx = tile_cost(dx.n, dx.nkb), c_w = tile_cost(n, nkb);
    // the work over the pairs, and half of the longest tile of imbalance
    const int64_t longest = std::max(c_w, tdx ? c_dx : 0);
    const int64_t cost = std::max((t13 + t2) * c_w + tdx * c_dx, longest * pairs) / pairs + longest / 2;
    if (cost <= best) best = cost, n_w = n;
  }
  const bool dx_split = d.dx && dx_fits;
  if (dx_split) {
    const bi_status st = launch_dx_split(d, M, H, I, s);
    if (st != BI_OK) return st;
  }
  const Mat dgu{d.dgu, 2 * I}, act{d.act, I};
  FfnBatch<3> b{};
  FfnMaps<3> m;
  int n = 0;
  bool ok = true;
  auto add = [&](const FfnGemm &p, Mat l, Mat r, uint64_t k_l, uint64_t k_r, uint64_t cols_l, uint64_t cols_r,
                 uint32_t box_r) {
    b.g[n] = p;
    ok = ok && make_tma_2d_bf16_ld(&m.a[n], l.p, k_l, cols_l, l.ld, kFK) &&
         make_tma_2d_bf16_ld(&m.b[n], r.p, k_r, cols_r, r.ld, box_r);
    ++n;
  };
  const bool with_dx = d.dx && !dx_split;
  const bool dx_first = with_dx && tile_cost(dx.n, dx.nkb) > tile_cost(n_w, nkb);
  auto add_dx = [&] { add(dx, Mat{d.w13, H}, dgu, 2 * I, M, H, 2 * I, dx.n / 2); };
  if (dx_first) add_dx();
  if (d.dw13) add(wgrad(2 * I, H, n_w, d.dw13), dgu, d.x, M, M, 2 * I, H, kFK);
  if (d.dw2) add(wgrad(H, I, n_w, d.dw2), d.dout, act, M, M, H, I, kFK);
  if (with_dx && !dx_first) add_dx();
  if (!ok) return BI_ERR_CUDA;
  if (n == 0) return BI_OK;
  for (int i = n; i < 3; ++i) m.a[i] = m.a[0], m.b[i] = m.b[0];  // (no tile uses them)
  return launch_ffn<kGrads, true>(m, b, s);
}

}  // namespace bimoe
