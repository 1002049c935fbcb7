// mx4_gemm.cu -- product of two matrices in the microscaled 4-bit form, plain
// or gated, on the block-scaled tensor-core path.
//
//   y = X W^T (+ addend),  or  act = silu(X Wg^T) * (X Wu^T)
//
// tcgen05.mma kind::mxf4 takes both operands as 4-bit codes and applies the
// scales itself, 64 k per MMA, summing in fp32.
//   * Weight rows are the MMA's rows, tokens its columns.  A stage is 256 k:
//     128-byte rows of codes by TMA (128-byte swizzle) and the scale tiles by
//     TMA, which tcgen05.cp spreads into tensor memory before the MMAs that use
//     them (cp and MMAs of one thread execute in order).
//   * One chain of MMAs over increasing k per output, whatever the tile: a
//     token's row has the same bits in every batch.
//   * Many tokens: CTA pairs (cta_group::2), 256 weight rows x up to 256 tokens,
//     each CTA staging its own rows of W and half of the tokens.  Few: one CTA
//     with 128 weight rows x up to 128 tokens (tiles of 64 or 32 rows, so that
//     more CTAs stream the weights, took the same time within 2 %).
//   * Two accumulators of 256 columns and the scales do not fit the 512 columns
//     of tensor memory: the second starts at column 224, and the epilogue drains
//     the 32 shared columns first and then lets the next tile's MMAs go.
//   * Eight epilogue warps, 32 rows x half of the columns each, take the tile to
//     registers before anything is stored.
//
// What bounds it, measured on a GB300.  An MMA of 128 rows x 256 columns x 64 k
// takes 128 cycles a CTA: 9.7 PFLOP/s at 1.95 GHz.  8192 x 8192 x 4096: 79.6 us,
// 6.9 PFLOP/s, a tile some 9900 cycles of which 8190 are MMAs (the rest: handing the
// accumulator over, about 1400, and waits for copies), 14 waves for 13.5; with
// K = 8192 7.6 PFLOP/s.  Gated 4096 x 4096 x 4096: 25.0 us, 5.5 PFLOP/s.  One CTA
// a tile of 192 tokens took 149 us for the first, pairs of 192 tokens, whose
// accumulators do not overlap, 89.6 (of 256 then 82.6; other sizes take 192, see
// the launch); blocks of 8 row tiles 84.9.  One token, 4096 x 2048: 3.8 us, latency
// (4.5 MB are 0.7 us of copying); gated 4096 x 4096 5.3 for one, 5.9 for 128.  An
// addend costs more than its bytes: 8192 x 4096 x 2048 32.6 us, with one 70.8.
#include <atomic>
#include <mutex>

#include "tile_epilogue.cuh"

namespace bimoe {

constexpr int kXThreads = 384;       // TMA and MMA warps (two idle), 8 epilogue warps
constexpr int kXRegsFew = 56, kXRegsMany = 224;  // 168 at launch: 128 x 56 + 256 x 224 = 384 x 168
constexpr int kXRows = 128;          // weight rows per CTA
constexpr int kXStageK = 256;        // values of k per stage
constexpr int kXABytes = kXRows * kXStageK / 2;
constexpr int scale_tiles(bool pair) { return pair ? 2 : 1; }  // scale tiles (128 tokens) that a token tile touches
constexpr int kXMaxStages = 12;
constexpr int kXAcc = 224;           // tensor-memory column of the second accumulator
constexpr int kXSfA = 480;           // scales of A: 4 columns per 128 k
constexpr int kXSfB = 488;           // scales of B: 8 columns (two row tiles) per 128 k
constexpr int kXSmem = 227 * 1024;

struct Mx4Gemm {
  int M, N;             // tokens, weight rows
  int nkb;              // stages of the reduction
  int n64;              // MMAs of the reduction
  int n;                // tokens per tile (the MMA's N)
  int m_tiles, n_tiles;
  int stages, stage_bytes;
  __nv_bfloat16 *y;
  int64_t ldy;
  const __nv_bfloat16 *addend;
  int64_t ld_add;
  int *err;
};

// Epilogue of one warp: 32 accumulator rows from row0, COLS/16 chunks of 16
// tokens from col0 (v[chunk][half of the rows], tmem_ld_16x16's order).
template <bool GATED, int CHUNKS>
__device__ __forceinline__ void mx4_epilogue(const Mx4Gemm &p, const uint32_t (&v)[CHUNKS][2][8], int row0, int col0,
                                             int ncols, uint32_t stage, int lane) {
  const int limit = min(ncols, p.M - col0);
  if (GATED) {
    // the first 16 rows are the gate values of 16 features, the others their up values
    const int f = row0 / 2;
    __nv_bfloat16 *y = p.y + static_cast<int64_t>(col0) * p.ldy + f;
    const RowsOut out{y, p.ldy, limit, p.N / 2 - f, rows_aligned(p.y, p.ldy)};
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c) {
      if (c * 16 >= limit) break;
      float act[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) act[j] = silu_mul(__uint_as_float(v[c][0][j]), __uint_as_float(v[c][1][j]));
      store_rows16(stage, act, c * 16, out, lane);
    }
  } else {
    const RowsOut out{p.y + static_cast<int64_t>(col0) * p.ldy + row0, p.ldy, limit, p.N - row0,
                      rows_aligned(p.y, p.ldy)};
    const RowsOut add{const_cast<__nv_bfloat16 *>(p.addend) + static_cast<int64_t>(col0) * p.ld_add + row0, p.ld_add,
                      limit, p.N - row0, rows_aligned(p.addend, p.ld_add)};
    uint4 aw[2][2] = {};  // the addend of a chunk, loaded while the one before is stored
    if (p.addend) load_rows32(add, 0, lane, aw[0]);
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c) {
      if (c * 16 >= limit) break;
      if (p.addend && (c + 1) * 16 < limit) load_rows32(add, (c + 1) * 16, lane, aw[(c + 1) & 1]);
      store_rows32(stage, v[c], c * 16, out, p.addend ? &add : nullptr, aw[c & 1], lane);
    }
  }
}

template <bool GATED, bool PAIR>
__global__ void __launch_bounds__(kXThreads, 1)
    mx4_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                    const __grid_constant__ CUtensorMap tmSA, const __grid_constant__ CUtensorMap tmSB,
                    const __grid_constant__ Mx4Gemm prm) {
  constexpr int kCols = PAIR ? 128 : 64;  // columns of an epilogue warp
  constexpr int kRows = PAIR ? 2 * kXRows : kXRows, kSfb = scale_tiles(PAIR);
  extern __shared__ uint8_t smem_raw[];
  uint8_t *aux = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint64_t *full = reinterpret_cast<uint64_t *>(aux);
  uint64_t *empty = full + kXMaxStages;
  uint64_t *tfull = empty + kXMaxStages;  // [2]
  uint64_t *tempty = tfull + 2;           // the columns that both accumulators use are drained
  uint64_t *drain = tempty + 1;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  uint8_t *tiles = aux + 1024;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int total = prm.m_tiles * prm.n_tiles;
  const uint32_t rank = PAIR ? cluster_ctarank() : 0u;
  const int unit0 = PAIR ? static_cast<int>(cluster_id_x()) : static_cast<int>(blockIdx.x);
  const int nunits = PAIR ? static_cast<int>(num_clusters_x()) : static_cast<int>(gridDim.x);
  const int b_rows = PAIR ? prm.n / 2 : prm.n;  // token rows that this CTA stages
  const int b_off = kXABytes, sfa_off = b_off + (b_rows * 128 + 1023) / 1024 * 1024, sfb_off = sfa_off + 1024;
  const uint32_t full0 = smem_u32(full), empty0 = smem_u32(empty), tfull0 = smem_u32(tfull), tempty0 = smem_u32(tempty),
                 tiles0 = smem_u32(tiles);

  if (threadIdx.x == 0) {
    for (int s = 0; s < prm.stages; ++s) {
      mbar_init(full0 + s * 8, 1);
      mbar_init(empty0 + s * 8, 1);
    }
    mbar_init(tfull0, 1);
    mbar_init(tfull0 + 8, 1);
    mbar_init(tempty0, PAIR ? 16 : 8);
    mbar_init(smem_u32(drain), 1);
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
    tma_prefetch_desc(&tmSA);
    tma_prefetch_desc(&tmSB);
  }
  if (warp == 2) {
    if (PAIR) {
      tmem_alloc_pair(smem_u32(tmem_slot), 512);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(smem_u32(tmem_slot), 512);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (PAIR) cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  griddep_wait();
  // the dependent grid may start: its CTAs need an SM of their own
  griddep_launch_dependents();

  auto wait = [&](uint32_t bar, uint32_t parity, volatile int *ab) {
    return PAIR ? mbar_wait_cl(bar, parity, ab, prm.err) : mbar_wait(bar, parity, ab, prm.err);
  };
  auto row_of = [&](int tile) { return tile / prm.n_tiles * kRows + static_cast<int>(rank) * kXRows; };
  auto col_of = [&](int tile) { return tile % prm.n_tiles * prm.n; };

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kXRegsFew));
    // the TMA and the MMA thread are alone in their warps: branches and barrier
    // waits of a lane that others wait for are several times slower
    if (warp == 0) {
      // -------------------------------------------------- TMA producer --
      if (elect_one()) {
        const uint32_t bytes =
            (PAIR ? 2u : 1u) * static_cast<uint32_t>((kXRows + b_rows) * 128 + (1 + kSfb) * 1024);
        uint32_t stage = 0, phase = 0, issued_mask = 0, issued_parity = 0;
        bool ok = true;
        for (int tile = unit0; tile < total && ok; tile += nunits) {
          const int row = row_of(tile), col = col_of(tile);
          for (int kb = 0; kb < prm.nkb; ++kb) {
            if (!wait(empty0 + stage * 8, phase ^ 1u, abort_flag)) {
              ok = false;
              break;
            }
            const uint32_t st = tiles0 + stage * static_cast<uint32_t>(prm.stage_bytes);
            if (PAIR) {
              // both CTAs' copies complete on the even CTA's barrier
              const uint32_t fb = mapa_shared(full0 + stage * 8, 0);
              if (rank == 0) mbar_arrive_expect_tx(full0 + stage * 8, bytes);
              tma_load_2d_pair(st, &tmA, fb, kb * 128, row);
              tma_load_2d_pair(st + b_off, &tmB, fb, kb * 128, col + static_cast<int>(rank) * b_rows);
              tma_load_2d_pair(st + sfa_off, &tmSA, fb, kb * 256, row / 128);
              tma_load_2d_pair(st + sfb_off, &tmSB, fb, kb * 256, col / 128);
            } else {
              const uint32_t fb = full0 + stage * 8;
              mbar_arrive_expect_tx(fb, bytes);
              tma_load_2d(st, &tmA, fb, kb * 128, row);
              tma_load_2d(st + b_off, &tmB, fb, kb * 128, col);
              tma_load_2d(st + sfa_off, &tmSA, fb, kb * 256, row / 128);
              tma_load_2d(st + sfb_off, &tmSB, fb, kb * 256, col / 128);
            }
            issued_mask |= 1u << stage;
            issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
            if (++stage == static_cast<uint32_t>(prm.stages)) {
              stage = 0;
              phase ^= 1u;
            }
          }
        }
        if (*abort_flag) {  // every copy this CTA started lands before it exits
          if (rank == 0) {
            for (int s = 0; s < prm.stages; ++s)
              if ((issued_mask >> s) & 1u) wait(full0 + s * 8, (issued_parity >> s) & 1u, nullptr);
          }
          if (PAIR) {
            // the odd CTA's copies complete on the even CTA's barriers: give them time to land
            const unsigned long long t0 = globaltimer_ns();
            while (globaltimer_ns() - t0 < 200000ull) {
            }
          }
        }
      } else {
        return;
      }
    } else if (warp == 1) {
      // ---------------------------------------------------- MMA issuer --
      if (rank == 0 && elect_one()) {
        const uint32_t idesc0 = idesc_mxf4(kRows, prm.n, 0), idesc1 = idesc_mxf4(kRows, prm.n, 1);
        const uint64_t a_first = sdesc_sw128(tiles0), b_first = sdesc_sw128(tiles0 + b_off);
        const uint64_t sa_first = sdesc_scales(tiles0 + sfa_off), sb_first = sdesc_scales(tiles0 + sfb_off);
        const uint32_t sfa = tmem_base + kXSfA, sfb0 = tmem_base + kXSfB;
        uint32_t stage = 0, phase = 0, at = 0, buf = 0, buf_phase = 0, drained = 0;
        bool ok = true, issued = false;
        for (int tile = unit0; tile < total && ok && !*abort_flag; tile += nunits) {
          // the last tile's columns that this accumulator shares are drained
          // (and so, long since, is the tile that used this accumulator)
          if (tile != unit0) {
            if (!wait(tempty0, drained, abort_flag)) break;
            drained ^= 1u;
          }
          tc_fence_after();
          const uint32_t d = tmem_base + buf * kXAcc;
          const uint32_t sfb = sfb0 + static_cast<uint32_t>(col_of(tile) % 128 / 32);  // the first tokens' column
          for (int kb = 0; kb < prm.nkb; ++kb) {
            if (!wait(full0 + stage * 8, phase, abort_flag)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const int mmas = min(4, prm.n64 - 4 * kb);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              if (PAIR) {
                tmem_copy_scales_pair(sfa + 4 * c, sa_first + (at + c * 32));
                tmem_copy_scales_pair(sfb0 + 8 * c, sb_first + (at + c * 32));
                tmem_copy_scales_pair(sfb0 + 8 * c + 4, sb_first + (at + 64 + c * 32));
              } else {
                tmem_copy_scales(sfa + 4 * c, sa_first + (at + c * 32));
                tmem_copy_scales(sfb0 + 8 * c, sb_first + (at + c * 32));
              }
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              if (k >= mmas) break;
              if (PAIR)
                umma_mxf4_pair(d, a_first + (at + k * 2), b_first + (at + k * 2), (k & 1) ? idesc1 : idesc0,
                               sfa + 4 * (k / 2), sfb + 8 * (k / 2), (kb | k) ? 1u : 0u);
              else
                umma_mxf4(d, a_first + (at + k * 2), b_first + (at + k * 2), (k & 1) ? idesc1 : idesc0,
                          sfa + 4 * (k / 2), sfb + 8 * (k / 2), (kb | k) ? 1u : 0u);
            }
            if (PAIR) umma_commit_pair(empty0 + stage * 8, 0x3);
            else umma_commit(empty0 + stage * 8);
            issued = true;
            at += static_cast<uint32_t>(prm.stage_bytes) / 16;
            if (++stage == static_cast<uint32_t>(prm.stages)) {
              stage = 0;
              phase ^= 1u;
              at = 0;
            }
          }
          if (!ok) break;
          if (PAIR) umma_commit_pair(tfull0 + buf * 8, 0x3);
          else umma_commit(tfull0 + buf * 8);
          buf ^= 1u;
          if (buf == 0) buf_phase ^= 1u;
        }
        if (PAIR || (*abort_flag && issued)) {
          // every MMA (pair: into both CTAs' tensor memory) has completed
          if (PAIR) umma_commit_pair(smem_u32(drain), 0x3);
          else umma_commit(smem_u32(drain));
          wait(smem_u32(drain), 0, nullptr);
        }
      } else {
        return;
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kXRegsMany));
    // -------------------------------------------------------- epilogue --
    const int q = warp & 3, h = (warp - 4) >> 2;
    // columns of this warp: half of the tile's (of 16 all for the first four warps)
    const int ncols = prm.n > 16 ? prm.n / 2 : (h == 0 ? prm.n : 0);
    const uint32_t staging = tiles0 + static_cast<uint32_t>(prm.stages * prm.stage_bytes + (warp - 4) * kStageBytes);
    uint32_t buf = 0, buf_phase = 0;
    for (int tile = unit0; tile < total; tile += nunits) {
      if (!__all_sync(0xffffffffu, wait(tfull0 + buf * 8, buf_phase, abort_flag) ? 1 : 0)) break;
      tc_fence_after();
      const uint32_t t = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + buf * kXAcc +
                         static_cast<uint32_t>(h * ncols);
      uint32_t v[kCols / 16][2][8];
      auto take = [&](int c) {  // chunk c of 16 columns
        tmem_ld_16x16(t + c * 16, v[c][0]);
        tmem_ld_16x16(t + (16u << 16) + c * 16, v[c][1]);
      };
      auto release = [&] {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (PAIR) mbar_arrive_cluster_relaxed(mapa_shared(tempty0, 0));
          else mbar_arrive_relaxed(tempty0);
        }
      };
      // first the columns that the other accumulator shares: the last 32 of the
      // first one, the first 32 of the second
      constexpr int kChunks = kCols / 16, kShared = (256 - kXAcc) / 16;
      if constexpr (PAIR) {
        if (buf == 0) {
#pragma unroll
          for (int c = kChunks - kShared; c < kChunks; ++c)
            if (c * 16 < ncols) take(c);
        } else {
#pragma unroll
          for (int c = 0; c < kShared; ++c)
            if (c * 16 < ncols) take(c);
        }
        tmem_ld_wait();
        release();
#pragma unroll
        for (int c = 0; c < kChunks; ++c)
          if (c * 16 < ncols && (buf == 0 ? c < kChunks - kShared : c >= kShared)) take(c);
      } else {
        // (up to 128 columns: nothing is shared, the other accumulator is free already)
        release();
#pragma unroll
        for (int c = 0; c < kChunks; ++c)
          if (c * 16 < ncols) take(c);
      }
      tmem_ld_wait();
      buf ^= 1u;
      if (buf == 0) buf_phase ^= 1u;
      if (ncols > 0)
        mx4_epilogue<GATED, kChunks>(prm, v, row_of(tile) + q * 32, col_of(tile) + h * ncols, ncols, staging, lane);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (PAIR) {
    // the even CTA's final commit: its last MMAs have left this CTA's memory too
    if (rank != 0 && threadIdx.x == 96) wait(smem_u32(drain), 0, nullptr);
    cluster_sync_rest();  // neither CTA leaves while the other may still signal its barriers
  }
  if (warp == 2) {
    tc_fence_after();
    if (PAIR) tmem_dealloc_pair(tmem_base, 512);
    else tmem_dealloc(tmem_base, 512);
  }
}

// ------------------------------------------------------------------- host --
template <bool GATED, bool PAIR>
static bi_status launch_mx4(const CUtensorMap (&maps)[4], const Mx4Gemm &p, cudaStream_t s) {
  static std::mutex mu;
  static int max_units[64] = {};  // CTAs or CTA pairs resident at once, per device
  static ContextSetup setup;      // the shared-memory attribute is per context
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64) {
    set_error("device ordinal %d out of range", dev);
    return BI_ERR_CUDA;
  }
  auto kern = mx4_gemm_kernel<GATED, PAIR>;
  {
    std::lock_guard<std::mutex> lk(mu);
    if (max_units[dev] == 0 || setup.pending(dev)) {
      int units = num_sms();
      cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kXSmem);
      if (e == cudaSuccess && PAIR) {
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 2;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.gridDim = dim3(2 * (num_sms() / 2));
        cfg.blockDim = dim3(kXThreads);
        cfg.dynamicSmemBytes = kXSmem;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        e = cudaOccupancyMaxActiveClusters(&units, kern, &cfg);
      }
      if (e != cudaSuccess || units <= 0) {
        cudaGetLastError();
        set_error("4-bit product set-up: %s (%d units)", cudaGetErrorString(e), units);
        return BI_ERR_CUDA;
      }
      max_units[dev] = units;
      setup.done(dev);
    }
  }
  const int64_t tiles = static_cast<int64_t>(p.m_tiles) * p.n_tiles;
  if (tiles > (int64_t(1) << 30)) {
    set_error("4-bit product with %lld tiles", (long long)tiles);
    return BI_ERR_UNSUPPORTED;
  }
  const int units = static_cast<int>(std::min<int64_t>(max_units[dev], tiles));
  const size_t smem = 2048 + static_cast<size_t>(p.stages) * p.stage_bytes + 8 * kStageBytes;
  return launch_chained(kern, dim3(PAIR ? 2 * units : units), dim3(kXThreads), smem, s, PAIR ? 2 : 1, maps[0], maps[1],
                        maps[2], maps[3], p);
}

static int div_up(int64_t a, int64_t b) { return static_cast<int>((a + b - 1) / b); }

// 0: the form of least estimated time; 1 to 3: always that row of kForms.
static std::atomic<int> g_mx4_form{0};

int set_mx4_form(int mode) { return g_mx4_form.exchange(mode); }

bi_status launch_mx4_gemm(const uint8_t *xq, const uint8_t *xs, const uint8_t *wq, const uint8_t *ws, Mat addend,
                          __nv_bfloat16 *y, int64_t ldy, bool gated, int64_t M, int64_t N, int64_t K, cudaStream_t s) {
  Mx4Gemm p{};
  p.M = static_cast<int>(M);
  p.N = static_cast<int>(N);
  p.nkb = div_up(K, kXStageK);
  p.n64 = div_up(K, 64);
  p.y = y;
  p.ldy = ldy;
  p.addend = addend.p;
  p.ld_add = addend.ld;
  p.err = device_error_word();
  // One CTA or a pair, and the tokens per tile: the least time by fits (10 ns) to
  // one to eight waves of N = 1024..32768, K = 1024..14336: a constant, and for
  // each wave a constant and the stages.  In one wave the single CTAs win (us,
  // single and pairs of 128: 4096 x 4096 gated, 256 tokens 6.5, 7.2; K = 14336,
  // 512 tokens 16.1, 16.8; N = 14336, one token 6.6, 9.0), past it larger tiles do
  // (8192 x 4096: 768 tokens 16.3 by single CTAs, 14.6 by pairs of 192; 1024
  // tokens 20.1, 18.4 and, by pairs of 256, 16.7).
  struct Form {
    bool pair;
    int n, once, wave, stage;
  };
  static constexpr Form kForms[] = {{false, 128, 400, 100, 18}, {true, 192, 620, 70, 20}, {true, 256, 620, 60, 28}};
  const int form = g_mx4_form.load();
  int64_t best = INT64_MAX;
  bool pair = false;
  for (const Form &f : kForms) {
    if (form != 0 && &f != &kForms[form - 1]) continue;
    const int64_t units = f.pair ? std::max(1, num_sms() / 2) : num_sms();
    const int64_t tiles = static_cast<int64_t>(div_up(N, f.pair ? 2 * kXRows : kXRows)) * div_up(M, f.n);
    const int64_t cost = f.once + (tiles + units - 1) / units * (f.wave + static_cast<int64_t>(f.stage) * p.nkb);
    if (cost < best) best = cost, pair = f.pair, p.n = f.n;
  }
  p.m_tiles = div_up(N, pair ? 2 * kXRows : kXRows);
  if (!pair) {
    // In one wave 64 tokens a tile if that leaves it one: what follows the last copy
    // is shorter (1001 x 2080, 100 tokens 6.7 us by a tile of 128, 5.4; 4096 x 2048,
    // 256 tokens 5.2, 4.3).  (Not 32: a tile begins at the tensor-memory column of its tokens'
    // scales, 32 tokens each, and an odd column is a misaligned address to the MMA.)
    if (static_cast<int64_t>(p.m_tiles) * div_up(M, 64) <= num_sms()) p.n = 64;
    // a single tile: no more than its tokens
    if (M <= p.n) p.n = M <= 16 ? 16 : div_up(M, 32) * 32;
  }
  p.n_tiles = div_up(M, p.n);
  const int b_rows = pair ? p.n / 2 : p.n;
  p.stage_bytes = kXABytes + div_up(b_rows * 128, 1024) * 1024 + 1024 + scale_tiles(pair) * 1024;
  p.stages = std::min(kXMaxStages, (kXSmem - 2048 - 8 * kStageBytes) / p.stage_bytes);
  CUtensorMap maps[4];
  const int64_t ktiles = div_up(K, 128);
  if (!make_tma_2d_u8(&maps[0], wq, N, K / 2, kXRows) ||
      !make_tma_2d_u8(&maps[1], xq, M, K / 2, b_rows) ||
      !make_tma_mx_scales(&maps[2], ws, div_up(N, 128), ktiles, 1) ||
      !make_tma_mx_scales(&maps[3], xs, div_up(M, 128), ktiles, scale_tiles(pair)))
    return BI_ERR_CUDA;
  if (pair) return gated ? launch_mx4<true, true>(maps, p, s) : launch_mx4<false, true>(maps, p, s);
  return gated ? launch_mx4<true, false>(maps, p, s) : launch_mx4<false, false>(maps, p, s);
}

}  // namespace bimoe
