// moe_grad.cu -- the row movements of the routed experts' backward pass and the
// gradient of the sigmoid top-k router.
//
// With s = x W^T (+ b), w = sigmoid(s) at a token's chosen experts and dw the
// gradient of those weights (the experts' backward pass gives it), the scores'
// gradient is c = dw w (1 - w) at the chosen experts and 0 elsewhere, so
//   dx[m] = sum over the slots of c W[id],
//   dW[e] = sum over the expert's tokens of c x[token],  db[e] = sum of c:
// sums over top_k rows of W and, grouped by expert, over the rows of x, instead
// of two products with a matrix of mostly zeros.
#include <mutex>

#include "train_internal.cuh"

namespace bimoe {

// Gradient of the score behind a sigmoid weight: one fixed fp32 sequence.
__device__ __forceinline__ float score_grad(float dw, float w) {
  return __fmul_rn(__fmul_rn(dw, w), __fsub_rn(1.0f, w));
}

// One warp per position; rows in 16-byte parts.  dwts (where given) is zeroed: the
// slots that are no pair of the grouping get no gradient later; and so are, with
// one slot a token, the result's rows of tokens without a valid one.
__global__ void __launch_bounds__(256) train_gather_kernel(const uint4 *__restrict__ rows, Groups g,
                                                           const int32_t *__restrict__ perm, int top_k, int row_vec,
                                                           uint4 *__restrict__ to, float *__restrict__ dwts, uint4 *zero,
                                                           const uint32_t *__restrict__ slots, int *err) {
  griddep_wait_small_release();
  const int p = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (p >= g.P) return;
  if (dwts && lane == 0) dwts[p] = 0.0f;
  if (zero && slots[p] == 0u)
    for (int c = lane; c < row_vec; c += 32) zero[static_cast<size_t>(p) * row_vec + c] = make_uint4(0, 0, 0, 0);
  const int npos = g.offsets[g.E];
  if (p == 0 && lane == 0 && (npos < 0 || npos > g.P)) report_error(err, BI_DEVERR_BAD_PERMUTATION);
  if (p >= npos) return;
  const int pair = perm[p];
  if (static_cast<unsigned>(pair) >= static_cast<unsigned>(g.P)) {
    if (lane == 0) report_error(err, BI_DEVERR_BAD_PERMUTATION);
    return;
  }
  const uint4 *src = rows + static_cast<size_t>(pair / top_k) * row_vec;
  uint4 *dst = to + static_cast<size_t>(p) * row_vec;
#pragma unroll 4
  for (int c = lane; c < row_vec; c += 32) dst[c] = src[c];
}

// dwts[perm[p]] = the parts of position p in order.
__device__ __forceinline__ void sum_dwts(const DwtsSum &d, int p) {
  if (p >= d.g.P || p >= d.g.offsets[d.g.E]) return;
  const int pair = d.perm[p];
  if (static_cast<unsigned>(pair) >= static_cast<unsigned>(d.g.P)) return;  // (reported by the gather)
  float s = 0.0f;
#pragma unroll 8
  for (int i = 0; i < d.nparts; ++i) s = __fadd_rn(s, d.parts[static_cast<int64_t>(i) * d.g.P + p]);
  d.dwts[pair] = s;
}
__global__ void __launch_bounds__(256) dwts_kernel(DwtsSum d) {
  griddep_wait_small_release();
  sum_dwts(d, blockIdx.x * 256 + threadIdx.x);
}

// Slots of a row that are pairs of the grouping: ids in range, each once.
__device__ __forceinline__ uint32_t valid_slots(const int32_t *ids, int top_k, int E) {
  uint32_t ok = 0u;
  for (int t = 0; t < top_k; ++t) {
    const int e = ids[t];
    bool v = e >= 0 && e < E;
    for (int u = 0; u < t; ++u) v = v && ids[u] != e;
    ok |= static_cast<uint32_t>(v) << t;
  }
  return ok;
}

__device__ __forceinline__ void add4(float4 &s, float4 v) {
  s.x = __fadd_rn(s.x, v.x);
  s.y = __fadd_rn(s.y, v.y);
  s.z = __fadd_rn(s.z, v.z);
  s.w = __fadd_rn(s.w, v.w);
}

// Four consecutive elements of dx per thread: the contributions in slot order,
// then the router's rows in slot order.
// The blocks from `blocks` on sum parts of dwts (a launch of its own took 3 us of a
// small step).
__global__ void __launch_bounds__(256) grad_combine_kernel(GradCombine a, unsigned blocks, DwtsSum d) {
  griddep_wait_small_release();
  if (blockIdx.x >= blocks) {
    sum_dwts(d, (blockIdx.x - blocks) * 256 + threadIdx.x);
    return;
  }
  const int H4 = static_cast<int>(a.H / 4);
  const int64_t idx = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (idx >= a.M * H4) return;
  const int64_t m = idx / H4;
  const int h4 = static_cast<int>(idx - m * H4);
  const uint32_t ok = a.slots ? a.slots[m] : valid_slots(a.ids + m * a.top_k, a.top_k, a.E);
  float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (a.contrib) {
    const float4 *c = reinterpret_cast<const float4 *>(a.contrib) + m * a.top_k * H4 + h4;
#pragma unroll 8
    for (int t = 0; t < a.top_k; ++t) {
      const float4 v = c[static_cast<int64_t>(t) * H4];
      if ((ok >> t) & 1u) add4(s, v);
    }
  }
  if (a.w) {
    for (int t = 0; t < a.top_k; ++t) {
      const int64_t q = m * a.top_k + t;
      const int e = a.ids[q];
      if (!((ok >> t) & 1u) || e < 0 || e >= a.E) continue;
      const float c = score_grad(a.dwts[q], a.wts[q]);
      const float4 w = reinterpret_cast<const float4 *>(a.w)[static_cast<int64_t>(e) * H4 + h4];
      s.x = __fmaf_rn(c, w.x, s.x);
      s.y = __fmaf_rn(c, w.y, s.y);
      s.z = __fmaf_rn(c, w.z, s.z);
      s.w = __fmaf_rn(c, w.w, s.w);
    }
    add4(s, make_float4(0.0f, 0.0f, 0.0f, 0.0f));  // (-0 to 0, as the other kernel's slots of c = 0 make it)
  }
  if (a.dx_f32) {
    reinterpret_cast<float4 *>(a.dx)[idx] = s;
  } else {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(s.x, s.y), hi = __floats2bfloat162_rn(s.z, s.w);
    reinterpret_cast<uint2 *>(a.dx)[idx] =
        make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
  }
}

// The same over columns of W in shared memory: a CTA holds kStageCols columns of
// all rows of W and takes every gridDim.y-th group of tokens, 16 lanes a token with
// four columns each.  A token's lanes first hold a slot each and leave its row's
// place and c in a table, two slots to a 16-byte word; a slot that is not valid has
// c = 0 and a row of zeros.  (4096 tokens, 256 experts, top 8, H=4096: rows of W from
// L2 100 us, staged with a slot's id and c by shuffles 44, by the table 33: the
// instructions a slot are the limit, shared memory would allow 15.)
constexpr int kStageCols = 64, kStageThreads = 512;

__device__ __forceinline__ void fma4(float4 &s, float c, float4 w) {
  asm("{\n\t.reg .b64 c, w, s;\n\t"
      "mov.b64 c, {%4, %4};\n\t"
      "mov.b64 w, {%5, %6};\n\tmov.b64 s, {%0, %1};\n\tfma.rn.f32x2 s, c, w, s;\n\tmov.b64 {%0, %1}, s;\n\t"
      "mov.b64 w, {%7, %8};\n\tmov.b64 s, {%2, %3};\n\tfma.rn.f32x2 s, c, w, s;\n\tmov.b64 {%2, %3}, s;\n\t}"
      : "+f"(s.x), "+f"(s.y), "+f"(s.z), "+f"(s.w)
      : "f"(c), "f"(w.x), "f"(w.y), "f"(w.z), "f"(w.w));
}

__global__ void __launch_bounds__(kStageThreads, 3) grad_combine_staged_kernel(GradCombine a) {
  extern __shared__ float4 w_s[];  // [E + 1][kStageCols / 4], the last row 0
  __shared__ __align__(16) float2 slot_s[kStageThreads];  // (place of the row in w_s, c) of a slot
  griddep_wait();
  griddep_launch_dependents();  // (the router's dW runs beside this: see there)
  const int64_t H4 = a.H / 4;
  const int c4 = blockIdx.x * (kStageCols / 4), lane = threadIdx.x & 15;
  const bool in = c4 + lane < H4;
  for (int i = threadIdx.x; i < (a.E + 1) * 16; i += kStageThreads)
    w_s[i] = in && i < a.E * 16 ? reinterpret_cast<const float4 *>(a.w)[static_cast<int64_t>(i >> 4) * H4 + c4 + lane]
                                : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  __syncthreads();
  constexpr int kTokens = kStageThreads / 16;
  const int64_t step = static_cast<int64_t>(gridDim.y) * kTokens;
  int64_t m = static_cast<int64_t>(blockIdx.y) * kTokens + (threadIdx.x >> 4);
  const float4 *slots = reinterpret_cast<const float4 *>(slot_s + (threadIdx.x & ~15));
  // the next token's slot is under way while this one's rows are added
  int next_id = -1;
  float next_dw = 0.0f, next_w = 0.0f;
  uint32_t next_slots = 0xffffffffu;
  const auto load = [&](int64_t token) {
    const bool slot = token < a.M && lane < a.top_k;
    const int64_t q = slot ? token * a.top_k + lane : 0;
    next_id = slot ? a.ids[q] : -1;
    next_dw = a.dwts[q];
    next_w = a.wts[q];
    if (a.slots) next_slots = token < a.M ? a.slots[token] : 0u;
  };
  load(m);
  for (int64_t m0 = static_cast<int64_t>(blockIdx.y) * kTokens; m0 < a.M; m0 += step, m += step) {
    const bool there = m < a.M;  // (lanes without a token take part in the exchange)
    const int id = next_id;
    const float c = score_grad(next_dw, next_w);
    bool ok = id >= 0 && id < a.E && ((next_slots >> lane) & 1u);
    load(m + step);
    if (!a.slots) {  // not an earlier slot's
      const uint32_t same = __match_any_sync(0xffffffffu, ok ? 2 * id + static_cast<int>((threadIdx.x >> 4) & 1) : -1);
      ok = ok && !(same & ((1u << (threadIdx.x & 31)) - 1u));
    }
    slot_s[threadIdx.x] = make_float2(__int_as_float((ok ? id : a.E) * 16), ok ? c : 0.0f);
    const uint32_t valid = __ballot_sync(0xffffffffu, ok) >> (threadIdx.x & 16);  // (and orders the table)
    __syncwarp();
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (a.contrib && there && in) {
      const float4 *k = reinterpret_cast<const float4 *>(a.contrib) + m * a.top_k * H4 + c4 + lane;
#pragma unroll 8
      for (int t = 0; t < a.top_k; ++t) {
        const float4 v = k[t * H4];
        if ((valid >> t) & 1u) add4(s, v);
      }
    }
#pragma unroll 4
    for (int t = 0; t < a.top_k; t += 2) {
      const float4 two = slots[t / 2];
      const float4 w0 = w_s[__float_as_int(two.x) + lane], w1 = w_s[__float_as_int(two.z) + lane];
      fma4(s, two.y, w0);
      fma4(s, two.w, w1);
    }
    add4(s, make_float4(0.0f, 0.0f, 0.0f, 0.0f));
    __syncwarp();
    if (!there || !in) continue;
    const int64_t at = m * H4 + c4 + lane;
    if (a.dx_f32) {
      reinterpret_cast<float4 *>(a.dx)[at] = s;
    } else {
      const __nv_bfloat162 lo = __floats2bfloat162_rn(s.x, s.y), hi = __floats2bfloat162_rn(s.z, s.w);
      reinterpret_cast<uint2 *>(a.dx)[at] =
          make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
    }
  }
}

// A CTA of 8 warps per expert and 256 columns of x, 8 a lane: the warps take the
// expert's positions in turn, kRouterUnroll rows under way at once, and their sums
// are added in order.  The positions' (token, c) come into shared memory
// kRouterBatch at a time, and the warps' sums are closed behind each batch, so that
// no running sum of a long group is longer than 64 products or the number of its
// batches (unclosed, 66048 equal products summed to 1.2e-4 too little).  Behind the
// kernel that stages W, `beside`: launched while that one runs and waiting for it
// only at the end, as it reads nothing that one writes (what came before is done
// when that one has begun).
// (4096 tokens, 256 experts, top 8, H=4096, with L2 emptied before: 50 us with groups
// of up to 1018 positions, 40 with even ones, the rows of x from L2 top_k times over,
// 268 MB.  Measured beside 58 with warm inputs and uneven groups: a warp's columns 512 or 1024 wide, so that (token, c) are made
// fewer times: 74 and 111 us, held up by the largest group; columns of x in shared
// memory, read once: 181 us, the latencies of a warp's experts one after another.)
constexpr int kRouterBatch = 512, kRouterUnroll = 4, kRouterWarps = 8, kRouterCols = 256;

// Eight elements as they lie in memory.
template <typename XT>
struct Row8 {
  uint32_t w[2 * sizeof(XT)];
  __device__ __forceinline__ float at(int j) const {
    if constexpr (sizeof(XT) == 4) return __uint_as_float(w[j]);
    else return __uint_as_float(j & 1 ? w[j / 2] & 0xffff0000u : w[j / 2] << 16);
  }
};
template <typename XT>
__device__ __forceinline__ Row8<XT> row8(const XT *p) {
  Row8<XT> r;
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(XT)) / 2; ++i) {
    const uint4 v = __ldg(reinterpret_cast<const uint4 *>(p) + i);
    r.w[4 * i] = v.x, r.w[4 * i + 1] = v.y, r.w[4 * i + 2] = v.z, r.w[4 * i + 3] = v.w;
  }
  return r;
}

template <typename XT>
__global__ void __launch_bounds__(32 * kRouterWarps, 5)
    router_dw_kernel(const float *__restrict__ dwts, const float *__restrict__ wts, const XT *__restrict__ x, Groups g,
                     const int32_t *__restrict__ perm, float *dw, float *dbias, int add, int H, int top_k, int beside,
                     int *err) {
  __shared__ __align__(16) float s[kRouterWarps][kRouterCols];  // 8 KB: each lane's sums of the batches so far
  __shared__ int token_s[kRouterBatch];
  __shared__ float c_s[kRouterBatch];
  if (!beside) griddep_wait_small_release();
  const int e = blockIdx.x, h0 = blockIdx.y * kRouterCols, warp = threadIdx.x >> 5;
  const int beg = g.offsets[e], end = g.offsets[e + 1];
  // beside: this grid is not done before dx' is, which later work takes for granted; with bad offsets neither
  const bool last = beside && blockIdx.x == 0 && blockIdx.y == 0;
  if (beg < 0 || end < beg || end > g.P) {
    if (threadIdx.x == 0) report_error(err, BI_DEVERR_BAD_PERMUTATION);
    if (last) griddep_wait();
    return;
  }
  const int col = (threadIdx.x & 31) * 8;
  const bool in = dw && h0 + col < H;  // H is a multiple of 8
  const XT *from = x + h0 + col;
  float acc[8] = {}, bias = 0.0f;
  // acc, this lane's sums of a batch, added to those of the batches before it
  float4 *own = reinterpret_cast<float4 *>(&s[warp][col]);
  const auto close = [&](bool first) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float4 t = make_float4(acc[4 * j], acc[4 * j + 1], acc[4 * j + 2], acc[4 * j + 3]);
      if (!first) add4(t, own[j]);
      own[j] = t;
    }
  };
  for (int b0 = beg; b0 < end; b0 += kRouterBatch) {
    if (b0 > beg) {
      close(b0 == beg + kRouterBatch);
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[j] = 0.0f;
    }
    const int n = min(kRouterBatch, end - b0);
    for (int i = threadIdx.x; i < n; i += 32 * kRouterWarps) {
      const int pair = perm[b0 + i];
      const bool ok = static_cast<unsigned>(pair) < static_cast<unsigned>(g.P);
      if (!ok) report_error(err, BI_DEVERR_BAD_PERMUTATION);
      token_s[i] = ok ? pair / top_k : -1;
      c_s[i] = ok ? score_grad(dwts[pair], wts[pair]) : 0.0f;
    }
    __syncthreads();
    if (threadIdx.x < 32 && dbias && h0 == 0) {
      float part = 0.0f;
      for (int i = threadIdx.x; i < n; i += 32) part = __fadd_rn(part, c_s[i]);
      bias = __fadd_rn(bias, part);
    }
    if (in) {
      for (int i0 = warp; i0 < n; i0 += kRouterWarps * kRouterUnroll) {
        // (loads without a condition and apart from their use, so that they are under way together: past the end
        // the last position's row again)
        Row8<XT> v[kRouterUnroll];
#pragma unroll
        for (int u = 0; u < kRouterUnroll; ++u)
          v[u] = row8(from + static_cast<int64_t>(max(token_s[min(i0 + u * kRouterWarps, n - 1)], 0)) * H);
#pragma unroll
        for (int u = 0; u < kRouterUnroll; ++u) {
          const int i = i0 + u * kRouterWarps;
          if (i >= n || token_s[i] < 0) continue;
          const float c = c_s[i];
#pragma unroll
          for (int j = 0; j < 8; ++j) acc[j] = __fmaf_rn(c, v[u].at(j), acc[j]);
        }
      }
    }
    __syncthreads();
  }
  close(end - beg <= kRouterBatch);
  __syncthreads();
  for (int i = threadIdx.x; i < kRouterCols && dw && h0 + i < H; i += 32 * kRouterWarps) {
    float t = 0.0f;
#pragma unroll
    for (int w = 0; w < kRouterWarps; ++w) t = __fadd_rn(t, s[w][i]);
    float *o = dw + static_cast<int64_t>(e) * H + h0 + i;
    *o = add ? __fadd_rn(*o, t) : t;
  }
  if (threadIdx.x < 32 && dbias && h0 == 0) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) bias = __fadd_rn(bias, __shfl_xor_sync(0xffffffffu, bias, d));
    if (threadIdx.x == 0) dbias[e] = add ? __fadd_rn(dbias[e], bias) : bias;
  }
  if (last) griddep_wait();
}

// ------------------------------------------------------------------- host --
bi_status launch_train_gather(const __nv_bfloat16 *rows, Groups g, const int32_t *perm, __nv_bfloat16 *to, float *dwts,
                              __nv_bfloat16 *zero, const uint32_t *slots, int64_t H, int32_t top_k, cudaStream_t s) {
  return launch_chained(train_gather_kernel, dim3((g.P + 7) / 8), dim3(256), 0, s, 1,
                        reinterpret_cast<const uint4 *>(rows), g, perm, top_k, static_cast<int>(H / 8),
                        reinterpret_cast<uint4 *>(to), dwts, reinterpret_cast<uint4 *>(zero), slots,
                        device_error_word());
}

bi_status launch_dwts(const DwtsSum &d, cudaStream_t s) {
  return launch_chained(dwts_kernel, dim3((d.g.P + 255) / 256), dim3(256), 0, s, 1, d);
}

// Staged where the tokens read W several times over.
static size_t staged_bytes(const GradCombine &a) { return static_cast<size_t>(a.E + 1) * kStageCols * sizeof(float); }
bool grad_combine_stages(const GradCombine &a) {
  return a.w && a.M * a.top_k > 4 * a.E && staged_bytes(a) <= 200 * 1024;
}

bi_status launch_grad_combine(const GradCombine &a, const DwtsSum *sum, cudaStream_t s) {
  const size_t smem = staged_bytes(a);
  if (grad_combine_stages(a)) {
    static std::mutex mu;
    static ContextSetup setup;  // the shared-memory attribute is per context
    int dev = 0;
    cudaGetDevice(&dev);
    {
      std::lock_guard<std::mutex> lk(mu);
      if (setup.pending(dev)) {
        const cudaError_t e =
            cudaFuncSetAttribute(grad_combine_staged_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 200 * 1024);
        if (e != cudaSuccess) {
          cudaGetLastError();
          set_error("cudaFuncSetAttribute: %s", cudaGetErrorString(e));
          return BI_ERR_CUDA;
        }
        setup.done(dev);
      }
    }
    // as few groups of tokens as fill the SMs; one CTA an SM beside the router's dW (dx and dW of 4096 tokens, 256
    // experts, top 8, H=4096: 83 us, three CTAs an SM 90; dx alone 45 and 33)
    const int cols = static_cast<int>((a.H + kStageCols - 1) / kStageCols);
    const int per_sm = static_cast<int>(std::max<size_t>(1, std::min<size_t>(a.beside ? 1 : 3, 220 * 1024 / (smem + 6 * 1024))));
    const int64_t groups = (a.M + kStageThreads / 16 - 1) / (kStageThreads / 16);
    const int64_t split = std::max<int64_t>(1, std::min<int64_t>(groups, num_sms() * per_sm / cols));
    return launch_chained(grad_combine_staged_kernel, dim3(cols, static_cast<unsigned>(split)), dim3(kStageThreads), smem,
                          s, 1, a);
  }
  const int64_t blocks = (a.M * (a.H / 4) + 255) / 256;
  const int64_t more = sum ? (sum->g.P + 255) / 256 : 0;
  if (blocks + more >= (int64_t(1) << 31)) {
    set_error("gradient combine of more than 2^31 blocks");
    return BI_ERR_UNSUPPORTED;
  }
  return launch_chained(grad_combine_kernel, dim3(static_cast<unsigned>(blocks + more)), dim3(256), 0, s, 1, a,
                        static_cast<unsigned>(blocks), sum ? *sum : DwtsSum{});
}

template <typename XT>
static bi_status router_dw_of(const float *dwts, const float *wts, const XT *x, Groups g, const int32_t *perm, float *dw,
                              float *dbias, bool add, bool beside, int H, int32_t top_k, cudaStream_t s) {
  const dim3 grid(g.E, dw ? (H + kRouterCols - 1) / kRouterCols : 1);
  return launch_chained(router_dw_kernel<XT>, grid, dim3(32 * kRouterWarps), 0, s, 1, dwts, wts, x, g, perm, dw, dbias, add ? 1 : 0, H,
                        top_k, beside ? 1 : 0, device_error_word());
}

bi_status launch_router_dw(const float *dwts, const float *wts, const void *x, bool x_f32, Groups g,
                           const int32_t *perm, float *dw, float *dbias, bool add, bool beside, int64_t H,
                           int32_t top_k, cudaStream_t s) {
  const int h = static_cast<int>(H);
  if (x_f32) return router_dw_of(dwts, wts, static_cast<const float *>(x), g, perm, dw, dbias, add, beside, h, top_k, s);
  return router_dw_of(dwts, wts, static_cast<const __nv_bfloat16 *>(x), g, perm, dw, dbias, add, beside, h, top_k, s);
}

}  // namespace bimoe
