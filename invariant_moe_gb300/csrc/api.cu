// api.cu -- the extern "C" entry points of libbimoe.so: argument checks,
// workspace layout, TMA descriptor encoding, and the device error word.
// All arithmetic happens in the kernels of router.cu, router_topk.cu, topk.cu,
// topk_window.cu, moe_route.cu, moe_gemm.cu, ffn.cu, mx4.cu, mx4_gemm.cu,
// grouped.cu, moe_grad.cu and layer_norm.cu.
#include <cstdarg>
#include <cstdio>
#include <atomic>
#include <mutex>
#include <utility>

#include "bimoe_internal.cuh"
#include "ffn_internal.cuh"
#include "train_internal.cuh"

namespace bimoe {

bi_status launch_router(const float *, const float *, const float *, float *, int64_t, int64_t,
                        int64_t, int, cudaStream_t);
bi_status launch_router_bf16(const void *, const float *, const float *, float *, int64_t, int64_t,
                             int64_t, int, cudaStream_t, unsigned *zero_words, int n_zero);
bi_status launch_topk_window(const float *, int64_t, const int64_t *, const int64_t *, int64_t,
                             int64_t, int32_t, int32_t *, cudaStream_t);
bi_status launch_router_negctl(const float *, const float *, const float *, float *, int64_t,
                               int64_t, int64_t, cudaStream_t);
bi_status launch_cast_bf16_f32(const void *, float *, int64_t, cudaStream_t);
bi_status launch_topk(const float *, int32_t *, float *, float *, int64_t, int64_t, int32_t,
                      cudaStream_t);
size_t permute_scratch_bytes(int64_t M, int64_t E);
bi_status launch_permute(const int32_t *, int32_t *, int32_t *, int64_t, int64_t, int32_t, void *,
                         cudaStream_t, uint32_t *slot_mask);
bi_status launch_gather(const void *, const int32_t *, const int32_t *, int64_t, int64_t, int64_t,
                        int32_t, void *, cudaStream_t);
bi_status launch_combine(const float *, void *, int64_t, int64_t, int32_t, bool, cudaStream_t,
                         const uint32_t *slot_mask);
bi_status launch_gate_up(const void *, const int32_t *, const int32_t *, const float *,
                         const void *, void *, int64_t, int64_t, int64_t, int32_t, int64_t,
                         cudaStream_t);
int set_gemm_variant(int v);
bi_status launch_gate_up_tokens(const void *, int64_t, const int32_t *, const int32_t *, const float *,
                                const void *, void *, int64_t, int64_t, int32_t, int64_t, cudaStream_t);
bool decode_path_ok(int64_t M, int64_t E, int32_t top_k);
size_t decode_counter_count(int64_t M, int64_t H);
bi_status launch_moe_decode(const void *, const int32_t *, const float *, const void *, const void *, void *,
                            float *, int *, void *, int64_t, int64_t, int64_t, int32_t, int64_t, cudaStream_t,
                            const float *scores, int32_t *ids_out, float *wts_out);
int set_decode_fused(int mode);
bool decode_fused_ok(int64_t M, int64_t H, int64_t E, int32_t top_k, int64_t I);
int64_t decode_fused_ready_count(int64_t M, int64_t E, int32_t top_k, int64_t I);
bi_status launch_moe_decode_fused(const void *, const void *, const void *, void *, float *, int *, unsigned *,
                                  void *, int64_t, int64_t, int64_t, int32_t, int64_t, cudaStream_t,
                                  const float *scores, int32_t *ids_out, float *wts_out);
// How bi_moe_forward feeds the gate/up GEMM its token rows: 0 automatic (the
// copy), 1 the gather kernel's contiguous copy, 2 gathered by the GEMM itself
// (tile::gather4).  Measured on GB300 at M=4096 the GEMM gathering its own
// rows is 3x slower (DSv4-shaped gate/up 4.31 ms against 1.45 ms; Qwen-shaped
// 0.339 against 0.220 ms): the TMA issues the 128-byte row gathers at about
// 20 cycles per row per SM, well below what the MMAs consume; at decode sizes
// the two are within noise.
static std::atomic<int> g_gate_up_feed{0};
static bool feed_in_gemm() { return g_gate_up_feed.load() == 2; }
bi_status launch_down(const void *, const int32_t *, const int32_t *, const void *, float *,
                      int64_t, int64_t, int64_t, int32_t, int64_t, cudaStream_t);
bi_status launch_fp32_fma_probe(float *, int64_t, int32_t, cudaStream_t);
bool router_topk_fused_supported(int64_t M, int64_t K, int64_t N, int32_t top_k);
template <typename XT>
bi_status launch_router_topk_fused(const XT *, const float *, const float *, float *, float *, int32_t *,
                                   float *, int64_t, int64_t, int64_t, int32_t, cudaStream_t);
// Batches up to this many rows take the one-kernel router + top-k (when its
// cluster can be scheduled); larger ones the router grid and the selection
// grid.  Both give the same bits.  0: the one-kernel path runs only when
// forced (schedule 10): measured on GB300 it is slower than the chained grids
// (DSv4 router shape, M=1: 10.9 us against 8.6 us; the 16 SMs of one
// cluster each stream 256 KB of the weight, and the two grids spread it over
// all SMs).
constexpr int64_t kFusedRouterTopkMaxM = 0;
bi_status launch_gather_routing(const int32_t *, const float *, const int32_t *, const int32_t *, int64_t,
                                int64_t, int64_t, int32_t *, float *, cudaStream_t);
bi_status launch_scatter_contrib(const float *, const int32_t *, const int32_t *, int64_t, int64_t, int64_t,
                                 float *, cudaStream_t);
bi_status launch_wait_timeout_probe(int, cudaStream_t);

// ------------------------------------------------------------ error state --
static thread_local char g_msg[512] = "";

void set_error(const char *fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_msg, sizeof g_msg, fmt, ap);
  va_end(ap);
}

// One word per device: kernels record the first BI_DEVERR_* they hit.
__device__ int g_device_error;

constexpr int kMaxDevices = 64;
static std::mutex g_mu;
static int *g_err_ptr[kMaxDevices] = {};
static ContextSetup g_err_ctx;
static int g_sms[kMaxDevices] = {};

static int current_device() {
  int d = 0;
  if (cudaGetDevice(&d) != cudaSuccess) return 0;
  return d;
}

typedef CUresult (*CtxGetCurrentFn)(CUcontext *);
typedef CUresult (*CtxGetIdFn)(CUcontext, unsigned long long *);

unsigned long long current_context_id() {
  static CtxGetCurrentFn get_current = nullptr;
  static CtxGetIdFn get_id = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuCtxGetCurrent", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      get_current = reinterpret_cast<CtxGetCurrentFn>(p);
    p = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuCtxGetId", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      get_id = reinterpret_cast<CtxGetIdFn>(p);
  });
  if (!get_current || !get_id) return 0;
  CUcontext c = nullptr;
  if (get_current(&c) != CUDA_SUCCESS || c == nullptr) return 0;
  unsigned long long id = 0;
  if (get_id(c, &id) != CUDA_SUCCESS) return 0;
  return id + 1;  // 0 stays "no context"
}

int *device_error_word() {
  const int d = current_device();
  if (d >= kMaxDevices) return nullptr;
  std::lock_guard<std::mutex> lk(g_mu);
  // the word's address belongs to the context the module is loaded in
  if (!g_err_ptr[d] || g_err_ctx.pending(d)) {
    void *p = nullptr;
    g_err_ptr[d] = nullptr;
    if (cudaGetSymbolAddress(&p, g_device_error) == cudaSuccess) {
      g_err_ptr[d] = static_cast<int *>(p);
      g_err_ctx.done(d);
    }
  }
  return g_err_ptr[d];
}

int num_sms() {
  const int d = current_device();
  if (d >= kMaxDevices) return 148;
  std::lock_guard<std::mutex> lk(g_mu);
  if (!g_sms[d]) {
    int v = 0;
    if (cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, d) != cudaSuccess || v <= 0) v = 148;
    g_sms[d] = v;
  }
  return g_sms[d];
}

// ------------------------------------------------------------ TMA encode --
typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                  const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                  const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

static EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}

bool make_tma_2d_f32(CUtensorMap *map, const void *base, uint64_t rows, uint64_t cols,
                     uint32_t box_rows) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) {
    set_error("cuTensorMapEncodeTiled is not available from the driver");
    return false;
  }
  const cuuint64_t dims[2] = {cols, rows};
  const cuuint64_t strides[1] = {cols * 4};
  const cuuint32_t box[2] = {32, box_rows};
  const cuuint32_t estr[2] = {1, 1};
  const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, const_cast<void *>(base), dims,
                        strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) {
    set_error("cuTensorMapEncodeTiled failed (%d) for fp32 [%llu x %llu]", (int)r,
              (unsigned long long)rows, (unsigned long long)cols);
    return false;
  }
  return true;
}

bool make_tma_2d_bf16_ld(CUtensorMap *map, const void *base, uint64_t rows, uint64_t cols, uint64_t ld,
                         uint32_t box_rows) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) {
    set_error("cuTensorMapEncodeTiled is not available from the driver");
    return false;
  }
  const cuuint64_t dims[2] = {cols, rows};
  const cuuint64_t strides[1] = {ld * 2};
  const cuuint32_t box[2] = {64, box_rows};
  const cuuint32_t estr[2] = {1, 1};
  const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(base), dims,
                        strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) {
    set_error("cuTensorMapEncodeTiled failed (%d) for [%llu x %llu]", (int)r,
              (unsigned long long)rows, (unsigned long long)cols);
    return false;
  }
  return true;
}

bool make_tma_2d_bf16(CUtensorMap *map, const void *base, uint64_t rows, uint64_t cols,
                      uint32_t box_rows) {
  return make_tma_2d_bf16_ld(map, base, rows, cols, cols, box_rows);
}

bool make_tma_3d(CUtensorMap *map, const void *base, bool f32, uint64_t E, uint64_t rows, uint64_t cols,
                 uint32_t box_rows) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) {
    set_error("cuTensorMapEncodeTiled is not available from the driver");
    return false;
  }
  const cuuint64_t dims[3] = {cols, rows, E};
  const uint64_t size = f32 ? 4 : 2;
  const cuuint64_t strides[2] = {cols * size, rows * cols * size};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(128 / size), box_rows, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = fn(map, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) {
    set_error("cuTensorMapEncodeTiled failed (%d) for %llu x [%llu x %llu]", (int)r, (unsigned long long)E,
              (unsigned long long)rows, (unsigned long long)cols);
    return false;
  }
  return true;
}

bool make_tma_mx_scales(CUtensorMap *map, const void *base, uint64_t row_tiles, uint64_t ktiles, uint32_t box_rows) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) {
    set_error("cuTensorMapEncodeTiled is not available from the driver");
    return false;
  }
  const cuuint64_t dims[2] = {ktiles * 128, row_tiles};  // 32-bit words
  const cuuint64_t strides[1] = {ktiles * 512};
  const cuuint32_t box[2] = {256, box_rows};
  const cuuint32_t estr[2] = {1, 1};
  const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_INT32, 2, const_cast<void *>(base), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) {
    set_error("cuTensorMapEncodeTiled failed (%d) for scale tiles [%llu x %llu]", (int)r,
              (unsigned long long)row_tiles, (unsigned long long)ktiles);
    return false;
  }
  return true;
}

bool make_tma_2d_u8(CUtensorMap *map, const void *base, uint64_t rows, uint64_t row_bytes, uint32_t box_rows) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) {
    set_error("cuTensorMapEncodeTiled is not available from the driver");
    return false;
  }
  const cuuint64_t dims[2] = {row_bytes, rows};
  const cuuint64_t strides[1] = {row_bytes};
  const cuuint32_t box[2] = {128, box_rows};
  const cuuint32_t estr[2] = {1, 1};
  const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) {
    set_error("cuTensorMapEncodeTiled failed (%d) for bytes [%llu x %llu]", (int)r, (unsigned long long)rows,
              (unsigned long long)row_bytes);
    return false;
  }
  return true;
}

bool make_tma_inter_bf16(CUtensorMap *map, const void *base, uint64_t rows, uint64_t I, uint64_t K,
                         uint32_t groups) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) {
    set_error("cuTensorMapEncodeTiled is not available from the driver");
    return false;
  }
  if (rows % 16 != 0 || I % 16 != 0) {
    set_error("interleaved weight map needs rows and I multiples of 16");
    return false;
  }
  const cuuint64_t dims[4] = {K, 16, 2, rows / 16};
  const cuuint64_t strides[3] = {K * 2, I * K * 2, 16 * K * 2};
  const cuuint32_t box[4] = {64, 16, 2, groups};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base), dims, strides, box,
                        estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) {
    set_error("cuTensorMapEncodeTiled failed (%d) for the interleaved map [%llu x %llu], I=%llu", (int)r,
              (unsigned long long)rows, (unsigned long long)K, (unsigned long long)I);
    return false;
  }
  return true;
}

// ------------------------------------------------------- MoE workspace --
static size_t align256(size_t v) { return (v + 255) / 256 * 256; }

struct MoeWorkspace {
  size_t offsets, perm, slot_mask, scratch, xperm, act, contrib, counters, gridbar, total;
};

static MoeWorkspace moe_layout(int64_t M, int64_t H, int64_t E, int32_t top_k, int64_t I) {
  MoeWorkspace w{};
  const size_t P = static_cast<size_t>(M) * top_k;
  size_t off = 0;
  w.offsets = off; off += align256((E + 1) * sizeof(int32_t));
  w.perm = off;    off += align256(P * sizeof(int32_t));
  w.slot_mask = off; off += align256(static_cast<size_t>(M) * sizeof(uint32_t));
  w.scratch = off; off += align256(permute_scratch_bytes(M, E));
  w.xperm = off;   off += align256(P * H * 2);
  w.act = off;     off += align256(P * I * 2);
  w.contrib = off; off += align256(P * H * sizeof(float));
  w.counters = off; off += align256(decode_counter_count(M, H) * sizeof(int));
  w.gridbar = off; off += 4096;  // the one-launch decode layer's ready counts (at most 1024)
  w.total = off;
  return w;
}

static bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

static bi_status check_moe_dims(int64_t M, int64_t H, int64_t E, int32_t top_k, int64_t I) {
  if (M < 0 || H <= 0 || E <= 0 || I <= 0) {
    set_error("negative or zero size (M=%lld H=%lld E=%lld I=%lld)", (long long)M, (long long)H,
              (long long)E, (long long)I);
    return BI_ERR_INVALID_ARG;
  }
  if (top_k < 1 || top_k > 16 || top_k > E) {
    set_error("top_k=%d outside [1, min(16, E)]", top_k);
    return BI_ERR_INVALID_ARG;
  }
  if (E > 1024 || H % 128 != 0 || I % 128 != 0) {
    set_error("unsupported MoE shape (needs H%%128==0, I%%128==0, E<=1024): H=%lld I=%lld E=%lld",
              (long long)H, (long long)I, (long long)E);
    return BI_ERR_UNSUPPORTED;
  }
  if (M * top_k >= (int64_t(1) << 31) || M * top_k * H >= (int64_t(1) << 40) ||
      E * 2 * I >= (int64_t(1) << 31) || E * H >= (int64_t(1) << 31)) {
    set_error("MoE sizes exceed the 32-bit index range");
    return BI_ERR_UNSUPPORTED;
  }
  return BI_OK;
}

}  // namespace bimoe

using namespace bimoe;

#define BI_REQUIRE(cond, code, ...) \
  do {                              \
    if (!(cond)) {                  \
      set_error(__VA_ARGS__);       \
      return code;                  \
    }                               \
  } while (0)

extern "C" {

BI_API const char *bi_status_str(bi_status s) {
  switch (s) {
    case BI_OK: return "BI_OK";
    case BI_ERR_INVALID_ARG: return "BI_ERR_INVALID_ARG";
    case BI_ERR_UNSUPPORTED: return "BI_ERR_UNSUPPORTED";
    case BI_ERR_WORKSPACE: return "BI_ERR_WORKSPACE";
    case BI_ERR_CUDA: return "BI_ERR_CUDA";
    case BI_ERR_DEVICE: return "BI_ERR_DEVICE";
  }
  return "BI_ERR_UNKNOWN";
}

BI_API const char *bi_last_error_message(void) { return g_msg; }

BI_API const char *bi_version(void) { return "bimoe 0.1 sm_103a"; }

BI_API bi_status bi_device_error(int32_t *code) {
  BI_REQUIRE(code, BI_ERR_INVALID_ARG, "code is NULL");
  int v = 0, zero = 0;
  cudaError_t e = cudaDeviceSynchronize();
  if (e == cudaSuccess) e = cudaMemcpyFromSymbol(&v, g_device_error, sizeof v);
  if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_device_error, &zero, sizeof zero);
  if (e != cudaSuccess) {
    set_error("reading the device error word: %s", cudaGetErrorString(e));
    return BI_ERR_CUDA;
  }
  *code = v;
  return BI_OK;
}

BI_API bi_status bi_cast_bf16_to_f32(const bi_bf16 *x, float *y, int64_t n, bi_stream_t stream) {
  BI_REQUIRE(n >= 0, BI_ERR_INVALID_ARG, "n < 0");
  if (n == 0) return BI_OK;
  BI_REQUIRE(x && y, BI_ERR_INVALID_ARG, "null pointer");
  return launch_cast_bf16_f32(x, y, n, reinterpret_cast<cudaStream_t>(stream));
}

static bi_status router_checks(const void *x, const float *w, float *y, int64_t M, int64_t K,
                               int64_t N) {
  BI_REQUIRE(M >= 0 && K > 0 && N > 0, BI_ERR_INVALID_ARG, "bad sizes M=%lld K=%lld N=%lld",
             (long long)M, (long long)K, (long long)N);
  BI_REQUIRE(M == 0 || (x && w && y), BI_ERR_INVALID_ARG, "null pointer");
  BI_REQUIRE(K % 128 == 0 && K <= 32768 && N <= 4096, BI_ERR_UNSUPPORTED,
             "router recipe needs K %% 128 == 0, K <= 32768, N <= 4096 (K=%lld N=%lld)",
             (long long)K, (long long)N);
  BI_REQUIRE(M * K < (int64_t(1) << 40) && M * N < (int64_t(1) << 31), BI_ERR_UNSUPPORTED,
             "router sizes exceed the index range");
  BI_REQUIRE(M == 0 || (aligned(x, 16) && aligned(w, 16)), BI_ERR_INVALID_ARG,
             "x and w must be 16-byte aligned");
  return BI_OK;
}

BI_API bi_status bi_router_gemm_schedule(const float *x, const float *w, const float *bias,
                                         float *y, int64_t M, int64_t K, int64_t N,
                                         int32_t schedule, bi_stream_t stream) {
  bi_status st = router_checks(x, w, y, M, K, N);
  if (st != BI_OK) return st;
  BI_REQUIRE(schedule >= 0 && schedule <= 9, BI_ERR_INVALID_ARG, "schedule %d", schedule);
  if (M == 0) return BI_OK;
  return launch_router(x, w, bias, y, M, K, N, schedule, reinterpret_cast<cudaStream_t>(stream));
}

BI_API bi_status bi_router_gemm(const float *x, const float *w, const float *bias, float *y,
                                int64_t M, int64_t K, int64_t N, bi_stream_t stream) {
  return bi_router_gemm_schedule(x, w, bias, y, M, K, N, 0, stream);
}

BI_API bi_status bi_router_gemm_bf16_schedule(const bi_bf16 *x, const float *w, const float *bias,
                                              float *y, int64_t M, int64_t K, int64_t N,
                                              int32_t schedule, bi_stream_t stream) {
  bi_status st = router_checks(x, w, y, M, K, N);
  if (st != BI_OK) return st;
  BI_REQUIRE(schedule >= 0 && schedule <= 9, BI_ERR_INVALID_ARG, "schedule %d", schedule);
  if (M == 0) return BI_OK;
  return launch_router_bf16(x, w, bias, y, M, K, N, schedule, reinterpret_cast<cudaStream_t>(stream), nullptr, 0);
}

BI_API bi_status bi_router_gemm_bf16(const bi_bf16 *x, const float *w, const float *bias, float *y,
                                     int64_t M, int64_t K, int64_t N, bi_stream_t stream) {
  return bi_router_gemm_bf16_schedule(x, w, bias, y, M, K, N, 0, stream);
}

BI_API bi_status bi_router_gemm_splitk_negctl(const float *x, const float *w, const float *bias,
                                              float *y, int64_t M, int64_t K, int64_t N,
                                              bi_stream_t stream) {
  bi_status st = router_checks(x, w, y, M, K, N);
  if (st != BI_OK) return st;
  if (M == 0) return BI_OK;
  return launch_router_negctl(x, w, bias, y, M, K, N, reinterpret_cast<cudaStream_t>(stream));
}

BI_API bi_status bi_topk(const float *scores, float *probs, int32_t *ids, float *wts, int64_t M,
                         int64_t E, int32_t top_k, bi_stream_t stream) {
  BI_REQUIRE(M >= 0, BI_ERR_INVALID_ARG, "M < 0");
  BI_REQUIRE(E >= 1 && E <= 512, BI_ERR_UNSUPPORTED, "E=%lld outside [1, 512]", (long long)E);
  BI_REQUIRE(top_k >= 1 && top_k <= 16 && top_k <= E, BI_ERR_INVALID_ARG,
             "top_k=%d outside [1, min(16, E)]", top_k);
  BI_REQUIRE(M * E < (int64_t(1) << 31), BI_ERR_UNSUPPORTED, "M*E exceeds the index range");
  if (M == 0) return BI_OK;
  BI_REQUIRE(scores && ids && wts, BI_ERR_INVALID_ARG, "null pointer");
  return launch_topk(scores, ids, wts, probs, M, E, top_k, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"

static bi_status launch_router_any(const float *x, const float *w, const float *b, float *y, int64_t M,
                                   int64_t K, int64_t N, int schedule, cudaStream_t s) {
  return launch_router(x, w, b, y, M, K, N, schedule, s);
}
static bi_status launch_router_any(const __nv_bfloat16 *x, const float *w, const float *b, float *y,
                                   int64_t M, int64_t K, int64_t N, int schedule, cudaStream_t s) {
  return launch_router_bf16(x, w, b, y, M, K, N, schedule, s, nullptr, 0);
}

// Router + selection: schedule 0 picks by M (the one-kernel path for small
// batches, else the router grid chained with the selection grid), 10 forces
// the one-kernel path, 1..9 force a router schedule followed by the selection
// grid.
template <typename XT>
static bi_status router_topk_impl(const XT *x, const float *w, const float *bias, float *y, float *probs,
                                  int32_t *ids, float *wts, int64_t M, int64_t K, int64_t N, int32_t top_k,
                                  int32_t schedule, bi_stream_t stream) {
  bi_status st = router_checks(x, w, y, M, K, N);
  if (st != BI_OK) return st;
  BI_REQUIRE(schedule >= 0 && schedule <= 10, BI_ERR_INVALID_ARG, "schedule %d", schedule);
  BI_REQUIRE(N <= 512, BI_ERR_UNSUPPORTED, "selection needs N <= 512 (N=%lld)", (long long)N);
  BI_REQUIRE(top_k >= 1 && top_k <= 16 && top_k <= N, BI_ERR_INVALID_ARG,
             "top_k=%d outside [1, min(16, N)]", top_k);
  if (M == 0) return BI_OK;
  BI_REQUIRE(ids && wts, BI_ERR_INVALID_ARG, "null pointer");
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (schedule == 10) return launch_router_topk_fused(x, w, bias, y, probs, ids, wts, M, K, N, top_k, s);
  if (schedule == 0 && M <= kFusedRouterTopkMaxM && router_topk_fused_supported(M, K, N, top_k)) {
    st = launch_router_topk_fused(x, w, bias, y, probs, ids, wts, M, K, N, top_k, s);
    if (st != BI_ERR_UNSUPPORTED) return st;  // else its cluster cannot be scheduled: two grids
  }
  if ((st = launch_router_any(x, w, bias, y, M, K, N, schedule, s)) != BI_OK) return st;
  return launch_topk(y, ids, wts, probs, M, N, top_k, s);
}

extern "C" {

BI_API bi_status bi_router_topk_schedule(const float *x, const float *w, const float *bias,
                                         float *y, float *probs, int32_t *ids, float *wts,
                                         int64_t M, int64_t K, int64_t N, int32_t top_k,
                                         int32_t schedule, bi_stream_t stream) {
  return router_topk_impl(x, w, bias, y, probs, ids, wts, M, K, N, top_k, schedule, stream);
}

BI_API bi_status bi_router_topk_bf16_schedule(const bi_bf16 *x, const float *w, const float *bias,
                                              float *y, float *probs, int32_t *ids, float *wts,
                                              int64_t M, int64_t K, int64_t N, int32_t top_k,
                                              int32_t schedule, bi_stream_t stream) {
  return router_topk_impl(reinterpret_cast<const __nv_bfloat16 *>(x), w, bias, y, probs, ids, wts, M, K, N,
                          top_k, schedule, stream);
}

BI_API bi_status bi_router_topk(const float *x, const float *w, const float *bias, float *y,
                                float *probs, int32_t *ids, float *wts, int64_t M, int64_t K,
                                int64_t N, int32_t top_k, bi_stream_t stream) {
  return bi_router_topk_schedule(x, w, bias, y, probs, ids, wts, M, K, N, top_k, 0, stream);
}

BI_API bi_status bi_router_topk_bf16(const bi_bf16 *x, const float *w, const float *bias, float *y,
                                     float *probs, int32_t *ids, float *wts, int64_t M, int64_t K,
                                     int64_t N, int32_t top_k, bi_stream_t stream) {
  return bi_router_topk_bf16_schedule(x, w, bias, y, probs, ids, wts, M, K, N, top_k, 0, stream);
}

BI_API bi_status bi_topk_window(const float *scores, int64_t ld, const int64_t *row_start,
                                const int64_t *row_end, int64_t n_rows, int64_t num_cols,
                                int32_t k, int32_t *out, bi_stream_t stream) {
  BI_REQUIRE(n_rows >= 0 && num_cols >= 0 && ld >= num_cols, BI_ERR_INVALID_ARG,
             "bad sizes n_rows=%lld num_cols=%lld ld=%lld", (long long)n_rows,
             (long long)num_cols, (long long)ld);
  BI_REQUIRE(num_cols <= 8192, BI_ERR_UNSUPPORTED, "num_cols=%lld > 8192", (long long)num_cols);
  BI_REQUIRE(k >= 1 && k <= 8192, BI_ERR_INVALID_ARG, "k=%d outside [1, 8192]", k);
  BI_REQUIRE(n_rows < (int64_t(1) << 31) && n_rows * ld < (int64_t(1) << 62), BI_ERR_UNSUPPORTED,
             "sizes exceed the index range");
  if (n_rows == 0) return BI_OK;
  BI_REQUIRE(out && (scores || num_cols == 0), BI_ERR_INVALID_ARG, "null pointer");
  return launch_topk_window(scores, ld, row_start, row_end, n_rows, num_cols, k, out,
                            reinterpret_cast<cudaStream_t>(stream));
}

BI_API bi_status bi_fp32_fma_probe(float *out, int64_t blocks, int32_t iters, bi_stream_t stream) {
  BI_REQUIRE(out && blocks > 0 && blocks < (int64_t(1) << 31) && iters > 0, BI_ERR_INVALID_ARG,
             "bad probe arguments");
  return launch_fp32_fma_probe(out, blocks, iters, reinterpret_cast<cudaStream_t>(stream));
}

BI_API bi_status bi_wait_timeout_probe(int32_t which, bi_stream_t stream) {
  BI_REQUIRE(which == 0 || which == 1, BI_ERR_INVALID_ARG, "wait probe %d not in {0, 1}", which);
  return launch_wait_timeout_probe(which, reinterpret_cast<cudaStream_t>(stream));
}

BI_API size_t bi_moe_workspace_bytes(int64_t M, int64_t H, int64_t E, int32_t top_k, int64_t I) {
  if (check_moe_dims(M, H, E, top_k, I) != BI_OK) return 0;
  return moe_layout(M, H, E, top_k, I).total;
}

BI_API size_t bi_moe_permute_workspace_bytes(int64_t M, int64_t E) {
  if (M < 0 || E <= 0) return 0;
  return align256(permute_scratch_bytes(M, E));
}

BI_API bi_status bi_moe_permute(const int32_t *ids, int32_t *offsets, int32_t *perm, int64_t M,
                                int64_t E, int32_t top_k, void *workspace, size_t workspace_bytes,
                                bi_stream_t stream) {
  BI_REQUIRE(M >= 0 && E >= 1 && E <= 1024, BI_ERR_INVALID_ARG, "bad sizes M=%lld E=%lld",
             (long long)M, (long long)E);
  BI_REQUIRE(top_k >= 1 && top_k <= 16 && top_k <= E, BI_ERR_INVALID_ARG, "top_k=%d", top_k);
  BI_REQUIRE(M * top_k < (int64_t(1) << 31), BI_ERR_UNSUPPORTED, "M*top_k exceeds int32");
  BI_REQUIRE(offsets, BI_ERR_INVALID_ARG, "offsets is NULL");
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (M == 0) {
    if (cudaMemsetAsync(offsets, 0, (E + 1) * sizeof(int32_t), s) != cudaSuccess) {
      set_error("cudaMemsetAsync failed");
      return BI_ERR_CUDA;
    }
    return BI_OK;
  }
  BI_REQUIRE(ids && perm && workspace, BI_ERR_INVALID_ARG, "null pointer");
  BI_REQUIRE(workspace_bytes >= bi_moe_permute_workspace_bytes(M, E), BI_ERR_WORKSPACE,
             "workspace %zu < %zu bytes", workspace_bytes, bi_moe_permute_workspace_bytes(M, E));
  return launch_permute(ids, offsets, perm, M, E, top_k, workspace, s, nullptr);
}

BI_API bi_status bi_moe_gather(const bi_bf16 *x, const int32_t *offsets, const int32_t *perm,
                               bi_bf16 *x_perm, int64_t M, int64_t H, int64_t E, int32_t top_k,
                               bi_stream_t stream) {
  BI_REQUIRE(M >= 0 && H > 0 && H % 8 == 0 && E >= 1, BI_ERR_INVALID_ARG, "bad sizes (H %% 8 == 0)");
  BI_REQUIRE(top_k >= 1 && top_k <= 16, BI_ERR_INVALID_ARG, "top_k=%d", top_k);
  BI_REQUIRE(M * top_k < (int64_t(1) << 31), BI_ERR_UNSUPPORTED, "M*top_k exceeds int32");
  if (M == 0) return BI_OK;
  BI_REQUIRE(x && offsets && perm && x_perm, BI_ERR_INVALID_ARG, "null pointer");
  BI_REQUIRE(aligned(x, 16) && aligned(x_perm, 16), BI_ERR_INVALID_ARG,
             "x and x_perm must be 16-byte aligned");
  return launch_gather(x, perm, offsets, M * top_k, H, E, top_k, x_perm,
                       reinterpret_cast<cudaStream_t>(stream));
}

BI_API bi_status bi_moe_gate_up(const bi_bf16 *x_perm, const int32_t *offsets, const int32_t *perm,
                                const float *wts, const bi_bf16 *w13, bi_bf16 *act, int64_t M,
                                int64_t H, int64_t E, int32_t top_k, int64_t I,
                                bi_stream_t stream) {
  bi_status st = check_moe_dims(M, H, E, top_k, I);
  if (st != BI_OK) return st;
  if (M == 0) return BI_OK;
  BI_REQUIRE(x_perm && offsets && perm && wts && w13 && act, BI_ERR_INVALID_ARG, "null pointer");
  BI_REQUIRE(aligned(x_perm, 16) && aligned(w13, 16), BI_ERR_INVALID_ARG,
             "x_perm/w13 must be 16-byte aligned");
  return launch_gate_up(x_perm, offsets, perm, wts, w13, act, M * top_k, H, E, top_k, I,
                        reinterpret_cast<cudaStream_t>(stream));
}

BI_API bi_status bi_moe_gate_up_tokens(const bi_bf16 *x, const int32_t *offsets, const int32_t *perm,
                                       const float *wts, const bi_bf16 *w13, bi_bf16 *act, int64_t M,
                                       int64_t H, int64_t E, int32_t top_k, int64_t I, bi_stream_t stream) {
  bi_status st = check_moe_dims(M, H, E, top_k, I);
  if (st != BI_OK) return st;
  if (M == 0) return BI_OK;
  BI_REQUIRE(x && offsets && perm && wts && w13 && act, BI_ERR_INVALID_ARG, "null pointer");
  BI_REQUIRE(aligned(x, 16) && aligned(w13, 16), BI_ERR_INVALID_ARG, "x/w13 must be 16-byte aligned");
  return launch_gate_up_tokens(x, M, offsets, perm, wts, w13, act, H, E, top_k, I,
                               reinterpret_cast<cudaStream_t>(stream));
}

BI_API bi_status bi_moe_down(const bi_bf16 *act, const int32_t *offsets, const int32_t *perm,
                             const bi_bf16 *w2, float *contrib, int64_t M, int64_t H, int64_t E,
                             int32_t top_k, int64_t I, bi_stream_t stream) {
  bi_status st = check_moe_dims(M, H, E, top_k, I);
  if (st != BI_OK) return st;
  if (M == 0) return BI_OK;
  BI_REQUIRE(act && offsets && perm && w2 && contrib, BI_ERR_INVALID_ARG, "null pointer");
  BI_REQUIRE(aligned(act, 16) && aligned(w2, 16), BI_ERR_INVALID_ARG,
             "act/w2 must be 16-byte aligned");
  return launch_down(act, offsets, perm, w2, contrib, M * top_k, H, E, top_k, I,
                     reinterpret_cast<cudaStream_t>(stream));
}

BI_API bi_status bi_moe_combine(const float *contrib, bi_bf16 *out, int64_t M, int64_t H,
                                int32_t top_k, bi_stream_t stream) {
  BI_REQUIRE(M >= 0 && H > 0 && H % 4 == 0, BI_ERR_INVALID_ARG, "bad sizes (H %% 4 == 0 needed)");
  BI_REQUIRE(top_k >= 1 && top_k <= 16, BI_ERR_INVALID_ARG, "top_k=%d", top_k);
  if (M == 0) return BI_OK;
  BI_REQUIRE(contrib && out, BI_ERR_INVALID_ARG, "null pointer");
  BI_REQUIRE(aligned(contrib, 16) && aligned(out, 8), BI_ERR_INVALID_ARG,
             "contrib must be 16-byte and out 8-byte aligned");
  return launch_combine(contrib, out, M, H, top_k, false, reinterpret_cast<cudaStream_t>(stream), nullptr);
}

BI_API bi_status bi_moe_combine_consume(float *contrib, bi_bf16 *out, int64_t M, int64_t H,
                                        int32_t top_k, bi_stream_t stream) {
  BI_REQUIRE(M >= 0 && H > 0 && H % 4 == 0, BI_ERR_INVALID_ARG, "bad sizes (H %% 4 == 0 needed)");
  BI_REQUIRE(top_k >= 1 && top_k <= 16, BI_ERR_INVALID_ARG, "top_k=%d", top_k);
  if (M == 0) return BI_OK;
  BI_REQUIRE(contrib && out, BI_ERR_INVALID_ARG, "null pointer");
  BI_REQUIRE(aligned(contrib, 16) && aligned(out, 8), BI_ERR_INVALID_ARG,
             "contrib must be 16-byte and out 8-byte aligned");
  return launch_combine(contrib, out, M, H, top_k, true, reinterpret_cast<cudaStream_t>(stream), nullptr);
}

BI_API bi_status bi_moe_gather_routing(const int32_t *ids, const float *wts, const int32_t *offsets,
                                       const int32_t *perm, int32_t *lid, float *pw, int64_t M, int64_t E,
                                       int32_t top_k, int64_t experts_per_rank, bi_stream_t stream) {
  BI_REQUIRE(M >= 0 && E >= 1 && E <= 1024, BI_ERR_INVALID_ARG, "bad sizes M=%lld E=%lld", (long long)M,
             (long long)E);
  BI_REQUIRE(top_k >= 1 && top_k <= 16 && top_k <= E, BI_ERR_INVALID_ARG, "top_k=%d", top_k);
  BI_REQUIRE(experts_per_rank >= 1 && experts_per_rank <= E && E % experts_per_rank == 0, BI_ERR_INVALID_ARG,
             "experts_per_rank=%lld must divide E=%lld", (long long)experts_per_rank, (long long)E);
  BI_REQUIRE(M * top_k < (int64_t(1) << 31), BI_ERR_UNSUPPORTED, "M*top_k exceeds int32");
  if (M == 0) return BI_OK;
  BI_REQUIRE(ids && wts && offsets && perm && lid && pw, BI_ERR_INVALID_ARG, "null pointer");
  return launch_gather_routing(ids, wts, offsets, perm, M * top_k, E, experts_per_rank, lid, pw,
                               reinterpret_cast<cudaStream_t>(stream));
}

BI_API bi_status bi_moe_scatter_contrib(const float *rows, const int32_t *offsets, const int32_t *perm,
                                        float *contrib, int64_t M, int64_t H, int64_t E, int32_t top_k,
                                        bi_stream_t stream) {
  BI_REQUIRE(M >= 0 && H > 0 && H % 4 == 0 && E >= 1 && E <= 1024, BI_ERR_INVALID_ARG,
             "bad sizes (H %% 4 == 0 needed)");
  BI_REQUIRE(top_k >= 1 && top_k <= 16, BI_ERR_INVALID_ARG, "top_k=%d", top_k);
  BI_REQUIRE(M * top_k < (int64_t(1) << 31), BI_ERR_UNSUPPORTED, "M*top_k exceeds int32");
  if (M == 0) return BI_OK;
  BI_REQUIRE(rows && offsets && perm && contrib, BI_ERR_INVALID_ARG, "null pointer");
  BI_REQUIRE(aligned(rows, 16) && aligned(contrib, 16), BI_ERR_INVALID_ARG,
             "rows and contrib must be 16-byte aligned");
  return launch_scatter_contrib(rows, offsets, perm, M * top_k, H, E, contrib,
                                reinterpret_cast<cudaStream_t>(stream));
}

BI_API bi_status bi_moe_forward(const bi_bf16 *x, const int32_t *ids, const float *wts,
                                const bi_bf16 *w13, const bi_bf16 *w2, bi_bf16 *out, int64_t M,
                                int64_t H, int64_t E, int32_t top_k, int64_t I, void *workspace,
                                size_t workspace_bytes, bi_stream_t stream) {
  bi_status st = check_moe_dims(M, H, E, top_k, I);
  if (st != BI_OK) return st;
  if (M == 0) return BI_OK;
  BI_REQUIRE(x && ids && wts && w13 && w2 && out && workspace, BI_ERR_INVALID_ARG, "null pointer");
  BI_REQUIRE(aligned(x, 16) && aligned(w13, 16) && aligned(w2, 16) && aligned(out, 8) &&
                 aligned(workspace, 256),
             BI_ERR_INVALID_ARG, "misaligned pointer (x/w13/w2 16 B, out 8 B, workspace 256 B)");
  const MoeWorkspace L = moe_layout(M, H, E, top_k, I);
  BI_REQUIRE(workspace_bytes >= L.total, BI_ERR_WORKSPACE, "workspace %zu < %zu bytes",
             workspace_bytes, L.total);
  char *ws = static_cast<char *>(workspace);
  int32_t *offsets = reinterpret_cast<int32_t *>(ws + L.offsets);
  int32_t *perm = reinterpret_cast<int32_t *>(ws + L.perm);
  void *xperm = ws + L.xperm;
  void *act = ws + L.act;
  float *contrib = reinterpret_cast<float *>(ws + L.contrib);
  uint32_t *slot_mask = reinterpret_cast<uint32_t *>(ws + L.slot_mask);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int64_t P = M * top_k;
  if (g_gate_up_feed.load() == 0 && decode_path_ok(M, E, top_k)) {
    // decode-sized batch: two launches, the routing derived inside the GEMMs
    // and the combine fused into the down GEMM
    return launch_moe_decode(x, ids, wts, w13, w2, act, contrib, reinterpret_cast<int *>(ws + L.counters), out,
                             M, H, E, top_k, I, s, nullptr, nullptr, nullptr);
  }
  if ((st = launch_permute(ids, offsets, perm, M, E, top_k, ws + L.scratch, s, slot_mask)) != BI_OK)
    return st;
  if (feed_in_gemm()) {
    // the gate/up GEMM gathers the token rows from x itself
    if ((st = launch_gate_up_tokens(x, M, offsets, perm, wts, w13, act, H, E, top_k, I, s)) != BI_OK)
      return st;
  } else {
    if ((st = launch_gather(x, perm, offsets, P, H, E, top_k, xperm, s)) != BI_OK) return st;
    if ((st = launch_gate_up(xperm, offsets, perm, wts, w13, act, P, H, E, top_k, I, s)) != BI_OK)
      return st;
  }
  if ((st = launch_down(act, offsets, perm, w2, contrib, P, H, E, top_k, I, s)) != BI_OK) return st;
  // a pair skipped for a bad id (recorded in the device error word) adds
  // nothing: the combine sums the slots the permutation marked valid
  return launch_combine(contrib, out, M, H, top_k, true, s, slot_mask);
}

BI_API bi_status bi_moe_layer(const bi_bf16 *x, const float *w_router, const float *bias,
                              const bi_bf16 *w13, const bi_bf16 *w2, bi_bf16 *out, float *scores,
                              int32_t *ids, float *wts, int64_t M, int64_t H, int64_t E, int32_t top_k,
                              int64_t I, void *workspace, size_t workspace_bytes, bi_stream_t stream) {
  bi_status st = check_moe_dims(M, H, E, top_k, I);
  if (st != BI_OK) return st;
  BI_REQUIRE(E <= 512, BI_ERR_UNSUPPORTED, "the layer's selection needs E <= 512 (E=%lld)", (long long)E);
  if ((st = router_checks(x, w_router, scores, M, H, E)) != BI_OK) return st;
  if (M == 0) return BI_OK;
  BI_REQUIRE(x && w_router && w13 && w2 && out && scores && ids && wts && workspace, BI_ERR_INVALID_ARG,
             "null pointer");
  BI_REQUIRE(aligned(x, 16) && aligned(w13, 16) && aligned(w2, 16) && aligned(out, 8) && aligned(workspace, 256),
             BI_ERR_INVALID_ARG, "misaligned pointer (x/w13/w2 16 B, out 8 B, workspace 256 B)");
  const MoeWorkspace L = moe_layout(M, H, E, top_k, I);
  BI_REQUIRE(workspace_bytes >= L.total, BI_ERR_WORKSPACE, "workspace %zu < %zu bytes", workspace_bytes, L.total);
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  char *ws = static_cast<char *>(workspace);
  const bool decode = g_gate_up_feed.load() == 0 && decode_path_ok(M, E, top_k);
  // decode-sized batch with the one-launch expert path: the router zeroes
  // its combine counters and ready counts (one range: the counters, the
  // padding after them, the ready counts)
  const bool fused = decode && decode_fused_ok(M, H, E, top_k, I);
  unsigned *zero_from = fused ? reinterpret_cast<unsigned *>(ws + L.counters) : nullptr;
  const int n_zero = fused ? static_cast<int>((L.gridbar - L.counters) / 4 + decode_fused_ready_count(M, E, top_k, I))
                           : 0;
  if ((st = launch_router_bf16(x, w_router, bias, scores, M, H, E, 0, s, zero_from, n_zero)) != BI_OK) return st;
  if (fused)
    return launch_moe_decode_fused(x, w13, w2, ws + L.act, reinterpret_cast<float *>(ws + L.contrib),
                                   reinterpret_cast<int *>(ws + L.counters), reinterpret_cast<unsigned *>(ws + L.gridbar),
                                   out, M, H, E, top_k, I, s, scores, ids, wts);
  if (decode) {
    // decode-sized batch: the gate/up GEMM selects the experts itself
    return launch_moe_decode(x, nullptr, nullptr, w13, w2, ws + L.act, reinterpret_cast<float *>(ws + L.contrib),
                             reinterpret_cast<int *>(ws + L.counters), out, M, H, E, top_k, I, s, scores, ids, wts);
  }
  if ((st = launch_topk(scores, ids, wts, nullptr, M, E, top_k, s)) != BI_OK) return st;
  return bi_moe_forward(x, ids, wts, w13, w2, out, M, H, E, top_k, I, workspace, workspace_bytes, stream);
}

}  // extern "C"

BI_API bi_status bi_moe_gate_up_feed(int32_t mode, int32_t *previous) {
  BI_REQUIRE(mode >= 0 && mode <= 2, BI_ERR_INVALID_ARG, "feed mode %d not in {0, 1, 2}", mode);
  const int old = g_gate_up_feed.exchange(mode);
  if (previous) *previous = old;
  return BI_OK;
}

BI_API bi_status bi_moe_decode_fused(int32_t mode, int32_t *previous) {
  BI_REQUIRE(mode == 0 || mode == 1, BI_ERR_INVALID_ARG, "decode layer mode %d not in {0, 1}", mode);
  const int old = bimoe::set_decode_fused(mode);
  if (previous) *previous = old;
  return BI_OK;
}

BI_API bi_status bi_moe_gemm_variant(int32_t variant, int32_t *previous) {
  BI_REQUIRE(variant >= 0 && variant <= 4, BI_ERR_INVALID_ARG, "variant %d not in {0, ..., 4}", variant);
  const int old = bimoe::set_gemm_variant(variant);
  if (previous) *previous = old;
  return BI_OK;
}

// -------------------------------------- dense gated feed-forward block --
static bi_status check_ffn_dims(int64_t M, int64_t H, int64_t I) {
  BI_REQUIRE(M >= 0 && H > 0 && I > 0, BI_ERR_INVALID_ARG, "negative or zero size (M=%lld H=%lld I=%lld)",
             (long long)M, (long long)H, (long long)I);
  BI_REQUIRE(H % 16 == 0 && I % 16 == 0, BI_ERR_UNSUPPORTED,
             "unsupported feed-forward shape (needs H %% 16 == 0, I %% 16 == 0): H=%lld I=%lld", (long long)H,
             (long long)I);
  BI_REQUIRE(M <= (int64_t(1) << 30) && H <= (int64_t(1) << 20) && I <= (int64_t(1) << 20), BI_ERR_UNSUPPORTED,
             "feed-forward sizes exceed the index range (M=%lld H=%lld I=%lld)", (long long)M, (long long)H,
             (long long)I);
  return BI_OK;
}

// A token matrix [M, cols] with row stride ld: 16-byte rows, as the copies want them.
static bi_status check_rows(const char *name, const void *p, int64_t ld, int64_t cols) {
  BI_REQUIRE(p, BI_ERR_INVALID_ARG, "%s is NULL", name);
  BI_REQUIRE(aligned(p, 16), BI_ERR_INVALID_ARG, "%s must be 16-byte aligned", name);
  BI_REQUIRE(ld >= cols && ld % 8 == 0 && ld <= (int64_t(1) << 30), BI_ERR_INVALID_ARG,
             "row stride of %s: %lld (needs a multiple of 8, at least %lld)", name, (long long)ld, (long long)cols);
  return BI_OK;
}

// Whether two matrices of `rows` rows share memory, rows of a and b bytes every lda and ldb bytes (with
// different strides: whether their ranges do).
static bool overlap_bytes(const void *p, int64_t lda, int64_t a, const void *q, int64_t ldb, int64_t b, int64_t rows) {
  uintptr_t at_p = reinterpret_cast<uintptr_t>(p), at_q = reinterpret_cast<uintptr_t>(q);
  if (at_p > at_q) {
    std::swap(at_p, at_q);
    std::swap(lda, ldb);
    std::swap(a, b);
  }
  const uintptr_t apart = at_q - at_p;
  if (apart >= static_cast<uintptr_t>((rows - 1) * lda + a)) return false;
  if (lda != ldb) return true;
  const int64_t at = static_cast<int64_t>(apart % static_cast<uintptr_t>(lda));
  return at < a || at > lda - b;
}
// The same of two bf16 matrices of `rows` x `cols` with row strides ldp and ldq (elements).
static bool overlap(const void *p, int64_t ldp, const void *q, int64_t ldq, int64_t rows, int64_t cols) {
  return overlap_bytes(p, ldp * 2, cols * 2, q, ldq * 2, cols * 2, rows);
}

// An array of a call (p may be null: not given).
struct Span {
  const char *name;
  const void *p;
  int64_t bytes;
};
static bool spans_meet(const Span &a, const Span &b) {
  const uintptr_t p = reinterpret_cast<uintptr_t>(a.p), q = reinterpret_cast<uintptr_t>(b.p);
  return p && q && p < q + static_cast<uintptr_t>(b.bytes) && q < p + static_cast<uintptr_t>(a.bytes);
}
// The results share no memory with one another nor with the operands; but `same` may be one of them, byte for byte,
// for results[0].
template <size_t R, size_t O>
static bi_status check_apart(const Span (&results)[R], const Span (&operands)[O], const void *same = nullptr) {
  for (size_t i = 0; i < R; ++i) {
    for (size_t j = i + 1; j < R; ++j)
      BI_REQUIRE(!spans_meet(results[i], results[j]), BI_ERR_INVALID_ARG, "%s and %s overlap", results[i].name,
                 results[j].name);
    for (const Span &o : operands)
      BI_REQUIRE(!spans_meet(results[i], o) || (i == 0 && o.p == same && results[0].p == same), BI_ERR_INVALID_ARG,
                 "%s overlaps %s", results[i].name, o.name);
  }
  return BI_OK;
}

static Mat mat(const bi_bf16 *p, int64_t ld) { return Mat{reinterpret_cast<const __nv_bfloat16 *>(p), ld}; }
static const __nv_bfloat16 *cbf(const void *p) { return static_cast<const __nv_bfloat16 *>(p); }
static __nv_bfloat16 *mbf(void *p) { return static_cast<__nv_bfloat16 *>(p); }

#define BI_TRY(call)                       \
  do {                                     \
    const bi_status st_ = (call);          \
    if (st_ != BI_OK) return st_;          \
  } while (0)

extern "C" {

BI_API size_t bi_ffn_workspace_bytes(int64_t M, int64_t H, int64_t I) {
  if (check_ffn_dims(M, H, I) != BI_OK) return 0;
  return std::max<size_t>(256, align256(static_cast<size_t>(M) * 2 * I * sizeof(bi_bf16)));
}

static bi_status ffn_forward_impl(const bi_bf16 *x, int64_t ldx, const bi_bf16 *w13, const bi_bf16 *w2,
                                  const bi_bf16 *addend, int64_t ld_addend, bi_bf16 *out, int64_t ldo, float *gu,
                                  void *act, int64_t M, int64_t H, int64_t I, bi_stream_t stream) {
  BI_TRY(check_rows("x", x, ldx, H));
  BI_TRY(check_rows("out", out, ldo, H));
  if (addend) BI_TRY(check_rows("addend", addend, ld_addend, H));
  BI_REQUIRE(w13 && w2, BI_ERR_INVALID_ARG, "null pointer");
  BI_REQUIRE(aligned(w13, 16) && aligned(w2, 16), BI_ERR_INVALID_ARG, "w13 and w2 must be 16-byte aligned");
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  BI_TRY(launch_ffn_gate_up(mat(x, ldx), cbf(w13), mbf(act), gu, M, H, I, s));
  return launch_ffn_down(cbf(act), cbf(w2), mat(addend, ld_addend), mbf(out), ldo, M, H, I, s);
}

BI_API bi_status bi_ffn_forward(const bi_bf16 *x, int64_t ldx, const bi_bf16 *w13, const bi_bf16 *w2,
                                const bi_bf16 *addend, int64_t ld_addend, bi_bf16 *out, int64_t ldo, int64_t M,
                                int64_t H, int64_t I, void *workspace, size_t workspace_bytes, bi_stream_t stream) {
  BI_TRY(check_ffn_dims(M, H, I));
  if (M == 0) return BI_OK;
  const size_t need = static_cast<size_t>(M) * I * sizeof(bi_bf16);
  BI_REQUIRE(workspace && aligned(workspace, 256), BI_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  BI_REQUIRE(workspace_bytes >= need, BI_ERR_WORKSPACE, "workspace %zu < %zu bytes", workspace_bytes, need);
  return ffn_forward_impl(x, ldx, w13, w2, addend, ld_addend, out, ldo, nullptr, workspace, M, H, I, stream);
}

BI_API bi_status bi_ffn_forward_train(const bi_bf16 *x, int64_t ldx, const bi_bf16 *w13, const bi_bf16 *w2,
                                      const bi_bf16 *addend, int64_t ld_addend, bi_bf16 *out, int64_t ldo, float *gu,
                                      bi_bf16 *act, int64_t M, int64_t H, int64_t I, bi_stream_t stream) {
  BI_TRY(check_ffn_dims(M, H, I));
  if (M == 0) return BI_OK;
  BI_REQUIRE(gu && act, BI_ERR_INVALID_ARG, "null pointer");
  BI_REQUIRE(aligned(gu, 16) && aligned(act, 16), BI_ERR_INVALID_ARG, "gu and act must be 16-byte aligned");
  return ffn_forward_impl(x, ldx, w13, w2, addend, ld_addend, out, ldo, gu, act, M, H, I, stream);
}

BI_API bi_status bi_ffn_backward(const bi_bf16 *dout, int64_t lddo, const bi_bf16 *x, int64_t ldx, const bi_bf16 *w13,
                                 const bi_bf16 *w2, const float *gu, const bi_bf16 *act, bi_bf16 *dx, int64_t lddx,
                                 void *dw13, void *dw2, int32_t grad_mode, int64_t M, int64_t H, int64_t I,
                                 void *workspace, size_t workspace_bytes, bi_stream_t stream) {
  BI_TRY(check_ffn_dims(M, H, I));
  BI_REQUIRE(grad_mode >= 0 && grad_mode <= 2, BI_ERR_INVALID_ARG, "grad_mode %d not in {0, 1, 2}", grad_mode);
  BI_REQUIRE(aligned(dw13, 16) && aligned(dw2, 16), BI_ERR_INVALID_ARG, "dw13 and dw2 must be 16-byte aligned");
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (M == 0) {
    // no tokens: the weight gradients are zero (or stay as they are, when added to)
    const size_t item = grad_mode == kGradBf16 ? 2 : 4;
    cudaError_t e = cudaSuccess;
    if (grad_mode != kGradF32Accumulate && dw13)
      e = cudaMemsetAsync(dw13, 0, static_cast<size_t>(2 * I) * H * item, s);
    if (e == cudaSuccess && grad_mode != kGradF32Accumulate && dw2)
      e = cudaMemsetAsync(dw2, 0, static_cast<size_t>(I) * H * item, s);
    BI_REQUIRE(e == cudaSuccess, BI_ERR_CUDA, "cudaMemsetAsync: %s", cudaGetErrorString(e));
    return BI_OK;
  }
  if (!dx && !dw13 && !dw2) return BI_OK;
  BI_TRY(check_rows("dout", dout, lddo, H));
  if (dx) BI_TRY(check_rows("dx", dx, lddx, H));
  if (dw13) BI_TRY(check_rows("x", x, ldx, H));
  BI_REQUIRE(w2 && gu && (w13 || !dx) && (act || !dw2), BI_ERR_INVALID_ARG, "null pointer");
  BI_REQUIRE(aligned(w13, 16) && aligned(w2, 16) && aligned(gu, 16) && aligned(act, 16), BI_ERR_INVALID_ARG,
             "w13, w2, gu and act must be 16-byte aligned");
  __nv_bfloat16 *dgu = mbf(workspace);
  if (dx || dw13) {
    const size_t need = static_cast<size_t>(M) * 2 * I * sizeof(bi_bf16);
    BI_REQUIRE(workspace && aligned(workspace, 256), BI_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
    BI_REQUIRE(workspace_bytes >= need, BI_ERR_WORKSPACE, "workspace %zu < %zu bytes", workspace_bytes, need);
    // dx is written beside the products that read dout (dW2) and x (dW13)
    BI_REQUIRE(!(dx && dw2 && overlap(dx, lddx, dout, lddo, M, H)), BI_ERR_INVALID_ARG, "dx and dout overlap");
    BI_REQUIRE(!(dx && dw13 && overlap(dx, lddx, x, ldx, M, H)), BI_ERR_INVALID_ARG, "dx and x overlap");
    BI_TRY(launch_ffn_dact(mat(dout, lddo), cbf(w2), gu, dgu, M, H, I, s));
  }
  const FfnGrads d{mat(dout, lddo), mat(x, ldx), dgu, cbf(act), cbf(w13), mbf(dx), lddx, dw13, dw2, grad_mode};
  return launch_ffn_grads(d, M, H, I, s);
}

BI_API bi_status bi_ffn_schedule(int32_t mode, int32_t *previous) {
  BI_REQUIRE(mode >= 0 && mode <= 2, BI_ERR_INVALID_ARG, "feed-forward schedule %d not in {0, 1, 2}", mode);
  const int old = bimoe::set_ffn_schedule(mode);
  if (previous) *previous = old;
  return BI_OK;
}

// ------------------------------------- microscaled 4-bit floating point --
static bi_status check_mx4_dims(const char *rows, int64_t R, int64_t K) {
  BI_REQUIRE(R >= 0 && K > 0, BI_ERR_INVALID_ARG, "bad sizes %s=%lld K=%lld", rows, (long long)R, (long long)K);
  BI_REQUIRE(K % kMxBlock == 0, BI_ERR_UNSUPPORTED, "K must be a multiple of 32 (K=%lld)", (long long)K);
  BI_REQUIRE(R <= (int64_t(1) << 30) && K <= (int64_t(1) << 20), BI_ERR_UNSUPPORTED,
             "sizes exceed the index range (%s=%lld K=%lld)", rows, (long long)R, (long long)K);
  return BI_OK;
}

BI_API size_t bi_mx4_scale_bytes(int64_t R, int64_t K) {
  if (check_mx4_dims("R", R, K) != BI_OK) return 0;
  return static_cast<size_t>((R + kMxTileRows - 1) / kMxTileRows) * ((K + 127) / 128) * kMxTileBytes;
}

BI_API bi_status bi_mx4_quantize(const void *x, int32_t x_f32, int64_t ldx, uint8_t *q, uint8_t *scales, int64_t R,
                                 int64_t K, bi_stream_t stream) {
  BI_TRY(check_mx4_dims("R", R, K));
  if (R == 0) return BI_OK;
  BI_TRY(check_rows("x", x, ldx, K));
  BI_REQUIRE(q && scales && aligned(q, 16) && aligned(scales, 16), BI_ERR_INVALID_ARG,
             "q and scales must be 16-byte aligned");
  return launch_mx4_quantize(x, x_f32 != 0, ldx, q, scales, R, K, reinterpret_cast<cudaStream_t>(stream));
}

BI_API bi_status bi_mx4_dequantize(const uint8_t *q, const uint8_t *scales, void *y, int32_t y_f32, int64_t ldy,
                                   int64_t R, int64_t K, bi_stream_t stream) {
  BI_TRY(check_mx4_dims("R", R, K));
  if (R == 0) return BI_OK;
  BI_TRY(check_rows("y", y, ldy, K));
  BI_REQUIRE(q && scales && aligned(q, 16) && aligned(scales, 16), BI_ERR_INVALID_ARG,
             "q and scales must be 16-byte aligned");
  return launch_mx4_dequantize(q, scales, y, y_f32 != 0, ldy, R, K, reinterpret_cast<cudaStream_t>(stream));
}

static bi_status mx4_product(const uint8_t *xq, const uint8_t *xs, const uint8_t *wq, const uint8_t *ws,
                             const bi_bf16 *addend, int64_t ld_addend, bi_bf16 *y, int64_t ldy, bool gated, int64_t M,
                             int64_t N, int64_t K, bi_stream_t stream) {
  BI_TRY(check_mx4_dims("M", M, K));
  BI_REQUIRE(N > 0, BI_ERR_INVALID_ARG, "bad size N=%lld", (long long)N);
  BI_REQUIRE(N <= (int64_t(1) << 22), BI_ERR_UNSUPPORTED, "N exceeds the index range (N=%lld)", (long long)N);
  if (M == 0) return BI_OK;
  BI_REQUIRE(xq && xs && wq && ws && y, BI_ERR_INVALID_ARG, "null pointer");
  BI_REQUIRE(aligned(xq, 16) && aligned(xs, 16) && aligned(wq, 16) && aligned(ws, 16), BI_ERR_INVALID_ARG,
             "codes and scales must be 16-byte aligned");
  const int64_t cols = gated ? N / 2 : N;
  BI_REQUIRE(ldy >= cols && ldy <= (int64_t(1) << 30), BI_ERR_INVALID_ARG, "row stride of y: %lld < %lld",
             (long long)ldy, (long long)cols);
  BI_REQUIRE(!addend || (ld_addend >= cols && ld_addend <= (int64_t(1) << 30)), BI_ERR_INVALID_ARG,
             "row stride of addend: %lld < %lld", (long long)ld_addend, (long long)cols);
  BI_REQUIRE(aligned(y, 2) && aligned(addend, 2), BI_ERR_INVALID_ARG, "y and addend must be 2-byte aligned");
  return launch_mx4_gemm(xq, xs, wq, ws, mat(addend, ld_addend), mbf(y), ldy, gated, M, N, K,
                         reinterpret_cast<cudaStream_t>(stream));
}

BI_API bi_status bi_mx4_gemm(const uint8_t *xq, const uint8_t *xs, const uint8_t *wq, const uint8_t *ws,
                             const bi_bf16 *addend, int64_t ld_addend, bi_bf16 *y, int64_t ldy, int64_t M, int64_t N,
                             int64_t K, bi_stream_t stream) {
  return mx4_product(xq, xs, wq, ws, addend, ld_addend, y, ldy, false, M, N, K, stream);
}

BI_API bi_status bi_mx4_gate_up(const uint8_t *xq, const uint8_t *xs, const uint8_t *w13q, const uint8_t *w13s,
                                bi_bf16 *act, int64_t ld_act, int64_t M, int64_t I, int64_t K, bi_stream_t stream) {
  BI_REQUIRE(I > 0, BI_ERR_INVALID_ARG, "bad size I=%lld", (long long)I);
  BI_REQUIRE(I % 16 == 0, BI_ERR_UNSUPPORTED, "I must be a multiple of 16 (I=%lld)", (long long)I);
  return mx4_product(xq, xs, w13q, w13s, nullptr, 0, act, ld_act, true, M, 2 * I, K, stream);
}

BI_API bi_status bi_mx4_form(int32_t mode, int32_t *previous) {
  BI_REQUIRE(mode >= 0 && mode <= 3, BI_ERR_INVALID_ARG, "4-bit product form %d not in {0, 1, 2, 3}", mode);
  const int old = bimoe::set_mx4_form(mode);
  if (previous) *previous = old;
  return BI_OK;
}

// ----------------------------------------- training a routed-experts layer --
static bi_status check_grouped(int64_t P, int64_t N, int64_t K, int64_t E, const int32_t *offsets) {
  BI_REQUIRE(P >= 0 && N > 0 && K > 0 && E > 0, BI_ERR_INVALID_ARG,
             "negative or zero size (P=%lld N=%lld K=%lld E=%lld)", (long long)P, (long long)N, (long long)K,
             (long long)E);
  BI_REQUIRE(N % 16 == 0 && K % 16 == 0, BI_ERR_UNSUPPORTED,
             "unsupported grouped product (needs N %% 16 == 0, K %% 16 == 0): N=%lld K=%lld", (long long)N, (long long)K);
  BI_REQUIRE(P <= (int64_t(1) << 30) && N <= (int64_t(1) << 20) && K <= (int64_t(1) << 20) && E <= 1024 &&
                 E * std::max(N, K) < (int64_t(1) << 31),
             BI_ERR_UNSUPPORTED, "grouped product sizes exceed the index range (P=%lld N=%lld K=%lld E=%lld)",
             (long long)P, (long long)N, (long long)K, (long long)E);
  BI_REQUIRE(P == 0 || offsets, BI_ERR_INVALID_ARG, "offsets is NULL");
  return BI_OK;
}

// y (or dx) = rows of x times the groups' matrices; out [P, cols_out], x [P, cols_in].
static bi_status grouped_rows(const char *in, const char *out, const bi_bf16 *x, int64_t ldx, const bi_bf16 *w, bool mn,
                              const int32_t *offsets, void *y, bool y_f32, int64_t ldy, int64_t P, int64_t cols_out,
                              int64_t cols_in, int64_t E, bi_stream_t stream) {
  if (P == 0) return BI_OK;
  BI_TRY(check_rows(in, x, ldx, cols_in));
  BI_TRY(check_rows(out, y, ldy, cols_out));
  BI_REQUIRE(w && aligned(w, 16), BI_ERR_INVALID_ARG, "w must be given and 16-byte aligned");
  const int64_t size = y_f32 ? 4 : 2, w_bytes = E * cols_out * cols_in * 2;
  BI_REQUIRE(!overlap_bytes(y, ldy * size, cols_out * size, x, ldx * 2, cols_in * 2, P), BI_ERR_INVALID_ARG,
             "%s and %s overlap", out, in);
  const uintptr_t y0 = reinterpret_cast<uintptr_t>(y), w0 = reinterpret_cast<uintptr_t>(w);
  BI_REQUIRE(y0 + static_cast<uintptr_t>(((P - 1) * ldy + cols_out) * size) <= w0 ||
                 w0 + static_cast<uintptr_t>(w_bytes) <= y0,
             BI_ERR_INVALID_ARG, "%s and w overlap", out);
  return launch_grouped_rows(mat(x, ldx), cbf(w), mn, Groups{offsets, static_cast<int>(E), static_cast<int>(P)}, y,
                             y_f32, ldy, cols_out, cols_in, reinterpret_cast<cudaStream_t>(stream));
}

BI_API bi_status bi_grouped_gemm(const bi_bf16 *x, int64_t ldx, const bi_bf16 *w, const int32_t *offsets, void *y,
                                 int32_t y_f32, int64_t ldy, int64_t P, int64_t N, int64_t K, int64_t E,
                                 bi_stream_t stream) {
  BI_TRY(check_grouped(P, N, K, E, offsets));
  return grouped_rows("x", "y", x, ldx, w, false, offsets, y, y_f32 != 0, ldy, P, N, K, E, stream);
}

BI_API bi_status bi_grouped_gemm_dx(const bi_bf16 *dy, int64_t lddy, const bi_bf16 *w, const int32_t *offsets, void *dx,
                                    int32_t dx_f32, int64_t lddx, int64_t P, int64_t N, int64_t K, int64_t E,
                                    bi_stream_t stream) {
  BI_TRY(check_grouped(P, N, K, E, offsets));
  return grouped_rows("dy", "dx", dy, lddy, w, true, offsets, dx, dx_f32 != 0, lddx, P, K, N, E, stream);
}

static size_t grad_size(int32_t grad_mode) { return grad_mode == kGradBf16 ? 2 : 4; }

// A gradient of `count` values over nothing: zero, or what it was.
static bi_status no_gradient(void *dw, int64_t count, int32_t grad_mode, cudaStream_t s) {
  if (!dw || grad_mode == kGradF32Accumulate) return BI_OK;
  const cudaError_t e = cudaMemsetAsync(dw, 0, static_cast<size_t>(count) * grad_size(grad_mode), s);
  BI_REQUIRE(e == cudaSuccess, BI_ERR_CUDA, "cudaMemsetAsync: %s", cudaGetErrorString(e));
  return BI_OK;
}

BI_API bi_status bi_grouped_gemm_dw(const bi_bf16 *dy, int64_t lddy, const bi_bf16 *x, int64_t ldx,
                                    const int32_t *offsets, void *dw, int32_t grad_mode, int64_t P, int64_t N,
                                    int64_t K, int64_t E, bi_stream_t stream) {
  BI_TRY(check_grouped(P, N, K, E, offsets));
  BI_REQUIRE(grad_mode >= 0 && grad_mode <= 2, BI_ERR_INVALID_ARG, "grad_mode %d not in {0, 1, 2}", grad_mode);
  BI_REQUIRE(dw && aligned(dw, 16), BI_ERR_INVALID_ARG, "dw must be given and 16-byte aligned");
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (P == 0) return no_gradient(dw, E * N * K, grad_mode, s);
  BI_TRY(check_rows("dy", dy, lddy, N));
  BI_TRY(check_rows("x", x, ldx, K));
  const int64_t bytes = E * N * K * static_cast<int64_t>(grad_size(grad_mode));
  const auto apart = [&](const void *p, int64_t ld, int64_t cols) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(dw), b = reinterpret_cast<uintptr_t>(p);
    return a + static_cast<uintptr_t>(bytes) <= b || b + static_cast<uintptr_t>(((P - 1) * ld + cols) * 2) <= a;
  };
  BI_REQUIRE(apart(dy, lddy, N) && apart(x, ldx, K), BI_ERR_INVALID_ARG, "dw overlaps dy or x");
  const GroupedDw d{mat(dy, lddy), mat(x, ldx), dw, N, K};
  return launch_grouped_dw(&d, 1, Groups{offsets, static_cast<int>(E), static_cast<int>(P)}, grad_mode, s);
}

// Workspace of the experts' training step: the forward and the backward pass use it in turn.
struct TrainWorkspace {
  size_t scratch, contrib, dout, dgu, parts, dwts, total;
};
static TrainWorkspace train_layout(int64_t M, int64_t H, int64_t E, int32_t top_k, int64_t I) {
  TrainWorkspace w{};
  const size_t P = static_cast<size_t>(M) * top_k;
  size_t off = 0;
  const auto take = [&](size_t bytes) {
    const size_t at = off;
    off += align256(bytes);
    return at;
  };
  w.contrib = take(P * H * sizeof(float));  // (one slot a token: for dx through the router only, which no size says)
  w.scratch = off;  // the forward's permutation; the backward's buffers take the same place
  const size_t scratch = align256(permute_scratch_bytes(M, E));
  w.dout = take(P * H * 2);
  w.dgu = take(P * 2 * I * 2);
  w.parts = take(P * (I / 32) * sizeof(float));
  w.dwts = take(P * sizeof(float));
  w.total = std::max<size_t>(256, std::max(off, w.scratch + scratch));
  return w;
}

BI_API size_t bi_moe_train_workspace_bytes(int64_t M, int64_t H, int64_t E, int32_t top_k, int64_t I) {
  if (check_moe_dims(M, H, E, top_k, I) != BI_OK) return 0;
  return train_layout(M, H, E, top_k, I).total;
}

BI_API bi_status bi_moe_forward_train(const bi_bf16 *x, const int32_t *ids, const float *wts, const bi_bf16 *w13,
                                      const bi_bf16 *w2, bi_bf16 *out, int32_t *offsets, int32_t *perm,
                                      uint32_t *slots, bi_bf16 *x_perm, float *gu, bi_bf16 *act, int64_t M, int64_t H,
                                      int64_t E, int32_t top_k, int64_t I, void *workspace, size_t workspace_bytes,
                                      bi_stream_t stream) {
  BI_TRY(check_moe_dims(M, H, E, top_k, I));
  if (M == 0) return BI_OK;
  BI_REQUIRE(x && ids && wts && w13 && w2 && out && offsets && perm && slots && x_perm && gu && act && workspace,
             BI_ERR_INVALID_ARG, "null pointer");
  BI_REQUIRE(aligned(x, 16) && aligned(w13, 16) && aligned(w2, 16) && aligned(out, 16) && aligned(x_perm, 16) &&
                 aligned(gu, 16) && aligned(act, 16) && aligned(workspace, 256),
             BI_ERR_INVALID_ARG, "misaligned pointer (x/w13/w2/out/x_perm/gu/act 16 B, workspace 256 B)");
  const TrainWorkspace L = train_layout(M, H, E, top_k, I);
  BI_REQUIRE(workspace_bytes >= L.total, BI_ERR_WORKSPACE, "workspace %zu < %zu bytes", workspace_bytes, L.total);
  const int64_t P = M * top_k;
  const Span results[] = {{"out", out, M * H * 2},      {"offsets", offsets, (E + 1) * 4}, {"perm", perm, P * 4},
                          {"slots", slots, M * 4},      {"x_perm", x_perm, P * H * 2},     {"gu", gu, P * 2 * I * 4},
                          {"act", act, P * I * 2}};
  const Span operands[] = {{"x", x, M * H * 2}, {"ids", ids, P * 4}, {"wts", wts, P * 4},
                           {"w13", w13, E * 2 * I * H * 2}, {"w2", w2, E * H * I * 2}};
  BI_TRY(check_apart(results, operands, x));
  char *ws = static_cast<char *>(workspace);
  float *contrib = reinterpret_cast<float *>(ws + L.contrib);
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const Groups g{offsets, static_cast<int>(E), static_cast<int>(P)};
  BI_TRY(launch_permute(ids, offsets, perm, M, E, top_k, ws + L.scratch, s, slots));
  // With one slot a token (the rows that an expert-parallel rank receives) nothing is summed: the down product's rows
  // are the result, rounded to bf16 where they are made (32768 rows, 32 groups,
  // H=4096, I=2048: forward 1335 us, without the separate sum 1145).
  const bool single = top_k == 1;
  BI_TRY(launch_train_gather(cbf(x), g, perm, mbf(x_perm), nullptr, single ? mbf(out) : nullptr, slots, H, top_k, s));
  BI_TRY(launch_train_gate_up(cbf(x_perm), g, perm, wts, cbf(w13), mbf(act), gu, H, I, s));
  if (single) return launch_train_down(cbf(act), g, perm, cbf(w2), mbf(out), H, I, s);
  BI_TRY(launch_down(act, offsets, perm, w2, contrib, P, H, E, top_k, I, s));
  return launch_combine(contrib, out, M, H, top_k, true, s, slots);
}

BI_API bi_status bi_moe_backward(const bi_bf16 *dout, const int32_t *ids, const float *wts, const bi_bf16 *w13,
                                 const bi_bf16 *w2, const int32_t *offsets, const int32_t *perm, const uint32_t *slots,
                                 const bi_bf16 *x_perm, const float *gu, const bi_bf16 *act, const float *w_router,
                                 bi_bf16 *dx, float *dwts, void *dw13, void *dw2, int32_t grad_mode, int64_t M,
                                 int64_t H, int64_t E, int32_t top_k, int64_t I, void *workspace,
                                 size_t workspace_bytes, bi_stream_t stream) {
  BI_TRY(check_moe_dims(M, H, E, top_k, I));
  BI_REQUIRE(grad_mode >= 0 && grad_mode <= 2, BI_ERR_INVALID_ARG, "grad_mode %d not in {0, 1, 2}", grad_mode);
  BI_REQUIRE(aligned(dw13, 16) && aligned(dw2, 16) && aligned(dx, 16), BI_ERR_INVALID_ARG,
             "dx, dw13 and dw2 must be 16-byte aligned");
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (M == 0) {
    BI_TRY(no_gradient(dw13, E * 2 * I * H, grad_mode, s));
    return no_gradient(dw2, E * H * I, grad_mode, s);
  }
  if (!dx && !dwts && !dw13 && !dw2) return BI_OK;
  BI_REQUIRE(dout && ids && wts && w13 && w2 && offsets && perm && slots && x_perm && gu && act && workspace,
             BI_ERR_INVALID_ARG, "null pointer");
  BI_REQUIRE(aligned(dout, 16) && aligned(w13, 16) && aligned(w2, 16) && aligned(x_perm, 16) && aligned(gu, 16) &&
                 aligned(act, 16) && aligned(w_router, 16) && aligned(workspace, 256),
             BI_ERR_INVALID_ARG, "misaligned pointer (dout/w13/w2/x_perm/gu/act/w_router 16 B, workspace 256 B)");
  const TrainWorkspace L = train_layout(M, H, E, top_k, I);
  BI_REQUIRE(workspace_bytes >= L.total, BI_ERR_WORKSPACE, "workspace %zu < %zu bytes", workspace_bytes, L.total);
  // dwts is set to zero first and dx may be; dw13 and dw2 come last, when only what is named here is still read
  const int64_t P = M * top_k, grad = static_cast<int64_t>(grad_size(grad_mode));
  const Span rows[] = {{"dx", dx, M * H * 2}, {"dwts", dwts, P * 4}};
  const Span all[] = {{"dout", dout, M * H * 2},     {"ids", ids, P * 4},
                      {"wts", wts, P * 4},           {"w13", w13, E * 2 * I * H * 2},
                      {"w2", w2, E * H * I * 2},     {"offsets", offsets, (E + 1) * 4},
                      {"perm", perm, P * 4},         {"slots", slots, M * 4},
                      {"x_perm", x_perm, P * H * 2}, {"gu", gu, P * 2 * I * 4},
                      {"act", act, P * I * 2},       {"w_router", w_router, E * H * 4}};
  const Span weights[] = {{"dw13", dw13, E * 2 * I * H * grad}, {"dw2", dw2, E * H * I * grad}};
  const Span late[] = {all[5], all[8], all[10], rows[0], rows[1]};
  BI_TRY(check_apart(rows, all, dout));
  BI_TRY(check_apart(weights, late));
  char *ws = static_cast<char *>(workspace);
  float *contrib = reinterpret_cast<float *>(ws + L.contrib), *parts = reinterpret_cast<float *>(ws + L.parts);
  __nv_bfloat16 *dout_perm = mbf(ws + L.dout), *dgu = mbf(ws + L.dgu);
  const Groups g{offsets, static_cast<int>(E), static_cast<int>(P)};
  const bool through_router = dx && w_router;
  if (through_router && !dwts) dwts = reinterpret_cast<float *>(ws + L.dwts);
  const bool single = dx && top_k == 1 && !through_router;  // as in the forward pass
  BI_TRY(launch_train_gather(cbf(dout), g, perm, dout_perm, dwts, single ? mbf(dx) : nullptr, slots, H, top_k, s));
  const DwtsSum sum{parts, static_cast<int>(I / 32), g, perm, dwts};
  const bool sum_beside = dx && !single && !through_router;  // in the launch that sums dx
  if (dx || dwts || dw13) {
    BI_TRY(launch_train_dact(dout_perm, g, perm, wts, cbf(w2), gu, dgu, dwts ? parts : nullptr, H, I, s));
    if (dwts && !sum_beside) BI_TRY(launch_dwts(sum, s));
  }
  if (single) {
    BI_TRY(launch_train_dx(dgu, g, perm, cbf(w13), dx, false, H, I, s));
  } else if (dx) {
    BI_TRY(launch_train_dx(dgu, g, perm, cbf(w13), contrib, true, H, I, s));
    BI_TRY(launch_grad_combine(GradCombine{contrib, slots, ids, wts, dwts, through_router ? w_router : nullptr, dx,
                                           false, M, H, static_cast<int>(E), top_k, false},
                               dwts && sum_beside ? &sum : nullptr, s));
  }
  GroupedDw d[2];
  int count = 0;
  if (dw13) d[count++] = GroupedDw{Mat{dgu, 2 * I}, mat(x_perm, H), dw13, 2 * I, H};
  if (dw2) d[count++] = GroupedDw{Mat{dout_perm, H}, mat(act, I), dw2, H, I};
  return count ? launch_grouped_dw(d, count, g, grad_mode, s) : BI_OK;
}

BI_API bi_status bi_router_backward(const float *dwts, const int32_t *ids, const float *wts, const void *x,
                                    int32_t x_f32, const float *w, const int32_t *offsets, const int32_t *perm,
                                    void *dx, float *dw, float *dbias, int32_t accumulate, int64_t M, int64_t H,
                                    int64_t E, int32_t top_k, bi_stream_t stream) {
  BI_REQUIRE(M >= 0 && H > 0 && E > 0, BI_ERR_INVALID_ARG, "negative or zero size (M=%lld H=%lld E=%lld)", (long long)M,
             (long long)H, (long long)E);
  BI_REQUIRE(top_k >= 1 && top_k <= 16 && top_k <= E, BI_ERR_INVALID_ARG, "top_k=%d outside [1, min(16, E)]", top_k);
  BI_REQUIRE(E <= 1024 && H % 8 == 0 && H <= (int64_t(1) << 20) && M * top_k < (int64_t(1) << 31), BI_ERR_UNSUPPORTED,
             "unsupported router gradient (needs H %% 8 == 0, E <= 1024): M=%lld H=%lld E=%lld", (long long)M,
             (long long)H, (long long)E);
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (M == 0) {
    const int32_t mode = accumulate ? kGradF32Accumulate : kGradF32;
    BI_TRY(no_gradient(dw, E * H, mode, s));
    return no_gradient(dbias, E, mode, s);
  }
  if (!dx && !dw && !dbias) return BI_OK;
  BI_REQUIRE(dwts && ids && wts && (x || !dw) && (w || !dx) && ((offsets && perm) || (!dw && !dbias)),
             BI_ERR_INVALID_ARG, "null pointer");
  BI_REQUIRE(aligned(x, 16) && aligned(w, 16) && aligned(dx, 16), BI_ERR_INVALID_ARG,
             "x, w and dx must be 16-byte aligned");
  // dw is summed while dx is stored; dx alone may be x, and dw alone w
  const int64_t slots = M * top_k * 4, x_bytes = M * H * (x_f32 ? 4 : 2), w_bytes = E * H * 4;
  const Span results[] = {{"dx", dx, x_bytes}, {"dw", dw, w_bytes}, {"dbias", dbias, E * 4}};
  const Span operands[] = {{"dwts", dwts, slots},     {"ids", ids, slots},
                           {"wts", wts, slots},       {"x", dw ? x : nullptr, x_bytes},
                           {"w", dx ? w : nullptr, w_bytes},
                           {"offsets", dw || dbias ? offsets : nullptr, (E + 1) * 4},
                           {"perm", dw || dbias ? perm : nullptr, slots}};
  BI_TRY(check_apart(results, operands));
  const GradCombine c{nullptr, nullptr, ids, wts, dwts, w, dx, x_f32 != 0, M, H, static_cast<int>(E), top_k,
                      dw || dbias};
  if (dx) BI_TRY(launch_grad_combine(c, nullptr, s));
  if (!dw && !dbias) return BI_OK;
  return launch_router_dw(dwts, wts, x, x_f32 != 0, Groups{offsets, static_cast<int>(E), static_cast<int>(M * top_k)},
                          perm, dw, dbias, accumulate != 0, dx && grad_combine_stages(c), H, top_k, s);
}

static bi_status check_norm(int64_t M, int64_t H) {
  BI_REQUIRE(M >= 0 && H > 0, BI_ERR_INVALID_ARG, "negative or zero size (M=%lld H=%lld)", (long long)M, (long long)H);
  BI_REQUIRE(H <= 16384 && M <= (int64_t(1) << 30), BI_ERR_UNSUPPORTED,
             "unsupported norm (needs H <= 16384, M <= 2^30): M=%lld H=%lld", (long long)M, (long long)H);
  return BI_OK;
}
// An array against the `rows` rows of a matrix, `bytes` each, every ld bytes.
static bool meets_rows(const Span &a, const void *m, int64_t ld, int64_t bytes, int64_t rows) {
  const uintptr_t p = reinterpret_cast<uintptr_t>(a.p), q = reinterpret_cast<uintptr_t>(m);
  if (!p || !spans_meet(a, Span{"", m, (rows - 1) * ld + bytes})) return false;
  const int64_t from = p > q ? static_cast<int64_t>(p - q) : 0, to = static_cast<int64_t>(p + a.bytes - q);
  return from % ld < bytes || (from / ld + 1) * ld < to;  // in its row, or reaching into the next
}
static bi_status check_norm_rows(const char *name, const void *p, int64_t ld, int64_t H, int32_t f32) {
  BI_REQUIRE(p, BI_ERR_INVALID_ARG, "%s is NULL", name);
  BI_REQUIRE(aligned(p, f32 ? 4 : 2), BI_ERR_INVALID_ARG, "%s must be aligned to its type", name);
  BI_REQUIRE(ld >= H && ld <= (int64_t(1) << 30), BI_ERR_INVALID_ARG, "row stride of %s: %lld (needs at least %lld)",
             name, (long long)ld, (long long)H);
  return BI_OK;
}

BI_API bi_status bi_layer_norm(const void *x, int32_t x_f32, int64_t ldx, const void *weight, const void *bias,
                               int32_t p_f32, float eps, void *y, int64_t ldy, float *mean, float *rstd, int64_t M,
                               int64_t H, bi_stream_t stream) {
  BI_TRY(check_norm(M, H));
  BI_REQUIRE(eps >= 0.0f, BI_ERR_INVALID_ARG, "eps must not be negative");
  if (M == 0) return BI_OK;
  BI_TRY(check_norm_rows("x", x, ldx, H, x_f32));
  BI_TRY(check_norm_rows("y", y, ldy, H, x_f32));
  BI_REQUIRE(aligned(weight, p_f32 ? 4 : 2) && aligned(bias, p_f32 ? 4 : 2) && aligned(mean, 4) && aligned(rstd, 4),
             BI_ERR_INVALID_ARG, "weight, bias, mean and rstd must be aligned to their type");
  const int64_t size = x_f32 ? 4 : 2;
  BI_REQUIRE((x == y && ldx == ldy) || !overlap_bytes(x, ldx * size, H * size, y, ldy * size, H * size, M),
             BI_ERR_INVALID_ARG, "x and y overlap (y may be x, with the same stride)");
  const Span params[] = {{"weight", weight, H * (p_f32 ? 4 : 2)}, {"bias", bias, H * (p_f32 ? 4 : 2)}};
  const Span stats[] = {{"mean", mean, M * 4}, {"rstd", rstd, M * 4}};
  BI_TRY(check_apart(stats, params));
  for (const Span &a : {params[0], params[1], stats[0], stats[1]})
    BI_REQUIRE(!meets_rows(a, y, ldy * size, H * size, M), BI_ERR_INVALID_ARG, "y overlaps %s", a.name);
  for (const Span &a : stats)
    BI_REQUIRE(!meets_rows(a, x, ldx * size, H * size, M), BI_ERR_INVALID_ARG, "%s overlaps x", a.name);
  return launch_layer_norm(x, x_f32 != 0, ldx, weight, bias, p_f32 != 0, eps, y, ldy, mean, rstd, M, H,
                           reinterpret_cast<cudaStream_t>(stream));
}

BI_API size_t bi_layer_norm_workspace_bytes(int64_t M, int64_t H) {
  if (check_norm(M, H) != BI_OK) return 0;
  return std::max<size_t>(256, align256(layer_norm_workspace_bytes(M, H)));
}

BI_API bi_status bi_layer_norm_backward(const void *dy, int64_t lddy, const void *x, int32_t x_f32, int64_t ldx,
                                        const void *weight, int32_t p_f32, const float *mean, const float *rstd,
                                        void *dx, int64_t lddx, float *dweight, float *dbias, int32_t accumulate,
                                        int64_t M, int64_t H, void *workspace, size_t workspace_bytes,
                                        bi_stream_t stream) {
  BI_TRY(check_norm(M, H));
  BI_REQUIRE(aligned(dweight, 4) && aligned(dbias, 4) && aligned(mean, 4) && aligned(rstd, 4) &&
                 aligned(weight, p_f32 ? 4 : 2),
             BI_ERR_INVALID_ARG, "weight, mean, rstd, dweight and dbias must be aligned to their type");
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (M == 0) {
    const int32_t mode = accumulate ? kGradF32Accumulate : kGradF32;
    BI_TRY(no_gradient(dweight, H, mode, s));
    return no_gradient(dbias, H, mode, s);
  }
  if (!dx && !dweight && !dbias) return BI_OK;
  BI_TRY(check_norm_rows("dy", dy, lddy, H, x_f32));
  BI_TRY(check_norm_rows("x", x, ldx, H, x_f32));
  BI_REQUIRE(mean && rstd, BI_ERR_INVALID_ARG, "null pointer");
  if (dx) {
    BI_TRY(check_norm_rows("dx", dx, lddx, H, x_f32));
    const int64_t size = x_f32 ? 4 : 2;
    BI_REQUIRE(((dx == dy && lddx == lddy) || !overlap_bytes(dx, lddx * size, H * size, dy, lddy * size, H * size, M)) &&
                   ((dx == x && lddx == ldx) || !overlap_bytes(dx, lddx * size, H * size, x, ldx * size, H * size, M)),
               BI_ERR_INVALID_ARG, "dx overlaps dy or x (it may be either, with the same stride)");
    for (const Span &a : {Span{"weight", weight, H * (p_f32 ? 4 : 2)}, Span{"mean", mean, M * 4},
                          Span{"rstd", rstd, M * 4}, Span{"dweight", dweight, H * 4}, Span{"dbias", dbias, H * 4}})
      BI_REQUIRE(!meets_rows(a, dx, lddx * size, H * size, M), BI_ERR_INVALID_ARG, "dx overlaps %s", a.name);
  }
  // (dweight and dbias are written when everything has been read)
  BI_REQUIRE(!spans_meet(Span{"dweight", dweight, H * 4}, Span{"dbias", dbias, H * 4}), BI_ERR_INVALID_ARG,
             "dweight and dbias overlap");
  if (dweight || dbias) {
    const size_t need = layer_norm_workspace_bytes(M, H);
    BI_REQUIRE(workspace && aligned(workspace, 16), BI_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
    BI_REQUIRE(workspace_bytes >= need, BI_ERR_WORKSPACE, "workspace %zu < %zu bytes", workspace_bytes, need);
  }
  return launch_layer_norm_backward(dy, lddy, x, x_f32 != 0, ldx, weight, p_f32 != 0, mean, rstd, dx, lddx, dweight,
                                    dbias, accumulate != 0, static_cast<float *>(workspace), M, H, s);
}

}  // extern "C"
