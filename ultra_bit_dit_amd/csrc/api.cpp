// C ABI of liblowbit: argument validation, dispatch and the per-stream
// workspace.  Every check runs on the host before any HIP call.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <map>
#include <numeric>
#include <mutex>
#include <utility>
#include <initializer_list>
#include <vector>

#include "../../include/lowbit.h"
#include "common.hpp"
#include "kv8.hpp"

using namespace lowbit;

namespace {

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

bool valid_fmt(int fmt) {
  return fmt == LOWBIT_BINARY || fmt == LOWBIT_TERNARY_2BIT || fmt == LOWBIT_TERNARY_BASE3;
}

// N * K and derived sizes must stay far from int64 overflow
bool shape_ok(int64_t N, int64_t K) {
  if (N < 1 || K < 1 || K % kGroup != 0) return false;
  if (N > (int64_t(1) << 40) || K > (int64_t(1) << 40)) return false;
  if (N > (int64_t(1) << 62) / K) return false;
  return true;
}

int hip_status(hipError_t e) { return e == hipSuccess ? LOWBIT_OK : LOWBIT_E_HIP; }

// ---- per-(device, stream) workspace, grown on demand.  A grown workspace
// serves the stream's later calls; the smaller one it replaces is retired,
// not freed, because kernels queued before the growth, and HIP graphs
// captured on the stream, may still use it.  Nothing waits for the stream.
// A stream being captured cannot grow its workspace (reserve it first).
// Retired and current workspaces are freed by lowbit_release_workspaces.
// The first kCounterBytes of a workspace hold the kernels' arrival counters
// (zeroed on the stream when the workspace is allocated; every launch leaves
// them zero).
struct Workspace {
  void* ptr = nullptr;
  size_t bytes = 0;
};
std::mutex g_ws_mutex;
std::map<std::pair<int, hipStream_t>, Workspace> g_ws;
std::vector<std::pair<int, void*>> g_retired;  // (device, workspace)

int workspace(hipStream_t s, size_t need, void** out) {
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess) return LOWBIT_E_HIP;
  std::lock_guard<std::mutex> lock(g_ws_mutex);
  Workspace& w = g_ws[{dev, s}];
  if (w.bytes < need) {
    hipStreamCaptureStatus cs = hipStreamCaptureStatusNone;
    if (hipStreamIsCapturing(s, &cs) != hipSuccess) return LOWBIT_E_HIP;
    if (cs != hipStreamCaptureStatusNone) return LOWBIT_E_NOMEM;
    const size_t sz = need < (1u << 20) ? (1u << 20) : need + need / 4;
    void* p = nullptr;
    if (hipMalloc(&p, sz) != hipSuccess) return LOWBIT_E_NOMEM;
    // the counter block must start at zero; kernels leave it zero
    if (hipMemsetAsync(p, 0, kCounterBytes, s) != hipSuccess) {
      (void)hipFree(p);
      return LOWBIT_E_HIP;
    }
    if (w.ptr) g_retired.push_back({dev, w.ptr});
    w.ptr = p;
    w.bytes = sz;
  }
  *out = w.ptr;
  return LOWBIT_OK;
}

size_t align_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

// ---- the allocation-free GEMV's scratch: one static device array per GPU,
// shared by every lowbit_gemv_noalloc call on that GPU.  Host code uses only
// the device address hipGetSymbolAddress returns for the current device
// (taken once per device, under g_scratch_mutex); the array's name on the
// host is not a device address.  Its first kCounterBytes hold the fused
// GEMV's arrival counters: zero when the code object is loaded (static
// storage), cleared again by a fill kernel on the first call's stream, and
// left zero by every launch.
constexpr size_t kScratchBytes = size_t(4) << 20;
static __device__ __align__(256) uint8_t scratch[kScratchBytes];
static_assert(kScratchBytes >= (size_t)kCounterBytes, "counters must fit the scratch");

__global__ void fill_zero_u32(uint32_t* p, int64_t n) {
  for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < n;
       i += (int64_t)gridDim.x * blockDim.x)
    p[i] = 0u;
}

std::mutex g_scratch_mutex;
std::map<int, void*> g_scratch;  // device -> address of `scratch` on it

int scratch_for_device(hipStream_t s, void** out) {
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess) return LOWBIT_E_HIP;
  std::lock_guard<std::mutex> lock(g_scratch_mutex);
  auto it = g_scratch.find(dev);
  if (it == g_scratch.end()) {
    void* ptr = nullptr;
    if (hipGetSymbolAddress(&ptr, HIP_SYMBOL(scratch)) != hipSuccess || !ptr) return LOWBIT_E_HIP;
    hipLaunchKernelGGL(fill_zero_u32, dim3(64), dim3(256), 0, s, (uint32_t*)ptr,
                       (int64_t)(kCounterBytes / 4));
    if (hipGetLastError() != hipSuccess) return LOWBIT_E_HIP;
    it = g_scratch.emplace(dev, ptr).first;
  }
  *out = it->second;
  return LOWBIT_OK;
}

// small-M product through the fused MFMA GEMV kernel (M * R <= 16 rows of A)
// with the workspace `ws` (counters first, zero)
int gemv_mfma_ws(int fmt, int64_t M, int64_t N, int64_t K, const void* pcodes,
                 const void* pscales, int x_dtype, const void* x, float x_scale,
                 const float* x_scales, int y_dtype, void* y, void* ws, hipStream_t s) {
  GemvArgs g;
  g.fmt = fmt;
  g.N = N;
  g.K = K;
  g.M = M;
  g.pcodes = pcodes;
  g.pscales = (const uint16_t*)pscales;
  g.xkind = x_dtype;
  g.x = x;
  g.x_scale = (x_dtype == LOWBIT_I8) ? x_scale : 1.0f;
  g.x_scales = x_scales;
  g.ykind = y_dtype;
  g.y = y;
  g.ws = ws;
  return hip_status(launch_gemv_mfma(g, s));
}

int run_gemv_mfma(int fmt, int64_t M, int64_t N, int64_t K, const void* pcodes,
                  const void* pscales, int x_dtype, const void* x, float x_scale,
                  const float* x_scales, int y_dtype, void* y, hipStream_t s) {
  if (cdiv(N, 16) > kMaxRowGroups) return LOWBIT_E_SHAPE;
  void* ws = nullptr;
  int rc = workspace(s, gemv_workspace_bytes(fmt, N, K, M, x_dtype), &ws);
  if (rc) return rc;
  return gemv_mfma_ws(fmt, M, N, K, pcodes, pscales, x_dtype, x, x_scale, x_scales, y_dtype, y,
                      ws, s);
}

// large-M product through the staged-tile MFMA GEMM
int run_gemm(int fmt, int64_t M, int64_t N, int64_t K, const void* pcodes, const void* pscales,
             int x_dtype, const void* X, const float* x_scales, int y_dtype, void* Y,
             hipStream_t s) {
  if (cdiv(N, 16) > (int64_t(1) << 40) / 16) return LOWBIT_E_SHAPE;
  void* ws = nullptr;
  int rc = workspace(s, gemm_workspace_bytes(fmt, x_dtype, M, N, K), &ws);
  if (rc) return rc;
  GemmArgs g;
  g.fmt = fmt;
  g.M = M;
  g.N = N;
  g.K = K;
  g.pcodes = pcodes;
  g.pscales = (const uint16_t*)pscales;
  g.xkind = x_dtype;
  g.x = X;
  g.x_scales = x_dtype != LOWBIT_BF16 && y_dtype != LOWBIT_I32 ? x_scales : nullptr;
  g.ykind = y_dtype;
  g.y = Y;
  g.ws = ws;
  return hip_status(launch_gemm(g, s));
}

// activation rows the batch-1 kernels take at once: 16 rows of A over the
// split terms of one row
int max_small_m(int fmt, int x_dtype) { return 16 / split_terms(fmt, x_dtype); }

// Workspace bytes a product needs: the path lowbit_gemm (or lowbit_gemv when
// M = 1) takes for these arguments.  Sign activations: the GEMM's need (the
// batch-1 sign GEMV of lowbit_gemv uses none, so this bounds both).
size_t product_workspace(int fmt, int64_t M, int64_t N, int64_t K, int x_dtype) {
  if (x_dtype != LOWBIT_SIGN1 && M <= max_small_m(fmt, x_dtype))
    return gemv_workspace_bytes(fmt, N, K, M, x_dtype);
  return gemm_workspace_bytes(fmt, x_dtype, M, N, K);
}

}  // namespace

extern "C" {

int lowbit_abi_version(void) { return LOWBIT_ABI_VERSION; }

const char* lowbit_status_str(int status) {
  switch (status) {
    case LOWBIT_OK: return "ok";
    case LOWBIT_E_NULL: return "null pointer";
    case LOWBIT_E_SHAPE: return "invalid shape (K must be a positive multiple of 128)";
    case LOWBIT_E_ALIGN: return "misaligned pointer";
    case LOWBIT_E_UNSUPPORTED: return "unsupported format / dtype combination";
    case LOWBIT_E_BADCODE: return "invalid code";
    case LOWBIT_E_HIP: return "HIP runtime error";
    case LOWBIT_E_NOMEM: return "workspace allocation failed (or needed growth during graph capture)";
    case LOWBIT_E_TOO_LARGE: return "product needs more scratch than the allocation-free call holds";
  }
  return "unknown status";
}

int lowbit_packed_bytes(int fmt, int64_t N, int64_t K, size_t* code_bytes, size_t* scale_bytes) {
  if (!code_bytes || !scale_bytes) return LOWBIT_E_NULL;
  if (!valid_fmt(fmt)) return LOWBIT_E_UNSUPPORTED;
  if (!shape_ok(N, K)) return LOWBIT_E_SHAPE;
  int64_t NB = cdiv(N, 16), G = K / kGroup;
  int64_t c = fmt == LOWBIT_BINARY ? NB * cdiv(G, 4) * 1024
              : fmt == LOWBIT_TERNARY_2BIT ? NB * cdiv(G, 2) * 1024
                                           : NB * cdiv(G, 8) * 3328;
  *code_bytes = (size_t)c;
  *scale_bytes = (size_t)(NB * cdiv(G, 4) * 128);
  return LOWBIT_OK;
}

int lowbit_pack(int fmt, int64_t N, int64_t K, const int8_t* codes, const uint16_t* scales,
                void* pcodes, void* pscales, int32_t* bad_code_count, void* stream) {
  if (!codes || !scales || !pcodes || !pscales) return LOWBIT_E_NULL;
  if (!valid_fmt(fmt)) return LOWBIT_E_UNSUPPORTED;
  if (!shape_ok(N, K)) return LOWBIT_E_SHAPE;
  if (!aligned(pcodes, 16) || !aligned(pscales, 16) || !aligned(scales, 2) ||
      (bad_code_count && !aligned(bad_code_count, 4)))
    return LOWBIT_E_ALIGN;
  return hip_status(launch_pack(fmt, N, K, codes, scales, pcodes, pscales, bad_code_count,
                                (hipStream_t)stream));
}

int lowbit_unpack(int fmt, int64_t N, int64_t K, const void* pcodes, const void* pscales,
                  int8_t* codes, uint16_t* scales, int32_t* bad_code_count, void* stream) {
  if (!codes || !scales || !pcodes || !pscales) return LOWBIT_E_NULL;
  if (!valid_fmt(fmt)) return LOWBIT_E_UNSUPPORTED;
  if (!shape_ok(N, K)) return LOWBIT_E_SHAPE;
  if (!aligned(pcodes, 16) || !aligned(pscales, 16) || !aligned(scales, 2) ||
      (bad_code_count && !aligned(bad_code_count, 4)))
    return LOWBIT_E_ALIGN;
  return hip_status(launch_unpack(fmt, N, K, pcodes, pscales, codes, scales, bad_code_count,
                                  (hipStream_t)stream));
}

int lowbit_quantize_act_i8(int64_t M, int64_t K, const uint16_t* X_bf16, int8_t* Q, float* s_x,
                           void* stream) {
  if (!X_bf16 || !Q || !s_x) return LOWBIT_E_NULL;
  if (M < 1 || K < 1 || M > (int64_t(1) << 31) || K > (int64_t(1) << 40)) return LOWBIT_E_SHAPE;
  if (!aligned(X_bf16, 2) || !aligned(s_x, 4)) return LOWBIT_E_ALIGN;
  return hip_status(launch_quantize_i8(M, K, X_bf16, Q, s_x, (hipStream_t)stream));
}

namespace {

// argument checks of lowbit_gemv (and its allocation-free variant)
int gemv_check(int fmt, int64_t N, int64_t K, const void* pcodes, const void* pscales,
               int x_dtype, const void* x, int y_dtype, void* y) {
  if (!pcodes || !x || !y) return LOWBIT_E_NULL;
  if (!valid_fmt(fmt)) return LOWBIT_E_UNSUPPORTED;
  if (!shape_ok(N, K)) return LOWBIT_E_SHAPE;
  const bool int_x = x_dtype == LOWBIT_I8 || x_dtype == LOWBIT_SIGN1;
  if (x_dtype < LOWBIT_F32 || x_dtype > LOWBIT_SIGN1) return LOWBIT_E_UNSUPPORTED;
  if (y_dtype != LOWBIT_F32 && y_dtype != LOWBIT_BF16 && y_dtype != LOWBIT_I32)
    return LOWBIT_E_UNSUPPORTED;
  if (y_dtype == LOWBIT_I32 && !(int_x && pscales == nullptr)) return LOWBIT_E_UNSUPPORTED;
  if (y_dtype != LOWBIT_I32 && !pscales) return LOWBIT_E_NULL;
  if (x_dtype == LOWBIT_SIGN1 && fmt != LOWBIT_BINARY) return LOWBIT_E_UNSUPPORTED;
  if (!aligned(pcodes, 16) || (pscales && !aligned(pscales, 16)) || !aligned(x, 16) ||
      !aligned(y, 4))
    return LOWBIT_E_ALIGN;
  if (x_dtype == LOWBIT_SIGN1 && K > kSignMaxK) return LOWBIT_E_SHAPE;  // sign words in LDS
  if (x_dtype != LOWBIT_SIGN1 && cdiv(N, 16) > kMaxRowGroups) return LOWBIT_E_SHAPE;
  return LOWBIT_OK;
}

int gemv_sign(int64_t N, int64_t K, const void* pcodes, const void* pscales, const void* x,
              float x_scale, int y_dtype, void* y, hipStream_t s) {
  SignArgs a;
  a.N = N;
  a.K = K;
  a.M = 1;
  a.pcodes = pcodes;
  a.pscales = (const uint16_t*)pscales;
  a.xbits = (const uint8_t*)x;
  a.alpha = x_scale;
  a.ykind = y_dtype;
  a.y = y;
  return hip_status(launch_gemv_sign(a, s));
}

}  // namespace

int lowbit_gemv(int fmt, int64_t N, int64_t K, const void* pcodes, const void* pscales,
                int x_dtype, const void* x, float x_scale, int y_dtype, void* y, void* stream) {
  const int rc = gemv_check(fmt, N, K, pcodes, pscales, x_dtype, x, y_dtype, y);
  if (rc) return rc;
  hipStream_t s = (hipStream_t)stream;
  if (x_dtype == LOWBIT_SIGN1) return gemv_sign(N, K, pcodes, pscales, x, x_scale, y_dtype, y, s);
  return run_gemv_mfma(fmt, 1, N, K, pcodes, pscales, x_dtype, x, x_scale, nullptr, y_dtype, y,
                       s);
}

int lowbit_gemv_noalloc(int fmt, int64_t N, int64_t K, const void* pcodes, const void* pscales,
                        int x_dtype, const void* x, float x_scale, int y_dtype, void* y,
                        void* stream) {
  const int rc = gemv_check(fmt, N, K, pcodes, pscales, x_dtype, x, y_dtype, y);
  if (rc) return rc;
  hipStream_t s = (hipStream_t)stream;
  if (x_dtype == LOWBIT_SIGN1) return gemv_sign(N, K, pcodes, pscales, x, x_scale, y_dtype, y, s);
  if (gemv_workspace_bytes(fmt, N, K, 1, x_dtype) > kScratchBytes) return LOWBIT_E_TOO_LARGE;
  void* ws = nullptr;
  const int r2 = scratch_for_device(s, &ws);
  if (r2) return r2;
  return gemv_mfma_ws(fmt, 1, N, K, pcodes, pscales, x_dtype, x, x_scale, nullptr, y_dtype, y, ws,
                      s);
}

int lowbit_gemm(int fmt, int64_t M, int64_t N, int64_t K, const void* pcodes, const void* pscales,
                int x_dtype, const void* X, const float* x_scales, int y_dtype, void* Y,
                void* stream) {
  if (!pcodes || !X || !Y) return LOWBIT_E_NULL;
  if (!valid_fmt(fmt)) return LOWBIT_E_UNSUPPORTED;
  if (!shape_ok(N, K) || M < 1 || M > (int64_t(1) << 31)) return LOWBIT_E_SHAPE;
  if (K > (int64_t(1) << 36)) return LOWBIT_E_SHAPE;  // 32-bit group indices of the GEMM
  const bool sign = x_dtype == LOWBIT_SIGN1;
  if (x_dtype != LOWBIT_BF16 && x_dtype != LOWBIT_I8 && !sign) return LOWBIT_E_UNSUPPORTED;
  if (y_dtype != LOWBIT_F32 && y_dtype != LOWBIT_BF16 && y_dtype != LOWBIT_I32)
    return LOWBIT_E_UNSUPPORTED;
  if (y_dtype == LOWBIT_I32 && !((x_dtype == LOWBIT_I8 || sign) && pscales == nullptr))
    return LOWBIT_E_UNSUPPORTED;
  if (y_dtype != LOWBIT_I32 && !pscales) return LOWBIT_E_NULL;
  if ((x_dtype == LOWBIT_I8 || sign) && y_dtype != LOWBIT_I32 && !x_scales) return LOWBIT_E_NULL;
  if (!aligned(pcodes, 16) || (pscales && !aligned(pscales, 16)) || !aligned(X, 16) ||
      !aligned(Y, 16) || (x_scales && !aligned(x_scales, 4)))
    return LOWBIT_E_ALIGN;
  hipStream_t s = (hipStream_t)stream;
  if (!sign && M <= max_small_m(fmt, x_dtype))
    return run_gemv_mfma(fmt, M, N, K, pcodes, pscales, x_dtype, X, 1.0f,
                         x_dtype == LOWBIT_I8 && y_dtype != LOWBIT_I32 ? x_scales : nullptr,
                         y_dtype, Y, s);
  return run_gemm(fmt, M, N, K, pcodes, pscales, x_dtype, X, x_scales, y_dtype, Y, s);
}

int lowbit_workspace_bytes(int fmt, int64_t M, int64_t N, int64_t K, int x_dtype, size_t* bytes) {
  if (!bytes) return LOWBIT_E_NULL;
  *bytes = 0;
  if (!valid_fmt(fmt)) return LOWBIT_E_UNSUPPORTED;
  if (x_dtype < LOWBIT_F32 || x_dtype > LOWBIT_SIGN1) return LOWBIT_E_UNSUPPORTED;
  if (!shape_ok(N, K) || M < 1 || M > (int64_t(1) << 31) || K > (int64_t(1) << 36))
    return LOWBIT_E_SHAPE;
  if (M > 1 && x_dtype == LOWBIT_F32) return LOWBIT_E_UNSUPPORTED;  // lowbit_gemm takes no F32
  *bytes = product_workspace(fmt, M, N, K, x_dtype);
  return LOWBIT_OK;
}

int lowbit_reserve_workspace(size_t bytes, void* stream) {
  void* ws = nullptr;
  return workspace((hipStream_t)stream, bytes, &ws);
}

int lowbit_release_workspaces(void) {
  std::lock_guard<std::mutex> lock(g_ws_mutex);
  int rc = LOWBIT_OK;
  int cur = 0;
  if (!g_ws.empty() || !g_retired.empty())
    if (hipGetDevice(&cur) != hipSuccess) return LOWBIT_E_HIP;
  std::vector<int> devs;
  for (auto& kv : g_ws) devs.push_back(kv.first.first);
  for (auto& r : g_retired) devs.push_back(r.first);
  std::sort(devs.begin(), devs.end());
  devs.erase(std::unique(devs.begin(), devs.end()), devs.end());
  for (int d : devs)  // queued kernels may still use a workspace
    if (hipSetDevice(d) != hipSuccess || hipDeviceSynchronize() != hipSuccess) rc = LOWBIT_E_HIP;
  auto release = [&](int dev, void* p) {
    if (hipSetDevice(dev) != hipSuccess || hipFree(p) != hipSuccess) rc = LOWBIT_E_HIP;
  };
  for (auto& kv : g_ws)
    if (kv.second.ptr) release(kv.first.first, kv.second.ptr);
  for (auto& r : g_retired) release(r.first, r.second);
  g_ws.clear();
  g_retired.clear();
  if (rc == LOWBIT_OK && hipSetDevice(cur) != hipSuccess) rc = LOWBIT_E_HIP;
  return rc;
}

struct lowbit_chain {
  void* plan;
};

int lowbit_chain_create_rows(int n_stages, const lowbit_gemv_stage* stages, int64_t rows,
                             int x_dtype, int y_dtype, lowbit_chain** chain) {
  if (!stages || !chain) return LOWBIT_E_NULL;
  *chain = nullptr;
  if (n_stages < 1) return LOWBIT_E_SHAPE;
  if (x_dtype != LOWBIT_F32 && x_dtype != LOWBIT_BF16) return LOWBIT_E_UNSUPPORTED;
  if (y_dtype != LOWBIT_F32 && y_dtype != LOWBIT_BF16) return LOWBIT_E_UNSUPPORTED;
  const int fmt = stages[0].fmt;
  if (!valid_fmt(fmt)) return LOWBIT_E_UNSUPPORTED;
  if (rows < 1 || rows > max_small_m(fmt, x_dtype)) return LOWBIT_E_SHAPE;
  std::vector<ChainStage> st(n_stages);
  for (int i = 0; i < n_stages; i++) {
    const lowbit_gemv_stage& g = stages[i];
    if (g.fmt != fmt) return LOWBIT_E_UNSUPPORTED;
    if (!g.pcodes || !g.pscales || !g.x || !g.y) return LOWBIT_E_NULL;
    if (!shape_ok(g.N, g.K) || cdiv(g.N, 16) > kMaxRowGroups) return LOWBIT_E_SHAPE;
    // a waiting stage reads x through a buffer descriptor (32-bit byte offsets)
    if (i > 0 && g.wait_prev && rows * g.K * (x_dtype == LOWBIT_F32 ? 4 : 2) > INT32_MAX)
      return LOWBIT_E_SHAPE;
    if (!aligned(g.pcodes, 16) || !aligned(g.pscales, 16) || !aligned(g.x, 16) || !aligned(g.y, 4))
      return LOWBIT_E_ALIGN;
    if (g.epilogue != LOWBIT_EPI_NONE && g.epilogue != LOWBIT_EPI_SILU_MUL) return LOWBIT_E_UNSUPPORTED;
    if (g.epilogue == LOWBIT_EPI_SILU_MUL && (g.N % 16 != 0 || rows != 1)) return LOWBIT_E_SHAPE;
    st[i] = ChainStage{fmt, g.N, g.K, g.pcodes, (const uint16_t*)g.pscales, g.x, g.y,
                       i > 0 && g.wait_prev ? 1 : 0, g.epilogue};
  }
  void* plan = nullptr;
  hipError_t e = chain_create(st.data(), n_stages, rows, x_dtype, y_dtype, &plan);
  if (e == hipErrorOutOfMemory) return LOWBIT_E_NOMEM;
  if (e != hipSuccess) return LOWBIT_E_HIP;
  *chain = new lowbit_chain{plan};
  return LOWBIT_OK;
}

int lowbit_chain_create(int n_stages, const lowbit_gemv_stage* stages, int x_dtype, int y_dtype,
                        lowbit_chain** chain) {
  return lowbit_chain_create_rows(n_stages, stages, 1, x_dtype, y_dtype, chain);
}

int lowbit_chain_run(lowbit_chain* chain, void* stream) {
  if (!chain) return LOWBIT_E_NULL;
  return hip_status(chain_run(chain->plan, (hipStream_t)stream));
}

int lowbit_chain_status(lowbit_chain* chain, int* failed_waits) {
  if (!chain || !failed_waits) return LOWBIT_E_NULL;
  return hip_status(chain_status(chain->plan, failed_waits));
}

int lowbit_chain_destroy(lowbit_chain* chain) {
  if (!chain) return LOWBIT_OK;
  const hipError_t e = hipDeviceSynchronize();
  chain_destroy(chain->plan);
  delete chain;
  return hip_status(e);
}

}  // extern "C"

int lowbit_hbm_read_probe(const void* src, int64_t bytes, uint32_t* out, void* stream) {
  if (!src || !out) return LOWBIT_E_NULL;
  if (bytes < 16 || bytes % 16 != 0) return LOWBIT_E_SHAPE;
  if (!aligned(src, 16) || !aligned(out, 4)) return LOWBIT_E_ALIGN;
  return hip_status(launch_hbm_read(src, bytes, out, (hipStream_t)stream));
}

int lowbit_quantize_weights(int fmt, int64_t N, int64_t K, const uint16_t* W_bf16,
                            const int8_t* signs, int8_t* codes, uint16_t* scales, void* stream) {
  if (!W_bf16 || !codes || !scales) return LOWBIT_E_NULL;
  if (!valid_fmt(fmt)) return LOWBIT_E_UNSUPPORTED;
  if (!shape_ok(N, K)) return LOWBIT_E_SHAPE;
  if (!aligned(W_bf16, 16) || !aligned(codes, 16) || (signs && !aligned(signs, 16)) ||
      !aligned(scales, 2))
    return LOWBIT_E_ALIGN;
  return hip_status(launch_quantize_weights(fmt, N, K, W_bf16, signs, codes, scales,
                                            (hipStream_t)stream));
}

int lowbit_rotate_act(int64_t M, int64_t K, const uint16_t* X_bf16, const int8_t* signs,
                      float* X_rot, void* stream) {
  if (!X_bf16 || !signs || !X_rot) return LOWBIT_E_NULL;
  if (!shape_ok(M, K)) return LOWBIT_E_SHAPE;
  if (!aligned(X_bf16, 2) || !aligned(X_rot, 4)) return LOWBIT_E_ALIGN;
  return hip_status(launch_rotate_act(M, K, X_bf16, signs, X_rot, (hipStream_t)stream));
}


// ------------------------------------------------ MXFP4 and the 8-bit cache

namespace {

// rows x K of an MXFP4 matrix: sizes far from overflow
bool mx_shape_ok(int64_t rows, int64_t K) {
  return rows >= 1 && K >= kMxBlock && K % kMxBlock == 0 && rows <= (int64_t(1) << 30) &&
         K <= (int64_t(1) << 30) && rows <= (int64_t(1) << 38) / K;
}

// sizes of an MXFP4 product
bool product_shape_ok(bool x4, int64_t M, int64_t N, int64_t K) {
  return mx_shape_ok(N, K) && mx_shape_ok(M, K) && N <= (int64_t(1) << 26) &&
         cdiv(M, 128) * cdiv(N, 128) <= (int64_t(1) << 23) && gemm_mxfp4_fits(x4, M, N, K);
}

}  // namespace

int lowbit_mxfp4_bytes(int64_t rows, int64_t K, size_t* code_bytes, size_t* scale_bytes) {
  if (!code_bytes || !scale_bytes) return LOWBIT_E_NULL;
  if (!mx_shape_ok(rows, K)) return LOWBIT_E_SHAPE;
  *code_bytes = (size_t)(cdiv(rows, 16) * mx_groups(K) * 1024);
  *scale_bytes = (size_t)(cdiv(rows, 16) * mx_quads(K) * 256);
  return LOWBIT_OK;
}

int lowbit_pack_mxfp4(int64_t rows, int64_t K, const uint8_t* codes, const uint8_t* scales, void* pcodes,
                      void* pscales, void* stream) {
  if (!codes || !scales || !pcodes || !pscales) return LOWBIT_E_NULL;
  if (!mx_shape_ok(rows, K)) return LOWBIT_E_SHAPE;
  if (!aligned(codes, 16) || !aligned(pcodes, 16) || !aligned(pscales, 16)) return LOWBIT_E_ALIGN;
  return hip_status(launch_pack_mxfp4(rows, K, codes, scales, pcodes, pscales, (hipStream_t)stream));
}

int lowbit_quantize_mxfp4(int64_t rows, int64_t K, int x_dtype, const void* X, int64_t x_stride, void* pcodes,
                          void* pscales, void* values, void* stream) {
  if (!X || !pcodes || !pscales) return LOWBIT_E_NULL;
  if (x_dtype != LOWBIT_F32 && x_dtype != LOWBIT_BF16) return LOWBIT_E_UNSUPPORTED;
  if (!mx_shape_ok(rows, K) || !quantize_mxfp4_fits(rows, K)) return LOWBIT_E_SHAPE;
  if (x_stride < K || x_stride > (int64_t(1) << 40)) return LOWBIT_E_SHAPE;
  const bool f32 = x_dtype == LOWBIT_F32;
  if (!aligned(X, 16) || x_stride % (f32 ? 4 : 8) != 0 || !aligned(pcodes, 16) || !aligned(pscales, 16) ||
      (values && !aligned(values, 16)))
    return LOWBIT_E_ALIGN;
  return hip_status(
      launch_quantize_mxfp4(rows, K, f32, X, x_stride, pcodes, pscales, values, (hipStream_t)stream));
}

int lowbit_gemm_mxfp4(int64_t M, int64_t N, int64_t K, const void* pcodes, const void* pscales, int x_dtype,
                      const void* X, int64_t x_stride, const void* x_pscales, int y_dtype, void* Y,
                      void* stream) {
  if (!pcodes || !pscales || !X || !Y) return LOWBIT_E_NULL;
  if (x_dtype != LOWBIT_BF16 && x_dtype != LOWBIT_MXFP4) return LOWBIT_E_UNSUPPORTED;
  if (y_dtype != LOWBIT_F32 && y_dtype != LOWBIT_BF16) return LOWBIT_E_UNSUPPORTED;
  const bool x4 = x_dtype == LOWBIT_MXFP4;
  if (x4 && !x_pscales) return LOWBIT_E_NULL;
  if (!product_shape_ok(x4, M, N, K)) return LOWBIT_E_SHAPE;
  if (!x4 && (x_stride < K || x_stride > (int64_t(1) << 40))) return LOWBIT_E_SHAPE;
  if (!aligned(pcodes, 16) || !aligned(pscales, 16) || !aligned(X, 16) || !aligned(Y, 16) ||
      (x4 && !aligned(x_pscales, 16)) || (!x4 && x_stride % 8 != 0))
    return LOWBIT_E_ALIGN;
  MxGemmArgs g;
  g.M = M;
  g.N = N;
  g.K = K;
  g.ld = x4 ? 0 : x_stride;
  g.pcodes = pcodes;
  g.pscales = pscales;
  g.x4 = x4;
  g.x = X;
  g.x_pscales = x_pscales;
  g.ykind = y_dtype;
  g.y = Y;
  g.ws = nullptr;
  const size_t need = gemm_mxfp4_workspace_bytes(x4, M, N, K);
  if (need) {
    const int rc = workspace((hipStream_t)stream, need, &g.ws);
    if (rc) return rc;
  }
  return hip_status(launch_gemm_mxfp4(g, (hipStream_t)stream));
}

int lowbit_gemm_mxfp4_workspace(int64_t M, int64_t N, int64_t K, int x_dtype, size_t* bytes) {
  if (!bytes) return LOWBIT_E_NULL;
  *bytes = 0;
  if (x_dtype != LOWBIT_BF16 && x_dtype != LOWBIT_MXFP4) return LOWBIT_E_UNSUPPORTED;
  if (!product_shape_ok(x_dtype == LOWBIT_MXFP4, M, N, K)) return LOWBIT_E_SHAPE;
  *bytes = gemm_mxfp4_workspace_bytes(x_dtype == LOWBIT_MXFP4, M, N, K);
  return LOWBIT_OK;
}

namespace {

// checks of a cache and a batch, and the kernels' view of them
int kv8_check(const lowbit_kv8* c, const lowbit_kv8_batch* b, KvArgs* out) {
  if (!c || !b) return LOWBIT_E_NULL;
  if (!c->k_codes || !c->v_codes || !c->k_scales || !c->v_scales || !b->page_table || !b->kv_lens)
    return LOWBIT_E_NULL;
  int lp = -1;
  for (int i = 4; i <= 7; i++)
    if (c->page_tokens == 1 << i) lp = i;
  if (lp < 0 || (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256)) return LOWBIT_E_UNSUPPORTED;
  if (c->kv_heads < 1 || c->kv_heads > 4096 || c->n_pages < 1 || c->n_pages > INT32_MAX) return LOWBIT_E_SHAPE;
  if (b->n_seqs < 1 || b->n_seqs > (1 << 20) || b->table_width < 1 || b->table_width > (1 << 26))
    return LOWBIT_E_SHAPE;
  if (b->total_q < 1 || b->total_q > (1 << 30) || b->max_q < 1 || b->max_q > b->total_q) return LOWBIT_E_SHAPE;
  if (!b->q_starts && b->total_q != b->n_seqs * b->max_q) return LOWBIT_E_SHAPE;
  if (b->max_kv < 1 || b->max_kv > (1 << 30) || b->max_kv > b->table_width * c->page_tokens) return LOWBIT_E_SHAPE;
  if (!aligned(c->k_codes, 16) || !aligned(c->v_codes, 16) || !aligned(b->page_table, 4) ||
      !aligned(b->kv_lens, 4) || (b->q_starts && !aligned(b->q_starts, 4)) ||
      (b->bad_pages && !aligned(b->bad_pages, 4)))
    return LOWBIT_E_ALIGN;
  out->n_pages = c->n_pages;
  out->H = c->kv_heads;
  out->D = c->head_dim;
  out->lp = lp;
  out->kc = (uint8_t*)c->k_codes;
  out->vc = (uint8_t*)c->v_codes;
  out->ks = c->k_scales;
  out->vs = c->v_scales;
  out->n_seqs = b->n_seqs;
  out->table = b->page_table;
  out->width = b->table_width;
  out->lens = b->kv_lens;
  out->starts = b->q_starts;
  out->total_q = b->total_q;
  out->max_q = b->max_q;
  out->max_kv = b->max_kv;
  out->bad = b->bad_pages;
  out->members = nullptr;
  out->member_count = out->n_members = out->member_q = 0;
  return LOWBIT_OK;
}

// query heads of a call: whole groups, rows that int counts, one grid
bool attention_heads_ok(const KvArgs& a, int64_t q_heads) {
  if (q_heads < 1 || q_heads > (1 << 16) || q_heads % a.H != 0) return false;
  const int64_t G = q_heads / a.H;
  return a.max_q * G <= (1 << 30) && attention_blocks(a, G) <= (1 << 22);
}

}  // namespace

int lowbit_kv8_append(const lowbit_kv8* cache, const lowbit_kv8_batch* batch, int dtype, const void* K,
                      const void* V, int64_t k_stride, int64_t v_stride, void* stream) {
  if (!K || !V) return LOWBIT_E_NULL;
  KvArgs a;
  const int rc = kv8_check(cache, batch, &a);
  if (rc) return rc;
  if (dtype != LOWBIT_F32 && dtype != LOWBIT_BF16) return LOWBIT_E_UNSUPPORTED;
  const int64_t row = (int64_t)a.H * a.D, most = int64_t(1) << 40;
  if (k_stride < row || v_stride < row || k_stride > most || v_stride > most) return LOWBIT_E_SHAPE;
  if (!kv8_append_fits(a)) return LOWBIT_E_SHAPE;
  const int step = dtype == LOWBIT_F32 ? 4 : 8;
  if (!aligned(K, 16) || !aligned(V, 16) || k_stride % step != 0 || v_stride % step != 0) return LOWBIT_E_ALIGN;
  return hip_status(launch_kv8_append(a, dtype == LOWBIT_F32, K, V, k_stride, v_stride, (hipStream_t)stream));
}

int lowbit_attention_kv8_workspace(const lowbit_kv8* cache, const lowbit_kv8_batch* batch, int64_t q_heads,
                                   size_t* bytes) {
  if (!bytes) return LOWBIT_E_NULL;
  *bytes = 0;
  KvArgs a;
  const int rc = kv8_check(cache, batch, &a);
  if (rc) return rc;
  if (!attention_heads_ok(a, q_heads)) return LOWBIT_E_SHAPE;
  *bytes = attention_workspace_bytes(a, q_heads / a.H);
  return LOWBIT_OK;
}

int lowbit_attention_kv8(const lowbit_kv8* cache, const lowbit_kv8_batch* batch, int64_t q_heads,
                         const uint16_t* Q_bf16, int64_t q_stride, float softmax_scale, int causal,
                         int64_t window, uint16_t* O_bf16, int64_t o_stride, float* lse, void* stream) {
  if (!Q_bf16 || !O_bf16) return LOWBIT_E_NULL;
  AttnArgs a;
  const int rc = kv8_check(cache, batch, &a.kv);
  if (rc) return rc;
  if (!attention_heads_ok(a.kv, q_heads)) return LOWBIT_E_SHAPE;
  const int64_t row = q_heads * a.kv.D, most = int64_t(1) << 40;
  if (q_stride < row || o_stride < row || q_stride > most || o_stride > most) return LOWBIT_E_SHAPE;
  a.scale2 = softmax_scale * 1.4426950408889634f;
  if (!(a.scale2 - a.scale2 == 0.0f)) return LOWBIT_E_UNSUPPORTED;  // infinite or NaN
  if (window < 0) return LOWBIT_E_SHAPE;
  a.G = q_heads / a.kv.H;
  if (!aligned(Q_bf16, 16) || !aligned(O_bf16, 16) || q_stride % 8 != 0 || o_stride % 8 != 0 ||
      (lse && !aligned(lse, 4)))
    return LOWBIT_E_ALIGN;
  a.Hq = q_heads;
  a.q = Q_bf16;
  a.q_stride = q_stride;
  a.causal = causal ? 1 : 0;
  a.window = window > (1 << 30) ? 0 : (int)window;  // wider than any sequence
  a.o = O_bf16;
  a.o_stride = o_stride;
  a.lse = lse;
  const size_t need = attention_workspace_bytes(a.kv, a.G);
  void* ws = nullptr;
  if (need) {
    const int r2 = workspace((hipStream_t)stream, need, &ws);
    if (r2) return r2;
  }
  return hip_status(launch_attention(a, ws, (hipStream_t)stream));
}

namespace {

// checks of what a call behind shared prefixes has in common with its workspace query
int prefix_check(const lowbit_kv8* cache, const lowbit_kv8_prefix* p, const lowbit_kv8_batch* batch, int64_t q_heads,
                 AttnArgs* a, PrefixPlan* plan) {
  KvArgs* const out = &a->prefix;
  if (!p) return LOWBIT_E_NULL;
  const int rc = kv8_check(cache, batch, &a->kv);
  if (rc) return rc;
  if (!p->page_table || !p->lens) return LOWBIT_E_NULL;
  if (p->n_groups < 1 || p->n_groups > (1 << 20) || p->table_width < 1 || p->table_width > (1 << 26))
    return LOWBIT_E_SHAPE;
  if (p->max_len < 1 || p->max_len > p->table_width * cache->page_tokens) return LOWBIT_E_SHAPE;
  if (p->max_len > (1 << 30) - batch->max_kv) return LOWBIT_E_SHAPE;  // positions behind the prefix are int
  if (p->seq_starts ? p->max_seqs < 1 || p->max_seqs > batch->n_seqs : batch->n_seqs % p->n_groups != 0)
    return LOWBIT_E_SHAPE;
  if (!aligned(p->page_table, 4) || !aligned(p->lens, 4) || (p->seq_starts && !aligned(p->seq_starts, 4)))
    return LOWBIT_E_ALIGN;
  const int64_t each = batch->n_seqs / p->n_groups, seqs = p->seq_starts ? p->max_seqs : each;
  *out = a->kv;
  out->n_seqs = p->n_groups;
  out->table = p->page_table;
  out->width = p->table_width;
  out->lens = p->lens;
  out->max_q = std::min(batch->total_q, seqs * batch->max_q);
  out->max_kv = p->max_len;
  out->members = p->seq_starts;
  out->member_count = each;
  out->n_members = batch->n_seqs;
  out->member_q = batch->max_q;
  if (!attention_heads_ok(a->kv, q_heads) || !attention_heads_ok(*out, q_heads)) return LOWBIT_E_SHAPE;
  if (a->kv.total_q * q_heads > (int64_t(1) << 38) / (a->kv.D + 4)) return LOWBIT_E_SHAPE;
  a->Hq = q_heads;
  a->G = q_heads / a->kv.H;
  // Starts may name more rows for a sequence than max_q, which only its own launch cuts: rows of a
  // group to be expected, and those that it may have.  (Of a key head int counts them: more than
  // 2^30 would take more workgroups than a launch has, so such calls go by their sequences.)
  a->group_q = std::max(out->max_q, batch->total_q / batch->n_seqs * seqs);
  out->max_q = batch->total_q;
  *plan = plan_prefix(*a);
  return plan->blocks <= (1 << 22) ? LOWBIT_OK : LOWBIT_E_SHAPE;
}

}  // namespace

int lowbit_attention_kv8_prefix_workspace(const lowbit_kv8* cache, const lowbit_kv8_prefix* prefix,
                                          const lowbit_kv8_batch* batch, int64_t q_heads, size_t* bytes) {
  if (!bytes) return LOWBIT_E_NULL;
  *bytes = 0;
  AttnArgs a = {};
  PrefixPlan plan;
  const int rc = prefix_check(cache, prefix, batch, q_heads, &a, &plan);
  if (rc) return rc;
  *bytes = attention_prefix_workspace_bytes(a);
  return LOWBIT_OK;
}

int lowbit_attention_kv8_prefix_launches(const lowbit_kv8* cache, const lowbit_kv8_prefix* prefix,
                                         const lowbit_kv8_batch* batch, int64_t q_heads, lowbit_kv8_prefix_plan* plan) {
  if (!plan) return LOWBIT_E_NULL;
  *plan = {};
  AttnArgs a = {};
  PrefixPlan p;
  const int rc = prefix_check(cache, prefix, batch, q_heads, &a, &p);
  if (rc) return rc;
  const bool few = p.nc > 0;
  plan->launches = p.behind ? 1 : 2;
  plan->tile_rows = few ? 16 * p.nc : p.rows;
  plan->tile_parts = !few ? p.parts : p.behind ? p.pieces : 0;
  plan->whole_tiles = p.behind && !few ? p.whole : 0;
  plan->own_rows = p.behind ? 0 : 16 * p.tail_nc;
  plan->own_parts = p.behind ? 0 : p.pieces;
  plan->weight_terms = few || p.fine ? 2 : 1;
  return LOWBIT_OK;
}

int lowbit_attention_kv8_prefix(const lowbit_kv8* cache, const lowbit_kv8_prefix* prefix,
                                const lowbit_kv8_batch* batch, int64_t q_heads, const uint16_t* Q_bf16,
                                int64_t q_stride, float softmax_scale, int causal, uint16_t* O_bf16,
                                int64_t o_stride, float* lse, void* stream) {
  if (!Q_bf16 || !O_bf16) return LOWBIT_E_NULL;
  AttnArgs a = {};
  PrefixPlan plan;
  const int rc = prefix_check(cache, prefix, batch, q_heads, &a, &plan);
  if (rc) return rc;
  const int64_t row = q_heads * a.kv.D, most = int64_t(1) << 40;
  if (q_stride < row || o_stride < row || q_stride > most || o_stride > most) return LOWBIT_E_SHAPE;
  a.scale2 = softmax_scale * 1.4426950408889634f;
  if (!(a.scale2 - a.scale2 == 0.0f)) return LOWBIT_E_UNSUPPORTED;  // infinite or NaN
  if (!aligned(Q_bf16, 16) || !aligned(O_bf16, 16) || q_stride % 8 != 0 || o_stride % 8 != 0 ||
      (lse && !aligned(lse, 4)))
    return LOWBIT_E_ALIGN;
  a.q = Q_bf16;
  a.q_stride = q_stride;
  a.causal = causal ? 1 : 0;
  a.o = O_bf16;
  a.o_stride = o_stride;
  a.lse = lse;
  void* ws = nullptr;
  const int r2 = workspace((hipStream_t)stream, attention_prefix_workspace_bytes(a), &ws);
  if (r2) return r2;
  return hip_status(launch_attention_prefix(a, plan, ws, (hipStream_t)stream));
}

// ------------------------------------------- heads of queries and keys; pages

namespace {

// n runs of bytes, `stride` apart (at least `bytes`)
struct Rows {
  uintptr_t at;
  int64_t bytes, stride, n;
};
// whether some run of a and some run of b share a byte
bool rows_meet(Rows a, Rows b) {
  if (!a.at || !b.at) return false;
  if (a.stride < b.stride) std::swap(a, b);
  auto end = [](const Rows& r) { return r.at + (uintptr_t)((r.n - 1) * r.stride + r.bytes); };
  if (end(a) <= b.at || end(b) <= a.at) return false;
  // Runs of a from the first that ends behind b's begin.  One that lies over b's begin or end meets it; of
  // the others the places between b's runs come again after stride / gcd runs.
  const int64_t gap = (int64_t)(b.at - a.at);
  const int64_t first = gap < a.bytes ? 0 : (gap - a.bytes) / a.stride + 1;
  const int64_t last = std::min(a.n, first + b.stride / std::gcd(a.stride, b.stride) + 2);
  for (int64_t i = first; i < last; i++) {
    const int64_t x = i * a.stride - gap;  // from b's begin
    const int64_t j = x < 0 ? 0 : std::min(x / b.stride, b.n - 1);
    if (j * b.stride < x + a.bytes && x < j * b.stride + b.bytes) return true;
    if (j + 1 < b.n && (j + 1) * b.stride < x + a.bytes) return true;
  }
  return false;
}

}  // namespace

int lowbit_qk_norm_rope(const lowbit_rope* rope, int x_dtype, const void* Q, int64_t q_heads, int64_t q_stride,
                        const float* q_weight, const void* K, int64_t kv_heads, int64_t k_stride,
                        const float* k_weight, float eps, int y_dtype, void* Q_out, int64_t qo_stride, void* K_out,
                        int64_t ko_stride, void* stream) {
  if (!rope || !Q || !Q_out || (kv_heads != 0 && (!K || !K_out))) return LOWBIT_E_NULL;
  const lowbit_rope& r = *rope;
  if (r.n_pairs != 0 && (!r.positions || !r.freqs)) return LOWBIT_E_NULL;
  for (int t : {x_dtype, y_dtype})
    if (t != LOWBIT_F32 && t != LOWBIT_BF16) return LOWBIT_E_UNSUPPORTED;
  if (r.head_dim < 8 || r.head_dim > 256 || r.head_dim % 8 != 0) return LOWBIT_E_UNSUPPORTED;
  if (r.n_pairs < 0 || r.n_pairs % 4 != 0 || 2 * (int64_t)r.n_pairs > r.head_dim) return LOWBIT_E_UNSUPPORTED;
  if (!(eps >= 0.f) || !(eps - eps == 0.f)) return LOWBIT_E_UNSUPPORTED;
  if (r.tokens < 1 || r.tokens > (1 << 30) || r.n_axes < 1 || r.n_axes > (1 << 16)) return LOWBIT_E_SHAPE;
  const int64_t most = int64_t(1) << 40;
  if (r.n_axes > 1 && r.n_pairs != 0 && (r.pos_stride < r.tokens || r.pos_stride > most)) return LOWBIT_E_SHAPE;
  if (q_heads < 1 || q_heads > (1 << 16) || kv_heads < 0 || kv_heads > (1 << 16)) return LOWBIT_E_SHAPE;
  const int64_t far = (int64_t(1) << 46) / r.tokens;  // rows beyond that lie in no address space
  auto bad_stride = [&](int64_t stride, int64_t heads) {
    return stride < heads * r.head_dim || stride > most || (r.tokens > 1 && stride > far);
  };
  if (bad_stride(q_stride, q_heads) || bad_stride(qo_stride, q_heads)) return LOWBIT_E_SHAPE;
  if (kv_heads && (bad_stride(k_stride, kv_heads) || bad_stride(ko_stride, kv_heads))) return LOWBIT_E_SHAPE;
  if (!aligned(Q, 16) || !aligned(Q_out, 16) || q_stride % 8 != 0 || qo_stride % 8 != 0) return LOWBIT_E_ALIGN;
  if (kv_heads && (!aligned(K, 16) || !aligned(K_out, 16) || k_stride % 8 != 0 || ko_stride % 8 != 0))
    return LOWBIT_E_ALIGN;
  if (r.n_pairs && (!aligned(r.positions, 4) || !aligned(r.freqs, 8) || (r.pair_axis && !aligned(r.pair_axis, 4))))
    return LOWBIT_E_ALIGN;
  if ((q_weight && !aligned(q_weight, 4)) || (k_weight && !aligned(k_weight, 4))) return LOWBIT_E_ALIGN;
  // Outputs share no byte with an input or each other, but for an output that is its input.
  const int xb = x_dtype == LOWBIT_F32 ? 4 : 2, yb = y_dtype == LOWBIT_F32 ? 4 : 2;
  auto rows = [&](const void* p, int64_t heads, int64_t stride, int bytes) {
    const int64_t row = heads * r.head_dim * bytes;
    return Rows{(uintptr_t)p, row, r.tokens > 1 ? stride * bytes : row, r.tokens};
  };
  auto run = [](const void* p, int64_t bytes) { return Rows{(uintptr_t)p, bytes, bytes, 1}; };
  const Rows none = {0, 0, 0, 0}, q = rows(Q, q_heads, q_stride, xb), qo = rows(Q_out, q_heads, qo_stride, yb);
  const Rows k = kv_heads ? rows(K, kv_heads, k_stride, xb) : none, ko = kv_heads ? rows(K_out, kv_heads, ko_stride, yb) : none;
  auto in_place = [&](const Rows& x, const Rows& y) { return x.at == y.at && xb == yb && x.stride == y.stride; };
  if ((!in_place(q, qo) && rows_meet(q, qo)) || (!in_place(k, ko) && rows_meet(k, ko)) || rows_meet(q, ko) || rows_meet(k, qo) ||
      rows_meet(qo, ko))
    return LOWBIT_E_UNSUPPORTED;
  for (const Rows& y : {qo, ko}) {
    for (const float* w : {q_weight, k_weight})
      if (rows_meet(y, run(w, 4 * (int64_t)r.head_dim))) return LOWBIT_E_UNSUPPORTED;
    if (r.n_pairs == 0) continue;
    const Rows positions = {(uintptr_t)r.positions, 4 * r.tokens, r.n_axes > 1 ? 4 * r.pos_stride : 4 * r.tokens, r.n_axes};
    if (rows_meet(y, positions) || rows_meet(y, run(r.freqs, 8 * (int64_t)r.n_pairs)) ||
        rows_meet(y, run(r.pair_axis, 4 * (int64_t)r.n_pairs)))
      return LOWBIT_E_UNSUPPORTED;
  }
  RopeArgs a;
  a.tokens = r.tokens;
  a.D = r.head_dim;
  a.pairs = r.n_pairs;
  a.adjacent = r.adjacent ? 1 : 0;
  a.axes = r.n_axes;
  a.Hq = (int)q_heads;
  a.Hk = (int)kv_heads;
  a.pos = r.positions;
  a.pos_stride = r.n_axes > 1 ? r.pos_stride : 0;
  a.freqs = r.freqs;
  a.pair_axis = r.pair_axis;
  a.eps = eps;
  a.inv_d = 1.0f / r.head_dim;
  a.qw = q_weight;
  a.kw = k_weight;
  a.q = Q;
  a.k = K;
  a.qo = Q_out;
  a.ko = K_out;
  a.q_stride = q_stride;
  a.k_stride = kv_heads ? k_stride : 0;
  a.qo_stride = qo_stride;
  a.ko_stride = kv_heads ? ko_stride : 0;
  return hip_status(launch_qk_norm_rope(a, x_dtype == LOWBIT_F32, y_dtype == LOWBIT_F32, (hipStream_t)stream));
}

namespace {

constexpr int64_t kMaxCachePages = int64_t(1) << 26, kMaxWidth = int64_t(1) << 26, kMaxCaches = 4096;

int log2_page(int page_tokens) {
  for (int i = 4; i <= 7; i++)
    if (page_tokens == 1 << i) return i;
  return -1;
}

// checks of a model's caches (its layers), which share pages and tables
int caches_check(const lowbit_kv8* c, int64_t n, std::vector<KvLayer>* out) {
  if (!c) return LOWBIT_E_NULL;
  if (n < 1 || n > kMaxCaches) return LOWBIT_E_SHAPE;
  for (int64_t i = 0; i < n; i++) {
    if (!c[i].k_codes || !c[i].v_codes || !c[i].k_scales || !c[i].v_scales) return LOWBIT_E_NULL;
    if (log2_page(c[i].page_tokens) < 0 || (c[i].head_dim != 64 && c[i].head_dim != 128 && c[i].head_dim != 256))
      return LOWBIT_E_UNSUPPORTED;
    if (c[i].n_pages < 1 || c[i].n_pages > kMaxCachePages || c[i].kv_heads < 1 || c[i].kv_heads > 4096)
      return LOWBIT_E_SHAPE;
    if (c[i].n_pages != c[0].n_pages || c[i].page_tokens != c[0].page_tokens) return LOWBIT_E_SHAPE;
    if (!aligned(c[i].k_codes, 16) || !aligned(c[i].v_codes, 16)) return LOWBIT_E_ALIGN;
    out->push_back(KvLayer{c[i].kv_heads, c[i].head_dim, (uint8_t*)c[i].k_codes, (uint8_t*)c[i].v_codes, c[i].k_scales,
                           c[i].v_scales});
  }
  return LOWBIT_OK;
}

bool fork_sizes_ok(int64_t n_pages, int page_tokens, int64_t n_seqs, int64_t n_new, int64_t max_grow) {
  return n_pages >= 1 && n_pages <= kMaxCachePages && n_seqs >= 0 && n_seqs <= (1 << 20) && n_new >= 0 &&
         n_new <= (1 << 20) && max_grow >= 0 && max_grow <= (1 << 30) &&
         n_new * (max_grow / page_tokens + 2) <= (1 << 30);
}
// whether an output shares a byte with an input or with another output
struct Span {
  const void* p;
  int64_t ints;
};
bool outputs_overlap(std::initializer_list<Span> in, std::initializer_list<Span> out) {
  auto meet = [](const Span& a, const Span& b) {
    const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
    return a.p && b.p && a.ints && b.ints && x < y + 4 * (uintptr_t)b.ints && y < x + 4 * (uintptr_t)a.ints;
  };
  for (const Span* o = out.begin(); o != out.end(); o++) {
    for (const Span& i : in)
      if (meet(*o, i)) return true;
    for (const Span* q = out.begin(); q != o; q++)
      if (meet(*o, *q)) return true;
  }
  return false;
}

bool table_ok(int64_t n_seqs, int64_t width) {
  return n_seqs == 0 || (width >= 1 && width <= kMaxWidth);
}

// runs f; C++ exceptions (of the host's memory) do not leave the library
template <class F>
int no_throw(F&& f) {
  try {
    return f();
  } catch (...) {
    return LOWBIT_E_NOMEM;
  }
}

}  // namespace

int lowbit_kv8_fork_workspace(int64_t n_pages, int page_tokens, int64_t n_caches, int64_t n_seqs, int64_t n_new,
                              int64_t max_grow, size_t* bytes) {
  if (!bytes) return LOWBIT_E_NULL;
  *bytes = 0;
  if (log2_page(page_tokens) < 0) return LOWBIT_E_UNSUPPORTED;
  if (n_caches < 1 || n_caches > kMaxCaches) return LOWBIT_E_SHAPE;
  if (!fork_sizes_ok(n_pages, page_tokens, n_seqs, n_new, max_grow)) return LOWBIT_E_SHAPE;
  ForkArgs a = {};
  a.n_pages = n_pages;
  a.n_layers = n_caches;
  a.lp = log2_page(page_tokens);
  a.n_seqs = n_seqs;
  a.n_new = n_new;
  a.max_grow = max_grow;
  *bytes = fork_workspace_bytes(a);
  return LOWBIT_OK;
}

int lowbit_kv8_fork_cut(const lowbit_kv8* caches, int64_t n_caches, int64_t n_seqs, const int32_t* page_table,
                        int64_t table_width, const int32_t* kv_lens, const int32_t* refs, int64_t n_new,
                        const int32_t* parents, const int32_t* grow, int64_t max_grow, int32_t* new_table,
                        int64_t new_width, int32_t* new_lens, int32_t* new_refs, int32_t* failed, int32_t* cut,
                        void* stream) {
  return no_throw([&]() -> int {
    std::vector<KvLayer> layers;
    const int rc = caches_check(caches, n_caches, &layers);
    if (rc) return rc;
    if (!refs || !new_refs || !failed) return LOWBIT_E_NULL;
    if (n_seqs != 0 && (!page_table || !kv_lens)) return LOWBIT_E_NULL;
    if (n_new != 0 && (!parents || !new_table || !new_lens)) return LOWBIT_E_NULL;
    const int P = caches[0].page_tokens;
    if (!fork_sizes_ok(caches[0].n_pages, P, n_seqs, n_new, max_grow)) return LOWBIT_E_SHAPE;
    if (!table_ok(n_seqs, table_width) || !table_ok(n_new, new_width)) return LOWBIT_E_SHAPE;
    for (const void* p : {(const void*)page_table, (const void*)kv_lens, (const void*)refs, (const void*)parents,
                          (const void*)grow, (const void*)new_table, (const void*)new_lens, (const void*)failed,
                          (const void*)cut})
      if (!aligned(p, 4)) return LOWBIT_E_ALIGN;
    if (!aligned(new_refs, 16)) return LOWBIT_E_ALIGN;
    ForkArgs a = {};
    a.n_pages = caches[0].n_pages;
    a.n_layers = n_caches;
    a.lp = log2_page(P);
    a.n_seqs = n_seqs;
    a.width = n_seqs ? table_width : 1;
    a.table = page_table;
    a.lens = kv_lens;
    a.refs = refs;
    a.n_new = n_new;
    a.new_width = n_new ? new_width : 1;
    a.max_grow = max_grow;
    a.parents = parents;
    a.grow = grow;
    a.new_table = new_table;
    a.new_lens = new_lens;
    a.new_refs = new_refs;
    a.failed = failed;
    a.cut = cut;
    if (!fork_fits(a)) return LOWBIT_E_SHAPE;
    if (outputs_overlap({{page_table, n_seqs * a.width}, {kv_lens, n_seqs}, {refs, a.n_pages}, {parents, n_new}, {grow, n_new}},
                        {{new_table, n_new * a.new_width}, {new_lens, n_new}, {new_refs, a.n_pages}, {failed, 1}, {cut, 1}}))
      return LOWBIT_E_UNSUPPORTED;
    void* ws = nullptr;
    const int r2 = workspace((hipStream_t)stream, fork_workspace_bytes(a), &ws);
    if (r2) return r2;
    return hip_status(launch_fork(a, layers.data(), ws, (hipStream_t)stream));
  });
}

int lowbit_kv8_fork(const lowbit_kv8* caches, int64_t n_caches, int64_t n_seqs, const int32_t* page_table,
                    int64_t table_width, const int32_t* kv_lens, const int32_t* refs, int64_t n_new,
                    const int32_t* parents, const int32_t* grow, int64_t max_grow, int32_t* new_table,
                    int64_t new_width, int32_t* new_lens, int32_t* new_refs, int32_t* failed, void* stream) {
  return lowbit_kv8_fork_cut(caches, n_caches, n_seqs, page_table, table_width, kv_lens, refs, n_new, parents, grow, max_grow,
                             new_table, new_width, new_lens, new_refs, failed, nullptr, stream);
}

int lowbit_kv8_compact_workspace(int64_t n_pages, int64_t n_caches, size_t* bytes) {
  if (!bytes) return LOWBIT_E_NULL;
  *bytes = 0;
  if (n_pages < 1 || n_pages > kMaxCachePages || n_caches < 1 || n_caches > kMaxCaches) return LOWBIT_E_SHAPE;
  CompactArgs a = {};
  a.n_pages = n_pages;
  a.n_layers = n_caches;
  *bytes = compact_workspace_bytes(a);
  return LOWBIT_OK;
}

int lowbit_kv8_compact(const lowbit_kv8* caches, int64_t n_caches, int64_t n_seqs, const int32_t* page_table,
                       int64_t table_width, const int32_t* kv_lens, const int32_t* refs, int32_t* new_table,
                       int32_t* new_refs, int32_t* remap, int32_t* live, void* stream) {
  return no_throw([&]() -> int {
    std::vector<KvLayer> layers;
    const int rc = caches_check(caches, n_caches, &layers);
    if (rc) return rc;
    if (!refs || !new_refs || !remap || !live) return LOWBIT_E_NULL;
    if (n_seqs != 0 && (!page_table || !kv_lens || !new_table)) return LOWBIT_E_NULL;
    if (n_seqs < 0 || n_seqs > (1 << 20) || !table_ok(n_seqs, table_width)) return LOWBIT_E_SHAPE;
    for (const void* p : {(const void*)page_table, (const void*)kv_lens, (const void*)refs, (const void*)new_table,
                          (const void*)new_refs, (const void*)remap, (const void*)live})
      if (!aligned(p, 4)) return LOWBIT_E_ALIGN;
    CompactArgs a = {};
    a.n_pages = caches[0].n_pages;
    a.n_layers = n_caches;
    a.lp = log2_page(caches[0].page_tokens);
    a.n_seqs = n_seqs;
    a.width = n_seqs ? table_width : 1;
    a.table = page_table;
    a.lens = kv_lens;
    a.refs = refs;
    a.new_table = new_table;
    a.new_refs = new_refs;
    a.remap = remap;
    a.live = live;
    if (!compact_fits(a)) return LOWBIT_E_SHAPE;
    if (outputs_overlap({{page_table, n_seqs * a.width}, {kv_lens, n_seqs}, {refs, a.n_pages}},
                        {{new_table, n_seqs * a.width}, {new_refs, a.n_pages}, {remap, a.n_pages}, {live, 1}}))
      return LOWBIT_E_UNSUPPORTED;
    void* ws = nullptr;
    const int r2 = workspace((hipStream_t)stream, compact_workspace_bytes(a), &ws);
    if (r2) return r2;
    return hip_status(launch_compact(a, layers.data(), ws, (hipStream_t)stream));
  });
}
