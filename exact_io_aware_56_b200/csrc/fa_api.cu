// C-ABI layer of libfa: argument checks, device check, TMA tensor maps,
// watchdog word, status strings. Declared in include/fa.h.

#include <atomic>
#include <cmath>
#include <cstdio>
#include <cstring>
#include <mutex>

#include "../../include/fa.h"
#include "../../include/fa_profile.h"
#include "../../include/fa_test.h"
#include "fa_internal.h"
#include "sm100.cuh"

namespace fa {
namespace {

__global__ void test_exp2_kernel(const float* x, float* yp, float* ye, int n) {
  for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < n; i += gridDim.x * blockDim.x) {
    yp[i] = exp2_poly(x[i]);
    ye[i] = ex2(x[i]);
  }
}

__global__ void test_exp2_accurate_kernel(const float* x, float* y, int n) {
  for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < n; i += gridDim.x * blockDim.x) y[i] = exp2_accurate(x[i]);
}

constexpr int kMaxDevices = 64;

// Device error word written by the kernels' watchdog.
__device__ unsigned int g_err_word;

std::atomic<uint64_t> g_budget_ns{2000000000ull};
std::atomic<int> g_fault{0};
std::atomic<void*> g_ev_pre{nullptr};
std::atomic<void*> g_ev_main{nullptr};
std::atomic<void*> g_ev_dec{nullptr};
thread_local char t_cuda_msg[256] = "no CUDA error recorded";

struct DevState {
  std::once_flag once;
  bool supported = false;
  unsigned int* err = nullptr;
  int sms = 0;
};
DevState g_dev[kMaxDevices];

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
std::once_flag g_encode_once;
EncodeTiledFn g_encode = nullptr;

int record_cuda(cudaError_t e) {
  snprintf(t_cuda_msg, sizeof(t_cuda_msg), "CUDA error %d: %s", static_cast<int>(e), cudaGetErrorString(e));
  return FA_ERR_CUDA;
}

// Checks the current device once: compute capability 10.0 (sm_100a) and the
// address of its error word. Returns FA_OK or an error status.
int device_state(DevState** out) {
  int dev = -1;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return record_cuda(e);
  if (dev < 0 || dev >= kMaxDevices) return FA_ERR_UNSUPPORTED;
  DevState& st = g_dev[dev];
  std::call_once(st.once, [&] {
    int major = 0, minor = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess) return;
    if (cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess) return;
    if (major != 10 || minor != 0) return;
    if (cudaDeviceGetAttribute(&st.sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || st.sms <= 0) return;
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_err_word) != cudaSuccess) return;
    st.err = static_cast<unsigned int*>(p);
    st.supported = true;
  });
  if (!st.supported) return FA_ERR_UNSUPPORTED;
  *out = &st;
  return FA_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int check_shape(int B, int Hq, int Hkv, int N, int d, int causal, float scale) {
  if (B <= 0 || Hq <= 0 || Hkv <= 0 || N <= 0) return FA_ERR_INVALID_ARGUMENT;
  if (causal != 0 && causal != 1) return FA_ERR_INVALID_ARGUMENT;
  if (!std::isfinite(scale) || !(scale > 0.f)) return FA_ERR_INVALID_ARGUMENT;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  if (Hq % Hkv != 0) return FA_ERR_UNSUPPORTED;
  // Index arithmetic limits: (B*Hq) fits the grid and a TMA coordinate; the
  // element count of one tensor stays below 2^40.
  const long long bh = static_cast<long long>(B) * Hq;
  if (bh > (1LL << 30)) return FA_ERR_UNSUPPORTED;
  if (bh * N * d >= (1LL << 40)) return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

int check_decode_shape(int B, int Hq, int Hkv, int Nq, int Nk, int d, int causal, float scale) {
  if (B <= 0 || Hq <= 0 || Hkv <= 0 || Nq <= 0 || Nk <= 0 || Nq > Nk) return FA_ERR_INVALID_ARGUMENT;
  if (causal != 0 && causal != 1) return FA_ERR_INVALID_ARGUMENT;
  if (!std::isfinite(scale) || !(scale > 0.f)) return FA_ERR_INVALID_ARGUMENT;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  if (Hq % Hkv != 0) return FA_ERR_UNSUPPORTED;
  // Query rows per KV head and (batch, KV head) pairs stay TMA coordinates;
  // element counts of the query and cache tensors stay below 2^40.
  const long long rows = static_cast<long long>(Hq / Hkv) * Nq;
  const long long bkv = static_cast<long long>(B) * Hkv;
  if (rows > (1LL << 30) || bkv > (1LL << 30)) return FA_ERR_UNSUPPORTED;
  if (bkv * rows * d >= (1LL << 40) || bkv * Nk * d >= (1LL << 40)) return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

LaunchCtl make_ctl(const DevState* st) {
  LaunchCtl c;
  c.err = st->err;
  c.budget_ns = g_budget_ns.load(std::memory_order_relaxed);
  c.fault = g_fault.load(std::memory_order_relaxed);
  c.ev_after_pre = static_cast<cudaEvent_t>(g_ev_pre.load(std::memory_order_relaxed));
  c.ev_after_main = static_cast<cudaEvent_t>(g_ev_main.load(std::memory_order_relaxed));
  return c;
}

}  // namespace

int check_current_device() {
  DevState* st = nullptr;
  return device_state(&st);
}

int record_cuda_error(cudaError_t e) { return record_cuda(e); }

namespace {
bool load_encode() {
  std::call_once(g_encode_once, [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      g_encode = reinterpret_cast<EncodeTiledFn>(fn);
  });
  return g_encode != nullptr;
}

bool encode_map(CUtensorMap* map, CUtensorMapDataType dtype, int elem_bytes, const void* base, int cols, int rows,
                int outer, int box_cols, int box_rows) {
  if (!load_encode()) return false;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows),
                        static_cast<cuuint64_t>(outer)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(cols) * elem_bytes,
                           static_cast<cuuint64_t>(cols) * elem_bytes * rows};
  cuuint32_t box[3] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_rows), 1};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = g_encode(map, dtype, 3, const_cast<void*>(base), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}
}  // namespace

bool encode_tile_map(CUtensorMap* map, const void* base, int cols, int rows, int outer, int box_rows) {
  return encode_map(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, base, cols, rows, outer, 64, box_rows);
}

bool encode_bf16_map(CUtensorMap* map, const void* base, int rank, const uint64_t* dims, const uint64_t* strides,
                     const uint32_t* box) {
  if (!load_encode()) return false;
  cuuint64_t d[5], st[4];
  cuuint32_t b[5], es[5];
  for (int i = 0; i < rank; ++i) {
    d[i] = dims[i];
    b[i] = box[i];
    es[i] = 1;
    // A dimension of one element is never stepped along: any valid stride.
    if (i > 0) st[i - 1] = dims[i] == 1 ? dims[0] * 2 : strides[i - 1];
  }
  return g_encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(base), d, st, b, es,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool encode_rows_map(CUtensorMap* map, const Rows& x, int T, int H, int d, int box_rows) {
  const uint64_t dims[3] = {static_cast<uint64_t>(d), static_cast<uint64_t>(T), static_cast<uint64_t>(H)};
  const uint64_t st[2] = {static_cast<uint64_t>(x.ts) * 2, static_cast<uint64_t>(x.hs) * 2};
  const uint32_t box[3] = {64, static_cast<uint32_t>(box_rows), 1};
  return encode_bf16_map(map, x.p, 3, dims, st, box);
}

bool encode_group_map(CUtensorMap* map, const Rows& x, int T, int Hkv, int r, int d, int tokens) {
  const uint64_t dims[4] = {static_cast<uint64_t>(d), static_cast<uint64_t>(r), static_cast<uint64_t>(T),
                            static_cast<uint64_t>(Hkv)};
  const uint64_t st[3] = {static_cast<uint64_t>(x.hs) * 2, static_cast<uint64_t>(x.ts) * 2,
                          static_cast<uint64_t>(x.hs) * 2 * r};
  const uint32_t box[4] = {64, static_cast<uint32_t>(r), static_cast<uint32_t>(tokens), 1};
  return encode_bf16_map(map, x.p, 4, dims, st, box);
}

bool encode_pages_map(CUtensorMap* map, const Pages& x, int n_pages, int Hkv, int page, int d, int box_rows) {
  const uint64_t dims[4] = {static_cast<uint64_t>(d), static_cast<uint64_t>(page), static_cast<uint64_t>(Hkv),
                            static_cast<uint64_t>(n_pages)};
  const uint64_t st[3] = {static_cast<uint64_t>(x.ss) * 2, static_cast<uint64_t>(x.hs) * 2,
                          static_cast<uint64_t>(x.ps) * 2};
  const uint32_t box[4] = {64, static_cast<uint32_t>(box_rows), 1, 1};
  return encode_bf16_map(map, x.p, 4, dims, st, box);
}

bool encode_f32_tile_map(CUtensorMap* map, const void* base, int cols, int rows, int outer, int box_cols,
                         int box_rows) {
  if (box_cols * 4 > 128) return false;
  return encode_map(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, base, cols, rows, outer, box_cols, box_rows);
}

}  // namespace fa

using namespace fa;

extern "C" {

static int fwd_impl(const void* q, const void* k, const void* v, void* o, void* o_resid, float* lse, int B,
                    int Hq, int Hkv, int N, int d, int causal, float scale, void* stream, int window = -1,
                    int prefix = 0) {
  if (window < -1 || prefix < 0) return FA_ERR_INVALID_ARGUMENT;
  if (!q || !k || !v || !o || !lse) return FA_ERR_INVALID_ARGUMENT;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(lse) ||
      !aligned16(o_resid))
    return FA_ERR_INVALID_ARGUMENT;
  int rc = check_shape(B, Hq, Hkv, N, d, causal, scale);
  if (rc != FA_OK) return rc;
  DevState* st = nullptr;
  if ((rc = device_state(&st)) != FA_OK) return rc;
  CUtensorMap tq, tk, tv, to, tr;
  if (!encode_tile_map(&tq, q, d, N, B * Hq, 128) || !encode_tile_map(&tk, k, d, N, B * Hkv, 128) ||
      !encode_tile_map(&tv, v, d, N, B * Hkv, 128) || !encode_tile_map(&to, o, d, N, B * Hq, 128) ||
      !encode_tile_map(&tr, o_resid ? o_resid : o, d, N, B * Hq, 128))
    return FA_ERR_UNSUPPORTED;
  AttnShape s{B, Hq, Hkv, N, d, causal, scale};
  s.window = window;
  s.prefix = prefix;
  cudaError_t e =
      launch_fwd(s, tq, tk, tv, to, tr, o, o_resid, lse, make_ctl(st), static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FA_OK : record_cuda(e);
}

int fa_fwd(const void* q, const void* k, const void* v, void* o, float* lse, int B, int Hq, int Hkv, int N,
           int d, int causal, float scale, void* stream) {
  return fwd_impl(q, k, v, o, nullptr, lse, B, Hq, Hkv, N, d, causal, scale, stream);
}

int fa_fwd_with_residual(const void* q, const void* k, const void* v, void* o, void* o_resid, float* lse, int B,
                         int Hq, int Hkv, int N, int d, int causal, float scale, void* stream) {
  if (!o_resid) return FA_ERR_INVALID_ARGUMENT;
  return fwd_impl(q, k, v, o, o_resid, lse, B, Hq, Hkv, N, d, causal, scale, stream);
}

size_t fa_bwd_workspace_bytes(int B, int Hq, int Hkv, int N, int d) {
  if (check_shape(B, Hq, Hkv, N, d, 0, 1.f) != FA_OK) return 0;
  AttnShape s{B, Hq, Hkv, N, d, 0, 1.f};
  return bwd_workspace_bytes(s);
}

static int bwd_impl(const void* q, const void* k, const void* v, const void* o, const void* o_resid,
                    const void* dout, const float* lse, void* dq, void* dk, void* dv, int B, int Hq, int Hkv, int N,
                    int d, int causal, float scale, void* workspace, size_t workspace_bytes, void* stream,
                    int window = -1, int prefix = 0) {
  if (window < -1 || prefix < 0) return FA_ERR_INVALID_ARGUMENT;
  if (!q || !k || !v || !o || !dout || !lse || !dq || !dk || !dv || !workspace) return FA_ERR_INVALID_ARGUMENT;
  const void* ptrs[] = {q, k, v, o, o_resid, dout, lse, dq, dk, dv, workspace};
  for (const void* p : ptrs)
    if (!aligned16(p)) return FA_ERR_INVALID_ARGUMENT;
  int rc = check_shape(B, Hq, Hkv, N, d, causal, scale);
  if (rc != FA_OK) return rc;
  AttnShape s{B, Hq, Hkv, N, d, causal, scale};
  s.window = window;
  s.prefix = prefix;
  if (workspace_bytes < bwd_workspace_bytes(s)) return FA_ERR_INVALID_ARGUMENT;
  DevState* st = nullptr;
  if ((rc = device_state(&st)) != FA_OK) return rc;
  // The backward streams 64-row query tiles past 128-row key tiles.
  CUtensorMap tq, tk, tv, tdo, tdk, tdv;
  if (!encode_tile_map(&tq, q, d, N, B * Hq, 64) || !encode_tile_map(&tk, k, d, N, B * Hkv, 128) ||
      !encode_tile_map(&tv, v, d, N, B * Hkv, 128) || !encode_tile_map(&tdo, dout, d, N, B * Hq, 64) ||
      !encode_tile_map(&tdk, dk, d, N, B * Hkv, 128) || !encode_tile_map(&tdv, dv, d, N, B * Hkv, 128))
    return FA_ERR_UNSUPPORTED;
  cudaError_t e = launch_bwd(s, tq, tk, tv, tdo, tdk, tdv, o, o_resid, dout, lse, dq, dk, dv, workspace, make_ctl(st),
                             static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FA_OK : record_cuda(e);
}

int fa_bwd(const void* q, const void* k, const void* v, const void* o, const void* dout, const float* lse,
           void* dq, void* dk, void* dv, int B, int Hq, int Hkv, int N, int d, int causal, float scale,
           void* workspace, size_t workspace_bytes, void* stream) {
  return bwd_impl(q, k, v, o, nullptr, dout, lse, dq, dk, dv, B, Hq, Hkv, N, d, causal, scale, workspace,
                  workspace_bytes, stream);
}

int fa_bwd_with_residual(const void* q, const void* k, const void* v, const void* o, const void* o_resid,
                         const void* dout, const float* lse, void* dq, void* dk, void* dv, int B, int Hq, int Hkv,
                         int N, int d, int causal, float scale, void* workspace, size_t workspace_bytes,
                         void* stream) {
  if (!o_resid) return FA_ERR_INVALID_ARGUMENT;
  return bwd_impl(q, k, v, o, o_resid, dout, lse, dq, dk, dv, B, Hq, Hkv, N, d, causal, scale, workspace,
                  workspace_bytes, stream);
}

int fa_fwd_masked(const void* q, const void* k, const void* v, void* o, void* o_resid, float* lse, int B, int Hq,
                  int Hkv, int N, int d, int window, int prefix, float scale, void* stream) {
  return fwd_impl(q, k, v, o, o_resid, lse, B, Hq, Hkv, N, d, 1, scale, stream, window, prefix);
}

int fa_bwd_masked(const void* q, const void* k, const void* v, const void* o, const void* o_resid, const void* dout,
                  const float* lse, void* dq, void* dk, void* dv, int B, int Hq, int Hkv, int N, int d, int window,
                  int prefix, float scale, void* workspace, size_t workspace_bytes, void* stream) {
  return bwd_impl(q, k, v, o, o_resid, dout, lse, dq, dk, dv, B, Hq, Hkv, N, d, 1, scale, workspace,
                  workspace_bytes, stream, window, prefix);
}

int fa_quantize_fp8(const void* x, void* codes, float* scales, int BH, int N, int d, int per_head, void* stream) {
  if (!x || !codes || !scales) return FA_ERR_INVALID_ARGUMENT;
  if (!aligned16(x) || !aligned16(codes) || (reinterpret_cast<uintptr_t>(scales) & 3u)) return FA_ERR_INVALID_ARGUMENT;
  if (BH <= 0 || N <= 0 || (per_head != 0 && per_head != 1)) return FA_ERR_INVALID_ARGUMENT;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  if (static_cast<long long>(BH) * N * d >= (1LL << 40)) return FA_ERR_UNSUPPORTED;
  DevState* st = nullptr;
  int rc = device_state(&st);
  if (rc != FA_OK) return rc;
  cudaError_t e = launch_quantize_fp8(x, codes, scales, BH, N, d, per_head, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FA_OK : record_cuda(e);
}

int fa_fwd_fp8(const void* q8, const float* sq, const void* k8, const float* sk, const void* v8, const float* sv,
               void* o, float* lse, int B, int Hq, int Hkv, int N, int d, int causal, float scale, void* stream) {
  if (!q8 || !sq || !k8 || !sk || !v8 || !sv || !o || !lse) return FA_ERR_INVALID_ARGUMENT;
  const void* ptrs[] = {q8, k8, v8, o, lse};
  for (const void* p : ptrs)
    if (!aligned16(p)) return FA_ERR_INVALID_ARGUMENT;
  const void* sptrs[] = {sq, sk, sv};
  for (const void* p : sptrs)
    if (reinterpret_cast<uintptr_t>(p) & 3u) return FA_ERR_INVALID_ARGUMENT;
  int rc = check_shape(B, Hq, Hkv, N, d, causal, scale);
  if (rc != FA_OK) return rc;
  if (d != 128) return FA_ERR_UNSUPPORTED;
  DevState* st = nullptr;
  if ((rc = device_state(&st)) != FA_OK) return rc;
  // e4m3 tensors: 128 one-byte columns per row, boxes of 128 columns x 128 rows.
  CUtensorMap tq, tk, tv, to;
  if (!encode_map(&tq, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, q8, d, N, B * Hq, 128, 128) ||
      !encode_map(&tk, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, k8, d, N, B * Hkv, 128, 128) ||
      !encode_map(&tv, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, v8, d, N, B * Hkv, 128, 128) ||
      !encode_tile_map(&to, o, d, N, B * Hq, 128))
    return FA_ERR_UNSUPPORTED;
  AttnShape s{B, Hq, Hkv, N, d, causal, scale};
  cudaError_t e =
      launch_fwd_fp8(s, tq, tk, tv, to, o, lse, sq, sk, sv, make_ctl(st), static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FA_OK : record_cuda(e);
}

size_t fa_decode_workspace_bytes(int B, int Hq, int Hkv, int Nq, int Nk, int d) {
  if (check_decode_shape(B, Hq, Hkv, Nq, Nk, d, 0, 1.f) != FA_OK) return 0;
  DecodeShape s{B, Hq, Hkv, Nq, Nk, d, 0, 1.f};
  return decode_workspace_bytes(s);
}

int fa_decode(const void* q, const void* k, const void* v, void* o, float* lse, int B, int Hq, int Hkv, int Nq,
              int Nk, int d, int causal, float scale, void* workspace, size_t workspace_bytes, void* stream) {
  if (!q || !k || !v || !o || !lse || !workspace) return FA_ERR_INVALID_ARGUMENT;
  const void* ptrs[] = {q, k, v, o, lse, workspace};
  for (const void* p : ptrs)
    if (!aligned16(p)) return FA_ERR_INVALID_ARGUMENT;
  int rc = check_decode_shape(B, Hq, Hkv, Nq, Nk, d, causal, scale);
  if (rc != FA_OK) return rc;
  DecodeShape s{B, Hq, Hkv, Nq, Nk, d, causal, scale};
  if (workspace_bytes < decode_workspace_bytes(s)) return FA_ERR_INVALID_ARGUMENT;
  DevState* st = nullptr;
  if ((rc = device_state(&st)) != FA_OK) return rc;
  const DecodePlan plan = make_decode_plan(s, st->sms);
  // The partials of this plan must fit the shape's workspace bound.
  if (static_cast<long long>(plan.G) * plan.MS > plan.W / plan.T + 2LL * plan.G) return FA_ERR_UNSUPPORTED;
  // Queries as [B*Hkv][R][d] (the query heads of a KV head are adjacent),
  // boxes of one row chunk; K and V as [B*Hkv][Nk][d], boxes of 128 keys.
  CUtensorMap tq, tk, tv;
  if (!encode_tile_map(&tq, q, d, plan.R, B * Hkv, 128 / plan.rho) || !encode_tile_map(&tk, k, d, Nk, B * Hkv, 128) ||
      !encode_tile_map(&tv, v, d, Nk, B * Hkv, 128))
    return FA_ERR_UNSUPPORTED;
  LaunchCtl ctl = make_ctl(st);
  ctl.ev_after_pre = nullptr;
  ctl.ev_after_main = static_cast<cudaEvent_t>(g_ev_dec.load(std::memory_order_relaxed));
  cudaError_t e = launch_decode(s, plan, tq, tk, tv, o, lse, workspace, ctl, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FA_OK : record_cuda(e);
}

const char* fa_status_string(int status) {
  switch (status) {
    case FA_OK:
      return "ok";
    case FA_ERR_INVALID_ARGUMENT:
      return "invalid argument (null or misaligned pointer, non-positive size, bad causal flag, "
             "non-finite or non-positive scale, or workspace too small)";
    case FA_ERR_UNSUPPORTED:
      return "unsupported (head dim not 64/128, Hq not a multiple of Hkv, size limit, or device is not "
             "compute capability 10.0)";
    case FA_ERR_CUDA:
      return t_cuda_msg;
    case FA_ERR_TIMEOUT:
      return "a kernel wait ran past the watchdog budget and the kernel gave up";
    case FA_ERR_DATA:
      return "sequence offsets, lengths or page numbers in device memory are out of range";
    default:
      return "unknown status";
  }
}

int fa_check_device_error(void* stream) {
  DevState* st = nullptr;
  int rc = device_state(&st);
  if (rc != FA_OK) return rc;
  cudaError_t e = cudaStreamSynchronize(static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return record_cuda(e);
  unsigned int word = 0;
  e = cudaMemcpy(&word, st->err, sizeof(word), cudaMemcpyDeviceToHost);
  if (e != cudaSuccess) return record_cuda(e);
  if (word == 0) return FA_OK;
  e = cudaMemset(st->err, 0, sizeof(word));
  if (e != cudaSuccess) return record_cuda(e);
  e = cudaDeviceSynchronize();
  if (e != cudaSuccess) return record_cuda(e);
  return (word & ~kErrData) != 0 ? FA_ERR_TIMEOUT : FA_ERR_DATA;
}

void fa_set_watchdog_ns(uint64_t ns) { g_budget_ns.store(ns < 1000000ull ? 1000000ull : ns); }

// ------------------------------------------ packed sequences, paged cache

// Strides: whole 16-byte pieces, positive where there is more than one
// element (a stride of zero would make rows share memory), and below TMA's
// 2^40 bytes.
static bool stride_ok(long long st, long long count) {
  return count <= 1 || (st > 0 && st % 8 == 0 && st < (1LL << 39));
}
static bool rows_ok(const fa_rows* x, int T, int H) {
  return x && x->data && aligned16(x->data) && stride_ok(x->token_stride, T) && stride_ok(x->head_stride, H);
}
static bool pages_ok(const fa_pages* x, int n_pages, int H, int page) {
  return x && x->data && aligned16(x->data) && stride_ok(x->page_stride, n_pages) && stride_ok(x->head_stride, H) &&
         stride_ok(x->slot_stride, page);
}
static Rows as_rows(const fa_rows* x) { return x ? Rows{x->data, x->token_stride, x->head_stride} : Rows{}; }
static Pages as_pages(const fa_pages* x) { return Pages{x->data, x->page_stride, x->head_stride, x->slot_stride}; }
static bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

static int check_seqs(int S, int T, int Hq, int Hkv, int d, int causal, float scale) {
  if (S < 0 || T < 0 || Hq <= 0 || Hkv <= 0) return FA_ERR_INVALID_ARGUMENT;
  if (causal != 0 && causal != 1) return FA_ERR_INVALID_ARGUMENT;
  if (!std::isfinite(scale) || !(scale > 0.f)) return FA_ERR_INVALID_ARGUMENT;
  if ((d != 64 && d != 128) || Hq % Hkv != 0 || Hq / Hkv > 128) return FA_ERR_UNSUPPORTED;
  if (Hq > (1 << 16) || T > (1 << 30) || S > (1 << 24)) return FA_ERR_UNSUPPORTED;
  // CTAs of one launch: (units of at least one token) * KV heads.
  if ((static_cast<long long>(T) + S + 4 * kShareCtas) * Hkv > 0x7fffffffLL) return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

static int check_cache(int n_pages, int page_size, int max_pages, int max_q) {
  if (n_pages < 0 || page_size <= 0 || max_pages < 0 || max_q < 0) return FA_ERR_INVALID_ARGUMENT;
  if (page_size % 8 != 0 || page_size > (1 << 20)) return FA_ERR_UNSUPPORTED;
  if (static_cast<long long>(max_pages) * page_size > (1 << 30)) return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

size_t fa_packed_fwd_workspace_bytes(int S, int T, int Hq, int Hkv, int d) {
  if (check_seqs(S, T, Hq, Hkv, d, 0, 1.f) != FA_OK) return 0;
  return packed_fwd_workspace_bytes(SeqShape{S, T, nullptr, Hq, Hkv, d, 0, 1.f}, nullptr);
}

int fa_packed_fwd(const fa_rows* q, const fa_rows* k, const fa_rows* v, const fa_rows* o, const fa_rows* o_resid,
                  float* lse, const int* cu_seqlens, int S, int T, int Hq, int Hkv, int d, int causal, float scale,
                  void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_seqs(S, T, Hq, Hkv, d, causal, scale);
  if (rc != FA_OK) return rc;
  if (S == 0 || T == 0) return FA_OK;
  if (!rows_ok(q, T, Hq) || !rows_ok(k, T, Hkv) || !rows_ok(v, T, Hkv) || !rows_ok(o, T, Hq) ||
      (o_resid && !rows_ok(o_resid, T, Hq)) || !lse || !aligned4(lse) || !cu_seqlens || !aligned4(cu_seqlens) ||
      !workspace || !aligned16(workspace))
    return FA_ERR_INVALID_ARGUMENT;
  const SeqShape s{S, T, cu_seqlens, Hq, Hkv, d, causal, scale};
  if (workspace_bytes < packed_fwd_workspace_bytes(s, nullptr)) return FA_ERR_INVALID_ARGUMENT;
  DevState* st = nullptr;
  if ((rc = device_state(&st)) != FA_OK) return rc;
  const int ctas = st->sms < kShareCtas ? st->sms : kShareCtas;
  cudaError_t e = launch_packed_fwd(s, nullptr, as_rows(q), as_rows(o), as_rows(o_resid), as_rows(k), as_rows(v),
                                    Pages{}, Pages{}, lse, workspace, ctas, make_ctl(st),
                                    static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FA_OK : record_cuda(e);
}

size_t fa_packed_bwd_workspace_bytes(int S, int T, int Hq, int Hkv, int d) {
  if (check_seqs(S, T, Hq, Hkv, d, 0, 1.f) != FA_OK) return 0;
  return packed_bwd_workspace_bytes(SeqShape{S, T, nullptr, Hq, Hkv, d, 0, 1.f});
}

int fa_packed_bwd(const fa_rows* q, const fa_rows* k, const fa_rows* v, const fa_rows* o, const fa_rows* o_resid,
                  const fa_rows* dout, const float* lse, const fa_rows* dq, const fa_rows* dk, const fa_rows* dv,
                  const int* cu_seqlens, int S, int T, int Hq, int Hkv, int d, int causal, float scale,
                  void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_seqs(S, T, Hq, Hkv, d, causal, scale);
  if (rc != FA_OK) return rc;
  if (S == 0 || T == 0) return FA_OK;
  if (!rows_ok(q, T, Hq) || !rows_ok(k, T, Hkv) || !rows_ok(v, T, Hkv) || !rows_ok(o, T, Hq) ||
      (o_resid && !rows_ok(o_resid, T, Hq)) || !rows_ok(dout, T, Hq) || !rows_ok(dq, T, Hq) || !rows_ok(dk, T, Hkv) ||
      !rows_ok(dv, T, Hkv) || !lse || !aligned4(lse) || !cu_seqlens || !aligned4(cu_seqlens) || !workspace ||
      !aligned16(workspace))
    return FA_ERR_INVALID_ARGUMENT;
  const SeqShape s{S, T, cu_seqlens, Hq, Hkv, d, causal, scale};
  if (workspace_bytes < packed_bwd_workspace_bytes(s)) return FA_ERR_INVALID_ARGUMENT;
  DevState* st = nullptr;
  if ((rc = device_state(&st)) != FA_OK) return rc;
  cudaError_t e = launch_packed_bwd(s, as_rows(q), as_rows(k), as_rows(v), as_rows(o), as_rows(o_resid), as_rows(dout),
                                    lse, as_rows(dq), as_rows(dk), as_rows(dv), workspace, make_ctl(st),
                                    static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FA_OK : record_cuda(e);
}

size_t fa_paged_fwd_workspace_bytes(int S, int T, int max_q, int Hq, int Hkv, int d, int page_size, int max_pages) {
  if (check_seqs(S, T, Hq, Hkv, d, 0, 1.f) != FA_OK || check_cache(0, page_size, max_pages, max_q) != FA_OK) return 0;
  const SeqShape s{S, T, nullptr, Hq, Hkv, d, 0, 1.f};
  CacheShape c{0, page_size, max_pages, nullptr, nullptr, 0, max_q < T ? max_q : T};
  return paged_few_rows(s, c) ? paged_few_workspace_bytes(s, c, kShareCtas)
                              : packed_fwd_workspace_bytes(s, &c);
}

int fa_paged_fwd(const fa_rows* q, const fa_pages* k_pages, const fa_pages* v_pages, const fa_rows* o, float* lse,
                 int n_pages, int page_size, const int* block_table, int64_t table_stride, int max_pages,
                 const int* seq_lens, const int* cu_seqlens, int S, int T, int max_q, int Hq, int Hkv, int d,
                 int causal, float scale, void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_seqs(S, T, Hq, Hkv, d, causal, scale);
  if (rc != FA_OK || (rc = check_cache(n_pages, page_size, max_pages, max_q)) != FA_OK) return rc;
  if (!cu_seqlens && S != T) return FA_ERR_INVALID_ARGUMENT;
  if (S == 0 || T == 0) return FA_OK;
  if (n_pages == 0 || max_pages == 0 || max_q == 0) return FA_ERR_INVALID_ARGUMENT;
  if (!rows_ok(q, T, Hq) || !rows_ok(o, T, Hq) || !pages_ok(k_pages, n_pages, Hkv, page_size) ||
      !pages_ok(v_pages, n_pages, Hkv, page_size) || !lse || !aligned4(lse) || !block_table || !aligned4(block_table) ||
      table_stride < (S > 1 ? max_pages : 0) || !seq_lens || !aligned4(seq_lens) || !aligned4(cu_seqlens) ||
      !workspace || !aligned16(workspace))
    return FA_ERR_INVALID_ARGUMENT;
  const SeqShape s{S, T, cu_seqlens, Hq, Hkv, d, causal, scale};
  const CacheShape c{n_pages, page_size, max_pages, seq_lens, block_table, table_stride, max_q < T ? max_q : T};
  const bool few = paged_few_rows(s, c);
  const size_t need = few ? paged_few_workspace_bytes(s, c, kShareCtas) : packed_fwd_workspace_bytes(s, &c);
  if (workspace_bytes < need) return FA_ERR_INVALID_ARGUMENT;
  DevState* st = nullptr;
  if ((rc = device_state(&st)) != FA_OK) return rc;
  const int ctas = st->sms < kShareCtas ? st->sms : kShareCtas;
  cudaError_t e =
      few ? launch_paged_few(s, c, as_rows(q), as_rows(o), as_pages(k_pages), as_pages(v_pages), lse, workspace, ctas,
                             make_ctl(st), static_cast<cudaStream_t>(stream))
          : launch_packed_fwd(s, &c, as_rows(q), as_rows(o), Rows{}, Rows{}, Rows{}, as_pages(k_pages),
                              as_pages(v_pages), lse, workspace, ctas, make_ctl(st), static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FA_OK : record_cuda(e);
}

// Checks the rotation's arguments and fills its shape.
static int rope_shape(RopeShape* s, int T, int Hq, int Hkv, int d, const int* positions, const double* inv_freq,
                      const int* sections, int n_sections, int interleaved, int inverse, bool need_positions) {
  if (T < 0 || Hq < 0 || Hkv < 0 || (interleaved != 0 && interleaved != 1) || (inverse != 0 && inverse != 1))
    return FA_ERR_INVALID_ARGUMENT;
  if (n_sections < 0 || (n_sections > 0 && !sections)) return FA_ERR_INVALID_ARGUMENT;
  if ((d != 64 && d != 128) || n_sections > 4) return FA_ERR_UNSUPPORTED;
  if (Hq > (1 << 16) || Hkv > (1 << 16) || T > (1 << 30)) return FA_ERR_UNSUPPORTED;
  *s = RopeShape{};
  int pairs = 0;
  for (int i = 0; i < n_sections; ++i) {
    if (sections[i] <= 0 || sections[i] > d) return FA_ERR_INVALID_ARGUMENT;
    pairs += sections[i];
    s->section_end[i] = pairs;
  }
  if (2 * pairs > d) return FA_ERR_INVALID_ARGUMENT;
  if (pairs % 8 != 0) return FA_ERR_UNSUPPORTED;
  if (pairs > 0 && (!inv_freq || (reinterpret_cast<uintptr_t>(inv_freq) & 7u))) return FA_ERR_INVALID_ARGUMENT;
  if (pairs > 0 && ((need_positions && !positions) || !aligned4(positions))) return FA_ERR_INVALID_ARGUMENT;
  s->T = T;
  s->Hq = Hq;
  s->Hkv = Hkv;
  s->d = d;
  s->pairs = pairs;
  s->interleaved = interleaved;
  s->sign = inverse ? -1.f : 1.f;
  s->positions = positions;
  s->inv_freq = inv_freq;
  s->n_sections = n_sections;
  return FA_OK;
}

int fa_rope(const fa_rows* q, const fa_rows* k, const fa_rows* q_out, const fa_rows* k_out, const int* positions,
            const double* inv_freq, const int* sections, int n_sections, int T, int Hq, int Hkv, int d,
            int interleaved, int inverse, void* stream) {
  RopeShape s;
  int rc = rope_shape(&s, T, Hq, Hkv, d, positions, inv_freq, sections, n_sections, interleaved, inverse, true);
  if (rc != FA_OK) return rc;
  if (s.pairs == 0 || Hq + Hkv == 0) return FA_ERR_INVALID_ARGUMENT;
  if (T == 0) return FA_OK;
  if ((Hq > 0 && (!rows_ok(q, T, Hq) || !rows_ok(q_out, T, Hq))) ||
      (Hkv > 0 && (!rows_ok(k, T, Hkv) || !rows_ok(k_out, T, Hkv))))
    return FA_ERR_INVALID_ARGUMENT;
  DevState* st = nullptr;
  if ((rc = device_state(&st)) != FA_OK) return rc;
  cudaError_t e = launch_rope(s, as_rows(Hq ? q : nullptr), as_rows(Hkv ? k : nullptr), as_rows(Hq ? q_out : nullptr),
                              as_rows(Hkv ? k_out : nullptr), static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FA_OK : record_cuda(e);
}

int fa_paged_append(const fa_rows* q, const fa_rows* k, const fa_rows* v, const fa_rows* q_out,
                    const fa_pages* k_pages, const fa_pages* v_pages, int n_pages, int page_size,
                    const int* block_table, int64_t table_stride, int max_pages, const int* seq_lens,
                    const int* cu_seqlens, int S, int T, const int* positions, const double* inv_freq,
                    const int* sections, int n_sections, int Hq, int Hkv, int d, int interleaved, void* stream) {
  if (S < 0 || Hkv <= 0) return FA_ERR_INVALID_ARGUMENT;
  RopeShape s;
  int rc = rope_shape(&s, T, Hq, Hkv, d, positions, inv_freq, sections, n_sections, interleaved, 0, n_sections > 1);
  if (rc != FA_OK || (rc = check_cache(n_pages, page_size, max_pages, 0)) != FA_OK) return rc;
  if (S > (1 << 24)) return FA_ERR_UNSUPPORTED;
  if (!cu_seqlens && S != T) return FA_ERR_INVALID_ARGUMENT;
  if (S == 0 || T == 0) return FA_OK;
  if (n_pages == 0 || max_pages == 0) return FA_ERR_INVALID_ARGUMENT;
  if ((Hq > 0 && (!rows_ok(q, T, Hq) || !rows_ok(q_out, T, Hq))) || !rows_ok(k, T, Hkv) || !rows_ok(v, T, Hkv) ||
      !pages_ok(k_pages, n_pages, Hkv, page_size) || !pages_ok(v_pages, n_pages, Hkv, page_size) || !block_table ||
      !aligned4(block_table) || table_stride < (S > 1 ? max_pages : 0) || !seq_lens || !aligned4(seq_lens) ||
      !aligned4(cu_seqlens))
    return FA_ERR_INVALID_ARGUMENT;
  DevState* st = nullptr;
  if ((rc = device_state(&st)) != FA_OK) return rc;
  const SeqShape seq{S, T, cu_seqlens, Hq, Hkv, d, 0, 1.f};
  const CacheShape c{n_pages, page_size, max_pages, seq_lens, block_table, table_stride, T};
  cudaError_t e = launch_paged_append(s, seq, c, as_rows(Hq ? q : nullptr), as_rows(k), as_rows(v),
                                      as_rows(Hq ? q_out : nullptr), as_pages(k_pages), as_pages(v_pages), st->err,
                                      static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FA_OK : record_cuda(e);
}

// Test hook, declared in include/fa_test.h: selects a deliberate stall
// (1 = the forward producer never loads the first K tile) so that the
// watchdog path can be exercised without faulting the GPU.
void fa_test_set_fault(int code) { g_fault.store(code); }

int fa_test_exp2(const float* x, float* y_poly, float* y_ex2, int n, void* stream) {
  if (!x || !y_poly || !y_ex2 || n < 0) return FA_ERR_INVALID_ARGUMENT;
  if (n == 0) return FA_OK;
  const int blocks = (n + 255) / 256 < 1184 ? (n + 255) / 256 : 1184;
  test_exp2_kernel<<<blocks, 256, 0, static_cast<cudaStream_t>(stream)>>>(x, y_poly, y_ex2, n);
  cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? FA_OK : record_cuda(e);
}

int fa_test_exp2_accurate(const float* x, float* y, int n, void* stream) {
  if (!x || !y || n < 0) return FA_ERR_INVALID_ARGUMENT;
  if (n == 0) return FA_OK;
  const int blocks = (n + 255) / 256 < 1184 ? (n + 255) / 256 : 1184;
  test_exp2_accurate_kernel<<<blocks, 256, 0, static_cast<cudaStream_t>(stream)>>>(x, y, n);
  cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? FA_OK : record_cuda(e);
}

int fa_test_decode_plan(int B, int Hq, int Hkv, int Nq, int Nk, int d, int num_ctas, long long* out) {
  if (!out || num_ctas < 1) return FA_ERR_INVALID_ARGUMENT;
  const int rc = check_decode_shape(B, Hq, Hkv, Nq, Nk, d, 0, 1.f);
  if (rc != FA_OK) return rc;
  const DecodeShape s{B, Hq, Hkv, Nq, Nk, d, 0, 1.f};
  const DecodePlan p = make_decode_plan(s, num_ctas);
  const long long v[8] = {p.W, p.T, p.G, p.MS, p.R, p.rho, p.rv, p.n_chunks};
  for (int i = 0; i < 8; ++i) out[i] = v[i];
  return FA_OK;
}

int fa_test_packed_layout(int S, int T, int Hq, int Hkv, int d, int page_size, int max_pages, int num_sms,
                          long long* out) {
  if (!out || num_sms < 1) return FA_ERR_INVALID_ARGUMENT;
  int rc = check_seqs(S, T, Hq, Hkv, d, 0, 1.f);
  if (rc != FA_OK || (page_size != 0 && (rc = check_cache(0, page_size, max_pages, T)) != FA_OK)) return rc;
  const SeqShape s{S, T, nullptr, Hq, Hkv, d, 0, 1.f};
  const CacheShape c{0, page_size, max_pages, nullptr, nullptr, 0, T};
  packed_fwd_layout(s, page_size ? &c : nullptr, num_sms < kShareCtas ? num_sms : kShareCtas, out);
  return FA_OK;
}

void fa_profile_set_decode_event(void* after_main) { g_ev_dec.store(after_main); }

void fa_profile_set_bwd_events(void* after_pre, void* after_main) {
  g_ev_pre.store(after_pre);
  g_ev_main.store(after_main);
}

}  // extern "C"
