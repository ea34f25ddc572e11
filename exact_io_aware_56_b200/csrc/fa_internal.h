// Internal interface between the C-ABI layer (fa_api.cpp) and the kernel
// launchers (fa_fwd.cu, fa_bwd.cu). Not installed, not part of the ABI.
#pragma once

#include <atomic>
#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace fa {

struct AttnShape {
  int B, Hq, Hkv, N, d;
  int causal;
  float scale;
  int window = -1;  // left window of the causal mask, -1 = none
  int prefix = 0;   // keys below this index are visible to every query
  // 0: no mask; 1: causal; 2: causal with a window and/or a prefix
  // (key j visible to query i iff (j <= i and i - j <= window) or j < prefix).
  int mask_kind() const { return !causal ? 0 : (window < 0 && prefix == 0 ? 1 : 2); }
};

struct LaunchCtl {
  unsigned int* err;        // device error word (watchdog)
  uint64_t budget_ns;       // watchdog budget per wait
  int fault;                // test-only fault injection selector (0 = none)
  cudaEvent_t ev_after_pre;   // optional timing events (see fa_profile.h)
  cudaEvent_t ev_after_main;
};

// Number of heads to schedule together so that their per-head working set
// (`bytes_per_head`) stays within a share of L2 that the resident CTAs can
// keep hot; at least 1, at most `heads`.
inline int l2_head_group(long long bytes_per_head, int heads) {
  constexpr long long kBudget = 48ll << 20;
  long long g = bytes_per_head > 0 ? kBudget / bytes_per_head : heads;
  if (g < 1) g = 1;
  if (g > heads) g = heads;
  return static_cast<int>(g);
}

// Encodes a 3-D bf16 tensor map over [outer][rows][cols] with a box of
// 64 columns x box_rows rows and 128-byte swizzle. Returns false on failure.
bool encode_tile_map(CUtensorMap* map, const void* base, int cols, int rows, int outer, int box_rows);

// Same for an fp32 tensor, box of box_cols x box_rows (box_cols * 4 <= 128).
bool encode_f32_tile_map(CUtensorMap* map, const void* base, int cols, int rows, int outer, int box_cols,
                         int box_rows);

// Checks that the current device is supported (compute capability 10.0),
// once per device, as every entry point does before its first launch.
// Returns FA_OK or the entry points' error status.
int check_current_device();

// Keeps `e` as the message of FA_ERR_CUDA for fa_status_string and returns
// FA_ERR_CUDA.
int record_cuda_error(cudaError_t e);

// o_resid may be null (no residual written). to and tr are bf16 tensor maps
// of o and o_resid laid out like q (tr unused without a residual).
cudaError_t launch_fwd(const AttnShape& s, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                       const CUtensorMap& to, const CUtensorMap& tr, void* o, void* o_resid, float* lse,
                       const LaunchCtl& ctl, cudaStream_t stream);

// FP8 mode (d = 128, masks 0 and 1): q, k, v are e4m3 codes behind 1-byte
// tensor maps with 128-column boxes; sq, sk, sv the block scales; to the
// bf16 tensor map of o.
cudaError_t launch_fwd_fp8(const AttnShape& s, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                           const CUtensorMap& to, void* o, float* lse, const float* sq, const float* sk,
                           const float* sv, const LaunchCtl& ctl, cudaStream_t stream);

// e4m3 block quantization of a bf16 tensor [BH][N][d]: scales per 128-row
// block ([BH][ceil(N/128)]) or per head ([BH]); see fa.h.
cudaError_t launch_quantize_fp8(const void* x, void* codes, float* scales, int BH, int N, int d, int per_head,
                                cudaStream_t stream);

size_t bwd_workspace_bytes(const AttnShape& s);

// tdk and tdv: bf16 tensor maps of dk and dv laid out like k (128-row boxes).
cudaError_t launch_bwd(const AttnShape& s, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                       const CUtensorMap& tdo, const CUtensorMap& tdk, const CUtensorMap& tdv, const void* o,
                       const void* o_resid, const void* dout, const float* lse, void* dq, void* dk, void* dv,
                       void* workspace, const LaunchCtl& ctl, cudaStream_t stream);

// Decode / short-query attention: Nq queries per head against an Nk-key
// cache, queries at the last Nq positions.
struct DecodeShape {
  int B, Hq, Hkv, Nq, Nk, d;
  int causal;
  float scale;
};

// At most this many CTAs run the decode kernel (one per SM up to here); the
// workspace bound below depends on it.
constexpr int kDecodeMaxCtas = 256;

// Stream-K partition of the decode work. Units are (batch, KV head, chunk of
// 128/rho query rows) with T key tiles of 128 keys each; the W = units * T
// tiles, in unit order, are cut into G contiguous runs of nearly equal
// length, run c being tiles [lo(c), lo(c+1)). A run touches at most MS units.
struct DecodePlan {
  long long W;
  int T, G, MS;
  int R;         // query rows per KV head: (Hq / Hkv) * Nq
  int rho;       // replication of the chunk's rows over the 128 lanes (4, 2 or 1)
  int rv;        // stored rows per copy and partial: min(128 / rho, R)
  int n_chunks;  // row chunks per KV head
  __host__ __device__ long long lo(long long c) const { return c * W / G; }
  // The run holding tile t: the largest c with lo(c) <= t.
  __host__ __device__ int cta_of(long long t) const { return static_cast<int>(((t + 1) * G + W - 1) / W) - 1; }
};

DecodePlan make_decode_plan(const DecodeShape& s, int num_ctas);

// Workspace for any plan of this shape with G <= kDecodeMaxCtas: partial O
// (fp32, d per row) and logsumexp for (units + 2 * G) partials of rho * rv rows
// (G * MS <= W / T + 2 G).
size_t decode_workspace_bytes(const DecodeShape& s);

cudaError_t launch_decode(const DecodeShape& s, const DecodePlan& plan, const CUtensorMap& tq,
                          const CUtensorMap& tk, const CUtensorMap& tv, void* o, float* lse, void* workspace,
                          const LaunchCtl& ctl, cudaStream_t stream);

// ------------------------------------------ packed sequences, paged cache

// Device views with strides in elements and contiguous rows of d elements:
// [tokens][heads][d] and [pages][heads][slots][d].
struct Rows {
  void* p;
  long long ts, hs;  // token and head stride
};
struct Pages {
  void* p;
  long long ps, hs, ss;  // page, head and slot stride
};

// Encodes a bf16 tensor map of `rank` dimensions (innermost first, strides
// in bytes of dimensions 1..rank-1) with a box of 64 columns and 128-byte
// swizzle. Returns false on failure.
bool encode_bf16_map(CUtensorMap* map, const void* base, int rank, const uint64_t* dims, const uint64_t* strides,
                     const uint32_t* box);

// Sequence layout of a packed call: sequence b holds tokens [cu[b], cu[b+1])
// of the T rows. cu == nullptr: one token each (S == T).
struct SeqShape {
  int S, T;
  const int* cu;
  int Hq, Hkv, d;
  int causal;
  float scale;
  int r() const { return Hq / Hkv; }
};

// Paged cache: sequence b's keys are the first lens[b] slots of the pages
// table[b * table_stride + 0, 1, ...].
struct CacheShape {
  int n_pages, page, max_pages;
  const int* lens;
  const int* table;
  long long table_stride;
  int max_q;  // no sequence of the call has more new tokens
};

// Rows per TMA box of a page: the largest power of two that divides both a
// page and a 128-key tile, so that no box straddles pages.
inline int page_box(int page) {
  int b = 1;
  while (b < 128 && page % (2 * b) == 0) b *= 2;
  return b;
}

// Sets a kernel's dynamic shared memory limit the first time that it is
// launched on a device (the call costs a microsecond of host time).
struct SmemOnce {
  std::atomic<uint64_t> done{0};  // one bit per device
  cudaError_t set(const void* kern, int bytes) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
    return e;
  }
};

// Launches a kernel that may start beside the one before it on the stream
// (programmatic dependent launch) and waits for it with pdl_wait().
template <typename... P, typename... A>
cudaError_t launch_dependent(void (*kern)(P...), dim3 grid, int threads, size_t smem, cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<P>(args)...);
}

// At most this many multiprocessors (a B200's) share the work that is cut along
// the keys; the workspace sizes depend on it.
constexpr int kShareCtas = 148;

// True when every sequence's query rows of a KV head fit one 128-row tile:
// these calls take the few-row kernel (fa_paged.cu), the others the prompt
// kernel (fa_packed.cu).
inline bool paged_few_rows(const SeqShape& s, const CacheShape& c) {
  return static_cast<long long>(s.r()) * c.max_q <= 128;
}

size_t paged_few_workspace_bytes(const SeqShape& s, const CacheShape& c, int ctas);
cudaError_t launch_paged_few(const SeqShape& s, const CacheShape& c, const Rows& q, const Rows& o, const Pages& k,
                             const Pages& v, float* lse, void* workspace, int sms, const LaunchCtl& ctl,
                             cudaStream_t stream);

// Work item of the prompt kernels (fa_plan.cuh): all that a CTA needs to
// start, in one load.
struct alignas(16) PlanItem {
  int base, n;   // the sequence's first row and its tokens
  int off;       // place of its first token (paged), else 0
  int tok0;      // first token of the item
  int j0, j1;    // forward: key tiles; backward: (head, query tile) steps
  int slot;      // part of a unit cut along its keys, -1: whole unit
  int seq;
  int kvh;       // KV head, where the items carry it
};

size_t packed_fwd_workspace_bytes(const SeqShape& s, const CacheShape* c);
// For tests: see fa_test_packed_layout.
void packed_fwd_layout(const SeqShape& s, const CacheShape* c, int sms, long long* out);
cudaError_t launch_packed_fwd(const SeqShape& s, const CacheShape* c, const Rows& q, const Rows& o, const Rows& resid,
                              const Rows& krows, const Rows& vrows, const Pages& kpages, const Pages& vpages,
                              float* lse, void* workspace, int sms, const LaunchCtl& ctl, cudaStream_t stream);

size_t packed_bwd_workspace_bytes(const SeqShape& s);
cudaError_t launch_packed_bwd(const SeqShape& s, const Rows& q, const Rows& k, const Rows& v, const Rows& o,
                              const Rows& resid, const Rows& dout, const float* lse, const Rows& dq, const Rows& dk,
                              const Rows& dv, void* workspace, const LaunchCtl& ctl, cudaStream_t stream);

// 3-D map of a [T][H][d] view, box_rows tokens of one head; and the 4-D map
// (d, heads of a KV group, tokens, KV heads) whose box is all r heads of a
// group times `tokens` tokens, in token-major order.
bool encode_rows_map(CUtensorMap* map, const Rows& x, int T, int H, int d, int box_rows);
bool encode_group_map(CUtensorMap* map, const Rows& x, int T, int Hkv, int r, int d, int tokens);
// 4-D map (d, slots, heads, pages) of a paged tensor, box_rows slots of one head.
bool encode_pages_map(CUtensorMap* map, const Pages& x, int n_pages, int Hkv, int page, int d, int box_rows);

// Sequence b's tokens [start, start + n), or n = 0 when its offsets or
// length are out of range. `lens`/`max_len` only for a paged cache.
struct SeqRange {
  int start, n, len;
  bool bad;
};
__host__ __device__ inline SeqRange seq_range(const int* cu, const int* lens, int b, int T, int max_q, long long max_len) {
  SeqRange x;
  x.start = cu ? cu[b] : b;
  const long long end = cu ? cu[b + 1] : static_cast<long long>(b) + 1;
  const long long n = end - x.start;
  x.len = lens ? lens[b] : static_cast<int>(n < 0 ? 0 : n);
  x.bad = x.start < 0 || n < 0 || end > T || n > max_q || x.len < 0 || x.len > max_len;
  x.n = x.bad ? 0 : static_cast<int>(n);
  return x;
}

// Rotary positions and the append to a paged cache (fa_rope.cu).
struct RopeShape {
  int T, Hq, Hkv, d;
  int pairs;          // rotated pairs (0: no rotation)
  int interleaved;    // pairs (2i, 2i + 1), else (i, i + pairs)
  float sign;         // -1: the inverse rotation
  const int* positions;  // [axes][T]
  const double* inv_freq;  // [pairs], radians per position
  int n_sections;
  int section_end[4];  // pair i goes by axis a for section_end[a-1] <= i < section_end[a]
};
cudaError_t launch_rope(const RopeShape& s, const Rows& q, const Rows& k, const Rows& q_out, const Rows& k_out,
                        cudaStream_t stream);
cudaError_t launch_paged_append(const RopeShape& s, const SeqShape& seq, const CacheShape& c, const Rows& q,
                                const Rows& k, const Rows& v, const Rows& q_out, const Pages& k_pages,
                                const Pages& v_pages, unsigned int* err, cudaStream_t stream);

}  // namespace fa
