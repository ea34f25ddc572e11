// Rotary positions of queries and keys, and the append of new keys and
// values to a paged cache (sm_100a).
//
// Pair i of a head, (x_a, x_b), is turned by the angle p f_i, p the token's
// position on the axis of i's section, f_i its frequency:
//   y_a = x_a cos - x_b sin,  y_b = x_b cos + x_a sin.
// The rotation is orthogonal, so its backward is the rotation by the negative
// angle (sign = -1). Elements behind the pairs are copied.
//
// Bound: HBM, every element read and written once. Angles: p f_i / 2 pi in
// float64, its fraction of a turn then goes to sincospi in float32: a float32
// angle at p = 10^5 would be off by 4e-3. One block takes a few tokens and
// computes their cosines and sines once, into shared memory, for all heads;
// a thread then turns eight pairs of one head per step (two 16-byte loads,
// two 16-byte stores). Measured at 16384 tokens, 32 + 8 heads, d = 128: 57.6
// us, 5.8 TB/s (a copy of the same tensors takes 58.1); with 39 registers
// (six blocks per SM instead of eight) and ordinary accesses 61.8; with four
// steps' loads ahead of the first store, in 80 registers, 75.
//
// The append adds to each token its place len_b - n_b + i in its sequence
// (found by a 32-way warp search of the offsets), and from the block table
// the page and slot that the turned key and the value go to; q is turned in
// the same launch, so that a decode step needs one.

#include <cuda_bf16.h>

#include "fa_internal.h"
#include "sm100.cuh"

namespace fa {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 16;  // tokens per block

struct RopeArgs {
  RopeShape s;
  Rows q, k, v, qo, ko;
  Pages kp, vp;
  const int* cu;
  const int* lens;
  const int* table;
  long long table_stride, max_len;
  int S, n_pages, page, tokens;  // tokens: per block
  unsigned int* err;
};

// The largest b in [0, S) with cu[b] <= t, or 0, by the whole warp.
__device__ __forceinline__ int find_token_seq(const int* cu, int S, int t, int lane) {
  int lo = 0, n = S;
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int k = lane * step;
    const bool le = k < n && (k == 0 || cu[lo + k] <= t);
    // Lanes up to the last that qualifies (offsets out of order may leave gaps).
    const int cnt = 32 - __clz(__ballot_sync(0xffffffffu, le));
    lo += (cnt - 1) * step;
    n = min(step, n - (cnt - 1) * step);
  }
  return lo;
}

// Streaming (evict-first) accesses: every element passes once.
__device__ __forceinline__ void load16(const __nv_bfloat16* p, uint4& x) { x = __ldcs(reinterpret_cast<const uint4*>(p)); }
__device__ __forceinline__ void store16(__nv_bfloat16* p, const uint4& x) { __stcs(reinterpret_cast<uint4*>(p), x); }

// Turns two bf16 pairs held as (a0, a1) in a and (b0, b1) in b.
__device__ __forceinline__ void turn2(uint32_t& a, uint32_t& b, const float2& t0, const float2& t1) {
  const float2 x = __bfloat1622float2(*reinterpret_cast<__nv_bfloat162*>(&a));
  const float2 y = __bfloat1622float2(*reinterpret_cast<__nv_bfloat162*>(&b));
  a = pack_bf16x2(x.x * t0.x - y.x * t0.y, x.y * t1.x - y.y * t1.y);
  b = pack_bf16x2(y.x * t0.x + x.x * t0.y, y.y * t1.x + x.y * t1.y);
}
// Turns one bf16 pair held in one register.
__device__ __forceinline__ void turn1(uint32_t& ab, const float2& t) {
  const float2 x = __bfloat1622float2(*reinterpret_cast<__nv_bfloat162*>(&ab));
  ab = pack_bf16x2(x.x * t.x - x.y * t.y, x.y * t.x + x.x * t.y);
}

template <bool APPEND>
__global__ void __launch_bounds__(kThreads, 8) rope_kernel(const RopeArgs a) {
  __shared__ float2 turns[kThreads];           // [token][pair]: cos, sin
  __shared__ long long k_at[kMaxTokens];       // page offset of the token's key, -1: none
  __shared__ long long v_at[kMaxTokens];
  __shared__ int place[kMaxTokens];            // place in the sequence
  __shared__ bool here[kMaxTokens];            // the token belongs to a sequence
  const int t0 = blockIdx.x * a.tokens;
  const int nt = min(a.tokens, a.s.T - t0);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if constexpr (APPEND) {
    for (int i = warp; i < nt; i += kThreads / 32) {
      const int t = t0 + i;
      const int b = a.cu ? find_token_seq(a.cu, a.S, t, lane) : t;
      if (lane == 0) {
        const SeqRange s = seq_range(a.cu, a.lens, b, a.s.T, a.s.T, a.max_len);
        const bool in = t >= s.start && t - s.start < s.n;
        const int at = s.len - s.n + (t - s.start);
        long long ka = -1, va = -1;
        if (s.bad) {
          atomicOr(a.err, kErrData);
        } else if (in && at >= 0) {
          const int pi = at / a.page;
          const int pg = a.table[static_cast<long long>(b) * a.table_stride + pi];
          if (pg >= 0 && pg < a.n_pages) {
            ka = pg * a.kp.ps + (at - pi * a.page) * a.kp.ss;
            va = pg * a.vp.ps + (at - pi * a.page) * a.vp.ss;
          } else {
            atomicOr(a.err, kErrData);
          }
        }
        k_at[i] = ka;
        v_at[i] = va;
        place[i] = at;
        here[i] = in;
      }
    }
    if (!a.s.positions) __syncthreads();
  }
  const int P = a.s.pairs;
  for (int x = threadIdx.x; x < nt * P; x += kThreads) {
    const int i = x / P, p = x - i * P;
    int axis = 0;
    while (axis < a.s.n_sections - 1 && p >= a.s.section_end[axis]) ++axis;
    const int pos = APPEND && !a.s.positions ? place[i] : a.s.positions[static_cast<long long>(axis) * a.s.T + t0 + i];
    const double turn = static_cast<double>(pos) * (a.s.inv_freq[p] * 0.15915494309189533577);
    float sn, cs;
    sincospif(static_cast<float>(2.0 * (turn - rint(turn))), &sn, &cs);
    turns[x] = make_float2(cs, sn * a.s.sign);
  }
  __syncthreads();
  // Steps of 16 elements: d / 16 for each head of q, then k, then v.
  const int per_head = a.s.d / 16;
  const int heads = a.s.Hq + a.s.Hkv * (APPEND ? 2 : 1);
  const int per_token = heads * per_head;
  for (int x = threadIdx.x; x < nt * per_token; x += kThreads) {
    const int i = x / per_token;
    const int y = x - i * per_token;
    const int head = y / per_head;
    const int c = y - head * per_head;
    const long long t = t0 + i;
    const __nv_bfloat16* src;
    __nv_bfloat16* dst;
    bool rotated = true;
    if (APPEND && !here[i]) continue;
    if (head < a.s.Hq) {
      src = static_cast<const __nv_bfloat16*>(a.q.p) + t * a.q.ts + head * a.q.hs;
      dst = static_cast<__nv_bfloat16*>(a.qo.p) + t * a.qo.ts + head * a.qo.hs;
    } else if (head < a.s.Hq + a.s.Hkv) {
      const int h = head - a.s.Hq;
      src = static_cast<const __nv_bfloat16*>(a.k.p) + t * a.k.ts + h * a.k.hs;
      if constexpr (APPEND) {
        if (k_at[i] < 0) continue;
        dst = static_cast<__nv_bfloat16*>(a.kp.p) + k_at[i] + h * a.kp.hs;
      } else {
        dst = static_cast<__nv_bfloat16*>(a.ko.p) + t * a.ko.ts + h * a.ko.hs;
      }
    } else {
      const int h = head - a.s.Hq - a.s.Hkv;
      if (v_at[i] < 0) continue;
      src = static_cast<const __nv_bfloat16*>(a.v.p) + t * a.v.ts + h * a.v.hs;
      dst = static_cast<__nv_bfloat16*>(a.vp.p) + v_at[i] + h * a.vp.hs;
      rotated = false;
    }
    // The step's two 16-byte pieces: the halves of eight pairs; or, for
    // neighbouring pairs and copies, one from each half of the head, so that
    // neighbouring threads take neighbouring pieces; or, behind pairs that
    // leave a rest, two of that.
    const bool halves = rotated && !a.s.interleaved && c * 8 < P;
    const bool rest = rotated && !a.s.interleaved && !halves;
    const int e0 = rest ? c * 16 : c * 8;
    const int e1 = halves ? P + c * 8 : (rest ? c * 16 + 8 : a.s.d / 2 + c * 8);
    uint4 u, w;
    load16(src + e0, u);
    load16(src + e1, w);
    uint32_t* pu = reinterpret_cast<uint32_t*>(&u);
    uint32_t* pw = reinterpret_cast<uint32_t*>(&w);
    if (halves) {
      const float2* tr = turns + i * P + c * 8;
#pragma unroll
      for (int e = 0; e < 4; ++e) turn2(pu[e], pw[e], tr[2 * e], tr[2 * e + 1]);
    } else if (rotated && !rest) {
      if (e0 / 2 < P)
#pragma unroll
        for (int e = 0; e < 4; ++e) turn1(pu[e], turns[i * P + e0 / 2 + e]);
      if (e1 / 2 < P)
#pragma unroll
        for (int e = 0; e < 4; ++e) turn1(pw[e], turns[i * P + e1 / 2 + e]);
    }
    store16(dst + e0, u);
    store16(dst + e1, w);
  }
}

// Tokens per block: as many as give each thread one angle, fewer where that
// would leave multiprocessors idle.
int tokens_per_block(int T, int pairs) {
  int n = pairs > 0 ? kThreads / pairs : kMaxTokens;
  if (n > kMaxTokens) n = kMaxTokens;
  if (n > T / 592) n = T / 592;
  return n < 1 ? 1 : n;
}

}  // namespace

cudaError_t launch_rope(const RopeShape& s, const Rows& q, const Rows& k, const Rows& q_out, const Rows& k_out,
                        cudaStream_t stream) {
  RopeArgs a{};
  a.s = s;
  a.q = q;
  a.k = k;
  a.qo = q_out;
  a.ko = k_out;
  a.tokens = tokens_per_block(s.T, s.pairs);
  rope_kernel<false><<<(s.T + a.tokens - 1) / a.tokens, kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_paged_append(const RopeShape& s, const SeqShape& seq, const CacheShape& c, const Rows& q,
                                const Rows& k, const Rows& v, const Rows& q_out, const Pages& k_pages,
                                const Pages& v_pages, unsigned int* err, cudaStream_t stream) {
  RopeArgs a{};
  a.s = s;
  a.q = q;
  a.k = k;
  a.v = v;
  a.qo = q_out;
  a.kp = k_pages;
  a.vp = v_pages;
  a.cu = seq.cu;
  a.lens = c.lens;
  a.table = c.table;
  a.table_stride = c.table_stride;
  a.max_len = static_cast<long long>(c.max_pages) * c.page;
  a.S = seq.S;
  a.n_pages = c.n_pages;
  a.page = c.page;
  a.tokens = tokens_per_block(s.T, s.pairs);
  a.err = err;
  rope_kernel<true><<<(s.T + a.tokens - 1) / a.tokens, kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace fa
