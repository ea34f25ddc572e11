// Work list of the packed-sequence kernels (fa_packed.cu, fa_bwd.cu).
//
// The sequences' offsets live on the device, so that captured graphs can be
// replayed on other lengths; what the host knows are the rows T and the
// number of sequences S. A one-block kernel lists the work: `unit` tokens of
// a sequence per item, longest items first (a counting sort by key tiles or
// loop length in shared memory, so that the last wave is short), and the main kernel's CTAs,
// launched for the largest possible count, leave when their item does not
// exist.
#pragma once

#include "fa_internal.h"
#include "sm100.cuh"

namespace fa {

struct PlanHeader {
  int items;   // items listed
  int splits;  // units cut along the keys (paged chunks)
  int pad[2];
};

// A unit cut along the keys: parts slot0, slot0 + 1, ... of the partial
// results, to be merged.
struct PlanSplit {
  int seq, tok0, slot0, parts;
};

struct PlanArgs {
  const int* cu;
  const int* lens;  // paged cache: lengths; nullptr: the sequences themselves
  int S, T, max_q;
  long long max_len;
  int unit;        // tokens per item
  int causal;
  int backward;    // items are key tiles of the backward, else query tokens of the forward
  int heads;       // CTAs per item (KV heads)
  int split_ctas;  // > 0: items may be cut so that this many CTAs are busy
  int sorted;      // 0: every CTA is resident at once, any order does
  PlanHeader* head;
  PlanItem* items;
  int* slots;      // per item: its part's slot, -1 when the unit is whole (nullptr: not wanted)
  PlanSplit* split_list;
  unsigned int* err;
};

constexpr int kPlanSeqs = 1024;    // sequences held in shared memory at a time
constexpr int kPlanBuckets = 1024;
// What starting and ending an item costs, in key tiles (partial results of
// 256 rows written and read again, one CTA's start).
constexpr float kPlanItemCost = 4.f;

struct PlanShared {
  int pre[kPlanSeqs + 1];  // units of the held sequences, summed
  int n[kPlanSeqs], len[kPlanSeqs];
  int hist[kPlanBuckets];
  int warp_sum[32];
  int cand[8];
  int most, n_splits, n_slots;
  unsigned int sum;
};

// Inclusive sum of `x` over the block of NT threads.
template <int NT>
__device__ __forceinline__ int plan_scan(int x, int* warp_sum, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sum[warp] = x;
  __syncthreads();
  int before = 0;
  total = 0;
#pragma unroll 4
  for (int i = 0; i < NT / 32; ++i) {
    const int y = warp_sum[i];
    if (i < warp) before += y;
    total += y;
  }
  __syncthreads();
  return x + before;
}

// Key tiles (128 keys) that the queries [tok0, tok0 + unit) of a sequence
// look at; at least one, which also writes the rows that see no key.
__host__ __device__ inline int plan_fwd_tiles(int n, int len, int tok0, int unit, int causal) {
  long long last = len - 1;  // last visible key
  if (causal) {
    const long long end = tok0 + unit < n ? tok0 + unit : n;
    last = static_cast<long long>(len) - n + end - 1;
  }
  return last < 0 ? 1 : static_cast<int>(last / 128) + 1;
}

// Writes the list; one block of NT threads. (Run once per call on cold
// instruction caches, it costs by the length of its code: loops are kept
// rolled, and the passes share theirs.)
template <int NT>
__device__ void plan_block(const PlanArgs& a, PlanShared& sh) {
  const int lane = threadIdx.x & 31;
  const bool one_chunk = a.S <= kPlanSeqs;
  bool bad = false;
  // Holds sequences [b0, b0 + kPlanSeqs); returns their units.
  auto load = [&](int b0) -> int {
    int base = 0;
#pragma unroll 1
    for (int i0 = 0; i0 < kPlanSeqs && b0 + i0 < a.S; i0 += NT) {
      const int i = i0 + threadIdx.x;
      int units = 0;
      if (b0 + i < a.S) {
        const SeqRange s = seq_range(a.cu, a.lens, b0 + i, a.T, a.max_q, a.max_len);
        bad |= s.bad;
        units = (s.n + a.unit - 1) / a.unit;
        sh.n[i] = s.n;
        sh.len[i] = s.len;
      }
      int total;
      const int x = plan_scan<NT>(units, sh.warp_sum, total);
      sh.pre[i + 1] = base + x;
      base += total;
    }
    if (threadIdx.x == 0) sh.pre[0] = 0;
    __syncthreads();
    return base;
  };
  // Unit u of the held sequences: its work (key tiles of the forward, 64-query
  // steps of the backward).
  auto unit_of = [&](int b0, int u, int& seq, int& tok0) -> int {
    int lo = 0, hi = min(kPlanSeqs, a.S - b0) - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (sh.pre[mid] <= u)
        lo = mid;
      else
        hi = mid - 1;
    }
    seq = b0 + lo;
    tok0 = (u - sh.pre[lo]) * a.unit;
    if (a.backward) return (sh.n[lo] + 63) / 64 - (a.causal ? tok0 / 64 : 0);
    return plan_fwd_tiles(sh.n[lo], sh.len[lo], tok0, a.unit, a.causal);
  };
  // f(u, seq, tok0, work) for every unit.
  int held_units = 0;
  auto each = [&](auto f) {
    int base = 0;
#pragma unroll 1
    for (int b0 = 0; b0 < a.S; b0 += kPlanSeqs) {
      const int units = one_chunk ? held_units : load(b0);
#pragma unroll 1
      for (int u = threadIdx.x; u < units; u += NT) {
        int seq, tok0;
        const int w = unit_of(b0, u, seq, tok0);
        f(base + u, seq, tok0, w);
      }
      base += units;
      if (!one_chunk) __syncthreads();
    }
  };
  for (int i = threadIdx.x; i < kPlanBuckets; i += NT) sh.hist[i] = 0;
  if (threadIdx.x < 8) sh.cand[threadIdx.x] = 0;
  if (threadIdx.x == 0) sh.most = sh.n_splits = sh.n_slots = sh.sum = 0;
  int U = 0;
  if (one_chunk) {
    U = held_units = load(0);
  } else {
#pragma unroll 1
    for (int b0 = 0; b0 < a.S; b0 += kPlanSeqs) {
      U += load(b0);
      __syncthreads();
    }
  }
  // Lengths or offsets out of range: nothing is listed (offsets out of order
  // could name more units than there is room for).
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0) {
      atomicOr(a.err, kErrData);
      *a.head = PlanHeader{0, 0, {0, 0}};
    }
    return;
  }
  if (!a.sorted && a.split_ctas == 0) {
    each([&](int u, int seq, int tok0, int w) {
      a.items[u] = PlanItem{seq, tok0, 0, w};
      if (a.slots) a.slots[u] = -1;
    });
    if (threadIdx.x == 0) *a.head = PlanHeader{U, 0, {0, 0}};
    return;
  }
  // Largest work there can be: sets the width of a bucket.
  long long most = a.backward ? a.T / 64 + 1 : a.max_len / 128 + 1;
  int L = 0x7fffffff;
  // Where the units are too few to fill the GPU evenly, cut them along the
  // keys: the longest length L among eight candidates that gives the least
  // estimate of the time, (all tiles and starts) / CTAs + half the longest
  // item, and no less than that item.
  if (a.split_ctas > 0 && static_cast<long long>(U) * a.heads < 2LL * a.split_ctas) {
    int my_max = 1;
    unsigned int my_sum = 0;  // below 2 * 148 units of at most 2^23 tiles: below 2^32
    each([&](int, int, int, int w) {
      my_max = max(my_max, w);
      my_sum += w;
    });
    my_max = __reduce_max_sync(0xffffffffu, my_max);
    my_sum = __reduce_add_sync(0xffffffffu, my_sum);
    if (lane == 0) {
      atomicMax(&sh.most, my_max);
      atomicAdd(&sh.sum, my_sum);
    }
    __syncthreads();
    most = sh.most;
    const long long all = static_cast<long long>(sh.sum) * a.heads;
    int len[8], cnt[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      // c = 0: whole units; else about split_ctas * (c + 1) / 4 items.
      const float l = ceilf(static_cast<float>(all) * 4.f / static_cast<float>(a.split_ctas * (c + 1)));
      len[c] = c == 0 ? sh.most : static_cast<int>(fminf(fmaxf(l, 4.f), static_cast<float>(sh.most)));
      cnt[c] = 0;
    }
    each([&](int, int, int, int w) {
#pragma unroll
      for (int c = 0; c < 8; ++c) cnt[c] += (w + len[c] - 1) / len[c];
    });
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const int x = __reduce_add_sync(0xffffffffu, cnt[c]);
      if (lane == 0 && x) atomicAdd(&sh.cand[c], x);
    }
    __syncthreads();
    float best = 0.f;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const float longest = static_cast<float>(len[c]) + kPlanItemCost;
      const float work = (static_cast<float>(all) + kPlanItemCost * sh.cand[c] * a.heads) / a.split_ctas;
      const float cost = fmaxf(work + 0.5f * longest, longest);
      if (c == 0 || cost < best) {
        best = cost;
        L = len[c];
      }
    }
  }
  int shift = 0;
  while ((most >> shift) >= kPlanBuckets) ++shift;
  // Longest first: bucket 0 holds the longest.
  auto bucket = [&](int w) { return kPlanBuckets - 1 - (w >> shift); };
  auto parts_of = [&](int w) { return w <= L ? 1 : (w + L - 1) / L; };
  // First pass: the buckets' sizes; second: the items, from their starts on.
  int run = 0;
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    each([&](int, int seq, int tok0, int w) {
      const int p = parts_of(w);
      int slot = -1;
      if (pass == 1 && p > 1) {
        slot = atomicAdd(&sh.n_slots, p);
        a.split_list[atomicAdd(&sh.n_splits, 1)] = PlanSplit{seq, tok0, slot, p};
      }
      // p parts of nearly equal length: w % p of them one longer.
      int j = 0;
#pragma unroll 1
      for (int k = 0; k < p; ++k) {
        const int n = p == 1 ? w : w / p + (k < w % p ? 1 : 0);
        const int at = atomicAdd(&sh.hist[bucket(n)], 1);
        if (pass == 1) {
          a.items[at] = PlanItem{seq, tok0, j, j + n};
          if (a.slots) a.slots[at] = p > 1 ? slot + k : -1;
        }
        j += n;
      }
    });
    __syncthreads();
    if (pass == 1) break;
#pragma unroll 1
    for (int i0 = 0; i0 < kPlanBuckets; i0 += NT) {
      const int i = i0 + threadIdx.x;
      const int h = sh.hist[i];
      int total;
      const int x = plan_scan<NT>(h, sh.warp_sum, total);
      sh.hist[i] = run + x - h;
      run += total;
    }
    __syncthreads();
  }
  if (threadIdx.x == 0) *a.head = PlanHeader{run, sh.n_splits, {0, 0}};
}

// Largest number of units: sum of ceil(n_b / unit) over S sequences of T
// tokens together.
inline long long plan_max_units(int S, int T, int unit) {
  const long long most = static_cast<long long>(T) / unit + S;
  return most < T ? most : T;
}

// Bytes of the plan, and its parts' offsets, for at most max_items items.
struct PlanLayout {
  size_t head, items, slots, splits, bytes;
};
inline PlanLayout plan_layout(long long max_items, int max_splits) {
  auto up = [](size_t x) { return (x + 15) / 16 * 16; };
  PlanLayout p;
  p.head = 0;
  p.items = up(sizeof(PlanHeader));
  p.slots = up(p.items + static_cast<size_t>(max_items) * sizeof(PlanItem));
  p.splits = up(p.slots + static_cast<size_t>(max_items) * 4);
  p.bytes = up(p.splits + static_cast<size_t>(max_splits) * sizeof(PlanSplit));
  return p;
}

}  // namespace fa
