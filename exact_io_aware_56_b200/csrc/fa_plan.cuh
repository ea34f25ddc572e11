// Work list of the packed-sequence kernels (fa_packed.cu, fa_bwd.cu).
//
// The sequences' offsets live on the device, so that captured graphs can be
// replayed on other lengths; what the host knows are the rows T and the
// number of sequences S. A one-block kernel lists the work: `unit` tokens of
// a sequence per item, longest items first (a counting sort by key tiles or
// loop length, so that the last wave is short), and the main kernel's CTAs,
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
  int max_splits;  // room of the split list
  int* upre;       // [S + 1] units, summed
  PlanHeader* head;
  PlanItem* items;
  int* slots;      // per item: its part's slot, -1 when the unit is whole
  PlanSplit* split_list;
  unsigned int* err;
};

constexpr int kPlanThreads = 1024;
constexpr int kPlanBuckets = 2048;
// What starting and ending an item costs, in key tiles (partial results of
// 256 rows written and read again, one CTA's start).
constexpr float kPlanItemCost = 4.f;

// Inclusive sum over the block; `total` receives the last thread's value.
__device__ __forceinline__ int plan_scan(int x, int* warp_sum, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sum[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int y = warp_sum[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int z = __shfl_up_sync(0xffffffffu, y, o);
      if (lane >= o) y += z;
    }
    warp_sum[lane] = y;
  }
  __syncthreads();
  if (warp) x += warp_sum[warp - 1];
  total = warp_sum[31];
  __syncthreads();
  return x;
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

static __global__ void __launch_bounds__(kPlanThreads) plan_kernel(const PlanArgs a) {
  pdl_launch_dependents();
  __shared__ int warp_sum[32];
  __shared__ int hist[kPlanBuckets];
  __shared__ int cand_items[8];
  __shared__ int max_work, split_len, n_splits, n_slots;
  __shared__ unsigned long long sum_work;
  int base = 0;
  bool bad = false;
  if (threadIdx.x == 0) {
    a.upre[0] = 0;
    max_work = 1;
    sum_work = 0;
    n_splits = n_slots = 0;
  }
  for (int i = threadIdx.x; i < kPlanBuckets; i += kPlanThreads) hist[i] = 0;
  if (threadIdx.x < 8) cand_items[threadIdx.x] = 0;
  for (int b0 = 0; b0 < a.S; b0 += kPlanThreads) {
    const int b = b0 + threadIdx.x;
    int units = 0;
    if (b < a.S) {
      const SeqRange s = seq_range(a.cu, a.lens, b, a.T, a.max_q, a.max_len);
      bad |= s.bad;
      units = (s.n + a.unit - 1) / a.unit;
    }
    int total;
    const int x = plan_scan(units, warp_sum, total);
    if (b < a.S) a.upre[b + 1] = base + x;
    base += total;
  }
  // Lengths or offsets out of range: nothing is listed (offsets out of order
  // could name more units than there is room for).
  bad = __syncthreads_or(bad);
  if (bad && threadIdx.x == 0) atomicOr(a.err, kErrData);
  const int U = bad ? 0 : base;
  // Unit u: its sequence, first token and work (key tiles of the forward,
  // 64-query steps of the backward).
  auto unit_of = [&](int u, PlanItem& it) -> int {
    int lo = 0, hi = a.S - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (a.upre[mid] <= u)
        lo = mid;
      else
        hi = mid - 1;
    }
    const SeqRange s = seq_range(a.cu, a.lens, lo, a.T, a.max_q, a.max_len);
    const int i = u - a.upre[lo];
    it.seq = lo;
    it.tok0 = i * a.unit;
    it.j0 = 0;
    if (a.backward) {
      const int steps = (s.n + 63) / 64;
      it.j1 = a.causal ? steps - it.tok0 / 64 : steps;
    } else {
      it.j1 = plan_fwd_tiles(s.n, s.len, it.tok0, a.unit, a.causal);
    }
    return it.j1;
  };
  int my_max = 1;
  unsigned long long my_sum = 0;
  for (int u = threadIdx.x; u < U; u += kPlanThreads) {
    PlanItem it;
    const int w = unit_of(u, it);
    my_max = max(my_max, w);
    my_sum += w;
  }
  atomicMax(&max_work, my_max);
  if (my_sum) atomicAdd(&sum_work, my_sum);
  __syncthreads();
  // Where the units are too few to fill the GPU evenly, cut them along the
  // keys: the longest length L among eight candidates that gives the least
  // estimate of the time, (all tiles and starts) / CTAs + half the longest
  // item, and no less than that item.
  if (threadIdx.x == 0) split_len = max_work;
  __syncthreads();
  if (a.split_ctas > 0 && static_cast<long long>(U) * a.heads < 2LL * a.split_ctas) {
    const unsigned long long all = sum_work * a.heads;
    int len[8];
    len[0] = max_work;
#pragma unroll
    for (int c = 1; c < 8; ++c) {
      // about split_ctas * (c + 1) / 4 items
      const unsigned long long l = (all * 4 + a.split_ctas * (c + 1) - 1) / (static_cast<unsigned long long>(a.split_ctas) * (c + 1));
      len[c] = static_cast<int>(l < 4 ? 4 : (l > static_cast<unsigned long long>(max_work) ? max_work : l));
    }
    int cnt[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    for (int u = threadIdx.x; u < U; u += kPlanThreads) {
      PlanItem it;
      const int w = unit_of(u, it);
#pragma unroll
      for (int c = 0; c < 8; ++c) cnt[c] += (w + len[c] - 1) / len[c];
    }
#pragma unroll
    for (int c = 0; c < 8; ++c)
      if (cnt[c]) atomicAdd(&cand_items[c], cnt[c]);
    __syncthreads();
    if (threadIdx.x == 0) {
      float best = 0.f;
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const float longest = static_cast<float>(len[c]) + kPlanItemCost;
        const float work = (static_cast<float>(all) + kPlanItemCost * cand_items[c] * a.heads) / a.split_ctas;
        const float cost = fmaxf(work + 0.5f * longest, longest);
        if (c == 0 || cost < best) {
          best = cost;
          split_len = len[c];
        }
      }
    }
    __syncthreads();
  }
  const int L = split_len;
  int shift = 0;
  while ((L >> shift) >= kPlanBuckets) ++shift;
  // Longest first: bucket 0 holds the longest.
  auto bucket = [&](int w) { return kPlanBuckets - 1 - (w >> shift); };
  auto parts_of = [&](int w) { return (w + L - 1) / L; };
  for (int u = threadIdx.x; u < U; u += kPlanThreads) {
    PlanItem it;
    const int w = unit_of(u, it);
    const int p = parts_of(w);
    // p parts of nearly equal length: w % p of them one longer.
    atomicAdd(&hist[bucket(w / p)], p - w % p);
    if (w % p) atomicAdd(&hist[bucket(w / p + 1)], w % p);
  }
  __syncthreads();
  int run = 0;
  for (int i0 = 0; i0 < kPlanBuckets; i0 += kPlanThreads) {
    const int i = i0 + threadIdx.x;
    const int h = hist[i];
    int total;
    const int x = plan_scan(h, warp_sum, total);
    hist[i] = run + x - h;
    run += total;
  }
  __syncthreads();
  for (int u = threadIdx.x; u < U; u += kPlanThreads) {
    PlanItem it;
    const int w = unit_of(u, it);
    const int p = parts_of(w);
    int slot = -1;
    if (p > 1) {
      slot = atomicAdd(&n_slots, p);
      a.split_list[atomicAdd(&n_splits, 1)] = PlanSplit{it.seq, it.tok0, slot, p};
    }
    int j = 0;
    for (int k = 0; k < p; ++k) {
      const int n = w / p + (k < w % p ? 1 : 0);
      const int at = atomicAdd(&hist[bucket(n)], 1);
      a.items[at] = PlanItem{it.seq, it.tok0, j, j + n};
      a.slots[at] = p > 1 ? slot + k : -1;
      j += n;
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) *a.head = PlanHeader{run, n_splits, {0, 0}};
}

// Largest number of units: sum of ceil(n_b / unit) over S sequences of T
// tokens together.
inline long long plan_max_units(int S, int T, int unit) {
  const long long most = static_cast<long long>(T) / unit + S;
  return most < T ? most : T;
}

// Bytes of the plan, and its parts' offsets, for at most max_items items.
struct PlanLayout {
  size_t head, upre, items, slots, splits, bytes;
};
inline PlanLayout plan_layout(int S, long long max_items, int max_splits) {
  auto up = [](size_t x) { return (x + 15) / 16 * 16; };
  PlanLayout p;
  p.head = 0;
  p.upre = up(sizeof(PlanHeader));
  p.items = up(p.upre + (static_cast<size_t>(S) + 1) * 4);
  p.slots = up(p.items + static_cast<size_t>(max_items) * sizeof(PlanItem));
  p.splits = up(p.slots + static_cast<size_t>(max_items) * 4);
  p.bytes = up(p.splits + static_cast<size_t>(max_splits) * sizeof(PlanSplit));
  return p;
}

}  // namespace fa
