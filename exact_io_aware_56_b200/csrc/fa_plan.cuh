// Work list of the packed-sequence kernels (fa_packed.cu, fa_bwd.cu).
//
// The sequences' offsets live on the device, so that captured graphs can be
// replayed on other lengths; what the host knows are the rows T and the
// number of sequences S. One block lists the work: `unit` tokens of a sequence
// per item, longest items first (a counting sort by key tiles or loop length
// in shared memory, so that the last wave is short). The forward's CTAs are
// resident and take items until none is left; the backward's, launched for the
// largest possible count, leave when their item does not exist.
//
// Few units leave most CTAs idle. The forward then cuts the whole work into one
// run per CTA (units cut by a run's end leave partial results), the backward
// each unit into parts of its steps.
#pragma once

#include "fa_internal.h"
#include "sm100.cuh"

namespace fa {

struct PlanHeader {
  int items;   // items listed
  int splits;  // units cut along the keys (paged chunks)
  int taken;   // forward: items taken by the CTAs beyond their first; of runs: units of more
               // than kMergeManyParts parts
  int runs;    // forward: CTA c takes items [run_first[c], run_first[c + 1]);
               // backward: the items are parts of units
};

// A unit and KV head cut along the keys: parts slot0, slot0 + 1, ... of the partial
// results, to be merged.
struct PlanSplit {
  int base, n, tok0, kvh, slot0, parts;
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
  int run_ctas;    // > 0: the work may be cut into this many runs
  int r;           // backward: query heads of a KV head, gone through one after another
  int part_ctas;   // backward: > 0: units may be cut into parts for this many CTAs
  int sorted;      // 0: every CTA is resident at once, any order does
  PlanHeader* head;
  PlanItem* items;
  int* run_first;
  PlanSplit* split_list;
  unsigned int* err;
};

constexpr int kPlanSeqs = 1024;    // sequences held in shared memory at a time
constexpr int kPlanBuckets = 1024;
// Units of more parts than this are merged by more warps.
constexpr int kMergeManyParts = 8;
// Backward: units times KV heads below which units may be cut into parts, for
// how many waves of CTAs at most, the least steps of a part, and what a CTA's
// start and end take, in steps. That units may be cut costs 1 to 9% even where
// none is (the accumulators of dK and dV are zeroed, the list looks at every
// unit twice), so not from 208 units on, where no cut was found to gain. GPU
// time of the backward, never cut against allowed: 206 units (13100 tokens, 8 + 2
// heads, d = 128, causal) 1229 -> 1090 us, 208 (3300, 32 + 8) 346 -> 351, 208
// (1600, 16 + 16, no mask) 85 -> 93, 304 (2048 tokens in 8, 16 + 16, d = 64) 37 -> 40.
// (fa.h names kPartUnits: dK and dV of fewer units may not repeat bit for bit.)
constexpr int kPartUnits = 208;
constexpr int kPartWaves = 3;
constexpr int kPartLeast = 6;
constexpr int kPartSteps = 5;
// Of more units than CTAs the estimate of whole units' time (mean per CTA plus
// the longest) is too long where they differ, and parts' additions are not in
// it: of 32 measured packs of 150 to 208 units that it would cut, the 18 that it
// had gain 62 steps or more gained up to 35% (one lost 1.4%), the 14 that it had
// gain 43 or less lost up to 27% (two of 1500 tokens, 16 + 8 heads, d = 128,
// causal: 89 -> 113 us).
constexpr int kPartGain = 48;
// Runs are made of fewer units times KV heads than this; more units are
// balanced well enough by taking them longest first (4 per CTA).
constexpr int kRunUnits = 4 * 148;
// Cost of a key tile, and of starting and ending an item, in quarters of a tile
// (measured at d = 128: 1.9 us a tile, 1.8 where only one of the two query tiles
// has tokens; 4 us an item. With one query tile's taken for three quarters and
// an item for 1.5 tiles, the last CTAs of a mix of chunks and single tokens
// ended at 153 us, the mean one at 129: 158.5 -> 147 us for the call).
constexpr int kCostTile = 4, kCostItem = 8;
// No run is shorter than this (about six key tiles), so that few units are not
// cut into more parts than their merge is worth; and no run end cuts off less
// than kRunLeast key tiles of a unit.
constexpr int kCostMerge = 36;  // the parts' stores and the merge kernel, about 14 us
constexpr int kRunCost = kCostItem + 6 * kCostTile;
constexpr int kRunLeast = 3;

// Taken one by one, longest first, the units end about when their mean cost per
// CTA plus most of the longest's has passed; runs end together, no earlier
// than the least run, and their merge follows.
__host__ __device__ inline bool plan_wants_runs(long long mean, long long most) {
  return mean + most * 4 / 5 > (mean > kRunCost ? mean : kRunCost) + kCostMerge;
}

struct PlanShared {
  int pre[kPlanSeqs + 1];  // units of the held sequences, summed
  int start[kPlanSeqs], n[kPlanSeqs], len[kPlanSeqs];
  int hist[kPlanBuckets];
  int warp_sum[32];
  int upos[kRunUnits + 1];  // units' costs, summed
  int most, n_splits, n_slots, n_many;
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
        sh.start[i] = s.start;
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
  // Unit u of the held sequences, as a whole item; returns its work (key
  // tiles of the forward, 64-query steps of the backward).
  auto unit_of = [&](int b0, int u, PlanItem& it) -> int {
    int lo = 0, hi = min(kPlanSeqs, a.S - b0) - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (sh.pre[mid] <= u)
        lo = mid;
      else
        hi = mid - 1;
    }
    const int n = sh.n[lo], tok0 = (u - sh.pre[lo]) * a.unit;
    const int w = a.backward ? (n + 63) / 64 - (a.causal ? tok0 / 64 : 0)
                             : plan_fwd_tiles(n, sh.len[lo], tok0, a.unit, a.causal);
    it = PlanItem{sh.start[lo], n, sh.len[lo] - n, tok0, 0, a.backward ? w * a.r : w, -1, b0 + lo, -1};
    return w;
  };
  // f(u, item, work) for every unit.
  int held_units = 0;
  auto each = [&](auto f) {
    int base = 0;
#pragma unroll 1
    for (int b0 = 0; b0 < a.S; b0 += kPlanSeqs) {
      const int units = one_chunk ? held_units : load(b0);
#pragma unroll 1
      for (int u = threadIdx.x; u < units; u += NT) {
        PlanItem it;
        const int w = unit_of(b0, u, it);
        f(base + u, it, w);
      }
      base += units;
      if (!one_chunk) __syncthreads();
    }
  };
  for (int i = threadIdx.x; i < kPlanBuckets; i += NT) sh.hist[i] = 0;
  if (threadIdx.x == 0) sh.most = sh.n_splits = sh.n_slots = sh.n_many = 0;
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
      *a.head = PlanHeader{0, 0, 0, 0};
    }
    return;
  }
  if (a.run_ctas > 0 && static_cast<long long>(U) * a.heads < kRunUnits) {
    // Cost of each unit, summed; a run is 1 / run_ctas of all units' and heads'.
    int total = 0, most = 0;
#pragma unroll 1
    for (int u0 = 0; u0 < U; u0 += NT) {
      const int u = u0 + threadIdx.x;
      int cost = 0, sum;
      if (u < U) {
        PlanItem it;
        const int w = unit_of(0, u, it);
        cost = kCostItem + w * kCostTile;
      }
      const int x = plan_scan<NT>(cost, sh.warp_sum, sum);
      if (u < U) sh.upos[u + 1] = total + x;
      total += sum;
      most = max(most, cost);
    }
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane == 0) atomicMax(&sh.most, most);
    if (threadIdx.x == 0) sh.upos[0] = 0;
    __syncthreads();
    const int mean = (total * a.heads + a.run_ctas - 1) / a.run_ctas;
    const int len = max(kRunCost, mean);
    if (plan_wants_runs(mean, sh.most)) {
      // First pass: the runs' sizes; second: the items, from their starts on.
#pragma unroll 1
      for (int pass = 0; pass < 2; ++pass) {
#pragma unroll 1
        for (int q = threadIdx.x; q < U * a.heads; q += NT) {
          const int u = q / a.heads;
          PlanItem it;
          const int w = unit_of(0, u, it);
          it.kvh = q - u * a.heads;
          const int cost = sh.upos[u + 1] - sh.upos[u];
          const int at = sh.upos[u] * a.heads + it.kvh * cost;
          // Key tile at which run r ends within this unit.
          auto end_tile = [&](int r) {
            const int x = (r + 1) * len - at;
            if (x >= cost) return w;
            const int j = (x - kCostItem) / kCostTile;
            return j < kRunLeast ? 0 : (j > w - kRunLeast ? w : j);
          };
          int parts = 0, done = 0;
#pragma unroll 1
          for (int r = at / len; done < w; ++r) {
            const int e = end_tile(r);
            if (e > done) ++parts;
            done = max(done, e);
          }
          if (pass == 1 && parts > 1) {
            it.slot = atomicAdd(&sh.n_slots, parts);
            if (parts > kMergeManyParts) atomicAdd(&sh.n_many, 1);
            a.split_list[atomicAdd(&sh.n_splits, 1)] = PlanSplit{it.base, it.n, it.tok0, it.kvh, it.slot, parts};
          }
          done = 0;
#pragma unroll 1
          for (int r = at / len; done < w; ++r) {
            const int e = end_tile(r);
            if (e <= done) continue;
            const int place = atomicAdd(&sh.hist[r], 1);
            it.j0 = done;
            it.j1 = done = e;
            if (pass == 1) a.items[place] = it;
            if (parts > 1) ++it.slot;
          }
        }
        __syncthreads();
        if (pass == 1) break;
        int run = 0;
#pragma unroll 1
        for (int i0 = 0; i0 < a.run_ctas; i0 += NT) {
          const int i = i0 + threadIdx.x;
          const int h = i < a.run_ctas ? sh.hist[i] : 0;
          int sum;
          const int x = run + plan_scan<NT>(h, sh.warp_sum, sum);
          if (i < a.run_ctas) {
            sh.hist[i] = x - h;
            a.run_first[i + 1] = x;
          }
          run += sum;
        }
        if (threadIdx.x == 0) a.run_first[0] = 0;
        __syncthreads();
      }
      if (threadIdx.x == 0) *a.head = PlanHeader{U * a.heads, sh.n_splits, sh.n_many, 1};
      return;
    }
  }
  // Backward with few units: each unit's (head, query tile) steps may be cut
  // into parts of at most len steps, which add up dK and dV in fp32. Parts for
  // one, two or three waves of CTAs against whole units, by what each takes at
  // most: waves times the longest part, or (whole units) the mean per CTA plus
  // the longest.
  int len = 0x7fffffff;
  bool parts_used = false;
  if (a.part_ctas > 0 && static_cast<long long>(U) * a.heads < kPartUnits) {
    int most = 0, steps = 0;
    each([&](int, const PlanItem& it, int) {
      steps += it.j1;
      most = max(most, it.j1);
    });
    most = __reduce_max_sync(0xffffffffu, most);
    steps = __reduce_add_sync(0xffffffffu, steps);
    if (lane == 0) {
      atomicMax(&sh.most, most);
      atomicAdd(&sh.n_slots, steps);
    }
    __syncthreads();
    const int waves = (U * a.heads + a.part_ctas - 1) / a.part_ctas;
    const int mean = (sh.n_slots + kPartSteps * U) * a.heads / a.part_ctas;
    const int whole = min(waves * (sh.most + kPartSteps), mean + sh.most + kPartSteps);
    int best = min(whole * 7 / 8, waves > 1 ? whole - kPartGain : whole);  // a cut has to gain that much
#pragma unroll 1
    for (int k = 1; k <= kPartWaves; ++k) {
      const int room = k * a.part_ctas / a.heads - U;  // parts of a KV head beyond one per unit
      if (room <= 0) continue;
      const int l = max(kPartLeast, (sh.n_slots + room - 1) / room);
      const int cost = k * (l + kPartSteps);
      if (cost < best) {
        best = cost;
        len = l;
        parts_used = true;
      }
    }
  }
  if (!parts_used && (!a.sorted || static_cast<long long>(U) * a.heads <= a.part_ctas)) {
    each([&](int u, const PlanItem& it, int) { a.items[u] = it; });
    if (threadIdx.x == 0) *a.head = PlanHeader{U, 0, 0, 0};
    return;
  }
  // Longest first: bucket 0 holds the longest.
  const long long most = a.backward ? (a.T / 64 + 1LL) * a.r : a.max_len / 128 + 1;
  int shift = 0;
  while ((most >> shift) >= kPlanBuckets) ++shift;
  // First pass: the buckets' sizes; second: the items, from their starts on.
  int run = 0;
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    each([&](int, PlanItem it, int) {
      const int all = it.j1, parts = parts_used ? (all + len - 1) / len : 1;
#pragma unroll 1
      for (int k = 0; k < parts; ++k) {
        const int n = parts == 1 ? all : all / parts + (k < all % parts ? 1 : 0);
        const int at = atomicAdd(&sh.hist[kPlanBuckets - 1 - (n >> shift)], 1);
        it.j1 = it.j0 + n;
        if (pass == 1) a.items[at] = it;
        it.j0 = it.j1;
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
  if (threadIdx.x == 0) *a.head = PlanHeader{run, 0, 0, parts_used ? 1 : 0};
}

__device__ __forceinline__ PlanItem load_item(const PlanItem* p) {
  const int4 a = reinterpret_cast<const int4*>(p)[0], b = reinterpret_cast<const int4*>(p)[1];
  return PlanItem{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w, p->kvh};
}

// Largest number of units: sum of ceil(n_b / unit) over S sequences of T
// tokens together.
inline long long plan_max_units(int S, int T, int unit) {
  const long long most = static_cast<long long>(T) / unit + S;
  return most < T ? most : T;
}

// Bytes of the plan, and its parts' offsets.
struct PlanLayout {
  size_t head, items, run_first, splits, bytes;
};
inline PlanLayout plan_layout(long long max_items, int max_runs, int max_splits) {
  auto up = [](size_t x) { return (x + 31) / 32 * 32; };
  PlanLayout p;
  p.head = 0;
  p.items = up(sizeof(PlanHeader));
  p.run_first = up(p.items + static_cast<size_t>(max_items) * sizeof(PlanItem));
  p.splits = up(p.run_first + (static_cast<size_t>(max_runs) + 1) * 4);
  p.bytes = up(p.splits + static_cast<size_t>(max_splits) * sizeof(PlanSplit));
  return p;
}

}  // namespace fa
