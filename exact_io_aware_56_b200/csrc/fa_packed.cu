// Forward attention over packed sequences, and over a paged cache for chunks
// of new tokens (sm_100a).
//
// Packed: sequence b is rows [cu[b], cu[b+1]) of q, k and v; every query sees
// the keys of its own sequence (all, or those not behind it). Paged: sequence
// b's n_b new tokens are the last of len_b cached ones, query i sees keys
// j <= len_b - n_b + i (causal) or j < len_b.
//   O_i = softmax(scale q_i K^T) V,  L_i = log sum_j e^(S_ij);  a row that
//   sees no key: O_i = 0, L_i = -inf.
//
// Bound: tensor cores and the exponential unit for long prompts, as in
// fa_fwd.cu, whose two forms this kernel follows: T = 2 query tiles per CTA
// at d = 128 (one CTA per SM), T = 1 at d = 64 (two CTAs per SM, separate P).
// What differs:
//  * A query tile is TT = 128 / r tokens times the r query heads of one KV
//    head (rows in token-major order), so that grouped heads share each K/V
//    tile in shared memory, short sequences fill their tiles r times better
//    than one head per tile would, and the causal edge is cut at TT tokens.
//  * The work comes from a list (fa_plan.cuh), longest first. CTAs stay
//    resident and take items until none is left; the next item's first K/V
//    tiles and Q load, and its first S products run, beside this one's last
//    softmax and epilogue. (One CTA per item spent 5.9 us of 44 per item on
//    starting, first loads and ending, at 16k packed tokens, d = 128.) Too
//    few units to fill the GPU evenly (chunks over a long cache, few heads) are
//    instead cut into one run per CTA of equal cost; units that a run's end cuts along
//    their keys leave O / l and logsumexp in the workspace and a second kernel
//    merges them.
//  * Tiles end where sequences do: scores of keys behind the end are replaced
//    by -inf; the V rows there, which may hold anything (the next sequence,
//    stale cache slots, NaN), are zeroed in shared memory before P V (warp
//    kFixWarp). O leaves by TMA in whole tiles (at d = 128 that takes 0.8 us
//    off an item against storing rows) or, where a tile holds rows that are
//    not this sequence's, row by row.
//
// Warp roles (w0 = 4T): 0..w0-1 softmax, w0 takes items and loads Q and K,
// w0+1 MMA and tensor memory, w0+2 loads V, w0+3 zeroes V rows behind the end.
// All rings and barrier phases run on across items. O_t needs no barrier of
// its own between items: P V of the next item follows p_ready, which the
// softmax warps of tile t give after their epilogue.

#include <cuda_bf16.h>
#include <math_constants.h>

#include "fa_internal.h"
#include "fa_merge.cuh"
#include "fa_plan.cuh"
#include "sm100.cuh"

namespace fa {
namespace {

constexpr int kBM = 128;  // rows per query tile
constexpr int kBN = 128;  // keys per tile
// Rescale thresholds of the running max, log2 units (as fa_fwd.cu: exact
// where the residual is written, so that the backward's D is; else lazy).
constexpr float kRescaleExact = 0.0f;
constexpr float kRescaleLazy = 8.0f;

template <int D>
struct PkCfg {
  static constexpr int T = D == 128 ? 2 : 1;
  static constexpr bool SEP = D == 64;  // P in its own tensor-memory columns
  static constexpr int kThreads = T == 1 ? 256 : 384;
  static constexpr int kMinBlocks = T == 1 ? 2 : 1;
  // Register shares (setmaxnreg) of a softmax warpgroup and of the other
  // warps' group: together what the launch gives the CTA (128 per thread in
  // two warpgroups, 168 in three).
  static constexpr int kLaunchRegs = T == 1 ? 128 : 168;
  static constexpr int kSoftmaxRegs = T == 1 ? 192 : 208;
  static constexpr int kOtherRegs = T == 1 ? 64 : 88;
  static_assert(T * kSoftmaxRegs + kOtherRegs == (T + 1) * kLaunchRegs, "register split");
  static constexpr int kProducerWarp = 4 * T;
  static constexpr int kMmaWarp = 4 * T + 1;
  static constexpr int kVProducerWarp = 4 * T + 2;
  static constexpr int kFixWarp = 4 * T + 3;
  static constexpr int kKStages = 2;
  static constexpr int kVStages = 2;
  static constexpr int kBoxBytes = kBN * 128;
  static constexpr int kBoxes = D / 64;
  static constexpr int kTileBytes = kBoxBytes * kBoxes;
  static constexpr int kOffQ = 0;
  static constexpr int kOffK = T * kTileBytes;
  static constexpr int kOffV = kOffK + kKStages * kTileBytes;
  // d = 128: whole output tiles leave by TMA through one 16-KB box (64
  // columns) per tile; at d = 64 each thread stores its own row.
  static constexpr bool kStaged = T == 2;
  static constexpr int kOffStage = kOffV + kVStages * kTileBytes;
  static constexpr int kOffBar = kOffStage + (kStaged ? T * 16384 : 0);
  static constexpr int kBarBytes = 512;
  static constexpr int kSmemBytes = kOffBar + kBarBytes + 1024;  // + alignment slack
  static constexpr uint32_t kTmemCols = T == 1 ? 256 : 512;
  static constexpr uint32_t kColO = T == 1 ? 128 : 256;
  static constexpr uint32_t kColP = 192;  // SEP
  static_assert(kSmemBytes <= 227 * 1024, "shared memory budget");
  static_assert(T == 1 ? (kSmemBytes <= 228 * 1024 / 2 - 1024 && 3 * kSmemBytes > 228 * 1024)
                       : kSmemBytes > 114 * 1024,
                "CTAs per SM");
};

struct PkArgs {
  PlanHeader* head;
  const PlanItem* items;
  const int* run_first;
  const PlanSplit* split_list;
  const int* table;  // paged
  long long table_stride;
  int n_pages, page, pb;
  Rows o, resid;
  float* lse;
  float* part_o;  // [slot][T * 128][D]
  float* part_l;
  int total, Hkv, r, TT, causal;
  // Packed, few units: no list; every CTA finds its units in cu itself.
  int direct, S, unit;
  const int* cu;
  int sectors;  // o (and its residual) can be stored 32 bytes at a time
  float scale_log2, rescale_tau;
  uint64_t item_ns;  // ample for the longest item that there can be
  LaunchCtl ctl;
};

struct PkBars {
  uint64_t q_full[2], q_empty[2];
  uint64_t k_full[2], k_empty[2];
  uint64_t v_full[2], v_land[2], v_empty[2];
  uint64_t s_full[2], p_ready[2][2], o_final[2];
  uint64_t s_free, pv_done;
  uint64_t epi_full[2], epi_free[2];  // output staging
  uint64_t item_full[2], item_empty[2];
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
  alignas(16) int4 item[2][2];  // taken items, and their KV heads
  int kvh[2];
};
static_assert(sizeof(PkBars) <= 512, "barrier block exceeds its shared-memory reservation");

constexpr int kPlanThreads = 512;
__global__ void __launch_bounds__(kPlanThreads) packed_plan_kernel(const PlanArgs a) {
  __shared__ PlanShared sh;
  pdl_launch_dependents();
  plan_block<kPlanThreads>(a, sh);
}

// Units of all sequences, by the whole warp; 0, and reported, where an offset
// is out of range.
__device__ __forceinline__ int direct_units(const PkArgs& a, int lane) {
  int n = 0;
  bool bad = false;
  for (int b = lane; b < a.S; b += 32) {
    const SeqRange s = seq_range(a.cu, nullptr, b, a.total, a.total, a.total);
    bad |= s.bad;
    n += (s.n + a.unit - 1) / a.unit;
  }
  if (__any_sync(0xffffffffu, bad)) {
    if (lane == 0 && blockIdx.x == 0) atomicOr(a.ctl.err, kErrData);
    return 0;
  }
  return __reduce_add_sync(0xffffffffu, n);
}

// Units of a sequence of n tokens that take fewer than w key tiles.
__device__ __forceinline__ int direct_less(const PkArgs& a, int n, int w) {
  if (n <= (w - 1) * kBN) return (n + a.unit - 1) / a.unit;
  return a.causal ? (w - 1) * kBN / a.unit : 0;
}

// The unit of this rank, by the whole warp. Where some CTAs take two units, of
// up to 32 sequences, one per lane: rank 0 takes the most key tiles; w, the
// rank's, by bisection of the number of units that take w or more. (17 short
// prompts of 16 heads, where a CTA's second unit could be one of the longest:
// 14.8 -> 13.5 us; the search itself costs 0.5 to 1 us.) Else, or of more
// sequences, which are shorter then: the last unit first, 32 sequences a step.
__device__ __forceinline__ PlanItem direct_item(const PkArgs& a, int units, int rank, int lane) {
  PlanItem it{};
  if (a.S <= 32 && units * a.Hkv > static_cast<int>(gridDim.x)) {
    SeqRange s{};
    if (lane < a.S) s = seq_range(a.cu, nullptr, lane, a.total, a.total, a.total);
    const int mine = (s.n + a.unit - 1) / a.unit;
    int w = 1, hi = (__reduce_max_sync(0xffffffffu, s.n) + kBN - 1) / kBN;
    int longer = 0;  // units of more than w key tiles
    while (w < hi) {
      const int mid = (w + hi + 1) / 2;
      const int n = __reduce_add_sync(0xffffffffu, mine - direct_less(a, s.n, mid));
      if (n > rank) {
        w = mid;
      } else {
        hi = mid - 1;
        longer = n;
      }
    }
    const int first = direct_less(a, s.n, w);
    const int same = direct_less(a, s.n, w + 1) - first;
    int end = same;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, end, o);
      if (lane >= o) end += y;
    }
    const int l = __ffs(__ballot_sync(0xffffffffu, end > rank - longer)) - 1;
    const int tok0 = (__shfl_sync(0xffffffffu, first + same - end, l) + rank - longer) * a.unit;
    return PlanItem{__shfl_sync(0xffffffffu, s.start, l), __shfl_sync(0xffffffffu, s.n, l), 0, tok0, 0, w, -1, l, -1};
  }
  const int u = units - 1 - rank;
  int before = 0;
  for (int b0 = 0; b0 < a.S; b0 += 32) {
    SeqRange s{};
    if (b0 + lane < a.S) s = seq_range(a.cu, nullptr, b0 + lane, a.total, a.total, a.total);
    const int mine = (s.n + a.unit - 1) / a.unit;
    int end = before + mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, end - before, o);
      if (lane >= o) end += y;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, end > u);
    if (hit) {
      const int l = __ffs(hit) - 1;
      const int n = __shfl_sync(0xffffffffu, s.n, l);
      const int tok0 = (u - __shfl_sync(0xffffffffu, end - mine, l)) * a.unit;
      it = PlanItem{__shfl_sync(0xffffffffu, s.start, l), n, 0, tok0, 0,
                    plan_fwd_tiles(n, n, tok0, a.unit, a.causal), -1, b0 + l, -1};
      break;
    }
    before = __shfl_sync(0xffffffffu, end, 31);
  }
  return it;
}

// An item as a CTA works on it: tile t holds tokens [tok_t[t], ...) and takes
// the first n_t[t] of the item's n key tiles.
struct Unit {
  PlanItem it;
  int kvh, n, n_t[2], tok_t[2];
  __device__ __forceinline__ int len() const { return it.off + it.n; }
  // Keys of the sequence in the item's u-th key tile (<= 0: none).
  __device__ __forceinline__ int keys(int u) const { return min(kBN, len() - (it.j0 + u) * kBN); }
};

template <int T>
__device__ __forceinline__ Unit make_unit(const PlanItem& it, int kvh, int TT, int causal) {
  Unit x;
  x.it = it;
  x.kvh = kvh;
  x.n_t[1] = 0;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    x.tok_t[t] = it.tok0 + t * TT;
    x.n_t[t] = 0;
    if (t < T && x.tok_t[t] < it.n)
      x.n_t[t] = max(0, min(it.j1, plan_fwd_tiles(it.n, x.len(), x.tok_t[t], TT, causal)) - it.j0);
  }
  x.n = max(x.n_t[0], x.n_t[1]);
  return x;
}

// RUNS: the work may be cut into runs, and units into parts. (Without, the
// kernel has no path for partial results: 1% at 16k packed tokens.)
template <int D, bool PAGED, bool RUNS>
__global__ void __launch_bounds__(PkCfg<D>::kThreads, PkCfg<D>::kMinBlocks)
    packed_fwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmO,
                      const __grid_constant__ CUtensorMap tmR, const PkArgs a) {
  using C = PkCfg<D>;
  constexpr int T = C::T;
  constexpr bool SEP = C::SEP;
  constexpr int KS = C::kKStages;
  constexpr int VS = C::kVStages;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + ((1024u - (raw_addr & 1023u)) & 1023u);
  PkBars* bars = reinterpret_cast<PkBars*>(smem + C::kOffBar);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bars->q_full[s], 1);
      mbar_init(&bars->q_empty[s], 1);
      mbar_init(&bars->v_full[s], 1);
      mbar_init(&bars->v_land[s], 1);
      mbar_init(&bars->v_empty[s], 1);
      mbar_init(&bars->s_full[s], 1);
      mbar_init(&bars->p_ready[s][0], kBM);
      mbar_init(&bars->p_ready[s][1], kBM);
      mbar_init(&bars->o_final[s], 1);
      mbar_init(&bars->epi_full[s], kBM);
      mbar_init(&bars->epi_free[s], 1);
      mbar_init(&bars->item_full[s], 1);
      mbar_init(&bars->item_empty[s], 4 * T + 3);  // softmax warps, MMA, V, fixer
    }
    for (int s = 0; s < KS; ++s) {
      mbar_init(&bars->k_full[s], 1);
      mbar_init(&bars->k_empty[s], 1);
    }
    mbar_init(&bars->s_free, kBM);
    mbar_init(&bars->pv_done, 1);
    mbar_init(&bars->drain, 1);
    bars->abort = 0;
    fence_mbar_init();
  }
  if (warp == C::kMmaWarp) {
    tmem_alloc(&bars->tmem_base, C::kTmemCols);
    tmem_relinquish();
  }
  // Without a list: the units, their loads beside the setup above.
  const bool direct = !PAGED && a.direct;
  int units = 0;
  if (direct && warp == C::kProducerWarp) units = direct_units(a, lane);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // Everything above ran beside the plan.
  pdl_launch_dependents();
  pdl_wait();
  const uint32_t tmem = bars->tmem_base;
  const Watch w{&bars->abort, a.ctl.err, a.ctl.budget_ns};
  // Waits that last as long as an item, whose key tiles take microseconds each.
  const Watch w_item{&bars->abort, a.ctl.err, a.ctl.budget_ns + a.item_ns};
  auto all = [](bool b) { return __all_sync(0xffffffffu, b); };

  // The i-th item of this CTA, from the producer; false: none is left, or a
  // wait gave up. Whole warp.
  auto next_unit = [&](int i, Unit& x) -> bool {
    const int s = i & 1;
    if (!all(wait_bar(&bars->item_full[s], (i >> 1) & 1, w_item))) return false;
    const int4 p = bars->item[s][0], q = bars->item[s][1];
    const int kvh = bars->kvh[s];
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars->item_empty[s]);
    x = make_unit<T>(PlanItem{p.x, p.y, p.z, p.w, q.x, q.y, q.z, q.w, kvh}, kvh, a.TT, a.causal);
    return p.y > 0;
  };
  // Page and slot of this lane's part of the u-th key tile (paged).
  auto page_of = [&](const Unit& x, int u, int& slot) -> int {
    slot = 0;
    int page_no = 0;
    if (lane * a.pb < x.keys(u)) {
      const int key = (x.it.j0 + u) * kBN + lane * a.pb;
      const int pi = key / a.page;
      slot = key - pi * a.page;
      page_no = a.table[static_cast<long long>(x.it.seq) * a.table_stride + pi];
      if (page_no < 0 || page_no >= a.n_pages) {
        page_no = a.n_pages;  // past the tensor: the copy fills zeros
        atomicOr(a.ctl.err, kErrData);
      }
    }
    return page_no;
  };
  // Copies the u-th key tile (K or V) to a stage; whole warp. Packed: one box
  // per 64 columns. Paged: lane i copies part i.
  auto load_tile = [&](const CUtensorMap* tm, uint64_t* bar, uint8_t* dst, const Unit& x, int u, int page_no, int slot) {
    if constexpr (PAGED) {
      const int parts = (max(0, x.keys(u)) + a.pb - 1) / a.pb;
      if (lane == 0) mbar_arrive_expect_tx(bar, static_cast<uint32_t>(parts) * a.pb * 128u * C::kBoxes);
      __syncwarp();
      if (lane < parts)
#pragma unroll
        for (int b = 0; b < C::kBoxes; ++b)
          tma_load_4d(tm, bar, dst + lane * a.pb * 128 + b * C::kBoxBytes, b * 64, slot, x.kvh, page_no);
    } else if (lane == 0) {
      mbar_arrive_expect_tx(bar, C::kTileBytes);
#pragma unroll
      for (int b = 0; b < C::kBoxes; ++b)
        tma_load_3d(tm, bar, dst + b * C::kBoxBytes, b * 64, x.it.base + (x.it.j0 + u) * kBN, x.kvh);
    }
  };

  if (warp >= 4 * T) {
    regs_dec<C::kOtherRegs>();
    if (warp == C::kProducerWarp) {
      // ------------------------------------------------ items, Q and K
      if (lane == 0) {
        tma_prefetch_desc(&tmQ);
        tma_prefetch_desc(&tmK);
      }
      // Items of the list times the KV heads, taken one by one; or, where the
      // plan cut the work into runs, this CTA's own items.
      const bool runs = RUNS && a.head->runs != 0;
      if (!direct) units = a.head->items;
      int idx = runs ? a.run_first[blockIdx.x] : blockIdx.x;
      const int total = runs ? a.run_first[blockIdx.x + 1] : units * a.Hkv;
      int kg = 0, q_uses[2] = {0, 0};
      bool ok = true;
      for (int i = 0; ok; ++i) {
        const int sl = i & 1;
        const bool more = idx < total;
        PlanItem it{};
        if (more) {
          if (direct)
            it = direct_item(a, units, idx / a.Hkv, lane);
          else
            it = load_item(a.items + (runs ? idx : idx / a.Hkv));
        }
        const int kvh = runs ? it.kvh : idx % a.Hkv;
        if (i >= 2 && !all(wait_bar(&bars->item_empty[sl], ((i >> 1) - 1) & 1, w_item))) break;
        int after = 0;
        if (lane == 0) {
          bars->item[sl][0] = make_int4(it.base, it.n, it.off, it.tok0);
          bars->item[sl][1] = make_int4(it.j0, it.j1, it.slot, it.seq);
          bars->kvh[sl] = kvh;
          mbar_arrive(&bars->item_full[sl]);
          if (more && !runs && !direct) after = atomicAdd(&a.head->taken, 1);  // arrives while this item's tiles load
        }
        if (!more) break;
        const Unit x = make_unit<T>(it, kvh, a.TT, a.causal);
        for (int u = 0; u < x.n; ++u) {
          const int s = kg % KS;
          int slot = 0, page_no = 0;
          if constexpr (PAGED) page_no = page_of(x, u, slot);
          if (kg >= KS && !(ok = all(wait_bar(&bars->k_empty[s], (kg / KS - 1) & 1, w)))) break;
          if (a.ctl.fault == 2 && kg == 0) {
            ok = false;  // test hook: K_0 never arrives
            break;
          }
          load_tile(&tmK, &bars->k_full[s], smem + C::kOffK + s * C::kTileBytes, x, u, page_no, slot);
          ++kg;
          if (u > 0) continue;
          // Q after the first key tile: its buffers free up later.
#pragma unroll
          for (int t = 0; t < T; ++t) {
            if (x.n_t[t] == 0) continue;
            if (q_uses[t] > 0 && !(ok = all(wait_bar(&bars->q_empty[t], (q_uses[t] - 1) & 1, w)))) break;
            if (lane == 0) {
              mbar_arrive_expect_tx(&bars->q_full[t], static_cast<uint32_t>(C::kBoxes) * a.TT * a.r * 128u);
#pragma unroll
              for (int b = 0; b < C::kBoxes; ++b)
                tma_load_4d(&tmQ, &bars->q_full[t], smem + C::kOffQ + t * C::kTileBytes + b * C::kBoxBytes, b * 64, 0,
                            it.base + x.tok_t[t], kvh);
            }
            ++q_uses[t];
          }
          if (!ok) break;
        }
        // (Without a list there are at most two items per CTA: the longest of the
        // second ones go to the CTAs of the shortest first ones.)
        if (runs)
          ++idx;
        else if (direct)
          idx = i > 0 ? total : 2 * gridDim.x - 1 - idx;
        else
          idx = gridDim.x + __shfl_sync(0xffffffffu, after, 0);
      }
      // Every copy issued must land before the CTA may exit.
#pragma unroll
      for (int t = 0; t < T; ++t)
        if (q_uses[t] > 0) drain_bar(&bars->q_full[t], (q_uses[t] - 1) & 1, w);
      for (int s = 0; s < KS; ++s)
        if (kg > s) drain_bar(&bars->k_full[s], ((kg - 1 - s) / KS) & 1, w);
    } else if (warp == C::kVProducerWarp) {
      // ----------------------------------------------------------- V producer
      if (lane == 0) tma_prefetch_desc(&tmV);
      int vg = 0;
      uint32_t tail_last = 0, land_par = 0;  // per stage: last use was a tail; parity of its next landing phase
      bool ok = true;
      Unit x;
      for (int i = 0; ok && next_unit(i, x); ++i) {
        for (int u = 0; u < x.n; ++u) {
          const int s = vg % VS;
          int slot = 0, page_no = 0;
          if constexpr (PAGED) page_no = page_of(x, u, slot);
          if (vg >= VS && !(ok = all(wait_bar(&bars->v_empty[s], (vg / VS - 1) & 1, w)))) break;
          // Only a sequence's last key tile can be short.
          const bool tail = x.keys(u) < kBN;
          load_tile(&tmV, tail ? &bars->v_land[s] : &bars->v_full[s], smem + C::kOffV + s * C::kTileBytes, x, u, page_no,
                    slot);
          tail_last = tail ? tail_last | (1u << s) : tail_last & ~(1u << s);
          if (tail) land_par ^= 1u << s;
          ++vg;
        }
      }
      for (int s = 0; s < VS; ++s)
        if (vg > s) {
          if ((tail_last >> s) & 1)
            drain_bar(&bars->v_land[s], ((land_par >> s) & 1) ^ 1, w);
          else
            drain_bar(&bars->v_full[s], ((vg - 1 - s) / VS) & 1, w);
        }
    } else if (warp == C::kFixWarp) {
      // -------------------------- V rows behind the sequence's last key
      int vg = 0;
      uint32_t land_par = 0;
      Unit x;
      for (int i = 0; next_unit(i, x); ++i) {
        vg += x.n;
        const int keys = max(0, x.keys(x.n - 1));
        if (keys == kBN) continue;
        const int s = (vg - 1) % VS;
        if (!all(wait_bar(&bars->v_land[s], (land_par >> s) & 1, w_item))) break;
        land_par ^= 1u << s;
#pragma unroll
        for (int b = 0; b < C::kBoxes; ++b) {
          uint4* box = reinterpret_cast<uint4*>(smem + C::kOffV + s * C::kTileBytes + b * C::kBoxBytes);
          for (int e = keys * 8 + lane; e < kBN * 8; e += 32) box[e] = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->v_full[s]);
      }
    } else if (warp == C::kMmaWarp) {
      // ----------------------------------------------------------- MMA issue
      const bool leader = elect_one();
      constexpr uint32_t idesc_qk = idesc_bf16(kBM, kBN, false, false);
      constexpr uint32_t idesc_pv = idesc_bf16(kBM, D, false, true);
      const uint32_t tS[2] = {tmem, tmem + 128u};
      const uint32_t tP[2] = {SEP ? tmem + C::kColP : tmem, tmem + 128u};
      const uint32_t tO[2] = {tmem + C::kColO, tmem + C::kColO + D};
      const uint64_t dQ = sdesc_sw128(smem_u32(smem + C::kOffQ), 16, 1024);
      const uint64_t dK = sdesc_sw128(smem_u32(smem + C::kOffK), 16, 1024);
      const uint64_t dV = sdesc_sw128(smem_u32(smem + C::kOffV), C::kBoxBytes, 1024);
      auto ofs_kmaj = [](int k) { return static_cast<uint32_t>((k / 4) * C::kBoxBytes + (k % 4) * 32); };
      // S_t = Q_t K^T, K in ring position g; `last`: the item's last use of Q_t.
      auto issue_s = [&](int t, int g, bool last) {
        const uint64_t qa = sdesc_step(dQ, t * C::kTileBytes);
        const uint64_t ka = sdesc_step(dK, (g % KS) * C::kTileBytes);
#pragma unroll
        for (int k = 0; k < D / 16; k += 4)
          mma_ss_x4(tS[t], sdesc_step(qa, ofs_kmaj(k)), sdesc_step(qa, ofs_kmaj(k + 1)), sdesc_step(qa, ofs_kmaj(k + 2)),
                    sdesc_step(qa, ofs_kmaj(k + 3)), sdesc_step(ka, ofs_kmaj(k)), sdesc_step(ka, ofs_kmaj(k + 1)),
                    sdesc_step(ka, ofs_kmaj(k + 2)), sdesc_step(ka, ofs_kmaj(k + 3)), idesc_qk, k > 0, leader);
        mma_commit(&bars->s_full[t], leader);
        if (last) mma_commit(&bars->q_empty[t], leader);
      };
      // Half h of O_t += P_t V (keys [64h, 64h + 64)), V in ring position g.
      auto issue_pv = [&](int t, int g, int h, bool first) {
        const uint64_t va = sdesc_step(dV, (g % VS) * C::kTileBytes);
        const int k = h * 4;
        mma_ts_x4(tO[t], tP[t] + k * 8, tP[t] + (k + 1) * 8, tP[t] + (k + 2) * 8, tP[t] + (k + 3) * 8,
                  sdesc_step(va, k * 2048), sdesc_step(va, (k + 1) * 2048), sdesc_step(va, (k + 2) * 2048),
                  sdesc_step(va, (k + 3) * 2048), idesc_pv, (!first || k > 0) ? 1u : 0u, leader);
      };
      // Ring position (K and V alike), and per query tile its key tiles and
      // items so far: the phases of the barriers.
      int g0 = 0, c_t[2] = {0, 0}, i_t[2] = {0, 0};
      bool ok = true;
      Unit x;
      for (int i = 0; ok && next_unit(i, x); ++i) {
        if (!(ok = all(wait_bar(&bars->k_full[g0 % KS], (g0 / KS) & 1, w)))) break;
#pragma unroll
        for (int t = 0; t < T; ++t) {
          if (x.n_t[t] == 0) continue;
          if (!(ok = all(wait_bar(&bars->q_full[t], i_t[t] & 1, w)))) break;
          tc_fence_after();
          issue_s(t, g0, x.n_t[t] == 1);
          ++i_t[t];
        }
        if (!ok) break;
        mma_commit(&bars->k_empty[g0 % KS], leader);
        for (int u = 0; ok && u < x.n; ++u) {
          const int g = g0 + u;
          const int s = g % VS;
          const uint32_t par = (g / VS) & 1;
          const int un = u + 1, gn = g + 1;
          if constexpr (SEP) {
            // S of the next key tile once the softmax has loaded this one.
            if (un < x.n) {
              if (!(ok = all(wait_bar(&bars->s_free, (c_t[0] + u) & 1, w)) && all(wait_bar(&bars->k_full[gn % KS], (gn / KS) & 1, w))))
                break;
              tc_fence_after();
              issue_s(0, gn, un == x.n - 1);
              mma_commit(&bars->k_empty[gn % KS], leader);
            }
          }
#pragma unroll
          for (int t = 0; t < T; ++t) {
            if (u >= x.n_t[t]) continue;
            const uint32_t pp = (c_t[t] + u) & 1;
            if (!(ok = all(wait_bar(&bars->p_ready[t][0], pp, w)) && all(wait_bar(&bars->v_full[s], par, w)))) break;
            tc_fence_after();
            issue_pv(t, g, 0, u == 0);
            if (!(ok = all(wait_bar(&bars->p_ready[t][1], pp, w)))) break;
            tc_fence_after();
            issue_pv(t, g, 1, u == 0);
            if constexpr (SEP) mma_commit(&bars->pv_done, leader);
            if (t == T - 1 || u >= x.n_t[T - 1]) mma_commit(&bars->v_empty[s], leader);
            if (u == x.n_t[t] - 1) mma_commit(&bars->o_final[t], leader);
            if (!SEP && un < x.n_t[t]) {
              if (!(ok = all(wait_bar(&bars->k_full[gn % KS], (gn / KS) & 1, w)))) break;
              tc_fence_after();
              issue_s(t, gn, un == x.n_t[t] - 1);
              if (t == T - 1 || un >= x.n_t[T - 1]) mma_commit(&bars->k_empty[gn % KS], leader);
            }
          }
        }
        g0 += x.n;
#pragma unroll
        for (int t = 0; t < T; ++t) c_t[t] += x.n_t[t];
      }
      // All MMAs issued by this thread must finish before tensor memory is freed.
      mma_commit(&bars->drain, leader);
      all(drain_bar(&bars->drain, 0, w));
    }
  } else {
    regs_inc<C::kSoftmaxRegs>();
    // ------------------------------------------------------------- softmax
    const int t = warp >> 2;
    const int quad = warp & 3;
    const int rw = quad * 32 + lane;  // row of the tile: token rw / r, head rw % r
    const int rw_tok = rw / a.r;
    const uint32_t lane_off = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t tS = tmem + lane_off + t * 128u;
    const uint32_t tPw = SEP ? tmem + lane_off + C::kColP : tS;
    const uint32_t tO = tmem + lane_off + C::kColO + t * D;
    const float sl2 = a.scale_log2;
    uint8_t* const stage = smem + C::kOffStage + t * 16384;
    const bool issuer = rw == 0;
    int c = 0, items = 0, boxes = 0;  // key tiles, items and staged boxes so far: the phases of the barriers
    bool ok = true;
    Unit x;
    for (int i = 0; ok && next_unit(i, x); ++i) {
      const int nt = T == 2 && t == 1 ? x.n_t[1] : x.n_t[0];
      const int tok0 = T == 2 && t == 1 ? x.tok_t[1] : x.tok_t[0];
      const int tok = tok0 + rw_tok;
      // Rows of other sequences, and rows that no token fills (128 % r of them,
      // whatever shared memory held), have no say in when O is rescaled:
      // results would depend on what lies beside a sequence.
      const bool mine = rw < a.TT * a.r && tok < x.it.n;
      const float tau = mine ? a.rescale_tau : CUDART_INF_F;
      // Last visible key of this row, and of the tile's first.
      const int lim = a.causal ? min(x.it.off + tok, x.len() - 1) : x.len() - 1;
      const int lim0 = a.causal ? min(x.it.off + tok0, x.len() - 1) : x.len() - 1;
      float m = -CUDART_INF_F;
      float l = 0.f;
      for (int u = 0; u < nt; ++u) {
        ok = all(wait_bar(&bars->s_full[t], (c + u) & 1, w));
        if (!ok) break;
        tc_fence_after();
        uint32_t sr[kBN];
        tmem_ld64x2(tS, sr);  // (no instruction may name more registers than the launch's share)
        if constexpr (SEP) {
          tc_fence_before();
          mbar_arrive(&bars->s_free);
        }
        const int k0 = (x.it.j0 + u) * kBN;
        if (k0 + kBN - 1 > lim0) {
#pragma unroll
          for (int e = 0; e < kBN; ++e)
            if (k0 + e > lim) sr[e] = __float_as_uint(-CUDART_INF_F);
        }
        // Row max as 8 independent partial maxima of three-input max.
        float pm[8];
#pragma unroll
        for (int y = 0; y < 8; ++y) pm[y] = fmaxf(__uint_as_float(sr[y]), __uint_as_float(sr[8 + y]));
#pragma unroll
        for (int e = 16; e < kBN; e += 16)
#pragma unroll
          for (int y = 0; y < 8; ++y)
            pm[y] = fmax3(pm[y], __uint_as_float(sr[e + y]), __uint_as_float(sr[e + 8 + y]));
        pm[0] = fmax3(pm[0], pm[1], pm[2]);
        pm[3] = fmax3(pm[3], pm[4], pm[5]);
        pm[6] = fmaxf(pm[6], pm[7]);
        const float m_cand = fmax3(pm[0], pm[3], pm[6]) * sl2;
        bool rescale = false;
        float alpha = 1.f;
        if (u == 0) {
          m = m_cand;  // -inf for a row that sees no key of this tile
        } else if (__any_sync(0xffffffffu, m_cand > m + tau)) {
          const float m_new = fmaxf(m, m_cand);
          alpha = m_new == -CUDART_INF_F ? 1.f : exp2_accurate(m - m_new);
          m = m_new;
          l *= alpha;
          rescale = true;
        }
        const float neg_m = m == -CUDART_INF_F ? 0.f : -m;
        if constexpr (SEP) {
          // (Before an item's first tile the last item's o_final has said so.)
          if (u > 0) {
            ok = all(wait_bar(&bars->pv_done, (c + u - 1) & 1, w));
            if (!ok) break;
            tc_fence_after();
          }
        }
        float ps[8];
#pragma unroll
        for (int y = 0; y < 8; ++y) ps[y] = 0.f;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int b = 2 * h; b < 2 * h + 2; ++b) {
            uint32_t pk[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              float x0, x1;
              ffma2(x0, x1, __uint_as_float(sr[b * 32 + 2 * e]), __uint_as_float(sr[b * 32 + 2 * e + 1]), sl2, sl2,
                    neg_m, neg_m);
              // All on the exponential unit: two of 32 on the FMA pipe, as in
              // fa_fwd.cu at d = 128, gained nothing here (678-685 us against
              // 672-679 at 16k packed tokens), and their error (1e-4) would
              // enter L.
              const float p0 = ex2(x0);
              const float p1 = ex2(x1);
              fadd2(ps[(2 * e) & 7], ps[(2 * e + 1) & 7], ps[(2 * e) & 7], ps[(2 * e + 1) & 7], p0, p1);
              // bf16: the type of V, which the weights meet in P V.
              pk[e] = pack_bf16x2(p0, p1);
            }
            tmem_st16(tPw + b * 16, pk);
          }
          if (h == 0 && rescale) {
#pragma unroll
            for (int b = 0; b < D / 32; ++b) {
              uint32_t o32[32];
              tmem_ld32(tO + b * 32, o32);
#pragma unroll
              for (int e = 0; e < 32; e += 2) {
                float y0, y1;
                fmul2(y0, y1, __uint_as_float(o32[e]), __uint_as_float(o32[e + 1]), alpha, alpha);
                o32[e] = __float_as_uint(y0);
                o32[e + 1] = __float_as_uint(y1);
              }
              tmem_st32(tO + b * 32, o32);
            }
          }
          tmem_st_wait();
          tc_fence_before();
          mbar_arrive(&bars->p_ready[t][h]);
        }
        l += ((ps[0] + ps[1]) + (ps[2] + ps[3])) + ((ps[4] + ps[5]) + (ps[6] + ps[7]));
      }
      if (ok && nt > 0) {
        ok = all(wait_bar(&bars->o_final[t], items & 1, w));
        ++items;
        c += nt;
      }
      if (!ok) break;
      tc_fence_after();
      const float inv_l = l == 0.f ? 0.f : 1.f / l;  // 0: no visible key (O is 0 there, or never written)
      const float L = l == 0.f ? -CUDART_INF_F : (m + lg2(l)) * 0.69314718055994530942f;
      const long long row = static_cast<long long>(x.it.base) + tok;
      const int head = x.kvh * a.r + rw - rw_tok * a.r;
      // 64 columns of this row's O, normalised.
      auto load_o = [&](int b, uint32_t (&oo)[64]) {
        uint32_t(&o0)[32] = *reinterpret_cast<uint32_t(*)[32]>(&oo[0]);
        uint32_t(&o1)[32] = *reinterpret_cast<uint32_t(*)[32]>(&oo[32]);
        if (nt == 0) {
          // A part of the unit's keys that this tile's rows do not reach.
#pragma unroll
          for (int e = 0; e < 64; ++e) oo[e] = 0u;
          return;
        }
        tmem_ld32_nowait(tO + b * 64, o0);
        tmem_ld32_nowait(tO + b * 64 + 32, o1);
        tmem_ld_wait(o0);
        tmem_ld_tie(o1);
#pragma unroll
        for (int e = 0; e < 64; ++e) oo[e] = __float_as_uint(__uint_as_float(oo[e]) * inv_l);
      };
      if (RUNS && x.it.slot >= 0) {
        const long long prow = static_cast<long long>(x.it.slot) * (T * kBM) + t * kBM + rw;
#pragma unroll
        for (int b = 0; b < D / 64; ++b) {
          uint32_t oo[64];
          load_o(b, oo);
          if (mine)
#pragma unroll
            for (int e = 0; e < 64; e += 8)
              store_sector(a.part_o + prow * D + b * 64 + e, *reinterpret_cast<uint32_t(*)[8]>(&oo[e]));
          __syncwarp();
        }
        if (mine) a.part_l[prow] = L;
        continue;
      }
      // 16 columns as bf16 (or their rounding residual), two per register.
      auto pack16 = [](const uint32_t* y, bool resid, uint32_t (&v)[8]) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float x0 = __uint_as_float(y[2 * e]), x1 = __uint_as_float(y[2 * e + 1]);
          v[e] = pack_bf16x2(x0, x1);
          if (resid) {
            const __nv_bfloat162 hi = *reinterpret_cast<const __nv_bfloat162*>(&v[e]);
            v[e] = pack_bf16x2(x0 - __low2float(hi), x1 - __high2float(hi));
          }
        }
      };
      constexpr int kBoxesO = D / 64;
      const int jobs = kBoxesO * (a.resid.p ? 2 : 1);
      if (C::kStaged && tok0 + a.TT <= x.it.n) {
        // A whole tile: boxes of 64 columns staged in the tensor map's swizzle.
        for (int b = 0; b < jobs; ++b, ++boxes) {
          const int col = b % kBoxesO;
          const bool resid = b >= kBoxesO;
          uint32_t oo[64];
          load_o(col, oo);
          if (boxes > 0) {
            // The staged box before this one has been read.
            if (issuer) {
              bulk_wait_read<0>();
              mbar_arrive(&bars->epi_free[t]);
            }
            __syncwarp();
            if (!(ok = all(wait_bar(&bars->epi_free[t], (boxes - 1) & 1, w)))) break;
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t v[8];
            pack16(oo + 16 * e, resid, v);
            *reinterpret_cast<uint4*>(stage + rw * 128 + (((2 * e) ^ (rw & 7)) << 4)) = make_uint4(v[0], v[1], v[2], v[3]);
            *reinterpret_cast<uint4*>(stage + rw * 128 + (((2 * e + 1) ^ (rw & 7)) << 4)) = make_uint4(v[4], v[5], v[6], v[7]);
          }
          fence_proxy_async_smem();
          mbar_arrive(&bars->epi_full[t]);
          // (After a timeout every lane leaves at a wait below or above.)
          if (issuer && wait_bar(&bars->epi_full[t], boxes & 1, w)) {
            tma_store_4d(resid ? &tmR : &tmO, stage, col * 64, 0, x.it.base + tok0, x.kvh);
            bulk_commit();
          }
          __syncwarp();
        }
      } else if (tok0 < x.it.n) {
        // Each thread stores its own row, whole 32-byte sectors at a time
        // where the view's alignment allows it.
        for (int b = 0; b < jobs; ++b) {
          const int col = b % kBoxesO;
          const bool resid = b >= kBoxesO;
          uint32_t oo[64];
          load_o(col, oo);
          if (mine) {
            const Rows& out = resid ? a.resid : a.o;
            __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(out.p) + row * out.ts + head * out.hs + col * 64;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint32_t v[8];
              pack16(oo + 16 * e, resid, v);
              if (a.sectors) {
                store_sector(dst + 16 * e, v);
              } else {
                reinterpret_cast<uint4*>(dst + 16 * e)[0] = make_uint4(v[0], v[1], v[2], v[3]);
                reinterpret_cast<uint4*>(dst + 16 * e)[1] = make_uint4(v[4], v[5], v[6], v[7]);
              }
            }
          }
          __syncwarp();
        }
      }
      if (mine) a.lse[static_cast<long long>(head) * a.total + row] = L;
    }
    if (issuer) bulk_wait_read<0>();  // a staged box, before the CTA exits
  }

  tc_fence_before();
  __syncthreads();
  if (warp == C::kMmaWarp) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// Merges the parts of the units that were cut along their keys: O = sum_p
// e^(L_p - L) O_p, L = log sum_p e^(L_p). Mostly two or three parts: a warp
// takes kMergeRows rows side by side (a row is one load per lane and part) to
// keep enough loads in flight (148 cut units of 256 rows took 16 us with one
// row per warp). Many parts (few units, a long cache): the block's warps share
// the parts of kMergeRows rows. Blocks go through (cut unit, group of rows)
// with the grid's stride, as the number of cut units is known on the device
// only.
constexpr int kMergeRows = 4;
template <int D>
__global__ void __launch_bounds__(128) packed_merge_kernel(const PkArgs a) {
  constexpr int rows = PkCfg<D>::T * kBM;
  constexpr int groups = rows / kMergeRows;
  constexpr int VW = D / 32;
  __shared__ float s_acc[4][kMergeRows][D], s_m[4][kMergeRows], s_den[4][kMergeRows];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  // First the units of few parts, four groups per block; then the others, if
  // there are any (the plan counts them).
  const int splits = a.head->splits;
  const int few_work = splits * (groups / 4), work = few_work + (a.head->taken > 0 ? splits * groups : 0);
#pragma unroll 1
  for (int g = blockIdx.x; g < work; g += gridDim.x) {
    const bool many = g >= few_work;
    const int in_pass = many ? g - few_work : g, per_unit = many ? groups : groups / 4;
    const PlanSplit sp = a.split_list[in_pass / per_unit];
    if ((sp.parts > kMergeManyParts) != many) continue;
    const int group = in_pass % per_unit;
    const int rw0 = (many ? group : group * 4 + warp) * kMergeRows;
    const long long part0 = static_cast<long long>(sp.slot0) * rows + rw0;
    // Rows of the tile, and of these the ones that hold a token: the others'
    // partials were never written.
    bool mine[kMergeRows];
    int tok[kMergeRows], head[kMergeRows];
    float acc[kMergeRows][VW], m[kMergeRows], den[kMergeRows];
#pragma unroll
    for (int i = 0; i < kMergeRows; ++i) {
      const int t = (rw0 + i) / kBM, rt = (rw0 + i) % kBM;
      tok[i] = sp.tok0 + t * a.TT + rt / a.r;
      head[i] = sp.kvh * a.r + rt % a.r;
      mine[i] = rt < a.TT * a.r && tok[i] < sp.n;
      m[i] = -CUDART_INF_F;
      den[i] = 0.f;
#pragma unroll
      for (int k = 0; k < VW; ++k) acc[i][k] = 0.f;
    }
    // One more part (or sum of parts) with maximum or logsumexp L, weight sum d
    // and weighted row x into row i.
    auto add = [&](int i, float L, float d, const float (&x)[VW]) {
      const float top = fmaxf(m[i], L);
      const float ref = top == -CUDART_INF_F ? 0.f : top;  // no key so far: every weight 0
      const float old = expf(m[i] - ref), wt = expf(L - ref);
      m[i] = top;
      den[i] = den[i] * old + wt * d;
#pragma unroll
      for (int k = 0; k < VW; ++k) acc[i][k] = acc[i][k] * old + (wt == 0.f ? 0.f : wt * x[k]);
    };
#pragma unroll 2
    for (int p = many ? warp : 0; p < sp.parts; p += many ? 4 : 1) {
      float L[kMergeRows], x[kMergeRows][VW];
#pragma unroll
      for (int i = 0; i < kMergeRows; ++i) {
        const long long at = part0 + static_cast<long long>(p) * rows + i;
        L[i] = mine[i] ? a.part_l[at] : -CUDART_INF_F;
        if (mine[i])
          load_vec(a.part_o + at * D + lane * VW, x[i]);
        else
#pragma unroll
          for (int k = 0; k < VW; ++k) x[i][k] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < kMergeRows; ++i) add(i, L[i], 1.f, x[i]);
    }
    if (many) {
      // The warps' sums, in warp order; warp 0 stores.
      __syncthreads();  // the last group's have been read
#pragma unroll
      for (int i = 0; i < kMergeRows; ++i) {
#pragma unroll
        for (int k = 0; k < VW; ++k) s_acc[warp][i][lane * VW + k] = acc[i][k];
        if (lane == 0) {
          s_m[warp][i] = m[i];
          s_den[warp][i] = den[i];
        }
      }
      __syncthreads();
      if (warp > 0) continue;
#pragma unroll
      for (int v = 1; v < 4; ++v)
#pragma unroll
        for (int i = 0; i < kMergeRows; ++i) {
          float x[VW];
#pragma unroll
          for (int k = 0; k < VW; ++k) x[k] = s_acc[v][i][lane * VW + k];
          add(i, s_m[v][i], s_den[v][i], x);
        }
    }
#pragma unroll
    for (int i = 0; i < kMergeRows; ++i) {
      if (!mine[i]) continue;
      const float inv = den[i] == 0.f ? 0.f : 1.f / den[i];
      const long long row = static_cast<long long>(sp.base) + tok[i];
      uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(a.o.p) + row * a.o.ts + head[i] * a.o.hs +
                                                  lane * VW);
      uint32_t* rst = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(a.resid.p) + row * a.resid.ts +
                                                  head[i] * a.resid.hs + lane * VW);
#pragma unroll
      for (int k = 0; k < VW / 2; ++k) {
        const float x0 = acc[i][2 * k] * inv, x1 = acc[i][2 * k + 1] * inv;
        const uint32_t o = pack_bf16x2(x0, x1);
        dst[k] = o;
        if (a.resid.p) {
          const __nv_bfloat162 hi = *reinterpret_cast<const __nv_bfloat162*>(&o);
          rst[k] = pack_bf16x2(x0 - __low2float(hi), x1 - __high2float(hi));
        }
      }
      if (lane == 0)
        a.lse[static_cast<long long>(head[i]) * a.total + row] = den[i] == 0.f ? -CUDART_INF_F : m[i] + logf(den[i]);
    }
  }
}

struct Layout {
  PlanLayout plan;
  int TT, unit;
  bool runs;            // the work may be cut into runs
  bool direct;          // no list
  int max_parts;
  long long max_items, key_tiles;
  long long grid;       // CTAs of the launch
  size_t off_o, off_l, bytes;
};

// What is laid out depends on the shape alone (kShareCtas, not the device's
// multiprocessors), as the size queries know no more: the choice of runs is not
// monotone in the CTAs. `sms`, at most kShareCtas, are those of the launch.
Layout make_layout(const SeqShape& s, const CacheShape* c, int sms) {
  Layout x;
  const int tiles = s.d == 128 ? 2 : 1;
  x.TT = kBM / s.r();
  x.unit = tiles * x.TT;
  x.max_items = plan_max_units(s.S, s.T, x.unit);
  // Runs where there can be so few units (the plan decides); of prompts fewer
  // than half the CTAs, as their keys are no more than their queries, and the
  // plan's way to runs and the merge's launch cost 4 us even where no unit is cut
  // (17 short prompts of 16 heads: 18.4 -> 22.5 us). The sums of their costs
  // stay in 32 bits.
  const int per_sm = tiles == 2 ? 1 : 2;
  const int most_ctas = per_sm * kShareCtas, ctas = per_sm * sms;
  const long long least = (static_cast<long long>(s.T) + x.unit - 1) / x.unit;
  const long long keys = c ? static_cast<long long>(c->max_pages) * c->page : s.T;
  const long long key_tiles = x.key_tiles = (keys + kBN - 1) / kBN + 1;
  x.runs = s.S <= kPlanSeqs && least * s.Hkv < static_cast<long long>(c ? kRunUnits : most_ctas / 2) &&
           (key_tiles + 4) * kCostTile * kRunUnits < (1LL << 31);
  // (The plan's own condition, for the longest units that there can be.)
  const long long most_cost = kCostItem + kCostTile * key_tiles;
  const long long mean_cost = x.max_items * s.Hkv * most_cost / most_ctas;
  if (!plan_wants_runs(mean_cost, most_cost)) x.runs = false;
  x.max_parts = 0;
  if (x.runs) {
    // Each run boundary adds an item and cuts at most one unit; the parts of a
    // unit are kRunLeast key tiles or more.
    const long long most = x.max_items * s.Hkv * (key_tiles / kRunLeast);
    x.max_parts = most < 2 * most_ctas ? static_cast<int>(most) : 2 * most_ctas;
    x.max_items += kRunUnits + most_ctas;
  }
  // At most two items per CTA: finding them in the offsets costs a CTA less
  // than the list's kernel before it (one prompt of 512 tokens, 8 + 1 heads, d =
  // 64: 12.2 -> 11.2 us; of 1054, 32 + 16 heads: 21.6 -> 18.9).
  x.direct = !c && !x.runs && x.max_items * s.Hkv <= 2 * ctas && s.S <= kPlanSeqs;
  x.grid = x.runs || x.max_items * s.Hkv > ctas ? ctas : x.max_items * s.Hkv;
  x.plan = plan_layout(x.max_items, x.runs ? most_ctas : 0, x.runs ? most_ctas : 0);
  x.off_o = x.plan.bytes;
  x.off_l = x.off_o + static_cast<size_t>(x.max_parts) * tiles * kBM * s.d * 4;
  x.bytes = x.off_l + static_cast<size_t>(x.max_parts) * tiles * kBM * 4 + 32;  // + alignment of the parts
  return x;
}

template <int D, bool PAGED, bool RUNS>
cudaError_t launch_t(const SeqShape& s, const CacheShape* c, const Layout& x, const CUtensorMap& tq,
                     const CUtensorMap& tk, const CUtensorMap& tv, const CUtensorMap& to, const CUtensorMap& tr,
                     const Rows& o, const Rows& resid, float* lse, void* workspace, int sms, const LaunchCtl& ctl,
                     cudaStream_t stream) {
  using C = PkCfg<D>;
  auto kern = packed_fwd_kernel<D, PAGED, RUNS>;
  static SmemOnce once;
  cudaError_t e = once.set(reinterpret_cast<const void*>(kern), C::kSmemBytes);
  if (e != cudaSuccess) return e;
  // With another launch count than the split's sum the softmax warps' increase
  // could never be granted.
  static const int launch_regs = [&] {
    cudaFuncAttributes at{};
    return cudaFuncGetAttributes(&at, kern) == cudaSuccess ? at.numRegs : -1;
  }();
  if (launch_regs != C::kLaunchRegs) return cudaErrorLaunchOutOfResources;
  uint8_t* ws = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(workspace) + 31) / 32 * 32);
  PlanArgs p{};
  p.cu = s.cu;
  p.lens = c ? c->lens : nullptr;
  p.S = s.S;
  p.T = s.T;
  p.max_q = c ? c->max_q : s.T;
  p.max_len = c ? static_cast<long long>(c->max_pages) * c->page : s.T;
  p.unit = x.unit;
  p.causal = s.causal;
  p.heads = s.Hkv;
  p.run_ctas = x.runs ? C::kMinBlocks * sms : 0;
  p.run_first = reinterpret_cast<int*>(ws + x.plan.run_first);
  p.sorted = x.max_items * s.Hkv > static_cast<long long>(C::kMinBlocks) * sms;
  p.head = reinterpret_cast<PlanHeader*>(ws + x.plan.head);
  p.items = reinterpret_cast<PlanItem*>(ws + x.plan.items);
  p.split_list = reinterpret_cast<PlanSplit*>(ws + x.plan.splits);
  p.err = ctl.err;
  PkArgs a{};
  a.head = p.head;
  a.items = p.items;
  a.split_list = p.split_list;
  a.run_first = p.run_first;
  if (c) {
    a.table = c->table;
    a.table_stride = c->table_stride;
    a.n_pages = c->n_pages;
    a.page = c->page;
    a.pb = page_box(c->page);
  }
  a.o = o;
  a.resid = resid;
  auto whole = [&](const Rows& y) {
    return (reinterpret_cast<uintptr_t>(y.p) % 32 == 0) && (s.T == 1 || y.ts % 16 == 0) && (s.Hq == 1 || y.hs % 16 == 0);
  };
  a.sectors = whole(o) && (!resid.p || whole(resid));
  a.lse = lse;
  a.part_o = reinterpret_cast<float*>(ws + x.off_o);
  a.part_l = reinterpret_cast<float*>(ws + x.off_l);
  a.total = s.T;
  a.Hkv = s.Hkv;
  a.r = s.r();
  a.TT = x.TT;
  a.causal = s.causal;
  a.scale_log2 = s.scale * 1.4426950408889634f;
  a.rescale_tau = resid.p ? kRescaleExact : kRescaleLazy;
  a.item_ns = static_cast<uint64_t>(x.key_tiles) * 20000;
  a.ctl = ctl;
  a.direct = x.direct;
  a.S = s.S;
  a.unit = x.unit;
  a.cu = s.cu;
  if (x.direct) {
    kern<<<static_cast<unsigned>(x.grid), C::kThreads, C::kSmemBytes, stream>>>(tq, tk, tv, to, tr, a);
    return cudaGetLastError();
  }
  packed_plan_kernel<<<1, kPlanThreads, 0, stream>>>(p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  e = launch_dependent(kern, dim3(static_cast<unsigned>(x.grid)), C::kThreads, C::kSmemBytes, stream, tq, tk, tv, to, tr,
                       a);
  if (e != cudaSuccess || !x.runs) return e;
  return launch_dependent(packed_merge_kernel<D>, dim3(8 * sms), 128, 0, stream, a);
}

}  // namespace

size_t packed_fwd_workspace_bytes(const SeqShape& s, const CacheShape* c) {
  return make_layout(s, c, kShareCtas).bytes;
}

void packed_fwd_layout(const SeqShape& s, const CacheShape* c, int sms, long long* out) {
  const Layout x = make_layout(s, c, sms);
  out[0] = static_cast<long long>(x.bytes);
  out[1] = x.runs;
  out[2] = x.direct;
  out[3] = x.max_items * s.Hkv;
  out[4] = x.grid;
}

cudaError_t launch_packed_fwd(const SeqShape& s, const CacheShape* c, const Rows& q, const Rows& o, const Rows& resid,
                              const Rows& krows, const Rows& vrows, const Pages& kpages, const Pages& vpages,
                              float* lse, void* workspace, int sms, const LaunchCtl& ctl, cudaStream_t stream) {
  const Layout x = make_layout(s, c, sms);
  CUtensorMap tq, tk, tv, to, tr;
  bool ok = encode_group_map(&tq, q, s.T, s.Hkv, s.r(), s.d, x.TT) &&
            encode_group_map(&to, o, s.T, s.Hkv, s.r(), s.d, x.TT) &&
            encode_group_map(&tr, resid.p ? resid : o, s.T, s.Hkv, s.r(), s.d, x.TT);
  if (c) {
    const int pb = page_box(c->page);
    ok = ok && encode_pages_map(&tk, kpages, c->n_pages, s.Hkv, c->page, s.d, pb) &&
         encode_pages_map(&tv, vpages, c->n_pages, s.Hkv, c->page, s.d, pb);
  } else {
    ok = ok && encode_rows_map(&tk, krows, s.T, s.Hkv, s.d, kBN) && encode_rows_map(&tv, vrows, s.T, s.Hkv, s.d, kBN);
  }
  if (!ok) return cudaErrorInvalidValue;
#define FA_ARGS s, c, x, tq, tk, tv, to, tr, o, resid, lse, workspace, sms, ctl, stream
  if (s.d == 64) {
    if (c) return launch_t<64, true, true>(FA_ARGS);
    return x.runs ? launch_t<64, false, true>(FA_ARGS) : launch_t<64, false, false>(FA_ARGS);
  }
  if (c) return launch_t<128, true, true>(FA_ARGS);
  return x.runs ? launch_t<128, false, true>(FA_ARGS) : launch_t<128, false, false>(FA_ARGS);
#undef FA_ARGS
}

}  // namespace fa
