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
//  * The work comes from a list (fa_plan.cuh), longest first. A unit of few
//    long rows (a chunk over a long cache, too few to fill the GPU) may be cut
//    along its keys; its parts leave O / l and logsumexp in the workspace and
//    a second kernel merges them.
//  * Tiles end where sequences do: scores of keys behind the end are replaced
//    by -inf; the V rows there, which may hold anything (the next sequence,
//    stale cache slots, NaN), are zeroed in shared memory before P V (warp
//    kFixWarp); rows are stored whole tiles at a time by TMA, or row by row
//    where the tile holds rows that are not this sequence's.
//
// Warp roles (w0 = 4T): 0..w0-1 softmax, w0 Q and K producer, w0+1 MMA and
// tensor memory, w0+2 V producer, w0+3 V rows behind the end.

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
// Register split of the one-tile form (as fa_fwd.cu).
constexpr int kSoftmaxRegs1 = 192;
constexpr int kOtherRegs1 = 64;
static_assert(kSoftmaxRegs1 + kOtherRegs1 == 2 * 128, "register split of the one-tile form");
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
  static constexpr int kProducerWarp = 4 * T;
  static constexpr int kMmaWarp = 4 * T + 1;
  static constexpr int kVProducerWarp = 4 * T + 2;
  static constexpr int kFixWarp = 4 * T + 3;
  static constexpr int kKStages = T == 1 ? 2 : 3;
  static constexpr int kVStages = 2;
  static constexpr int kBoxBytes = kBN * 128;
  static constexpr int kBoxes = D / 64;
  static constexpr int kTileBytes = kBoxBytes * kBoxes;
  static constexpr int kOffQ = 0;
  static constexpr int kOffK = T * kTileBytes;
  static constexpr int kOffV = kOffK + kKStages * kTileBytes;
  static constexpr int kOffBar = kOffV + kVStages * kTileBytes;
  static constexpr int kBarBytes = 512;
  // Output staging: two 16-KB boxes per tile; the Q_t buffer at d = 128, the
  // Q buffer and a box of its own at d = 64.
  static constexpr int kOffStage = (kOffBar + kBarBytes + 1023) / 1024 * 1024;
  static constexpr int kSmemBytes = (T == 1 ? kOffStage + 16384 : kOffBar + kBarBytes) + 1024;
  static constexpr uint32_t kTmemCols = T == 1 ? 256 : 512;
  static constexpr uint32_t kColO = T == 1 ? 128 : 256;
  static constexpr uint32_t kColP = 192;  // SEP
  static_assert(kSmemBytes <= 227 * 1024, "shared memory budget");
  static_assert(T == 1 ? (kSmemBytes <= 228 * 1024 / 2 - 1024 && 3 * kSmemBytes > 228 * 1024)
                       : kSmemBytes > 114 * 1024,
                "CTAs per SM");
};

struct PkArgs {
  const PlanHeader* head;
  const PlanItem* items;
  const int* slots;
  const PlanSplit* split_list;
  const int* cu;
  const int* lens;  // paged
  const int* table;
  long long table_stride;
  int n_pages, page, pb;
  Rows o, resid;
  float* lse;
  float* part_o;  // [slot][KV head][T * 128][D]
  float* part_l;
  int total, Hkv, r, TT, causal;
  float scale_log2, rescale_tau;
  LaunchCtl ctl;
};

struct PkBars {
  uint64_t q_full;
  uint64_t k_full[3], v_full[2], v_land[2], k_empty[3], v_empty[2];
  uint64_t s_full[2], p_ready[2][2], o_final[2];
  uint64_t s_free, pv_done;
  uint64_t epi_full[2][2], epi_free[2];  // epi_full: [tile][staging box]
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
};
static_assert(sizeof(PkBars) <= 512, "barrier block exceeds its shared-memory reservation");

constexpr int kPlanThreads = 512;
__global__ void __launch_bounds__(kPlanThreads) packed_plan_kernel(const PlanArgs a) {
  __shared__ PlanShared sh;
  pdl_launch_dependents();
  plan_block<kPlanThreads>(a, sh);
}

template <int D, bool PAGED>
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
    mbar_init(&bars->q_full, 1);
    for (int s = 0; s < KS; ++s) {
      mbar_init(&bars->k_full[s], 1);
      mbar_init(&bars->k_empty[s], 1);
    }
    for (int s = 0; s < VS; ++s) {
      mbar_init(&bars->v_full[s], 1);
      mbar_init(&bars->v_land[s], 1);
      mbar_init(&bars->v_empty[s], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&bars->s_full[t], 1);
      mbar_init(&bars->p_ready[t][0], kBM);
      mbar_init(&bars->p_ready[t][1], kBM);
      mbar_init(&bars->o_final[t], 1);
      mbar_init(&bars->epi_full[t][0], kBM);
      mbar_init(&bars->epi_full[t][1], kBM);
      mbar_init(&bars->epi_free[t], 1);
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
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // Everything above ran beside the plan.
  pdl_launch_dependents();
  pdl_wait();
  const int item_no = blockIdx.x / a.Hkv;
  if (item_no >= a.head->items) {
    if (warp == C::kMmaWarp) tmem_dealloc(bars->tmem_base, C::kTmemCols);
    return;
  }
  const int kvh = blockIdx.x - item_no * a.Hkv;
  const PlanItem item = a.items[item_no];
  const int tok_base = a.cu ? a.cu[item.seq] : item.seq;  // the sequence's first row
  const int n_tok = a.cu ? a.cu[item.seq + 1] - tok_base : 1;
  const int len = PAGED ? a.lens[item.seq] : n_tok;
  const int off = len - n_tok;  // place of the first new token
  // Tile t: tokens [tok0 + t TT, ...), key tiles [j0, j0 + n_t).
  int n_t[2] = {0, 0}, tok_t[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    tok_t[t] = item.tok0 + t * a.TT;
    if (t < T && tok_t[t] < n_tok)
      n_t[t] = max(0, min(item.j1, plan_fwd_tiles(n_tok, len, tok_t[t], a.TT, a.causal)) - item.j0);
  }
  const int n = max(n_t[0], n_t[1]);  // stream length

  const uint32_t tmem = bars->tmem_base;
  const Watch w{&bars->abort, a.ctl.err, a.ctl.budget_ns};
  auto all = [](bool b) { return __all_sync(0xffffffffu, b); };

  // Copies key tile j of the sequence (K or V) to a stage; whole warp.
  // Packed: one box per 64 columns. Paged: lane i copies part i.
  auto keys_of = [&](int j) { return max(0, min(kBN, len - j * kBN)); };
  auto page_of = [&](int j, int& slot) -> int {
    slot = 0;
    int page_no = 0;
    if (lane * a.pb < keys_of(j)) {
      const int key = j * kBN + lane * a.pb;
      const int pi = key / a.page;
      slot = key - pi * a.page;
      page_no = a.table[static_cast<long long>(item.seq) * a.table_stride + pi];
      if (page_no < 0 || page_no >= a.n_pages) {
        page_no = a.n_pages;  // past the tensor: the copy fills zeros
        atomicOr(a.ctl.err, kErrData);
      }
    }
    return page_no;
  };
  auto load_tile = [&](const CUtensorMap* tm, uint64_t* bar, uint8_t* dst, int j, int page_no, int slot) {
    if constexpr (PAGED) {
      const int parts = (keys_of(j) + a.pb - 1) / a.pb;
      if (lane == 0) mbar_arrive_expect_tx(bar, static_cast<uint32_t>(parts) * a.pb * 128u * C::kBoxes);
      __syncwarp();
      if (lane < parts)
#pragma unroll
        for (int x = 0; x < C::kBoxes; ++x)
          tma_load_4d(tm, bar, dst + lane * a.pb * 128 + x * C::kBoxBytes, x * 64, slot, kvh, page_no);
    } else if (lane == 0) {
      mbar_arrive_expect_tx(bar, C::kTileBytes);
#pragma unroll
      for (int x = 0; x < C::kBoxes; ++x)
        tma_load_3d(tm, bar, dst + x * C::kBoxBytes, x * 64, tok_base + j * kBN, kvh);
    }
  };

  if (warp >= 4 * T) {
    if constexpr (T == 1) regs_dec<kOtherRegs1>();
    if (warp == C::kProducerWarp) {
      // ------------------------------------------------------- Q, K producer
      int issued = 0;
      if (lane == 0) {
        tma_prefetch_desc(&tmQ);
        tma_prefetch_desc(&tmK);
        const int tiles = T == 2 && n_t[1] > 0 ? 2 : 1;
        mbar_arrive_expect_tx(&bars->q_full, static_cast<uint32_t>(tiles * C::kBoxes) * a.TT * a.r * 128u);
        for (int t = 0; t < tiles; ++t)
#pragma unroll
          for (int x = 0; x < C::kBoxes; ++x)
            tma_load_4d(&tmQ, &bars->q_full, smem + C::kOffQ + t * C::kTileBytes + x * C::kBoxBytes, x * 64, 0,
                        tok_base + tok_t[t], kvh);
      }
      __syncwarp();
      for (int u = 0; u < n; ++u) {
        const int s = u % KS;
        int slot = 0, page_no = 0;
        if constexpr (PAGED) page_no = page_of(item.j0 + u, slot);
        if (u >= KS && !all(wait_bar(&bars->k_empty[s], (u / KS - 1) & 1, w))) break;
        load_tile(&tmK, &bars->k_full[s], smem + C::kOffK + s * C::kTileBytes, item.j0 + u, page_no, slot);
        issued = u + 1;
      }
      // Every copy issued must land before the CTA may exit.
      drain_bar(&bars->q_full, 0, w);
      for (int s = 0; s < KS; ++s)
        if (issued > s) drain_bar(&bars->k_full[s], ((issued - 1 - s) / KS) & 1, w);
    } else if (warp == C::kVProducerWarp) {
      // ----------------------------------------------------------- V producer
      if (lane == 0) tma_prefetch_desc(&tmV);
      int issued = 0;
      bool tail_issued = false;
      for (int u = 0; u < n; ++u) {
        const int s = u % VS;
        int slot = 0, page_no = 0;
        if constexpr (PAGED) page_no = page_of(item.j0 + u, slot);
        if (u >= VS && !all(wait_bar(&bars->v_empty[s], (u / VS - 1) & 1, w))) break;
        // Only the sequence's last key tile can be short.
        const bool tail = keys_of(item.j0 + u) < kBN;
        load_tile(&tmV, tail ? &bars->v_land[s] : &bars->v_full[s], smem + C::kOffV + s * C::kTileBytes, item.j0 + u,
                  page_no, slot);
        if (tail)
          tail_issued = true;
        else
          issued = u + 1;
      }
      for (int s = 0; s < VS; ++s) {
        if (issued > s) drain_bar(&bars->v_full[s], ((issued - 1 - s) / VS) & 1, w);
        if (tail_issued && s == (n - 1) % VS) drain_bar(&bars->v_land[s], 0, w);
      }
    } else if (warp == C::kFixWarp) {
      // -------------------------- V rows behind the sequence's last key
      const int keys = n > 0 ? keys_of(item.j0 + n - 1) : kBN;
      if (keys < kBN) {
        const int s = (n - 1) % VS;
        if (all(wait_bar(&bars->v_land[s], 0, w))) {
#pragma unroll
          for (int x = 0; x < C::kBoxes; ++x) {
            uint4* box = reinterpret_cast<uint4*>(smem + C::kOffV + s * C::kTileBytes + x * C::kBoxBytes);
            for (int i = keys * 8 + lane; i < kBN * 8; i += 32) box[i] = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars->v_full[s]);
        }
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
      auto issue_s = [&](int t, int u) {
        const uint64_t qa = sdesc_step(dQ, t * C::kTileBytes);
        const uint64_t ka = sdesc_step(dK, (u % KS) * C::kTileBytes);
#pragma unroll
        for (int k = 0; k < D / 16; k += 4)
          mma_ss_x4(tS[t], sdesc_step(qa, ofs_kmaj(k)), sdesc_step(qa, ofs_kmaj(k + 1)), sdesc_step(qa, ofs_kmaj(k + 2)),
                    sdesc_step(qa, ofs_kmaj(k + 3)), sdesc_step(ka, ofs_kmaj(k)), sdesc_step(ka, ofs_kmaj(k + 1)),
                    sdesc_step(ka, ofs_kmaj(k + 2)), sdesc_step(ka, ofs_kmaj(k + 3)), idesc_qk, k > 0, leader);
        mma_commit(&bars->s_full[t], leader);
      };
      // Half h of P V: keys [64h, 64h + 64).
      auto issue_pv = [&](int t, int u, int h) {
        const uint64_t va = sdesc_step(dV, (u % VS) * C::kTileBytes);
        const int k = h * 4;
        mma_ts_x4(tO[t], tP[t] + k * 8, tP[t] + (k + 1) * 8, tP[t] + (k + 2) * 8, tP[t] + (k + 3) * 8,
                  sdesc_step(va, k * 2048), sdesc_step(va, (k + 1) * 2048), sdesc_step(va, (k + 2) * 2048),
                  sdesc_step(va, (k + 3) * 2048), idesc_pv, (u > 0 || k > 0) ? 1u : 0u, leader);
      };
      bool ok = all(wait_bar(&bars->q_full, 0, w));
      if (ok && n > 0) ok = all(wait_bar(&bars->k_full[0], 0, w));
      if (ok && n > 0) {
        tc_fence_after();
#pragma unroll
        for (int t = 0; t < T; ++t)
          if (n_t[t] > 0) issue_s(t, 0);
        mma_commit(&bars->k_empty[0], leader);
      }
      for (int u = 0; ok && u < n; ++u) {
        const int s = u % VS;
        const uint32_t par = (u / VS) & 1;
        const int un = u + 1;
        if constexpr (SEP) {
          // S of the next key tile once the softmax has loaded this one.
          if (un < n) {
            if (!(ok = all(wait_bar(&bars->s_free, u & 1, w)) && all(wait_bar(&bars->k_full[un % KS], (un / KS) & 1, w))))
              break;
            tc_fence_after();
            issue_s(0, un);
            mma_commit(&bars->k_empty[un % KS], leader);
          }
        }
#pragma unroll
        for (int t = 0; t < T; ++t) {
          if (u >= n_t[t]) continue;
          const bool last_user = t == T - 1 || u >= n_t[T - 1];
          if (!(ok = all(wait_bar(&bars->p_ready[t][0], u & 1, w)) && all(wait_bar(&bars->v_full[s], par, w)))) break;
          tc_fence_after();
          issue_pv(t, u, 0);
          if (!(ok = all(wait_bar(&bars->p_ready[t][1], u & 1, w)))) break;
          tc_fence_after();
          issue_pv(t, u, 1);
          if constexpr (SEP) mma_commit(&bars->pv_done, leader);
          if (last_user) mma_commit(&bars->v_empty[s], leader);
          if (u == n_t[t] - 1) mma_commit(&bars->o_final[t], leader);
          if (!SEP && un < n_t[t]) {
            if (!(ok = all(wait_bar(&bars->k_full[un % KS], (un / KS) & 1, w)))) break;
            tc_fence_after();
            issue_s(t, un);
            if (t == T - 1 || un >= n_t[T - 1]) mma_commit(&bars->k_empty[un % KS], leader);
          }
        }
      }
      // All MMAs issued by this thread must finish before tensor memory is freed.
      mma_commit(&bars->drain, leader);
      all(drain_bar(&bars->drain, 0, w));
    }
  } else {
    if constexpr (T == 1) regs_inc<kSoftmaxRegs1>();
    // ------------------------------------------------------------- softmax
    const int t = warp >> 2;
    const int quad = warp & 3;
    const int rw = quad * 32 + lane;  // row of the tile: token rw / r, head rw % r
    const uint32_t lane_off = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t tS = tmem + lane_off + t * 128u;
    const uint32_t tPw = SEP ? tmem + lane_off + C::kColP : tS;
    const uint32_t tO = tmem + lane_off + C::kColO + t * D;
    const int nt = T == 2 && t == 1 ? n_t[1] : n_t[0];
    const int tok0 = T == 2 && t == 1 ? tok_t[1] : tok_t[0];
    const int tok = tok0 + rw / a.r;
    const bool mine = rw < a.TT * a.r && tok < n_tok;
    // Last visible key of this row, and of the tile's first.
    const int lim = a.causal ? min(off + tok, len - 1) : len - 1;
    const int lim0 = a.causal ? min(off + tok0, len - 1) : len - 1;
    const float sl2 = a.scale_log2;
    float m = -CUDART_INF_F;
    float l = 0.f;
    bool ok = true;
    for (int u = 0; u < nt; ++u) {
      ok = all(wait_bar(&bars->s_full[t], u & 1, w));
      if (!ok) break;
      tc_fence_after();
      uint32_t sr[kBN];
      if constexpr (T == 1)
        tmem_ld64x2(tS, sr);
      else
        tmem_ld128(tS, sr);
      if constexpr (SEP) {
        tc_fence_before();
        mbar_arrive(&bars->s_free);
      }
      const int k0 = (item.j0 + u) * kBN;
      if (k0 + kBN - 1 > lim0) {
#pragma unroll
        for (int i = 0; i < kBN; ++i)
          if (k0 + i > lim) sr[i] = __float_as_uint(-CUDART_INF_F);
      }
      // Row max as 8 independent partial maxima of three-input max.
      float pm[8];
#pragma unroll
      for (int x = 0; x < 8; ++x) pm[x] = fmaxf(__uint_as_float(sr[x]), __uint_as_float(sr[8 + x]));
#pragma unroll
      for (int i = 16; i < kBN; i += 16)
#pragma unroll
        for (int x = 0; x < 8; ++x)
          pm[x] = fmax3(pm[x], __uint_as_float(sr[i + x]), __uint_as_float(sr[i + 8 + x]));
      pm[0] = fmax3(pm[0], pm[1], pm[2]);
      pm[3] = fmax3(pm[3], pm[4], pm[5]);
      pm[6] = fmaxf(pm[6], pm[7]);
      const float m_cand = fmax3(pm[0], pm[3], pm[6]) * sl2;
      bool rescale = false;
      float alpha = 1.f;
      if (u == 0) {
        m = m_cand;  // -inf for a row that sees no key of this tile
      } else if (__any_sync(0xffffffffu, m_cand > m + a.rescale_tau)) {
        const float m_new = fmaxf(m, m_cand);
        alpha = m_new == -CUDART_INF_F ? 1.f : exp2_accurate(m - m_new);
        m = m_new;
        l *= alpha;
        rescale = true;
      }
      const float neg_m = m == -CUDART_INF_F ? 0.f : -m;
      if constexpr (SEP) {
        if (u > 0) {
          ok = all(wait_bar(&bars->pv_done, (u - 1) & 1, w));
          if (!ok) break;
          tc_fence_after();
        }
      }
      float ps[8];
#pragma unroll
      for (int x = 0; x < 8; ++x) ps[x] = 0.f;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int c = 2 * h; c < 2 * h + 2; ++c) {
          uint32_t pk[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float x0, x1;
            ffma2(x0, x1, __uint_as_float(sr[c * 32 + 2 * i]), __uint_as_float(sr[c * 32 + 2 * i + 1]), sl2, sl2,
                  neg_m, neg_m);
            // Shares of the FMA pipe as in fa_fwd.cu (2 of 32 at d = 128,
            // none at d = 64 causal).
            constexpr int kPoly = D == 128 ? 2 : 0;
            const float p0 = (2 * i < kPoly) ? exp2_poly(x0) : ex2(x0);
            const float p1 = (2 * i + 1 < kPoly) ? exp2_poly(x1) : ex2(x1);
            fadd2(ps[(2 * i) & 7], ps[(2 * i + 1) & 7], ps[(2 * i) & 7], ps[(2 * i + 1) & 7], p0, p1);
            // bf16: the type of V, which the weights meet in P V.
            pk[i] = pack_bf16x2(p0, p1);
          }
          tmem_st16(tPw + c * 16, pk);
        }
        if (h == 0 && rescale) {
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            uint32_t o32[32];
            tmem_ld32(tO + c * 32, o32);
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              float y0, y1;
              fmul2(y0, y1, __uint_as_float(o32[i]), __uint_as_float(o32[i + 1]), alpha, alpha);
              o32[i] = __float_as_uint(y0);
              o32[i + 1] = __float_as_uint(y1);
            }
            tmem_st32(tO + c * 32, o32);
          }
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&bars->p_ready[t][h]);
      }
      l += ((ps[0] + ps[1]) + (ps[2] + ps[3])) + ((ps[4] + ps[5]) + (ps[6] + ps[7]));
    }
    if (ok && nt > 0) ok = all(wait_bar(&bars->o_final[t], 0, w));
    if (ok) {
      tc_fence_after();
      const float inv_l = l == 0.f ? 0.f : 1.f / l;  // 0: no visible key (O is 0 there, or never written)
      const float L = l == 0.f ? -CUDART_INF_F : (m + lg2(l)) * 0.69314718055994530942f;
      const int slot = a.slots[item_no];
      const long long row = static_cast<long long>(tok_base) + tok;
      const int head = kvh * a.r + rw % a.r;
      // 64 columns of this row's O, normalised.
      auto load_o = [&](int x, uint32_t (&oo)[64]) {
        uint32_t(&o0)[32] = *reinterpret_cast<uint32_t(*)[32]>(&oo[0]);
        uint32_t(&o1)[32] = *reinterpret_cast<uint32_t(*)[32]>(&oo[32]);
        if (nt == 0) {
          // A part of the unit's keys that this tile's rows do not reach.
#pragma unroll
          for (int i = 0; i < 64; ++i) oo[i] = 0u;
          return;
        }
        tmem_ld32_nowait(tO + x * 64, o0);
        tmem_ld32_nowait(tO + x * 64 + 32, o1);
        tmem_ld_wait(o0);
        tmem_ld_tie(o1);
#pragma unroll
        for (int i = 0; i < 64; ++i) oo[i] = __float_as_uint(__uint_as_float(oo[i]) * inv_l);
      };
      // Eight columns as bf16, or their rounding residual.
      auto pack8 = [](const uint32_t* y, bool resid) {
        uint4 v;
        uint32_t* pv = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float x0 = __uint_as_float(y[2 * e]), x1 = __uint_as_float(y[2 * e + 1]);
          pv[e] = pack_bf16x2(x0, x1);
          if (resid) {
            const __nv_bfloat162 hi = *reinterpret_cast<const __nv_bfloat162*>(&pv[e]);
            pv[e] = pack_bf16x2(x0 - __low2float(hi), x1 - __high2float(hi));
          }
        }
        return v;
      };
      if (PAGED && slot >= 0) {
        const long long prow = (static_cast<long long>(slot) * a.Hkv + kvh) * (T * kBM) + t * kBM + rw;
#pragma unroll
        for (int x = 0; x < D / 64; ++x) {
          uint32_t oo[64];
          load_o(x, oo);
          if (mine) {
            uint4* dst = reinterpret_cast<uint4*>(a.part_o + prow * D + x * 64);
#pragma unroll
            for (int i = 0; i < 16; ++i) dst[i] = make_uint4(oo[4 * i], oo[4 * i + 1], oo[4 * i + 2], oo[4 * i + 3]);
          }
        }
        if (mine) a.part_l[prow] = L;
      } else {
        constexpr int kBoxesO = D / 64;
        const int jobs = kBoxesO * (a.resid.p ? 2 : 1);
        if (tok0 + a.TT <= n_tok) {
          // A whole tile: boxes staged in shared memory in the tensor map's
          // swizzle and stored by TMA, two at a time (as fa_fwd.cu).
          uint8_t* const slots[2] = {smem + C::kOffQ + (T == 1 ? 0 : t * C::kTileBytes),
                                     T == 1 ? smem + C::kOffStage : smem + C::kOffQ + t * C::kTileBytes + 16384};
          const bool issuer = rw == 0;
          for (int i = 0; i < jobs; ++i) {
            const int x = i % kBoxesO;
            const bool resid = i >= kBoxesO;
            uint8_t* st = slots[i % 2];
            if (i >= 2 && !(ok = all(wait_bar(&bars->epi_free[t], (i - 2) & 1, w)))) break;
            uint32_t oo[64];
            load_o(x, oo);
#pragma unroll
            for (int cc = 0; cc < 8; ++cc)
              *reinterpret_cast<uint4*>(st + rw * 128 + ((cc ^ (rw & 7)) << 4)) = pack8(oo + 8 * cc, resid);
            fence_proxy_async_smem();
            // A barrier for each box: a fast warp arrives for the second
            // before a slow one has for the first.
            mbar_arrive(&bars->epi_full[t][i & 1]);
            // (On a timeout every lane leaves at the next wait for epi_free.)
            if (issuer && (ok = wait_bar(&bars->epi_full[t][i & 1], (i >> 1) & 1, w))) {
              tma_store_4d(resid ? &tmR : &tmO, st, x * 64, 0, tok_base + tok0, kvh);
              bulk_commit();
              if (i + 1 < jobs && i + 1 >= 2) {
                bulk_wait_read<1>();
                mbar_arrive(&bars->epi_free[t]);
              }
            }
          }
          if (issuer) bulk_wait_read<0>();  // before the CTA exits
        } else if (tok0 < n_tok) {
          for (int i = 0; i < jobs; ++i) {
            const int x = i % kBoxesO;
            const bool resid = i >= kBoxesO;
            uint32_t oo[64];
            load_o(x, oo);
            if (mine) {
              const Rows& out = resid ? a.resid : a.o;
              uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(out.p) + row * out.ts + head * out.hs + x * 64);
#pragma unroll
              for (int cc = 0; cc < 8; ++cc) dst[cc] = pack8(oo + 8 * cc, resid);
            }
          }
        }
        if (mine) a.lse[static_cast<long long>(head) * a.total + row] = L;
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == C::kMmaWarp) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// Merges the parts of the units that were cut along their keys, one warp per
// row. Grid (KV heads, groups of four rows, units).
template <int D>
__global__ void __launch_bounds__(128) packed_merge_kernel(const PkArgs a) {
  pdl_wait();
  if (static_cast<int>(blockIdx.z) >= a.head->splits) return;
  constexpr int rows = PkCfg<D>::T * kBM;
  const PlanSplit sp = a.split_list[blockIdx.z];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rw = blockIdx.y * 4 + warp;
  const int t = rw / kBM, rt = rw % kBM;
  const int kvh = blockIdx.x;
  const int tok_base = a.cu ? a.cu[sp.seq] : sp.seq;
  const int n_tok = a.cu ? a.cu[sp.seq + 1] - tok_base : 1;
  const int tok = sp.tok0 + t * a.TT + rt / a.r;
  if (rt >= a.TT * a.r || tok >= n_tok) return;
  const int head = kvh * a.r + rt % a.r;
  const long long row = static_cast<long long>(tok_base) + tok;
  merge_row<D>(a.part_o, a.part_l, (static_cast<long long>(sp.slot0) * a.Hkv + kvh) * rows + rw,
               static_cast<long long>(a.Hkv) * rows, sp.parts,
               static_cast<__nv_bfloat16*>(a.o.p) + row * a.o.ts + head * a.o.hs,
               a.lse + static_cast<long long>(head) * a.total + row, lane);
}

struct Layout {
  PlanLayout plan;
  int TT, unit, max_splits;
  long long max_items, max_parts;  // parts: slots * KV heads
  size_t off_o, off_l, bytes;
};

Layout make_layout(const SeqShape& s, const CacheShape* c, int ctas) {
  Layout x;
  const int tiles = s.d == 128 ? 2 : 1;
  x.TT = kBM / s.r();
  x.unit = tiles * x.TT;
  const long long units = plan_max_units(s.S, s.T, x.unit);
  x.max_items = units;
  x.max_splits = 0;
  x.max_parts = 0;
  // Units are cut only where they are fewer than two per CTA (see plan_kernel).
  const long long least = (static_cast<long long>(s.T) + x.unit - 1) / x.unit;
  if (c && least * s.Hkv < 2LL * ctas) {
    const long long tiles_most = (static_cast<long long>(c->max_pages) * c->page + kBN - 1) / kBN;
    long long parts = units * s.Hkv * ((tiles_most + 3) / 4);
    if (parts > 4LL * ctas) parts = 4LL * ctas;
    x.max_parts = parts + s.Hkv;
    x.max_splits = 2 * ctas / s.Hkv + 1;
    if (x.max_splits > units) x.max_splits = static_cast<int>(units);
    x.max_items += 4LL * ctas / s.Hkv + 1;
  }
  x.plan = plan_layout(x.max_items, x.max_splits);
  x.off_o = x.plan.bytes;
  x.off_l = x.off_o + static_cast<size_t>(x.max_parts) * tiles * kBM * s.d * 4;
  x.bytes = x.off_l + static_cast<size_t>(x.max_parts) * tiles * kBM * 4;
  return x;
}

template <int D, bool PAGED>
cudaError_t launch_t(const SeqShape& s, const CacheShape* c, const Layout& x, const CUtensorMap& tq,
                     const CUtensorMap& tk, const CUtensorMap& tv, const CUtensorMap& to, const CUtensorMap& tr,
                     const Rows& o, const Rows& resid, float* lse, void* workspace, int sms, const LaunchCtl& ctl,
                     cudaStream_t stream) {
  using C = PkCfg<D>;
  auto kern = packed_fwd_kernel<D, PAGED>;
  static SmemOnce once;
  cudaError_t e = once.set(reinterpret_cast<const void*>(kern), C::kSmemBytes);
  if (e != cudaSuccess) return e;
  if constexpr (C::T == 1) {
    // The register split hands out exactly what a launch at 128 registers
    // per thread gives the CTA.
    static const int launch_regs = [&] {
      cudaFuncAttributes at{};
      return cudaFuncGetAttributes(&at, kern) == cudaSuccess ? at.numRegs : -1;
    }();
    if (launch_regs != 128) return cudaErrorLaunchOutOfResources;
  }
  uint8_t* ws = static_cast<uint8_t*>(workspace);
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
  p.split_ctas = x.max_parts > 0 ? sms : 0;
  p.sorted = x.max_items * s.Hkv > static_cast<long long>(C::kMinBlocks) * sms;
  p.head = reinterpret_cast<PlanHeader*>(ws + x.plan.head);
  p.items = reinterpret_cast<PlanItem*>(ws + x.plan.items);
  p.slots = reinterpret_cast<int*>(ws + x.plan.slots);
  p.split_list = reinterpret_cast<PlanSplit*>(ws + x.plan.splits);
  p.err = ctl.err;
  PkArgs a{};
  a.head = p.head;
  a.items = p.items;
  a.slots = p.slots;
  a.split_list = p.split_list;
  a.cu = s.cu;
  if (c) {
    a.lens = c->lens;
    a.table = c->table;
    a.table_stride = c->table_stride;
    a.n_pages = c->n_pages;
    a.page = c->page;
    a.pb = page_box(c->page);
  }
  a.o = o;
  a.resid = resid;
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
  a.ctl = ctl;
  const long long grid = x.max_items * s.Hkv;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  packed_plan_kernel<<<1, kPlanThreads, 0, stream>>>(p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  e = launch_dependent(kern, dim3(static_cast<unsigned>(grid)), C::kThreads, C::kSmemBytes, stream, tq, tk, tv, to, tr,
                       a);
  if (e != cudaSuccess || x.max_splits == 0) return e;
  return launch_dependent(packed_merge_kernel<D>, dim3(s.Hkv, C::T * kBM / 4, x.max_splits), 128, 0, stream, a);
}

}  // namespace

size_t packed_fwd_workspace_bytes(const SeqShape& s, const CacheShape* c, int ctas) {
  return make_layout(s, c, ctas).bytes;
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
  if (s.d == 64) return c ? launch_t<64, true>(FA_ARGS) : launch_t<64, false>(FA_ARGS);
  return c ? launch_t<128, true>(FA_ARGS) : launch_t<128, false>(FA_ARGS);
#undef FA_ARGS
}

}  // namespace fa
