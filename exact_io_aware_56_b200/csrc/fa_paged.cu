// Attention of a few new tokens per sequence over a paged KV cache
// (sm_100a): single-token decode, drafted tokens, short chunks. Sequence b
// has n_b new tokens, the last n_b of its len_b cached ones; its keys lie in
// the first len_b slots of the pages that its row of the block table names.
//
//   S_ij = scale q_i k_j for keys j <= len_b - n_b + i (causal) or j < len_b,
//   O_i = softmax(S_i) V,  L_i = log sum_j e^(S_ij);  no key: O_i = 0, L_i = -inf.
//
// Bound: the cache is read once for a handful of rows, so by HBM bandwidth
// (4 Hkv d len_b bytes per sequence). As in fa_decode.cu, every query head
// of a KV head shares its K/V stream, and the 128-key tiles of all (sequence,
// KV head) units, concatenated, are cut into equal contiguous runs, one per
// SM ("stream-K"): one wave, no tail, whatever the mix of lengths. A run's
// part of a unit is a segment; a second kernel merges a unit's segments by
// their logsumexp. The lengths live on the device, so that a captured graph
// can be replayed as sequences grow: every warp sums the sequences' tiles
// itself (32 sequences per step), which for tens of sequences costs less
// than a kernel before this one (measured: 3.5 us of 109 at 32 sequences).
//
// A tile's keys come by TMA, one box per page part (page_box() rows); page
// numbers are looked up by the producer warp's lanes in parallel. Slots
// behind len_b may hold anything, NaN included: their scores are replaced by
// -inf, and the V rows of a sequence's last tile are zeroed in shared memory
// before P V reads them (0 * NaN is NaN).
//
// Rows: slot rr of a unit is token rr / r, head rr % r of the group. They are
// replicated RHO times over the 128 tensor-memory lanes (RHO = 4 up to 32
// rows, 2 up to 64, else 1); copy c runs its own online softmax over key
// columns [c * 128/RHO, (c+1) * 128/RHO) of every tile, so that the
// exponentials spread over all four softmax warps; the copies are merged
// like segments.
//
// Warp roles (224 threads): 0-3 softmax, one thread per tensor-memory lane;
// 4 TMA producer; 5 tensor-memory owner and MMA issuer (warp-uniform loop,
// one elected lane issues); 6 zeroes the V rows behind a sequence's end.
// Tensor memory (512 columns): [0,256) S_0, S_1 | [256,384) P_0, P_1 |
// [384,...) O_0 (, O_1 at d = 64). The ordering argument is fa_decode.cu's:
// S_(j+1) is issued before P_j V_j, so a complete S_(j+1) means that the P
// buffer it pairs with is free; O is rescaled only after pv_done of the
// previous tile; p_ready is a barrier per tile parity, as a fast warp arrives
// for tile j + 1 before a slow one has for tile j.

#include <cuda_bf16.h>
#include <math_constants.h>

#include "fa_internal.h"
#include "fa_merge.cuh"
#include "sm100.cuh"

namespace fa {
namespace {

constexpr int kT = 128;  // keys per tile = tensor-memory lanes = row slots
constexpr int kThreads = 224;
constexpr int kProducer = 4;
constexpr int kMma = 5;
constexpr int kFixer = 6;
constexpr uint32_t kColS = 0;
constexpr uint32_t kColP = 256;
constexpr uint32_t kColO = 384;

template <int D>
struct Cfg {
  static constexpr int kStages = (D == 128) ? 3 : 6;
  static constexpr int kQBufs = (D == 128) ? 1 : 2;
  static constexpr int kOBufs = (kColO + 2 * D <= 512) ? 2 : 1;
  static constexpr int kBoxBytes = kT * 128;  // 128 rows x 64 bf16 columns
  static constexpr int kBoxes = D / 64;
  static constexpr int kTileBytes = kBoxBytes * kBoxes;
  static constexpr int kOffQ = 0;
  static constexpr int kOffK = kQBufs * kTileBytes;
  static constexpr int kOffV = kOffK + kStages * kTileBytes;
  static constexpr int kOffBar = kOffV + kStages * kTileBytes;
  static constexpr int kSmemBytes = kOffBar + 384 + 1024;  // + alignment slack
  static constexpr uint32_t kTmemCols = 512;
  static_assert(kSmemBytes <= 227 * 1024, "shared memory budget");
  static_assert(kSmemBytes > 114 * 1024, "one CTA per SM (owns all tensor memory)");
  static_assert(kColO + kOBufs * D <= kTmemCols, "tensor memory budget");
};

struct Args {
  float* part_o;        // [S * Hkv + G][RHO][rv][D] partial O / l
  float* part_l;        // [S * Hkv + G][RHO][rv] partial logsumexp (natural log, -inf: no key)
  long long* tile_pre;  // [S + 1] tiles of a unit of each sequence, summed (written for the merge)
  const int* cu;
  const int* lens;
  const int* table;
  long long table_stride, max_len;
  int S, T, max_q, Hkv, r, n_pages, page, pb, causal, rv, q_tokens;
  float scale_log2;
  LaunchCtl ctl;
};

struct Bars {
  uint64_t q_full[2], q_empty[2];
  uint64_t k_full[6], v_full[6], v_land[6], kv_empty[6];
  uint64_t s_full[2], p_ready[2], pv_done;
  uint64_t o_full[2], o_empty[2];
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
};
static_assert(sizeof(Bars) <= 384, "barrier block exceeds its shared-memory reservation");

// Runs: one per CTA, but none empty (the merge counts on it), and of few units
// over long caches none so short that merging a unit's partials takes longer
// than the tiles it saves: of T tiles a unit in runs of k the longest run takes
// 0.9 k us and the merge 0.06 rho T / k us (measured), least at
// k = sqrt(0.07 rho T). Five sequences of up to 7.5k
// keys, one KV head: 27.4 -> 20.6 us.
__device__ __forceinline__ int runs_of(long long W, int ctas, int rho, int units) {
  const int k = max(1, static_cast<int>(sqrtf(0.07f * rho * static_cast<float>(W) / units)));
  const long long runs = W / k;
  return runs < ctas ? (runs < 1 ? 1 : static_cast<int>(runs)) : ctas;
}
// First tile of run c of G; in 32 bits where they hold it (W G < 2^31).
__device__ __forceinline__ long long run_lo(int c, long long W, int G) {
  if (W <= (1 << 22)) return static_cast<unsigned>(c) * static_cast<unsigned>(W) / static_cast<unsigned>(G);
  return c * W / G;
}
// The run holding tile t: the largest c with run_lo(c) <= t.
__device__ __forceinline__ int run_of(long long t, long long W, int G) {
  if (W <= (1 << 22)) {
    const unsigned w = static_cast<unsigned>(W);
    return static_cast<int>(((static_cast<unsigned>(t) + 1) * G + w - 1) / w) - 1;
  }
  return static_cast<int>(((t + 1) * G + W - 1) / W) - 1;
}

// Tiles of a unit of sequence b: one at least where there are new tokens.
__device__ __forceinline__ int seq_tiles(const Args& a, int b, bool& bad) {
  const SeqRange s = seq_range(a.cu, a.lens, b, a.T, a.max_q, a.max_len);
  bad |= s.bad;
  return s.n > 0 ? max(1, (s.len + kT - 1) / kT) : 0;
}

// Walks the tiles of a run [lo, hi): sequence b, KV head kvh, tile j of the
// unit's T, segment e of the run.
struct Cursor {
  long long t, t_lo, t_hi;
  int b, kvh, j, T, e;
  __device__ __forceinline__ bool first() const { return t == t_lo || j == 0; }
  __device__ __forceinline__ bool last() const { return t == t_hi - 1 || j == T - 1; }
  __device__ __forceinline__ bool done() const { return t >= t_hi; }
  __device__ __forceinline__ void next(const Args& a) {
    ++t;
    if (++j == T) {
      j = 0;
      ++e;
      if (++kvh == a.Hkv) {
        kvh = 0;
        if (t < t_hi) {
          bool bad = false;
          do T = seq_tiles(a, ++b, bad);
          while (T == 0);  // ends: tile t < t_hi <= W lies in a later sequence
        }
      }
    }
  }
};

__device__ __forceinline__ long long warp_scan(long long x, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

// This CTA's run, by the whole warp. Lane i first sums the tiles of the i-th
// 32nd of the sequences; the 32nd that holds the run's first tile is then
// looked through 32 sequences at a time. W: all tiles; 0 (no work at all)
// where a length or an offset is out of range.
__device__ __forceinline__ Cursor first_tile(const Args& a, int rho, int lane, long long& W, bool& bad) {
  const int per = (a.S + 31) / 32;
  long long mine = 0;
  bad = false;
  for (int i = 0; i < per; ++i) {
    const int b = lane * per + i;
    if (b < a.S) mine += seq_tiles(a, b, bad);
  }
  bad = __any_sync(0xffffffffu, bad);
  const long long incl = warp_scan(mine, lane);
  W = bad ? 0 : __shfl_sync(0xffffffffu, incl, 31) * a.Hkv;
  const int G = runs_of(W, gridDim.x, rho, a.S * a.Hkv);
  Cursor c;
  c.t = c.t_lo = run_lo(min(static_cast<int>(blockIdx.x), G), W, G);
  c.t_hi = run_lo(min(static_cast<int>(blockIdx.x) + 1, G), W, G);
  c.b = c.kvh = c.j = c.e = 0;
  c.T = 1;
  if (c.done()) return c;
  // The first lane whose part ends behind the tile.
  const int part = __ffs(__ballot_sync(0xffffffffu, incl * a.Hkv > c.t)) - 1;
  long long before = __shfl_sync(0xffffffffu, incl - mine, part);
  for (int i0 = 0; i0 < per; i0 += 32) {
    const int b = part * per + i0 + lane;
    bool unused = false;
    const int tiles = i0 + lane < per && b < a.S ? seq_tiles(a, b, unused) : 0;
    const long long in = before + warp_scan(tiles, lane);
    const unsigned hit = __ballot_sync(0xffffffffu, in * a.Hkv > c.t);
    if (hit) {
      const int l = __ffs(hit) - 1;
      c.b = part * per + i0 + l;
      c.T = __shfl_sync(0xffffffffu, tiles, l);
      const long long in_seq = c.t - (__shfl_sync(0xffffffffu, in, l) - c.T) * a.Hkv;
      c.kvh = static_cast<int>(static_cast<unsigned long long>(in_seq) / static_cast<unsigned>(c.T));
      c.j = static_cast<int>(in_seq - static_cast<long long>(c.kvh) * c.T);
      break;
    }
    before = __shfl_sync(0xffffffffu, in, 31);
  }
  return c;
}

template <int D, int RHO>
__global__ void __launch_bounds__(kThreads, 1)
    paged_few_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, const Args a) {
  using C = Cfg<D>;
  constexpr int ST = C::kStages;
  constexpr int QB = C::kQBufs;
  constexpr int OB = C::kOBufs;
  constexpr int RB = kT / RHO;  // rows per copy
  constexpr int CW = kT / RHO;  // key columns per copy
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + ((1024u - (raw_addr & 1023u)) & 1023u);
  Bars* bars = reinterpret_cast<Bars*>(smem + C::kOffBar);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int b = 0; b < 2; ++b) {
      mbar_init(&bars->q_full[b], 1);
      mbar_init(&bars->q_empty[b], 1);
      mbar_init(&bars->o_full[b], 1);
      mbar_init(&bars->o_empty[b], kT);
      mbar_init(&bars->s_full[b], 1);
      mbar_init(&bars->p_ready[b], kT);
    }
    for (int s = 0; s < ST; ++s) {
      mbar_init(&bars->k_full[s], 1);
      mbar_init(&bars->v_full[s], 1);
      mbar_init(&bars->v_land[s], 1);
      mbar_init(&bars->kv_empty[s], 1);
    }
    mbar_init(&bars->pv_done, 1);
    mbar_init(&bars->drain, 1);
    bars->abort = 0;
    fence_mbar_init();
  }
  if (warp == kMma) {
    tmem_alloc(&bars->tmem_base, C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  const Watch w{&bars->abort, a.ctl.err, a.ctl.budget_ns};
  pdl_launch_dependents();  // the merge kernel may be scheduled; it waits for this grid's end

  long long W;
  bool bad;
  const Cursor start = first_tile(a, RHO, lane, W, bad);
  const long long t_lo = start.t_lo;
  auto all = [](bool b) { return __all_sync(0xffffffffu, b); };

  if (warp == kProducer) {
    // ------------------------------------------------------------ producer
    // All 32 lanes: lane i loads part i of the tile (a page or a part of one).
    if (lane == 0) {
      tma_prefetch_desc(&tmQ);
      tma_prefetch_desc(&tmK);
      tma_prefetch_desc(&tmV);
    }
    int len = 0, tok = 0, last_b = -1;
    int issued = 0, q_issued = 0;
    uint32_t tail_last = 0, land_par = 0;  // per stage: last use was a tail; parity of its next landing phase
    for (Cursor ta = start; !ta.done(); ta.next(a)) {
      if (ta.b != last_b) {
        last_b = ta.b;
        len = a.lens[ta.b];
        tok = a.cu ? a.cu[ta.b] : ta.b;
      }
      const int g = static_cast<int>(ta.t - t_lo);
      const int s = g % ST;
      const int keys = min(kT, len - ta.j * kT);  // <= 0: a sequence without keys
      const bool tail = keys < kT;
      const int parts = keys > 0 ? (keys + a.pb - 1) / a.pb : 0;
      int page_no = 0, slot = 0;
      if (lane < parts) {
        const int key = ta.j * kT + lane * a.pb;
        const int pi = key / a.page;
        slot = key - pi * a.page;
        page_no = a.table[static_cast<long long>(ta.b) * a.table_stride + pi];
        if (page_no < 0 || page_no >= a.n_pages) {
          // Past the tensor: the copy fills zeros.
          page_no = a.n_pages;
          atomicOr(a.ctl.err, kErrData);
        }
      }
      if (g >= ST && !all(wait_bar(&bars->kv_empty[s], (g / ST - 1) & 1, w))) break;
      const uint32_t bytes = static_cast<uint32_t>(parts) * a.pb * 128u * C::kBoxes;
      uint64_t* v_bar = tail ? &bars->v_land[s] : &bars->v_full[s];
      if (a.ctl.fault == 3) break;  // test hook: K_0 never arrives
      if (lane == 0) {
        mbar_arrive_expect_tx(&bars->k_full[s], bytes);
        mbar_arrive_expect_tx(v_bar, bytes);
      }
      __syncwarp();
      if (lane < parts) {
        uint8_t* dk = smem + C::kOffK + s * C::kTileBytes + lane * a.pb * 128;
        uint8_t* dv = smem + C::kOffV + s * C::kTileBytes + lane * a.pb * 128;
#pragma unroll
        for (int x = 0; x < C::kBoxes; ++x)
          tma_load_4d(&tmK, &bars->k_full[s], dk + x * C::kBoxBytes, x * 64, slot, ta.kvh, page_no);
#pragma unroll
        for (int x = 0; x < C::kBoxes; ++x)
          tma_load_4d(&tmV, v_bar, dv + x * C::kBoxBytes, x * 64, slot, ta.kvh, page_no);
      }
      tail_last = tail ? tail_last | (1u << s) : tail_last & ~(1u << s);
      if (tail) land_par ^= 1u << s;
      issued = g + 1;
      if (ta.first()) {
        // The segment's Q, after its first K/V tile is on its way.
        const int qb = ta.e % QB;
        if (ta.e >= QB && !all(wait_bar(&bars->q_empty[qb], (ta.e / QB - 1) & 1, w))) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(&bars->q_full[qb],
                                static_cast<uint32_t>(RHO * C::kBoxes) * a.q_tokens * a.r * 128u);
#pragma unroll
          for (int x = 0; x < C::kBoxes; ++x)
#pragma unroll
            for (int c = 0; c < RHO; ++c)
              tma_load_4d(&tmQ, &bars->q_full[qb],
                          smem + C::kOffQ + qb * C::kTileBytes + x * C::kBoxBytes + c * RB * 128, x * 64, 0, tok,
                          ta.kvh);
        }
        q_issued = ta.e + 1;
      }
    }
    // Every copy issued must land before the CTA may exit.
    for (int b = 0; b < QB; ++b)
      if (q_issued > b) drain_bar(&bars->q_full[b], ((q_issued - 1 - b) / QB) & 1, w);
    for (int s = 0; s < ST; ++s)
      if (issued > s) {
        const uint32_t par = ((issued - 1 - s) / ST) & 1;
        drain_bar(&bars->k_full[s], par, w);
        if ((tail_last >> s) & 1)
          drain_bar(&bars->v_land[s], ((land_par >> s) & 1) ^ 1, w);
        else
          drain_bar(&bars->v_full[s], par, w);
      }
  } else if (warp == kFixer) {
    // ------------------------------ V rows behind the sequence's last key
    if (blockIdx.x == 0) {
      // Also the merge's sums, and what there is to report.
      if (bad && lane == 0) atomicOr(a.ctl.err, kErrData);
      long long before = 0;
      for (int b0 = 0; b0 < a.S; b0 += 32) {
        bool unused = false;
        const long long x = before + warp_scan(b0 + lane < a.S && !bad ? seq_tiles(a, b0 + lane, unused) : 0, lane);
        if (b0 + lane < a.S) a.tile_pre[b0 + lane + 1] = x;
        before = __shfl_sync(0xffffffffu, x, 31);
      }
      if (lane == 0) a.tile_pre[0] = 0;
    }
    int len = 0, last_b = -1;
    uint32_t land_par = 0;
    // A tail may be the last of a long run, whose tiles take 1 to 2 us each.
    const Watch w_run{&bars->abort, a.ctl.err, a.ctl.budget_ns + static_cast<uint64_t>(start.t_hi - t_lo) * 20000};
    for (Cursor ta = start; !ta.done(); ta.next(a)) {
      if (ta.b != last_b) {
        last_b = ta.b;
        len = a.lens[ta.b];
      }
      const int keys = max(0, min(kT, len - ta.j * kT));
      if (keys == kT) continue;
      const int s = static_cast<int>(ta.t - t_lo) % ST;
      if (!all(wait_bar(&bars->v_land[s], (land_par >> s) & 1, w_run))) break;
      land_par ^= 1u << s;
      // A 128-byte row's 16-byte pieces stay within it under the swizzle.
#pragma unroll
      for (int x = 0; x < C::kBoxes; ++x) {
        uint4* box = reinterpret_cast<uint4*>(smem + C::kOffV + s * C::kTileBytes + x * C::kBoxBytes);
        for (int i = keys * 8 + lane; i < kT * 8; i += 32) box[i] = make_uint4(0, 0, 0, 0);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->v_full[s]);
    }
  } else if (warp == kMma) {
    // ----------------------------------------------------------- MMA issue
    const bool leader = elect_one();
    if (!start.done()) {
      constexpr uint32_t idesc_qk = idesc_bf16(kT, kT, false, false);
      constexpr uint32_t idesc_pv = idesc_bf16(kT, D, false, true);
      const uint64_t dQ = sdesc_sw128(smem_u32(smem + C::kOffQ), 16, 1024);
      const uint64_t dK = sdesc_sw128(smem_u32(smem + C::kOffK), 16, 1024);
      const uint64_t dV = sdesc_sw128(smem_u32(smem + C::kOffV), C::kBoxBytes, 1024);
      auto ofs_kmaj = [](int k) { return static_cast<uint32_t>((k / 4) * C::kBoxBytes + (k % 4) * 32); };
      // S_t = Q K_t^T into S buffer (t - t_lo) & 1.
      auto issue_s = [&](const Cursor& ta) -> bool {
        const int g = static_cast<int>(ta.t - t_lo);
        const int s = g % ST;
        const int qb = ta.e % QB;
        if (ta.first() && !all(wait_bar(&bars->q_full[qb], (ta.e / QB) & 1, w))) return false;
        if (!all(wait_bar(&bars->k_full[s], (g / ST) & 1, w))) return false;
        tc_fence_after();
        const uint64_t qa = sdesc_step(dQ, qb * C::kTileBytes);
        const uint64_t ka = sdesc_step(dK, s * C::kTileBytes);
        const uint32_t d_s = tmem + kColS + (g & 1) * kT;
#pragma unroll
        for (int k = 0; k < D / 16; k += 4)
          mma_ss_x4(d_s, sdesc_step(qa, ofs_kmaj(k)), sdesc_step(qa, ofs_kmaj(k + 1)), sdesc_step(qa, ofs_kmaj(k + 2)),
                    sdesc_step(qa, ofs_kmaj(k + 3)), sdesc_step(ka, ofs_kmaj(k)), sdesc_step(ka, ofs_kmaj(k + 1)),
                    sdesc_step(ka, ofs_kmaj(k + 2)), sdesc_step(ka, ofs_kmaj(k + 3)), idesc_qk, k > 0, leader);
        mma_commit(&bars->s_full[g & 1], leader);
        if (ta.last()) mma_commit(&bars->q_empty[qb], leader);  // the segment's last read of its Q buffer
        return true;
      };
      // O += P_t V_t.
      auto issue_pv = [&](const Cursor& ta) -> bool {
        const int g = static_cast<int>(ta.t - t_lo);
        const int s = g % ST;
        const int ob = ta.e % OB;
        if (!all(wait_bar(&bars->p_ready[g & 1], (g >> 1) & 1, w)) || !all(wait_bar(&bars->v_full[s], (g / ST) & 1, w))) return false;
        const bool first = ta.first();
        if (first && ta.e >= OB && !all(wait_bar(&bars->o_empty[ob], ((ta.e / OB) - 1) & 1, w))) return false;
        tc_fence_after();
        const uint64_t va = sdesc_step(dV, s * C::kTileBytes);
        const uint32_t d_o = tmem + kColO + ob * D;
        const uint32_t a_p = tmem + kColP + (g & 1) * 64;
#pragma unroll
        for (int k = 0; k < kT / 16; k += 4)
          mma_ts_x4(d_o, a_p + k * 8, a_p + (k + 1) * 8, a_p + (k + 2) * 8, a_p + (k + 3) * 8,
                    sdesc_step(va, k * 2048), sdesc_step(va, (k + 1) * 2048), sdesc_step(va, (k + 2) * 2048),
                    sdesc_step(va, (k + 3) * 2048), idesc_pv, (!first || k > 0) ? 1u : 0u, leader);
        mma_commit(&bars->kv_empty[s], leader);
        mma_commit(&bars->pv_done, leader);
        if (ta.last()) mma_commit(&bars->o_full[ob], leader);
        return true;
      };
      Cursor cur = start, nxt = start;
      bool ok = issue_s(nxt);
      for (nxt.next(a); ok && !cur.done(); cur.next(a), nxt.next(a)) {
        const bool more = !nxt.done();
        // With one Q buffer the next segment's Q lands only after this
        // segment's last S: hand P_t V_t to the tensor pipe before waiting.
        if (QB == 1 && more && nxt.first()) {
          ok = issue_pv(cur) && issue_s(nxt);
        } else {
          ok = (!more || issue_s(nxt)) && issue_pv(cur);
        }
      }
      // All MMAs issued by this thread must finish before tensor memory is freed.
      mma_commit(&bars->drain, leader);
      all(drain_bar(&bars->drain, 0, w));
    }
  } else {
    // ------------------------------------------------------------- softmax
    const int slot = warp * 32 + lane;  // tensor-memory lane = row slot
    const int cp = slot / RB;           // copy: key columns [cp*CW, cp*CW + CW) of each tile
    const int rr = slot - cp * RB;      // row of the unit
    const int row_tok = rr / a.r;
    const uint32_t lane_off = static_cast<uint32_t>(warp * 32) << 16;
    const float sl2 = a.scale_log2;
    if (RHO > 1) {
      // P columns of the other copies stay zero for the whole kernel.
      uint32_t z[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) z[i] = 0u;
#pragma unroll
      for (int c = 0; c < 8; ++c) tmem_st16(tmem + lane_off + kColP + c * 16, z);
      tmem_st_wait();
    }
    float m = -CUDART_INF_F;
    float l = 0.f;
    int lim = 0, last_b = -1;  // last visible key
    bool valid = false;
    for (Cursor ta = start; !ta.done(); ta.next(a)) {
      const int g = static_cast<int>(ta.t - t_lo);
      const bool first = ta.first();
      const int ob = ta.e % OB;
      const uint32_t tS = tmem + lane_off + kColS + (g & 1) * kT;
      const uint32_t tP = tmem + lane_off + kColP + (g & 1) * 64;
      const uint32_t tO = tmem + lane_off + kColO + ob * D;
      if (ta.b != last_b) {
        last_b = ta.b;
        const int n = a.cu ? a.cu[ta.b + 1] - a.cu[ta.b] : 1;
        const int len = a.lens[ta.b];
        valid = row_tok < n;
        lim = a.causal ? min(len - n + row_tok, len - 1) : len - 1;
      }
      if (first) {
        m = -CUDART_INF_F;
        l = 0.f;
      }
      if (!all(wait_bar(&bars->s_full[g & 1], (g >> 1) & 1, w))) break;
      tc_fence_after();
      uint32_t sr[CW];
      if constexpr (CW == 128) {
        tmem_ld128(tS, sr);
      } else {
#pragma unroll
        for (int c = 0; c < CW / 32; ++c) {
          uint32_t t32[32];
          tmem_ld32(tS + cp * CW + c * 32, t32);
#pragma unroll
          for (int i = 0; i < 32; ++i) sr[c * 32 + i] = t32[i];
        }
      }
      const int k0 = ta.j * kT + cp * CW;
      if (k0 + CW - 1 > lim) {
#pragma unroll
        for (int i = 0; i < CW; ++i)
          if (k0 + i > lim) sr[i] = __float_as_uint(-CUDART_INF_F);
      }
      float pm[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) pm[u] = fmaxf(__uint_as_float(sr[u]), __uint_as_float(sr[8 + u]));
#pragma unroll
      for (int i = 16; i < CW; i += 16)
#pragma unroll
        for (int u = 0; u < 8; ++u)
          pm[u] = fmax3(pm[u], __uint_as_float(sr[i + u]), __uint_as_float(sr[i + 8 + u]));
      pm[0] = fmax3(pm[0], pm[1], pm[2]);
      pm[3] = fmax3(pm[3], pm[4], pm[5]);
      pm[6] = fmaxf(pm[6], pm[7]);
      const float m_cand = fmax3(pm[0], pm[3], pm[6]) * sl2;
      bool rescale = false;
      float alpha = 1.f;
      if (first) {
        m = m_cand;
      } else if (__any_sync(0xffffffffu, m_cand > m)) {
        const float m_new = fmaxf(m, m_cand);
        alpha = (m_new == -CUDART_INF_F) ? 1.f : ex2(m - m_new);
        m = m_new;
        l *= alpha;
        rescale = true;
      }
      // A row with no visible key so far keeps m = -inf; its masked
      // scores must give exp(-inf) = 0, not exp(-inf + inf).
      const float neg_m = (m == -CUDART_INF_F) ? 0.f : -m;
      float ps[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) ps[u] = 0.f;
#pragma unroll
      for (int c = 0; c < CW / 32; ++c) {
        uint32_t pk[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          // Exponent arguments and partial sums two at a time (packed f32x2).
          float x0, x1;
          ffma2(x0, x1, __uint_as_float(sr[c * 32 + 2 * i]), __uint_as_float(sr[c * 32 + 2 * i + 1]), sl2, sl2,
                neg_m, neg_m);
          const float p0 = ex2(x0);
          const float p1 = ex2(x1);
          fadd2(ps[(2 * i) & 7], ps[(2 * i + 1) & 7], ps[(2 * i) & 7], ps[(2 * i + 1) & 7], p0, p1);
          // bf16: the type of V, which the weights meet in P V.
          pk[i] = pack_bf16x2(p0, p1);
        }
        tmem_st16(tP + cp * (CW / 2) + c * 16, pk);
      }
      const float sum = ((ps[0] + ps[1]) + (ps[2] + ps[3])) + ((ps[4] + ps[5]) + (ps[6] + ps[7]));
      if (rescale) {
        // O may still be receiving the previous tile's product.
        if (!all(wait_bar(&bars->pv_done, (g - 1) & 1, w))) break;
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o32[32];
          tmem_ld32(tO + c * 32, o32);
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            float x0, x1;
            fmul2(x0, x1, __uint_as_float(o32[i]), __uint_as_float(o32[i + 1]), alpha, alpha);
            o32[i] = __float_as_uint(x0);
            o32[i + 1] = __float_as_uint(x1);
          }
          tmem_st32(tO + c * 32, o32);
        }
      }
      l += sum;
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(&bars->p_ready[g & 1]);
      if (ta.last()) {
        if (!all(wait_bar(&bars->o_full[ob], (ta.e / OB) & 1, w))) break;
        tc_fence_after();
        // Partial of this copy: O / l and logsumexp, or zeros and -inf when
        // no key of the segment is visible to the row. Unit + run numbers the
        // segments without gaps in either: from one segment to the next, the
        // unit or the run (or both) grow by one.
        const long long part = static_cast<long long>(ta.b) * a.Hkv + ta.kvh + blockIdx.x;
        const long long prow = (part * RHO + cp) * a.rv + rr;
        const float inv_l = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t oo[32];
          tmem_ld32(tO + c * 32, oo);
          if (valid) {
            float4* dst = reinterpret_cast<float4*>(a.part_o + prow * D + c * 32);
#pragma unroll
            for (int i = 0; i < 8; ++i)
              dst[i] = make_float4(__uint_as_float(oo[4 * i]) * inv_l, __uint_as_float(oo[4 * i + 1]) * inv_l,
                                   __uint_as_float(oo[4 * i + 2]) * inv_l, __uint_as_float(oo[4 * i + 3]) * inv_l);
          }
        }
        if (valid) a.part_l[prow] = l == 0.f ? -CUDART_INF_F : (m + lg2(l)) * 0.69314718055994530942f;
        tc_fence_before();
        mbar_arrive(&bars->o_empty[ob]);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMma) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// Merges the partials of a unit's rows (every copy of every segment), one
// warp per row; grid (S * Hkv, groups of four rows).
template <int D>
__global__ void __launch_bounds__(128)
    paged_few_merge_kernel(const Args a, int ctas, int rho, Rows o, float* __restrict__ lse) {
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int b = blockIdx.x / a.Hkv;
  const int kvh = blockIdx.x - b * a.Hkv;
  const int rr = blockIdx.y * 4 + warp;
  const int tok0 = a.cu ? a.cu[b] : b;
  const int n = a.cu ? a.cu[b + 1] - tok0 : 1;
  pdl_wait();
  const long long pre = a.tile_pre[b];
  const int Tb = static_cast<int>(a.tile_pre[b + 1] - pre);
  const long long W = a.tile_pre[a.S] * a.Hkv;
  if (Tb == 0 || rr >= n * a.r) return;
  const int G = runs_of(W, ctas, rho, a.S * a.Hkv);
  const long long first = pre * a.Hkv + static_cast<long long>(kvh) * Tb;
  const int c0 = run_of(first, W, G);
  const int n_parts = (run_of(first + Tb - 1, W, G) - c0 + 1) * rho;
  // Partial p = (run c0 + p / rho, copy p % rho).
  const long long row0 = (static_cast<long long>(blockIdx.x) + c0) * rho * a.rv + rr;
  const int tok = tok0 + rr / a.r;
  const int h = kvh * a.r + rr % a.r;
  merge_row<D>(a.part_o, a.part_l, row0, a.rv, n_parts, static_cast<__nv_bfloat16*>(o.p) + tok * o.ts + h * o.hs,
               lse + static_cast<long long>(h) * a.T + tok, lane);
}

struct Plan {
  int rho, rv, q_tokens, G;
  size_t off_l, off_pre, bytes;
};

Plan make_plan(const SeqShape& s, const CacheShape& c, int ctas) {
  Plan p;
  const int rows = s.r() * c.max_q;
  p.rho = rows <= 32 ? 4 : (rows <= 64 ? 2 : 1);
  p.rv = rows;
  p.q_tokens = (kT / p.rho) / s.r();
  if (p.q_tokens > c.max_q) p.q_tokens = c.max_q;
  // No more runs than there can be tiles.
  const long long tiles = static_cast<long long>(s.S) * s.Hkv *
                          ((static_cast<long long>(c.max_pages) * c.page + kT - 1) / kT);
  p.G = tiles < ctas ? static_cast<int>(tiles < 1 ? 1 : tiles) : ctas;
  const size_t parts = (static_cast<size_t>(s.S) * s.Hkv + ctas) * p.rho * p.rv;
  p.off_l = parts * s.d * 4;
  p.off_pre = (p.off_l + parts * 4 + 15) / 16 * 16;
  p.bytes = p.off_pre + (static_cast<size_t>(s.S) + 1) * 8;
  return p;
}

template <int D, int RHO>
cudaError_t launch_t(const SeqShape& s, const CacheShape& c, const Plan& p, const CUtensorMap& tq,
                     const CUtensorMap& tk, const CUtensorMap& tv, const Rows& o, float* lse, void* workspace,
                     const LaunchCtl& ctl, cudaStream_t stream) {
  using C = Cfg<D>;
  auto kern = paged_few_kernel<D, RHO>;
  static SmemOnce once;
  cudaError_t e = once.set(reinterpret_cast<const void*>(kern), C::kSmemBytes);
  if (e != cudaSuccess) return e;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  Args a;
  a.part_o = reinterpret_cast<float*>(ws);
  a.part_l = reinterpret_cast<float*>(ws + p.off_l);
  a.tile_pre = reinterpret_cast<long long*>(ws + p.off_pre);
  a.cu = s.cu;
  a.lens = c.lens;
  a.table = c.table;
  a.table_stride = c.table_stride;
  a.max_len = static_cast<long long>(c.max_pages) * c.page;
  a.S = s.S;
  a.T = s.T;
  a.max_q = c.max_q;
  a.Hkv = s.Hkv;
  a.r = s.r();
  a.n_pages = c.n_pages;
  a.page = c.page;
  a.pb = page_box(c.page);
  a.causal = s.causal;
  a.rv = p.rv;
  a.q_tokens = p.q_tokens;
  a.scale_log2 = s.scale * 1.4426950408889634f;
  a.ctl = ctl;
  kern<<<p.G, kThreads, C::kSmemBytes, stream>>>(tq, tk, tv, a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  return launch_dependent(paged_few_merge_kernel<D>, dim3(s.S * s.Hkv, (p.rv + 3) / 4), 128, 0, stream, a, p.G, RHO,
                          o, lse);
}

}  // namespace

size_t paged_few_workspace_bytes(const SeqShape& s, const CacheShape& c, int ctas) {
  return make_plan(s, c, ctas).bytes;
}

cudaError_t launch_paged_few(const SeqShape& s, const CacheShape& c, const Rows& q, const Rows& o, const Pages& k,
                             const Pages& v, float* lse, void* workspace, int sms, const LaunchCtl& ctl,
                             cudaStream_t stream) {
  const Plan p = make_plan(s, c, sms);
  CUtensorMap tq, tk, tv;
  const int pb = page_box(c.page);
  if (!encode_group_map(&tq, q, s.T, s.Hkv, s.r(), s.d, p.q_tokens) ||
      !encode_pages_map(&tk, k, c.n_pages, s.Hkv, c.page, s.d, pb) ||
      !encode_pages_map(&tv, v, c.n_pages, s.Hkv, c.page, s.d, pb))
    return cudaErrorInvalidValue;
#define FA_ARGS s, c, p, tq, tk, tv, o, lse, workspace, ctl, stream
  if (s.d == 64) {
    if (p.rho == 4) return launch_t<64, 4>(FA_ARGS);
    if (p.rho == 2) return launch_t<64, 2>(FA_ARGS);
    return launch_t<64, 1>(FA_ARGS);
  }
  if (p.rho == 4) return launch_t<128, 4>(FA_ARGS);
  if (p.rho == 2) return launch_t<128, 2>(FA_ARGS);
  return launch_t<128, 1>(FA_ARGS);
#undef FA_ARGS
}

}  // namespace fa
