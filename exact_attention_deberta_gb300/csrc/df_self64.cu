// Causal attention with a window and sinks, forward, head sizes to 64, where there is more work
// than a round of the SMs (df_cross64.cu's SELF form has clusters for less), on tcgen05 (bf16 / fp16
// I/O, fp32 accumulation and softmax).
//
//   s_ij = scale q_i.k_j,  o_i = sum_j exp(s_ij - lse_i) v_j  over the keys j that i sees
//   (df_cross.cuh); a row that sees none gets zeros and lse = -inf.
//
// A window's query tile meets some ten key tiles, so that its end counts: where both softmax
// warpgroups take turns at one query tile and join their sums, it takes as long as eight key tiles.
// Here an item is two query tiles that follow one another, one for each warpgroup: each key tile is
// loaded once for both, a warpgroup ends its tile by itself, and its ends lie beside the other's
// tiles, since it may run two key tiles ahead.  A key tile that only one of them sees is a step of
// that one alone.
//   warp 0      finds the items, loads both Q tiles (two buffers), K and V by TMA;
//   warp 1      issues S = Q.K^T, key tile by key tile, first for warpgroup 0, then 1;
//   warps 3, 2  issue O_w += P.V for warpgroup 0 and 1 (a V tile is free when both have), and zero
//               the rows of V whose keys do not count first;
//   warps 4-11  softmax: one thread per row, P (rounded to the I/O type) written over its S.
// Three score buffers rotate over the steps of both.
//
// Keys that a row does not see: the scores of a tile that not every row sees whole become -inf in
// registers, in code of its own (in place in tensor memory, as the whole tile's code is shorter then:
// 546 us against 481 with a window of 1024; by a minimum with infinities, a block for each end of the
// window: 523), by bits that are found before the scores are awaited (481 -> 461; 549 -> 514 with 4 sinks).
// The loop's length in instructions and what its warps spill decide here: a split of 224 and 56
// registers, which spills, took 506 us where this one took 483.
//
// Measured (GB300, bf16): 16 x 12 heads, 8192 tokens, a window of 1024: 460 us, 841 TFLOP/s of what is
// seen, with 4 sinks 511 to 519 (one query tile an item: 658 and 729); 4 x 12 heads, 8192 tokens, no window:
// 356 us, 1160 TFLOP/s (412); 64 x 12 heads of 512: 61 us (96).  A step, a key tile for one warpgroup, takes
// it some 2000 cycles, of which softmax is 1560 and 260 are a wait for its scores; an item's end takes
// 2400, its beginning 1200 (stamps of the SM clock, before the last change).
#include "df_cross_fwd.cuh"

namespace dfa {

namespace {

using namespace ptx;

constexpr int kThreads = 384;
constexpr int kRegs = 168;  // launched; after the split eight softmax warps have 216, four others 72
static_assert(256 * 216 + 128 * 72 <= kThreads * kRegs, "setmaxnreg.inc must not wait");
constexpr uint32_t kItemRing = 4;

struct PairSmem {
  static constexpr int D = 64;
  static constexpr int kStages = 4;                                 // K tiles, and V tiles, in flight
  static constexpr uint32_t kTileBytes = kBoxBytes;
  static constexpr uint32_t q = 0;                                  // [2 buffers][2 warpgroups][Q tile]
  static constexpr uint32_t k = q + 4 * kTileBytes;                 // [kStages][K tile]
  static constexpr uint32_t v = k + kStages * kTileBytes;           // [kStages][V tile]
  static constexpr uint32_t rows = v + kStages * kTileBytes;        // [8 softmax warps] on their way out
  static constexpr uint32_t bars = rows + 8 * kRowStage;
  // q_full, q_empty [2]; k_full, k_empty, v_full, v_empty [kStages]; buf_free, drain [3];
  // s_full, p_full, pv_done [2][4]; item_full, item_empty; claim
  static constexpr int kBars = 4 + 4 * kStages + 6 + 24 + 2 * (int)kItemRing + 1;
  static constexpr uint32_t ring = (bars + kBars * 8 + 15) & ~15u;  // CrossItem slots of 32 bytes
  static constexpr uint32_t cur = ring + 32 * kItemRing;            // [2 warpgroups][2] current items
  static constexpr uint32_t claim = cur + 128;                      // 16 bytes
  static constexpr uint32_t misc = claim + 16;                      // abort flag, tmem slot
  static constexpr uint32_t bytes = misc + 16;
  static constexpr uint32_t alloc = bytes + 1024;
  static_assert(alloc <= 232448, "shared memory of one CTA");
};

// The key tiles of an item, `n` of both query tiles together: the first warpgroup sees the first
// `na`, the second all but `skip` from `from` on (none where it has no rows).
struct PairTiles {
  CrossBand band;
  int n, na, from;
  unsigned skip;
  __device__ __forceinline__ bool sees(int w, int t) const {
    return w == 0 ? t < na : (unsigned)(t - from) >= skip;
  }
};
__device__ __forceinline__ PairTiles pair_tiles(const CrossArgs& a, const CrossItem& it) {
  PairTiles p;
  p.band = key_band(a, it);
  p.n = band_tiles(p.band, it.no);
  CrossItem part = it;
  part.nr = min(it.nr, a.tpt);
  clip_causal(part);
  p.na = min(p.n, band_tiles(p.band, part.no));
  part.no = it.no;
  part.p0 = it.p0 + a.tpt;
  const bool second = it.nr > a.tpt;
  p.from = second ? p.band.sinks : 0;
  p.skip = second ? (unsigned)(key_band(a, part).skip - p.band.skip) : UINT_MAX;
  return p;
}

// LO: what the rounding of the results drops is asked for too.
template <bool BF16, bool LO>
__global__ void __launch_bounds__(kThreads, 1) self64_kernel(const FwdArgs args, const __grid_constant__ FwdMaps maps) {
  using SL = PairSmem;
  constexpr int D = SL::D;
  constexpr uint32_t R = SL::kStages;
  constexpr uint32_t kIdescQK = idesc_f16(128, 128, BF16 ? 1 : 0, 0, 0);
  constexpr uint32_t kIdescPV = idesc_f16(128, D, BF16 ? 1 : 0, 0, 1);
  using T = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
  // tensor-memory columns: three score buffers (step g of the CTA uses g % 3), two O
  static_assert(tmem_region_fits(384, 2u * D, 512), "scores and two O accumulators in 512 columns");
  constexpr uint32_t kItemReaders = 5;  // three issuing warps, a reader of each softmax warpgroup

  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t* sQ = sm + SL::q;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + SL::bars);
  uint64_t* q_full = bars;
  uint64_t* q_empty = bars + 2;
  uint64_t* k_full = bars + 4;
  uint64_t* k_empty = k_full + R;
  uint64_t* v_full = k_empty + R;
  uint64_t* v_empty = v_full + R;      // both P.V warps
  uint64_t* buf_free = v_empty + R;    // [3] the P.V that read the buffer is done
  uint64_t* drain = buf_free + 3;      // [3], one per issuing warp
  // [wg][n & 3]: S of the n-th step of wg computed; its four warps stored P of it; P.V of it done.
  // (By its own steps, not by buffers: a warpgroup without rows in some items is far ahead of the
  // other's steps.)  A warp may be through with steps n + 1 and n + 2 before a sibling has stored
  // n, but not with n + 3: its scores wait for a buffer that P.V of n, or of a step behind it, frees.
  uint64_t* s_full = drain + 3;
  uint64_t* p_full = s_full + 8;
  uint64_t* pv_done = p_full + 8;
  uint64_t* item_full = pv_done + 8;
  uint64_t* item_empty = item_full + kItemRing;
  uint64_t* claim_bar = item_empty + kItemRing;
  auto ring_slot = [&](uint32_t c) { return reinterpret_cast<CrossItem*>(sm + SL::ring + 32 * (c % kItemRing)); };
  volatile int* s_abort = reinterpret_cast<volatile int*>(sm + SL::misc);
  uint32_t* tslot = reinterpret_cast<uint32_t*>(sm + SL::misc + 4);

  const CrossArgs& a = args.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int b = 0; b < 2; ++b) {
      mbar_init(q_full + b, 1);
      mbar_init(q_empty + b, 1);
    }
    for (uint32_t s = 0; s < R; ++s) {
      mbar_init(k_full + s, 1);
      mbar_init(k_empty + s, 1);
      mbar_init(v_full + s, 1);
      mbar_init(v_empty + s, 2);
    }
    for (int b = 0; b < 3; ++b) {
      mbar_init(buf_free + b, 1);
      mbar_init(drain + b, 1);
    }
    for (int b = 0; b < 8; ++b) {
      mbar_init(s_full + b, 1);
      mbar_init(p_full + b, 4);
      mbar_init(pv_done + b, 1);
    }
    for (uint32_t b = 0; b < kItemRing; ++b) {
      mbar_init(item_full + b, 1);
      mbar_init(item_empty + b, kItemReaders);
    }
    mbar_init(claim_bar, 1);
    *s_abort = 0;
    mbar_fence_init();
    tma_prefetch_desc(&maps.q);
    tma_prefetch_desc(&maps.k);
    tma_prefetch_desc(&maps.v);
  }
  if (warp == 1) {
    tmem_alloc(tslot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;
  auto tS = [&](int b) { return tmem + 128u * b; };
  auto tO = [&](int b) { return tmem + 384u + (uint32_t)D * b; };

  const unsigned long long budget = a.budget;
  // the c-th item handed out, for one thread; hk = -1 at the end or after an abort
  auto read_item = [&](uint32_t c) {
    const uint32_t slot = c % kItemRing;
    CrossItem it;
    it.r0 = it.nr = it.o0 = it.no = it.b = it.p0 = it.q0 = 0;
    it.hk = -1;
    if (cross_wait(item_full + slot, (c / kItemRing) & 1, budget, s_abort)) {
      it = *ring_slot(c);
      mbar_arrive(item_empty + slot);
    }
    return it;
  };

  if (warp == 0) {
    // ------------------------------------------------------------ items and loads
    setmaxnreg_dec<72>();
    // (the whole warp runs every step, and one lane of it issues)
    TileWalk<true> walk;
    walk.together = heads_together(a);
    TileClaim claim = {claim_bar, reinterpret_cast<uint4*>(sm + SL::claim)};
    uint32_t g = 0, qc = 0, k_issued = 0, v_issued = 0;
    int mask_b = -1, mask_n = 0;  // the last masked row measured
    bool ok = true;               // a wait ran out: nothing is loaded after it
    long long number = blockIdx.x;
    // K or V rows [row, row + 128) into stage s
    auto load = [&](const CUtensorMap* map, uint32_t tiles, uint64_t* full, uint64_t* empty, uint32_t gs, int head, int row,
                    uint32_t& issued) {
      const uint32_t s = gs % R;
      ok = ok && cross_wait(empty + s, ((gs / R) & 1) ^ 1, budget, s_abort);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) return;
      if (elect_one()) {
        mbar_expect_tx(full + s, SL::kTileBytes);
        tma_load_3d(sm + tiles + s * SL::kTileBytes, map, 0, head, row, full + s);
      }
      __syncwarp();
      issued = gs + 1;
    };
    for (uint32_t c = 0;; ++c) {
      CrossItem it = walk.find(a, query_side(a), key_side(a), 2 * a.tpt, number);
      const uint32_t slot = c % kItemRing;
      if (a.key_mask && it.hk >= 0) {  // key tiles behind the last valid key are not visited
        if (it.b != mask_b) mask_n = masked_length(a.key_mask + (size_t)it.b * a.Lk, it.no);
        mask_b = it.b;
        it.no = mask_n;
      }
      clip_causal(it);
      bool room = true;
      if (c >= kItemRing) room = cross_wait(item_empty + slot, ((c / kItemRing) - 1) & 1, budget, s_abort);
      if (__any_sync(0xffffffffu, *s_abort || !room)) it.hk = -1;
      if (lane == 0 && room) {
        *ring_slot(c) = it;
        mbar_arrive(item_full + slot);
      }
      if (it.hk < 0) break;
      const CrossBand band = key_band(a, it);
      const int nt = band_tiles(band, it.no);
      if (nt > 0) {
        const uint32_t qb = qc & 1;
        ok = ok && cross_wait(q_empty + qb, ((qc >> 1) & 1) ^ 1, budget, s_abort);
        ok = __all_sync(0xffffffffu, ok);
        if (ok) {
          if (elect_one()) {
            const bool second = it.nr > a.tpt;
            const uint32_t box = (uint32_t)(a.G * a.tpt) * 128u;
            mbar_expect_tx(q_full + qb, second ? 2 * box : box);
            tma_load_3d(sQ + 2 * qb * SL::kTileBytes, &maps.q, 0, it.hk * a.G, it.r0, q_full + qb);
            if (second)
              tma_load_3d(sQ + (2 * qb + 1) * SL::kTileBytes, &maps.q, 0, it.hk * a.G, it.r0 + a.tpt, q_full + qb);
          }
          __syncwarp();
          ++qc;
        }
      }
      // K(t) goes out before V(t - 1): the next scores must not wait until P.V has
      // freed a V tile.  The next item is asked for two tiles before this one's end.
      const int ask_at = max(0, nt - 2);
      auto row_at = [&](int t) { return it.o0 + band.tile(t) * 128; };
#pragma unroll 1
      for (int t = 0; t <= nt; ++t) {
        if (t == ask_at) claim.ask();
        if (t < nt) load(&maps.k, SL::k, k_full, k_empty, g + t, it.hk, row_at(t), k_issued);
        if (t > 0) load(&maps.v, SL::v, v_full, v_empty, g + t - 1, it.hk, row_at(t - 1), v_issued);
      }
      g += nt;
      number = claim.answer(budget, s_abort);
    }
    // no copy may still be landing when the CTA leaves
    if (elect_one()) {
#pragma unroll 1
      for (uint32_t n = k_issued > R ? k_issued - R : 0; n < k_issued; ++n)
        mbar_wait(k_full + n % R, (n / R) & 1, kDrainBudget);
#pragma unroll 1
      for (uint32_t n = v_issued > R ? v_issued - R : 0; n < v_issued; ++n)
        mbar_wait(v_full + n % R, (n / R) & 1, kDrainBudget);
#pragma unroll 1
      for (uint32_t n = qc > 2 ? qc - 2 : 0; n < qc; ++n) mbar_wait(q_full + (n & 1), (n >> 1) & 1, kDrainBudget);
    }
    __syncwarp();
  } else if (warp < 4) {
    // ------------------------------------------------------------ MMA issuers
    // (whole warps, so that the one that issues a P.V can zero rows of V first)
    setmaxnreg_dec<72>();
    const bool qk_role = warp == 1;
    const int pv_wg = warp == 3 ? 0 : 1;  // the warpgroup whose steps this warp multiplies
    uint32_t g = 0, qc = 0, pn = 0;       // key tiles and items before this one, steps whose P has been consumed
    uint32_t n0 = 0, n1 = 0;              // the warpgroups' steps whose S has been issued
    uint32_t sb = 0, phase = 0;           // buffer of the next step of both, and how often it came round
    auto pass = [&](bool step) {
      sb += step;
      phase ^= sb == 3;
      sb = sb == 3 ? 0 : sb;
    };
    const uint32_t to = uniform(tO(pv_wg));
    const uint32_t q_addr = smem_u32(sQ), k_addr = smem_u32(sm + SL::k), v_addr = smem_u32(sm + SL::v);
    bool ok = true;                       // a wait that ran out ends this warp's products
    for (uint32_t c = 0;; ++c) {
      CrossItem it;
      if (lane == 0) it = read_item(c);
      it.hk = __shfl_sync(0xffffffffu, it.hk, 0);
      if (it.hk < 0) break;
      it.no = __shfl_sync(0xffffffffu, it.no, 0);
      it.nr = __shfl_sync(0xffffffffu, it.nr, 0);
      it.p0 = __shfl_sync(0xffffffffu, it.p0, 0);
      it.b = __shfl_sync(0xffffffffu, it.b, 0);
      const PairTiles pt = pair_tiles(a, it);
      if (pt.n == 0) continue;
      if (qk_role) {
        const uint32_t qb = qc & 1;
        ok = ok && cross_wait(q_full + qb, (qc >> 1) & 1, budget, s_abort);
#pragma unroll 1
        for (int t = 0; t < pt.n; ++t) {
          const uint32_t gs = g + t, s = gs % R;
          const uint64_t dk = uniform(sdesc_sw128(k_addr + s * SL::kTileBytes, 16, 1024));
          ok = ok && cross_wait(k_full + s, (gs / R) & 1, budget, s_abort);
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            if (!pt.sees(w, t)) continue;
            const uint64_t dq = uniform(sdesc_sw128(q_addr + (2 * qb + w) * SL::kTileBytes, 16, 1024));
            const uint32_t ts = uniform(tS(sb));
            // (the first time round the buffer is free: the phase before its first)
            ok = ok && cross_wait(buf_free + sb, phase ^ 1, budget, s_abort);
            ok = __all_sync(0xffffffffu, ok);
            if (ok) {
              tc_fence_after();
              if (elect_one()) {
#pragma unroll
                for (int k = 0; k < D / 16; ++k) mma_ss(ts, dq + kmajor_step(k), dk + kmajor_step(k), kIdescQK, k > 0);
                mma_commit(s_full + 4 * w + (w == 0 ? n0 & 3 : n1 & 3));
              }
              __syncwarp();
            }
            if (w == 0)
              ++n0;
            else
              ++n1;
            pass(true);
          }
          ok = __all_sync(0xffffffffu, ok);
          if (ok && elect_one()) mma_commit(k_empty + s);
          __syncwarp();
        }
        if (ok && elect_one()) mma_commit(q_empty + qb);
        ++qc;
        __syncwarp();
      } else {
        uint32_t first = 0;  // 0: the item's first product begins its sums
#pragma unroll 1
        for (int t = 0; t < pt.n; ++t) {
          const uint32_t gs = g + t, s = gs % R;
          pass(pv_wg == 1 && pt.sees(0, t));
          if (!pt.sees(pv_wg, t)) {
            // (not before the tile has come: the arrival would count for the one before)
            ok = ok && cross_wait(v_full + s, (gs / R) & 1, budget, s_abort);
            ok = __all_sync(0xffffffffu, ok);
            if (ok && lane == 0) mbar_arrive(v_empty + s);
            __syncwarp();
          } else {
            const uint64_t dv = uniform(vtile_desc(v_addr + s * SL::kTileBytes, 0));
            const uint32_t tp = uniform(tS(sb)), add = uniform(first);  // P overwrote its S
            const int kt = pt.band.tile(t), left = it.no - kt * 128;
            const bool partial = a.key_mask || left < 128;
            ok = ok && cross_wait(p_full + 4 * pv_wg + (pn & 3), (pn >> 2) & 1, budget, s_abort);
            ok = ok && cross_wait(v_full + s, (gs / R) & 1, budget, s_abort);
            ok = __all_sync(0xffffffffu, ok);
            if (ok) {
              if (partial) {  // (the other warp may do the same beside this one: the zeros are the same)
                uint32_t bits[4];
                const uint8_t* mask = a.key_mask ? a.key_mask + (size_t)it.b * a.Lk + (size_t)kt * 128 : nullptr;
                if (!key_bits(mask, left, bits)) zero_rows<4, 1>(sm + SL::v + s * SL::kTileBytes, bits);
                __syncwarp();
              }
              tc_fence_after();
              if (elect_one()) {
#pragma unroll
                for (int k = 0; k < 128 / 16; ++k)
                  mma_ts(to, tp + 8 * k, dv + vtile_step(k), kIdescPV, k > 0 ? 1u : add);
                mma_commit(buf_free + sb);
                mma_commit(pv_done + 4 * pv_wg + (pn & 3));
                mma_commit(v_empty + s);
              }
              __syncwarp();
            }
            first = 1;
            ++pn;
            pass(true);
          }
          pass(pv_wg == 0 && pt.sees(1, t));
        }
      }
      g += pt.n;
    }
    if (elect_one()) {
      uint64_t* my_drain = drain + (warp - 1);
      mma_commit(my_drain);
      mbar_wait(my_drain, 0, kDrainBudget);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ softmax warpgroups
    setmaxnreg_inc<216>();
    const int wg = (warp - 4) >> 2;
    const int quad = warp & 3;               // TMEM lane quadrant of this warp
    const int row = quad * 32 + lane;
    const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
    const float ks = a.kscale;
    const float2 ks2 = make_float2(ks, ks);
    const uint32_t tOw = tO(wg) + lane_off;
    const int row_tok = row / a.G, row_head = row - row_tok * a.G;
    CrossItem* s_cur = reinterpret_cast<CrossItem*>(sm + SL::cur) + 2 * wg;
    uint32_t own = 0;                        // this warpgroup's steps so far
    uint32_t sb = 0;                         // buffer of the next step of both
    auto pass = [&](bool step) {
      sb += step;
      sb = sb == 3 ? 0 : sb;
    };
    auto pv_wait = [&](uint32_t n) {  // until P.V of its n-th step is done
      cross_wait(pv_done + 4 * wg + (n & 3), (n >> 2) & 1, budget, s_abort);
    };
    // One thread takes each item from the ring and leaves it in s_cur; the warpgroup reads
    // it behind its barrier, so that all of it runs the same list even after a wait
    // has run out.
    const bool reader = quad == 0 && lane == 0;
    uint32_t c = 1;  // items taken, of which the last but one is current at an item's end
    if (reader) s_cur[0] = read_item(0);
    named_sync(3 + wg, 128);
    for (;;) {
      // (what a step needs of the item is read again, and is in no register beside the scores)
      const volatile CrossItem* it = s_cur + (~c & 1);
      if (it->hk < 0) break;
      PairTiles pt;
      {
        CrossItem x;
        x.nr = it->nr;
        x.no = it->no;
        x.p0 = it->p0;
        pt = pair_tiles(a, x);
      }
      const bool row_in = row_tok < min(it->nr - wg * a.tpt, a.tpt);
      // a row block without a valid row needs no weights: its P may hold anything,
      // since a row of P only reaches its own row of O
      const bool warp_in = __any_sync(0xffffffffu, row_in);
      float m_run = -INFINITY, l_run = 0.f;
      bool o_has = false;
#pragma unroll 1
      for (int t = 0; t < pt.n; ++t) {
        pass(wg == 1 && pt.sees(0, t));
        if (pt.sees(wg, t)) {
          const uint32_t tSw = tmem + 128u * sb + lane_off;
          // (found while the scores are on their way; keys behind the sequence's last lie behind every row)
          const int first = 128 * pt.band.tile(t), p0 = it->p0 + wg * a.tpt;
          const bool cut = !seen_whole(a, p0, min(it->nr - wg * a.tpt, a.tpt), first), part = cut || a.key_mask;
          uint32_t bits[4] = {~0u, ~0u, ~0u, ~0u};
          if (a.key_mask) key_bits(a.key_mask + (size_t)it->b * a.Lk + first, it->no - first, bits);
          if (cut) {
#pragma unroll
            for (int w = 0; w < 4; ++w) bits[w] &= seen_bits(a, p0 + row_tok, first + 32 * w);
          }
          cross_wait(s_full + 4 * wg + (own & 3), (own >> 2) & 1, budget, s_abort);
          __syncwarp();
          tc_fence_after();
          if (warp_in) {
            float x[128];
            {
              uint32_t r0[32], r1[32], r2[32], r3[32];
              tmem_ld32(tSw, r0);
              tmem_ld32(tSw + 32, r1);
              tmem_ld32(tSw + 64, r2);
              tmem_ld32(tSw + 96, r3);
              tmem_ld_wait4(r0, r1, r2, r3);
#pragma unroll
              for (int e = 0; e < 32; ++e) {
                x[e] = __uint_as_float(r0[e]);
                x[32 + e] = __uint_as_float(r1[e]);
                x[64 + e] = __uint_as_float(r2[e]);
                x[96 + e] = __uint_as_float(r3[e]);
              }
            }
            if (__builtin_expect(part, 0)) {
#pragma unroll
              for (int j = 0; j < 128; ++j)
                if (!((bits[j >> 5] >> (j & 31)) & 1u)) x[j] = -INFINITY;
            }
            // row maximum of the raw scores (the scale is positive)
            float mx[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) mx[e] = -INFINITY;
#pragma unroll
            for (int j = 0; j < 128; j += 4) {
              const int e = (j >> 2) & 3;
              mx[2 * e] = fmax3(mx[2 * e], x[j], x[j + 1]);
              mx[2 * e + 1] = fmax3(mx[2 * e + 1], x[j + 2], x[j + 3]);
            }
            const float mt = fmaxf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])),
                                   fmaxf(fmaxf(mx[4], mx[5]), fmaxf(mx[6], mx[7]))) * ks - kBelow<BF16>;
            // the base of the exponentials moves only when it would grow by more
            // than 2^8: numerator and denominator share it, so the result is exact
            float rescale = 1.f;
            const bool rebase = mt > m_run + 8.f;
            if (rebase) {
              rescale = ex2(m_run - mt);
              m_run = mt;
              l_run *= rescale;
            }
            const bool rescaled = __any_sync(0xffffffffu, rebase && o_has);
            const float shift = m_run == -INFINITY ? INFINITY : m_run;  // no finite score yet: every p is 0
            const float2 nshift = make_float2(-shift, -shift);
            {
              uint32_t r[32];
              float2 acc[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) acc[e] = make_float2(0.f, 0.f);
#pragma unroll
              for (int h = 0; h < 2; ++h) {
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                  const float2 z = fma2(make_float2(x[64 * h + 2 * e], x[64 * h + 2 * e + 1]), ks2, nshift);
                  const float2 pp = make_float2(ex2(z.x), ex2(z.y));
                  acc[e & 3] = add2(acc[e & 3], pp);
                  r[e] = BF16 ? pack_bf16x2(pp.x, pp.y) : pack_f16x2(pp.x, pp.y);
                }
                tmem_st32(tSw + 32 * h, r);  // P overwrites the S it came from
              }
              const float2 s01 = add2(acc[0], acc[1]), s23 = add2(acc[2], acc[3]);
              l_run += (s01.x + s23.x) + (s01.y + s23.y);
            }
            if (rescaled) {
              // this warpgroup's previous P.V must be done
              pv_wait(own - 1);
              __syncwarp();
              tc_fence_after();
              uint32_t r[32];
#pragma unroll 1
              for (int h = 0; h < D / 32; ++h) {
                tmem_ld32(tOw + 32 * h, r);
                tmem_ld_wait(r);
#pragma unroll
                for (int e = 0; e < 32; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * rescale);
                tmem_st32(tOw + 32 * h, r);
              }
            }
            tmem_st_wait();
          }
          tc_fence_before();
          __syncwarp();
          mbar_arrive_if(lane == 0, p_full + 4 * wg + (own & 3));
          o_has = true;
          ++own;
          pass(true);
        }
        pass(wg == 0 && pt.sees(1, t));
      }
      // ---- the item's end
      if (reader) s_cur[c & 1] = read_item(c);  // the next one
      ++c;
      if (o_has) pv_wait(own - 1);  // its last P.V
      __syncwarp();
      tc_fence_after();
      // (a NaN among the scores of keys that count is in l, and stays in the row)
      const float inv = l_run != 0.f ? rcp(l_run) : 0.f;
      const bool any = o_has && l_run != 0.f;
      // (With what the rounding drops, rows go by way of shared memory: a thread's own row is a line for
      // each of a warp's 32, which two results' stores wait for: 16 x 12 heads, 8192 tokens, a window of 1024,
      // 565 -> 518 us; one result's do not, and the code is shorter: 493 -> 481.)
      if constexpr (LO) {
        const size_t row0 = (size_t)(it->r0 + wg * a.tpt) * a.H + (size_t)it->hk * a.G;
        const int rel = row_in && *s_abort == 0 ? row_tok * a.H + row_head : -1;
        uint8_t* stage = sm + SL::rows + (warp - 4) * kRowStage;
        T* const out = static_cast<T*>(args.out) + row0 * a.d;
        T* const out_lo = static_cast<T*>(args.out_lo) + row0 * a.d;
#pragma unroll 1
        for (int col = 0; warp_in && col < D && col < a.d; col += 32) {
          uint32_t r[32], w[16];
          tmem_ld32(tOw + col, r);
          tmem_ld_wait(r);
#pragma unroll
          for (int e = 0; e < 32; ++e) r[e] = any ? __float_as_uint(__uint_as_float(r[e]) * inv) : 0u;
#pragma unroll
          for (int e = 0; e < 16; ++e) w[e] = pack2<BF16>(__uint_as_float(r[2 * e]), __uint_as_float(r[2 * e + 1]));
          store_rows32(stage, w, rel, out + col, a.d, a.d - col);
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            T h[2];
            *reinterpret_cast<uint32_t*>(h) = w[e];
            w[e] = pack2<BF16>(__uint_as_float(r[2 * e]) - IO<T>::to_f(h[0]),
                               __uint_as_float(r[2 * e + 1]) - IO<T>::to_f(h[1]));
          }
          store_rows32(stage, w, rel, out_lo + col, a.d, a.d - col);
        }
        if (args.lse && rel >= 0) args.lse[row0 + rel] = l_run != 0.f ? (m_run + lg2(l_run)) * kLn2 : -INFINITY;
      } else {
        const size_t orow = ((size_t)(it->r0 + wg * a.tpt + row_tok) * a.H + (size_t)it->hk * a.G + row_head);
#pragma unroll 1
        for (int col = 0; warp_in && col < D; col += 16) {
          uint32_t r[16];
          tmem_ld16(tOw + col, r);
          tmem_ld_wait(r);
          if (!row_in || *s_abort != 0) continue;
#pragma unroll
          for (int e = 0; e < 16; e += 8) {
            if (col + e >= a.d) continue;
            float o[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) o[k] = any ? __uint_as_float(r[e + k]) * inv : 0.f;
            store_rounded<T, 8>(static_cast<T*>(args.out) + orow * a.d + col + e, nullptr, o);
          }
        }
        if (args.lse && row_in && *s_abort == 0) args.lse[orow] = l_run != 0.f ? (m_run + lg2(l_run)) * kLn2 : -INFINITY;
      }
      tc_fence_before();
      named_sync(3 + wg, 128);  // every thread has read O; s_cur[c & 1] is there
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
  if (threadIdx.x == 0) cross_report(s_abort, a.status);
}

template <bool BF16, bool LO>
cudaError_t launch(const FwdArgs& a, const FwdMaps& maps, int grid, cudaStream_t s) {
  auto kernel = self64_kernel<BF16, LO>;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = prepare_kernel((const void*)kernel, (int)PairSmem::alloc, kRegs, &done);
  return e != cudaSuccess ? e : launch_clusters(kernel, a, maps, grid, kThreads, PairSmem::alloc, s);
}

}  // namespace

cudaError_t launch_self64(const FwdArgs& a, const FwdMaps& maps, bool bf16, int grid, cudaStream_t s) {
  if (a.out_lo) return bf16 ? launch<true, true>(a, maps, grid, s) : launch<false, true>(a, maps, grid, s);
  return bf16 ? launch<true, false>(a, maps, grid, s) : launch<false, false>(a, maps, grid, s);
}

}  // namespace dfa
