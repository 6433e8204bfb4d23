// Cross attention, forward, head sizes to 64 (df_cross128.cu: to 128): queries
// [B, Lq] or packed, keys and values of another length [B, Lk] or packed, query
// heads that share key heads, on tcgen05 (bf16 / fp16 I/O, fp32 accumulation and
// softmax).
//
//   s_ij = scale q_i.k_j,  o_i = sum_j exp(s_ij - lse_i) v_j,
//   lse_i = log sum_j exp s_ij          over the valid keys j of i's sequence;
// a row without a valid key gets zeros and lse = -inf.
//
// One CTA per SM takes query tiles (128 rows, df_cross.cuh) in turn.  The key
// tiles (128 keys) of an item alternate between two softmax warpgroups with
// independent (max, sum, O), so that the tensor core works for one while the other
// exponentiates; the two are merged at the end of the item.  Three score buffers
// in tensor memory let S run ahead of the softmax.
//   warp 0      finds the items and loads Q (two buffers), K and V (a ring each, a
//               stage freed by the product that read it) by TMA;
//   warp 1      issues S = Q.K^T;
//   warps 3, 2  issue O_w += P.V for warpgroup 0 and 1, and zero the rows of V whose
//               keys do not count first;
//   warps 4-11  softmax: one thread per row, P (rounded to the I/O type) written
//               over its S.
// Keys that do not count (a tail tile's rows behind the sequence, key_mask) get
// weight 0 by selection, not by arithmetic, and their rows of V are zeroed in
// shared memory before P.V, so that whatever they hold (NaN, infinities, the
// next sequence) stays out.  Warps without a valid row skip the softmax.
//
// Few query tiles, long keys: a cluster of CTAs shares one item, each with a
// part of the key tiles; the partial (max, sum, O) are joined through
// distributed shared memory, so no workspace and no second launch is needed.
//
// Measured (GB300): 16 x 12 heads, 2048 queries x 8192 keys, bf16: 721 to 758 us by
// machine and inputs, 1088 to 1144 TFLOP/s.  A tile of 128 x 128 scores takes about 1020 cycles of an SM; its
// products take 618 of the tensor core (P.V, 64 columns wide, runs at two thirds
// of its rate), its exponentials 512.  What is left is latency: a score buffer goes
// around S, softmax (1470 cycles), P.V, S in about 3 x 1020.  Of what would shorten
// that, P in columns of its own (two score buffers: 857 us, with the warpgroups
// taking turns 914), P.V in two halves (810), scores read twice in short loops
// (828) and one warp issuing both products in order (1138) were slower (735 at the
// time).
//
// SELF: causal attention with a window and sinks (df_cross.cuh) where there is little of it
// (df_self64.cu: more).  Key tiles that no row of an item sees are not on its list; where some
// row does not see a key, a thread finds its row's bits from two positions, and a tile that
// every row sees whole takes the path without bits.  Sequences' query tiles run from the last,
// which has the most keys, to the first.  Measured: 12 heads, one sequence of 1024 tokens: 12 us,
// 2048: 16; 8 heads of 4096: 25 us, 690 TFLOP/s of what is seen (4 flops a score and column).
#include "df_cross_fwd.cuh"

namespace dfa {

namespace {

using namespace ptx;

constexpr int kThreads = 384;
constexpr int kRegs = 168;  // launched; after the split eight softmax warps have 224, four others 56
static_assert(256 * 224 + 128 * 56 <= kThreads * kRegs, "setmaxnreg.inc must not wait");
constexpr uint32_t kItemRing = 4;

struct FwdSmem {
  static constexpr int D = 64;
  static constexpr int kStages = 4;                                 // K tiles, and V tiles, in flight
  static constexpr uint32_t kTileBytes = kBoxBytes;
  static constexpr uint32_t q = 0;                                  // [2][Q tile]
  static constexpr uint32_t k = q + 2 * kTileBytes;                 // [kStages][K tile]
  static constexpr uint32_t v = k + kStages * kTileBytes;           // [kStages][V tile]
  static constexpr uint32_t ml = v + kStages * kTileBytes;          // float4 [2 warpgroups, a cluster's][128]
  static constexpr uint32_t bars = ml + 3 * 128 * 16;
  // q_full, q_empty [2]; k_full, k_empty, v_full, v_empty [kStages]; s_full,
  // buf_free, drain [3]; p_full, pv_done [4]; item_full, item_empty; claim
  static constexpr int kBars = 4 + 4 * kStages + 9 + 8 + 2 * (int)kItemRing + 1;
  static constexpr uint32_t ring = (bars + kBars * 8 + 15) & ~15u;  // CrossItem slots of 32 bytes
  static constexpr uint32_t cur = ring + 32 * kItemRing;            // the softmax warpgroups' current item
  static constexpr uint32_t claim = cur + 64;                       // 16 bytes
  static constexpr uint32_t misc = claim + 16;                      // abort flag, tmem slot
  static constexpr uint32_t bytes = misc + 16;
  static constexpr uint32_t alloc = bytes + 1024;
  static_assert(alloc <= 232448, "shared memory of one CTA");
  // the join of a cluster: O [128][D] fp32 over the (then idle) K tiles
  static_assert(128 * D * 4 <= kStages * kTileBytes, "O fits over K");
};

template <bool BF16, bool SELF>
__global__ void __launch_bounds__(kThreads, 1) cross64_kernel(const FwdArgs args, const __grid_constant__ FwdMaps maps) {
  using SL = FwdSmem;
  constexpr int D = SL::D;
  constexpr uint32_t R = SL::kStages;
  constexpr uint32_t kIdescQK = idesc_f16(128, 128, BF16 ? 1 : 0, 0, 0);
  constexpr uint32_t kIdescPV = idesc_f16(128, D, BF16 ? 1 : 0, 0, 1);
  using T = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
  // tensor-memory columns: three score buffers (tile G of the CTA uses G % 3), two O
  static_assert(tmem_region_fits(384, 2u * D, 512), "scores and two O accumulators in 512 columns");
  constexpr uint32_t kItemReaders = 4;  // three issuing warps, the softmax warpgroups' reader

  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t* sQ = sm + SL::q;
  float4* sML = reinterpret_cast<float4*>(sm + SL::ml);
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + SL::bars);
  uint64_t* q_full = bars;
  uint64_t* q_empty = bars + 2;
  uint64_t* k_full = bars + 4;
  uint64_t* k_empty = k_full + R;
  uint64_t* v_full = k_empty + R;
  uint64_t* v_empty = v_full + R;
  uint64_t* s_full = v_empty + R;      // [3] S of the buffer computed
  uint64_t* buf_free = s_full + 3;     // [3] the P.V that read the buffer is done
  uint64_t* drain = buf_free + 3;      // [3], one per issuing warp
  // [wg][k & 1]: the four warps of wg stored P of its k-th tile; P.V of it done.  Two
  // of each per warpgroup because a warp may be through with its next tile before a
  // sibling has stored this one, or before this one's P.V is done; it is never two
  // ahead, since its next S but one waits for a P.V issued behind this phase.
  uint64_t* p_full = drain + 3;
  uint64_t* pv_done = p_full + 4;
  uint64_t* item_full = pv_done + 4;
  uint64_t* item_empty = item_full + kItemRing;
  uint64_t* claim_bar = item_empty + kItemRing;
  auto ring_slot = [&](uint32_t c) { return reinterpret_cast<CrossItem*>(sm + SL::ring + 32 * (c % kItemRing)); };
  CrossItem* s_cur = reinterpret_cast<CrossItem*>(sm + SL::cur);
  volatile int* s_abort = reinterpret_cast<volatile int*>(sm + SL::misc);
  uint32_t* tslot = reinterpret_cast<uint32_t*>(sm + SL::misc + 4);

  const CrossArgs& a = args.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int b = 0; b < 2; ++b) {
      mbar_init(q_full + b, 1);
      mbar_init(q_empty + b, 1);
    }
    for (uint32_t s = 0; s < 4 * R; ++s) mbar_init(k_full + s, 1);
    for (int b = 0; b < 3; ++b) {
      mbar_init(s_full + b, 1);
      mbar_init(buf_free + b, 1);
      mbar_init(drain + b, 1);
    }
    for (int b = 0; b < 4; ++b) {
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
  const uint32_t rank = args.splits > 1 ? cluster_rank() : 0u;
  // an item's key tiles, and this CTA's part of them
  auto band_of = [&](const CrossItem& it) { return SELF ? key_band(a, it) : CrossBand{0, 0}; };
  auto part = [&](const CrossItem& it, const CrossBand& band, int* t0) { return key_part(args, it, band, rank, t0); };
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
    setmaxnreg_dec<56>();
    // (the whole warp runs every step, and one lane of it issues: this loop's length
    // in instructions is what a tile's period comes down to)
    TileWalk<SELF> walk;
    if (SELF) walk.together = heads_together(a);
    TileClaim claim = {claim_bar, reinterpret_cast<uint4*>(sm + SL::claim)};
    uint32_t g = 0, qc = 0, k_issued = 0, v_issued = 0;
    int mask_b = -1, mask_n = 0;  // the last masked row measured
    bool ok = true;               // a wait ran out: nothing is loaded after it
    long long number = blockIdx.x / args.splits;
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
      CrossItem it = walk.find(a, query_side(a), key_side(a), a.tpt, number);
      const uint32_t slot = c % kItemRing;
      if (a.key_mask && it.hk >= 0) {  // key tiles behind the last valid key are not visited
        if (it.b != mask_b) mask_n = masked_length(a.key_mask + (size_t)it.b * a.Lk, it.no);
        mask_b = it.b;
        it.no = mask_n;
      }
      if (SELF) clip_causal(it);
      bool room = true;
      if (c >= kItemRing) room = cross_wait(item_empty + slot, ((c / kItemRing) - 1) & 1, budget, s_abort);
      if (__any_sync(0xffffffffu, *s_abort || !room)) it.hk = -1;
      if (lane == 0 && room) {
        *ring_slot(c) = it;
        mbar_arrive(item_full + slot);
      }
      if (it.hk < 0) break;
      int t0;
      const CrossBand band = band_of(it);
      const int nt = part(it, band, &t0);
      if (nt > 0) {
        const uint32_t qb = qc & 1;
        ok = ok && cross_wait(q_empty + qb, ((qc >> 1) & 1) ^ 1, budget, s_abort);
        ok = __all_sync(0xffffffffu, ok);
        if (ok) {
          if (elect_one()) {
            mbar_expect_tx(q_full + qb, (uint32_t)(a.G * a.tpt) * 128u);
            tma_load_3d(sQ + qb * SL::kTileBytes, &maps.q, 0, it.hk * a.G, it.r0, q_full + qb);
          }
          __syncwarp();
          ++qc;
        }
      }
      // K(t) goes out before V(t - 1): the next scores must not wait until P.V has
      // freed a V tile.
      // The next item is asked for two tiles before this one's end: early enough to be
      // answered by then, late enough to leave it to a CTA that is through sooner.
      const int ask_at = args.splits > 1 ? -1 : max(0, nt - 2);
      auto row_at = [&](int t) { return it.o0 + (SELF ? band.tile(t0 + t) : t0 + t) * 128; };
#pragma unroll 1
      for (int t = 0; t <= nt; ++t) {
        if (t == ask_at) claim.ask();
        if (t < nt) load(&maps.k, SL::k, k_full, k_empty, g + t, it.hk, row_at(t), k_issued);
        if (t > 0) load(&maps.v, SL::v, v_full, v_empty, g + t - 1, it.hk, row_at(t - 1), v_issued);
      }
      g += nt;
      number = args.splits > 1 ? -1 : claim.answer(budget, s_abort);
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
    setmaxnreg_dec<56>();
    const bool qk_role = warp == 1;
    const int pv_wg = warp == 3 ? 0 : 1;  // the warpgroup whose tiles this warp multiplies
    uint32_t g = 0, qc = 0, pn = 0;       // key tiles and items before this one, tiles whose P has been consumed
    const uint32_t to = uniform(tO(pv_wg));
    const uint32_t q_addr = smem_u32(sQ), k_addr = smem_u32(sm + SL::k), v_addr = smem_u32(sm + SL::v);
    bool ok = true;                       // a wait that ran out ends this warp's products
    for (uint32_t c = 0;; ++c) {
      CrossItem it;
      if (lane == 0) it = read_item(c);
      it.hk = __shfl_sync(0xffffffffu, it.hk, 0);
      if (it.hk < 0) break;
      it.no = __shfl_sync(0xffffffffu, it.no, 0);
      if (SELF) it.p0 = __shfl_sync(0xffffffffu, it.p0, 0);
      it.b = __shfl_sync(0xffffffffu, it.b, 0);
      int t0;
      const CrossBand band = band_of(it);
      const int nt = part(it, band, &t0);
      if (nt == 0) continue;
      if (qk_role) {
        const uint32_t qb = qc & 1;
        ok = ok && cross_wait(q_full + qb, (qc >> 1) & 1, budget, s_abort);
        const uint64_t dq = uniform(sdesc_sw128(q_addr + qb * SL::kTileBytes, 16, 1024));
#pragma unroll 1
        for (int t = 0; t < nt; ++t) {
          const uint32_t gs = g + t, s = gs % R, sb = gs % 3;
          const uint64_t dk = uniform(sdesc_sw128(k_addr + s * SL::kTileBytes, 16, 1024));
          const uint32_t ts = uniform(tS(sb));
          if (gs >= 3) ok = ok && cross_wait(buf_free + sb, ((gs - 3) / 3) & 1, budget, s_abort);
          ok = ok && cross_wait(k_full + s, (gs / R) & 1, budget, s_abort);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) continue;
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < D / 16; ++k) mma_ss(ts, dq + kmajor_step(k), dk + kmajor_step(k), kIdescQK, k > 0);
            mma_commit(s_full + sb);
            mma_commit(k_empty + s);
          }
          __syncwarp();
        }
        ok = __all_sync(0xffffffffu, ok);
        if (ok && elect_one()) mma_commit(q_empty + qb);
        ++qc;
        __syncwarp();
      } else {
#pragma unroll 1
        for (int t = pv_wg; t < nt; t += 2, ++pn) {
          const uint32_t gs = g + t, s = gs % R, sb = gs % 3;
          const uint64_t dv = uniform(vtile_desc(v_addr + s * SL::kTileBytes, 0));
          const uint32_t tp = uniform(tS(sb)), first = uniform(t >= 2 ? 1u : 0u);  // P(t) overwrote its S
          const int kt = SELF ? band.tile(t0 + t) : t0 + t, left = it.no - kt * 128;
          const bool partial = a.key_mask || left < 128;
          // P of this tile says that S was there, so that P.V of the stage's previous
          // tile is done: the wait for V sees its own phase
          ok = ok && cross_wait(p_full + 2 * pv_wg + (pn & 1), (pn >> 1) & 1, budget, s_abort);
          ok = ok && cross_wait(v_full + s, (gs / R) & 1, budget, s_abort);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) continue;
          if (partial) {
            uint32_t bits[4];
            const uint8_t* mask = a.key_mask ? a.key_mask + (size_t)it.b * a.Lk + (size_t)kt * 128 : nullptr;
            if (!key_bits(mask, left, bits)) zero_rows<4, 1>(sm + SL::v + s * SL::kTileBytes, bits);
            __syncwarp();
          }
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < 128 / 16; ++k)
              mma_ts(to, tp + 8 * k, dv + vtile_step(k), kIdescPV, k > 0 ? 1u : first);
            mma_commit(buf_free + sb);
            mma_commit(pv_done + 2 * pv_wg + (pn & 1));
            mma_commit(v_empty + s);
          }
          __syncwarp();
        }
      }
      g += nt;
    }
    if (elect_one()) {
      uint64_t* my_drain = drain + (warp - 1);
      mma_commit(my_drain);
      mbar_wait(my_drain, 0, kDrainBudget);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ softmax warpgroups
    setmaxnreg_inc<224>();
    const int wg = (warp - 4) >> 2;
    const int quad = warp & 3;               // TMEM lane quadrant of this warp
    const int row = quad * 32 + lane;
    const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
    const float ks = a.kscale;
    const float2 ks2 = make_float2(ks, ks);
    const uint32_t tOw = tO(wg) + lane_off;
    const int row_tok = row / a.G, row_head = row - row_tok * a.G;
    uint32_t own = 0, gbase = 0;  // this warpgroup's tiles, and the CTA's before the item
    auto pv_wait = [&](uint32_t n) {  // until P.V of its n-th tile is done
      cross_wait(pv_done + 2 * wg + (n & 1), (n >> 1) & 1, budget, s_abort);
    };
    // One thread takes each item from the ring and leaves it in s_cur; all 256 read
    // it behind their barrier, so that they run the same list even after a wait
    // has run out.
    const bool reader = warp == 4 && lane == 0;
    uint32_t c = 1;  // items taken, of which the last but one is current at an item's end
    if (reader) s_cur[0] = read_item(0);
    named_sync(3, 256);
    for (;;) {
      const CrossItem it = s_cur[~c & 1];
      if (it.hk < 0) break;
      int t0;
      const CrossBand band = band_of(it);
      const int nt = part(it, band, &t0);
      const bool row_in = row_tok < it.nr;
      // a row block without a valid row needs no weights: its P may hold anything,
      // since a row of P only reaches its own row of O
      const bool warp_in = __any_sync(0xffffffffu, row_in);
      float m_run = -INFINITY, l_run = 0.f;
      bool o_has = false;
      const int whole = a.key_mask ? 0 : it.no / 128 - t0;  // tiles of which every key counts
      uint32_t sb = (gbase + wg) % 3, phase = ((gbase + wg) / 3) & 1;  // of tile gbase + t
      for (int t = wg; t < nt; t += 2, ++own) {
        const uint32_t tSw = tmem + 128u * sb + lane_off;
        cross_wait(s_full + sb, phase, budget, s_abort);
        __syncwarp();
        tc_fence_after();
        if (warp_in) {
          const int kt = SELF ? band.tile(t0 + t) : t0 + t;
          const bool cut = SELF && !seen_whole(a, it.p0, it.nr, kt * 128);
          if (SELF ? a.key_mask || it.no < kt * 128 + 128 || cut : t >= whole) {
            const int left = it.no - kt * 128;
            uint32_t bits[4];
            const bool all = key_bits(a.key_mask ? a.key_mask + (size_t)it.b * a.Lk + (size_t)kt * 128 : nullptr, left, bits);
            if (SELF && cut) {
#pragma unroll
              for (int w = 0; w < 4; ++w) bits[w] &= seen_bits(a, it.p0 + row_tok, kt * 128 + 32 * w);
            }
            if (!all || cut) {
              // the scores of keys that do not count become -inf in place (kept out of
              // the straight code below, which the instruction caches have to hold)
#pragma unroll 1
              for (int w = 0; w < 4; ++w) {
                const uint32_t word = w == 0 ? bits[0] : w == 1 ? bits[1] : w == 2 ? bits[2] : bits[3];
                uint32_t r[32];
                tmem_ld32(tSw + 32 * w, r);
                tmem_ld_wait(r);
#pragma unroll
                for (int j = 0; j < 32; ++j)
                  if (!((word >> j) & 1u)) r[j] = 0xff800000u;
                tmem_st32(tSw + 32 * w, r);
              }
              tmem_st_wait();
            }
          }
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
              tmem_st32(tSw + 32 * h, r);  // P(t) overwrites the S it came from
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
        mbar_arrive_if(lane == 0, p_full + 2 * wg + (own & 1));
        o_has = true;
        sb += 2;
        if (sb >= 3) {
          sb -= 3;
          phase ^= 1;
        }
      }
      // ---- the item's end: both warpgroups' states together
      if (reader) s_cur[c & 1] = read_item(c);  // the next one
      ++c;
      if (wg < nt) pv_wait(own - 1);  // its last P.V
      __syncwarp();
      tc_fence_after();
      sML[wg * 128 + row] = make_float4(m_run, l_run, o_has ? 1.f : 0.f, 0.f);
      // (each thread goes on to read both warpgroups' O, and has waited for its own one's
      // P.V only: the barrier has to order the other's tensor memory too)
      tc_fence_before();
      named_sync(3, 256);
      tc_fence_after();
      const float4 s0 = sML[row], s1 = sML[128 + row];
      const bool h0 = s0.z != 0.f, h1 = s1.z != 0.f;
      const float m = fmaxf(s0.x, s1.x);
      const float f0 = (h0 && m != -INFINITY) ? ex2(s0.x - m) : 0.f;
      const float f1 = (h1 && m != -INFINITY) ? ex2(s1.x - m) : 0.f;
      const float l = s0.y * f0 + s1.y * f1;
      const bool alone = args.splits == 1;
      // (a NaN among the scores of keys that count is in l, and stays in the row)
      const float inv = !alone ? 1.f : (l != 0.f ? rcp(l) : 0.f);
      const size_t orow = ((size_t)(it.r0 + row_tok) * a.H + (size_t)it.hk * a.G + row_head);
      float* sO = reinterpret_cast<float*>(sm + SL::k);  // a cluster's join: the K tiles are idle by then
#pragma unroll 1
      for (int col = wg * (D / 2); warp_in && col < (wg + 1) * (D / 2); col += 16) {
        uint32_t ra[16], rb[16];
        tmem_ld16(tO(0) + lane_off + col, ra);
        tmem_ld16(tO(1) + lane_off + col, rb);
        tmem_ld_wait(ra);
        tmem_ld_wait(rb);
        if (!row_in || *s_abort != 0) continue;
#pragma unroll
        for (int e = 0; e < 16; e += 8) {
          float o[8];
#pragma unroll
          for (int k = 0; k < 8; ++k)
            o[k] = ((f0 > 0.f ? __uint_as_float(ra[e + k]) * f0 : 0.f) +
                    (f1 > 0.f ? __uint_as_float(rb[e + k]) * f1 : 0.f)) * inv;
          if (!alone) {
#pragma unroll
            for (int k = 0; k < 8; k += 4)
              *reinterpret_cast<float4*>(sO + o_piece<D>(row, (col + e + k) / 4)) =
                  make_float4(o[k], o[k + 1], o[k + 2], o[k + 3]);
          } else if (col + e < a.d) {
            const size_t at = orow * a.d + col + e;
            store_rounded<T, 8>(static_cast<T*>(args.out) + at,
                                args.out_lo ? static_cast<T*>(args.out_lo) + at : nullptr, o);
          }
        }
      }
      if (!alone) {
        if (wg == 0) sML[256 + row] = make_float4(m, l, 0.f, 0.f);
      } else if (args.lse && wg == 0 && row_in && *s_abort == 0) {
        args.lse[orow] = l != 0.f ? (m + lg2(l)) * kLn2 : -INFINITY;
      }
      tc_fence_before();
      named_sync(3, 256);  // every thread has read sML and s_cur[c & 1]
      gbase += nt;
      if (!alone) break;  // one item per cluster; s_cur stays for the join
    }
  }

  if (args.splits > 1) {
    cluster_sync();
    if (warp >= 4 && s_cur->hk >= 0)
      join_cluster<T, D>(args, *s_cur, rank, (int)threadIdx.x - 128, 256, smem_u32(sML + 256), smem_u32(sm + SL::k));
    cluster_sync();  // no CTA leaves while another one reads its shared memory
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
  if (threadIdx.x == 0) cross_report(s_abort, a.status);
}

template <bool BF16, bool SELF>
cudaError_t launch(const FwdArgs& a, const FwdMaps& maps, int grid, cudaStream_t s) {
  auto kernel = cross64_kernel<BF16, SELF>;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = prepare_kernel((const void*)kernel, (int)FwdSmem::alloc, kRegs, &done);
  return e != cudaSuccess ? e : launch_clusters(kernel, a, maps, grid, kThreads, FwdSmem::alloc, s);
}

}  // namespace

cudaError_t launch_cross64(const FwdArgs& a, const FwdMaps& maps, bool bf16, bool self, int grid, cudaStream_t s) {
  if (self) return bf16 ? launch<true, true>(a, maps, grid, s) : launch<false, true>(a, maps, grid, s);
  return bf16 ? launch<true, false>(a, maps, grid, s) : launch<false, false>(a, maps, grid, s);
}

}  // namespace dfa
