// Causal attention with a window and sinks, forward, head sizes 72 to 128, where there is more work
// than a round of the SMs (df_cross128.cu's SELF form has clusters for less), on tcgen05 (bf16 / fp16
// I/O, fp32 accumulation and softmax).
//
//   s_ij = scale q_i.k_j,  o_i = sum_j exp(s_ij - lse_i) v_j  over the keys j that i sees
//   (df_cross.cuh); a row that sees none gets zeros and lse = -inf.
//
// An item is two query tiles that follow one another, one for each team of eight softmax warps, with
// a Q, K and V tile, tensor-memory columns and an issuer of its own: where both teams take turns at
// one query tile and join their sums, a window's items (some ten key tiles) end as often as they
// begin.  Here a team ends by itself, beside the other one's tiles.
//   warp 0       finds the items and loads Q, K and V of both teams by TMA;
//   warps 1, 2   issue S = Q.K^T and O += P.V for team 0 and 1;
//   warp 3       per V tile: zeroes the rows of keys that do not count, hands it on;
//   warps 4-19   softmax: a row's scores are shared by two threads (a half of the
//                columns each), which exchange their maxima through shared memory;
//                P (rounded to the I/O type) overwrites the scores it came from.
// Keys that do not count get weight 0 by selection, by bits that are found before the scores are awaited,
// and their rows of V are zeroed, as in df_cross128.cu; 32 columns that no row of a warp sees get no
// exponentials.
//
// Measured (GB300, bf16): 8 x 16 heads, 8192 tokens, d = 128, a window of 1024: 491 us, 1050 TFLOP/s of what
// is seen (one query tile an item: 614); 16 x 16 heads sharing 4, 2048 tokens: 253 us, 1088 TFLOP/s (301);
// 64 x 16 heads sharing 4, 512 tokens: 127 us (162).  Without a window, items are long and the gain is
// smaller: 2 x 16 heads sharing 4, 8192 tokens: 394 us, 1395 TFLOP/s (422).
#include "df_cross_fwd.cuh"

namespace dfa {

namespace {

using namespace ptx;

constexpr int kThreads = 640, kSoftmaxThreads = 512;
// registers per thread: launched, and after the split (softmax, others)
constexpr int kRegs = 96, kSoftmaxRegs = 104, kOtherRegs = 64;
static_assert(kSoftmaxThreads * kSoftmaxRegs + 128 * kOtherRegs <= kThreads * kRegs, "setmaxnreg.inc must not wait");
constexpr uint32_t kItemRing = 4;

struct TeamSmem {
  static constexpr int D = 128;
  static constexpr int kChunks = D / 64;
  static constexpr int kKeys = kFwdKeys;
  static constexpr uint32_t kQBytes = kChunks * kBoxBytes;
  static constexpr uint32_t kKVBox = kKeys * 128;                   // a 64-column box of a key tile
  static constexpr uint32_t kTileBytes = kChunks * kKVBox;
  static constexpr uint32_t q = 0;                                  // [2 teams][Q tile]
  static constexpr uint32_t k = q + 2 * kQBytes;               // [2 teams][K tile]
  static constexpr uint32_t v = k + 2 * kTileBytes;       // the same of V
  static constexpr uint32_t ml = v + 2 * kTileBytes;      // float2 (max, sum) [4 warpgroups][128]
  static constexpr uint32_t mx = ml + 4 * 128 * 8;                  // float [2 tiles][4 warpgroups][128]: row maxima
  static constexpr uint32_t rows = mx + 2 * 4 * 128 * 4;                   // int2 [128]: a row's token, and its place from the tile's first
  static constexpr uint32_t stage = rows + 128 * 8;                  // [16 warps] rows on their way out
  static constexpr uint32_t bars = stage + 16 * kRowStage;
  // q_full, q_empty [2]; k_full, k_empty, v_full, v_ready, v_empty [2];
  // s_full, p_full, o_final, drain [2]; exp_done [2][4]; item_full, item_empty; claim
  static constexpr int kBars = 30 + 2 * (int)kItemRing + 1;
  static constexpr uint32_t ring = (bars + kBars * 8 + 15) & ~15u;  // CrossItem slots of 32 bytes
  static constexpr uint32_t cur = ring + 32 * kItemRing;            // [2 teams][2] current items
  static constexpr uint32_t claim = cur + 128;                      // 16 bytes
  static constexpr uint32_t misc = claim + 16;                      // abort flag, tmem slot
  static constexpr uint32_t bytes = misc + 16;
  static constexpr uint32_t alloc = bytes + 1024;
  static_assert(alloc <= 232448, "shared memory of one CTA");
};

// A team's query tile of an item: the first or the second.
__device__ __forceinline__ CrossItem team_item(const CrossArgs& a, CrossItem it, int w) {
  it.r0 += w * a.tpt;
  it.p0 += w * a.tpt;
  it.nr = min(it.nr - w * a.tpt, a.tpt);
  if (it.nr <= 0) it.no = 0;
  clip_causal(it);
  return it;
}

// 64 columns of a warp's rows, o = a f, rounded, and (out_lo) what that rounding dropped, 32 at a time by
// way of shared memory (16 at a time: 606 us against 590 for 8 x 16 heads sharing 4, 8192 tokens, a window
// of 1024 and 4 sinks, 663 against 637 with what rounding drops).
template <bool BF16, typename T>
__device__ __forceinline__ void store_own(const FwdArgs& args, uint8_t* stage, uint32_t ta, float f, bool empty, int rel,
                                          size_t row0, int col) {
  const int d = args.c.d;
  const float2 f2 = make_float2(f, f);
#pragma unroll 1
  for (int end = min(col + 64, d); col < end; col += 32, ta += 32) {
    uint32_t r[32], w[16];
    tmem_ld32(ta, r);
    tmem_ld_wait(r);
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const float2 o = mul2(make_float2(__uint_as_float(r[2 * e]), __uint_as_float(r[2 * e + 1])), f2);
      r[2 * e] = empty ? 0u : __float_as_uint(o.x);
      r[2 * e + 1] = empty ? 0u : __float_as_uint(o.y);
      w[e] = pack2<BF16>(__uint_as_float(r[2 * e]), __uint_as_float(r[2 * e + 1]));
    }
    store_rows32(stage, w, rel, static_cast<T*>(args.out) + row0 * d + col, d, d - col);
    if (!args.out_lo) continue;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      T h[2];
      *reinterpret_cast<uint32_t*>(h) = w[e];
      w[e] = pack2<BF16>(__uint_as_float(r[2 * e]) - IO<T>::to_f(h[0]), __uint_as_float(r[2 * e + 1]) - IO<T>::to_f(h[1]));
    }
    store_rows32(stage, w, rel, static_cast<T*>(args.out_lo) + row0 * d + col, d, d - col);
  }
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads, 1) self128_kernel(const FwdArgs args, const __grid_constant__ FwdMaps maps) {
  using SL = TeamSmem;
  constexpr int D = SL::D;
  constexpr int kChunks = SL::kChunks;
  constexpr int kKeys = SL::kKeys, kWords = kKeys / 32;
  constexpr uint32_t kIdescQK = idesc_f16(128, kKeys, BF16 ? 1 : 0, 0, 0);
  constexpr uint32_t kIdescPV = idesc_f16(128, D, BF16 ? 1 : 0, 0, 1);
  using T = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
  // Tensor-memory columns of a team: S, of which P takes the first half of each
  // half, then O.
  static_assert(tmem_region_fits(256 + kKeys, D, 512), "S and O of two teams in 512 columns");
  constexpr uint32_t kItemReaders = 5;  // two issuers, warp 3, a reader of each team

  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t* sQ = sm + SL::q;
  float2* sML = reinterpret_cast<float2*>(sm + SL::ml);
  float* sMax = reinterpret_cast<float*>(sm + SL::mx);
  int2* sRow = reinterpret_cast<int2*>(sm + SL::rows);
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + SL::bars);
  uint64_t* q_full = bars;              // [team], as the next ones
  uint64_t* q_empty = bars + 2;
  uint64_t* k_full = bars + 4;
  uint64_t* k_empty = k_full + 2;
  uint64_t* v_full = k_empty + 2;
  uint64_t* v_ready = v_full + 2;   // landed, rows that do not count zeroed
  uint64_t* v_empty = v_ready + 2;
  uint64_t* s_full = v_empty + 2;       // S computed
  uint64_t* p_full = s_full + 2;        // its eight warps have stored P
  uint64_t* o_final = p_full + 2;       // every P.V of the item done
  uint64_t* drain = o_final + 2;
  uint64_t* exp_done = drain + 2;       // [team][n & 3]: its eight warps are through with its n-th tile's exponentials
  uint64_t* item_full = exp_done + 8;
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
      mbar_init(s_full + b, 1);
      mbar_init(p_full + b, 8);
      for (int n = 0; n < 4; ++n) mbar_init(exp_done + 4 * b + n, 8);
      mbar_init(o_final + b, 1);
      mbar_init(drain + b, 1);
    }
    for (uint32_t s = 0; s < 10; ++s) mbar_init(k_full + s, 1);
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
  if (threadIdx.x < 128) {
    const int tok = threadIdx.x / a.G;
    sRow[threadIdx.x] = make_int2(tok, tok * a.H + (int)threadIdx.x - tok * a.G);
  }
  if (warp == 1) {
    tmem_alloc(tslot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;
  auto tS = [&](int w) { return tmem + 256u * w; };
  auto tO = [&](int w) { return tmem + 256u * w + kKeys; };

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
    setmaxnreg_dec<kOtherRegs>();
    // (the whole warp runs every step, and one lane of it issues)
    TileWalk<true> walk;
    walk.together = heads_together(a);
    TileClaim claim = {claim_bar, reinterpret_cast<uint4*>(sm + SL::claim)};
    uint32_t kn0 = 0, kn1 = 0, vn0 = 0, vn1 = 0;  // tiles loaded for each team
    uint32_t qn0 = 0, qn1 = 0;
    int mask_b = -1, mask_n = 0;  // the last masked row measured
    bool ok = true;               // a wait ran out: nothing is loaded after it
    long long number = blockIdx.x;
    // K or V rows [row, row + 128) for a team, its n-th tile
    auto load = [&](const CUtensorMap* map, uint32_t tiles, uint64_t* full, uint64_t* empty, int w, uint32_t& n, int head,
                    int row) {
      ok = ok && cross_wait(empty + w, (n & 1) ^ 1, budget, s_abort);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) return;
      if (elect_one()) {
        uint8_t* dst = sm + tiles + w * SL::kTileBytes;
        mbar_expect_tx(full + w, SL::kTileBytes);
        for (int ch = 0; ch < kChunks; ++ch) tma_load_3d(dst + ch * SL::kKVBox, map, ch * 64, head, row, full + w);
      }
      __syncwarp();
      ++n;
    };
    for (uint32_t c = 0;; ++c) {
      CrossItem it = walk.find(a, query_side(a), key_side(a), 2 * a.tpt, number);
      const uint32_t slot = c % kItemRing;
      if (a.key_mask && it.hk >= 0) {  // key tiles behind the last valid key are not visited
        if (it.b != mask_b) mask_n = masked_length(a.key_mask + (size_t)it.b * a.Lk, it.no);
        mask_b = it.b;
        it.no = mask_n;
      }
      bool room = true;
      if (c >= kItemRing) room = cross_wait(item_empty + slot, ((c / kItemRing) - 1) & 1, budget, s_abort);
      if (__any_sync(0xffffffffu, *s_abort || !room)) it.hk = -1;
      if (lane == 0 && room) {
        *ring_slot(c) = it;
        mbar_arrive(item_full + slot);
      }
      if (it.hk < 0) break;
      const CrossItem i0 = team_item(a, it, 0), i1 = team_item(a, it, 1);
      const CrossBand b0 = key_band(a, i0), b1 = key_band(a, i1);
      const int n0 = band_tiles(b0, i0.no), n1 = band_tiles(b1, i1.no), most = max(n0, n1);
      auto load_q = [&](int w, int row, uint32_t& n) {
        ok = ok && cross_wait(q_empty + w, (n & 1) ^ 1, budget, s_abort);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) return;
        if (elect_one()) {
          mbar_expect_tx(q_full + w, kChunks * (uint32_t)(a.G * a.tpt) * 128u);
          for (int ch = 0; ch < kChunks; ++ch)
            tma_load_3d(sQ + w * SL::kQBytes + ch * kBoxBytes, &maps.q, ch * 64, it.hk * a.G, row, q_full + w);
        }
        __syncwarp();
        ++n;
      };
      if (n0 > 0) load_q(0, i0.r0, qn0);
      // K of a team's next tile goes out behind V of this one, before the other team's: in the order in
      // which the products free their stages.  The next item is asked for two tiles before this one's end.
      const int ask_at = max(-1, most - 2);
#pragma unroll 1
      for (int t = -1; t < max(most, 0); ++t) {
        if (t == ask_at) claim.ask();
        if (t >= 0 && t < n0) load(&maps.v, SL::v, v_full, v_empty, 0, vn0, it.hk, i0.o0 + b0.tile(t) * kKeys);
        if (t + 1 < n0) load(&maps.k, SL::k, k_full, k_empty, 0, kn0, it.hk, i0.o0 + b0.tile(t + 1) * kKeys);
        if (t < 0 && n1 > 0) load_q(1, i1.r0, qn1);
        if (t >= 0 && t < n1) load(&maps.v, SL::v, v_full, v_empty, 1, vn1, it.hk, i1.o0 + b1.tile(t) * kKeys);
        if (t + 1 < n1) load(&maps.k, SL::k, k_full, k_empty, 1, kn1, it.hk, i1.o0 + b1.tile(t + 1) * kKeys);
      }
      number = claim.answer(budget, s_abort);
    }
    // no copy may still be landing when the CTA leaves
    if (elect_one()) {
      for (int w = 0; w < 2; ++w) {
        const uint32_t kn = w ? kn1 : kn0, vn = w ? vn1 : vn0, qn = w ? qn1 : qn0;
        if (kn > 0) mbar_wait(k_full + w, (kn - 1) & 1, kDrainBudget);
        if (vn > 0) mbar_wait(v_full + w, (vn - 1) & 1, kDrainBudget);
        if (qn > 0) mbar_wait(q_full + w, (qn - 1) & 1, kDrainBudget);
      }
    }
    __syncwarp();
  } else if (warp < 3) {
    // ------------------------------------------------------------ MMA issuers
    setmaxnreg_dec<kOtherRegs>();
    const int wg = warp - 1;        // the team whose tiles this warp multiplies
    uint32_t qn = 0, kn = 0, vn = 0;
    const uint64_t dq = uniform(sdesc_sw128(smem_u32(sQ + wg * SL::kQBytes), 16, 1024));
    const uint32_t ts = uniform(tS(wg)), to = uniform(tO(wg));
    const uint64_t dk = uniform(sdesc_sw128(smem_u32(sm + SL::k + wg * SL::kTileBytes), 16, 1024));
    const uint64_t dv = uniform(sdesc_sw128(smem_u32(sm + SL::v + wg * SL::kTileBytes), SL::kKVBox, 1024));
    bool ok = true;                 // a wait that ran out ends this warp's products
    for (uint32_t c = 0;; ++c) {
      CrossItem it;
      if (lane == 0) it = read_item(c);
      it.hk = __shfl_sync(0xffffffffu, it.hk, 0);
      if (it.hk < 0) break;
      it.no = __shfl_sync(0xffffffffu, it.no, 0);
      it.nr = __shfl_sync(0xffffffffu, it.nr, 0);
      it.p0 = __shfl_sync(0xffffffffu, it.p0, 0);
      it = team_item(a, it, wg);
      const int nt = band_tiles(key_band(a, it), it.no);
      if (nt == 0) continue;
      ok = ok && cross_wait(q_full + wg, qn & 1, budget, s_abort);
      ++qn;
      // (P(t) overwrote its S: QK(t + 1) stands behind P(t).V in this warp's order)
      auto issue_qk = [&](bool last) {
        ok = ok && cross_wait(k_full + wg, kn & 1, budget, s_abort);
        ok = __all_sync(0xffffffffu, ok);
        ++kn;
        if (!ok) return;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
            mma_ss(ts, dq + kmajor_step(k), dk + (((k >> 2) * SL::kKVBox + (k & 3) * 32) >> 4), kIdescQK, k > 0);
          mma_commit(s_full + wg);
          mma_commit(k_empty + wg);
          if (last) mma_commit(q_empty + wg);
        }
        __syncwarp();
      };
      issue_qk(nt == 1);
#pragma unroll 1
      for (int t = 0; t < nt; ++t) {
        ok = ok && cross_wait(v_ready + wg, vn & 1, budget, s_abort);
        ok = ok && cross_wait(p_full + wg, vn & 1, budget, s_abort);
        ok = __all_sync(0xffffffffu, ok);
        ++vn;
        if (ok) {
          const uint32_t first = uniform(t > 0 ? 1u : 0u);
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < kKeys / 16; ++k)
              mma_ts(to, ts + 8 * k + (k >= kKeys / 32 ? kKeys / 4 : 0), dv + vtile_step(k), kIdescPV, k > 0 ? 1u : first);
            mma_commit(v_empty + wg);
          }
          __syncwarp();
        }
        if (t + 1 < nt) issue_qk(t + 2 == nt);
      }
      ok = __all_sync(0xffffffffu, ok);
      if (ok && elect_one()) mma_commit(o_final + wg);
      __syncwarp();
    }
    if (elect_one()) {
      mma_commit(drain + wg);
      mbar_wait(drain + wg, 0, kDrainBudget);
    }
    __syncwarp();
  } else if (warp == 3) {
    // ------------------------------------------------------------ V tiles
    setmaxnreg_dec<kOtherRegs>();
    uint32_t vn0 = 0, vn1 = 0;
    bool ok = true;
    for (uint32_t c = 0;; ++c) {
      CrossItem it;
      if (lane == 0) it = read_item(c);
      it.hk = __shfl_sync(0xffffffffu, it.hk, 0);
      if (it.hk < 0) break;
      it.no = __shfl_sync(0xffffffffu, it.no, 0);
      it.nr = __shfl_sync(0xffffffffu, it.nr, 0);
      it.p0 = __shfl_sync(0xffffffffu, it.p0, 0);
      it.b = __shfl_sync(0xffffffffu, it.b, 0);
      const CrossItem i0 = team_item(a, it, 0), i1 = team_item(a, it, 1);
      const CrossBand b0 = key_band(a, i0), b1 = key_band(a, i1);
      const int n0 = band_tiles(b0, i0.no), n1 = band_tiles(b1, i1.no);
#pragma unroll 1
      for (int u = 0; u < 2 * max(n0, n1); ++u) {
        const int w = u & 1, t = u >> 1;
        if (t >= (w ? n1 : n0)) continue;
        const uint32_t n = w ? vn1 : vn0;
        vn0 += !w;
        vn1 += w;
        const int kt = w ? b1.tile(t) : b0.tile(t), left = (w ? i1.no : i0.no) - kt * kKeys;
        uint32_t bits[kWords];
        bool whole = left >= kKeys && !a.key_mask;
        if (!whole)
          whole = key_bits(a.key_mask ? a.key_mask + (size_t)it.b * a.Lk + (size_t)kt * kKeys : nullptr, left, bits);
        ok = ok && cross_wait(v_full + w, n & 1, budget, s_abort);
        ok = __all_sync(0xffffffffu, ok);
        if (ok && !whole) zero_rows<kWords, kChunks>(sm + SL::v + w * SL::kTileBytes, bits);
        __syncwarp();
        if (ok && lane == 0) mbar_arrive(v_ready + w);
      }
    }
  } else {
    // ------------------------------------------------------------ softmax
    setmaxnreg_inc<kSoftmaxRegs>();
    const int group = (warp - 4) >> 2;       // warpgroup 0 .. 3
    const int wg = group >> 1;               // team
    const int half = group & 1;              // which half of the tile's keys
    const int quad = warp & 3;               // TMEM lane quadrant of this warp
    const int row = quad * 32 + lane;
    const int pair_bar = 1 + wg * 4 + quad;  // this warp and the one with the rows' other columns
    const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
    const float ks = a.kscale;
    const float2 ks2 = make_float2(ks, ks);
    const uint32_t tSw = tS(wg) + lane_off + (kKeys / 2) * half;  // this thread's scores, and its P
    const uint32_t tOw = tO(wg) + lane_off + (D / 2) * half;
    uint32_t n = 0, other_n = 0, ic = 0;  // tiles of this and (before the item) the other team, items with a tile of this one
    // One thread takes each item from the ring and leaves it in s_cur; the team reads
    // it behind its barrier, so that all of it runs the same list even after a wait
    // has run out.
    const bool reader = half == 0 && quad == 0 && lane == 0;
    CrossItem* s_cur = reinterpret_cast<CrossItem*>(sm + SL::cur) + 2 * wg;
    uint32_t c = 1;  // items taken, of which the last but one is current at an item's end
    if (reader) s_cur[0] = read_item(0);
    named_sync(9 + wg, 256);
    for (;;) {
      CrossItem it = s_cur[~c & 1];
      if (it.hk < 0) break;
      const CrossItem other = team_item(a, it, 1 - wg);
      const int other_nt = band_tiles(key_band(a, other), other.no);
      it = team_item(a, it, wg);
      const CrossBand band = key_band(a, it);
      const int nt = band_tiles(band, it.no);
      // a row block without a valid row needs no weights: its P may hold anything,
      // since a row of P only reaches its own row of O
      const bool warp_in = __any_sync(0xffffffffu, sRow[row].x < it.nr);
      float m_run = -INFINITY, l_run = 0.f;  // l_run: this thread's columns only
      bool o_has = false;
      // The teams take turns at the exponentials, in the order (item, tile, team): left alone they
      // fall into step, exponentiate together and leave the tensor core idle meanwhile (df_cross128.cu).
      // A tile waits for the other team's last one before it in that order, but an item's first, while
      // the other team has tiles of the item, for the one before that: an end lies beside the other's
      // last tile.  While a team waits for tile m, the other one may be through with m + 2, not with m + 3:
      // that waits for the one before which this team stands.  So m's phase is told from the next of four.
      for (int t = 0; t < nt; ++t, ++n) {
        // (found while the scores are on their way)
        const int first = kKeys * band.tile(t), left = it.no - first;
        const bool cut = !seen_whole(a, it.p0, it.nr, first);
        bool part = false, live0 = true, live1 = true;  // live: whether any of this thread's columns counts in its warp
        uint32_t b0 = ~0u, b1 = ~0u;
        if (a.key_mask || left < kKeys || cut) {
          uint32_t bits[kWords];
          part = !key_bits(a.key_mask ? a.key_mask + (size_t)it.b * a.Lk + first : nullptr, left, bits) || cut;
          b0 = half ? bits[kWords / 2] : bits[0];
          b1 = half ? bits[kWords / 2 + 1] : bits[1];
          if (cut) {
            const int p = it.p0 + sRow[row].x, mine = first + (kKeys / 2) * half;
            b0 &= seen_bits(a, p, mine);
            b1 &= seen_bits(a, p, mine + 32);
            live0 = __any_sync(0xffffffffu, b0 != 0);
            live1 = __any_sync(0xffffffffu, b1 != 0);
          }
        }
        cross_wait(s_full + wg, n & 1, budget, s_abort);
        __syncwarp();
        tc_fence_after();
        if (warp_in) {
          uint32_t r0[32], r1[32];
          tmem_ld32(tSw, r0);
          tmem_ld32(tSw + 32, r1);
          tmem_ld_wait2(r0, r1);
          if (part) {
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              if (!((b0 >> j) & 1u)) r0[j] = 0xff800000u;  // -infinity
              if (!((b1 >> j) & 1u)) r1[j] = 0xff800000u;
            }
          }
          // row maximum of the raw scores (the scale is positive)
          float mx0 = -INFINITY, mx1 = -INFINITY, mx2 = -INFINITY, mx3 = -INFINITY;
#pragma unroll
          for (int j = 0; j < 32; j += 4) {
            mx0 = fmax3(mx0, __uint_as_float(r0[j]), __uint_as_float(r0[j + 1]));
            mx1 = fmax3(mx1, __uint_as_float(r0[j + 2]), __uint_as_float(r0[j + 3]));
            mx2 = fmax3(mx2, __uint_as_float(r1[j]), __uint_as_float(r1[j + 1]));
            mx3 = fmax3(mx3, __uint_as_float(r1[j + 2]), __uint_as_float(r1[j + 3]));
          }
          const float mine = fmaxf(fmaxf(mx0, mx1), fmaxf(mx2, mx3));
          float* slot = sMax + ((n & 1) * 4 + wg * 2) * 128 + row;
          slot[half * 128] = mine;
          named_sync(pair_bar, 64);
          const float mt = fmaxf(mine, slot[(1 - half) * 128]) * ks - kBelow<BF16>;
          // the base of the exponentials moves only when it would grow by more
          // than 2^8: numerator and denominator share it, so the result is exact
          float rescale = 1.f;
          const bool rebase = mt > m_run + 8.f;
          if (rebase) {
            rescale = ex2(m_run - mt);
            m_run = mt;
            l_run *= rescale;
          }
          const int before = (int)other_n + min(t + wg, other_nt) - (t == 0 && other_nt > 0 ? 2 : 1);  // the tile to wait for
          if (before >= 0) cross_wait(exp_done + 4 * (1 - wg) + (before & 3), (before >> 2) & 1, budget, s_abort);
          __syncwarp();
          const float shift = m_run == -INFINITY ? INFINITY : m_run;  // no finite score yet: every p is 0
          const float2 nshift = make_float2(-shift, -shift);
          float2 acc0 = make_float2(0.f, 0.f), acc1 = acc0;
          auto exp_of = [&](const uint32_t (&r)[32], uint32_t to) {
            uint32_t w[16];
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
              const float2 z0 = fma2(make_float2(__uint_as_float(r[2 * e]), __uint_as_float(r[2 * e + 1])), ks2, nshift);
              const float2 z1 =
                  fma2(make_float2(__uint_as_float(r[2 * e + 2]), __uint_as_float(r[2 * e + 3])), ks2, nshift);
              const float2 p0 = make_float2(ex2(z0.x), ex2(z0.y)), p1 = make_float2(ex2(z1.x), ex2(z1.y));
              acc0 = add2(acc0, p0);
              acc1 = add2(acc1, p1);
              w[e] = BF16 ? pack_bf16x2(p0.x, p0.y) : pack_f16x2(p0.x, p0.y);
              w[e + 1] = BF16 ? pack_bf16x2(p1.x, p1.y) : pack_f16x2(p1.x, p1.y);
            }
            tmem_st16(to, w);
          };
          auto zeros = [&](uint32_t to) {
            uint32_t w[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) w[e] = 0u;
            tmem_st16(to, w);
          };
          // (P's 16 columns of a chunk fall on scores that are in registers)
          if (live0) {
            exp_of(r0, tSw);
          } else {
            zeros(tSw);
          }
          if (live1) {
            exp_of(r1, tSw + 16);
          } else {
            zeros(tSw + 16);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(exp_done + 4 * wg + (n & 3));
          l_run += (acc0.x + acc1.x) + (acc0.y + acc1.y);
          if (o_has && __any_sync(0xffffffffu, rebase)) {
            uint32_t r[16];
#pragma unroll 1
            for (int h = 0; h < D / 2; h += 16) {
              tmem_ld16(tOw + h, r);
              tmem_ld_wait(r);
#pragma unroll
              for (int e = 0; e < 16; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * rescale);
              tmem_st16(tOw + h, r);
            }
          }
          tmem_st_wait();
        } else {
          // the same hand-off without the work
          __syncwarp();
          if (lane == 0) mbar_arrive(exp_done + 4 * wg + (n & 3));
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full + wg);
        o_has = true;
      }
      // ---- the item's end
      if (reader) s_cur[c & 1] = read_item(c);  // the next one
      ++c;
      sML[group * 128 + row] = make_float2(m_run, l_run);
      if (nt > 0) cross_wait(o_final + wg, ic++ & 1, budget, s_abort);
      named_sync(pair_bar, 64);
      tc_fence_after();
      const float l = l_run + sML[(group ^ 1) * 128 + row].y;
      // (-infinity: without a key that counts; what O holds then comes to nothing)
      const float inv = l != 0.f ? rcp(l) : 0.f;
      // (what only the results' places need is formed again here: held over the loop
      // above, it would spill there)
      const CrossItem end = team_item(a, s_cur[c & 1], wg);
      uint32_t tid;
      asm volatile("mov.u32 %0, %%tid.x;" : "=r"(tid));
      const int2 place = sRow[tid & 127];
      const size_t row0 = (size_t)end.r0 * a.H + (size_t)end.hk * a.G;
      const int rel = place.x < end.nr && *s_abort == 0 ? place.y : -1;
      const int c0 = (D / 2) * half;
      if (warp_in && c0 < a.d)
        store_own<BF16, T>(args, sm + SL::stage + ((tid >> 5) - 4) * kRowStage, tOw, inv, nt == 0 || l == 0.f, rel, row0, c0);
      if (args.lse && c0 == 0 && rel >= 0) args.lse[row0 + rel] = l != 0.f ? (m_run + lg2(l)) * kLn2 : -INFINITY;
      tc_fence_before();
      named_sync(9 + wg, 256);  // every thread has read sML and s_cur[c & 1], and the next item is there
      other_n += other_nt;
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
  if (threadIdx.x == 0) cross_report(s_abort, a.status);
}

template <bool BF16>
cudaError_t launch(const FwdArgs& a, const FwdMaps& maps, int grid, cudaStream_t s) {
  auto kernel = self128_kernel<BF16>;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = prepare_kernel((const void*)kernel, (int)TeamSmem::alloc, kRegs, &done);
  return e != cudaSuccess ? e : launch_clusters(kernel, a, maps, grid, kThreads, TeamSmem::alloc, s);
}

}  // namespace

cudaError_t launch_self128(const FwdArgs& a, const FwdMaps& maps, bool bf16, int grid, cudaStream_t s) {
  return bf16 ? launch<true>(a, maps, grid, s) : launch<false>(a, maps, grid, s);
}

}  // namespace dfa
