// Cross attention, forward, head sizes 72 to 128 (df_cross64.cu: to 64, with the
// conventions of both): queries [B, Lq] or packed, keys and values of another
// length [B, Lk] or packed, query heads that share key heads, on tcgen05 (bf16 /
// fp16 I/O, fp32 accumulation and softmax).
//
//   s_ij = scale q_i.k_j,  o_i = sum_j exp(s_ij - lse_i) v_j,
//   lse_i = log sum_j exp s_ij          over the valid keys j of i's sequence;
// a row without a valid key gets zeros and lse = -inf.
//
// One CTA per SM takes query tiles (128 rows, df_cross.cuh) in turn.  The key
// tiles (128 keys) of an item alternate between two teams of eight softmax warps
// that share nothing until the item's end: each has its own (max, sum, O), its own
// K and V stages, tensor-memory columns and MMA-issuing thread, so that the tensor
// core works for one while the other exponentiates.
//   warp 0       finds the items and loads Q, K and V by TMA;
//   warps 1, 2   issue S = Q.K^T and O += P.V for team 0 and 1;
//   warp 3       per V tile: zeroes the rows of keys that do not count, hands it on;
//   warps 4-19   softmax: a row's scores are shared by two threads (a half of the
//                columns each), which exchange their maxima through shared memory;
//                P (rounded to the I/O type) overwrites the scores it came from.
// Keys that do not count (a tail tile's rows behind the sequence, key_mask) get
// weight 0 by selection, not by arithmetic, and their rows of V are zeroed in
// shared memory before P.V, so that whatever they hold (NaN, infinities, the
// next sequence) stays out.  Warps without a valid row skip the softmax.
//
// Few query tiles, long keys: a cluster of CTAs shares one item, each with a
// part of the key tiles; the partial (max, sum, O) are joined through
// distributed shared memory, so no workspace and no second launch is needed.
//
// Measured (GB300): 19 x 8 heads, 2048 queries x 8192 keys, d = 128, bf16: 943 to
// 959 us, 1361 to 1384 TFLOP/s.  A tile of 128 x 128 scores takes about 1800 cycles of an SM, of
// which its products are 1034; the rest is the chain S, softmax, P.V, next S of
// each team, which two teams do not fill (a third has no tensor memory).  Two CTAs
// of one team each per SM, whose ends overlap better but which cannot take turns,
// took 1094 us where this layout took 1034.  An item's end costs about 5000 cycles:
// its code has left the instruction caches by then, so it is kept short.
//
// SELF: causal attention with a window and sinks where there is little of it (df_self128.cu: more),
// as in df_cross64.cu; 32 columns that no row of a warp sees get no exponentials.  Measured:
// 8 heads, one sequence of 4096 tokens, bf16: 35 us, 980 TFLOP/s of what is seen; 4 of 1024: 22 us.
#include "df_cross_fwd.cuh"

namespace dfa {

namespace {

using namespace ptx;

constexpr int kThreads = 640, kSoftmaxThreads = 512;
// registers per thread: launched, and after the split (softmax, others)
constexpr int kRegs = 96, kSoftmaxRegs = 104, kOtherRegs = 64;
static_assert(kSoftmaxThreads * kSoftmaxRegs + 128 * kOtherRegs <= kThreads * kRegs, "setmaxnreg.inc must not wait");
constexpr uint32_t kItemRing = 4;

struct FwdSmem {
  static constexpr int D = 128;
  static constexpr int kChunks = D / 64;
  static constexpr int kKeys = kFwdKeys;
  static constexpr int kQBufs = 2;   // Q tiles in flight
  static constexpr uint32_t kQBytes = kChunks * kBoxBytes;
  static constexpr uint32_t kKVBox = kKeys * 128;                   // a 64-column box of a key tile
  static constexpr uint32_t kTileBytes = kChunks * kKVBox;
  static constexpr uint32_t q = 0;                                  // [kQBufs][Q tile]
  static constexpr uint32_t k = q + kQBufs * kQBytes;               // [2 teams][K tile]
  static constexpr uint32_t v = k + 2 * kTileBytes;       // the same of V
  static constexpr uint32_t ml = v + 2 * kTileBytes;      // float2 (max, sum) [4 warpgroups][128]
  static constexpr uint32_t mx = ml + 4 * 128 * 8;                  // float [2 tiles][4 warpgroups][128]: row maxima
  static constexpr uint32_t mj = mx + 2 * 4 * 128 * 4;              // float4 [128]: a cluster's (max, sum)
  static constexpr uint32_t rows = mj + 128 * 16;                   // int2 [128]: a row's token, and its place from the tile's first
  static constexpr uint32_t stage = rows + 128 * 8;                  // [16 warps] rows on their way out
  static constexpr uint32_t bars = stage + 16 * kRowStage;
  // q_full, q_empty [2]; k_full, k_empty, v_full, v_ready, v_empty [2];
  // s_full, p_full, exp_done, o_final, drain [2]; item_full, item_empty; claim
  static constexpr int kBars = 24 + 2 * (int)kItemRing + 1;
  static constexpr uint32_t ring = (bars + kBars * 8 + 15) & ~15u;  // CrossItem slots of 32 bytes
  static constexpr uint32_t cur = ring + 32 * kItemRing;            // the softmax threads' current item
  static constexpr uint32_t claim = cur + 64;                       // 16 bytes
  static constexpr uint32_t misc = claim + 16;                      // abort flag, tmem slot
  static constexpr uint32_t bytes = misc + 16;
  static constexpr uint32_t alloc = bytes + 1024;
  static_assert(alloc <= 232448, "shared memory of one CTA");
  // the join of a cluster: O [128][D] fp32 over the (then idle) K and V tiles
  static_assert(128 * D * 4 <= 4 * kTileBytes, "O fits over K and V");
};

// 32 columns of a warp's rows from the two teams' O: o = a fa + b fb, rounded, and
// (out_lo) what that rounding dropped.  A step of 16 columns at a time changes hands
// through 1 KB of shared memory, so that rows go out as 32 bytes each.  (A short
// loop: code that runs once per item has left the instruction caches by then.)
template <bool BF16, typename T>
__device__ __forceinline__ void store_merged(const FwdArgs& args, uint8_t* stage, uint32_t ta, uint32_t tb, float fa,
                                             float fb, bool empty, int rel, size_t row0, int col) {
  const int lane = threadIdx.x & 31, d = args.c.d;
  const float2 fa2 = make_float2(fa, fa), fb2 = make_float2(fb, fb);
  uint8_t* mine = stage + lane * 32 + 16 * ((lane >> 2) & 1);  // the row's first 8 columns; the others at ^ 16
#pragma unroll 1
  for (int end = min(col + 32, d); col < end; col += 16, ta += 16, tb += 16) {
    uint32_t ra[16], rb[16];
    tmem_ld16(ta, ra);
    tmem_ld16(tb, rb);
    tmem_ld_wait(ra);
    tmem_ld_wait(rb);
    uint32_t hi[8], lo[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float2 b = mul2(make_float2(__uint_as_float(rb[2 * e]), __uint_as_float(rb[2 * e + 1])), fb2);
      if (fb == 0.f) b = make_float2(0.f, 0.f);  // (its O may hold anything)
      const float2 o = fma2(make_float2(__uint_as_float(ra[2 * e]), __uint_as_float(ra[2 * e + 1])), fa2, b);
      hi[e] = empty ? 0u : pack2<BF16>(o.x, o.y);
      const T* t = reinterpret_cast<const T*>(&hi[e]);
      lo[e] = empty ? 0u : pack2<BF16>(o.x - IO<T>::to_f(t[0]), o.y - IO<T>::to_f(t[1]));
    }
    const size_t at = row0 * d + col;
#pragma unroll
    for (int pass = 0; pass < 2; ++pass) {
      if (pass == 1 && !args.out_lo) break;
      const uint32_t (&w)[8] = pass ? lo : hi;
      *reinterpret_cast<uint4*>(mine) = make_uint4(w[0], w[1], w[2], w[3]);
      *reinterpret_cast<uint4*>((uintptr_t)mine ^ 16) = make_uint4(w[4], w[5], w[6], w[7]);
      __syncwarp();
      T* dst = static_cast<T*>(pass ? args.out_lo : args.out) + at + 8 * (lane & 1);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = 16 * i + (lane >> 1);
        const uint4 v = *reinterpret_cast<const uint4*>(stage + r * 32 + 16 * ((lane ^ (r >> 2)) & 1));
        const int to = __shfl_sync(0xffffffffu, rel, r);
        if (to >= 0 && col + 8 * (lane & 1) < d) *reinterpret_cast<uint4*>(dst + (size_t)to * d) = v;
      }
      __syncwarp();
    }
  }
}

// One step of 16 columns of one row, not rounded, for a cluster's join.
__device__ __forceinline__ void keep_merged(float* dst, uint32_t ta, uint32_t tb, float fa, float fb, int row, int col) {
  uint32_t ra[16], rb[16];
  tmem_ld16(ta, ra);
  tmem_ld16(tb, rb);
  tmem_ld_wait(ra);
  tmem_ld_wait(rb);
#pragma unroll
  for (int e = 0; e < 16; e += 4) {
    float o[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      o[k] = (fa > 0.f ? __uint_as_float(ra[e + k]) * fa : 0.f) + (fb > 0.f ? __uint_as_float(rb[e + k]) * fb : 0.f);
    *reinterpret_cast<float4*>(dst + o_piece<FwdSmem::D>(row, (col + e) / 4)) = make_float4(o[0], o[1], o[2], o[3]);
  }
}

template <bool BF16, bool SELF>
__global__ void __launch_bounds__(kThreads, 1) cross128_kernel(const FwdArgs args, const __grid_constant__ FwdMaps maps) {
  using SL = FwdSmem;
  constexpr int D = SL::D;
  constexpr int kChunks = SL::kChunks;
  constexpr int kKeys = SL::kKeys, kWords = kKeys / 32;
  constexpr uint32_t kQBufs = SL::kQBufs;
  constexpr uint32_t kIdescQK = idesc_f16(128, kKeys, BF16 ? 1 : 0, 0, 0);
  constexpr uint32_t kIdescPV = idesc_f16(128, D, BF16 ? 1 : 0, 0, 1);
  using T = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
  // Tensor-memory columns of a team: S, of which P takes the first half of each
  // half, then O.
  static_assert(tmem_region_fits(256 + kKeys, D, 512), "S and O of two teams in 512 columns");
  constexpr uint32_t kItemReaders = 4;  // two issuers, warp 3, the softmax threads' reader

  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t* sQ = sm + SL::q;
  float2* sML = reinterpret_cast<float2*>(sm + SL::ml);
  float* sMax = reinterpret_cast<float*>(sm + SL::mx);
  float4* sJoin = reinterpret_cast<float4*>(sm + SL::mj);
  int2* sRow = reinterpret_cast<int2*>(sm + SL::rows);
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + SL::bars);
  uint64_t* q_full = bars;
  uint64_t* q_empty = bars + 2;
  uint64_t* k_full = bars + 4;          // [team], as the next four
  uint64_t* k_empty = k_full + 2;
  uint64_t* v_full = k_empty + 2;
  uint64_t* v_ready = v_full + 2;   // landed, rows that do not count zeroed
  uint64_t* v_empty = v_ready + 2;
  uint64_t* s_full = v_empty + 2;   // [team], as the next four: S computed
  uint64_t* p_full = s_full + 2;        // its eight warps have stored P
  uint64_t* exp_done = p_full + 2;     // its eight warps are through with a tile's exponentials
  uint64_t* o_final = exp_done + 2;     // every P.V of the item done
  uint64_t* drain = o_final + 2;
  uint64_t* item_full = drain + 2;
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
      mbar_init(q_empty + b, 2);
      mbar_init(s_full + b, 1);
      mbar_init(p_full + b, 8);
      mbar_init(exp_done + b, 8);
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
    setmaxnreg_dec<kOtherRegs>();
    // (the whole warp runs every step, and one lane of it issues)
    TileWalk<SELF> walk;
    if (SELF) walk.together = heads_together(a);
    TileClaim claim = {claim_bar, reinterpret_cast<uint4*>(sm + SL::claim)};
    uint32_t kn0 = 0, kn1 = 0, vn0 = 0, vn1 = 0;  // tiles loaded for each team
    uint32_t qc = 0;
    int mask_b = -1, mask_n = 0;  // the last masked row measured
    bool ok = true;               // a wait ran out: nothing is loaded after it
    long long number = blockIdx.x / args.splits;
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
        const uint32_t qb = qc % kQBufs;
        ok = ok && cross_wait(q_empty + qb, ((qc / kQBufs) & 1) ^ 1, budget, s_abort);
        ok = __all_sync(0xffffffffu, ok);
        if (ok) {
          if (elect_one()) {
            mbar_expect_tx(q_full + qb, kChunks * (uint32_t)(a.G * a.tpt) * 128u);
            for (int ch = 0; ch < kChunks; ++ch)
              tma_load_3d(sQ + qb * SL::kQBytes + ch * kBoxBytes, &maps.q, ch * 64, it.hk * a.G, it.r0, q_full + qb);
          }
          __syncwarp();
          ++qc;
        }
      }
      // K(t + 2) goes out behind V(t), before V(t + 1): in the order in which the
      // products free their stages.
      // The next item is asked for two tiles before this one's end: early enough to be
      // answered by then, late enough to leave it to a CTA that is through sooner.
      const int ask_at = args.splits > 1 ? INT_MAX : max(-2, nt - 2);
      auto row_at = [&](int t) { return it.o0 + (SELF ? band.tile(t0 + t) : t0 + t) * kKeys; };
#pragma unroll 1
      for (int t = -2; t < max(nt, -1); ++t) {
        const int w = t & 1;
        if (t == ask_at) claim.ask();
        if (t >= 0) load(&maps.v, SL::v, v_full, v_empty, w, w ? vn1 : vn0, it.hk, row_at(t));
        if (t + 2 < nt) load(&maps.k, SL::k, k_full, k_empty, w, w ? kn1 : kn0, it.hk, row_at(t + 2));
      }
      number = args.splits > 1 ? -1 : claim.answer(budget, s_abort);
    }
    // no copy may still be landing when the CTA leaves
    if (elect_one()) {
      for (int w = 0; w < 2; ++w) {
        const uint32_t kn = w ? kn1 : kn0, vn = w ? vn1 : vn0;
        if (kn > 0) mbar_wait(k_full + w, (kn - 1) & 1, kDrainBudget);
        if (vn > 0) mbar_wait(v_full + w, (vn - 1) & 1, kDrainBudget);
      }
#pragma unroll 1
      for (uint32_t n = qc > kQBufs ? qc - kQBufs : 0; n < qc; ++n)
        mbar_wait(q_full + n % kQBufs, (n / kQBufs) & 1, kDrainBudget);
    }
    __syncwarp();
  } else if (warp < 3) {
    // ------------------------------------------------------------ MMA issuers
    setmaxnreg_dec<kOtherRegs>();
    const int wg = warp - 1;        // the team whose tiles (t = wg, wg + 2, ...) this warp multiplies
    uint32_t qc = 0, kn = 0, vn = 0;
    const uint32_t q_addr = smem_u32(sQ);
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
      if (SELF) it.p0 = __shfl_sync(0xffffffffu, it.p0, 0);
      int t0;
      const CrossBand band = band_of(it);
      const int nt = part(it, band, &t0);
      if (nt == 0) continue;
      const uint32_t qb = qc % kQBufs;
      ok = ok && cross_wait(q_full + qb, (qc / kQBufs) & 1, budget, s_abort);
      const uint64_t dq = uniform(sdesc_sw128(q_addr + qb * SL::kQBytes, 16, 1024));
      ++qc;
      // (P(t) overwrote its S: QK(t + 2) stands behind P(t).V in this warp's order)
      auto issue_qk = [&]() {
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
        }
        __syncwarp();
      };
      if (wg < nt) issue_qk();
#pragma unroll 1
      for (int t = wg; t < nt; t += 2) {
        ok = ok && cross_wait(v_ready + wg, vn & 1, budget, s_abort);
        ok = ok && cross_wait(p_full + wg, vn & 1, budget, s_abort);
        ok = __all_sync(0xffffffffu, ok);
        ++vn;
        if (ok) {
          const uint32_t first = uniform(t >= 2 ? 1u : 0u);
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < kKeys / 16; ++k)
              mma_ts(to, ts + 8 * k + (k >= kKeys / 32 ? kKeys / 4 : 0), dv + vtile_step(k), kIdescPV, k > 0 ? 1u : first);
            mma_commit(v_empty + wg);
          }
          __syncwarp();
        }
        if (t + 2 < nt) issue_qk();
      }
      ok = __all_sync(0xffffffffu, ok);
      if (ok && elect_one()) {
        // (a team without a tile waits for nothing here: its issuer may be items ahead)
        if (wg < nt) mma_commit(o_final + wg);
        mma_commit(q_empty + qb);
      }
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
      if (SELF) it.p0 = __shfl_sync(0xffffffffu, it.p0, 0);
      it.b = __shfl_sync(0xffffffffu, it.b, 0);
      int t0;
      const CrossBand band = band_of(it);
      const int nt = part(it, band, &t0);
#pragma unroll 1
      for (int t = 0; t < nt; ++t) {
        const int w = t & 1;
        const uint32_t n = w ? vn1 : vn0;
        vn0 += !w;
        vn1 += w;
        const int kt = SELF ? band.tile(t0 + t) : t0 + t, left = it.no - kt * kKeys;
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
    uint32_t n = 0, other_n = 0, ic = 0;  // tiles of this and the other team, items with a tile of this one
    // One thread takes each item from the ring and leaves it in s_cur; all 512 read
    // it behind their barrier, so that they run the same list even after a wait
    // has run out.
    const bool reader = warp == 4 && lane == 0;
    uint32_t c = 1;  // items taken, of which the last but one is current at an item's end
    if (reader) s_cur[0] = read_item(0);
    named_sync(9, kSoftmaxThreads);
    for (;;) {
      const CrossItem it = s_cur[~c & 1];
      if (it.hk < 0) break;
      int t0;
      const CrossBand band = band_of(it);
      const int nt = part(it, band, &t0);
      // a row block without a valid row needs no weights: its P may hold anything,
      // since a row of P only reaches its own row of O
      const bool warp_in = __any_sync(0xffffffffu, sRow[row].x < it.nr);
      float m_run = -INFINITY, l_run = 0.f;  // l_run: this thread's columns only
      bool o_has = false;
      // The teams take turns at the exponentials, in the order of the tiles: left
      // alone they fall into step, exponentiate together and leave the tensor core
      // idle meanwhile (19 x 8 heads, 2048 x 8192: 944 us with turns, 1066 without).
      // Within an item neither gets two phases ahead of the other's wait; at its end
      // both meet.
      // tile t = 2 i + w of the item is team w's i-th: the other one's t - 1 has the
      // number other_n + (t - 1) / 2 among its own
      for (int t = wg; t < nt; t += 2, ++n) {
        cross_wait(s_full + wg, n & 1, budget, s_abort);
        __syncwarp();
        tc_fence_after();
        if (warp_in) {
          uint32_t r0[32], r1[32];
          tmem_ld32(tSw, r0);
          tmem_ld32(tSw + 32, r1);
          tmem_ld_wait2(r0, r1);
          const int kt = SELF ? band.tile(t0 + t) : t0 + t, left = it.no - kt * kKeys;
          const bool cut = SELF && !seen_whole(a, it.p0, it.nr, kt * kKeys);
          bool live0 = true, live1 = true;  // SELF: whether any of this thread's columns counts in its warp
          if (a.key_mask || left < kKeys || cut) {
            uint32_t bits[kWords];
            const bool all =
                key_bits(a.key_mask ? a.key_mask + (size_t)it.b * a.Lk + (size_t)kt * kKeys : nullptr, left, bits);
            if (!all || cut) {
              uint32_t b0 = half ? bits[kWords / 2] : bits[0], b1 = half ? bits[kWords / 2 + 1] : bits[1];
              if (SELF && cut) {
                const int p = it.p0 + sRow[row].x, first = kt * kKeys + (kKeys / 2) * half;
                b0 &= seen_bits(a, p, first);
                b1 &= seen_bits(a, p, first + 32);
                live0 = __any_sync(0xffffffffu, b0 != 0);
                live1 = __any_sync(0xffffffffu, b1 != 0);
              }
#pragma unroll
              for (int j = 0; j < 32; ++j) {
                if (!((b0 >> j) & 1u)) r0[j] = 0xff800000u;  // -infinity
                if (!((b1 >> j) & 1u)) r1[j] = 0xff800000u;
              }
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
          if (t > 0) cross_wait(exp_done + (1 - wg), (other_n + ((t - 1) >> 1)) & 1, budget, s_abort);
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
          if (!SELF || live0) {
            exp_of(r0, tSw);
          } else {
            zeros(tSw);
          }
          if (!SELF || live1) {
            exp_of(r1, tSw + 16);
          } else {
            zeros(tSw + 16);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(exp_done + wg);
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
          if (lane == 0) mbar_arrive(exp_done + wg);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full + wg);
        o_has = true;
      }
      // ---- the item's end: both teams' states together
      if (reader) s_cur[c & 1] = read_item(c);  // the next one
      ++c;
      if (wg < nt) cross_wait(o_final + wg, ic++ & 1, budget, s_abort);
      __syncwarp();
      tc_fence_after();
      sML[group * 128 + row] = make_float2(m_run, l_run);
      // (each thread goes on to read both teams' O, and has waited for its own one's P.V
      // only: the barrier has to order the other's tensor memory too)
      tc_fence_before();
      named_sync(9, kSoftmaxThreads);
      tc_fence_after();
      const float2 s0 = sML[row], s1 = sML[128 + row], s2 = sML[256 + row], s3 = sML[384 + row];
      const float m = fmaxf(s0.x, s2.x);
      // a team without a tile, or without a valid key, has -infinity: its O is not read
      const float f0 = s0.x != -INFINITY ? ex2(s0.x - m) : 0.f;
      const float f1 = s2.x != -INFINITY ? ex2(s2.x - m) : 0.f;
      const float l = (s0.y + s1.y) * f0 + (s2.y + s3.y) * f1;
      const bool alone = args.splits == 1;
      const float inv = !alone ? 1.f : (l != 0.f ? rcp(l) : 0.f);
      // (what only the results' places need is formed again here: held over the loop
      // above, it would spill there)
      const CrossItem end = s_cur[c & 1];
      uint32_t tid;
      asm volatile("mov.u32 %0, %%tid.x;" : "=r"(tid));
      const int end_row = tid & 127;
      const int2 place = sRow[end_row];
      const size_t row0 = (size_t)end.r0 * a.H + (size_t)end.hk * a.G;
      const int rel = place.x < end.nr && *s_abort == 0 ? place.y : -1;
      const int c0 = (((int)tid - 128) >> 7) * (D / 4);  // each of a row's four threads writes a quarter of its columns
      const uint32_t ta = tO(0) + ((tid & 96u) << 16), tb = ta + 256u;
      if (alone) {
        if (warp_in && c0 < a.d)
          store_merged<BF16, T>(args, sm + SL::stage + ((tid >> 5) - 4) * kRowStage, ta + c0, tb + c0, f0 * inv, f1 * inv,
                                nt == 0, rel, row0, c0);
        if (args.lse && c0 == 0 && rel >= 0) args.lse[row0 + rel] = l != 0.f ? (m + lg2(l)) * kLn2 : -INFINITY;
      } else {
        float* sO = reinterpret_cast<float*>(sm + SL::k);  // K and V are idle by then
        if (warp_in) {
#pragma unroll 1
          for (int col = c0; col < c0 + D / 4; col += 16)
            keep_merged(sO, ta + col, tb + col, f0, f1, end_row, col);
        }
        if (c0 == 0) sJoin[end_row] = make_float4(m, l, 0.f, 0.f);
      }
      tc_fence_before();
      named_sync(9, kSoftmaxThreads);  // every thread has read sML and s_cur[c & 1]
      other_n += wg ? (nt + 1) >> 1 : nt >> 1;
      if (!alone) break;  // one item per cluster; s_cur stays for the join
    }
  }

  if (args.splits > 1) {
    cluster_sync();
    if (warp >= 4 && s_cur->hk >= 0)
      join_cluster<T, D>(args, *s_cur, rank, (int)threadIdx.x - 128, kSoftmaxThreads, smem_u32(sJoin), smem_u32(sm + SL::k));
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
  auto kernel = cross128_kernel<BF16, SELF>;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = prepare_kernel((const void*)kernel, (int)FwdSmem::alloc, kRegs, &done);
  return e != cudaSuccess ? e : launch_clusters(kernel, a, maps, grid, kThreads, FwdSmem::alloc, s);
}

}  // namespace

cudaError_t launch_cross128(const FwdArgs& a, const FwdMaps& maps, bool bf16, bool self, int grid, cudaStream_t s) {
  if (self) return bf16 ? launch<true, true>(a, maps, grid, s) : launch<false, true>(a, maps, grid, s);
  return bf16 ? launch<true, false>(a, maps, grid, s) : launch<false, false>(a, maps, grid, s);
}

}  // namespace dfa
