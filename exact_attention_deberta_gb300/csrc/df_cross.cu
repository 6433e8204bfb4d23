// Cross attention, forward: queries [B, Lq] or packed, keys and values of
// another length [B, Lk] or packed, query heads that share key heads, on
// tcgen05 (bf16 / fp16 I/O, fp32 accumulation and softmax).
//
//   s_ij = scale q_i.k_j,  o_i = sum_j exp(s_ij - lse_i) v_j,
//   lse_i = log sum_j exp s_ij          over the valid keys j of i's sequence;
// a row without a valid key gets zeros and lse = -inf.
//
// One CTA per SM takes query tiles (128 rows, df_cross.cuh) in turn.  The key
// tiles (128 keys) of an item alternate between two softmax warpgroups with
// independent (max, sum, O) states, so that the tensor core works for one while
// the other exponentiates; the two are merged at the end of the item.
//   warp 0      finds the items and loads Q (two buffers) and K, V (a ring of
//               buffers, K(t) and V(t) in turn, each freed by the product that
//               read it) by TMA;
//   warp 1      issues S = Q.K^T into tensor memory (three score buffers at
//               D = 64, two at D = 128 where it also issues the P.V);
//   warps 3, 2  at D = 64 issue O_w += P.V for warpgroup 0 and 1;
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
#include "df_cross.cuh"

#include <cudaTypedefs.h>
#include <math.h>

#include <algorithm>
#include <type_traits>

namespace dfa {

namespace {

using namespace ptx;

constexpr int kThreads = 384;
constexpr uint32_t kItemRing = 4;

struct FwdArgs {
  CrossArgs c;
  void* out;
  void* out_lo;  // or NULL
  float* lse;    // or NULL
  int splits;    // CTAs per item (cluster size)
};

struct FwdMaps {
  CUtensorMap q, k, v;
};

template <int D>
struct FwdSmem {
  static constexpr int kChunks = D / 64;
  static constexpr int kRing = D == 64 ? 10 : 4;  // K and V tiles in flight
  static constexpr uint32_t kTileBytes = kChunks * kBoxBytes;
  static constexpr uint32_t q = 0;                                  // [2][Q tile]
  static constexpr uint32_t kv = q + 2 * kTileBytes;                // [kRing][K or V tile]
  static constexpr uint32_t ml = kv + kRing * kTileBytes;           // float4 [2 warpgroups, their join][128]
  static constexpr uint32_t bars = ml + 3 * 128 * 16;
  // q_full[2], q_empty[2], full[R], empty[R], s_full[3], p_full[4], buf_free[3],
  // o_final, drain[3], item_full, item_empty
  static constexpr int kBars = 4 + 2 * kRing + 3 + 4 + 3 + 1 + 3 + 2 * (int)kItemRing;
  static constexpr uint32_t ring = (bars + kBars * 8 + 15) & ~15u;  // CrossItem slots of 32 bytes
  static constexpr uint32_t cur = ring + 32 * kItemRing;            // the softmax warpgroups' current item
  static constexpr uint32_t misc = cur + 32;                        // abort flag, tmem slot
  static constexpr uint32_t bytes = misc + 16;
  static constexpr uint32_t alloc = bytes + 1024;
  static_assert(alloc <= 232448, "shared memory of one CTA");
  // the join of a cluster: O [128][D] fp32 over the (then idle) K/V ring
  static_assert(128 * D * 4 <= kRing * kTileBytes, "O fits over the ring");
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ float4 ld_cluster(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

constexpr float kLn2 = 0.69314718055994531f;

// Word offset of a 4-column piece of a row in a cluster's join buffer (pieces
// rotated by row, so that the rows of a warp fall in different banks).
template <int D>
__device__ __forceinline__ int o_piece(int row, int piece) {
  return row * D + 4 * ((piece + row) % (D / 4));
}

// N consecutive output values of a row, rounded to the I/O type, and (lo) what
// that rounding dropped.
template <typename T, int N>
__device__ __forceinline__ void store_rounded(T* out, T* lo, const float (&o)[N]) {
  using Vec = typename std::conditional<N == 8, uint4, uint2>::type;
  __align__(16) T h[N];
#pragma unroll
  for (int e = 0; e < N; ++e) h[e] = IO<T>::from_f(o[e]);
  *reinterpret_cast<Vec*>(out) = *reinterpret_cast<const Vec*>(h);
  if (lo) {
    __align__(16) T l[N];
#pragma unroll
    for (int e = 0; e < N; ++e) l[e] = IO<T>::from_f(o[e] - IO<T>::to_f(h[e]));
    *reinterpret_cast<Vec*>(lo) = *reinterpret_cast<const Vec*>(l);
  }
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads, 1) cross_fwd_kernel(const FwdArgs args, const __grid_constant__ FwdMaps maps) {
  using SL = FwdSmem<D>;
  constexpr int kChunks = SL::kChunks;
  constexpr uint32_t R = SL::kRing;
  constexpr uint32_t kIdescQK = idesc_f16(128, 128, BF16 ? 1 : 0, 0, 0);
  constexpr uint32_t kIdescPV = idesc_f16(128, D, BF16 ? 1 : 0, 0, 1);
  using T = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
  // D = 64: three score buffers and two O accumulators; D = 128: two and two.
  constexpr bool kTriS = D == 64;
  constexpr uint32_t kScoreBufs = kTriS ? 3u : 2u, kOFirst = 128u * kScoreBufs;
  static_assert(tmem_region_fits(kOFirst, 2u * D, 512), "scores and two O accumulators in 512 columns");
  constexpr uint32_t kItemReaders = (kTriS ? 3 : 1) + 1;  // the issuing threads, the softmax warpgroups' reader

  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t* sQ = sm + SL::q;
  uint8_t* sKV = sm + SL::kv;
  float4* sML = reinterpret_cast<float4*>(sm + SL::ml);
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + SL::bars);
  uint64_t* q_full = bars;
  uint64_t* q_empty = bars + 2;
  uint64_t* full = bars + 4;
  uint64_t* empty = full + R;
  uint64_t* s_full = empty + R;        // [3] S of the buffer computed
  uint64_t* p_full = s_full + 3;       // [wg][k & 1]: the four warps of wg stored P of its k-th tile
  uint64_t* buf_free = p_full + 4;     // [3] D = 64: the P.V that read the buffer is done
  uint64_t* o_final = buf_free + 3;    // D = 128: every P.V of the item is done
  uint64_t* drain = o_final + 1;       // [3], one per issuing thread
  uint64_t* item_full = drain + 3;
  uint64_t* item_empty = item_full + kItemRing;
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
    for (uint32_t s = 0; s < R; ++s) {
      mbar_init(full + s, 1);
      mbar_init(empty + s, 1);
    }
    for (int b = 0; b < 3; ++b) {
      mbar_init(s_full + b, 1);
      mbar_init(buf_free + b, 1);
      mbar_init(drain + b, 1);
    }
    for (int b = 0; b < 4; ++b) mbar_init(p_full + b, 4);
    mbar_init(o_final, 1);
    for (uint32_t b = 0; b < kItemRing; ++b) {
      mbar_init(item_full + b, 1);
      mbar_init(item_empty + b, kItemReaders);
    }
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
  auto tO = [&](int b) { return tmem + kOFirst + (uint32_t)D * b; };

  const unsigned long long budget = a.budget;
  int32_t* status = a.status;
  const uint32_t rank = args.splits > 1 ? cluster_rank() : 0u;
  // this CTA's key tiles [t0, t0 + nt) of an item
  auto part = [&](const CrossItem& it, int* t0) {
    const int all = (it.no + 127) >> 7;
    *t0 = (int)((long long)all * rank / args.splits);
    return (int)((long long)all * (rank + 1) / args.splits) - *t0;
  };
  // the c-th item handed out, for one thread; hk = -1 at the end or after an abort
  auto read_item = [&](uint32_t c) {
    const uint32_t slot = c % kItemRing;
    CrossItem it;
    it.r0 = it.nr = it.o0 = it.no = it.b = 0;
    it.hk = -1;
    if (cross_wait(item_full + slot, (c / kItemRing) & 1, budget, s_abort, status)) {
      it = *ring_slot(c);
      mbar_arrive(item_empty + slot);
    }
    return it;
  };

  if (warp == 0) {
    // ------------------------------------------------------------ items and loads
    setmaxnreg_dec<56>();
    TileWalk walk;
    uint32_t u = 0, qc = 0, u_issued = 0, q_issued = 0;
    const int clusters = gridDim.x / args.splits, first = blockIdx.x / args.splits;
    for (uint32_t c = 0;; ++c) {
      CrossItem it = walk.find(a, query_side(a), key_side(a), a.tpt, (long long)first + (long long)c * clusters);
      const uint32_t slot = c % kItemRing;
      bool ok = true;
      if (lane == 0) {
        if (c >= kItemRing) ok = cross_wait(item_empty + slot, ((c / kItemRing) - 1) & 1, budget, s_abort, status);
        if (*s_abort || !ok) it.hk = -1;
        if (ok) {
          *ring_slot(c) = it;
          mbar_arrive(item_full + slot);
        }
        int t0;
        const int nt = it.hk < 0 ? 0 : part(it, &t0);
        if (nt > 0) {
          const int qb = qc & 1;
          if (cross_wait(q_empty + qb, ((qc >> 1) & 1) ^ 1, budget, s_abort, status)) {
            const uint32_t box = (uint32_t)(a.G * a.tpt) * 128u;
            mbar_expect_tx(q_full + qb, kChunks * box);
            for (int ch = 0; ch < kChunks; ++ch)
              tma_load_3d(sQ + qb * SL::kTileBytes + ch * kBoxBytes, &maps.q, ch * 64, it.hk * a.G, it.r0, q_full + qb);
            q_issued = qc + 1;
          }
          ++qc;
          for (int t = 0; t < nt; ++t) {
            const int row = it.o0 + (t0 + t) * 128;
#pragma unroll
            for (int kv = 0; kv < 2; ++kv, ++u) {
              const uint32_t s = u % R;
              if (cross_wait(empty + s, ((u / R) & 1) ^ 1, budget, s_abort, status)) {
                mbar_expect_tx(full + s, SL::kTileBytes);
                for (int ch = 0; ch < kChunks; ++ch)
                  tma_load_3d(sKV + s * SL::kTileBytes + ch * kBoxBytes, kv ? &maps.v : &maps.k, ch * 64, it.hk, row,
                              full + s);
                u_issued = u + 1;
              }
            }
          }
        }
      }
      if (__shfl_sync(0xffffffffu, it.hk, 0) < 0) break;
    }
    if (lane == 0) {
      // no copy may still be landing when the CTA leaves
      for (uint32_t k = u_issued > R ? u_issued - R : 0; k < u_issued; ++k)
        mbar_wait(full + k % R, (k / R) & 1, kDrainBudget);
      for (uint32_t k = q_issued > 2 ? q_issued - 2 : 0; k < q_issued; ++k)
        mbar_wait(q_full + (k & 1), (k >> 1) & 1, kDrainBudget);
    }
  } else if (warp < 4) {
    // ------------------------------------------------------------ MMA issuers
    setmaxnreg_dec<56>();
    if (lane == 0 && (kTriS || warp == 1)) {
      const bool qk_role = warp == 1;
      const int pv_wg = warp == 3 ? 0 : 1;  // D = 64: the warpgroup whose tiles this thread multiplies
      uint32_t g = 0, qc = 0;               // key tiles and items before this one
      uint32_t pn[2] = {0, 0};              // tiles of warpgroup b whose P has been consumed
      const uint32_t kv_addr = smem_u32(sKV);
      for (uint32_t c = 0;; ++c) {
        const CrossItem it = read_item(c);
        if (it.hk < 0) break;
        int t0;
        const int nt = part(it, &t0);
        if (nt == 0) continue;
        const int qb = qc & 1;
        const uint8_t* sQb = sQ + qb * SL::kTileBytes;
        const bool q_ok = !qk_role || cross_wait(q_full + qb, (qc >> 1) & 1, budget, s_abort, status);
        ++qc;
        auto issue_qk = [&](int t) {
          const uint32_t gs = g + t, uk = 2 * gs, uv = uk + 1;
          const int sb = kTriS ? (int)(gs % 3) : (t & 1);
          bool ok = q_ok;
          if (kTriS && gs >= 3) ok = cross_wait(buf_free + sb, ((gs - 3) / 3) & 1, budget, s_abort, status) && ok;
          ok = cross_wait(full + uk % R, (uk / R) & 1, budget, s_abort, status) && ok;
          // V too: S complete then says that both tiles of t have landed, for the
          // softmax threads that zero rows of V and for the P.V after them
          ok = cross_wait(full + uv % R, (uv / R) & 1, budget, s_abort, status) && ok;
          if (ok) {
            const uint64_t dq = kmajor_desc(sQb, 0);
            const uint64_t dk = kmajor_desc(sKV + (uk % R) * SL::kTileBytes, 0);
            tc_fence_after();
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
              mma_ss(tS(sb), dq + kmajor_step(k), dk + kmajor_step(k), kIdescQK, k > 0);
            mma_commit(s_full + sb);
            mma_commit(empty + uk % R);
          }
        };
        auto issue_pv = [&](int t) {
          const int b = t & 1;
          const uint32_t gs = g + t, uv = 2 * gs + 1;
          const uint32_t k = pn[b]++;
          if (cross_wait(p_full + 2 * b + (k & 1), (k >> 1) & 1, budget, s_abort, status)) {
            const uint64_t dv = vtile_desc(kv_addr + (uv % R) * SL::kTileBytes, 0);
            tc_fence_after();
            const uint32_t tP = tS(kTriS ? (int)(gs % 3) : b);  // P(t) overwrote its S
#pragma unroll
            for (int kk = 0; kk < 128 / 16; ++kk)
              mma_ts(tO(b), tP + 8 * kk, dv + vtile_step(kk), kIdescPV, (kk > 0 || t >= 2) ? 1u : 0u);
            mma_commit(empty + uv % R);
            if (kTriS) mma_commit(buf_free + (gs % 3));
          }
        };
        if (kTriS) {
          if (qk_role) {
            for (int t = 0; t < nt; ++t) issue_qk(t);
          } else {
            for (int t = pv_wg; t < nt; t += 2) issue_pv(t);
          }
        } else {
          // P overwrites S: QK(t) follows P(t - 2).V in the same pipe
          for (int t = 0; t <= nt; ++t) {
            if (t < nt) issue_qk(t);
            if (t >= 1) issue_pv(t - 1);
          }
        }
        g += nt;
        if (qk_role) mma_commit(q_empty + qb);
        if (!kTriS) mma_commit(o_final);
      }
      uint64_t* my_drain = drain + (warp == 1 ? 0 : warp == 3 ? 1 : 2);
      mma_commit(my_drain);
      mbar_wait(my_drain, 0, kDrainBudget);
    }
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
    uint32_t sc = 0, ic = 0, own = 0, gbase = 0;  // gbase: key tiles before the item
    // One thread takes each item from the ring and leaves it in s_cur; all 256 read
    // it behind their barrier, so that they run the same list even after a wait
    // has run out.
    const bool reader = warp == 4 && lane == 0;
    uint32_t c = 0;
    if (reader) *s_cur = read_item(c++);
    named_sync(3, 256);
    for (;;) {
      const CrossItem it = *s_cur;
      if (it.hk < 0) break;
      int t0;
      const int nt = part(it, &t0);
      const bool row_in = row_tok < it.nr;
      // a row block without a valid row needs no weights: its P may hold anything,
      // since a row of P only reaches its own row of O
      const bool warp_in = __any_sync(0xffffffffu, row_in);
      float m_run = -INFINITY, l_run = 0.f;
      bool o_has = false;
      for (int t = wg; t < nt; t += 2, ++own) {
        const uint32_t G = gbase + t;
        const int sb = kTriS ? (int)(G % 3) : wg;
        const uint32_t tSw = tmem + 128u * sb + lane_off;
        // which keys of the tile count, one bit each
        const int left = it.no - (t0 + t) * 128;
        uint32_t bits[4];
        bool whole = left >= 128;
        if (a.key_mask) {
          const uint8_t* mrow = a.key_mask + (size_t)it.b * a.Lk + (size_t)(t0 + t) * 128;
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const int j = 32 * w + lane;
            bits[w] = __ballot_sync(0xffffffffu, j < left && mrow[j] != 0);
          }
          whole = (bits[0] & bits[1] & bits[2] & bits[3]) == 0xffffffffu;
        } else {
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const int n = left - 32 * w;
            bits[w] = n >= 32 ? 0xffffffffu : (n <= 0 ? 0u : (1u << n) - 1u);
          }
        }
        cross_wait(s_full + sb, kTriS ? (G / 3) & 1 : sc & 1, budget, s_abort, status);
        ++sc;
        __syncwarp();
        tc_fence_after();
        if (!whole) {
          // thread `row` of the warpgroup zeroes key row `row` of V
          uint32_t word = bits[0];
          word = quad == 1 ? bits[1] : word;
          word = quad == 2 ? bits[2] : word;
          word = quad == 3 ? bits[3] : word;
          if (!((word >> lane) & 1u)) {
            uint8_t* v = sKV + ((2 * G + 1) % R) * SL::kTileBytes + row * 128;
#pragma unroll
            for (int ch = 0; ch < kChunks; ++ch)
#pragma unroll
              for (int e = 0; e < 8; ++e)
                *reinterpret_cast<uint4*>(v + ch * kBoxBytes + 16 * e) = make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
        }
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
          if (!whole) {
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
                                 fmaxf(fmaxf(mx[4], mx[5]), fmaxf(mx[6], mx[7]))) * ks;
          // the base of the exponentials moves only when it would grow by more
          // than 2^8: numerator and denominator share it, so the result is exact
          float rescale = 1.f;
          const bool rebase = mt > m_run + 8.f;
          if (rebase) {
            rescale = ex2(m_run - mt);
            m_run = mt;
            l_run *= rescale;
          }
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
          if (o_has && __any_sync(0xffffffffu, rebase)) {
            // this warpgroup's previous P.V must be done (at D = 128 the score MMA
            // of t already followed it in the same pipe)
            if (kTriS) {
              cross_wait(buf_free + (G - 2) % 3, ((G - 2) / 3) & 1, budget, s_abort, status);
              __syncwarp();
              tc_fence_after();
            }
            uint32_t r[32];
#pragma unroll
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
        if (lane == 0) mbar_arrive(p_full + 2 * wg + (own & 1));
        o_has = true;
      }
      // ---- the item's end: both warpgroups' states together
      if (nt > 0) {
        if (kTriS) {
          if (wg < nt) {
            const uint32_t G = gbase + wg + 2 * ((nt - 1 - wg) / 2);
            cross_wait(buf_free + G % 3, (G / 3) & 1, budget, s_abort, status);
          }
        } else {
          cross_wait(o_final, ic & 1, budget, s_abort, status);
          ++ic;
        }
      }
      __syncwarp();
      tc_fence_after();
      sML[wg * 128 + row] = make_float4(m_run, l_run, o_has ? 1.f : 0.f, 0.f);
      named_sync(3, 256);
      const float4 s0 = sML[row], s1 = sML[128 + row];
      const bool h0 = s0.z != 0.f, h1 = s1.z != 0.f;
      const float m = fmaxf(s0.x, s1.x);
      const float f0 = (h0 && m != -INFINITY) ? ex2(s0.x - m) : 0.f;
      const float f1 = (h1 && m != -INFINITY) ? ex2(s1.x - m) : 0.f;
      const float l = s0.y * f0 + s1.y * f1;
      const bool alone = args.splits == 1;
      const float inv = !alone ? 1.f : (l > 0.f ? 1.f / l : 0.f);
      const size_t orow = ((size_t)(it.r0 + row_tok) * a.H + (size_t)it.hk * a.G + row_head);
      float* sO = reinterpret_cast<float*>(sKV);  // a cluster's join: the ring is idle by then
#pragma unroll
      for (int h = 0; h < D / 64; ++h) {
        const int col = wg * (D / 2) + 32 * h;
        uint32_t ra[32], rb[32];
        if (warp_in) {
          tmem_ld32(tO(0) + lane_off + col, ra);
          tmem_ld32(tO(1) + lane_off + col, rb);
          tmem_ld_wait(ra);
          tmem_ld_wait(rb);
        }
        if (row_in && *s_abort == 0) {
#pragma unroll
          for (int e = 0; e < 32; e += 8) {
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
      }
      if (!alone) {
        if (wg == 0) sML[256 + row] = make_float4(m, l, 0.f, 0.f);
      } else if (args.lse && wg == 0 && row_in && *s_abort == 0) {
        args.lse[orow] = l > 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
      }
      tc_fence_before();
      named_sync(3, 256);  // every thread has read s_cur and sML
      gbase += nt;
      if (!alone) break;  // one item per cluster; s_cur stays for the join
      if (reader) *s_cur = read_item(c++);
      named_sync(3, 256);
    }
  }

  if (args.splits > 1) {
    cluster_sync();
    if (warp >= 4 && s_cur->hk >= 0) {
      const CrossItem it = *s_cur;
      const uint32_t ml_addr = smem_u32(sML + 256), o_addr = smem_u32(sKV);
      constexpr int kPieces = D / 4;
      for (int i = (int)rank * 256 + (int)threadIdx.x - 128; i < 128 * kPieces; i += 256 * args.splits) {
        const int row = i / kPieces, piece = i - row * kPieces;
        const int tok = row / a.G;
        if (tok >= it.nr || 4 * piece >= a.d) continue;
        float m = -INFINITY, l = 0.f;
        for (int r = 0; r < args.splits; ++r) m = fmaxf(m, ld_cluster(map_rank(ml_addr + 16 * row, r)).x);
        float o[4] = {0.f, 0.f, 0.f, 0.f};
        for (int r = 0; r < args.splits; ++r) {
          const float4 s = ld_cluster(map_rank(ml_addr + 16 * row, r));
          const float f = m != -INFINITY ? ex2(s.x - m) : 0.f;
          if (f > 0.f) {
            const float4 v = ld_cluster(map_rank(o_addr + 4 * o_piece<D>(row, piece), r));
            l += s.y * f;
            o[0] += v.x * f;
            o[1] += v.y * f;
            o[2] += v.z * f;
            o[3] += v.w * f;
          }
        }
        const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) o[k] *= inv;
        const size_t orow = (size_t)(it.r0 + tok) * a.H + (size_t)it.hk * a.G + (row - tok * a.G);
        const size_t at = orow * a.d + 4 * piece;
        store_rounded<T, 4>(static_cast<T*>(args.out) + at, args.out_lo ? static_cast<T*>(args.out_lo) + at : nullptr,
                            o);
        if (args.lse && piece == 0) args.lse[orow] = l > 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
      }
    }
    cluster_sync();  // no CTA leaves while another one reads its shared memory
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  if (!fn) {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  }
  return fn;
}

template <int D, bool BF16>
cudaError_t launch_fwd(const FwdArgs& a, const FwdMaps& maps, int grid, cudaStream_t s) {
  auto kernel = cross_fwd_kernel<D, BF16>;
  const uint32_t bytes = FwdSmem<D>::alloc;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = prepare_kernel((const void*)kernel, (int)bytes, kThreads, &done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = a.splits;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.splits > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, a, maps);
}

bool al16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

}  // namespace

bool encode_heads(CUtensorMap* m, const void* base, long long rows, int heads, int d, bool bf16, int box_heads,
                  int box_rows) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)rows};
  const cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)d * heads * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_rows};
  const cuuint32_t es[3] = {1, 1, 1};
  return enc(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(base),
             dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t prepare_kernel(const void* kernel, int bytes, int threads, std::atomic<uint64_t>* done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (dev < 64 && (done->load(std::memory_order_acquire) & bit)) return cudaSuccess;
  cudaFuncAttributes fa;
  e = cudaFuncGetAttributes(&fa, kernel);
  if (e != cudaSuccess) return e;
  if (fa.numRegs * threads < 256 * 224 + 128 * 56) return cudaErrorInvalidConfiguration;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev < 64) done->fetch_or(bit, std::memory_order_release);
  return e;
}

int device_sms() {
  static int sms = 0;
  if (!sms) {
    int dev = 0;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (sms <= 0) sms = 1;
  }
  return sms;
}

long long cross_query_tiles(const CrossArgs& a) {
  const long long per = (a.Lq + a.tpt - 1) / a.tpt;
  if (!a.cu_q) return per * a.B * a.Hk;
  // packed: every sequence and the rows behind the last one end in a tile of their own
  return ((long long)a.Tq / a.tpt + a.B + 1) * a.Hk;
}

df_status cross_check(const void* q, const void* k, const void* v, const uint8_t* key_mask, const int32_t* cu_q,
                      const int32_t* cu_k, int B, int H, int Hk, int Lq, int Lk, int total_q, int total_k, int d,
                      float scale, df_dtype dtype, int32_t* status, CrossArgs* a) {
  if (B < 0 || H < 1 || Hk < 1 || H % Hk != 0 || Lq < 0 || Lk < 0 || total_q < 0 || total_k < 0 || d < 1)
    return DF_ERR_INVALID_ARG;
  if (dtype != DF_BF16 && dtype != DF_FP16 && dtype != DF_FP32) return DF_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !(scale <= 3.0e38f) || (key_mask && cu_k)) return DF_ERR_INVALID_ARG;
  if (!cu_q && (long long)B * Lq != total_q) return DF_ERR_INVALID_ARG;
  if (!cu_k && (long long)B * Lk != total_k) return DF_ERR_INVALID_ARG;
  if (dtype == DF_FP32 || d % 8 != 0 || d > 128 || H / Hk > 128) return DF_ERR_UNSUPPORTED;
  if (total_q > (1 << 30) || total_k > (1 << 30)) return DF_ERR_UNSUPPORTED;
  if ((total_q > 0 && !q) || (total_k > 0 && (!k || !v))) return DF_ERR_INVALID_ARG;
  if (!al16(q) || !al16(k) || !al16(v) || ((uintptr_t)cu_q & 3u) != 0 || ((uintptr_t)cu_k & 3u) != 0)
    return DF_ERR_ALIGNMENT;
  a->key_mask = key_mask;
  a->cu_q = cu_q;
  a->cu_k = cu_k;
  a->B = B;
  a->H = H;
  a->Hk = Hk;
  a->G = H / Hk;
  a->Lq = Lq;
  a->Lk = Lk;
  a->Tq = total_q;
  a->Tk = total_k;
  a->d = d;
  a->tpt = 128 / a->G;
  a->scale = scale;
  a->kscale = (float)((double)scale * 1.4426950408889634);
  a->status = status;
  a->budget = wait_budget();
  return DF_OK;
}

}  // namespace dfa

using namespace dfa;

extern "C" df_status df_cross_attn_fwd(const void* q, const void* k, const void* v, const uint8_t* key_mask,
                                       const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k, int B, int H, int Hk,
                                       int Lq, int Lk, int total_q, int total_k, int d, float scale, df_dtype dtype,
                                       void* out, void* out_lo, float* lse, int32_t* status, df_stream_t stream) {
  FwdArgs a;
  const df_status st = cross_check(q, k, v, key_mask, cu_seqlens_q, cu_seqlens_k, B, H, Hk, Lq, Lk, total_q, total_k,
                                   d, scale, dtype, status, &a.c);
  if (st != DF_OK) return st;
  if (total_q == 0) return DF_OK;
  if (!out) return DF_ERR_INVALID_ARG;
  if (!al16(out) || !al16(out_lo) || ((uintptr_t)lse & 3u) != 0) return DF_ERR_ALIGNMENT;
  a.out = out;
  a.out_lo = out_lo;
  a.lse = lse;
  const bool bf16 = dtype == DF_BF16;
  FwdMaps maps;
  // without keys no copy of k or v is made: the maps then describe q
  const void* kp = total_k > 0 ? k : q;
  const void* vp = total_k > 0 ? v : q;
  const long long krows = total_k > 0 ? total_k : total_q;
  const int kheads = total_k > 0 ? Hk : H;
  if (!encode_heads(&maps.q, q, total_q, H, d, bf16, a.c.G, a.c.tpt) ||
      !encode_heads(&maps.k, kp, krows, kheads, d, bf16, 1, 128) ||
      !encode_heads(&maps.v, vp, krows, kheads, d, bf16, 1, 128))
    return DF_ERR_CUDA;
  const long long items = cross_query_tiles(a.c);
  const int sms = device_sms();
  a.splits = 1;
  const int key_tiles = (Lk + 127) / 128;
  while (a.splits < 8 && items * a.splits * 2 <= sms && a.splits * 2 <= key_tiles) a.splits *= 2;
  const int grid = a.splits > 1 ? (int)items * a.splits : (int)std::min<long long>(items, sms);
  cudaStream_t s = (cudaStream_t)stream;
  const cudaError_t e = d <= 64 ? (bf16 ? launch_fwd<64, true>(a, maps, grid, s) : launch_fwd<64, false>(a, maps, grid, s))
                                : (bf16 ? launch_fwd<128, true>(a, maps, grid, s) : launch_fwd<128, false>(a, maps, grid, s));
  return e == cudaSuccess ? DF_OK : DF_ERR_CUDA;
}
