// Cross attention, backward, on tcgen05 (bf16 / fp16 I/O, fp32 accumulation).
// With p_ij = exp(scale q_i.k_j - lse_i), D_i = dout_i.out_i and
// dS_ij = p_ij (dout_i.v_j - D_i):
//   dq_i = scale sum_j dS_ij k_j,  dk_j = scale sum_i dS_ij q_i,
//   dv_j = sum_i p_ij dout_i       (sums over i also run over the query heads
//                                   that share the key head).
//
// Three launches.  row_stats (fp16: group_stats) forms D_i from out + out_lo (fp32 sums; the rounding
// of out alone would leave 2^-9 |dout||v| where few keys carry a row) and puts it
// beside the row's lse in log2 units.  Two runs of one kernel then recompute the
// scores tile by tile: for a tile of keys it streams the queries past (dk, dv),
// for a tile of queries the keys (dq).  Five products would do with atomic sums
// into dq; seven without atomics keep every sum in tensor memory in a fixed order,
// so equal inputs give equal bits.
//
// Per 128 x 128 tile and half h of the streamed rows (64 columns each):
//   S = X0.Y0^T, dP = X1.Y1^T         into tensor memory (64 + 64 columns)
//   P, dS                             by warpgroup h, rounded to the I/O type,
//                                     written over S and dP
//   acc0 += dS.Y0 (dk or dq), acc1 += P.Y1 (dv; rows of P that do not count are 0)
// (X the resident, Y the streamed tiles.)  Three such (S, dP) buffers rotate (two
// where the sums leave no more columns: dk, dv at D = 128), so that the tensor core
// runs the next half's products while both warpgroups are busy.
//   warp 0        items and TMA loads
//   warps 1, 2    issue S and dP, warps 3, 4 the sums acc0 and acc1 (one issuer for
//                 each: two for all four took 1.81 ms where these took 1.57)
//   warp 5        per streamed tile: the rows' (lse, D) or the keys' mask bits into
//                 shared memory, and zeros over streamed rows that do not count
//                 (they are the reduction dimension of the second products); fp16:
//                 the resident rows' scales beside the item's first tile
//   warps 8-15    P and dS, one thread per resident row; the epilogue
//
// Measured (GB300, bf16): 16 x 12 heads, 2048 queries x 8192 keys, d = 64: 2.30 to 2.35 ms
// (10 flops per score and column: 877 to 896 TFLOP/s; with the two products that are done
// twice 1228 to 1255); 19 x 8 heads, d = 128: 3.39 to 3.46 ms (943 to 963; 1321 to 1348);
// fp16: 2.57 and 3.64.  Bound by the tensor core:
// S and dP in halves of 64 columns run at two thirds of its rate, so a 128 x 128 tile
// takes at least 1498 (keys) or 1138 (queries) cycles at d = 64 and takes about 1700
// and 1290; 2591 and 2074 at d = 128, and takes about 3500 and 2600 (only two buffers
// in the first).  Whole tiles (128 columns) would leave one buffer and no overlap.
//
// fp16: dS spans too wide a range for its exponent, so it is held times a power of two,
// taken back in fp32 at the end: the one that takes a bound of |dS| just below 2^15, for
// each resident row by itself.  Query tiles, row i: |dS_ij| <= |dout_i| max_j |v_j| +
// |D_i|; key tiles, row j: |dS_ij| <= max_i |dout_i| |v_j| + max_i |D_i|, the maxima over
// the sequence and the heads that share a key head (group_stats).  So nothing overflows,
// whatever v holds, a row keeps its digits beside rows of far larger dout or v, and
// what is lost below fp16's smallest step is 2^-40 of the row's bound.  P (at most 1) is
// held times 2^14.  bf16 needs none of this.
#include "df_cross.cuh"

#include <algorithm>
#include <type_traits>

namespace dfa {

namespace {

using namespace ptx;

constexpr int kThreads = 512, kFirst = 8;  // warps kFirst .. form P and dS, the others feed them
// registers per thread: launched, and after the split (P and dS, others)
constexpr int kRegs = 128, kSoftmaxRegs = 176, kOtherRegs = 72;
static_assert(256 * kSoftmaxRegs + 256 * kOtherRegs <= kThreads * kRegs, "setmaxnreg.inc must not wait");
constexpr uint32_t kItemRing = 4;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kPShift = 14.f, kPUnit = 1.f / 16384.f;  // fp16: P is held as 2^14 p

struct BwdArgs {
  CrossArgs c;
  const float2* stat;      // [Tq][H]: lse in log2 units (+inf without keys), D
  // fp16: |dout_i| [Tq][H], and [3][Tq][H], at the first query row of a sequence and the
  // first head of a group, the largest |dout_i|, |D_i| and |v_j| of the two, as bits.
  // |v_j| itself stands in the first four bytes of the key's row of dv until that is written.
  const float* norm;
  const uint32_t* top;
  void* out0;              // dk or dq
  void* out1;              // dv
  int after_keys;          // the key tiles' launch is the one before
};

struct BwdMaps {
  CUtensorMap x0, x1, y0, y1;
};

// ------------------------------------------------------------- row statistics
// |x|^2 of the row at `x`, and x (o + r) where o (and r) is given: (x (o + r), |x|^2).  Four
// lanes share a row, 8 columns of every 32 each.
template <typename T>
__device__ __forceinline__ float2 row_sums(const T* x, const T* o, const T* r, int d) {
  float sq = 0.f, sum = 0.f;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int c = 32 * k + 8 * (threadIdx.x & 3);
    if (c >= d) break;
    uint4 x4 = *reinterpret_cast<const uint4*>(x + c), o4 = make_uint4(0u, 0u, 0u, 0u), r4 = o4;
    if (o) o4 = *reinterpret_cast<const uint4*>(o + c);
    if (r) r4 = *reinterpret_cast<const uint4*>(r + c);
    const T *xe = reinterpret_cast<const T*>(&x4), *oe = reinterpret_cast<const T*>(&o4),
            *re = reinterpret_cast<const T*>(&r4);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float f = IO<T>::to_f(xe[e]);
      sq += f * f;
      if (o) sum += (IO<T>::to_f(oe[e]) + IO<T>::to_f(re[e])) * f;
    }
  }
#pragma unroll
  for (int m = 1; m < 4; m <<= 1) {
    sq += __shfl_xor_sync(0xffffffffu, sq, m);
    if (o) sum += __shfl_xor_sync(0xffffffffu, sum, m);
  }
  return make_float2(sum, sq);
}
__device__ __forceinline__ float2 row_stat(float lse, float D) {
  return make_float2(lse == -INFINITY ? INFINITY : lse * kLog2e, D);
}

template <typename T>
__global__ void __launch_bounds__(256) row_stats(const T* __restrict__ out, const T* __restrict__ out_lo,
                                                 const T* __restrict__ dout, const float* __restrict__ lse, int d,
                                                 long long rows, float2* __restrict__ stat) {
  allow_dependent_launch();
  const long long row = (long long)blockIdx.x * 64 + (threadIdx.x >> 2);
  const bool in = row < rows;
  const size_t at = in ? (size_t)row * d : 0;
  const float l = in ? lse[row] : 0.f;
  const float D = row_sums(dout + at, out + at, out_lo ? out_lo + at : nullptr, in ? d : 0).x;
  if (in && (threadIdx.x & 3) == 0) stat[row] = row_stat(l, D);
}

// fp16: the statistics of the rows of every sequence, their norms, those of its keys (at the
// head of dv's rows), and the largest of each (BwdArgs::top, zero before).  `parts`
// blocks share a sequence; a warp takes a step at a time: `span` rows of a group (a
// token's, where more heads share a key head), or `span` keys of a head.  Rows without a
// valid key, keys that do not count and what is not finite are left out of the maxima
// (the order in which warps raise those does not matter).  Bound by latency where there
// is little to do, so the code is short (eight rows at a time, in loops), and by HBM
// else: 4 x 12 heads, 77 x 300, d = 64: 5.3 us; 2048 x 8192: 29 us (88 MB).
__global__ void __launch_bounds__(256) group_stats(const CrossArgs a, int parts, int span, const __half* __restrict__ out,
                                                   const __half* __restrict__ out_lo, const __half* __restrict__ dout,
                                                   const float* __restrict__ lse, const __half* __restrict__ v,
                                                   float2* __restrict__ stat, float* __restrict__ norm, uint32_t* top,
                                                   __half* __restrict__ dv) {
  allow_dependent_launch();
  const int lane = threadIdx.x & 31, b = blockIdx.x / parts;
  const int warps = parts * 8, warp = (blockIdx.x - b * parts) * 8 + (threadIdx.x >> 5);
  int q0, k0;
  const int nq = seq_rows(query_side(a), b, nullptr, &q0), nk = seq_rows(key_side(a), b, nullptr, &k0);
  if (nq == 0 || nk == 0) return;
  const size_t plane = (size_t)a.Tq * a.H;
  const int tokens = max(1, span / a.G), per_q = (nq + tokens - 1) / tokens, per_k = (nk + span - 1) / span;
  const long long q_steps = (long long)per_q * a.Hk, steps = q_steps + (long long)per_k * a.Hk;
  for (long long u = warp; u < steps; u += warps) {
    const bool queries = u < q_steps;
    const int i = (int)(queries ? u : u - q_steps), per = queries ? per_q : per_k, hk = i / per;
    uint32_t* p0 = top + (size_t)q0 * a.H + hk * a.G + (queries ? 0 : 2 * plane);
    float m0 = 0.f, m1 = 0.f;
    if (queries) {
      const int t0 = (i - hk * per) * tokens, n = min(tokens, nq - t0) * a.G;
#pragma unroll 1
      for (int r0 = 0; r0 < n; r0 += 8) {
        const int r = min(r0 + (lane >> 2), n - 1), tok = r / a.G;  // (the last one again where there are fewer)
        const size_t row = (size_t)(q0 + t0 + tok) * a.H + hk * a.G + (r - tok * a.G), at = row * a.d;
        const float l = lse[row];
        const float2 s = row_sums(dout + at, out + at, out_lo ? out_lo + at : nullptr, a.d);
        const float x = sqrtf(s.y);
        const bool counts = l != -INFINITY && x <= 3.0e38f;
        if ((lane & 3) == 0) {
          stat[row] = row_stat(l, s.x);
          norm[row] = counts ? x : 0.f;
        }
        if (counts) m0 = fmaxf(m0, x);
        if (counts && fabsf(s.x) <= 3.0e38f) m1 = fmaxf(m1, fabsf(s.x));
      }
    } else {
      const int j0 = (i - hk * per) * span + (lane >> 2);
#pragma unroll 1
      for (int j = j0; j < j0 + span; j += 8) {
        const bool in = j < nk;
        const size_t at = in ? ((size_t)(k0 + j) * a.Hk + hk) * a.d : 0;
        const bool counts = in && (!a.key_mask || a.key_mask[(size_t)b * a.Lk + j] != 0);
        const float x = sqrtf(row_sums<__half>(v + at, nullptr, nullptr, in ? a.d : 0).y);
        if (in && (lane & 3) == 0) *reinterpret_cast<float*>(dv + at) = x;
        if (counts && x <= 3.0e38f) m0 = fmaxf(m0, x);
      }
    }
    // not negative: their bits are in order
    const uint32_t b0 = __reduce_max_sync(0xffffffffu, __float_as_uint(m0));
    const uint32_t b1 = __reduce_max_sync(0xffffffffu, __float_as_uint(m1));
    if (lane < (queries ? 2 : 1)) {
      uint32_t* p = p0 + lane * plane;
      const uint32_t mine = lane ? b1 : b0;
      if (mine > *static_cast<volatile uint32_t*>(p)) atomicMax(p, mine);
    }
  }
}

// The power of two that takes x y + z, a bound of |dS| (2^-48 .. 2^40 for fp16 rows),
// below 2^15.  (Short code: it runs once per item.  A bound of 0, or one that is not
// finite, gets the ends of the range.)
__device__ __forceinline__ float ds_scale(float x, float y, float z) {
  const uint32_t e = __float_as_uint(fmaf(x, y, z)) >> 23;  // below 2^(e - 126)
  return __uint_as_float((254u + 14u - min(max(e, 60u), 200u)) << 23);
}

// fp16: the scales of a resident tile's rows 32 w + lane (one warp).  Those of keys that do
// not count may be any power of two.
template <bool KEYS, typename T>
__device__ __forceinline__ void resident_scales(const BwdArgs& args, const CrossItem& it, float (&scales)[4]) {
  const CrossArgs& a = args.c;
  const size_t plane = (size_t)a.Tq * a.H;
  const int first = KEYS ? it.o0 : a.cu_q ? min(max(a.cu_q[it.b], 0), a.Tq - 1) : it.b * a.Lq;
  const uint32_t* top = args.top + (size_t)first * a.H + it.hk * a.G;
  const float x = __uint_as_float(top[KEYS ? 0 : 2 * plane]), z = KEYS ? __uint_as_float(top[plane]) : 0.f;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const int r = 32 * w + (threadIdx.x & 31), tok = KEYS ? r : r / a.G;
    scales[w] = 1.f;
    if (tok >= it.nr) continue;
    if (KEYS) {
      const T* dv = static_cast<const T*>(args.out1) + ((size_t)(it.r0 + r) * a.Hk + it.hk) * a.d;
      scales[w] = ds_scale(x, *reinterpret_cast<const float*>(dv), z);
    } else {
      const size_t row = (size_t)(it.r0 + tok) * a.H + it.hk * a.G + (r - tok * a.G);
      scales[w] = ds_scale(x, args.norm[row], fabsf(args.stat[row].y));
    }
  }
}

// ------------------------------------------------------------ the tile kernel
template <int D, bool BF16>
struct BwdSmem {
  static constexpr int kChunks = D / 64;
  static constexpr int kRes = D == 64 ? 2 : 1;     // resident pairs
  static constexpr int kStages = D == 64 ? 4 : 2;  // streamed pairs
  static constexpr uint32_t kTileBytes = kChunks * kBoxBytes;
  static constexpr uint32_t x = 0;                                   // [kRes][X0 | X1]
  static constexpr uint32_t y = x + kRes * 2 * kTileBytes;           // [kStages][Y0 | Y1]
  static constexpr uint32_t col = y + kStages * 2 * kTileBytes;      // [kStages]: float -lse [128], -D [128]; or 4 mask words
  static constexpr uint32_t stage = col + kStages * 1024;            // [8 warps] rows on their way out
  static constexpr uint32_t bars = stage + 8 * kRowStage;
  // x_full, x_empty [kRes]; full, ready, empty [kStages]; s_full, p_full, ds_free,
  // p_free [3];
  // acc_full, acc_free; drain [4]; item_full, item_empty; claim
  static constexpr int kBars = 2 * kRes + 3 * kStages + 12 + 6 + 2 * (int)kItemRing + 1;
  static constexpr uint32_t ring = (bars + kBars * 8 + 15) & ~15u;
  static constexpr uint32_t cur = ring + 32 * kItemRing;
  static constexpr uint32_t claim = cur + 64;  // 16 bytes
  static constexpr uint32_t misc = claim + 16;
  static constexpr uint32_t scale = misc + 16;  // fp16: float [kStages][128], the resident rows' scales
  static constexpr uint32_t bytes = scale + (BF16 ? 0 : kStages * 512);
  static constexpr uint32_t alloc = bytes + 1024;
  static_assert(alloc <= 232448, "shared memory of one CTA");
};

// KEYS: the resident rows are keys (K, V), the streamed ones queries (Q, dout).
template <int D, bool BF16, bool KEYS>
__global__ void __launch_bounds__(kThreads, 1) cross_bwd_kernel(const BwdArgs args, const __grid_constant__ BwdMaps maps) {
  using SL = BwdSmem<D, BF16>;
  constexpr int kChunks = SL::kChunks;
  constexpr uint32_t kRes = SL::kRes, kStages = SL::kStages;
  constexpr uint32_t kIdescS = idesc_f16(128, 64, BF16 ? 1 : 0, 0, 0);
  constexpr uint32_t kIdescAcc = idesc_f16(128, D, BF16 ? 1 : 0, 0, 1);
  using T = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
  // sums first, then the (S, dP) buffers: half u of the CTA (two per streamed tile)
  // uses buffer u mod kBufs
  constexpr uint32_t kAccCols = (KEYS ? 2u : 1u) * D, kBufs = kAccCols <= 128 ? 3u : 2u;
  static_assert(tmem_region_fits(kAccCols, 128 * kBufs, 512), "sums and score buffers in 512 columns");
  constexpr uint32_t kSums = KEYS ? 2 : 1;           // issuers of sums
  constexpr uint32_t kItemReaders = 2 + kSums + 2;  // the issuers, warp 5, the warpgroups' reader

  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + SL::bars);
  uint64_t* x_full = bars;
  uint64_t* x_empty = x_full + kRes;
  uint64_t* full = x_empty + kRes;
  uint64_t* ready = full + kStages;   // landed, rows that do not count zeroed, columns' values written
  uint64_t* empty = ready + kStages;
  // [buffer]: S and dP computed; P and dS written; the sums have read dS, and P
  uint64_t* s_full = empty + kStages;
  uint64_t* p_full = s_full + 3;
  uint64_t* ds_free = p_full + 3;
  uint64_t* p_free = ds_free + 3;
  uint64_t* acc_full = p_free + 3;
  uint64_t* acc_free = acc_full + 1;
  uint64_t* drain = acc_free + 1;      // [4], one per issuing thread
  uint64_t* item_full = drain + 4;
  uint64_t* item_empty = item_full + kItemRing;
  uint64_t* claim_bar = item_empty + kItemRing;
  auto ring_slot = [&](uint32_t c) { return reinterpret_cast<CrossItem*>(sm + SL::ring + 32 * (c % kItemRing)); };
  CrossItem* s_cur = reinterpret_cast<CrossItem*>(sm + SL::cur);
  volatile int* s_abort = reinterpret_cast<volatile int*>(sm + SL::misc);
  uint32_t* tslot = reinterpret_cast<uint32_t*>(sm + SL::misc + 4);

  const CrossArgs& a = args.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (uint32_t b = 0; b < kRes; ++b) {
      mbar_init(x_full + b, 1);
      mbar_init(x_empty + b, 2);
    }
    for (uint32_t s = 0; s < kStages; ++s) {
      mbar_init(full + s, 1);
      mbar_init(ready + s, 1);
      mbar_init(empty + s, kSums);
    }
    for (int b = 0; b < 3; ++b) {
      mbar_init(s_full + b, 2);
      mbar_init(p_full + b, 4);
      mbar_init(ds_free + b, 1);
      mbar_init(p_free + b, 1);
    }
    for (int b = 0; b < 4; ++b) mbar_init(drain + b, 1);
    mbar_init(acc_full, kSums);
    mbar_init(acc_free, 8);
    for (uint32_t b = 0; b < kItemRing; ++b) {
      mbar_init(item_full + b, 1);
      mbar_init(item_empty + b, kItemReaders);
    }
    mbar_init(claim_bar, 1);
    *s_abort = 0;
    mbar_fence_init();
    tma_prefetch_desc(&maps.x0);
    tma_prefetch_desc(&maps.x1);
    tma_prefetch_desc(&maps.y0);
    tma_prefetch_desc(&maps.y1);
  }
  if (warp == 1) {
    tmem_alloc(tslot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;
  // Keys: row_stats has finished; once every CTA stands here (and so none is left to
  // be launched), those of the query tiles may take the SMs that run dry.  They need
  // nothing that the key tiles write, only the end of their launch before their own.
  if (KEYS || !args.after_keys) grid_dependency_wait();
  if (KEYS) allow_dependent_launch();
  const uint32_t tAcc0 = tmem, tAcc1 = tmem + D;
  auto tS = [&](uint32_t b) { return tmem + kAccCols + 128u * b; };
  auto tdP = [&](uint32_t b) { return tmem + kAccCols + 128u * b + 64u; };

  const unsigned long long budget = a.budget;
  const int x_step = KEYS ? 128 : a.tpt, y_step = KEYS ? a.tpt : 128;  // tokens per tile
  auto y_tiles = [&](const CrossItem& it) { return (it.no + y_step - 1) / y_step; };
  auto read_item = [&](uint32_t c) {  // one thread: the c-th item handed out, hk = -1 at the end
    const uint32_t slot = c % kItemRing;
    CrossItem it;
    it.r0 = it.nr = it.o0 = it.no = it.b = 0;
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
    // (the whole warp runs every step, and one lane of it issues; so do the warps of
    // the products)
    TileWalk walk;
    TileClaim claim = {claim_bar, reinterpret_cast<uint4*>(sm + SL::claim)};
    uint32_t g = 0, xc = 0, g_issued = 0, x_issued = 0;
    const uint32_t q_box = (uint32_t)(a.G * a.tpt) * 128u;  // bytes of a 64-column box of a query tile
    const uint32_t x_box = KEYS ? kBoxBytes : q_box, y_box = KEYS ? q_box : kBoxBytes;
    long long number = blockIdx.x;
    int mask_b = -1, mask_n = 0;  // the last masked row measured
    bool ok = true;               // a wait ran out: nothing is loaded after it
    // a tile of each of two tensors
    auto load = [&](const CUtensorMap* m0, const CUtensorMap* m1, uint8_t* dst, uint32_t box, int head, int row,
                    uint64_t* bar) {
      if (elect_one()) {
        mbar_expect_tx(bar, 2 * kChunks * box);
        for (int ch = 0; ch < kChunks; ++ch) {
          tma_load_3d(dst + ch * kBoxBytes, m0, ch * 64, head, row, bar);
          tma_load_3d(dst + SL::kTileBytes + ch * kBoxBytes, m1, ch * 64, head, row, bar);
        }
      }
      __syncwarp();
    };
    for (uint32_t c = 0;; ++c) {
      CrossItem it = walk.find(a, KEYS ? key_side(a) : query_side(a), KEYS ? query_side(a) : key_side(a), x_step, number);
      if (a.key_mask && it.hk >= 0) {
        // nothing is streamed past 128 keys that do not count, and no keys behind the
        // last one that does
        if (KEYS) {
          if (masked_length(a.key_mask + it.r0, it.nr) == 0) it.no = 0;
        } else {
          if (it.b != mask_b) mask_n = masked_length(a.key_mask + (size_t)it.b * a.Lk, it.no);
          mask_b = it.b;
          it.no = mask_n;
        }
      }
      const uint32_t slot = c % kItemRing;
      bool room = true;
      if (c >= kItemRing) room = cross_wait(item_empty + slot, ((c / kItemRing) - 1) & 1, budget, s_abort);
      if (__any_sync(0xffffffffu, *s_abort || !room)) it.hk = -1;
      if (lane == 0 && room) {
        *ring_slot(c) = it;
        mbar_arrive(item_full + slot);
      }
      if (it.hk < 0) break;
      const int nt = y_tiles(it);
      const int x_head = KEYS ? it.hk : it.hk * a.G, y_head = KEYS ? it.hk * a.G : it.hk;
      if (nt > 0) {
        const uint32_t xb = xc % kRes;
        ok = ok && cross_wait(x_empty + xb, ((xc / kRes) & 1) ^ 1, budget, s_abort);
        ok = __all_sync(0xffffffffu, ok);
        if (ok) {
          load(&maps.x0, &maps.x1, sm + SL::x + xb * 2 * SL::kTileBytes, x_box, x_head, it.r0, x_full + xb);
          x_issued = xc + 1;
        }
        ++xc;
      }
      // the next item is asked for two tiles before this one's end
      const int ask_at = max(0, nt - 2);
#pragma unroll 1
      for (int t = 0; t < max(nt, 1); ++t) {
        if (t == ask_at) claim.ask();
        if (t >= nt) break;
        const uint32_t s = g % kStages;
        ok = ok && cross_wait(empty + s, ((g / kStages) & 1) ^ 1, budget, s_abort);
        ok = __all_sync(0xffffffffu, ok);
        ++g;
        if (!ok) continue;
        load(&maps.y0, &maps.y1, sm + SL::y + s * 2 * SL::kTileBytes, y_box, y_head, it.o0 + t * y_step, full + s);
        g_issued = g;
      }
      number = claim.answer(budget, s_abort);
    }
    // no copy may still be landing when the CTA leaves
    if (elect_one()) {
#pragma unroll 1
      for (uint32_t k = g_issued > kStages ? g_issued - kStages : 0; k < g_issued; ++k)
        mbar_wait(full + k % kStages, (k / kStages) & 1, kDrainBudget);
#pragma unroll 1
      for (uint32_t k = x_issued > kRes ? x_issued - kRes : 0; k < x_issued; ++k)
        mbar_wait(x_full + k % kRes, (k / kRes) & 1, kDrainBudget);
    }
    __syncwarp();
  } else if (warp <= 2) {
    // ------------------------------------------------------------ S (warp 1), dP (warp 2)
    setmaxnreg_dec<kOtherRegs>();
    const uint32_t which = warp - 1;
    const uint32_t tD = tmem + kAccCols + 64u * which;
    // a buffer's columns may be written again once the sums have read what stands
    // there; without dv the columns of S hold no P, and its readers are done with
    // dS's arrival
    uint64_t* free_bar = which ? ds_free : KEYS ? p_free : p_full;
    uint32_t g = 0, xc = 0;  // streamed tiles and items before this one
    bool ok = true;          // a wait that ran out ends this warp's products
    for (uint32_t c = 0;; ++c) {
      CrossItem it;
      if (lane == 0) it = read_item(c);
      it.hk = __shfl_sync(0xffffffffu, it.hk, 0);
      if (it.hk < 0) break;
      it.no = __shfl_sync(0xffffffffu, it.no, 0);
      const int nt = y_tiles(it);
      if (nt == 0) continue;
      const uint32_t xb = xc % kRes;
      ok = ok && cross_wait(x_full + xb, (xc / kRes) & 1, budget, s_abort);
      const uint64_t dx = uniform(sdesc_sw128(smem_u32(sm + SL::x + (xb * 2 + which) * SL::kTileBytes), 16, 1024));
#pragma unroll 1
      for (int t = 0; t < nt; ++t, ++g) {
        const uint32_t s = g % kStages;
        ok = ok && cross_wait(ready + s, (g / kStages) & 1, budget, s_abort);
        const uint32_t y_addr = smem_u32(sm + SL::y + (s * 2 + which) * SL::kTileBytes);
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          const uint32_t u = 2 * g + h, b = u % kBufs;
          const uint64_t dy = uniform(sdesc_sw128(y_addr + h * 8192, 16, 1024));
          const uint32_t to = uniform(tD + 128u * b);
          if (u >= kBufs) ok = ok && cross_wait(free_bar + b, (u / kBufs - 1) & 1, budget, s_abort);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) continue;
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < D / 16; ++k) mma_ss(to, dx + kmajor_step(k), dy + kmajor_step(k), kIdescS, k > 0);
            mma_commit(s_full + b);
          }
          __syncwarp();
        }
      }
      if (ok && elect_one()) mma_commit(x_empty + xb);
      __syncwarp();
      ++xc;
    }
    if (elect_one()) {
      mma_commit(drain + which);
      mbar_wait(drain + which, 0, kDrainBudget);
    }
    __syncwarp();
  } else if (warp <= 4) {
    // ------------------------------------------------------------ sums: dS.Y0 (warp 3), P.Y1 (warp 4)
    setmaxnreg_dec<kOtherRegs>();
    const uint32_t which = warp - 3;
    if (which < kSums) {
      const uint32_t tA = tmem + kAccCols + (which ? 0u : 64u), tD = uniform(which ? tAcc1 : tAcc0);
      uint64_t* free_bar = which ? p_free : ds_free;
      uint32_t g = 0, xc = 0;
      bool ok = true;
      for (uint32_t c = 0;; ++c) {
        CrossItem it;
        if (lane == 0) it = read_item(c);
        it.hk = __shfl_sync(0xffffffffu, it.hk, 0);
        if (it.hk < 0) break;
        it.no = __shfl_sync(0xffffffffu, it.no, 0);
        const int nt = y_tiles(it);
        if (nt == 0) continue;
        // the epilogue has read the previous item's sums
        if (xc > 0) ok = ok && cross_wait(acc_free, (xc - 1) & 1, budget, s_abort);
#pragma unroll 1
        for (int t = 0; t < nt; ++t, ++g) {
          const uint32_t s = g % kStages;
          const uint32_t y_addr = smem_u32(sm + SL::y + (s * 2 + which) * SL::kTileBytes);
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {
            const uint32_t u = 2 * g + h, b = u % kBufs;
            const uint64_t dy = uniform(vtile_desc(y_addr, 4 * h));
            const uint32_t from = uniform(tA + 128u * b);
            const uint32_t first = uniform(t == 0 && h == 0 ? 0u : 1u);
            ok = ok && cross_wait(p_full + b, (u / kBufs) & 1, budget, s_abort);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) continue;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
              for (int k = 0; k < 4; ++k) mma_ts(tD, from + 8 * k, dy + vtile_step(k), kIdescAcc, k > 0 ? 1u : first);
              mma_commit(free_bar + b);
              // (the scores of both halves, which read the stage too, stood before P)
              if (h == 1) mma_commit(empty + s);
            }
            __syncwarp();
          }
        }
        if (ok && elect_one()) mma_commit(acc_full);
        __syncwarp();
        ++xc;
      }
      if (elect_one()) {
        mma_commit(drain + 2 + which);
        mbar_wait(drain + 2 + which, 0, kDrainBudget);
      }
      __syncwarp();
    }
  } else if (warp == 5) {
    // ------------------------------------------------------------ streamed rows
    setmaxnreg_dec<kOtherRegs>();
    uint32_t g = 0;
    bool ok = true;
    for (uint32_t c = 0;; ++c) {
      CrossItem it;
      if (lane == 0) it = read_item(c);
      it.hk = __shfl_sync(0xffffffffu, it.hk, 0);
      if (it.hk < 0) break;
      it.o0 = __shfl_sync(0xffffffffu, it.o0, 0);
      it.no = __shfl_sync(0xffffffffu, it.no, 0);
      it.b = __shfl_sync(0xffffffffu, it.b, 0);
      if (!BF16) {
        it.r0 = __shfl_sync(0xffffffffu, it.r0, 0);
        it.nr = __shfl_sync(0xffffffffu, it.nr, 0);
      }
      const int nt = y_tiles(it);
#pragma unroll 1
      for (int t = 0; t < nt; ++t, ++g) {
        const uint32_t s = g % kStages;
        float scales[4];
        if (!BF16 && t == 0) resident_scales<KEYS, T>(args, it, scales);
        const int left = it.no - t * y_step;  // tokens of the tile (and behind it)
        uint32_t bits[4];
        float2 st[4];
        bool whole = true;
        if constexpr (KEYS) {
          const float2* stat = args.stat + (size_t)(it.o0 + t * y_step) * a.H + it.hk * a.G;
          const int tokens = min(left, a.tpt);
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const int r = 32 * w + lane, tok = r / a.G;
            const bool in = tok < tokens;
            st[w] = in ? stat[(size_t)tok * a.H + (r - tok * a.G)] : make_float2(INFINITY, 0.f);
            bits[w] = __ballot_sync(0xffffffffu, in);
          }
          whole = (bits[0] & bits[1] & bits[2] & bits[3]) == 0xffffffffu;
        } else {
          whole = key_bits(a.key_mask ? a.key_mask + (size_t)it.b * a.Lk + (size_t)t * 128 : nullptr, left, bits);
        }
        ok = ok && cross_wait(full + s, (g / kStages) & 1, budget, s_abort);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) continue;
        uint8_t* sY = sm + SL::y + s * 2 * SL::kTileBytes;
        if (!BF16 && t == 0) {
#pragma unroll
          for (int w = 0; w < 4; ++w) reinterpret_cast<float*>(sm + SL::scale + s * 512)[32 * w + lane] = scales[w];
        }
        if (!whole) {
          zero_rows<4, kChunks>(sY, bits);
          if (KEYS) zero_rows<4, kChunks>(sY + SL::kTileBytes, bits);
        }
        if constexpr (KEYS) {
          float* col = reinterpret_cast<float*>(sm + SL::col + s * 1024);
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            col[32 * w + lane] = (BF16 ? 0.f : kPShift) - st[w].x;
            col[128 + 32 * w + lane] = -st[w].y;
          }
        } else if (lane < 4) {
          reinterpret_cast<uint32_t*>(sm + SL::col + s * 1024)[lane] =
              lane == 0 ? bits[0] : lane == 1 ? bits[1] : lane == 2 ? bits[2] : bits[3];
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(ready + s);
      }
    }
  } else if (warp < kFirst) {
    setmaxnreg_dec<kOtherRegs>();
  } else {
    // ------------------------------------------------------------ P, dS and the epilogue
    setmaxnreg_inc<kSoftmaxRegs>();
    const int h = (warp - kFirst) >> 2;
    const int quad = warp & 3;
    const int row = quad * 32 + lane;        // resident row
    const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
    const float ks = a.kscale;
    const float2 ks2 = make_float2(ks, ks);
    const float scale0 = a.scale;              // dk, dq
    const float scale1 = BF16 ? 1.f : kPUnit;  // dv
    const int row_tok = KEYS ? row : row / a.G, row_head = KEYS ? 0 : row - row_tok * a.G;
    const bool reader = warp == kFirst && lane == 0;
    uint32_t g = 0, xc = 0, c = 1;  // c: items taken, of which the last but one is current at an item's end
    if (reader) s_cur[0] = read_item(0);
    named_sync(3, 256);
    for (;;) {
      const CrossItem it = s_cur[~c & 1];
      if (it.hk < 0) break;
      const int nt = y_tiles(it);
      const bool stored = row_tok < it.nr;   // the resident row belongs to the sequence
      bool row_in = stored;
      float nl = -INFINITY, nd = 0.f;  // -lse, -D
      if (KEYS) {
        const long long key = (long long)it.r0 + row;  // in [B, Lk] layout this is also the mask's index
        if (row_in && a.key_mask) row_in = a.key_mask[key] != 0;
      } else if (row_in) {
        const float2 st = args.stat[(size_t)(it.r0 + row_tok) * a.H + it.hk * a.G + row_head];
        nl = (BF16 ? 0.f : kPShift) - st.x;
        nd = -st.y;
      }
      const uint32_t rows_in = __ballot_sync(0xffffffffu, row_in);
      float ds_mul = kPUnit;  // fp16: the row's scale, on P as it is held
      const float2 nl2 = make_float2(nl, nl), nd2 = make_float2(nd, nd);
      for (int t = 0; t < nt; ++t) {
        const uint32_t s = (g + t) % kStages, u = 2 * (g + t) + h, b = u % kBufs;
        // (the buffer's previous half is the other warpgroup's u - 3 at three buffers;
        // its scores stand before those of u - 2, which this warp has seen)
        cross_wait(s_full + b, (u / kBufs) & 1, budget, s_abort);
        __syncwarp();
        tc_fence_after();
        const float* col = reinterpret_cast<const float*>(sm + SL::col + s * 1024);
        if (!BF16 && t == 0) ds_mul = reinterpret_cast<const float*>(sm + SL::scale + s * 512)[row] * kPUnit;
        if constexpr (KEYS) {
          // A thread takes two columns of every eight in four rows (lane / 4 + 8 r),
          // not 64 columns of one row: it then reads a quarter of the columns' values
          // from shared memory (one row per thread: 898 us against 835 on 8 x 12 heads,
          // 2048 x 8192, d = 64)
          const int c2 = 64 * h + 2 * (lane & 3);
          // (32 columns at a time, in a loop that the instruction caches hold: 707 us
          // unrolled against 677 for the launch of that shape)
#pragma unroll 1
          for (int q = 0; q < 2; ++q) {
            uint32_t rs0[16], rs1[16], rd0[16], rd1[16];
            const uint32_t at = lane_off + 32 * q;
            tmem_ld_rows16(tS(b) + at, rs0);
            tmem_ld_rows16(tdP(b) + at, rd0);
            tmem_ld_rows16(tS(b) + at + (16u << 16), rs1);
            tmem_ld_rows16(tdP(b) + at + (16u << 16), rd1);
            float2 nl[4], nd[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              nl[j] = *reinterpret_cast<const float2*>(col + c2 + 32 * q + 8 * j);
              nd[j] = *reinterpret_cast<const float2*>(col + 128 + c2 + 32 * q + 8 * j);
            }
            tmem_ld_wait(rs0);
            tmem_ld_wait(rd0);
            tmem_ld_wait(rs1);
            tmem_ld_wait(rd1);
            auto half_rows = [&](const uint32_t (&rs)[16], const uint32_t (&rd)[16], int i) {
              uint32_t wp[8], wd[8];
              // (fp16: the scales of this thread's rows, fetched here: held over the loop they spill)
              const float m0 = BF16 ? 1.f : __shfl_sync(0xffffffffu, ds_mul, 16 * i + (lane >> 2));
              const float m1 = BF16 ? 1.f : __shfl_sync(0xffffffffu, ds_mul, 16 * i + 8 + (lane >> 2));
              const float2 mul[2] = {make_float2(m0, m0), make_float2(m1, m1)};
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const int j = e >> 1, k = 4 * j + 2 * (e & 1);
                const float2 z = fma2(make_float2(__uint_as_float(rs[k]), __uint_as_float(rs[k + 1])), ks2, nl[j]);
                const float2 p = make_float2(ex2(z.x), ex2(z.y));
                float2 ds = mul2(p, add2(make_float2(__uint_as_float(rd[k]), __uint_as_float(rd[k + 1])), nd[j]));
                if (!BF16) ds = mul2(ds, mul[e & 1]);
                wp[e] = BF16 ? pack_bf16x2(p.x, p.y) : pack_f16x2(p.x, p.y);
                wd[e] = BF16 ? pack_bf16x2(ds.x, ds.y) : pack_f16x2(ds.x, ds.y);
              }
              if (rows_in != 0xffffffffu) {
                // what does not count has weight 0 whatever its row held
#pragma unroll
                for (int e = 0; e < 8; ++e)
                  if (!((rows_in >> (16 * i + 8 * (e & 1) + (lane >> 2))) & 1u)) wp[e] = wd[e] = 0u;
              }
              const uint32_t to = lane_off + 16 * q + ((uint32_t)(16 * i) << 16);
              tmem_st_rows16(tS(b) + to, wp);
              tmem_st_rows16(tdP(b) + to, wd);
            };
            half_rows(rs0, rd0, 0);
            half_rows(rs1, rd1, 1);
          }
        } else {
          // 32 columns at a time, the second loads in flight meanwhile
          uint32_t rs0[32], rd0[32], rs1[32], rd1[32];
          tmem_ld32(tS(b) + lane_off, rs0);
          tmem_ld32(tdP(b) + lane_off, rd0);
          tmem_ld_wait2(rs0, rd0);
          tmem_ld32(tS(b) + lane_off + 32, rs1);
          tmem_ld32(tdP(b) + lane_off + 32, rd1);
          auto columns = [&](const uint32_t (&rs)[32], const uint32_t (&rd)[32], int q) {
            uint32_t wd[16];
            const uint32_t bits = reinterpret_cast<const uint32_t*>(col)[2 * h + q];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float2 z =
                  fma2(make_float2(__uint_as_float(rs[2 * e]), __uint_as_float(rs[2 * e + 1])), ks2, nl2);
              const float2 p = make_float2(ex2(z.x), ex2(z.y));
              float2 ds = mul2(p, add2(make_float2(__uint_as_float(rd[2 * e]), __uint_as_float(rd[2 * e + 1])), nd2));
              if (!BF16) ds = mul2(ds, make_float2(ds_mul, ds_mul));
              wd[e] = BF16 ? pack_bf16x2(ds.x, ds.y) : pack_f16x2(ds.x, ds.y);
            }
            if (bits != 0xffffffffu) {
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const uint32_t two = (bits >> (2 * e)) & 3u;
                wd[e] &= (two & 1u ? 0xffffu : 0u) | (two & 2u ? 0xffff0000u : 0u);
              }
            }
            tmem_st16(tdP(b) + lane_off + 16 * q, wd);
          };
          columns(rs0, rd0, 0);
          tmem_ld_wait2(rs1, rd1);
          columns(rs1, rd1, 1);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full + b);
      }
      // ---- the item's results
      if (reader) s_cur[c & 1] = read_item(c);  // the next one
      ++c;
      if (nt > 0) cross_wait(acc_full, xc & 1, budget, s_abort);
      __syncwarp();
      tc_fence_after();
      const int heads = KEYS ? a.Hk : a.H;
      const size_t row0 = (size_t)it.r0 * heads + (KEYS ? it.hk : it.hk * a.G);
      const int rel = stored && *s_abort == 0 ? row_tok * heads + row_head : -1;
      // KEYS: warpgroup 0 writes dk, 1 dv; else each half of dq's columns
      const uint32_t tA = (KEYS && h == 1 ? tAcc1 : tAcc0) + lane_off;
      T* dst = static_cast<T*>(KEYS && h == 1 ? args.out1 : args.out0) + row0 * a.d;
      const float mul = KEYS && h == 1 ? scale1 : BF16 ? scale0 : scale0 / (ds_mul / kPUnit);
      const int c0 = KEYS ? 0 : h * (D / 2), c1 = KEYS ? D : c0 + D / 2;
      // The sums of a key that does not count are of 0 times rows that may not be finite.  (A
      // mask: a choice by condition here cost the key tiles' loop 3 % of its time.)
      const uint32_t keep = nt > 0 && (!KEYS || ((rows_in >> lane) & 1u)) ? 0xffffffffu : 0u;
#pragma unroll 1
      for (int cc = c0; cc < min(c1, a.d); cc += 32) {
        uint32_t r[32], w[16];
        tmem_ld32(tA + cc, r);
        tmem_ld_wait(r);
#pragma unroll
        for (int e = 0; e < 16; ++e)
          w[e] = keep & pack2<BF16>(__uint_as_float(r[2 * e]) * mul, __uint_as_float(r[2 * e + 1]) * mul);
        store_rows32<T>(sm + SL::stage + (warp - kFirst) * kRowStage, w, rel, dst + cc, a.d, a.d - cc);
      }
      tc_fence_before();
      __syncwarp();
      if (nt > 0) {
        if (lane == 0) mbar_arrive(acc_free);
        ++xc;
      }
      g += nt;
      named_sync(3, 256);  // the next item is there, and every thread has read s_cur[c & 1]
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
  if (threadIdx.x == 0) cross_report(s_abort, a.status);
  if (!KEYS && args.after_keys) grid_dependency_wait();
}

template <int D, bool BF16, bool KEYS>
cudaError_t launch_tiles(const BwdArgs& a, const BwdMaps& maps, long long items, cudaStream_t s) {
  if (items == 0) return cudaSuccess;
  auto kernel = cross_bwd_kernel<D, BF16, KEYS>;
  const uint32_t bytes = BwdSmem<D, BF16>::alloc;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = prepare_kernel((const void*)kernel, (int)bytes, kRegs, &done);
  if (e != cudaSuccess) return e;
  return launch_after_plan(kernel, (int)items, kThreads, bytes, s, a, maps);
}

template <int D, bool BF16>
cudaError_t launch_both(BwdArgs a, const BwdMaps& km, const BwdMaps& qm, void* dq, void* dk, void* dv,
                        cudaStream_t s) {
  const long long key_items = a.c.cu_k ? ((long long)a.c.Tk / 128 + a.c.B + 1) * a.c.Hk
                                       : (long long)((a.c.Lk + 127) / 128) * a.c.B * a.c.Hk;
  a.after_keys = 0;
  if (a.c.Tk > 0 && key_items > 0) {
    a.after_keys = 1;
    a.out0 = dk;
    a.out1 = dv;
    const cudaError_t e = launch_tiles<D, BF16, true>(a, km, key_items, s);
    if (e != cudaSuccess) return e;
  }
  if (a.c.Tq > 0) {
    a.out0 = dq;
    a.out1 = nullptr;
    return launch_tiles<D, BF16, false>(a, qm, cross_query_tiles(a.c), s);
  }
  return cudaSuccess;
}

void launch_stats(const void* out, const void* out_lo, const void* dout, const float* lse, const CrossArgs& c,
                  float2* stat, cudaStream_t s) {
  using T = __nv_bfloat16;
  const long long rows = (long long)c.Tq * c.H;
  row_stats<T><<<(unsigned)((rows + 63) / 64), 256, 0, s>>>(static_cast<const T*>(out), static_cast<const T*>(out_lo),
                                                           static_cast<const T*>(dout), lse, c.d, rows, stat);
}

void launch_group_stats(const void* out, const void* out_lo, const void* dout, const float* lse, const void* v,
                        const CrossArgs& c, float2* stat, float* norm, uint32_t* top, void* dv, cudaStream_t s) {
  using T = __half;
  // a step for each warp, in at most eight blocks an SM (by the stated lengths); steps of
  // eight rows, one round trip to memory each, where they are that few
  const long long most = std::max(1ll, 8ll * device_sms() / c.B);
  auto blocks = [&](long long span) {
    return (c.Hk * ((c.Lk + span - 1) / span + ((long long)c.Lq * c.G + span - 1) / span) + 7) / 8;
  };
  const int span = blocks(8) <= most ? 8 : 32;
  const int parts = (int)std::min(std::max(1ll, blocks(span)), most);
  group_stats<<<parts * c.B, 256, 0, s>>>(c, parts, span, static_cast<const T*>(out), static_cast<const T*>(out_lo),
                                          static_cast<const T*>(dout), lse, static_cast<const T*>(v), stat, norm, top,
                                          static_cast<T*>(dv));
}

bool al16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

}  // namespace
}  // namespace dfa

using namespace dfa;

extern "C" size_t df_cross_attn_bwd_workspace_size(int total_q, int H) {
  if (total_q < 0 || total_q > (1 << 30) || H < 1 || (long long)total_q * H > (1ll << 34)) return 0;
  // stat, norm and top (the last two for fp16)
  const size_t rows = (size_t)total_q * H;
  return up256(rows * sizeof(float2)) + up256(rows * sizeof(float)) + up256(3 * rows * sizeof(uint32_t)) + 256;
}

extern "C" df_status df_cross_attn_bwd(const void* q, const void* k, const void* v, const void* out, const void* out_lo,
                                       const float* lse, const void* dout, const uint8_t* key_mask,
                                       const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k, int B, int H, int Hk,
                                       int Lq, int Lk, int total_q, int total_k, int d, float scale, df_dtype dtype,
                                       void* dq, void* dk, void* dv, int32_t* status, void* workspace,
                                       size_t workspace_bytes, df_stream_t stream) {
  BwdArgs a;
  const df_status st = cross_check(q, k, v, key_mask, cu_seqlens_q, cu_seqlens_k, B, H, Hk, Lq, Lk, total_q, total_k,
                                   d, scale, dtype, status, &a.c);
  if (st != DF_OK) return st;
  if ((total_q > 0 && (!out || !lse || !dout || !dq)) || (total_k > 0 && (!dk || !dv))) return DF_ERR_INVALID_ARG;
  if (!al16(out) || !al16(out_lo) || !al16(dout) || !al16(dq) || !al16(dk) || !al16(dv) || ((uintptr_t)lse & 3u) != 0 ||
      ((uintptr_t)workspace & 255u) != 0)
    return DF_ERR_ALIGNMENT;
  const size_t need = df_cross_attn_bwd_workspace_size(total_q, H);
  if (need == 0) return DF_ERR_UNSUPPORTED;
  if (!workspace || workspace_bytes < need) return DF_ERR_WORKSPACE;
  if (total_q == 0 && total_k == 0) return DF_OK;
  const size_t q_bytes = (size_t)total_q * H * d * 2, k_bytes = (size_t)total_k * Hk * d * 2;
  const size_t cu_bytes = ((size_t)B + 1) * 4;
  if (overlapping({{dq, q_bytes}, {dk, k_bytes}, {dv, k_bytes}, {workspace, need}},
                  {{q, q_bytes}, {k, k_bytes}, {v, k_bytes}, {out, q_bytes}, {out_lo, q_bytes}, {dout, q_bytes},
                   {lse, (size_t)total_q * H * 4}, {key_mask, (size_t)total_k}, {cu_seqlens_q, cu_bytes},
                   {cu_seqlens_k, cu_bytes}}))
    return DF_ERR_INVALID_ARG;
  cudaStream_t s = (cudaStream_t)stream;
  const bool bf16 = dtype == DF_BF16;
  const size_t rows = (size_t)total_q * H;
  char* base = static_cast<char*>(workspace);
  float2* stat = reinterpret_cast<float2*>(base);
  float* norm = bf16 ? nullptr : reinterpret_cast<float*>(base + up256(rows * sizeof(float2)));
  uint32_t* top =
      bf16 ? nullptr : reinterpret_cast<uint32_t*>(base + up256(rows * sizeof(float2)) + up256(rows * sizeof(float)));
  a.stat = stat;
  a.norm = norm;
  a.top = top;
  if (total_q > 0 && bf16) {
    launch_stats(out, out_lo, dout, lse, a.c, stat, s);
  } else if (total_q > 0 && total_k > 0 && B > 0) {
    if (cudaMemsetAsync(top, 0, 3 * rows * sizeof(uint32_t), s) != cudaSuccess) return DF_ERR_CUDA;
    launch_group_stats(out, out_lo, dout, lse, v, a.c, stat, norm, top, dv, s);
  }
  if (cudaGetLastError() != cudaSuccess) return DF_ERR_CUDA;
  // a side without rows is never copied from: its maps then describe the other one
  const bool has_q = total_q > 0, has_k = total_k > 0;
  const void* qp = has_q ? q : k;
  const void* gp = has_q ? dout : k;
  const void* kp = has_k ? k : q;
  const void* vp = has_k ? v : q;
  const int q_heads = has_q ? H : Hk, k_heads = has_k ? Hk : H;
  const long long q_rows = has_q ? total_q : total_k, k_rows = has_k ? total_k : total_q;
  CUtensorMap mq, mg, mk, mv;
  if (!encode_heads(&mq, qp, q_rows, q_heads, d, bf16, a.c.G, a.c.tpt) ||
      !encode_heads(&mg, gp, q_rows, q_heads, d, bf16, a.c.G, a.c.tpt) ||
      !encode_heads(&mk, kp, k_rows, k_heads, d, bf16, 1, 128) ||
      !encode_heads(&mv, vp, k_rows, k_heads, d, bf16, 1, 128))
    return DF_ERR_CUDA;
  const BwdMaps key_maps = {mk, mv, mq, mg}, query_maps = {mq, mg, mk, mv};
  const cudaError_t e =
      d <= 64 ? (bf16 ? launch_both<64, true>(a, key_maps, query_maps, dq, dk, dv, s)
                      : launch_both<64, false>(a, key_maps, query_maps, dq, dk, dv, s))
              : (bf16 ? launch_both<128, true>(a, key_maps, query_maps, dq, dk, dv, s)
                      : launch_both<128, false>(a, key_maps, query_maps, dq, dk, dv, s));
  return e == cudaSuccess ? DF_OK : DF_ERR_CUDA;
}
