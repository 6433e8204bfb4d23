// Attention of a few queries for each sequence to the 8-bit cache: single tokens and short
// runs of them (causal, with a window and sinks), or queries that see every token held (the
// encoder's states).
//
//   s_ij = scale ks_j (q_i . ck_j),  o_i = sum_j exp(s_ij - lse_i) vs_j cv_j
// over the visible tokens j, with codes ck, cv and scales ks, vs of j's block.
//
// Bound by reading the cache once: 2 d + 1/2 bytes a token and key head, for 4 d G n flops.  So
// nothing but the tensor core's old instructions (m16n8k16: a tile of 16 query rows, one block
// of 16 keys) stands between the bytes and the sums:
//   - A CTA has four warps, each on its own: a ring of bulk copies (two blocks' records, one
//     contiguous piece where they are on one page) in shared memory, waits, products. Nothing
//     in the loop meets another warp (WR > 1: query rows that do not fit 16 are shared out, and
//     WR warps read the same ring).
//   - Codes become fp16 exactly (one instruction for two). The scale of K multiplies scores, that
//     of V the products of a block, both in fp32.
//   - The order of keys in a block is free, and so is that of columns in a sum: lane (g, t) =
//     (lane / 4, lane % 4) takes 8 columns of a K row at once and 4 tokens x 4 columns of V,
//     transposed by byte permutes; key i of lane t is 4 i + ((t + 2 (i & 1)) & 3), for which
//     neither read meets a bank conflict and the scores a lane gets are the weights it needs.
//   - A weight is held times 2^14, so that fp16 keeps its digits down to 2^-28 of the largest.
// Sequences are cut over the CTAs of a cluster where there are few of them; the parts are joined
// through distributed shared memory, without a workspace or a second launch.
#include <limits.h>

#include <algorithm>

#include "df_cache.cuh"
#include "df_cross_fwd.cuh"

namespace dfa {
namespace {

using namespace ptx;

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kTile = 32;  // keys of a copy: two blocks
constexpr float kUp = 14.f;

struct DecodeArgs {
  CacheView c;
  const void* q;
  const int32_t* cu_q;  // [B + 1] or NULL
  void* out;
  float* lse;           // or NULL
  int B, H, G, Lq, Tq;
  int row_tiles;        // CTAs that share a sequence's query rows
  int splits;           // and its keys (cluster size)
  int causal, window, sinks, bf16;
  float kscale;         // scale log2(e)
  int32_t* status;
  unsigned long long budget;
};

template <int SLABS, int WR>
struct DecodeSmem {
  static constexpr int D = 32 * SLABS;
  static constexpr int kRings = kWarps / WR;
  static constexpr int kStages = SLABS == 1 ? 6 : SLABS == 2 ? 3 : 2;
  static constexpr uint32_t kRecord = 32 * D + 16;
  static constexpr uint32_t kStageBytes = 2 * kRecord;
  static constexpr uint32_t ring = 0;  // [kRings][kStages][two records]
  static constexpr uint32_t ring_bytes = kRings * kStages * kStageBytes;
  // after the loop, over the ring: each warp's O, and the CTA's
  static constexpr int kPitch = D + 4;
  static constexpr uint32_t o_warp = 0;  // float [kWarps][16][kPitch]
  static constexpr uint32_t o_cta = kWarps * 16 * kPitch * 4;  // float [16 WR][D]
  static constexpr uint32_t joined = o_cta + 16 * WR * D * 4;
  static constexpr uint32_t ml_warp = (ring_bytes > joined ? ring_bytes : joined);  // float2 [kWarps][16]
  static constexpr uint32_t ml_cta = ml_warp + kWarps * 16 * 8;                     // float4 [16 WR]
  static constexpr uint32_t bars = ml_cta + 64 * 16;                                // full, empty [kRings][kStages]
  static constexpr uint32_t have = bars + 2 * kRings * kStages * 8;                 // int [kRings][kStages]
  static constexpr uint32_t misc = have + kRings * kStages * 4;
  static constexpr uint32_t bytes = misc + 16;
  static_assert(bytes <= 232448 && o_cta % 16 == 0 && joined % 16 == 0 && ml_warp % 16 == 0 && bars % 8 == 0, "layout");
};

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The same onto zeros.
__device__ __forceinline__ void mma_f16_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
// Four e4m3 codes as two pairs of fp16.
__device__ __forceinline__ void codes4_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 x, y;\n\tmov.b32 {x, y}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, x;\n\tcvt.rn.f16x2.e4m3x2 %1, y;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}
__device__ __forceinline__ uint2 lds64(uint32_t at) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t at) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ void bulk_load(uint32_t dst, unsigned long long src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// The tokens that a tile of query rows, at positions p0 .. p1, sees: those before `head` and
// those from lo to end - 1; in tiles of kTile, the first `heads` and then those from `skip`
// tiles further on.
struct Reach {
  int head, lo, end, heads, skip, tiles;
  __device__ __forceinline__ int tile(int t) const { return t < heads ? t : t + skip; }
  __device__ __forceinline__ bool any(int first, int n) const {
    return first < end && (first < head || first + n > lo);
  }
};
__device__ __forceinline__ Reach reach_of(const DecodeArgs& a, int held, int p0, int p1) {
  Reach r;
  r.end = a.causal ? max(min(held, p1 + 1), 0) : held;
  r.lo = a.causal && a.window != 0 ? max(p0 - a.window + 1, 0) : 0;
  r.lo = min(r.lo, r.end);
  r.head = min(a.sinks, r.lo);
  r.heads = (r.head + kTile - 1) / kTile;
  r.skip = max(r.lo / kTile - r.heads, 0);
  r.tiles = (r.end + kTile - 1) / kTile - r.skip;
  return r;
}

// HALF: at most 8 query rows (the tile's upper half is empty).
template <int SLABS, int WR, bool HALF>
__global__ void __launch_bounds__(kThreads) decode_kernel(const DecodeArgs a) {
  using SL = DecodeSmem<SLABS, WR>;
  constexpr int D = SL::D, S = SL::kStages, R = SL::kRings;
  constexpr int kHalves = HALF ? 1 : 2;
  extern __shared__ __align__(128) uint8_t sm[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group = warp / WR, part = warp % WR;  // the warp's ring, and its 16 query rows
  const int g = lane >> 2, t = lane & 3;
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + SL::bars) + group * S;
  uint64_t* empty = reinterpret_cast<uint64_t*>(sm + SL::bars) + (R + group) * S;
  volatile int* have = reinterpret_cast<volatile int*>(sm + SL::have) + group * S;
  volatile int* s_abort = reinterpret_cast<volatile int*>(sm + SL::misc);
  if (threadIdx.x == 0) {
    for (int i = 0; i < R * S; ++i) {
      mbar_init(reinterpret_cast<uint64_t*>(sm + SL::bars) + i, 1);
      mbar_init(reinterpret_cast<uint64_t*>(sm + SL::bars) + R * S + i, WR);
    }
    *s_abort = 0;
    mbar_fence_init();
  }
  __syncthreads();

  // ---- the CTA's work: sequence, key head, query rows, part of the keys
  const int split = blockIdx.x % a.splits;
  int rest = blockIdx.x / a.splits;
  const int rt = rest % a.row_tiles;
  rest /= a.row_tiles;
  const int hk = rest % a.c.Hk;
  int b = rest / a.c.Hk;
  // Sequences in the order of their lengths, the longest first, so that the launch's last CTAs
  // are short ones.
  if (a.B > 1 && a.B <= kThreads) {
    int* lens = reinterpret_cast<int*>(sm + SL::ml_cta);
    int* which = reinterpret_cast<int*>(sm + SL::ml_warp);
    const int n = threadIdx.x < a.B ? a.c.lengths[threadIdx.x] : 0;
    lens[threadIdx.x] = n;
    __syncthreads();
    int rank = 0;
    for (int i = 0; i < a.B; ++i) rank += lens[i] > n || (lens[i] == n && i < threadIdx.x);
    if (threadIdx.x < a.B && rank == b) *which = threadIdx.x;
    __syncthreads();
    b = *which;
  }
  int q0;
  const CrossSide side = {a.cu_q, a.Lq, a.Tq};
  int nq = seq_rows(side, b, a.status, &q0);
  int held = a.c.lengths[b];
  if (held < 0 || held > a.c.max_pages * a.c.page) {  // (the product is at most 2^30)
    held = 0;
    if (threadIdx.x == 0) cross_fail(a.status, (int)DF_ERR_INVALID_ARG);
  }
  if (nq > a.Lq) {  // rows that the launch has no CTA for
    if (threadIdx.x == 0) cross_fail(a.status, (int)DF_ERR_INVALID_ARG);
    nq = a.Lq;
  }
  const int rows = nq * a.G, r0 = rt * 16 * WR;  // rows: token r / G, head r % G
  const int nr = min(16 * WR, rows - r0);
  const int p_first = held - nq;                 // position of the sequence's first query
  const int p0 = p_first + r0 / a.G, p1 = p_first + (r0 + max(nr, 1) - 1) / a.G;
  Reach reach = reach_of(a, held, p0, p1);
  if (nr <= 0) reach.tiles = 0;
  // this CTA's tiles, of which its rings take every R-th
  const int first = (int)((long long)reach.tiles * split / a.splits);
  const int count = (int)((long long)reach.tiles * (split + 1) / a.splits) - first;
  const int mine = (count - group + R - 1) / R;

  // ---- copies: tile i of this ring into stage i % S
  const bool producer = part == 0;
  const uint32_t ring = smem_u32(sm + SL::ring) + group * S * SL::kStageBytes;
  int held_at = -1;  // this ring's tiles held_at + lane: the records of their two blocks (0: no copy)
  unsigned long long rec0 = 0, rec1 = 0;
  int issued = 0;
  auto tile_first = [&](int i) { return reach.tile(first + group + R * i) * kTile; };
  auto issue = [&](int i) {  // (a converged warp)
    if (held_at < 0 || i >= held_at + 32) {
      held_at = i;
      const int k0 = tile_first(i + lane);
      const bool in = i + lane < mine;
      auto record = [&](int key) -> unsigned long long {
        if (!in || !reach.any(key, kBlock)) return 0;
        const int id = page_of(a.c, b, key / kBlock);
        if (id >= 0) return (unsigned long long)record_of(a.c, id, hk, key / kBlock);
        cross_fail(a.status, (int)DF_ERR_INVALID_ARG);  // tokens without a page
        return 0;
      };
      rec0 = record(k0);
      rec1 = record(k0 + kBlock);
    }
    const unsigned long long x0 = __shfl_sync(0xffffffffu, rec0, i - held_at), x1 = __shfl_sync(0xffffffffu, rec1, i - held_at);
    const int s = i % S;
    if (lane == 0) {
      const uint32_t dst = ring + s * SL::kStageBytes;
      have[s] = (x0 != 0 ? 1 : 0) | (x1 != 0 ? 2 : 0);
      mbar_expect_tx(full + s, ((x0 != 0 ? 1u : 0u) + (x1 != 0 ? 1u : 0u)) * SL::kRecord);
      if (x0 != 0 && x1 == x0 + SL::kRecord) {
        bulk_load(dst, x0, 2 * SL::kRecord, full + s);
      } else {
        if (x0 != 0) bulk_load(dst, x0, SL::kRecord, full + s);
        if (x1 != 0) bulk_load(dst + SL::kRecord, x1, SL::kRecord, full + s);
      }
    }
    __syncwarp();
    issued = i + 1;
  };
  if (producer)
    for (int i = 0; i < min(S, mine); ++i) issue(i);

  // ---- query rows g and g + 8 of the warp, as fp16 (bf16: times a power of two, exactly)
  uint32_t qa[SLABS][2][4];
  float ks_row[2];
  int pos[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r = r0 + 16 * part + g + 8 * h;
    const bool in = r < rows && h < kHalves;
    pos[h] = in ? p_first + r / a.G : INT_MIN;
    ks_row[h] = a.kscale;
    uint4 v[SLABS];
    const uint4* src = reinterpret_cast<const uint4*>(
        static_cast<const uint16_t*>(a.q) + ((size_t)(q0 + (in ? r / a.G : 0)) * a.H + (size_t)hk * a.G + (in ? r % a.G : 0)) * D + 8 * t);
#pragma unroll
    for (int c = 0; c < SLABS; ++c) v[c] = in ? src[4 * c] : make_uint4(0u, 0u, 0u, 0u);
    if (a.bf16) {
      uint32_t top = 0;
#pragma unroll
      for (int c = 0; c < SLABS; ++c) {
        const uint32_t w[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) top = max(top, max(w[e] & 0x7fffu, (w[e] >> 16) & 0x7fffu));
      }
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const uint32_t e = min(max(top >> 7, 1u), 253u);  // the largest is below 2^(e - 126)
      const float down = __uint_as_float((254u - e) << 23);
      ks_row[h] = a.kscale * __uint_as_float(e << 23);
#pragma unroll
      for (int c = 0; c < SLABS; ++c) {
        uint32_t* w = reinterpret_cast<uint32_t*>(&v[c]);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          w[i] = pack_f16x2(__uint_as_float(w[i] << 16) * down, __uint_as_float(w[i] & 0xffff0000u) * down);
      }
    }
#pragma unroll
    for (int c = 0; c < SLABS; ++c) {
      qa[c][0][h] = v[c].x;
      qa[c][0][2 + h] = v[c].y;
      qa[c][1][h] = v[c].z;
      qa[c][1][2 + h] = v[c].w;
    }
  }

  // ---- the loop
  float o[SLABS][4][4];
#pragma unroll
  for (int c = 0; c < SLABS; ++c)
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[c][m][e] = 0.f;
  float m_run[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.f, 0.f};
  // bytes from a record's start to this lane's reads: K row of key (g / 2, 2 j + g % 2), V row of key (t, i)
  auto key_of = [](int tt, int i) { return 4 * i + ((tt + 2 * (i & 1)) & 3); };
  const bool rows_here = 16 * part < nr;
  bool ok = true;
  int done = 0;
#pragma unroll 1
  for (int i = 0; i < mine; ++i) {
    const int s = i % S;
    ok = ok && cross_wait(full + s, (i / S) & 1, a.budget, s_abort);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) break;
    done = i + 1;
    const uint32_t base = ring + s * SL::kStageBytes;
    const int first_key = tile_first(i), here = have[s];
    // every key of the tile counts for every row of the CTA
    const bool whole = here == 3 && (!a.causal ? first_key + kTile <= held
                                               : first_key + kTile <= p0 + 1 &&
                                                     (a.window == 0 || p1 - a.window < first_key || first_key + kTile <= a.sinks));
    if (rows_here) {
      float sc[2][2][4], vs[2];
#pragma unroll
      for (int blk = 0; blk < 2; ++blk) {
        const uint32_t rec = base + blk * SL::kRecord;
        const uint2 sw = lds64(rec + 32 * D);
        const float ksc = __uint_as_float(sw.x);
        vs[blk] = (here >> blk) & 1 ? __uint_as_float(sw.y) : 0.f;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float acc[4];
          const uint32_t row = rec + 32 * key_of(g >> 1, 2 * j + (g & 1)) + 8 * t;
#pragma unroll
          for (int c = 0; c < SLABS; ++c) {
            const uint2 w = lds64(row + 512 * c);
            uint32_t b0, b1;
            codes4_f16(w.x, b0, b1);
            if (c == 0)
              mma_f16_first(acc, qa[c][0], b0, b1);
            else
              mma_f16(acc, qa[c][0], b0, b1);
            codes4_f16(w.y, b0, b1);
            mma_f16(acc, qa[c][1], b0, b1);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[blk][j][e] = acc[e] * ksc * ks_row[e >> 1];
        }
      }
      uint32_t gone = 0;  // of this lane's keys (t, i), bit 4 blk + i: those that no row counts
      if (!whole) {
#pragma unroll
        for (int blk = 0; blk < 2; ++blk)
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const int key = first_key + kBlock * blk + key_of(t, 2 * j + x);
              const bool there = (here >> blk) & 1 && reach.any(key, 1);
              if (!there) gone |= 1u << (4 * blk + 2 * j + x);
#pragma unroll
              for (int h = 0; h < kHalves; ++h) {
                const bool seen = there && (!a.causal || (key <= pos[h] && (a.window == 0 || key > pos[h] - a.window || key < a.sinks)));
                if (!seen) sc[blk][j][2 * h + x] = -INFINITY;
              }
            }
      }
      uint32_t pa[2][4];
#pragma unroll
      for (int h = 0; h < kHalves; ++h) {
        float mt = fmaxf(fmaxf(fmaxf(sc[0][0][2 * h], sc[0][0][2 * h + 1]), fmaxf(sc[0][1][2 * h], sc[0][1][2 * h + 1])),
                         fmaxf(fmaxf(sc[1][0][2 * h], sc[1][0][2 * h + 1]), fmaxf(sc[1][1][2 * h], sc[1][1][2 * h + 1])));
        mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 1));
        mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 2)) - kUp;
        if (__any_sync(0xffffffffu, mt > m_run[h])) {
          const float m_new = fmaxf(m_run[h], mt);
          const float f = m_new > m_run[h] ? ex2(m_run[h] - m_new) : 1.f;
          m_run[h] = m_new;
          l_run[h] *= f;
#pragma unroll
          for (int c = 0; c < SLABS; ++c)
#pragma unroll
            for (int m = 0; m < 4; ++m) {
              o[c][m][2 * h] *= f;
              o[c][m][2 * h + 1] *= f;
            }
        }
        const float shift = m_run[h] == -INFINITY ? INFINITY : m_run[h];
        float sum = 0.f;
#pragma unroll
        for (int blk = 0; blk < 2; ++blk)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float x = ex2(sc[blk][j][2 * h] - shift), y = ex2(sc[blk][j][2 * h + 1] - shift);
            sum += x + y;
            pa[blk][2 * j + h] = pack_f16x2(x, y);
          }
        l_run[h] += sum;
      }
      if (HALF) pa[0][1] = pa[0][3] = pa[1][1] = pa[1][3] = 0u;
#pragma unroll
      for (int blk = 0; blk < 2; ++blk) {
        const uint32_t rec = base + blk * SL::kRecord + 16 * D + 4 * g;
#pragma unroll
        for (int c = 0; c < SLABS; ++c) {
          uint32_t w[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) w[x] = lds32(rec + 512 * c + 32 * key_of(t, x));
          if (!whole) {
#pragma unroll
            for (int x = 0; x < 4; ++x)
              if ((gone >> (4 * blk + x)) & 1u) w[x] = 0u;
          }
          // four tokens of four columns -> four columns of four tokens
#pragma unroll
          for (int two = 0; two < 2; ++two) {  // columns 2 two, 2 two + 1
            uint32_t x[2], y[2];
            codes4_f16(prmt(w[0], w[1], two ? 0x7362 : 0x5140), x[0], x[1]);
            codes4_f16(prmt(w[2], w[3], two ? 0x7362 : 0x5140), y[0], y[1]);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float acc[4];
              float(&to)[4] = o[c][2 * two + e];
              mma_f16_first(acc, pa[blk], x[e], y[e]);
#pragma unroll
              for (int h = 0; h < kHalves; ++h) {
                const float2 sum = fma2(make_float2(acc[2 * h], acc[2 * h + 1]), make_float2(vs[blk], vs[blk]),
                                        make_float2(to[2 * h], to[2 * h + 1]));
                to[2 * h] = sum.x;
                to[2 * h + 1] = sum.y;
              }
            }
          }
        }
      }
    }
    __syncwarp();
    if (WR > 1 && lane == 0) mbar_arrive(empty + s);
    if (producer && i + S < mine) {
      if (WR > 1) {
        ok = cross_wait(empty + s, (i / S) & 1, a.budget, s_abort);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
      }
      issue(i + S);
    }
  }
  // a wait ran out: no copy may still be landing when the ring is used again
  if (producer)
    for (int i = done; i < issued; ++i) mbar_wait(full + i % S, (i / S) & 1, kDrainBudget);
  __syncthreads();

  // ---- the CTA's rows: its warps' parts together
  float* so = reinterpret_cast<float*>(sm + SL::o_warp);
  float2* sml = reinterpret_cast<float2*>(sm + SL::ml_warp);
#pragma unroll
  for (int h = 0; h < kHalves; ++h) {
    float l = l_run[h];
    l += __shfl_xor_sync(0xffffffffu, l, 1);
    l += __shfl_xor_sync(0xffffffffu, l, 2);
    const int r = warp * 16 + g + 8 * h;
    if (t == 0) sml[r] = make_float2(m_run[h], l);
#pragma unroll
    for (int c = 0; c < SLABS; ++c)
#pragma unroll
      for (int x = 0; x < 2; ++x)
        *reinterpret_cast<float4*>(so + r * SL::kPitch + 32 * c + 8 * t + 4 * x) =
            make_float4(o[c][0][2 * h + x], o[c][1][2 * h + x], o[c][2][2 * h + x], o[c][3][2 * h + x]);
  }
  __syncthreads();
  constexpr int kPieces = D / 4;
  const bool alone = a.splits == 1;
  float4* s_ml = reinterpret_cast<float4*>(sm + SL::ml_cta);
  float* s_o = reinterpret_cast<float*>(sm + SL::o_cta);
  const bool failed = *s_abort != 0;
  auto store = [&](int row, int piece, float m, float l, float (&v)[4]) {
    const float inv = l != 0.f ? rcp(l) : 0.f;  // (a NaN stays one)
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] *= inv;
    const int r = r0 + row;
    const size_t at = (size_t)(q0 + r / a.G) * a.H + (size_t)hk * a.G + r % a.G;
    uint32_t lo, hi;
    if (a.bf16) {
      lo = pack_bf16x2(v[0], v[1]);
      hi = pack_bf16x2(v[2], v[3]);
    } else {
      lo = pack_f16x2(v[0], v[1]);
      hi = pack_f16x2(v[2], v[3]);
    }
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at * D + 4 * piece) = make_uint2(lo, hi);
    if (a.lse && piece == 0) a.lse[at] = l != 0.f ? (m + lg2(l)) * kLn2 : -INFINITY;
  };
  for (int i = threadIdx.x; i < max(nr, 0) * kPieces; i += kThreads) {
    const int row = i / kPieces, piece = i - row * kPieces;
    const int w0 = row >> 4, rr = row & 15;
    float m = -INFINITY, l = 0.f, v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < R; ++k) m = fmaxf(m, sml[(k * WR + w0) * 16 + rr].x);
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const int at = (k * WR + w0) * 16 + rr;
      const float2 s = sml[at];
      const float f = s.x != -INFINITY ? ex2(s.x - m) : 0.f;
      l += f > 0.f || s.y != s.y ? s.y * (f > 0.f ? f : 1.f) : 0.f;
      const float4 x = *reinterpret_cast<const float4*>(so + at * SL::kPitch + 4 * piece);
      if (f > 0.f) {
        v[0] += f * x.x;
        v[1] += f * x.y;
        v[2] += f * x.z;
        v[3] += f * x.w;
      }
    }
    if (alone) {
      if (!failed) store(row, piece, m, l, v);
    } else {
      *reinterpret_cast<float4*>(s_o + row * D + 4 * piece) = make_float4(v[0], v[1], v[2], v[3]);
      if (piece == 0) s_ml[row] = make_float4(m, l, 0.f, 0.f);
    }
  }
  if (!alone) {
    cluster_sync();
    const uint32_t o_addr = smem_u32(s_o), ml_addr = smem_u32(s_ml);
    for (int i = split * kThreads + threadIdx.x; i < max(nr, 0) * kPieces; i += kThreads * a.splits) {
      const int row = i / kPieces, piece = i - row * kPieces;
      float m = -INFINITY, l = 0.f, v[4] = {0.f, 0.f, 0.f, 0.f};
      for (int k = 0; k < a.splits; ++k) m = fmaxf(m, ld_cluster(map_rank(ml_addr + 16 * row, k)).x);
      for (int k = 0; k < a.splits; ++k) {
        const float4 s = ld_cluster(map_rank(ml_addr + 16 * row, k));
        const float f = s.x != -INFINITY ? ex2(s.x - m) : 0.f;
        l += f > 0.f || s.y != s.y ? s.y * (f > 0.f ? f : 1.f) : 0.f;
        if (f > 0.f) {
          const float4 x = ld_cluster(map_rank(o_addr + 4 * (row * D + 4 * piece), k));
          v[0] += f * x.x;
          v[1] += f * x.y;
          v[2] += f * x.z;
          v[3] += f * x.w;
        }
      }
      if (!failed) store(row, piece, m, l, v);
    }
    cluster_sync();  // no CTA leaves while another one reads its shared memory
  }
  if (threadIdx.x == 0) cross_report(s_abort, a.status);
}

// CTAs of `items` that share one, 1 to 8 (a cluster): the number for which the CTAs' rounds,
// each as long as its share of the tiles and what it costs to begin and to join, are shortest.
int splits_for(long long items, long long tiles, int rings, long long slots) {
  constexpr long long kBegin = 6;  // in tiles of a warp
  int best = 1;
  long long least = LLONG_MAX;
  for (int n = 1; n <= 8; ++n) {
    const long long rounds = (items * n + slots - 1) / slots;
    const long long cost = rounds * ((tiles + (long long)n * rings - 1) / (n * rings) + kBegin);
    if (cost < least) {
      least = cost;
      best = n;
    }
  }
  return best;
}

template <int SLABS, int WR, bool HALF>
cudaError_t launch(DecodeArgs a, long long tiles, cudaStream_t s) {
  auto kernel = decode_kernel<SLABS, WR, HALF>;
  constexpr int bytes = DecodeSmem<SLABS, WR>::bytes;
  static std::atomic<uint64_t> done{0};
  static std::atomic<int> resident{0};  // CTAs an SM holds
  cudaError_t e = prepare_kernel((const void*)kernel, bytes, 0, &done);
  if (e != cudaSuccess) return e;
  int per_sm = resident.load(std::memory_order_relaxed);
  if (per_sm == 0) {
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, kThreads, bytes);
    if (e != cudaSuccess) return e;
    per_sm = std::max(per_sm, 1);
    resident.store(per_sm, std::memory_order_relaxed);
  }
  const long long items = (long long)a.B * a.c.Hk * a.row_tiles;
  a.splits = splits_for(items, tiles, kWarps / WR, (long long)device_sms() * per_sm);
  if (items * a.splits > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  const int grid = (int)(items * a.splits);
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
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <int SLABS>
cudaError_t launch_rows(const DecodeArgs& a, int wr, bool half, long long tiles, cudaStream_t s) {
  if (half) return launch<SLABS, 1, true>(a, tiles, s);
  return wr == 1 ? launch<SLABS, 1, false>(a, tiles, s)
                 : wr == 2 ? launch<SLABS, 2, false>(a, tiles, s) : launch<SLABS, 4, false>(a, tiles, s);
}

bool al16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

}  // namespace
}  // namespace dfa

using namespace dfa;

extern "C" df_status df_cache_attn(const void* q, const int32_t* cu_seqlens_q, int B, int H, int Hk, int Lq, int total_q,
                                   int d, float scale, int causal, int window, int sinks, df_dtype dtype,
                                   const void* cache, int n_pages, int page, const int32_t* pages, int max_pages,
                                   const int32_t* lengths, int max_length, void* out, float* lse, int32_t* status,
                                   df_stream_t stream) {
  DecodeArgs a;
  if (dtype != DF_BF16 && dtype != DF_FP16 && dtype != DF_FP32) return DF_ERR_INVALID_ARG;
  df_status st = cache_check(cache, pages, lengths, B, Hk, d, page, n_pages, max_pages, &a.c);
  if (st != DF_OK) return st;
  if (H < 1 || H % Hk != 0 || Lq < 0 || total_q < 0 || max_length < 0 || !(scale > 0.f) || !(scale <= 2.0e38f))
    return DF_ERR_INVALID_ARG;
  if (!self_reach(&window, &sinks) || (!causal && (window != 0 || sinks != 0))) return DF_ERR_INVALID_ARG;
  if (!cu_seqlens_q && (long long)B * Lq != total_q) return DF_ERR_INVALID_ARG;
  if (dtype == DF_FP32 || total_q > (1 << 30) || H > 65536 || (long long)Lq * (H / Hk) > (1 << 30)) return DF_ERR_UNSUPPORTED;
  if (((uintptr_t)cu_seqlens_q & 3u) != 0 || ((uintptr_t)lse & 3u) != 0) return DF_ERR_ALIGNMENT;
  if (total_q == 0 || B == 0 || Lq == 0) return DF_OK;
  if (!q || !out) return DF_ERR_INVALID_ARG;
  if (!al16(q) || !al16(out)) return DF_ERR_ALIGNMENT;
  const size_t bytes = (size_t)total_q * H * d * 2;
  if (overlapping({{out, bytes}, {lse, (size_t)total_q * H * 4}},
                  {{q, bytes}, {cache, cache_bytes(Hk, d, page, n_pages)}, {pages, (size_t)B * max_pages * 4},
                   {lengths, (size_t)B * 4}, {cu_seqlens_q, ((size_t)B + 1) * 4}}))
    return DF_ERR_INVALID_ARG;
  a.q = q;
  a.cu_q = cu_seqlens_q;
  a.out = out;
  a.lse = lse;
  a.B = B;
  a.H = H;
  a.G = H / Hk;
  a.Lq = Lq;
  a.Tq = total_q;
  a.causal = causal != 0;
  a.window = window;
  a.sinks = sinks;
  a.bf16 = dtype == DF_BF16;
  a.kscale = (float)((double)scale * 1.4426950408889634);
  a.status = status;
  a.budget = wait_budget();
  const int rows = Lq * a.G;
  const int wr = rows <= 16 ? 1 : rows <= 32 ? 2 : 4;
  a.row_tiles = (rows + 16 * wr - 1) / (16 * wr);
  if ((long long)B * Hk * a.row_tiles > 0x7fffffffll / 8) return DF_ERR_UNSUPPORTED;
  // the tokens that a tile of rows sees at most, in tiles
  long long tiles = ((long long)std::min<long long>(max_length, (long long)max_pages * page) + kTile - 1) / kTile;
  if (window > 0) tiles = std::min<long long>(tiles, ((long long)window + Lq + sinks) / kTile + 3);
  cudaStream_t s = (cudaStream_t)stream;
  const bool half = rows <= 8;
  cudaError_t e;
  switch (d / 32) {
    case 1: e = launch_rows<1>(a, wr, half, tiles, s); break;
    case 2: e = launch_rows<2>(a, wr, half, tiles, s); break;
    case 3: e = launch_rows<3>(a, wr, half, tiles, s); break;
    default: e = launch_rows<4>(a, wr, half, tiles, s); break;
  }
  return e == cudaSuccess ? DF_OK : DF_ERR_CUDA;
}
