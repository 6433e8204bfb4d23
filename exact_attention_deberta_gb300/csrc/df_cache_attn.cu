// Attention of a few queries for each sequence to the 8-bit cache: single tokens and short
// runs of them (causal, with a window and sinks), or queries that see every token held (the
// encoder's states).
//
//   s_ij = scale ks_j (q_i . ck_j),  o_i = sum_j exp(s_ij - lse_i) vs_j cv_j
// over the visible tokens j, with codes ck, cv and scales ks, vs of j's block.
//
// Bound by reading the cache once: 2 d + 1 bytes a token and key head, for 4 d G n flops.  So
// nothing but the tensor core's old instructions (m16n8k16: a tile of 16 query rows, one block
// of 16 keys) stands between the bytes and the sums:
//   - A CTA has four warps (or eight), each on its own: a ring of bulk copies (two blocks' records, one
//     contiguous piece where they are on one page) in shared memory, waits, products. Nothing
//     in the loop meets another warp (WR > 1: query rows that do not fit 16 are shared out, and
//     WR warps read the same ring).
//   - Codes become fp16 exactly (one instruction for two). The scale of K multiplies scores, that
//     of V the products of a block, both in fp32.
//   - The order of keys in a block is free, and so is that of columns in a sum: lane (g, t) =
//     (lane / 4, lane % 4) takes 8 columns of a K row at once and 4 tokens x 4 columns of V,
//     transposed by byte permutes; key i of lane t is 4 i + ((t + 2 (i & 1)) & 3), for which
//     neither read meets a bank conflict and the scores a lane gets are the weights it needs.
//   - A weight is held times 2^14, so that fp16 keeps its digits down to 2^-28 of the largest; the scale of
//     V takes that back, so that O is a sum of weights of 1 at most.
// Sequences are cut over the CTAs of a cluster where there are few of them; the parts are joined
// through distributed shared memory, without a workspace or a second launch.
//
// Measured (GB300): 64 requests of up to 8192 tokens, 24 heads, d = 64, bf16 (1.0 GB): 161 us, 6.3 TB/s;
// 64 sequences of up to 4096 states, 4 key heads of 4 heads, d = 128, fp16: 40 us, 4.3 TB/s; 16 x 4
// tokens of 32 heads sharing 8, a window of 4096, d = 128, bf16: 39 us, 3.5 TB/s; one request of 512
// tokens, 12 heads: 6.5 us. A tile of 32 keys takes a warp some 650 instructions at d = 128, and alone
// on its scheduler 2600 cycles: most of them wait for a result of the one before (counters: an
// instruction every 4 cycles, no pipe above a fifth). So long rows are bound by the number of warps,
// 12 an SM where the records of d = 128 lie in shared memory (8 with all 16 rows in registers).
#include <limits.h>

#include <algorithm>

#include "df_cache.cuh"
#include "df_cross_fwd.cuh"

namespace dfa {
namespace {

using namespace ptx;

// A tile is the keys of one copy: two blocks.  (Four at d = 64: 166 us where two take 160, for 24
// heads and 64 requests of up to 8192 tokens; one at d = 128: the same as two.)
constexpr int NB = 2, kKeys = NB * kBlock;
static_assert(NB == 2, "the scales of a tile's values are a pair");
constexpr float kUp = 14.f, kDown = 1.f / 16384.f;  // (2^-14)

struct DecodeArgs {
  CacheView c;
  const void* q;
  const int32_t* cu_q;  // [B + 1] or NULL
  void* out;
  float* lse;           // or NULL
  int B, H, G, Lq, Tq;
  unsigned by_G;        // 65536 / G + 1
  int row_tiles;        // CTAs that share a sequence's query rows
  int splits;           // and its keys (cluster size)
  int longest_first;    // (at most a CTA's threads)
  int causal, window, sinks, bf16;
  float kscale;         // scale log2(e)
  int32_t* status;
  unsigned long long budget;
};

template <int SLABS, int WR, int WARPS>
struct DecodeSmem {
  static constexpr int D = 32 * SLABS;
  static constexpr int kRings = WARPS / WR;
  static constexpr int kStages = SLABS == 1 ? 6 : SLABS == 2 ? 3 : 2;
  static constexpr uint32_t kRecord = 32 * D + 16;
  static constexpr uint32_t kStageBytes = NB * kRecord;
  static constexpr uint32_t ring = 0;  // [kRings][kStages][records of a tile]
  static constexpr uint32_t ring_bytes = kRings * kStages * kStageBytes;
  // after the loop, over the ring: each warp's O, and the CTA's
  static constexpr int kPitch = D + 4;
  static constexpr uint32_t o_warp = 0;  // float [WARPS][16][kPitch]
  static constexpr uint32_t o_cta = WARPS * 16 * kPitch * 4;  // float [16 WR][D]
  static constexpr uint32_t joined = o_cta + 16 * WR * D * 4;
  static constexpr uint32_t ml_warp = (ring_bytes > joined ? ring_bytes : joined);  // float2 [WARPS][16]
  static constexpr uint32_t ml_cta = ml_warp + WARPS * 16 * 8;                     // float4 [16 WR]
  static constexpr uint32_t bars = ml_cta + 64 * 16;                                // full, empty [kRings][kStages]
  static constexpr uint32_t have = bars + 2 * kRings * kStages * 8;                 // int [kRings][kStages]
  static constexpr uint32_t recs = (have + kRings * kStages * 4 + 7) & ~7u;  // 64-bit [kRings][32 tiles][blocks]: records to copy
  static constexpr uint32_t reach = recs + kRings * 32 * NB * 8;
  static constexpr uint32_t misc = reach + 32;
  static constexpr uint32_t bytes = (misc + 4 + 15) & ~15u;
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

// As cross_wait.  A copy lands within the time that one try may sleep, so that a budget below that
// has to bound the try as well.
__device__ __forceinline__ bool ring_wait(uint64_t* bar, uint32_t parity, unsigned long long budget,
                                          volatile int* abort) {
  if (budget > 100000) return cross_wait(bar, parity, budget, abort);
  const long long t0 = clock64();
  do {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    if (done) return true;
    if ((unsigned long long)(clock64() - t0) > budget) *abort = 1;
  } while (*abort == 0);
  return false;
}

// The tokens that a tile of query rows, at positions p0 .. p1, sees: those before `head` and
// those from lo to end - 1; in tiles of kKeys, the first `heads` and then those from `skip`
// tiles further on.
struct Reach {
  int head, lo, end, heads, skip, tiles;
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
  r.heads = (r.head + kKeys - 1) / kKeys;
  r.skip = max(r.lo / kKeys - r.heads, 0);
  r.tiles = (r.end + kKeys - 1) / kKeys - r.skip;
  return r;
}

// The query rows of a CTA or worker and what they see.
struct Rows {
  int b, hk, nr;     // `nr` rows, token by token and head by head within the key head's G
  int t0, h0;        // the first one's token (of the sequence's queries) and head
  int q0, held;      // the sequence's first row of q; tokens held
  int p0, p1;        // positions of the first and the last row
  // Row i: its token, counted from t0, and its head
  __device__ __forceinline__ void place(const DecodeArgs& a, int i, int* token, int* head) const {
    const int x = h0 + i;  // below 192: the product is exact
    *token = (int)((unsigned)x * a.by_G >> 16);
    *head = x - *token * a.G;
  }
};
// A sequence's queries and tokens, as far as they can be believed (`tell`: what cannot is reported).
__device__ __forceinline__ void sequence(const DecodeArgs& a, int b, bool tell, int* q0, int* nq, int* held) {
  const CrossSide side = {a.cu_q, a.Lq, a.Tq};
  *nq = seq_rows(side, b, tell ? a.status : nullptr, q0);
  *held = a.c.lengths[b];
  const bool bad = *held < 0 || *held > a.c.max_pages * a.c.page;  // (the product is at most 2^30)
  if (bad) *held = 0;
  if (tell && (bad || *nq > a.Lq)) cross_fail(a.status, (int)DF_ERR_INVALID_ARG);
}
__device__ __forceinline__ Rows rows_of(const DecodeArgs& a, int b, int hk, int rt, int per_tile, bool tell) {
  Rows w;
  int nq;
  sequence(a, b, tell, &w.q0, &nq, &w.held);
  w.b = b;
  w.hk = hk;
  // (rows beyond Lq, for which there may be no worker, are left alone)
  w.nr = min(per_tile, min(nq, a.Lq) * a.G - rt * per_tile);
  w.t0 = rt * per_tile / a.G;
  w.h0 = rt * per_tile - w.t0 * a.G;
  w.p0 = w.held - nq + w.t0;
  int last, head;
  w.place(a, max(w.nr, 1) - 1, &last, &head);
  w.p1 = w.p0 + last;
  return w;
}

// The records of the NB blocks from token `key` on (a multiple of 16), 0 where nothing is to be
// copied: blocks of which no token is seen, and those without a page.
__device__ __forceinline__ void records_at(const DecodeArgs& a, const Reach& reach, int b, int hk, int key,
                                           unsigned long long (&rec)[NB]) {
  const unsigned per = (unsigned)a.c.page / kBlock;
  unsigned at = (unsigned)key / kBlock / per, in = (unsigned)key / kBlock - at * per;
  unsigned long long first = 0;  // the page's first record of the head
  bool looked = false;
#pragma unroll
  for (int k = 0; k < NB; ++k) {
    rec[k] = 0;
    if (reach.any(key + k * kBlock, kBlock)) {
      if (!looked) {
        const int id = at < (unsigned)a.c.max_pages ? a.c.pages[(size_t)b * a.c.max_pages + at] : -1;
        const bool good = (unsigned)id < (unsigned)a.c.n_pages;
        if (!good) cross_fail(a.status, (int)DF_ERR_INVALID_ARG);  // tokens without a page
        first = good ? (unsigned long long)(a.c.base + ((size_t)id * a.c.Hk + hk) * per * record_bytes(a.c.d)) : 0;
        looked = true;
      }
      if (first != 0) rec[k] = first + (unsigned long long)in * record_bytes(a.c.d);
    }
    if (++in == per) {
      in = 0;
      ++at;
      looked = false;
    }
  }
}

// Key i of lane t's four in a block.
__device__ __forceinline__ int key_of(int t, int i) { return 4 * i + ((t + 2 * (i & 1)) & 3); }

// A warp's 16 query rows and their running state; HALF: the upper 8 are empty.
template <int SLABS, bool HALF, bool ACROSS>
struct Softmax {
  static constexpr int D = 32 * SLABS, kHalves = HALF ? 1 : 2;
  static constexpr uint32_t kRecord = 32 * D + 16;
  int whole_from, whole_to;  // tiles that begin in between have no key that a row does not see
  uint32_t qa[SLABS][2][4];  // the rows as fp16, operands of the scores
  float ks_row[2];
  int pos[2];                // rows g and g + 8: their positions
  float o[SLABS][4][4];
  float m_run[2], l_run[2];  // l_run: this lane's keys only

  // (bf16 rows become fp16 times a power of two, exactly down to 2^-32 of a row's largest, which comes to
  // 2^15 .. 65280: fp16's smallest step is 2^-24, and eight digits are to stand above it)
  __device__ __forceinline__ void begin(const DecodeArgs& a, const Rows& w, int part) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    whole_to = (a.causal ? min(w.p0 + 1, w.held) : w.held) - kKeys;
    whole_from = a.causal && a.window != 0 ? w.p1 - a.window + 1 : 0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int i = 16 * part + g + 8 * h;
      const bool in = i < w.nr && h < kHalves;
      int token = 0, head = 0;
      if (in) w.place(a, i, &token, &head);
      pos[h] = in ? w.p0 + token : INT_MIN;
      ks_row[h] = a.kscale;
      m_run[h] = -INFINITY;
      l_run[h] = 0.f;
      uint4 v[SLABS];
      const uint4* src = reinterpret_cast<const uint4*>(
          static_cast<const uint16_t*>(a.q) +
          ((size_t)(w.q0 + w.t0 + token) * a.H + w.hk * a.G + head) * D + 8 * t);
#pragma unroll
      for (int c = 0; c < SLABS; ++c) v[c] = in ? src[4 * c] : make_uint4(0u, 0u, 0u, 0u);
      if (a.bf16) {
        uint32_t top = 0;
#pragma unroll
        for (int c = 0; c < SLABS; ++c) {
          const uint32_t x[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) top = max(top, max(x[e] & 0x7fffu, (x[e] >> 16) & 0x7fffu));
        }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // the largest is below 2^(e - 126); where it is below 2^-94, every step of bf16 is one of fp16 at 33
        const uint32_t e = min(max(top >> 7, 33u), 254u);
        const float down = __uint_as_float((269u - e) << 23);  // 2^(142 - e)
        ks_row[h] = a.kscale * __uint_as_float((e - 15u) << 23);
#pragma unroll
        for (int c = 0; c < SLABS; ++c) {
          uint32_t* x = reinterpret_cast<uint32_t*>(&v[c]);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            x[i] = pack_f16x2(__uint_as_float(x[i] << 16) * down, __uint_as_float(x[i] & 0xffff0000u) * down);
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
#pragma unroll
    for (int c = 0; c < SLABS; ++c)
#pragma unroll
      for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[c][m][e] = 0.f;
  }

  // One tile: its records at `base` (shared memory), of which those in `here` were copied.
  __device__ __forceinline__ void tile(const DecodeArgs& a, const Reach* reach, uint32_t base, int first_key,
                                       int here) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    // every key of the tile counts for every row
    const bool whole = here == (1 << NB) - 1 && first_key <= whole_to &&
                       (first_key >= whole_from || first_key + kKeys <= a.sinks);
    float sc[NB][2][4], vs[NB], f[NB][kHalves];
#pragma unroll
    for (int blk = 0; blk < NB; ++blk) {
      const uint32_t rec = base + blk * kRecord;
      const uint2 sw = lds64(rec + 32 * D);
      // (positive, so that a score of -infinity stays one)
#pragma unroll
      for (int h = 0; h < kHalves; ++h) f[blk][h] = fmaxf(__uint_as_float(sw.x) * ks_row[h], 1.17549435e-38f);
      vs[blk] = __uint_as_float(sw.y);
    }
    // Products in the order of their sums, or, so that those that follow one another are of different
    // sums, slab by slab of all keys: long rows that leave the registers for it (d = 128, a key head's
    // 4 heads, one request of 65536 tokens: 53 -> 48 us; 8 rows of 16 tokens: 107 -> 102; but d = 64,
    // 64 requests: 161 -> 162, and 16 rows of d = 128: 33.1 -> 33.8).
    constexpr int kOuter = ACROSS ? 1 : 2 * NB, kInner = ACROSS ? 2 * NB : 1;
#pragma unroll
    for (int out = 0; out < kOuter; ++out)
#pragma unroll
      for (int c = 0; c < SLABS; ++c) {
        uint2 x[kInner];
#pragma unroll
        for (int i = 0; i < kInner; ++i) {
          const int at = out + i, blk = at >> 1, j = at & 1;
          x[i] = lds64(base + blk * kRecord + 32 * key_of(g >> 1, 2 * j + (g & 1)) + 8 * t + 512 * c);
        }
#pragma unroll
        for (int part = 0; part < 2; ++part)
#pragma unroll
          for (int i = 0; i < kInner; ++i) {
            float(&to)[4] = sc[(out + i) >> 1][(out + i) & 1];
            uint32_t b0, b1;
            codes4_f16(part ? x[i].y : x[i].x, b0, b1);
            if (c == 0 && part == 0)
              mma_f16_first(to, qa[0][0], b0, b1);
            else
              mma_f16(to, qa[c][part], b0, b1);
          }
      }
    uint32_t gone = 0;  // of this lane's keys (t, i), bit 4 blk + i: those that no row counts
    if (!whole) {
#pragma unroll
      for (int blk = 0; blk < NB; ++blk) {
        if (!((here >> blk) & 1)) {  // (its scales are not there either)
          vs[blk] = 0.f;
#pragma unroll
          for (int h = 0; h < kHalves; ++h) f[blk][h] = 1.f;
        }
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int key = first_key + kBlock * blk + key_of(t, 2 * j + x);
            const bool there = (here >> blk) & 1 && reach->any(key, 1);
            if (!there) gone |= 1u << (4 * blk + 2 * j + x);
#pragma unroll
            for (int h = 0; h < kHalves; ++h) {
              const bool seen =
                  there && (!a.causal || (key <= pos[h] && (a.window == 0 || key > pos[h] - a.window || key < a.sinks)));
              if (!seen) sc[blk][j][2 * h + x] = -INFINITY;
            }
          }
      }
    }
    uint32_t pa[NB][4];
#pragma unroll
    for (int h = 0; h < kHalves; ++h) {
      float mt = -INFINITY;
#pragma unroll
      for (int blk = 0; blk < NB; ++blk) {
        const float top = fmaxf(fmaxf(sc[blk][0][2 * h], sc[blk][0][2 * h + 1]), fmaxf(sc[blk][1][2 * h], sc[blk][1][2 * h + 1]));
        mt = fmaxf(mt, top * f[blk][h]);
      }
      mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 1));
      mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 2)) - kUp;
      if (__any_sync(0xffffffffu, mt > m_run[h])) {
        const float m_new = fmaxf(m_run[h], mt);
        const float down = m_new > m_run[h] ? ex2(m_run[h] - m_new) : 1.f;
        m_run[h] = m_new;
        l_run[h] *= down;
#pragma unroll
        for (int c = 0; c < SLABS; ++c)
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            o[c][m][2 * h] *= down;
            o[c][m][2 * h + 1] *= down;
          }
      }
      const float shift = m_run[h] == -INFINITY ? -INFINITY : -m_run[h];
      float2 sum = make_float2(0.f, 0.f);
#pragma unroll
      for (int blk = 0; blk < NB; ++blk)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float2 z = fma2(make_float2(sc[blk][j][2 * h], sc[blk][j][2 * h + 1]), make_float2(f[blk][h], f[blk][h]),
                                make_float2(shift, shift));
          const float2 p = make_float2(ex2(z.x), ex2(z.y));
          sum = add2(sum, p);
          pa[blk][2 * j + h] = pack_f16x2(p.x, p.y);
        }
      l_run[h] += sum.x + sum.y;
    }
    // The weights' 2^14 taken back (a scale is 2^-100 at least).  Here, not where the scales are read: 4 tokens of
    // 32 heads, a window of 4096: 38.3 us without it, 38.6, and 39.2 there.
    {
      const float2 both = mul2(make_float2(vs[0], vs[1]), make_float2(kDown, kDown));
      vs[0] = both.x;
      vs[1] = both.y;
    }
    if (HALF) {
#pragma unroll
      for (int blk = 0; blk < NB; ++blk) pa[blk][1] = pa[blk][3] = 0u;
    }
#pragma unroll
    for (int blk = 0; blk < NB; ++blk) {
      __syncwarp();  // (keeps the next block's loads, and so their registers, behind this one's products)
      const uint32_t rec = base + blk * kRecord + 16 * D + 4 * g;
#pragma unroll
      for (int c = 0; c < SLABS; ++c) {
        uint32_t v[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) v[x] = lds32(rec + 512 * c + 32 * key_of(t, x));
        if (!whole) {
#pragma unroll
          for (int x = 0; x < 4; ++x)
            if ((gone >> (4 * blk + x)) & 1u) v[x] = 0u;
        }
        // four tokens of four columns -> four columns of four tokens
#pragma unroll
        for (int two = 0; two < 2; ++two) {  // columns 2 two, 2 two + 1
          uint32_t x[2], y[2];
          codes4_f16(prmt(v[0], v[1], two ? 0x7362 : 0x5140), x[0], x[1]);
          codes4_f16(prmt(v[2], v[3], two ? 0x7362 : 0x5140), y[0], y[1]);
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

  // The sum of row g + 8 h over the lanes that share it.
  __device__ __forceinline__ float row_sum(int h) const {
    float l = l_run[h];
    l += __shfl_xor_sync(0xffffffffu, l, 1);
    return l + __shfl_xor_sync(0xffffffffu, l, 2);
  }
  // Columns 32 c + 8 t + 4 x .. + 3 of row g + 8 h.
  __device__ __forceinline__ float4 piece(int h, int c, int x) const {
    return make_float4(o[c][0][2 * h + x], o[c][1][2 * h + x], o[c][2][2 * h + x], o[c][3][2 * h + x]);
  }
};

// What stands for s (its maximum and sum) in a join whose maximum is m: the factor of its O and its sum.
// (Products of the two keep a NaN, and make one of an infinite maximum, of whose row all weights are 0.)
__device__ __forceinline__ float join_factor(float s_max, float m) { return s_max != -INFINITY ? ex2(s_max - m) : 0.f; }
__device__ __forceinline__ void add_scaled(float (&v)[4], float f, const float4& x) {
  if (!(f > 0.f)) return;
  v[0] += f * x.x;
  v[1] += f * x.y;
  v[2] += f * x.z;
  v[3] += f * x.w;
}

// Four columns of query row i, divided by the row's sum and rounded; the first
// ones bring lse.
__device__ __forceinline__ void store4(const DecodeArgs& a, const Rows& w, int i, int D, int piece, float m, float l,
                                       const float (&v)[4]) {
  const float inv = l != 0.f ? rcp(l * kDown) : 0.f;  // (a NaN stays one)
  int token, head;
  w.place(a, i, &token, &head);
  const size_t at = (size_t)(w.q0 + w.t0 + token) * a.H + w.hk * a.G + head;
  // (fp16: held values may be larger, 65504 is as 65536; what reading back clips is clipped here)
  auto pack = [&](float x, float y) {
    if (a.bf16) return pack_bf16x2(x, y);
    return pack_f16x2(fabsf(x) > 65504.f ? copysignf(65504.f, x) : x, fabsf(y) > 65504.f ? copysignf(65504.f, y) : y);
  };
  const uint32_t lo = pack(v[0] * inv, v[1] * inv), hi = pack(v[2] * inv, v[3] * inv);
  *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at * D + 4 * piece) = make_uint2(lo, hi);
  if (a.lse && piece == 0) a.lse[at] = l != 0.f ? (m + lg2(l)) * kLn2 : -INFINITY;
}

// The copies of a ring: tiles 0 .. count - 1, tile i into stage i % S.  `find(i, x)` gives the
// records of tile i's blocks (0: none); a lane does that for one tile of every 32 and leaves them
// in shared memory, the first one with its low bit set where the others follow it (records
// start on 16 bytes), so that one copy brings them all.
template <int S, uint32_t RECORD, typename Find>
struct Feeder {
  Find find;
  uint32_t ring;
  uint64_t* full;
  volatile int* have;
  volatile unsigned long long* recs;  // [32][NB]
  int count, issued = 0;

  // Tile i into stage s (a converged warp).
  __device__ __forceinline__ void issue(int i, int s) {
    const int lane = threadIdx.x & 31;
    if ((i & 31) == 0) {
      unsigned long long x[NB];
#pragma unroll
      for (int k = 0; k < NB; ++k) x[k] = 0;
      if (i + lane < count) find(i + lane, x);
      bool follow = x[0] != 0;
#pragma unroll
      for (int k = 1; k < NB; ++k) follow = follow && x[k] == x[0] + k * RECORD;
      recs[lane * NB] = follow ? x[0] | 1 : x[0];
#pragma unroll
      for (int k = 1; k < NB; ++k) recs[lane * NB + k] = x[k];
      __syncwarp();
    }
    if (lane == 0) {
      const volatile unsigned long long* mine = recs + (i & 31) * NB;
      const uint32_t dst = ring + s * NB * RECORD;
      const unsigned long long x0 = mine[0];
      if (x0 & 1) {
        have[s] = (1 << NB) - 1;
        mbar_expect_tx(full + s, NB * RECORD);
        bulk_load(dst, x0 - 1, NB * RECORD, full + s);
      } else {
        int here = 0;
        for (int k = 0; k < NB; ++k) here |= (mine[k] != 0 ? 1 : 0) << k;
        have[s] = here;
        mbar_expect_tx(full + s, __popc(here) * RECORD);
#pragma unroll 1
        for (int k = 0; k < NB; ++k)
          if ((here >> k) & 1) bulk_load(dst + k * RECORD, mine[k], RECORD, full + s);
      }
    }
    __syncwarp();
    issued = i + 1;
  }
  __device__ __forceinline__ void drain(int done) const {
    for (int i = done; i < issued; ++i) mbar_wait(full + i % S, (i / S) & 1, kDrainBudget);
  }
};

// The stage of a ring's current tile, and how often the ring has gone round.
template <int S>
struct Stage {
  int at = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next() {
    if (++at == S) {
      at = 0;
      phase ^= 1;
    }
  }
};

template <typename SL>
__device__ __forceinline__ void init_bars(uint8_t* sm, int wr) {
  constexpr int n = SL::kRings * SL::kStages;
  if (threadIdx.x < 2 * n) {
    mbar_init(reinterpret_cast<uint64_t*>(sm + SL::bars) + threadIdx.x, threadIdx.x < n ? 1 : wr);
    mbar_fence_init();
  }
  if (threadIdx.x == 0) *reinterpret_cast<volatile int*>(sm + SL::misc) = 0;
  __syncthreads();
}

// A CTA, or a cluster of them, for each sequence, key head and tile of query rows.
template <int SLABS, int WR, bool HALF, int WARPS>
__global__ void __launch_bounds__(32 * WARPS) decode_kernel(const DecodeArgs a) {
  using SL = DecodeSmem<SLABS, WR, WARPS>;
  constexpr int kThreads = 32 * WARPS;
  static_assert(2 * SL::kRings * SL::kStages <= kThreads && kThreads <= 256, "a thread for each barrier, room for lengths");
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
  init_bars<SL>(sm, WR);

  const int split = blockIdx.x % a.splits;
  int rest = blockIdx.x / a.splits;
  const int rt = rest % a.row_tiles;
  rest /= a.row_tiles;
  int b = rest / a.c.Hk;
  // Sequences in the order of their lengths, the longest first, so that a launch's last CTAs
  // are short ones.
  if (a.longest_first) {
    int4* lens = reinterpret_cast<int4*>(sm + SL::ml_cta);
    int* which = reinterpret_cast<int*>(sm + SL::ml_warp);
    const int me = threadIdx.x, n = me < a.B ? a.c.lengths[me] : INT_MIN;
    reinterpret_cast<int*>(lens)[me] = n;
    __syncthreads();
    int rank = 0;  // sequences before this thread's
    for (int i = 0; i < a.B; i += 4) {
      const int4 x = lens[i / 4];
      rank += (x.x > n || (x.x == n && i < me)) + (x.y > n || (x.y == n && i + 1 < me)) +
              (x.z > n || (x.z == n && i + 2 < me)) + (x.w > n || (x.w == n && i + 3 < me));
    }
    if (me < a.B && rank == b) *which = me;
    __syncthreads();
    b = *which;
  }
  const Rows w = rows_of(a, b, rest % a.c.Hk, rt, 16 * WR, threadIdx.x == 0);
  // (what only the finding of records and the tiles at an end need stays out of the registers)
  Reach* s_reach = reinterpret_cast<Reach*>(sm + SL::reach);
  if (threadIdx.x == 0) {
    Reach reach = reach_of(a, w.held, w.p0, w.p1);
    if (w.nr <= 0) reach.tiles = 0;
    *s_reach = reach;
  }
  __syncthreads();
  const int tiles = s_reach->tiles, heads = s_reach->heads, skip = s_reach->skip;
  // this CTA's tiles, of which its rings take every R-th
  const int first = (int)((long long)tiles * split / a.splits);
  const int count = (int)((long long)tiles * (split + 1) / a.splits) - first;
  const int mine = (count - group + R - 1) / R;
  auto tile_first = [&](int i) {
    const int t = first + group + R * i;
    return (t < heads ? t : t + skip) * kKeys;
  };
  auto find = [&](int i, unsigned long long (&x)[NB]) { records_at(a, *s_reach, w.b, w.hk, tile_first(i), x); };
  const bool producer = part == 0;
  const uint32_t ring = smem_u32(sm + SL::ring) + group * S * SL::kStageBytes;
  Feeder<S, SL::kRecord, decltype(find)> feed = {
      find, ring, full, have, reinterpret_cast<volatile unsigned long long*>(sm + SL::recs) + group * 32 * NB, mine};
  if (producer)
    for (int i = 0; i < min(S, mine); ++i) feed.issue(i, i);

  Softmax<SLABS, HALF, SLABS >= 3 && (HALF || WR == 4)> st;
  st.begin(a, w, part);
  const bool rows_here = 16 * part < w.nr;
  bool ok = true;
  int done = 0;
  Stage<S> stage;
#pragma unroll 1
  for (int i = 0; i < mine; ++i, stage.next()) {
    const int s = stage.at;
    ok = __all_sync(0xffffffffu, ring_wait(full + s, stage.phase, a.budget, s_abort));
    if (!ok) break;
    done = i + 1;
    if (rows_here) st.tile(a, s_reach, ring + s * SL::kStageBytes, tile_first(i), have[s]);
    __syncwarp();
    if (WR > 1 && lane == 0) mbar_arrive(empty + s);
    if (producer && i + S < mine) {
      if (WR > 1 && !__all_sync(0xffffffffu, ring_wait(empty + s, stage.phase, a.budget, s_abort))) break;
      feed.issue(i + S, s);
    }
  }
  // a wait ran out: no copy may still be landing when the ring is used again
  if (producer) feed.drain(done);
  __syncthreads();

  // ---- the CTA's rows: its warps' parts together
  float* so = reinterpret_cast<float*>(sm + SL::o_warp);
  float2* sml = reinterpret_cast<float2*>(sm + SL::ml_warp);
#pragma unroll
  for (int h = 0; h < kHalves; ++h) {
    const float l = st.row_sum(h);
    const int r = warp * 16 + g + 8 * h;
    if (t == 0) sml[r] = make_float2(st.m_run[h], l);
#pragma unroll
    for (int c = 0; c < SLABS; ++c)
#pragma unroll
      for (int x = 0; x < 2; ++x)
        *reinterpret_cast<float4*>(so + r * SL::kPitch + 32 * c + 8 * t + 4 * x) = st.piece(h, c, x);
  }
  __syncthreads();
  constexpr int kPieces = D / 4;
  const bool alone = a.splits == 1;
  float4* s_ml = reinterpret_cast<float4*>(sm + SL::ml_cta);
  float* s_o = reinterpret_cast<float*>(sm + SL::o_cta);
  const bool failed = *s_abort != 0;
  for (int i = threadIdx.x; i < max(w.nr, 0) * kPieces; i += kThreads) {
    const int row = i / kPieces, piece = i - row * kPieces;
    const int at = (row >> 4) * 16 + (row & 15);
    float m = -INFINITY, l = 0.f, v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < R; ++k) m = fmaxf(m, sml[k * WR * 16 + at].x);
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const float2 s = sml[k * WR * 16 + at];
      const float f = join_factor(s.x, m);
      l += __fmul_rn(s.y, f);
      add_scaled(v, f, *reinterpret_cast<const float4*>(so + (k * WR * 16 + at) * SL::kPitch + 4 * piece));
    }
    if (alone) {
      if (!failed) store4(a, w, row, D, piece, m, l, v);
    } else {
      *reinterpret_cast<float4*>(s_o + row * D + 4 * piece) = make_float4(v[0], v[1], v[2], v[3]);
      if (piece == 0) s_ml[row] = make_float4(m, l, 0.f, 0.f);
    }
  }
  if (!alone) {
    cluster_sync();
    const uint32_t o_addr = smem_u32(s_o), ml_addr = smem_u32(s_ml);
    for (int i = split * kThreads + threadIdx.x; i < max(w.nr, 0) * kPieces; i += kThreads * a.splits) {
      const int row = i / kPieces, piece = i - row * kPieces;
      float m = -INFINITY, l = 0.f, v[4] = {0.f, 0.f, 0.f, 0.f};
      for (int k = 0; k < a.splits; ++k) m = fmaxf(m, ld_cluster(map_rank(ml_addr + 16 * row, k)).x);
      for (int k = 0; k < a.splits; ++k) {
        const float4 s = ld_cluster(map_rank(ml_addr + 16 * row, k));
        const float f = join_factor(s.x, m);
        l += __fmul_rn(s.y, f);
        if (f > 0.f) add_scaled(v, f, ld_cluster(map_rank(o_addr + 4 * (row * D + 4 * piece), k)));
      }
      if (!failed) store4(a, w, row, D, piece, m, l, v);
    }
    cluster_sync();  // no CTA leaves while another one reads its shared memory
  }
  if (threadIdx.x == 0) cross_report(s_abort, a.status);
}

// Cluster sizes, and how many clusters of each a device holds at a time (found once for a kernel and device;
// clusters stay within a part of the GPU, so that it is not the CTAs' number over their size).
constexpr int kSizes[] = {1, 2, 3, 4, 6, 8, 12, 16}, kSizeCount = 8;
struct Residency {
  std::atomic<bool> known{false};
  std::atomic<int> clusters[kSizeCount] = {};
};
constexpr int kDevices = 64;

// The current device's table of `all`, or, of a device beyond those, *own filled anew.
template <typename Kernel>
cudaError_t find_residency(Kernel kernel, int threads, int bytes, Residency (&all)[kDevices], Residency* own, Residency** found) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  Residency* r = *found = dev < kDevices ? all + dev : own;
  if (r->known.load(std::memory_order_acquire)) return e;
  e = cudaFuncSetAttribute((const void*)kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  for (int i = 0; i < kSizeCount && e == cudaSuccess; ++i) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kSizes[i]);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = bytes;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kSizes[i];
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    e = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg);
    r->clusters[i].store(n, std::memory_order_relaxed);
  }
  if (e == cudaSuccess) r->known.store(true, std::memory_order_release);
  return e;
}

// CTAs that share an item (a cluster): the number for which the rounds, each as long as a CTA's
// share of the tiles and what it costs to begin and to join, are shortest; their cost, in tiles of a
// warp. (8 key heads of 4 query heads, d = 128, one request: 16384 tokens 141 us with one CTA
// each, 24 with 8, 18 with 16; four requests of 8192: 75 with one, 25 with 4, 20 with 8, 31 with 16.)
long long splits_for(long long items, long long tiles, int rings, const Residency& r, int* splits, long long* rounds) {
  constexpr long long kBegin = 6;
  long long least = LLONG_MAX;
  for (int i = 0; i < kSizeCount; ++i) {
    const long long n = kSizes[i], held = r.clusters[i].load(std::memory_order_relaxed);
    if (held < 1) continue;
    const long long turns = (items + held - 1) / held;
    const long long cost = turns * ((tiles + n * rings - 1) / (n * rings) + kBegin);
    if (cost < least) {
      least = cost;
      *splits = (int)n;
      *rounds = turns;
    }
  }
  return least;
}

// Warps that share a ring, by the query rows.
int warps_a_ring(int rows) { return rows <= 16 ? 1 : rows <= 32 ? 2 : 4; }

template <int SLABS, int WR, bool HALF, int WARPS>
struct Launch {
  static constexpr int bytes = DecodeSmem<SLABS, WR, WARPS>::bytes, threads = 32 * WARPS;
  int splits = 1;
  long long rounds = 0, cost = LLONG_MAX;

  cudaError_t plan(long long items, long long tiles) {
    static std::atomic<uint64_t> done{0};
    static Residency all[kDevices];
    Residency own, *held = nullptr;
    auto kernel = decode_kernel<SLABS, WR, HALF, WARPS>;
    cudaError_t e = prepare_kernel((const void*)kernel, bytes, 0, &done);
    if (e == cudaSuccess) e = find_residency(kernel, threads, bytes, all, &own, &held);
    if (e == cudaSuccess) cost = splits_for(items, tiles, WARPS / WR, *held, &splits, &rounds);
    return e;
  }
  cudaError_t run(DecodeArgs a, long long items, cudaStream_t s) const {
    a.splits = splits;
    a.longest_first = a.B > 1 && a.B <= threads && items * splits > device_sms();
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(items * splits));
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = splits;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = splits > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, decode_kernel<SLABS, WR, HALF, WARPS>, a);
  }
};

template <int SLABS, int WR, bool HALF>
cudaError_t launch(const DecodeArgs& a, long long tiles, cudaStream_t s) {
  const long long items = (long long)a.B * a.c.Hk * a.row_tiles;
  Launch<SLABS, WR, HALF, 4> four;
  cudaError_t e = four.plan(items, tiles);
  if (e != cudaSuccess) return e;
  // Few items of long rows: eight warps a CTA, for a cluster's size is limited, and what a tile takes a
  // warp is latency (8 key heads of 4 heads, d = 128, one request: 4096 tokens 9.8 -> 8.4 us, 16384
  // 18.4 -> 15.4, 65536 48 -> 37). In more than one round four are as good or better, their CTAs' ends
  // and beginnings overlap (200 requests of 1000 tokens: 75 us, with eight 129); d = 64 gains nothing
  // (2 requests of 16384, 24 heads: 24.5, with eight 29.2).
  if constexpr (HALF && SLABS >= 3) {
    Launch<SLABS, WR, HALF, 8> eight;
    e = eight.plan(items, tiles);
    if (e != cudaSuccess) return e;
    if (eight.rounds == 1 && eight.cost <= four.cost) return eight.run(a, items, s);
  }
  return four.run(a, items, s);
}

template <int SLABS>
cudaError_t launch_rows(const DecodeArgs& a, int wr, long long tiles, cudaStream_t s) {
  if (a.Lq * a.G <= 8) return launch<SLABS, 1, true>(a, tiles, s);
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
  if (dtype == DF_FP32 || total_q > (1 << 30) || H / Hk > 128 || (long long)Lq * (H / Hk) > (1 << 30)) return DF_ERR_UNSUPPORTED;
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
  a.by_G = 65536u / a.G + 1;
  a.Lq = Lq;
  a.Tq = total_q;
  a.causal = causal != 0;
  a.window = window;
  a.sinks = sinks;
  a.bf16 = dtype == DF_BF16;
  a.kscale = (float)((double)scale * 1.4426950408889634);
  a.status = status;
  a.budget = wait_budget();
  const int wr = warps_a_ring(Lq * a.G);
  a.row_tiles = (Lq * a.G + 16 * wr - 1) / (16 * wr);
  if ((long long)B * Hk * a.row_tiles > 0x7fffffffll / 16) return DF_ERR_UNSUPPORTED;
  long long tiles = (std::min<long long>(max_length, (long long)max_pages * page) + kKeys - 1) / kKeys;
  if (window > 0) tiles = std::min<long long>(tiles, ((long long)window + Lq + sinks) / kKeys + 3);
  cudaStream_t s = (cudaStream_t)stream;
  cudaError_t e;
  switch (d / 32) {
    case 1: e = launch_rows<1>(a, wr, tiles, s); break;
    case 2: e = launch_rows<2>(a, wr, tiles, s); break;
    case 3: e = launch_rows<3>(a, wr, tiles, s); break;
    default: e = launch_rows<4>(a, wr, tiles, s); break;
  }
  return e == cudaSuccess ? DF_OK : DF_ERR_CUDA;
}
