// Shared pieces of the cross-attention kernels (queries of one length against
// keys and values of another): the call's arguments, the list of query tiles,
// the tensor maps and the bounded waits.
//
// A query tile holds 128 rows: `tpt` = floor(128 / G) consecutive tokens times
// the G query heads that share one key head, head fastest, so that row r is
// token r / G and head r % G.  Shared key heads are then read once for all of
// their query heads and a single-token call still fills G rows of its tile.
// Head sizes that are not 64 or 128 run as the next of the two: the tensor
// maps end a row at d, and a copy fills the columns behind it with zeros.
#pragma once

#include <limits.h>

#include <atomic>

#include "df_tc_common.cuh"

namespace dfa {

struct CrossArgs {
  const uint8_t* key_mask;   // [B, Lk] or NULL
  const int32_t* cu_q;       // [B + 1] or NULL: queries are [B, Lq]
  const int32_t* cu_k;       // [B + 1] or NULL: keys are [B, Lk]
  int B, H, Hk, G, Lq, Lk, Tq, Tk, d;
  int tpt;                   // tokens per query tile
  float kscale;              // scale * log2(e)
  float scale;
  int32_t* status;
  unsigned long long budget;
};

// A tile of one side's rows (queries, or keys in the backward's key kernel)
// against all rows of its sequence on the other side.
struct CrossItem {
  int r0;   // first token of the tile
  int nr;   // its tokens that belong to the sequence, at least 1
  int o0;   // first token of the sequence's other side
  int no;   // tokens there
  int hk;   // key head; -1 ends the list
  int b;    // batch row (for key_mask)
};

// The sequences' rows on one side of a call.
struct CrossSide {
  const int32_t* cu;  // or NULL: B sequences of len tokens each
  int len, total;
};

__device__ __forceinline__ CrossSide query_side(const CrossArgs& a) { return {a.cu_q, a.Lq, a.Tq}; }
__device__ __forceinline__ CrossSide key_side(const CrossArgs& a) { return {a.cu_k, a.Lk, a.Tk}; }

__device__ __forceinline__ void cross_fail(int32_t* status, int code) {
  if (status) atomicCAS(status, 0, code);
}

// Rows [*start, *start + n) of sequence b; a sequence whose offsets are not
// 0 <= cu[b] <= cu[b + 1] <= total is taken as empty and reported.
__device__ __forceinline__ int seq_rows(const CrossSide& side, int b, int32_t* status, int* start) {
  if (!side.cu) {
    *start = b * side.len;
    return side.len;
  }
  const int s = side.cu[b], e = side.cu[b + 1];
  if (s < 0 || e < s || e > side.total) {
    cross_fail(status, (int)DF_ERR_INVALID_ARG);
    *start = 0;
    return 0;
  }
  *start = s;
  return e - s;
}

// Bounded wait that gives up as soon as another role of the CTA has; the control
// flow after it stays the same either way.  (What ran out is reported once, by
// cross_report at the kernel's end: this code stands in the kernels some thirty times.)
__device__ __forceinline__ bool cross_wait(uint64_t* bar, uint32_t parity, unsigned long long budget,
                                           volatile int* abort) {
  if (ptx::mbar_try_wait(bar, parity)) return true;
  const long long t0 = clock64();
  do {
    if (ptx::mbar_try_wait(bar, parity)) return true;
    if ((unsigned long long)(clock64() - t0) > budget) *abort = 1;
  } while (*abort == 0);
  return false;
}
// One thread, behind the CTA's last wait.
__device__ __forceinline__ void cross_report(volatile int* abort, int32_t* status) {
  if (*abort != 0) cross_fail(status, (int)DF_ERR_DEVICE_TIMEOUT);
}

// 3-D tiled load: column, head, token.
__device__ __forceinline__ void tma_load_3d(void* dst, const void* tmap, int c0, int c1, int c2, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(ptx::smem_u32(dst)),
      "l"((uint64_t)tmap), "r"(c0), "r"(c1), "r"(c2), "r"(ptx::smem_u32(bar))
      : "memory");
}

// Which of the 32 W keys of a tile count, one bit each (warp-collective): the
// first `left` ones, and of those the ones that the mask (at the tile's first key,
// or NULL) holds valid.  True if all do.
template <int W>
__device__ __forceinline__ bool key_bits(const uint8_t* mask, int left, uint32_t (&bits)[W]) {
  const int lane = threadIdx.x & 31;
  uint32_t all = 0xffffffffu;
#pragma unroll
  for (int w = 0; w < W; ++w) {
    const int j = 32 * w + lane;
    bits[w] = __ballot_sync(0xffffffffu, j < left && (!mask || mask[j] != 0));
    all &= bits[w];
  }
  return all == 0xffffffffu;
}

// Zeroes the rows of a tile of 32 W rows whose bit is 0 (one warp): a row is 128
// bytes of each 64-column box, however swizzled.
template <int W, int CHUNKS>
__device__ __forceinline__ void zero_rows(uint8_t* tile, const uint32_t (&bits)[W]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int w = 0; w < W; ++w) {
    if ((bits[w] >> lane) & 1u) continue;
#pragma unroll 1
    for (int ch = 0; ch < CHUNKS; ++ch)
#pragma unroll
      for (int e = 0; e < 8; ++e)
        *reinterpret_cast<uint4*>(tile + (ch * 32 * W + 32 * w + lane) * 128 + 16 * e) = make_uint4(0u, 0u, 0u, 0u);
  }
  ptx::fence_proxy_async_smem();
}

template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float x, float y) {
  return BF16 ? ptx::pack_bf16x2(x, y) : ptx::pack_f16x2(x, y);
}

// A warp's 32 rows of results, 32 columns each (16 words, packed), one row per
// thread, to memory: row by row a store would touch 32 lines 16 bytes at a time,
// so the rows change hands through 1 KB of shared memory of the warp's own (16
// rows at a time) and go out as 64 bytes each.  `rel` is the thread's row (-1: not
// stored) behind `dst`, the first column of row 0; `left` columns exist from there
// on.
constexpr int kRowStage = 1024;
template <typename T>
__device__ __forceinline__ void store_rows32(uint8_t* stage, const uint32_t (&w)[16], int rel, T* dst, int d, int left) {
  const int lane = threadIdx.x & 31, c = lane & 3;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    if ((lane >> 4) == half) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        *reinterpret_cast<uint4*>(stage + (lane & 15) * 64 + 16 * (e ^ ((lane >> 1) & 3))) =
            make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = 8 * i + (lane >> 2);
      const uint4 v = *reinterpret_cast<const uint4*>(stage + r * 64 + 16 * (c ^ ((r >> 1) & 3)));
      const int to = __shfl_sync(0xffffffffu, rel, 16 * half + r);
      if (to >= 0 && 8 * c < left) *reinterpret_cast<uint4*>(dst + (size_t)to * d + 8 * c) = v;
    }
    __syncwarp();
  }
}

// Keys of a masked row up to its last valid one (warp-collective).
__device__ __forceinline__ int masked_length(const uint8_t* mask, int n) {
  const int lane = threadIdx.x & 31;
  for (int end = n; end > 0; end -= 512) {
    int last = -1;  // 16 loads in flight per lane
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int j = end - 1 - lane - 32 * i;
      if (j >= 0 && mask[j] != 0) last = max(last, j);
    }
    last = __reduce_max_sync(0xffffffffu, last);
    if (last >= 0) return last + 1;
  }
  return 0;
}

// Finds the tiles of one side by number, warp-collectively.  Tiles of `step`
// tokens are numbered by sequence, then key head, then position; in packed mode
// the rows behind the last sequence count as one more sequence, whose other
// side is empty.  The walk over packed sequences goes on from the last call's number,
// in either direction.
struct TileWalk {
  int b0 = 0;          // sequences b0 .. b0 + 31 are the lanes' current ones
  long long done = 0;  // tiles of the sequences before b0

  __device__ __forceinline__ CrossItem find(const CrossArgs& a, const CrossSide& rows, const CrossSide& other,
                                            int step, long long number) {
    const int lane = threadIdx.x & 31;
    CrossItem it;
    it.hk = -1;
    it.r0 = it.nr = it.o0 = it.no = it.b = 0;
    if (number < 0) return it;
    int first, len, tiles, at;  // the sequence's rows and tiles, the tile's number in it
    if (!rows.cu) {
      tiles = (rows.len + step - 1) / step;
      const long long per = (long long)tiles * a.Hk;
      if (number >= per * a.B) return it;
      it.b = (int)(number / per);
      at = (int)(number - it.b * per);
      first = it.b * rows.len;
      len = rows.len;
    } else {
      for (;;) {
        bool back = number < done;
        if (back && b0 == 0) {  // (only with offsets that change meanwhile)
          back = false;
          done = 0;
        }
        if (back) b0 -= 32;
        if (b0 > a.B) return it;
        const int b = b0 + lane;
        int start = 0, n = 0;
        if (b < a.B) {
          n = seq_rows(rows, b, a.status, &start);
        } else if (b == a.B) {
          start = min(max(rows.cu[a.B], 0), rows.total);
          n = rows.total - start;
        }
        const int nt = (n + step - 1) / step;
        const long long own = (long long)nt * a.Hk;
        long long incl = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const long long u = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += u;
        }
        const long long total = __shfl_sync(0xffffffffu, incl, 31);
        if (back) done -= total;
        if (number < done) continue;
        if (number >= done + total) {
          done += total;
          b0 += 32;
          continue;
        }
        const int src = __ffs(__ballot_sync(0xffffffffu, number < done + incl)) - 1;
        at = (int)(number - done - __shfl_sync(0xffffffffu, incl - own, src));
        tiles = __shfl_sync(0xffffffffu, nt, src);
        first = __shfl_sync(0xffffffffu, start, src);
        len = __shfl_sync(0xffffffffu, n, src);
        it.b = b0 + src;
        break;
      }
    }
    it.hk = at / tiles;
    const int tok = (at - it.hk * tiles) * step;
    it.r0 = first + tok;
    it.nr = min(step, len - tok);
    if (it.b < a.B) it.no = seq_rows(other, it.b, a.status, &it.o0);
    return it;
  }
};

// Work for the next turn of a CTA.  The grid has a CTA for every tile; one that
// runs takes over the number of one that has not been launched yet (cluster launch
// control), so that tiles of unequal cost spread evenly without a counter in
// memory, which concurrent calls and replayed graphs would have to share.
struct TileClaim {
  uint64_t* bar;    // one arrival
  uint4* response;  // 16 bytes of shared memory
  uint32_t asked = 0;

  // (both for a converged warp) Nothing may be asked again once an answer was -1.
  __device__ __forceinline__ void ask() {
    if (ptx::elect_one()) {
      ptx::mbar_expect_tx(bar, 16);
      asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                       ptx::smem_u32(response)),
                   "r"(ptx::smem_u32(bar))
                   : "memory");
    }
    __syncwarp();
    ++asked;
  }
  // The tile number taken over, or -1 when none is left.
  __device__ __forceinline__ long long answer(unsigned long long budget, volatile int* abort) {
    const bool ok = cross_wait(bar, (asked - 1) & 1, budget, abort);
    // (the response must not be written into a CTA that has left)
    if (!ok) ptx::mbar_wait(bar, (asked - 1) & 1, kDrainBudget);
    uint32_t taken, x;
    asm volatile(
        "{\n\t.reg .b128 r;\n\t.reg .pred p;\n\t"
        "ld.shared.b128 r, [%2];\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t"
        "mov.u32 %1, 0;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, r;\n\t}\n"
        : "=r"(taken), "=r"(x)
        : "r"(ptx::smem_u32(response))
        : "memory");
    ptx::fence_proxy_async_smem();  // this read before the next response's write
    const bool mine = __all_sync(0xffffffffu, ok) && taken;
    return mine ? (long long)x : -1;
  }
};

// Host side (df_cross.cu): [rows][heads][d] 16-bit rows in boxes of 64 columns,
// box_heads heads and box_rows rows, 128-byte swizzle.
bool encode_heads(CUtensorMap* m, const void* base, long long rows, int heads, int d, bool bf16, int box_heads,
                  int box_rows);
int device_sms();
// Allows `kernel` its dynamic shared memory on the current device (once per
// device) and checks that it is launched with at least `regs` registers a thread,
// those that its setmaxnreg split counts on (the .inc would wait for the rest).
cudaError_t prepare_kernel(const void* kernel, int bytes, int regs, std::atomic<uint64_t>* done);
// Argument checks and arguments shared by the forward and the backward.
df_status cross_check(const void* q, const void* k, const void* v, const uint8_t* key_mask, const int32_t* cu_q,
                      const int32_t* cu_k, int B, int H, int Hk, int Lq, int Lk, int total_q, int total_k, int d,
                      float scale, df_dtype dtype, int32_t* status, CrossArgs* a);
// An upper bound of the number of query tiles.
long long cross_query_tiles(const CrossArgs& a);
unsigned long long wait_budget();

}  // namespace dfa
