// Shared pieces of the 8-bit cache's kernels: the record of a block and the way to it.
//
// A block is 16 tokens of one key head.  Its record holds the keys' and the values' e4m3
// codes and a scale of each; a page is page / 16 records of every head,
// [n_pages][Hk][page / 16][32 d + 16 bytes]:
//   0       keys' codes, [d / 32][16 tokens][32 columns]
//   16 d    values' codes, likewise
//   32 d    keys' scale, values' scale (fp32), 8 bytes unused
// so that a run of tokens of one head is one contiguous copy with all that belongs to it, and
// the reads of an attention's lanes (a token's 32 columns behind the next one's) meet no bank
// conflict.
#pragma once

#include "df_cross.cuh"

namespace dfa {

constexpr int kBlock = 16;  // tokens

__host__ __device__ constexpr int record_bytes(int d) { return 32 * d + 16; }

struct CacheView {
  uint8_t* base;
  const int32_t* pages;    // [B][max_pages]
  const int32_t* lengths;  // [B]
  int Hk, d, page, n_pages, max_pages;
};

// The page of block `blk` of sequence b, or -1 where the table holds none.
__device__ __forceinline__ int page_of(const CacheView& c, int b, int blk) {
  const int at = (int)((unsigned)blk * kBlock / (unsigned)c.page);
  if (at >= c.max_pages) return -1;
  const int id = c.pages[(size_t)b * c.max_pages + at];
  return (unsigned)id < (unsigned)c.n_pages ? id : -1;
}
__device__ __forceinline__ uint8_t* record_of(const CacheView& c, int page_id, int head, int blk) {
  const unsigned per = c.page / kBlock;
  return c.base + (((size_t)page_id * c.Hk + head) * per + (unsigned)blk % per) * record_bytes(c.d);
}

// Two e4m3 codes as fp16 (exact).
__device__ __forceinline__ uint32_t codes_f16(uint16_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(two));
  return h;
}
// Two values as e4m3 codes, `lo` in the lower byte (nearest even; at most 448 in magnitude).
__device__ __forceinline__ uint16_t f32_codes(float lo, float hi) {
  uint16_t c;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(hi), "f"(lo));
  return c;
}

// Host side (df_cache.cu): checks that the entry points share; fills *c.
df_status cache_check(const void* cache, const int32_t* pages, const int32_t* lengths, int B, int Hk, int d, int page,
                      int n_pages, int max_pages, CacheView* c);
inline size_t cache_bytes(int Hk, int d, int page, int n_pages) {
  return (size_t)n_pages * Hk * (page / kBlock) * record_bytes(d);
}

}  // namespace dfa
