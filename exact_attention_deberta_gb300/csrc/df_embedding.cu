// Embedding lookup with scaling, out[t] = scale * table[ids[t]], and the
// gradient of the table, grad[v] (+)= scale * sum_{t: ids[t] = v} dout[t].
//
// Lookup: a warp per token, or per four tokens where there are many, 16-byte vectors;
// HBM bound (each row that the ids reach is read once, the repeats come from L2, each
// output row is written once): 131072 x 768, bf16: 41 to 44 us.
//
// Gradient.  Adding rows with atomics would make the last bits depend on the
// order of arrival, so the tokens are sorted by id first (a stable radix sort
// of (id, position) pairs) and every row of the table is then the sum of one
// run of the sorted list, in ascending position:
//   1. sort.  Few tokens (to 8192; to 2048 where nothing has to be zeroed): one block, 8
//      bits per pass, pairs in shared memory.  More: tiles of 512 or 2048 keys, at most 10 bits per pass (two passes for
//      ids below 2^20); a pass counts the digits of each tile, scans each
//      digit's counts over the tiles, and scatters (rank inside the tile by warp
//      digit matching, so that equal digits keep their order).  Ids that pass no
//      gradient (the padding id, ids outside the table) sort behind every other
//      one and are left out.  The sort is latency bound and leaves HBM idle, so
//      the same launches also zero the table in further blocks (rows that tokens
//      reach are written again in step 2).
//   2. sums: a warp takes 32 consecutive entries of the sorted list (8 where there
//      are few) and 256 columns (8 per lane), adds rows in fp32 while the id stays
//      the same and writes each finished run.  A run that crosses into the next
//      warp's entries leaves one partial row per warp in the workspace.
//   3. join: the warp of the chunk in which such a run begins adds its partial
//      rows in order; long runs are shared by the eight warps of the block.
// Each launch may be scheduled while the one before it drains (programmatic
// dependent launch); it waits before its first access to global memory.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "df_common.cuh"

namespace dfa {
namespace {

constexpr int kSortThreads = 256;
constexpr int kMaxDigitBits = 10;
constexpr int kSlice = 256;                             // columns per warp of the sums

__device__ __forceinline__ void load8(const float* p, float (&f)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
  f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}

// Eight values as loaded, converted where they are added.
template <typename T>
struct Raw8 {
  uint4 v[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int e = 0; e < (int)sizeof(T) / 2; ++e) v[e] = reinterpret_cast<const uint4*>(p)[e];
  }
  __device__ __forceinline__ void add_to(float (&acc)[8]) const {
    const T* h = reinterpret_cast<const T*>(v);
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] += IO<T>::to_f(h[e]);
  }
};

template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&f)[8]) {
  if constexpr (sizeof(T) == 2) {
    uint4 v;
    T* h = reinterpret_cast<T*>(&v);
#pragma unroll
    for (int e = 0; e < 8; ++e) h[e] = IO<T>::from_f(f[e]);
    *reinterpret_cast<uint4*>(p) = v;
  } else {
    *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(f[4], f[5], f[6], f[7]);
  }
}

template <typename T>
__device__ __forceinline__ void store8_past_l2(T* p, const float (&f)[8]) {
  uint4 v[sizeof(T) / 2];
  store8<T>(reinterpret_cast<T*>(v), f);
#pragma unroll
  for (int e = 0; e < (int)sizeof(T) / 2; ++e) __stcs(reinterpret_cast<uint4*>(p) + e, v[e]);
}

// The id is kept from here on and not read again, whatever the compiler would make of it: the
// value that is checked against the table is the one that is used, also where another
// stream writes the ids meanwhile.
__device__ __forceinline__ long long load_id(const void* ids, int ids64, size_t t) {
  long long id = ids64 ? (long long)static_cast<const int64_t*>(ids)[t] : (long long)static_cast<const int32_t*>(ids)[t];
  asm("" : "+l"(id));
  return id;
}

// A warp takes R consecutive tokens, R rows of loads in flight per 256 columns.
// The output is written past L2 (evict first), which is left to the table's rows.
template <typename T, int R>
__global__ void __launch_bounds__(256) lookup_kernel(const void* __restrict__ ids, int ids64, int tokens,
                                                     const T* __restrict__ table, int V, int N, float scale,
                                                     T* __restrict__ out, int32_t* status) {
  const int lane = threadIdx.x & 31;
  const int t0 = (blockIdx.x * 8 + (threadIdx.x >> 5)) * R;
  if (t0 >= tokens) return;
  const T* src[R];
  bool in[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const long long id = t0 + r < tokens ? load_id(ids, ids64, t0 + r) : 0;
    in[r] = id >= 0 && id < V;
    if (!in[r] && lane == 0 && status) atomicCAS(status, 0, (int32_t)DF_ERR_INVALID_ARG);
    src[r] = table + (size_t)(in[r] ? id : 0) * N;
  }
  T* dst = out + (size_t)t0 * N;
  for (int c = lane * 8; c < N; c += 256) {
    Raw8<T> raw[R];
#pragma unroll
    for (int r = 0; r < R; ++r) raw[r].load(src[r] + c);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      raw[r].add_to(f);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = in[r] ? f[e] * scale : 0.f;
      if (t0 + r < tokens) store8_past_l2<T>(dst + (size_t)r * N + c, f);
    }
  }
}

// ---------------------------------------------------------------- sort by id
// A key is the id, or V for a token that passes no gradient.
struct SortArgs {
  const void* ids;      // first pass: the caller's ids
  int ids64;
  uint32_t* key;        // sorted by the passes before; the first pass fills it from the ids
  const uint32_t* pos;  // (so that ids which change meanwhile cannot lead it astray)
  uint32_t* key_out;
  uint32_t* pos_out;
  uint32_t* hist;       // [tiles][digits]
  uint32_t* total;      // [digits]
  int n, tiles, V, pad, first, shift, bits;
  int32_t* status;
  // blocks from `blocks` on zero 16-byte pieces [fill_begin, fill_end) of the table
  int blocks;
  uint4* fill;
  size_t fill_begin, fill_end;
};

// Lets the next launch be scheduled and waits for the previous one.
__device__ __forceinline__ void start_after_previous() {
  allow_dependent_launch();
  grid_dependency_wait();
}

// A block without sorting work: its share of the zeros.
__device__ __forceinline__ void fill_share(const SortArgs& a) {
  const size_t step = (size_t)(gridDim.x - a.blocks) * blockDim.x;
  for (size_t i = a.fill_begin + (size_t)(blockIdx.x - a.blocks) * blockDim.x + threadIdx.x; i < a.fill_end; i += step)
    a.fill[i] = make_uint4(0u, 0u, 0u, 0u);
}

__device__ __forceinline__ uint32_t sort_key(const SortArgs& a, int i) {
  if (!a.first) return a.key[i];
  const long long id = load_id(a.ids, a.ids64, i);
  const bool in = id >= 0 && id < a.V;
  if (!in && a.status) atomicCAS(a.status, 0, (int32_t)DF_ERR_INVALID_ARG);
  return in && id != a.pad ? (uint32_t)id : (uint32_t)a.V;
}

// Exclusive prefix of one value per thread over a block of at most 1024 threads.
__device__ __forceinline__ uint32_t block_exclusive(uint32_t own, uint32_t* warp_sum) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t incl = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t u = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += u;
  }
  if (lane == 31) warp_sum[warp] = incl;
  __syncthreads();
  uint32_t before = 0;
  for (int w = 0; w < warp; ++w) before += warp_sum[w];
  __syncthreads();
  return before + incl - own;
}

// Rank of each lane's digit among equal ones of the warp's keys so far (rounds of
// 32 keys in lane order); `cnt` holds the warp's counts.
__device__ __forceinline__ uint32_t digit_rank(uint32_t d, bool valid, uint32_t* cnt, int lane) {
  const uint32_t same = __match_any_sync(0xffffffffu, valid ? d : 0xffffffffu);
  const uint32_t before = __popc(same & ((1u << lane) - 1u));
  uint32_t start = 0;
  if (valid && before == 0) {
    start = cnt[d];
    cnt[d] = start + __popc(same);
  }
  start = __shfl_sync(0xffffffffu, start, __ffs(same) - 1);
  __syncwarp();
  return start + before;
}

// (ITEMS keys per thread, in both kernels)
template <int ITEMS>
__global__ void __launch_bounds__(kSortThreads) digit_counts(const SortArgs a) {
  start_after_previous();
  if ((int)blockIdx.x >= a.blocks) return fill_share(a);
  __shared__ uint32_t cnt[1 << kMaxDigitBits];
  const int digits = 1 << a.bits;
  uint32_t key[ITEMS];
  const int base = blockIdx.x * (kSortThreads * ITEMS);
#pragma unroll
  for (int k = 0; k < ITEMS; ++k) {
    const int i = base + k * kSortThreads + threadIdx.x;
    key[k] = i < a.n ? sort_key(a, i) : 0u;
    if (a.first && i < a.n) a.key[i] = key[k];
  }
  for (int d = threadIdx.x; d < digits; d += kSortThreads) cnt[d] = 0;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < ITEMS; ++k)
    if (base + k * kSortThreads + (int)threadIdx.x < a.n) atomicAdd(&cnt[(key[k] >> a.shift) & (digits - 1)], 1u);
  __syncthreads();
  for (int d = threadIdx.x; d < digits; d += kSortThreads) a.hist[(size_t)blockIdx.x * digits + d] = cnt[d];
}

// Each digit's counts become exclusive prefixes over the tiles: block d / 32 takes
// 32 digits (lane = digit, so rows of hist are read whole), its eight warps eight
// ranges of tiles.
__global__ void __launch_bounds__(256) scan_over_tiles(const SortArgs a) {
  start_after_previous();
  if ((int)blockIdx.x >= a.blocks) return fill_share(a);
  __shared__ uint32_t sums[8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int digits = 1 << a.bits, d = blockIdx.x * 32 + lane;
  const int per = (a.tiles + 7) / 8, t0 = min(a.tiles, warp * per), t1 = min(a.tiles, t0 + per);
  const bool in = d < digits;
  uint32_t s = 0;
#pragma unroll 8
  for (int t = t0; t < t1; ++t) s += in ? a.hist[(size_t)t * digits + d] : 0u;
  sums[warp][lane] = s;
  __syncthreads();
  uint32_t run = 0, all = 0;
#pragma unroll
  for (int w = 0; w < 8; ++w) {
    if (w < warp) run += sums[w][lane];
    all += sums[w][lane];
  }
  if (!in) return;
  if (warp == 0) a.total[d] = all;
#pragma unroll 8
  for (int t = t0; t < t1; ++t) {
    const uint32_t c = a.hist[(size_t)t * digits + d];
    a.hist[(size_t)t * digits + d] = run;
    run += c;
  }
}

// Writes a tile's pairs to their places.  Each warp of the tile owns
// 32 ITEMS consecutive keys in rounds of 32, so that (warp, round, lane) is the
// original order.
template <int ITEMS>
__global__ void __launch_bounds__(kSortThreads) scatter_by_digit(const SortArgs a) {
  start_after_previous();
  if ((int)blockIdx.x >= a.blocks) return fill_share(a);
  constexpr int kWarps = kSortThreads / 32, kPer = (1 << kMaxDigitBits) / kSortThreads;
  __shared__ uint32_t cnt[kWarps][1 << kMaxDigitBits];
  __shared__ uint32_t warp_sum[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int digits = 1 << a.bits;
  const int base = blockIdx.x * (kSortThreads * ITEMS) + warp * (ITEMS * 32);
  uint32_t key[ITEMS], pos[ITEMS], rank[ITEMS];
#pragma unroll
  for (int k = 0; k < ITEMS; ++k) {
    const int i = base + k * 32 + lane;
    key[k] = i < a.n ? a.key[i] : 0u;
    pos[k] = a.first ? (uint32_t)i : (i < a.n ? a.pos[i] : 0u);
  }
  // thread t's digits: t kPer .. t kPer + kPer - 1
  uint32_t tot[kPer], own = 0;
#pragma unroll
  for (int e = 0; e < kPer; ++e) {
    const int d = threadIdx.x * kPer + e;
    tot[e] = d < digits ? a.total[d] : 0u;
    own += tot[e];
  }
  for (int d = threadIdx.x; d < digits; d += kSortThreads)
#pragma unroll
    for (int w = 0; w < kWarps; ++w) cnt[w][d] = 0;
  uint32_t at_digit = block_exclusive(own, warp_sum);  // (also: the counts are cleared)
#pragma unroll
  for (int k = 0; k < ITEMS; ++k)
    rank[k] = digit_rank((key[k] >> a.shift) & (digits - 1), base + k * 32 + lane < a.n, cnt[warp], lane);
  __syncthreads();
#pragma unroll
  for (int e = 0; e < kPer; ++e) {
    const int d = threadIdx.x * kPer + e;
    if (d < digits) {
      uint32_t at = at_digit + a.hist[(size_t)blockIdx.x * digits + d];
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const uint32_t c = cnt[w][d];
        cnt[w][d] = at;
        at += c;
      }
    }
    at_digit += tot[e];
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < ITEMS; ++k) {
    if (base + k * 32 + lane >= a.n) continue;
    const uint32_t to = cnt[warp][(key[k] >> a.shift) & (digits - 1)] + rank[k];
    if (to >= (uint32_t)a.n) continue;  // only with a workspace that another call writes
    a.key_out[to] = key[k];
    a.pos_out[to] = pos[k];
  }
}

// The whole sort of at most kSmallSort tokens in block 0.
constexpr int kSmallSort = 8192, kSmallBits = 8, kSmallThreads = 1024;
constexpr size_t kSmallSmem = (size_t)kSmallSort * 8 + 32 * (1 << kSmallBits) * 4 + 128;

__global__ void __launch_bounds__(kSmallThreads) sort_small(const SortArgs a, int passes) {
  start_after_previous();
  if ((int)blockIdx.x >= a.blocks) return fill_share(a);
  extern __shared__ uint32_t sh[];
  uint32_t* s_key = sh;
  uint32_t* s_pos = sh + kSmallSort;
  uint32_t* cnt = s_pos + kSmallSort;  // [32 warps][256]
  uint32_t* warp_sum = cnt + 32 * (1 << kSmallBits);
  constexpr int kDigits = 1 << kSmallBits;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // rounds that hold keys: as few as the tokens need, the same for every warp
  const int rounds = (a.n + kSmallThreads - 1) / kSmallThreads;
  const int base = warp * rounds * 32;
  uint32_t key[8], pos[8], rank[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int i = base + k * 32 + lane;
    const bool in = k < rounds && i < a.n;
    key[k] = in ? sort_key(a, i) : 0u;
    pos[k] = (uint32_t)i;
  }
  for (int p = 0; p < passes; ++p) {
    const int shift = p * kSmallBits;
    for (int d = threadIdx.x; d < 32 * kDigits; d += kSmallThreads) cnt[d] = 0;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < rounds)
        rank[k] = digit_rank((key[k] >> shift) & (kDigits - 1), base + k * 32 + lane < a.n, cnt + warp * kDigits, lane);
    __syncthreads();
    uint32_t all = 0;
    if (threadIdx.x < kDigits)
      for (int w = 0; w < 32; ++w) {
        const uint32_t c = cnt[w * kDigits + threadIdx.x];
        cnt[w * kDigits + threadIdx.x] = all;
        all += c;
      }
    const uint32_t start = block_exclusive(all, warp_sum);
    if (threadIdx.x < kDigits)
      for (int w = 0; w < 32; ++w) cnt[w * kDigits + threadIdx.x] += start;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < rounds && base + k * 32 + lane < a.n) {
        const uint32_t to = cnt[warp * kDigits + ((key[k] >> shift) & (kDigits - 1))] + rank[k];
        s_key[to] = key[k];
        s_pos[to] = pos[k];
      }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int i = base + k * 32 + lane;
      if (k < rounds && i < a.n) {
        key[k] = s_key[i];
        pos[k] = s_pos[i];
      }
    }
    __syncthreads();
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int i = base + k * 32 + lane;
    if (k < rounds && i < a.n) {
      a.key_out[i] = key[k];
      a.pos_out[i] = pos[k];
    }
  }
}

// ------------------------------------------------------------ sums over runs
struct SumArgs {
  const uint32_t* key;  // sorted; entries >= V pass no gradient
  const uint32_t* pos;
  int n, V, N, chunks, accumulate;
  float scale;
  float* part;          // [chunks][2][N]: the run that began before the chunk, the one that goes on behind it
  float* grad;          // [V][N]
};

__device__ __forceinline__ void write_row(const SumArgs& a, uint32_t v, int c, const float (&acc)[8]) {
  if (v >= (uint32_t)a.V) return;
  float* p = a.grad + (size_t)v * a.N + c;
  float f[8];
  if (a.accumulate) load8(p, f);
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] = a.accumulate ? f[e] + acc[e] * a.scale : acc[e] * a.scale;
  store8<float>(p, f);
}

template <typename T, int CHUNK>
__global__ void __launch_bounds__(256, sizeof(T) == 2 ? 4 : 2) sum_runs(const SumArgs a, const T* dout) {
  start_after_previous();
  const int lane = threadIdx.x & 31;
  const int chunk = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (chunk >= a.chunks) return;
  const int c = blockIdx.y * kSlice + lane * 8;
  const bool col = c < a.N;
  const int i0 = chunk * CHUNK, cnt = min(CHUNK, a.n - i0);
  const uint32_t my_key = lane < cnt ? a.key[i0 + lane] : 0xffffffffu;
  const uint32_t my_pos = lane < cnt ? min(a.pos[i0 + lane], (uint32_t)a.n - 1u) : 0u;
  const uint32_t before = chunk > 0 ? a.key[i0 - 1] : 0xffffffffu;
  const uint32_t after = i0 + CHUNK < a.n ? a.key[i0 + CHUNK] : 0xffffffffu;
  // entries that pass a gradient stand at the front
  const int live = __popc(__ballot_sync(0xffffffffu, my_key < (uint32_t)a.V));
  if (live == 0) return;
  float acc[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) acc[e] = 0.f;
  uint32_t cur = __shfl_sync(0xffffffffu, my_key, 0);
  bool head = before == cur;  // the current run began in an earlier chunk
  for (int k0 = 0; k0 < live; k0 += 8) {
    Raw8<T> f[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const uint32_t p = __shfl_sync(0xffffffffu, my_pos, k0 + u);
      if (col && k0 + u < live) f[u].load(dout + (size_t)p * a.N + c);
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const uint32_t key = __shfl_sync(0xffffffffu, my_key, k0 + u);
      if (k0 + u >= live) break;
      if (key != cur) {
        if (col) {
          if (head) store8<float>(a.part + (size_t)chunk * 2 * a.N + c, acc);
          else write_row(a, cur, c, acc);
        }
        cur = key;
        head = false;
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = 0.f;
      }
      if (col) f[u].add_to(acc);
    }
  }
  if (col) {
    const bool on = live == CHUNK && after == cur;
    if (head) store8<float>(a.part + (size_t)chunk * 2 * a.N + c, acc);
    else if (on) store8<float>(a.part + ((size_t)chunk * 2 + 1) * a.N + c, acc);
    else write_row(a, cur, c, acc);
  }
}

// Runs longer than this many chunks are added by the block's eight warps together.
constexpr int kLongRun = 16;

// Sum of the partial rows of chunks [k0, k1), four loads in flight (eight would
// halve the resident warps, and most runs are short).
__device__ __forceinline__ void add_partials(const SumArgs& a, int k0, int k1, int c, float (&acc)[8]) {
#pragma unroll 1
  for (int k = k0; k < k1; k += 4) {
    Raw8<float> f[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (k + u < k1) f[u].load(a.part + (size_t)(k + u) * 2 * a.N + c);
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (k + u < k1) f[u].add_to(acc);
  }
}

template <int CHUNK>
__global__ void __launch_bounds__(256, 4) join_runs(const SumArgs a) {
  start_after_previous();
  __shared__ int s_end[8];
  __shared__ float s_part[8][kSlice];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int chunk = blockIdx.x * 8 + warp;
  const int c = blockIdx.y * kSlice + lane * 8;
  const bool col = c < a.N;
  // only where a run begins in this chunk and goes on behind it
  uint32_t v = 0;
  bool begins = false;
  if (chunk + 1 < a.chunks) {
    const int i0 = chunk * CHUNK;
    v = a.key[i0 + CHUNK - 1];
    begins = v < (uint32_t)a.V && a.key[i0 + CHUNK] == v &&
             !(a.key[i0] == v && chunk > 0 && a.key[i0 - 1] == v);
  }
  int end = 0;  // the first chunk whose first entry lies behind the run
  if (begins) {
    auto in_run = [&](int k) { return k < a.chunks && a.key[(size_t)k * CHUNK] == v; };
    uint32_t m = __ballot_sync(0xffffffffu, in_run(chunk + 2 + lane));
    end = chunk + 2 + (m == 0xffffffffu ? 32 : __ffs(~m) - 1);
    if (m == 0xffffffffu) {
      int hi = a.chunks;  // chunk end - 1 is in the run, hi is not; 32 probes at a time
      while (hi - end > 0) {
        const int step = (hi - end + 31) / 32;
        const int k = end - 1 + step * (lane + 1);
        m = __ballot_sync(0xffffffffu, k < hi && in_run(k));
        const int n = m == 0xffffffffu ? 32 : __ffs(~m) - 1;
        end += step * n;
        hi = min(hi, end - 1 + step);
      }
    }
  }
  const bool is_long = begins && end - chunk > kLongRun;
  if (lane == 0) s_end[warp] = is_long ? end : 0;
  float acc[8];
  if (begins && !is_long && col) {
    load8(a.part + ((size_t)chunk * 2 + 1) * a.N + c, acc);
    add_partials(a, chunk + 1, end, c, acc);
    write_row(a, v, c, acc);
  }
  __syncthreads();
  for (int w = 0; w < 8; ++w) {
    const int e = s_end[w], first = blockIdx.x * 8 + w;
    if (e == 0) continue;  // the same for the whole block
    const int per = (e - first - 1 + 7) / 8, k0 = min(e, first + 1 + warp * per), k1 = min(e, k0 + per);
#pragma unroll
    for (int x = 0; x < 8; ++x) acc[x] = 0.f;
    if (col) {
      add_partials(a, k0, k1, c, acc);
#pragma unroll
      for (int x = 0; x < 8; ++x) s_part[warp][lane * 8 + x] = acc[x];
    }
    __syncthreads();
    if (warp == w && col) {
      load8(a.part + ((size_t)first * 2 + 1) * a.N + c, acc);
      for (int u = 0; u < 8; ++u)
#pragma unroll
        for (int x = 0; x < 8; ++x) acc[x] += s_part[u][lane * 8 + x];
      write_row(a, v, c, acc);
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------------ host side
int sm_count() {
  static int sms = 0;
  if (!sms) {
    int dev = 0;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (sms <= 0) sms = 1;
  }
  return sms;
}

size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

struct GradLayout {
  size_t key[2], pos[2], hist, digit_total, part, total;
  int items, tiles, chunk, chunks, bits, passes;
  bool small;
};

GradLayout grad_layout(int T, int N, int V, bool zeroed) {
  GradLayout l;
  // keys per thread of a sorting block: small tiles spread few tokens over the SMs,
  // large ones leave fewer counts to scan (whole gradient, ten in a graph, 768 wide: 32768
  // tokens into 50000 rows 57 us at 2, 63 at 8; 65536: 71, 77; 131072 into 128100: 153, 133)
  l.items = T <= 65536 ? 2 : 8;
  l.tiles = (T + kSortThreads * l.items - 1) / (kSortThreads * l.items);
  // short chunks spread few tokens over more warps, long ones leave fewer partial
  // rows (whole gradient, bf16; 8192 x 1024: 46 us at 8, 58 at 32; 32768 x 768: 57, 58;
  // 65536 x 768: 85, 71; 131072 x 768: 161, 133)
  l.chunk = T <= 32768 ? 8 : 32;
  l.chunks = (T + l.chunk - 1) / l.chunk;
  int key_bits = 1;  // keys 0 .. V
  while (key_bits < 32 && ((unsigned long long)V >> key_bits) != 0) ++key_bits;
  // one block sorts what the zero fill hides (2048 x 768 into 50000 rows: 35 us, 34 in
  // tiles; 8192 x 1024: 46, 50), or few tokens (added to the table: 17, 22; 35, 30)
  l.small = T <= (zeroed ? kSmallSort : 2048);
  const int most = l.small ? kSmallBits : kMaxDigitBits;
  l.passes = (key_bits + most - 1) / most;
  l.bits = (key_bits + l.passes - 1) / l.passes;
  size_t at = 0;
  for (int b = 0; b < 2; ++b) {
    l.key[b] = at;
    at += up256((size_t)T * 4);
    l.pos[b] = at;
    at += up256((size_t)T * 4);
  }
  l.hist = at;
  at += up256(((size_t)l.tiles << l.bits) * 4);
  l.digit_total = at;
  at += up256((size_t)4 << kMaxDigitBits);
  l.part = at;
  at += up256((size_t)l.chunks * 2 * N * 4);
  l.total = at;
  return l;
}

bool al16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

df_status check_sizes(int T, int N, int V) {
  if (T < 0 || T > (1 << 30) || N < 1 || V < 1) return DF_ERR_INVALID_ARG;
  if (N % 8 != 0 || N > 65536) return DF_ERR_UNSUPPORTED;
  return DF_OK;
}

template <typename T>
void launch_lookup(const void* ids, int ids64, int n, const void* table, int V, int N, float scale, void* out,
                   int32_t* status, cudaStream_t s) {
  // four rows per warp once that still leaves every SM its resident warps (131072 x
  // 768: 40.7 us, 43.5 with one; 38912: 12.4, 12.8; 8192 x 1024: 5.5, 5.0; 2048: 4.0, 3.2)
  if (n >= 4 * 64 * sm_count())
    lookup_kernel<T, 4><<<(n + 31) / 32, 256, 0, s>>>(ids, ids64, n, static_cast<const T*>(table), V, N, scale,
                                                      static_cast<T*>(out), status);
  else
    lookup_kernel<T, 1><<<(n + 7) / 8, 256, 0, s>>>(ids, ids64, n, static_cast<const T*>(table), V, N, scale,
                                                    static_cast<T*>(out), status);
}

template <typename... Params, typename... Args>
bool launch_next(void (*kernel)(Params...), dim3 grid, int threads, size_t smem, cudaStream_t s, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess;
}

template <typename T, int CHUNK>
bool launch_sums(const SumArgs& a, const void* dout, cudaStream_t s) {
  const dim3 grid((a.chunks + 7) / 8, (a.N + kSlice - 1) / kSlice);
  return launch_next(sum_runs<T, CHUNK>, grid, 256, 0, s, a, static_cast<const T*>(dout)) &&
         launch_next(join_runs<CHUNK>, grid, 256, 0, s, a);
}

template <typename T>
bool launch_sums(const SumArgs& a, int chunk, const void* dout, cudaStream_t s) {
  return chunk == 8 ? launch_sums<T, 8>(a, dout, s) : launch_sums<T, 32>(a, dout, s);
}

}  // namespace
}  // namespace dfa

using namespace dfa;

extern "C" df_status df_embedding(const void* ids, int ids_64, int T, const void* table, int V, int N, float scale,
                                  void* out, df_dtype dtype, int32_t* status, df_stream_t stream) {
  const df_status st = check_sizes(T, N, V);
  if (st != DF_OK) return st;
  if (dtype != DF_BF16 && dtype != DF_FP16 && dtype != DF_FP32) return DF_ERR_INVALID_ARG;
  if (T == 0) return DF_OK;
  if (!ids || !table || !out) return DF_ERR_INVALID_ARG;
  if (((uintptr_t)ids & (ids_64 ? 7u : 3u)) != 0 || !al16(table) || !al16(out)) return DF_ERR_ALIGNMENT;
  const size_t row = (size_t)N * (dtype == DF_FP32 ? 4 : 2);
  if (overlapping({{out, T * row}}, {{ids, (size_t)T * (ids_64 ? 8 : 4)}, {table, V * row}})) return DF_ERR_INVALID_ARG;
  cudaStream_t s = (cudaStream_t)stream;
  if (dtype == DF_BF16) launch_lookup<__nv_bfloat16>(ids, ids_64, T, table, V, N, scale, out, status, s);
  else if (dtype == DF_FP16) launch_lookup<__half>(ids, ids_64, T, table, V, N, scale, out, status, s);
  else launch_lookup<float>(ids, ids_64, T, table, V, N, scale, out, status, s);
  return cudaGetLastError() == cudaSuccess ? DF_OK : DF_ERR_CUDA;
}

extern "C" size_t df_embedding_bwd_workspace_size(int T, int N, int V) {
  if (check_sizes(T, N, V) != DF_OK) return 0;
  return std::max({grad_layout(T, N, V, false).total, grad_layout(T, N, V, true).total, (size_t)256});
}

extern "C" df_status df_embedding_bwd(const void* ids, int ids_64, int T, const void* dout, int V, int N,
                                      float scale, int padding_idx, int accumulate, float* grad, df_dtype dtype,
                                      int32_t* status, void* workspace, size_t workspace_bytes,
                                      df_stream_t stream) {
  const df_status st = check_sizes(T, N, V);
  if (st != DF_OK) return st;
  if (dtype != DF_BF16 && dtype != DF_FP16 && dtype != DF_FP32) return DF_ERR_INVALID_ARG;
  if (!grad || padding_idx < -1 || padding_idx >= V || (T > 0 && (!ids || !dout))) return DF_ERR_INVALID_ARG;
  if (((uintptr_t)ids & (ids_64 ? 7u : 3u)) != 0 || !al16(dout) || !al16(grad) || ((uintptr_t)workspace & 255u) != 0)
    return DF_ERR_ALIGNMENT;
  const GradLayout l = grad_layout(T, N, V, !accumulate);
  if (!workspace || workspace_bytes < std::max<size_t>(l.total, 256)) return DF_ERR_WORKSPACE;
  if (overlapping({{grad, (size_t)V * N * 4}, {workspace, l.total}},
                  {{ids, (size_t)T * (ids_64 ? 8 : 4)}, {dout, (size_t)T * N * (dtype == DF_FP32 ? 4 : 2)}}))
    return DF_ERR_INVALID_ARG;
  cudaStream_t s = (cudaStream_t)stream;
  if (T == 0) {
    if (!accumulate && cudaMemsetAsync(grad, 0, (size_t)V * N * 4, s) != cudaSuccess) return DF_ERR_CUDA;
    return DF_OK;
  }
  char* base = static_cast<char*>(workspace);
  SortArgs a;
  a.ids = ids;
  a.ids64 = ids_64;
  a.hist = reinterpret_cast<uint32_t*>(base + l.hist);
  a.total = reinterpret_cast<uint32_t*>(base + l.digit_total);
  a.n = T;
  a.tiles = l.tiles;
  a.V = V;
  a.pad = padding_idx;
  a.bits = l.bits;
  a.status = status;
  a.fill = reinterpret_cast<uint4*>(grad);
  const size_t pieces = accumulate ? 0 : (size_t)V * N / 4;
  // The launches' shares of the zeros, as long as each takes by itself: 3 : 3 : 5 for
  // counts, scan and scatter.
  const size_t unit = pieces / (l.small ? 1 : 11 * (size_t)l.passes) + 1;
  size_t filled = 0;
  // the next launch's grid: its sorting blocks, and blocks that zero its share
  auto grid_for = [&](int blocks, int threads, int share) {
    a.blocks = blocks;
    a.fill_begin = filled;
    filled = a.fill_end = std::min(pieces, filled + share * unit);
    const size_t most = (size_t)sm_count() * (2048 / threads);
    return dim3((unsigned)(blocks + std::min(most, (a.fill_end - a.fill_begin + threads - 1) / threads)));
  };
  if (l.small) {
    if (cudaFuncSetAttribute(sort_small, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmallSmem) != cudaSuccess)
      return DF_ERR_CUDA;
    a.first = 1;
    a.shift = 0;
    a.key_out = reinterpret_cast<uint32_t*>(base + l.key[0]);
    a.pos_out = reinterpret_cast<uint32_t*>(base + l.pos[0]);
    const dim3 grid = grid_for(1, kSmallThreads, 1);
    if (!launch_next(sort_small, grid, kSmallThreads, kSmallSmem, s, a, l.passes)) return DF_ERR_CUDA;
  } else {
    const bool few = l.items == 2;
    for (int p = 0; p < l.passes; ++p) {
      a.first = p == 0;
      a.shift = p * l.bits;
      a.key = reinterpret_cast<uint32_t*>(base + l.key[(p + 1) & 1]);
      a.pos = reinterpret_cast<const uint32_t*>(base + l.pos[(p + 1) & 1]);
      a.key_out = reinterpret_cast<uint32_t*>(base + l.key[p & 1]);
      a.pos_out = reinterpret_cast<uint32_t*>(base + l.pos[p & 1]);
      dim3 grid = grid_for(l.tiles, kSortThreads, 3);
      if (!launch_next(few ? digit_counts<2> : digit_counts<8>, grid, kSortThreads, 0, s, a)) return DF_ERR_CUDA;
      grid = grid_for(((1 << l.bits) + 31) / 32, 256, 3);
      if (!launch_next(scan_over_tiles, grid, 256, 0, s, a)) return DF_ERR_CUDA;
      grid = grid_for(l.tiles, kSortThreads, 5);
      if (!launch_next(few ? scatter_by_digit<2> : scatter_by_digit<8>, grid, kSortThreads, 0, s, a)) return DF_ERR_CUDA;
    }
  }
  SumArgs u;
  u.key = a.key_out;  // of the last pass
  u.pos = a.pos_out;
  u.n = T;
  u.V = V;
  u.N = N;
  u.chunks = l.chunks;
  u.accumulate = accumulate;
  u.scale = scale;
  u.part = reinterpret_cast<float*>(base + l.part);
  u.grad = grad;
  const bool ok = dtype == DF_BF16   ? launch_sums<__nv_bfloat16>(u, l.chunk, dout, s)
                  : dtype == DF_FP16 ? launch_sums<__half>(u, l.chunk, dout, s)
                                     : launch_sums<float>(u, l.chunk, dout, s);
  return ok ? DF_OK : DF_ERR_CUDA;
}
