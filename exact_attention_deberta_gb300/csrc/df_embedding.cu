// Embedding lookup with scaling, out[t] = scale * table[ids[t]], and the
// gradient of the table, grad[v] (+)= scale * sum_{t: ids[t] = v} dout[t].
//
// Lookup: one warp per token, 16-byte vectors; HBM bound (each row that the
// ids reach is read once, the repeats come from L2, each output row is written
// once).
//
// Gradient.  Adding rows with atomics would make the last bits depend on the
// order of arrival, so the tokens are sorted by id first (a stable radix sort
// of (id, position) pairs) and every row of the table is then the sum of one
// run of the sorted list, in ascending position:
//   1. sort: least-significant digit first, at most 10 bits per pass (two
//      passes for ids below 2^20).  A pass counts the digits of each 2048-key
//      tile, scans the counts digit-major in one block, and scatters the tiles
//      (rank inside the tile by warp digit matching, so that equal digits keep
//      their order).  Ids that pass no gradient (the padding id, ids outside
//      the table) sort behind every other one and are left out.
//   2. sums: a warp takes 32 consecutive entries of the sorted list and 256
//      columns (8 per lane), adds rows in fp32 while the id stays the same and
//      writes each finished run.  A run that crosses a 32-entry boundary leaves
//      one partial row per chunk in the workspace.
//   3. join: the warp of the chunk in which such a run begins adds its partial
//      rows in order.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "df_common.cuh"

namespace dfa {
namespace {

constexpr int kSortThreads = 256;
constexpr int kSortItems = 8;                           // keys per thread
constexpr int kSortTile = kSortThreads * kSortItems;    // keys per block
constexpr int kMaxDigitBits = 10;
constexpr int kChunk = 32;                              // sorted entries per warp of the sums
constexpr int kSlice = 256;                             // columns per warp of the sums

template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&f)[8]) {
  if constexpr (sizeof(T) == 2) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    const T* h = reinterpret_cast<const T*>(&v);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = IO<T>::to_f(h[e]);
  } else {
    const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
}

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

__device__ __forceinline__ long long load_id(const void* ids, int ids64, size_t t) {
  return ids64 ? (long long)static_cast<const int64_t*>(ids)[t] : (long long)static_cast<const int32_t*>(ids)[t];
}

template <typename T>
__global__ void __launch_bounds__(256) lookup_kernel(const void* __restrict__ ids, int ids64, int tokens,
                                                     const T* __restrict__ table, int V, int N, float scale,
                                                     T* __restrict__ out, int32_t* status) {
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (t >= tokens) return;
  const long long id = load_id(ids, ids64, t);
  const bool in = id >= 0 && id < V;
  if (!in && lane == 0 && status) atomicCAS(status, 0, (int32_t)DF_ERR_INVALID_ARG);
  const T* src = table + (size_t)(in ? id : 0) * N;
  T* dst = out + (size_t)t * N;
  for (int c = lane * 8; c < N; c += 256) {
    float f[8];
    if (in) load8<T>(src + c, f);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = in ? f[e] * scale : 0.f;
    store8<T>(dst + c, f);
  }
}

// ---------------------------------------------------------------- sort by id
// A key is the id, or V for a token that passes no gradient.
struct SortArgs {
  const void* ids;      // first pass: the caller's ids
  int ids64;
  const uint32_t* key;  // later passes
  const uint32_t* pos;
  uint32_t* key_out;
  uint32_t* pos_out;
  uint32_t* hist;       // [digits][tiles]
  int n, tiles, V, pad, first, shift, bits;
  int32_t* status;
};

__device__ __forceinline__ uint32_t sort_key(const SortArgs& a, int i) {
  if (!a.first) return a.key[i];
  const long long id = load_id(a.ids, a.ids64, i);
  const bool in = id >= 0 && id < a.V;
  if (!in && a.status) atomicCAS(a.status, 0, (int32_t)DF_ERR_INVALID_ARG);
  return in && id != a.pad ? (uint32_t)id : (uint32_t)a.V;
}

__global__ void __launch_bounds__(kSortThreads) digit_counts(const SortArgs a) {
  __shared__ uint32_t cnt[1 << kMaxDigitBits];
  const int digits = 1 << a.bits;
  for (int d = threadIdx.x; d < digits; d += kSortThreads) cnt[d] = 0;
  __syncthreads();
  const int base = blockIdx.x * kSortTile;
#pragma unroll
  for (int k = 0; k < kSortItems; ++k) {
    const int i = base + k * kSortThreads + threadIdx.x;
    if (i < a.n) atomicAdd(&cnt[(sort_key(a, i) >> a.shift) & (digits - 1)], 1u);
  }
  __syncthreads();
  for (int d = threadIdx.x; d < digits; d += kSortThreads) a.hist[(size_t)d * a.tiles + blockIdx.x] = cnt[d];
}

// Exclusive prefix over m counts, one block of 1024 threads; each thread owns a
// contiguous range.
__global__ void __launch_bounds__(1024) scan_digit_counts(uint32_t* __restrict__ h, int m) {
  __shared__ uint32_t warp_sum[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t carry = 0;
  for (int base = 0; base < m; base += 4096) {
    const int i = base + threadIdx.x * 4;
    uint32_t v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = i + e < m ? h[i + e] : 0u;
    const uint32_t own = v[0] + v[1] + v[2] + v[3];
    uint32_t incl = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t u = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += u;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    if (warp == 0) {
      uint32_t w = warp_sum[lane];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t u = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += u;
      }
      warp_sum[lane] = w;
    }
    __syncthreads();
    uint32_t run = carry + (warp ? warp_sum[warp - 1] : 0u) + incl - own;
    carry += warp_sum[31];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (i + e < m) {
        h[i + e] = run;
        run += v[e];
      }
    __syncthreads();  // warp_sum is written again
  }
}

// Writes a tile's pairs to their places.  Warp w of the tile owns keys
// [w 256, w 256 + 256) in rounds of 32, so that (warp, round, lane) is the
// original order; equal digits of a round are ranked by lane.
__global__ void __launch_bounds__(kSortThreads) scatter_by_digit(const SortArgs a) {
  constexpr int kWarps = kSortThreads / 32;
  __shared__ uint32_t cnt[kWarps][1 << kMaxDigitBits];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int digits = 1 << a.bits;
  for (int d = threadIdx.x; d < digits; d += kSortThreads)
#pragma unroll
    for (int w = 0; w < kWarps; ++w) cnt[w][d] = 0;
  __syncthreads();
  const int base = blockIdx.x * kSortTile + warp * (kSortItems * 32);
  uint32_t key[kSortItems], rank[kSortItems];
#pragma unroll
  for (int k = 0; k < kSortItems; ++k) {
    const int i = base + k * 32 + lane;
    key[k] = i < a.n ? sort_key(a, i) : 0u;
  }
#pragma unroll
  for (int k = 0; k < kSortItems; ++k) {
    const int i = base + k * 32 + lane;
    const bool valid = i < a.n;
    const uint32_t d = (key[k] >> a.shift) & (digits - 1);
    const uint32_t same = __match_any_sync(0xffffffffu, valid ? d : 0xffffffffu);
    const uint32_t before = __popc(same & ((1u << lane) - 1u));
    uint32_t start = 0;
    if (valid && before == 0) {
      start = cnt[warp][d];
      cnt[warp][d] = start + __popc(same);
    }
    rank[k] = before + __shfl_sync(0xffffffffu, start, __ffs(same) - 1);
    __syncwarp();
  }
  __syncthreads();
  // the tile's place for each digit, then each warp's
  for (int d = threadIdx.x; d < digits; d += kSortThreads) {
    uint32_t at = a.hist[(size_t)d * a.tiles + blockIdx.x];
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const uint32_t c = cnt[w][d];
      cnt[w][d] = at;
      at += c;
    }
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kSortItems; ++k) {
    const int i = base + k * 32 + lane;
    if (i >= a.n) continue;
    const uint32_t d = (key[k] >> a.shift) & (digits - 1);
    const uint32_t to = cnt[warp][d] + rank[k];
    a.key_out[to] = key[k];
    a.pos_out[to] = a.first ? (uint32_t)i : a.pos[i];
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
  float* p = a.grad + (size_t)v * a.N + c;
  float f[8];
  if (a.accumulate) load8<float>(p, f);
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] = a.accumulate ? f[e] + acc[e] * a.scale : acc[e] * a.scale;
  store8<float>(p, f);
}

template <typename T>
__global__ void __launch_bounds__(256) sum_runs(const SumArgs a, const T* __restrict__ dout) {
  const int lane = threadIdx.x & 31;
  const int chunk = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (chunk >= a.chunks) return;
  const int c = blockIdx.y * kSlice + lane * 8;
  const bool col = c < a.N;
  const int i0 = chunk * kChunk, cnt = min(kChunk, a.n - i0);
  const uint32_t my_key = lane < cnt ? a.key[i0 + lane] : 0xffffffffu;
  const uint32_t my_pos = lane < cnt ? a.pos[i0 + lane] : 0u;
  const uint32_t before = chunk > 0 ? a.key[i0 - 1] : 0xffffffffu;
  const uint32_t after = i0 + kChunk < a.n ? a.key[i0 + kChunk] : 0xffffffffu;
  // entries that pass a gradient stand at the front
  const int live = __popc(__ballot_sync(0xffffffffu, my_key < (uint32_t)a.V));
  if (live == 0) return;
  float acc[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) acc[e] = 0.f;
  uint32_t cur = __shfl_sync(0xffffffffu, my_key, 0);
  bool head = before == cur;  // the current run began in an earlier chunk
  for (int k0 = 0; k0 < live; k0 += 8) {
    float f[8][8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const uint32_t p = __shfl_sync(0xffffffffu, my_pos, k0 + u);
      if (col && k0 + u < live) load8<T>(dout + (size_t)p * a.N + c, f[u]);
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
      if (col) {
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] += f[u][e];
      }
    }
  }
  if (col) {
    const bool on = live == kChunk && after == cur;
    if (head) store8<float>(a.part + (size_t)chunk * 2 * a.N + c, acc);
    else if (on) store8<float>(a.part + ((size_t)chunk * 2 + 1) * a.N + c, acc);
    else write_row(a, cur, c, acc);
  }
}

__global__ void __launch_bounds__(256) join_runs(const SumArgs a) {
  const int lane = threadIdx.x & 31;
  const int chunk = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (chunk + 1 >= a.chunks) return;
  const int i0 = chunk * kChunk;
  const uint32_t v = a.key[i0 + kChunk - 1];
  // only where a run begins in this chunk and goes on behind it
  if (v >= (uint32_t)a.V || a.key[i0 + kChunk] != v) return;
  if (a.key[i0] == v && chunk > 0 && a.key[i0 - 1] == v) return;
  const int c = blockIdx.y * kSlice + lane * 8;
  if (c >= a.N) return;
  float acc[8], f[8];
  load8<float>(a.part + ((size_t)chunk * 2 + 1) * a.N + c, acc);
  for (int k = chunk + 1; k < a.chunks && a.key[(size_t)k * kChunk] == v; ++k) {
    load8<float>(a.part + (size_t)k * 2 * a.N + c, f);
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] += f[e];
  }
  write_row(a, v, c, acc);
}

// ------------------------------------------------------------------ host side
size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

struct GradLayout {
  size_t key[2], pos[2], hist, part, total;
  int tiles, chunks, bits, passes;
};

GradLayout grad_layout(int T, int N, int V) {
  GradLayout l;
  l.tiles = (T + kSortTile - 1) / kSortTile;
  l.chunks = (T + kChunk - 1) / kChunk;
  int key_bits = 1;  // keys 0 .. V
  while (key_bits < 32 && ((unsigned long long)V >> key_bits) != 0) ++key_bits;
  l.passes = (key_bits + kMaxDigitBits - 1) / kMaxDigitBits;
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
  lookup_kernel<T><<<(n + 7) / 8, 256, 0, s>>>(ids, ids64, n, static_cast<const T*>(table), V, N, scale,
                                               static_cast<T*>(out), status);
}

template <typename T>
void launch_sums(const SumArgs& a, const void* dout, dim3 grid, cudaStream_t s) {
  sum_runs<T><<<grid, 256, 0, s>>>(a, static_cast<const T*>(dout));
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
  cudaStream_t s = (cudaStream_t)stream;
  if (dtype == DF_BF16) launch_lookup<__nv_bfloat16>(ids, ids_64, T, table, V, N, scale, out, status, s);
  else if (dtype == DF_FP16) launch_lookup<__half>(ids, ids_64, T, table, V, N, scale, out, status, s);
  else launch_lookup<float>(ids, ids_64, T, table, V, N, scale, out, status, s);
  return cudaGetLastError() == cudaSuccess ? DF_OK : DF_ERR_CUDA;
}

extern "C" size_t df_embedding_bwd_workspace_size(int T, int N, int V) {
  if (check_sizes(T, N, V) != DF_OK) return 0;
  return std::max<size_t>(grad_layout(T, N, V).total, 256);
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
  const GradLayout l = grad_layout(T, N, V);
  if (!workspace || workspace_bytes < std::max<size_t>(l.total, 256)) return DF_ERR_WORKSPACE;
  cudaStream_t s = (cudaStream_t)stream;
  if (!accumulate && cudaMemsetAsync(grad, 0, (size_t)V * N * 4, s) != cudaSuccess) return DF_ERR_CUDA;
  if (T == 0) return DF_OK;
  char* base = static_cast<char*>(workspace);
  SortArgs a;
  a.ids = ids;
  a.ids64 = ids_64;
  a.hist = reinterpret_cast<uint32_t*>(base + l.hist);
  a.n = T;
  a.tiles = l.tiles;
  a.V = V;
  a.pad = padding_idx;
  a.bits = l.bits;
  a.status = status;
  for (int p = 0; p < l.passes; ++p) {
    a.first = p == 0;
    a.shift = p * l.bits;
    a.key = reinterpret_cast<const uint32_t*>(base + l.key[(p + 1) & 1]);
    a.pos = reinterpret_cast<const uint32_t*>(base + l.pos[(p + 1) & 1]);
    a.key_out = reinterpret_cast<uint32_t*>(base + l.key[p & 1]);
    a.pos_out = reinterpret_cast<uint32_t*>(base + l.pos[p & 1]);
    digit_counts<<<l.tiles, kSortThreads, 0, s>>>(a);
    scan_digit_counts<<<1, 1024, 0, s>>>(a.hist, l.tiles << l.bits);
    scatter_by_digit<<<l.tiles, kSortThreads, 0, s>>>(a);
  }
  SumArgs u;
  u.key = a.key_out;
  u.pos = a.pos_out;
  u.n = T;
  u.V = V;
  u.N = N;
  u.chunks = l.chunks;
  u.accumulate = accumulate;
  u.scale = scale;
  u.part = reinterpret_cast<float*>(base + l.part);
  u.grad = grad;
  const dim3 grid((l.chunks + 7) / 8, (N + kSlice - 1) / kSlice);
  if (dtype == DF_BF16) launch_sums<__nv_bfloat16>(u, dout, grid, s);
  else if (dtype == DF_FP16) launch_sums<__half>(u, dout, grid, s);
  else launch_sums<float>(u, dout, grid, s);
  join_runs<<<grid, 256, 0, s>>>(u);
  return cudaGetLastError() == cudaSuccess ? DF_OK : DF_ERR_CUDA;
}
