// Cross attention, forward: what the kernels of the two tensor-core head sizes
// (df_cross64.cu, df_cross128.cu) share.
#pragma once

#include <type_traits>

#include "df_cross.cuh"

namespace dfa {

struct FwdArgs {
  CrossArgs c;
  void* out;
  void* out_lo;  // or NULL
  float* lse;    // or NULL
  int splits;    // CTAs per item (cluster size, 2^split_bits)
  int split_bits;
};

struct FwdMaps {
  CUtensorMap q, k, v;
};

cudaError_t launch_cross64(const FwdArgs& a, const FwdMaps& maps, bool bf16, bool self, int grid, cudaStream_t s);
cudaError_t launch_self64(const FwdArgs& a, const FwdMaps& maps, bool bf16, int grid, cudaStream_t s);
cudaError_t launch_self128(const FwdArgs& a, const FwdMaps& maps, bool bf16, int grid, cudaStream_t s);
cudaError_t launch_cross128(const FwdArgs& a, const FwdMaps& maps, bool bf16, bool self, int grid, cudaStream_t s);
constexpr int kFwdKeys = 128;  // keys per tile

// The base of a row's exponentials stands this many binary orders below its maximum.  A
// weight is then at most 2^(kBelow + 8) (the base moves by more than 2^8 only), and fp16
// holds weights down to 2^-21 of the largest with all their digits, and below that in steps
// of 2^-31 of it.  With the base at the maximum, weights of 2^-25 came to nothing, which is
// all that is left where the large ones meet values of 0.  The row's sum and O share the
// base, so nothing else changes.  bf16 has the range anyway.
template <bool BF16>
constexpr float kBelow = BF16 ? 0.f : 7.f;

// Key tiles of a band among `keys` keys.
__device__ __forceinline__ int band_tiles(const CrossBand& band, int keys) {
  const int all = (keys + 127) / 128;
  return max(all - band.skip, min(band.sinks, all));
}
// This CTA's key tiles [*t0, *t0 + n) of an item (of those that it meets); returns n.
__device__ __forceinline__ int key_part(const FwdArgs& args, const CrossItem& it, const CrossBand& band, uint32_t rank,
                                        int* t0) {
  const unsigned all = max((it.no + kFwdKeys - 1) / kFwdKeys - band.skip, band.sinks);
  *t0 = (int)((all * rank) >> args.split_bits);
  return (int)((all * (rank + 1)) >> args.split_bits) - *t0;
}

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

// 1 / x and log2 x by the hardware's approximations (a unit and 2^-22 off, of sums whose
// exponentials are that much off themselves; short, for code that runs once per item
// and has left the instruction caches by then).
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

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

// A cluster's join: every CTA has left its (max, sum) per row and its
// un-normalised O in shared memory; thread i of `threads` in each CTA adds up its
// share of the rows' 4-column pieces over all of them.
template <typename T, int D>
__device__ __forceinline__ void join_cluster(const FwdArgs& args, const CrossItem& it, uint32_t rank, int i0, int threads,
                                             uint32_t ml_addr, uint32_t o_addr) {
  const CrossArgs& a = args.c;
  constexpr int kPieces = D / 4;
  for (int i = (int)rank * threads + i0; i < 128 * kPieces; i += threads * args.splits) {
    const int row = i / kPieces, piece = i - row * kPieces;
    const int tok = row / a.G;
    if (tok >= it.nr || 4 * piece >= a.d) continue;
    float m = -INFINITY, l = 0.f;
    for (int r = 0; r < args.splits; ++r) m = fmaxf(m, ld_cluster(map_rank(ml_addr + 16 * row, r)).x);
    float o[4] = {0.f, 0.f, 0.f, 0.f};
    for (int r = 0; r < args.splits; ++r) {
      const float4 s = ld_cluster(map_rank(ml_addr + 16 * row, r));
      const float f = m != -INFINITY ? ex2(s.x - m) : 0.f;
      l += s.y * f;  // (NaN even where f is 0)
      if (f > 0.f) {
        const float4 v = ld_cluster(map_rank(o_addr + 4 * o_piece<D>(row, piece), r));
        o[0] += v.x * f;
        o[1] += v.y * f;
        o[2] += v.z * f;
        o[3] += v.w * f;
      }
    }
    const float inv = l != 0.f ? rcp(l) : 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) o[k] *= inv;
    const size_t orow = (size_t)(it.r0 + tok) * a.H + (size_t)it.hk * a.G + (row - tok * a.G);
    const size_t at = orow * a.d + 4 * piece;
    store_rounded<T, 4>(static_cast<T*>(args.out) + at, args.out_lo ? static_cast<T*>(args.out_lo) + at : nullptr,
                        o);
    if (args.lse && piece == 0) args.lse[orow] = l != 0.f ? (m + lg2(l)) * kLn2 : -INFINITY;
  }
}

template <typename... Params>
cudaError_t launch_clusters(void (*kernel)(Params...), const FwdArgs& a, const FwdMaps& maps, int grid, int threads,
                            uint32_t bytes, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
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

}  // namespace dfa
