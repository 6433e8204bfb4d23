// The 8-bit cache: tokens appended to it, and read back in 16 bits.
//
// A block of 16 tokens of one head has one scale, the least power of two s with
// max |x| <= 448 s; its codes are e4m3(x / s) (with the largest s, which 1.75 2^127 asks for, 240 at most:
// 255 would round to 256, an infinity; 240 is off by less than e4m3's half a step still).  A power of two makes x / s exact, so that the
// one rounding is that of the code, and lets a block that is filled token by token grow its
// scale: the codes that it holds are halved as often as the scale doubles, which changes
// nothing above e4m3's subnormals.
//
// A warp takes the keys or the values of one block and head at a time, several one after another
// where there is much to do (what it costs to find a block is then paid once for them): 4 lanes a
// token's 32 columns, 8 tokens at a time, so that its loads are 64-byte runs and its stores
// 256-byte ones.  HBM bound.
//
// Measured (GB300): 64 ragged prompts of up to 8192 tokens, 12 heads, d = 64, bf16, appended and
// read back: 465 us, 6.4 TB/s; a token for each of 64 sequences of 499, 8 heads, d = 128, fp16, whose
// rows are then read: 30 us, 4.2 TB/s.
#include <math.h>

#include <algorithm>

#include "df_cache.cuh"

namespace dfa {
namespace {

struct StoreArgs {
  CacheView c;
  void *k, *v;        // [.., Hk, d]: read (append) or written (read)
  const int32_t* cu;  // [B + 1], or NULL: `len` rows of each sequence
  int B, len, total;
  long long slots;    // blocks that warps look for, over all sequences
  int pairs, warps;   // of the 2 Hk (head, keys or values) of a block: those that a warp takes, warps a block
  int32_t* status;
};

// Blocks are numbered so that no prefix sum is needed: a sequence of n rows that begins at
// row r has at most n / 16 + 2 blocks, and so those numbered from r / 16 + 2 b on to itself.
__device__ __forceinline__ long long slot_of(const StoreArgs& a, int b) {
  if (!a.cu) return (long long)b * (a.len / kBlock + 2);
  const int r = b <= a.B ? a.cu[b] : a.total;
  return (r > 0 ? r : 0) / kBlock + 2ll * b;
}
// The sequence of a slot, of b < seqs: the last whose first slot is not behind it.
__device__ __forceinline__ int sequence_of(const StoreArgs& a, int seqs, long long slot) {
  if (!a.cu) return (int)(slot / (a.len / kBlock + 2));
  int lo = 0, hi = seqs;  // slot_of(lo) <= slot, hi too far
  while (hi - lo > 1) {
    const int mid = lo + (hi - lo) / 2;
    if (slot_of(a, mid) <= slot)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// The least power of two s, from 2^-100 on, with top <= 448 s; top >= 0, finite.
__device__ __forceinline__ float block_scale(float top) {
  const uint32_t u = __float_as_uint(top);
  int e = (int)(u >> 23) - 127;           // top = m 2^e, m in [1, 2)
  e += ((u & 0x7fffffu) > 0x600000u) - 8;  // 448 = 1.75 2^8
  e = max(e, -100);
  return __uint_as_float((uint32_t)(e + 127) << 23);
}
// 1 / s of a power of two from 2^-100 to 2^120
__device__ __forceinline__ float inverse_scale(float s) { return __uint_as_float(0x7f000000u - __float_as_uint(s)); }

__device__ __forceinline__ float finite_or_nan(float x) { return fabsf(x) <= 3.4028235e38f ? x : __uint_as_float(0x7fffffffu); }

// The larger magnitudes of two pairs (a NaN gives way to the other).
__device__ __forceinline__ __nv_bfloat162 top2(__nv_bfloat162 m, __nv_bfloat162 x) { return __hmax2(m, __habs2(x)); }
__device__ __forceinline__ __half2 top2(__half2 m, __half2 x) { return __hmax2(m, __habs2(x)); }
template <typename T>
using Pair = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;

// The largest scale, of which a code above 240 would stand for an infinity.
constexpr float kTopScale = 1.329227995784916e36f;  // 2^120

// Eight values times inv, a power of two, as codes, `most` in magnitude at most; infinities as NaN.
template <typename T>
__device__ __forceinline__ uint2 codes8(const uint4& v, float inv, float most) {
  const T* e = reinterpret_cast<const T*>(&v);
  auto times = [&](T x) {
    const float f = finite_or_nan(IO<T>::to_f(x)) * inv;
    return fabsf(f) > most ? copysignf(most, f) : f;  // (a NaN stays one)
  };
  uint16_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = f32_codes(times(e[2 * i]), times(e[2 * i + 1]));
  return make_uint2(w[0] | (uint32_t)w[1] << 16, w[2] | (uint32_t)w[3] << 16);
}
// The same for values without an infinity and smaller scales, fewer instructions.  Products of 16-bit values with a
// power of two are exact where they matter: what leaves the normal range is far below half of
// the smallest code.  fp16: inv must be one, 2^-16 .. 2^15.
__device__ __forceinline__ uint2 finite_codes8(const uint4& v, __nv_bfloat162 inv) {
  const uint32_t x[4] = {v.x, v.y, v.z, v.w};
  uint16_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 y = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&x[i]), inv);
    const uint32_t u = *reinterpret_cast<const uint32_t*>(&y);
    w[i] = f32_codes(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
  }
  return make_uint2(w[0] | (uint32_t)w[1] << 16, w[2] | (uint32_t)w[3] << 16);
}
__device__ __forceinline__ uint2 finite_codes8(const uint4& v, __half2 inv) {
  const uint32_t x[4] = {v.x, v.y, v.z, v.w};
  uint16_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 y = __hmul2(*reinterpret_cast<const __half2*>(&x[i]), inv);
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(w[i]) : "r"(*reinterpret_cast<const uint32_t*>(&y)));
  }
  return make_uint2(w[0] | (uint32_t)w[1] << 16, w[2] | (uint32_t)w[3] << 16);
}
__device__ __forceinline__ __nv_bfloat162 both(float x, __nv_bfloat162) { return __float2bfloat162_rn(x); }
__device__ __forceinline__ __half2 both(float x, __half2) { return __float2half2_rn(x); }

// A warp's block and its first (head, keys or values): false behind the last one.
__device__ __forceinline__ bool warp_block(const StoreArgs& a, long long* slot, int* pair) {
  const unsigned id = blockIdx.x * 8u + (threadIdx.x >> 5);  // (below 2^31)
  const unsigned at = id / (unsigned)a.warps;
  *slot = at;
  *pair = (int)(id - at * a.warps) * a.pairs;
  return *slot < a.slots;
}
// Each sequence is looked over once.
__device__ __forceinline__ void look_over(const StoreArgs& a, long long slot, int pair) {
  if (slot >= a.B || pair != 0 || (threadIdx.x & 31) != 0) return;
  const CrossSide rows = {a.cu, a.len, a.total};
  int at;
  seq_rows(rows, (int)slot, a.status, &at);
  if (a.c.lengths[slot] < 0) cross_fail(a.status, (int)DF_ERR_INVALID_ARG);
}

template <typename T, int SLABS>
__global__ void __launch_bounds__(256) append_kernel(const StoreArgs a) {
  constexpr int D = 32 * SLABS;
  const int lane = threadIdx.x & 31;
  long long slot;
  int pair;
  if (!warp_block(a, &slot, &pair)) return;
  look_over(a, slot, pair);
  const int b = sequence_of(a, a.B, slot);
  if (b >= a.B) return;
  const CrossSide rows = {a.cu, a.len, a.total};
  int first;
  const int n = seq_rows(rows, b, nullptr, &first), held = a.c.lengths[b];
  if (n == 0 || held < 0) return;
  // the sequence's blocks from its first new token on, of which the first holds `part` older ones (k
  // below 0: a slot of the rows in front of the first sequence, whose blocks are none of the call's)
  const int k = (int)(slot - slot_of(a, b)), part = held % kBlock;
  if (k < 0 || (long long)k * kBlock >= part + n) return;
  const int blk = held / kBlock + k;
  const int from = k == 0 ? part : 0;                  // the block's tokens from here on are new,
  const int to = min(kBlock, part + n - k * kBlock);  // up to here
  const int id = page_of(a.c, b, blk);
  if (id < 0) {
    if (lane == 0) cross_fail(a.status, (int)DF_ERR_INVALID_ARG);
    return;
  }
  const int piece = lane & 3, row0 = lane >> 2;
  const long long step = (long long)a.c.Hk * D;  // elements from token to token
  const long long base = ((long long)first + k * kBlock - part + row0) * step + 8 * piece;  // the lane's, in head 0
  const size_t stride = (size_t)(a.c.page / kBlock) * record_bytes(D);  // from head to head of a page
  uint8_t* rec0 = record_of(a.c, id, 0, blk);
  const int last = min(pair + a.pairs, 2 * a.c.Hk);
#pragma unroll 1
  for (int p = pair; p < last; ++p) {
    const int which = p & 1, head = p >> 1;
    uint8_t* rec = rec0 + head * stride;
    uint8_t* codes = rec + 16 * D * which + 32 * row0 + 8 * piece;
    float* scale_at = reinterpret_cast<float*>(rec + 32 * D + 4 * which);
    const T* x = static_cast<const T*>(which ? a.v : a.k) + base + head * D;
    uint4 v[2 * SLABS];
#pragma unroll
    for (int j = 0; j < 2 * SLABS; ++j) {
      const int row = row0 + 8 * (j & 1);
      v[j] = make_uint4(0u, 0u, 0u, 0u);
      if (row >= from && row < to) v[j] = *reinterpret_cast<const uint4*>(x + (j & 1 ? 8 * step : 0) + 32 * (j >> 1));
    }
    Pair<T> m2 = both(0.f, Pair<T>());
#pragma unroll
    for (int j = 0; j < 2 * SLABS; ++j) {
      const Pair<T>* e = reinterpret_cast<const Pair<T>*>(&v[j]);
#pragma unroll
      for (int i = 0; i < 4; ++i) m2 = top2(m2, e[i]);
    }
    const uint32_t m = *reinterpret_cast<const uint32_t*>(&m2);
    const uint32_t bits = __reduce_max_sync(0xffffffffu, max(m & 0xffffu, m >> 16));  // (magnitudes: in order)
    const uint16_t half_bits = (uint16_t)bits;
    float top = IO<T>::to_f(*reinterpret_cast<const T*>(&half_bits));
    const bool finite = top <= 3.4028235e38f;
    if (!finite) {  // an infinity among them: the largest of the others
      top = 0.f;
#pragma unroll
      for (int j = 0; j < 2 * SLABS; ++j) {
        const T* e = reinterpret_cast<const T*>(&v[j]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float f = fabsf(IO<T>::to_f(e[i]));
          if (f <= 3.4028235e38f) top = fmaxf(top, f);
        }
      }
      top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
    }
    float s = block_scale(top);
    float grown = 1.f;  // old scale / new scale
    if (from > 0) {
      const float old = *scale_at;
      s = fmaxf(s, old);
      grown = old * inverse_scale(s);
    }
    const float inv = inverse_scale(s);
    __syncwarp();  // every lane has read the scale
    auto code_of = [&](int j) { return reinterpret_cast<uint2*>(codes + 512 * (j >> 1) + 256 * (j & 1)); };
    const bool plain = finite && (std::is_same<T, __half>::value ? inv >= 1.52587890625e-5f && inv <= 32768.f : s < kTopScale);
    if (plain) {
      const Pair<T> inv2 = both(inv, Pair<T>());
#pragma unroll
      for (int j = 0; j < 2 * SLABS; ++j)
        if (row0 + 8 * (j & 1) >= from && row0 + 8 * (j & 1) < to) *code_of(j) = finite_codes8(v[j], inv2);
    } else {
#pragma unroll
      for (int j = 0; j < 2 * SLABS; ++j)
        if (row0 + 8 * (j & 1) >= from && row0 + 8 * (j & 1) < to) *code_of(j) = codes8<T>(v[j], inv, s < kTopScale ? 448.f : 240.f);
    }
    if (from > 0 && grown != 1.f) {  // the block's scale has grown: its older codes again
#pragma unroll 1
      for (int j = 0; j < 2 * SLABS; ++j) {
        if (row0 + 8 * (j & 1) >= from) continue;
        const uint2 kept = *code_of(j);
        uint16_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t h = codes_f16((uint16_t)((i < 2 ? kept.x : kept.y) >> (16 * (i & 1))));
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
          w[i] = f32_codes(f.x * grown, f.y * grown);
        }
        *code_of(j) = make_uint2(w[0] | (uint32_t)w[1] << 16, w[2] | (uint32_t)w[3] << 16);
      }
    }
    if (lane == 0) *scale_at = s;
  }
}

template <typename T>
__device__ __forceinline__ T rounded(float f) {
  if constexpr (sizeof(T) == 2 && std::is_same<T, __half>::value) f = fminf(fmaxf(f, -65504.f), 65504.f) + (f != f ? f : 0.f);
  return IO<T>::from_f(f);
}

template <typename T, int SLABS>
__global__ void __launch_bounds__(256) read_kernel(const StoreArgs a) {
  constexpr int D = 32 * SLABS;
  const int lane = threadIdx.x & 31;
  long long slot;
  int pair;
  if (!warp_block(a, &slot, &pair)) return;
  look_over(a, slot, pair);
  // (packed: the rows behind the last sequence count as one more, which holds nothing)
  const int seqs = a.cu ? a.B + 1 : a.B;
  const int b = sequence_of(a, seqs, slot);
  if (b >= seqs) return;
  const CrossSide rows = {a.cu, a.len, a.total};
  int first, n, held = 0;
  if (b < a.B) {
    n = seq_rows(rows, b, nullptr, &first);
    held = max(a.c.lengths[b], 0);
  } else {
    first = min(max(a.cu[a.B], 0), a.total);
    n = a.total - first;
  }
  const int blk = (int)(slot - slot_of(a, b));
  if (blk < 0 || (long long)blk * kBlock >= n) return;  // (below 0: a slot of the rows in front of the first sequence)
  const int here = min(kBlock, n - blk * kBlock);  // rows of the block,
  int left = min(held - blk * kBlock, here);       // of which the cache holds these
  int id = 0;
  if (left > 0) {
    id = page_of(a.c, b, blk);
    if (id < 0) {
      if (lane == 0) cross_fail(a.status, (int)DF_ERR_INVALID_ARG);
      left = 0;
    }
  }
  const int piece = lane & 3, row0 = lane >> 2;
  const long long step = (long long)a.c.Hk * D;
  const long long base = (first + (long long)blk * kBlock + row0) * step + 8 * piece;
  const size_t stride = (size_t)(a.c.page / kBlock) * record_bytes(D);
  const uint8_t* rec0 = left > 0 ? record_of(a.c, id, 0, blk) : nullptr;
  const int last = min(pair + a.pairs, 2 * a.c.Hk);
#pragma unroll 1
  for (int p = pair; p < last; ++p) {
    const int which = p & 1, head = p >> 1;
    const uint8_t* rec = rec0 + head * stride;
    T* y = static_cast<T*>(which ? a.v : a.k) + base + head * D;
    float s = 0.f;
    uint2 v[2 * SLABS];
#pragma unroll
    for (int j = 0; j < 2 * SLABS; ++j) {
      v[j] = make_uint2(0u, 0u);
      if (row0 + 8 * (j & 1) < left)
        v[j] = *reinterpret_cast<const uint2*>(rec + 16 * D * which + 512 * (j >> 1) + 256 * (j & 1) + 32 * row0 + 8 * piece);
    }
    if (left > 0) s = *reinterpret_cast<const float*>(rec + 32 * D + 4 * which);
#pragma unroll
    for (int j = 0; j < 2 * SLABS; ++j) {
      const int row = row0 + 8 * (j & 1);
      if (row >= here) continue;
      alignas(16) T e[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t h = codes_f16((uint16_t)((i < 2 ? v[j].x : v[j].y) >> (16 * (i & 1))));
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
        e[2 * i] = rounded<T>(row < left ? f.x * s : 0.f);
        e[2 * i + 1] = rounded<T>(row < left ? f.y * s : 0.f);
      }
      uint4* at = reinterpret_cast<uint4*>(y + (j & 1 ? 8 * step : 0) + 32 * (j >> 1));
#pragma unroll
      for (int i = 0; i < (int)sizeof(T) / 2; ++i) at[i] = reinterpret_cast<const uint4*>(e)[i];
    }
  }
}

bool al16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

template <bool READ, typename T>
cudaError_t launch(StoreArgs a, cudaStream_t s) {
  // one pair a warp where there are few, up to eight while some 2^16 warps are left; reading, two where
  // one each would be more than a round of the SMs' warps (64 sequences of 500 rows, 8 heads, d = 128,
  // after a token each was appended: 32.5 -> 30.0 us; four: 32.8)
  const long long all = a.slots * a.c.Hk * 2;
  a.pairs = (int)std::min<long long>(8, std::max<long long>(READ && all > 16384 ? 2 : 1, all >> 16));
  a.warps = (2 * a.c.Hk + a.pairs - 1) / a.pairs;
  const long long blocks = (a.slots * a.warps + 7) / 8;
  if (blocks > 0x7fffffffll / 8) return cudaErrorInvalidConfiguration;
  void (*kernel)(StoreArgs) = nullptr;
  switch (a.c.d / 32) {
    case 1: kernel = READ ? read_kernel<T, 1> : append_kernel<T, 1>; break;
    case 2: kernel = READ ? read_kernel<T, 2> : append_kernel<T, 2>; break;
    case 3: kernel = READ ? read_kernel<T, 3> : append_kernel<T, 3>; break;
    default: kernel = READ ? read_kernel<T, 4> : append_kernel<T, 4>; break;
  }
  kernel<<<(unsigned)blocks, 256, 0, s>>>(a);
  return cudaGetLastError();
}

// What both calls check of their rows; fills the rest of *a.
df_status rows_check(const int32_t* cu, int B, int len, int total, StoreArgs* a) {
  if (len < 0 || total < 0 || (!cu && (long long)B * len != total)) return DF_ERR_INVALID_ARG;
  if (total > (1 << 30)) return DF_ERR_UNSUPPORTED;
  if (((uintptr_t)cu & 3u) != 0) return DF_ERR_ALIGNMENT;
  a->cu = cu;
  a->B = B;
  a->len = len;
  a->total = total;
  a->slots = cu ? (long long)total / kBlock + 2ll * (B + 1) + 1 : (long long)B * (len / kBlock + 2);
  return DF_OK;
}

}  // namespace

df_status cache_check(const void* cache, const int32_t* pages, const int32_t* lengths, int B, int Hk, int d, int page,
                      int n_pages, int max_pages, CacheView* c) {
  if (B < 0 || Hk < 1 || d < 1 || page < 1 || n_pages < 0 || max_pages < 0) return DF_ERR_INVALID_ARG;
  if (d % 32 != 0 || d > 128 || page % kBlock != 0 || page > (1 << 20) || Hk > 65536) return DF_ERR_UNSUPPORTED;
  if ((long long)max_pages * page > (1ll << 30)) return DF_ERR_UNSUPPORTED;
  if ((n_pages > 0 && !cache) || (B > 0 && (!lengths || (max_pages > 0 && !pages)))) return DF_ERR_INVALID_ARG;
  if (!al16(cache) || (((uintptr_t)pages | (uintptr_t)lengths) & 3u) != 0) return DF_ERR_ALIGNMENT;
  c->base = const_cast<uint8_t*>(static_cast<const uint8_t*>(cache));
  c->pages = pages;
  c->lengths = lengths;
  c->Hk = Hk;
  c->d = d;
  c->page = page;
  c->n_pages = n_pages;
  c->max_pages = max_pages;
  return DF_OK;
}

}  // namespace dfa

using namespace dfa;

extern "C" size_t df_cache_bytes(int n_pages, int Hk, int page, int d) {
  CacheView c;
  static const int32_t none = 0;
  if (n_pages < 1 || cache_check(&none - ((uintptr_t)&none % 16) / 4, &none, &none, 0, Hk, d, page, n_pages, 0, &c) != DF_OK)
    return 0;
  return cache_bytes(Hk, d, page, n_pages);
}

extern "C" df_status df_cache_append(const void* k, const void* v, const int32_t* cu_seqlens, int B, int Hk, int n,
                                     int total, int d, df_dtype dtype, void* cache, int n_pages, int page,
                                     const int32_t* pages, int max_pages, const int32_t* lengths, int32_t* status,
                                     df_stream_t stream) {
  StoreArgs a;
  if (dtype != DF_BF16 && dtype != DF_FP16 && dtype != DF_FP32) return DF_ERR_INVALID_ARG;
  df_status st = cache_check(cache, pages, lengths, B, Hk, d, page, n_pages, max_pages, &a.c);
  if (st == DF_OK) st = rows_check(cu_seqlens, B, n, total, &a);
  if (st != DF_OK) return st;
  if (dtype == DF_FP32) return DF_ERR_UNSUPPORTED;
  if (total == 0 || B == 0) return DF_OK;
  if (!k || !v) return DF_ERR_INVALID_ARG;
  if (!al16(k) || !al16(v)) return DF_ERR_ALIGNMENT;
  const size_t bytes = (size_t)total * Hk * d * 2;
  if (overlapping({{cache, cache_bytes(Hk, d, page, n_pages)}},
                  {{k, bytes}, {v, bytes}, {pages, (size_t)B * max_pages * 4}, {lengths, (size_t)B * 4},
                   {cu_seqlens, ((size_t)B + 1) * 4}}))
    return DF_ERR_INVALID_ARG;
  a.k = const_cast<void*>(k);
  a.v = const_cast<void*>(v);
  a.status = status;
  cudaStream_t s = (cudaStream_t)stream;
  const cudaError_t e = dtype == DF_BF16 ? launch<false, __nv_bfloat16>(a, s) : launch<false, __half>(a, s);
  return e == cudaSuccess ? DF_OK : DF_ERR_CUDA;
}

extern "C" df_status df_cache_read(const void* cache, int n_pages, int page, const int32_t* pages, int max_pages,
                                   const int32_t* lengths, const int32_t* cu_seqlens, int B, int Hk, int n, int total,
                                   int d, df_dtype dtype, void* k, void* v, int32_t* status, df_stream_t stream) {
  StoreArgs a;
  if (dtype != DF_BF16 && dtype != DF_FP16 && dtype != DF_FP32) return DF_ERR_INVALID_ARG;
  df_status st = cache_check(cache, pages, lengths, B, Hk, d, page, n_pages, max_pages, &a.c);
  if (st == DF_OK) st = rows_check(cu_seqlens, B, n, total, &a);
  if (st != DF_OK) return st;
  if (total == 0) return DF_OK;
  if (!k || !v) return DF_ERR_INVALID_ARG;
  if (!al16(k) || !al16(v)) return DF_ERR_ALIGNMENT;
  const size_t bytes = (size_t)total * Hk * d * (dtype == DF_FP32 ? 4 : 2);
  if (overlapping({{k, bytes}, {v, bytes}},
                  {{cache, cache_bytes(Hk, d, page, n_pages)}, {pages, (size_t)B * max_pages * 4}, {lengths, (size_t)B * 4},
                   {cu_seqlens, ((size_t)B + 1) * 4}}))
    return DF_ERR_INVALID_ARG;
  a.k = k;
  a.v = v;
  a.status = status;
  cudaStream_t s = (cudaStream_t)stream;
  const cudaError_t e = dtype == DF_BF16   ? launch<true, __nv_bfloat16>(a, s)
                        : dtype == DF_FP16 ? launch<true, __half>(a, s)
                                           : launch<true, float>(a, s);
  return e == cudaSuccess ? DF_OK : DF_ERR_CUDA;
}
