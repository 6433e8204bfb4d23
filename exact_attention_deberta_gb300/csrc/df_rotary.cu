// Rotary positions: the columns of a head are rotated in pairs by an angle that grows with
// the token's position, y_a = A (x_a cos t - x_b sin t), y_b = A (x_b cos t + x_a sin t),
// t = position * f of the pair.  Pairs are (i, i + rot / 2) or (2i, 2i + 1), i < rot / 2;
// the columns from rot on are copied.  The inverse rotation is the gradient.
//
// Frequencies are held as turns a position in units of 2^-64 of a turn, so that an
// integer product modulo 2^64 is the angle without its whole turns, exactly: far positions
// cost no digits (position * f in fp32 is off by 0.06 rad at a million) and no fp64.  Of
// that angle the quarter turns are taken off as integers; what is left, at most an eighth
// of a turn, is rounded to fp32 for the sine and cosine.
//
// A thread keeps the sines and cosines of one vector of columns in registers and rotates
// that vector in several heads, two at a time in flight; neighbouring lanes take
// neighbouring columns, then heads, so that a warp's loads are whole lines.  HBM bound.
//
// Measured (GB300): 131072 tokens, 24 heads, d = 64, bf16: 131 us, 6.2 TB/s (four heads in
// flight: 146, one: 137; 24 heads a thread: 137); 8191 tokens, 20 heads, d = 128, 48 columns
// rotated in interleaved pairs, fp16: 19 us, 4.4 TB/s (one share of 2^20 threads: 23).
#include <math.h>

#include <algorithm>

#include "df_common.cuh"

namespace dfa {
namespace {

struct RotaryArgs {
  const void* x[2];
  void* y[2];
  long long xs[2], ys[2];  // elements between tokens
  int heads0, heads;       // of the first tensor, of both
  const void* pos;
  const uint64_t* turns;
  int T, d, rot;
  int chunks, groups;      // vectors of a head that threads take, threads that share its heads
  float amplitude;
  int pos_64, inter, inverse;
  int few;                 // fewer than 2^32 threads
};

// sin and cos of `phase` turns / 2^64.
__device__ __forceinline__ float2 sincos_turns(uint64_t phase) {
  const uint32_t u = (uint32_t)(phase >> 32);
  const uint32_t q = (u + 0x20000000u) >> 30;       // the nearest quarter turn
  const int r = (int)(u - (q << 30));               // 2^-32 turns from there, below 2^29
  float s, c;
  sincospif((float)r * 4.656612873077393e-10f, &s, &c);  // in half turns, at most 1 / 4
  if (q & 1) {
    const float t = s;
    s = c;
    c = -t;
  }
  return q & 2 ? make_float2(-s, -c) : make_float2(s, c);
}

template <typename T, int N>
struct Vec {
  using Word = typename std::conditional<
      N * sizeof(T) == 16, uint4,
      typename std::conditional<N * sizeof(T) == 8, uint2,
                                typename std::conditional<N * sizeof(T) == 4, uint32_t, uint16_t>::type>::type>::type;
  union {
    Word w;
    T e[N];
  };
  __device__ __forceinline__ Vec() {}
  __device__ __forceinline__ void load(const T* p) { w = *reinterpret_cast<const Word*>(p); }
  __device__ __forceinline__ void store(T* p) const { *reinterpret_cast<Word*>(p) = w; }
};

// N columns a vector.  Half layout: a thread takes vector c of the first half and its
// partner; interleaved: a vector holds N / 2 pairs (N = 1: the pair's columns one by one).
template <typename T, int N, bool INTER>
__global__ void __launch_bounds__(256) rotary_kernel(const RotaryArgs a) {
  constexpr int kPairs = INTER && N > 1 ? N / 2 : N;
  constexpr bool kTwo = !INTER || N == 1;  // two vectors
  constexpr int kFlight = 2;
  int c, g;
  long long t;
  if (a.few) {  // (32-bit divisions)
    const unsigned id = blockIdx.x * 256u + threadIdx.x, rest = id / (unsigned)a.chunks;
    c = (int)(id - rest * a.chunks);
    t = rest / (unsigned)a.groups;
    g = (int)(rest - (unsigned)t * a.groups);
  } else {
    const long long id = (long long)blockIdx.x * 256 + threadIdx.x, rest = id / a.chunks;
    c = (int)(id - rest * a.chunks);
    t = rest / a.groups;
    g = (int)(rest - t * a.groups);
  }
  if (t >= a.T) return;
  const int turned = a.rot / 2 / kPairs;  // chunks that are rotated
  const bool rotate = c < turned;
  // the vector's first column, and its partner's
  const int c0 = rotate ? (INTER ? 2 * kPairs * c : N * c) : a.rot + N * (c - turned);
  const int c1 = INTER ? c0 + 1 : c0 + a.rot / 2;
  float cs[kPairs], sn[kPairs];
  if (rotate) {
    const uint64_t p = a.pos_64 ? (uint64_t) static_cast<const int64_t*>(a.pos)[t]
                                : (uint64_t)(int64_t) static_cast<const int32_t*>(a.pos)[t];
#pragma unroll
    for (int e = 0; e < kPairs; ++e) {
      const float2 sc = sincos_turns(p * a.turns[kPairs * c + e]);
      sn[e] = (a.inverse ? -sc.x : sc.x) * a.amplitude;
      cs[e] = sc.y * a.amplitude;
    }
  }
  auto from = [&](int h) {
    const int i = h >= a.heads0;
    return static_cast<const T*>(a.x[i]) + t * a.xs[i] + (long long)(i ? h - a.heads0 : h) * a.d;
  };
  auto to = [&](int h) {
    const int i = h >= a.heads0;
    return static_cast<T*>(a.y[i]) + t * a.ys[i] + (long long)(i ? h - a.heads0 : h) * a.d;
  };
  for (int h0 = g; h0 < a.heads; h0 += kFlight * a.groups) {
    Vec<T, N> v[kFlight], w[kFlight];
#pragma unroll
    for (int k = 0; k < kFlight; ++k) {
      const int h = h0 + k * a.groups;
      if (h >= a.heads) break;
      const T* x = from(h);
      v[k].load(x + c0);
      if (kTwo && rotate) w[k].load(x + c1);
    }
#pragma unroll
    for (int k = 0; k < kFlight; ++k) {
      const int h = h0 + k * a.groups;
      if (h >= a.heads) break;
      T* y = to(h);
      if (rotate) {
#pragma unroll
        for (int e = 0; e < kPairs; ++e) {
          T& p = kTwo ? v[k].e[e] : v[k].e[2 * e];
          T& q = kTwo ? w[k].e[e] : v[k].e[2 * e + 1];
          const float x0 = IO<T>::to_f(p), x1 = IO<T>::to_f(q);
          p = IO<T>::from_f(x0 * cs[e] - x1 * sn[e]);
          q = IO<T>::from_f(x1 * cs[e] + x0 * sn[e]);
        }
        if (kTwo) w[k].store(y + c1);
      }
      v[k].store(y + c0);
    }
  }
}

template <typename T, int N>
cudaError_t launch(RotaryArgs a, cudaStream_t s) {
  const int pairs = a.inter && N > 1 ? N / 2 : N;
  a.chunks = a.rot / 2 / pairs + (a.d - a.rot) / N;
  // heads a thread: as many as leave some 2^19 threads, to twelve (the sines are formed once
  // for all of them); one where there is little to do
  const long long all = (long long)a.T * a.chunks;
  const long long share = std::min<long long>(12, std::max<long long>(1, all * a.heads >> 19));
  a.groups = (int)((a.heads + share - 1) / share);
  const long long blocks = (all * a.groups + 255) / 256;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  a.few = blocks < 1 << 24;
  if (a.inter)
    rotary_kernel<T, N, true><<<(unsigned)blocks, 256, 0, s>>>(a);
  else
    rotary_kernel<T, N, false><<<(unsigned)blocks, 256, 0, s>>>(a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_widest(const RotaryArgs& a, int n, cudaStream_t s) {
  if constexpr (sizeof(T) == 2)
    if (n >= 8) return launch<T, 8>(a, s);
  if (n >= 4) return launch<T, 4>(a, s);
  return n >= 2 ? launch<T, 2>(a, s) : launch<T, 1>(a, s);
}

// Whether rows of `w` bytes every `s` bytes from p on and others from q on share no byte.
bool rows_apart(const void* p, long long sp, long long wp, const void* q, long long sq, long long wq, long long rows) {
  const uintptr_t a = (uintptr_t)p, b = (uintptr_t)q;
  const uintptr_t a1 = a + (rows - 1) * sp + wp, b1 = b + (rows - 1) * sq + wq;
  if (a1 <= b || b1 <= a) return true;
  if (sp != sq) return false;
  const long long off = (long long)((b > a ? b - a : a - b) % (uintptr_t)sp);  // from the lower one's row
  const long long low = b > a ? wp : wq, high = b > a ? wq : wp;
  return off >= low && sp - off >= high;
}

}  // namespace
}  // namespace dfa

using namespace dfa;

extern "C" df_status df_rotary_table(int rot, double base, double factor, double original_len, double low, double high,
                                     uint64_t* turns) {
  if (!turns || rot < 2 || rot % 2 != 0 || rot > 65536) return DF_ERR_INVALID_ARG;
  if (!(base > 0.) || !isfinite(base) || !(factor > 0.) || !isfinite(factor)) return DF_ERR_INVALID_ARG;
  if (!(original_len >= 0.) || !isfinite(original_len)) return DF_ERR_INVALID_ARG;
  if (original_len > 0. && (!(low < high) || !isfinite(low) || !isfinite(high))) return DF_ERR_INVALID_ARG;
  const double two_pi = 6.283185307179586476925286766559;
  for (int i = 0; i < rot / 2; ++i) {
    const double f = pow(base, -2.0 * i / rot);
    double keep = 0.;
    if (original_len > 0.) keep = fmin(1., fmax(0., (original_len * f / two_pi - low) / (high - low)));
    const double turn = f * (keep + (1. - keep) / factor) / two_pi;
    if (!isfinite(turn)) return DF_ERR_INVALID_ARG;
    // 2^-64 turns: the whole turns fall out; 53 digits in two steps of 32 bits
    const double part = turn - floor(turn);
    const double hi = floor(ldexp(part, 32));
    turns[i] = ((uint64_t)hi << 32) + (uint64_t)ldexp(ldexp(part, 32) - hi, 32);
  }
  return DF_OK;
}

extern "C" df_status df_rotary(const void* x, int heads, long long x_stride, void* out, long long out_stride,
                               const void* x2, int heads2, long long x2_stride, void* out2, long long out2_stride,
                               const void* positions, int pos_64, int T, int d, int rot, int interleaved, int inverse,
                               const uint64_t* turns, float amplitude, df_dtype dtype, df_stream_t stream) {
  const int n = heads2 != 0 ? 2 : 1;
  const int h[2] = {heads, heads2};
  const void* from[2] = {x, x2};
  void* to[2] = {out, out2};
  const long long xs[2] = {x_stride, x2_stride}, ys[2] = {out_stride, out2_stride};
  if (T < 0 || T > (1 << 30) || d < 1 || rot < 2 || rot % 2 != 0 || rot > d || !(fabsf(amplitude) <= 3.0e38f))
    return DF_ERR_INVALID_ARG;
  if (dtype != DF_BF16 && dtype != DF_FP16 && dtype != DF_FP32) return DF_ERR_INVALID_ARG;
  if (d > 65536) return DF_ERR_UNSUPPORTED;
  const int size = dtype == DF_FP32 ? 4 : 2;
  RotaryArgs a = {};
  for (int i = 0; i < n; ++i) {
    if (h[i] < 1 || h[i] > 65536) return DF_ERR_INVALID_ARG;
    const long long width = (long long)h[i] * d;
    if (T > 1 && (xs[i] < width || ys[i] < width)) return DF_ERR_INVALID_ARG;
    if (xs[i] < 0 || ys[i] < 0 || xs[i] > (1ll << 31) || ys[i] > (1ll << 31))
      return DF_ERR_INVALID_ARG;
  }
  if (T == 0) return DF_OK;
  if (!positions || !turns) return DF_ERR_INVALID_ARG;
  if (((uintptr_t)positions & (pos_64 ? 7u : 3u)) != 0 || ((uintptr_t)turns & 7u) != 0) return DF_ERR_ALIGNMENT;
  // the widest vector that the pairs, the columns behind them and every row start on
  int width = 16 / size;
  while (width > 1 && ((interleaved ? rot : rot / 2) % width != 0 || (d - rot) % width != 0)) width /= 2;
  for (int i = 0; i < n; ++i) {
    if (!from[i] || !to[i]) return DF_ERR_INVALID_ARG;
    if (((uintptr_t)from[i] | (uintptr_t)to[i]) % size != 0) return DF_ERR_ALIGNMENT;
    while (width > 1 && (((uintptr_t)from[i] | (uintptr_t)to[i]) % (width * size) != 0 || d % width != 0 ||
                         (T > 1 && (xs[i] % width != 0 || ys[i] % width != 0))))
      width /= 2;
    a.x[i] = from[i];
    a.y[i] = to[i];
    a.xs[i] = xs[i];
    a.ys[i] = ys[i];
    a.heads += h[i];
  }
  a.heads0 = heads;
  for (int i = 0; i < n; ++i) {
    const long long wi = (long long)h[i] * d * size, si = T > 1 ? ys[i] * size : wi;
    for (int j = 0; j < n; ++j) {
      const long long wj = (long long)h[j] * d * size, sj = T > 1 ? xs[j] * size : wj;
      const bool in_place = i == j && to[i] == from[j] && (T == 1 || ys[i] == xs[j]);
      if (!in_place && !rows_apart(to[i], si, wi, from[j], sj, wj, T)) return DF_ERR_INVALID_ARG;
      if (j > i && !rows_apart(to[i], si, wi, to[j], T > 1 ? ys[j] * size : wj, wj, T)) return DF_ERR_INVALID_ARG;
    }
    const size_t bytes = (size_t)((T - 1) * si + wi);
    if (overlapping({{to[i], bytes}}, {{positions, (size_t)T * (pos_64 ? 8 : 4)}, {turns, (size_t)rot * 4}}))
      return DF_ERR_INVALID_ARG;
  }
  a.pos = positions;
  a.pos_64 = pos_64;
  a.turns = turns;
  a.T = T;
  a.d = d;
  a.rot = rot;
  a.amplitude = amplitude;
  a.inter = interleaved != 0;
  a.inverse = inverse != 0;
  cudaStream_t s = (cudaStream_t)stream;
  const cudaError_t e = dtype == DF_BF16   ? launch_widest<__nv_bfloat16>(a, width, s)
                        : dtype == DF_FP16 ? launch_widest<__half>(a, width, s)
                                           : launch_widest<float>(a, width, s);
  return e == cudaSuccess ? DF_OK : DF_ERR_CUDA;
}
