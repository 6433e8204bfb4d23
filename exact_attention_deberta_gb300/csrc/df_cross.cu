// Cross attention: host side of the forward (argument checks, tensor maps, the
// choice of kernel and split) and what the backward shares with it.
#include "df_cross_fwd.cuh"

#include <cudaTypedefs.h>
#include <math.h>

#include <algorithm>

namespace dfa {

namespace {

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  if (!fn) {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  }
  return fn;
}

bool al16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

}  // namespace

bool encode_heads(CUtensorMap* m, const void* base, long long rows, int heads, int d, bool bf16, int box_heads,
                  int box_rows) {
  auto enc = tensor_map_encoder();
  if (!enc) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)rows};
  const cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)d * heads * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_rows};
  const cuuint32_t es[3] = {1, 1, 1};
  return enc(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(base),
             dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t prepare_kernel(const void* kernel, int bytes, int regs, std::atomic<uint64_t>* done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (dev < 64 && (done->load(std::memory_order_acquire) & bit)) return cudaSuccess;
  cudaFuncAttributes fa;
  e = cudaFuncGetAttributes(&fa, kernel);
  if (e != cudaSuccess) return e;
  if (fa.numRegs < regs) return cudaErrorInvalidConfiguration;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev < 64) done->fetch_or(bit, std::memory_order_release);
  return e;
}

int device_sms() {
  static int sms = 0;
  if (!sms) {
    int dev = 0;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (sms <= 0) sms = 1;
  }
  return sms;
}

long long cross_query_tiles(const CrossArgs& a) {
  const long long per = (a.Lq + a.tpt - 1) / a.tpt;
  if (!a.cu_q) return per * a.B * a.Hk;
  // packed: every sequence and the rows behind the last one end in a tile of their own
  return ((long long)a.Tq / a.tpt + a.B + 1) * a.Hk;
}

df_status cross_check(const void* q, const void* k, const void* v, const uint8_t* key_mask, const int32_t* cu_q,
                      const int32_t* cu_k, int B, int H, int Hk, int Lq, int Lk, int total_q, int total_k, int d,
                      float scale, df_dtype dtype, int32_t* status, CrossArgs* a) {
  if (B < 0 || H < 1 || Hk < 1 || H % Hk != 0 || Lq < 0 || Lk < 0 || total_q < 0 || total_k < 0 || d < 1)
    return DF_ERR_INVALID_ARG;
  if (dtype != DF_BF16 && dtype != DF_FP16 && dtype != DF_FP32) return DF_ERR_INVALID_ARG;
  // (scale log2(e) is finite too)
  if (!(scale > 0.f) || !(scale <= 2.0e38f) || (key_mask && cu_k)) return DF_ERR_INVALID_ARG;
  if (!cu_q && (long long)B * Lq != total_q) return DF_ERR_INVALID_ARG;
  if (!cu_k && (long long)B * Lk != total_k) return DF_ERR_INVALID_ARG;
  if (dtype == DF_FP32 || d % 8 != 0 || d > 128 || H / Hk > 128) return DF_ERR_UNSUPPORTED;
  if (total_q > (1 << 30) || total_k > (1 << 30)) return DF_ERR_UNSUPPORTED;
  // a grid has a CTA for every tile
  if ((long long)Hk * ((long long)std::max(total_q, total_k) + B + 1) > 0x7fffffffll) return DF_ERR_UNSUPPORTED;
  if ((total_q > 0 && !q) || (total_k > 0 && (!k || !v))) return DF_ERR_INVALID_ARG;
  if (!al16(q) || !al16(k) || !al16(v) || ((uintptr_t)cu_q & 3u) != 0 || ((uintptr_t)cu_k & 3u) != 0)
    return DF_ERR_ALIGNMENT;
  a->key_mask = key_mask;
  a->cu_q = cu_q;
  a->cu_k = cu_k;
  a->B = B;
  a->H = H;
  a->Hk = Hk;
  a->G = H / Hk;
  a->Lq = Lq;
  a->Lk = Lk;
  a->Tq = total_q;
  a->Tk = total_k;
  a->d = d;
  a->tpt = 128 / a->G;
  a->scale = scale;
  a->kscale = (float)((double)scale * 1.4426950408889634);
  a->status = status;
  a->budget = wait_budget();
  return DF_OK;
}

}  // namespace dfa

using namespace dfa;

extern "C" df_status df_cross_attn_fwd(const void* q, const void* k, const void* v, const uint8_t* key_mask,
                                       const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k, int B, int H, int Hk,
                                       int Lq, int Lk, int total_q, int total_k, int d, float scale, df_dtype dtype,
                                       void* out, void* out_lo, float* lse, int32_t* status, df_stream_t stream) {
  FwdArgs a;
  const df_status st = cross_check(q, k, v, key_mask, cu_seqlens_q, cu_seqlens_k, B, H, Hk, Lq, Lk, total_q, total_k,
                                   d, scale, dtype, status, &a.c);
  if (st != DF_OK) return st;
  if (total_q == 0) return DF_OK;
  if (!out) return DF_ERR_INVALID_ARG;
  if (!al16(out) || !al16(out_lo) || ((uintptr_t)lse & 3u) != 0) return DF_ERR_ALIGNMENT;
  const size_t q_bytes = (size_t)total_q * H * d * 2, k_bytes = (size_t)total_k * Hk * d * 2;
  const size_t cu_bytes = ((size_t)B + 1) * 4;
  if (overlapping({{out, q_bytes}, {out_lo, q_bytes}, {lse, (size_t)total_q * H * 4}},
                  {{q, q_bytes}, {k, k_bytes}, {v, k_bytes}, {key_mask, (size_t)total_k}, {cu_seqlens_q, cu_bytes},
                   {cu_seqlens_k, cu_bytes}}))
    return DF_ERR_INVALID_ARG;
  a.out = out;
  a.out_lo = out_lo;
  a.lse = lse;
  const bool bf16 = dtype == DF_BF16;
  FwdMaps maps;
  // without keys no copy of k or v is made: the maps then describe q
  const void* kp = total_k > 0 ? k : q;
  const void* vp = total_k > 0 ? v : q;
  const long long krows = total_k > 0 ? total_k : total_q;
  const int kheads = total_k > 0 ? Hk : H;
  if (!encode_heads(&maps.q, q, total_q, H, d, bf16, a.c.G, a.c.tpt) ||
      !encode_heads(&maps.k, kp, krows, kheads, d, bf16, 1, kFwdKeys) ||
      !encode_heads(&maps.v, vp, krows, kheads, d, bf16, 1, kFwdKeys))
    return DF_ERR_CUDA;
  const long long items = cross_query_tiles(a.c);
  const int sms = device_sms();
  // Fewer items than half the SMs: clusters share them, with at least two key tiles
  // for each CTA (both warpgroups at work).  12 heads, one query, 8192 keys: 12 us
  // against 36 without; 8 heads, d = 128, 64 queries, 4096 keys: 13 against 38; 4 x
  // 12 heads, 33 queries, 300 keys: 9.3 against 10.9 with a tile for each.
  a.splits = 1;
  const int key_tiles = (Lk + kFwdKeys - 1) / kFwdKeys;
  while (a.splits < 8 && items * a.splits * 2 <= sms && a.splits * 4 <= key_tiles) a.splits *= 2;
  a.split_bits = a.splits == 8 ? 3 : a.splits / 2;
  const int grid = (int)items * a.splits;
  cudaStream_t s = (cudaStream_t)stream;
  const cudaError_t e = d <= 64 ? launch_cross64(a, maps, bf16, grid, s) : launch_cross128(a, maps, bf16, grid, s);
  return e == cudaSuccess ? DF_OK : DF_ERR_CUDA;
}
