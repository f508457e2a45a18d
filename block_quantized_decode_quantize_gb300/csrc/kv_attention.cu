// Attention over the paged 8-bit KV cache (layouts and arithmetic in memra.h).
//
// The simplest form: a CTA to a query row and head, a warp to every fourth key, one pass
// with a running maximum and sum for each warp, joined at the end.
#include <cuda_bf16.h>

#include "common.cuh"

namespace memra {
namespace {

struct AttnArgs {
  const void* q;
  int64_t T, Hq, stride_t, stride_h;
  const int8_t *kq, *vq;
  const float *kd, *vd;
  int64_t n_pages, max_pages;
  int Hkv, page, D, block;
  const int32_t *table, *kv_lens, *cu_q;
  int64_t B, window;
  float scale;
  void* out;
  float* lse;
  int32_t* status;
};

__device__ __forceinline__ float value(const float* p) { return *p; }
__device__ __forceinline__ float value(const uint16_t* p) {
  return __uint_as_float((uint32_t)*p << 16);
}
__device__ __forceinline__ void store(float* p, float v) { *p = v; }
__device__ __forceinline__ void store(uint16_t* p, float v) {
  *p = __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

template <typename T, int kD>
__global__ void __launch_bounds__(128) attention_rows_kernel(AttnArgs a) {
  constexpr int kPer = kD / 32;
  __shared__ float sm[4], sl[4], so[4][kD];
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = blockIdx.x / a.Hq;
  const int hq = (int)(blockIdx.x % a.Hq), h = hq / (int)(a.Hq / a.Hkv);
  int64_t b = 0;
  while (b < a.B && a.cu_q[b + 1] <= t) ++b;
  int64_t lo = 0, hi = 0;
  if (b < a.B) {
    int64_t len = a.kv_lens[b];
    if (len > a.max_pages * a.page) {
      len = a.max_pages * a.page;
      if (a.status != nullptr && threadIdx.x == 0) atomicOr(a.status, 1);
    }
    hi = len - (a.cu_q[b + 1] - t) + 1;
    if (hi > len) hi = len;
    if (a.window > 0 && hi > a.window) lo = hi - a.window;
  }
  const T* q = static_cast<const T*>(a.q) + t * a.stride_t + hq * a.stride_h;
  float x[kPer], o[kPer];
  for (int i = 0; i < kPer; ++i) {
    x[i] = value(q + lane * kPer + i);
    o[i] = 0.0f;
  }
  float m = -INFINITY, l = 0.0f;
  for (int64_t j = lo + warp; j < hi; j += 4) {
    const int64_t page = a.table[b * a.max_pages + j / a.page];
    if (page < 0 || page >= a.n_pages) {
      if (a.status != nullptr && lane == 0) atomicOr(a.status, 1);
      continue;
    }
    const int off = (int)(j % a.page);
    const int64_t head = page * a.Hkv + h;
    const int64_t row = (head * a.page + off) * kD + lane * kPer;
    const int64_t sc = head * (a.page / a.block) + off / a.block;
    float s = 0.0f;
    for (int i = 0; i < kPer; ++i) s += x[i] * (float)a.kq[row + i];
    for (int w = 16; w > 0; w >>= 1) s += __shfl_xor_sync(kFullMask, s, w);
    s *= a.kd[sc] * a.scale;
    const float mn = fmaxf(m, s), keep = expf(m - mn), p = expf(s - mn);
    const float pv = p * a.vd[sc];
    l = l * keep + p;
    m = mn;
    for (int i = 0; i < kPer; ++i) o[i] = o[i] * keep + pv * (float)a.vq[row + i];
  }
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
  for (int i = 0; i < kPer; ++i) so[warp][lane * kPer + i] = o[i];
  __syncthreads();
  const float mx = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3]));
  float sum = 0.0f, f[4];
  for (int w = 0; w < 4; ++w) {
    f[w] = sm[w] == -INFINITY ? 0.0f : expf(sm[w] - mx);
    sum += f[w] * sl[w];
  }
  T* out = static_cast<T*>(a.out) + (t * a.Hq + hq) * kD;
  for (int i = threadIdx.x; i < kD; i += 128) {
    float v = 0.0f;
    for (int w = 0; w < 4; ++w) v += f[w] * so[w][i];
    store(out + i, sum > 0.0f ? v / sum : 0.0f);
  }
  if (a.lse != nullptr && threadIdx.x == 0)
    a.lse[t * a.Hq + hq] = sum > 0.0f ? mx + logf(sum) : -INFINITY;
}

template <typename T>
cudaError_t launch_rows(const AttnArgs& a, cudaStream_t stream) {
  const dim3 grid((unsigned)(a.T * a.Hq)), block(128);
  if (a.D == 64) return launch_kernel(attention_rows_kernel<T, 64>, grid, block, 0, stream, a);
  if (a.D == 128) return launch_kernel(attention_rows_kernel<T, 128>, grid, block, 0, stream, a);
  return launch_kernel(attention_rows_kernel<T, 256>, grid, block, 0, stream, a);
}

}  // namespace
}  // namespace memra

using namespace memra;

extern "C" memra_status memra_kv_attention_q8(
    const void* q, int32_t dtype, int64_t T, int64_t Hq, int64_t stride_t, int64_t stride_h,
    const int8_t* kq, const float* kd, const int8_t* vq, const float* vd, int64_t n_pages,
    int64_t Hkv, int64_t page_size, int64_t D, int64_t block, const int32_t* block_table,
    int64_t B, int64_t max_pages, const int32_t* kv_lens, const int32_t* cu_q, float scale,
    int64_t window, void* out, float* lse, void* workspace, int32_t* dev_status,
    cudaStream_t stream) {
  if (T < 0 || B < 0 || Hkv < 1 || Hq < 1 || Hq % Hkv != 0 || n_pages < 0 || max_pages < 0)
    return MEMRA_ERR_INVALID_ARG;
  if (stride_t < 0 || stride_h < 0 || window < 0) return MEMRA_ERR_INVALID_ARG;
  if (dtype != MEMRA_BF16 && dtype != MEMRA_F32) return MEMRA_ERR_INVALID_ARG;
  if (page_size < 16 || page_size % 16 != 0 || block < 1 || page_size % block != 0)
    return MEMRA_ERR_INVALID_ARG;
  if (D != 64 && D != 128 && D != 256) return MEMRA_ERR_UNSUPPORTED;
  if (page_size > MEMRA_MAX_KV_PAGE || Hkv > 65535 || n_pages > INT32_MAX / page_size ||
      max_pages > INT32_MAX / page_size || T > INT32_MAX / Hq || B > (1 << 24))
    return MEMRA_ERR_UNSUPPORTED;
  if (T == 0) return MEMRA_OK;
  if (!q || !out || !workspace || !cu_q) return MEMRA_ERR_INVALID_ARG;
  if (B > 0 && (!kv_lens || (max_pages > 0 && !block_table))) return MEMRA_ERR_INVALID_ARG;
  if (n_pages > 0 && (!kq || !kd || !vq || !vd)) return MEMRA_ERR_INVALID_ARG;
  const int per16 = dtype == MEMRA_BF16 ? 8 : 4;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(kq, 16) || !aligned(vq, 16) ||
      !aligned(workspace, 16) || stride_t % per16 != 0 || stride_h % per16 != 0)
    return MEMRA_ERR_ALIGNMENT;
  const void* words[] = {kd, vd, block_table, kv_lens, cu_q, lse, dev_status};
  for (const void* p : words)
    if (!aligned(p, 4)) return MEMRA_ERR_ALIGNMENT;
  AttnArgs a;
  a.q = q;
  a.T = T;
  a.Hq = Hq;
  a.stride_t = stride_t;
  a.stride_h = stride_h;
  a.kq = kq;
  a.vq = vq;
  a.kd = kd;
  a.vd = vd;
  a.n_pages = n_pages;
  a.max_pages = max_pages;
  a.Hkv = (int)Hkv;
  a.page = (int)page_size;
  a.D = (int)D;
  a.block = (int)block;
  a.table = block_table;
  a.kv_lens = kv_lens;
  a.cu_q = cu_q;
  a.B = B;
  a.window = window;
  a.scale = scale;
  a.out = out;
  a.lse = lse;
  a.status = dev_status;
  const cudaError_t e =
      dtype == MEMRA_BF16 ? launch_rows<uint16_t>(a, stream) : launch_rows<float>(a, stream);
  if (e != cudaSuccess) return cuda_fail(e);
  return MEMRA_OK;
}
