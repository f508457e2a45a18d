// Routing to experts: scores, balance bias, groups, top-k and renormalised weights.
//
// One warp takes a token.  Lane i holds experts 128c + 4i + j (c < kChunks, j < 4) in
// registers, so a row of logits is read once in 16-byte (bf16: 8-byte) pieces; scores,
// ranks and choice never leave the warp.  A rank is kept as an order-preserving uint32
// of its fp32 value, which lets one redux.sync find the warp's maximum.
#include "common.cuh"

namespace memra {
namespace {

constexpr int kRouteWarps = 4;

// Bits of v in an order that compares as unsigned; 0 lies below every value (taken).
__device__ __forceinline__ uint32_t rank_of(float v) {
  const uint32_t u = __float_as_uint(v);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t r) {
  return __uint_as_float((r & 0x80000000u) ? (r & 0x7fffffffu) : ~r);
}

struct RouteArgs {
  const void* logits;
  int64_t T, stride_t;
  int E;
  const float* bias;
  int score, n_groups, topk_groups, group_top, top_k, renormalize, vec;
  float scale;
  int32_t* ids;
  float* gate_w;
};

template <typename T>
__device__ __forceinline__ float logit_at(const T* p);
template <>
__device__ __forceinline__ float logit_at<float>(const float* p) { return *p; }
template <>
__device__ __forceinline__ float logit_at<uint16_t>(const uint16_t* p) {
  return __uint_as_float((uint32_t)*p << 16);
}
__device__ __forceinline__ void logits4(const float* p, float v[4]) {
  const float4 a = *reinterpret_cast<const float4*>(p);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
}
__device__ __forceinline__ void logits4(const uint16_t* p, float v[4]) {
  const uint2 a = *reinterpret_cast<const uint2*>(p);
  v[0] = __uint_as_float(a.x << 16); v[1] = __uint_as_float(a.x & 0xffff0000u);
  v[2] = __uint_as_float(a.y << 16); v[3] = __uint_as_float(a.y & 0xffff0000u);
}

template <int kChunks, typename T>
__global__ void __launch_bounds__(kRouteWarps * 32) route_kernel(RouteArgs a) {
  constexpr int kVals = 4 * kChunks;
  extern __shared__ float rows[];  // [kRouteWarps][E], with groups only
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = (int64_t)blockIdx.x * kRouteWarps + warp;
  if (t >= a.T) return;
  const T* row = static_cast<const T*>(a.logits) + t * a.stride_t;
  const float kInf = __int_as_float(0x7f800000);

  float s[kVals];
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
    const int e = 128 * c + 4 * lane;
    if (a.vec) {
      if (e < a.E) logits4(row + e, s + 4 * c);
      else s[4 * c] = s[4 * c + 1] = s[4 * c + 2] = s[4 * c + 3] = -kInf;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) s[4 * c + j] = e + j < a.E ? logit_at<T>(row + e + j) : -kInf;
    }
  }
#pragma unroll
  for (int i = 0; i < kVals; ++i)  // NaN -> -inf (fmaxf drops it), +inf -> the largest finite value
    s[i] = fminf(fmaxf(s[i], -kInf), 3.402823466e38f);

  uint32_t masked = 0;  // bit i: value i is a masked expert or none
#pragma unroll
  for (int i = 0; i < kVals; ++i) masked |= (s[i] == -kInf ? 1u : 0u) << i;
  if (a.score == MEMRA_SCORE_SOFTMAX) {
    float m = s[0];
#pragma unroll
    for (int i = 1; i < kVals; ++i) m = fmaxf(m, s[i]);
    m = value_of(__reduce_max_sync(kFullMask, rank_of(m)));
    float z = 0.0f;
#pragma unroll
    for (int i = 0; i < kVals; ++i) {
      s[i] = (masked >> i) & 1u ? 0.0f : exp_cody_waite(__fsub_rn(s[i], m));
      z = __fadd_rn(z, s[i]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) z = __fadd_rn(z, __shfl_xor_sync(kFullMask, z, o));
#pragma unroll
    for (int i = 0; i < kVals; ++i) s[i] = (masked >> i) & 1u ? 0.0f : __fdiv_rn(s[i], z);
  } else {
#pragma unroll
    for (int i = 0; i < kVals; ++i)
      s[i] = (masked >> i) & 1u ? 0.0f
                                : __fdiv_rn(1.0f, __fadd_rn(1.0f, exp_cody_waite(-s[i])));
  }

  uint32_t r[kVals];
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = 4 * c + j, e = 128 * c + 4 * lane + j;
      float v = s[i];
      if (a.bias != nullptr && e < a.E) v = __fadd_rn(v, a.bias[e]);
      if ((masked >> i) & 1u) v = -kInf;
      r[i] = e < a.E ? rank_of(v) : 0u;
    }
  }

  if (a.n_groups > 1) {
    // Lane g reads group g's values from shared memory, each lane starting elsewhere in
    // its group so that groups of 32 do not meet in one bank.
    float* mine = rows + warp * a.E;
#pragma unroll
    for (int c = 0; c < kChunks; ++c)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int e = 128 * c + 4 * lane + j;
        if (e < a.E) mine[e] = value_of(r[4 * c + j]);
      }
    __syncwarp();
    const int size = a.E / a.n_groups;
    float g1 = -kInf, g2 = -kInf;
    if (lane < a.n_groups) {
      int at = lane % size;
      for (int i = 0; i < size; ++i) {
        const float v = mine[lane * size + at];
        g2 = fmaxf(g2, fminf(g1, v));
        g1 = fmaxf(g1, v);
        at = at + 1 == size ? 0 : at + 1;
      }
    }
    const float g = a.group_top == 1 ? g1 : __fadd_rn(g1, g2);
    int before = 0;
    for (int o = 0; o < a.n_groups; ++o) {
      const float other = __shfl_sync(kFullMask, g, o);
      before += (other > g || (other == g && o < lane)) ? 1 : 0;
    }
    const uint32_t keep =
        __ballot_sync(kFullMask, lane < a.n_groups && before < a.topk_groups);
    const uint32_t none = rank_of(-kInf);
#pragma unroll
    for (int c = 0; c < kChunks; ++c)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int e = 128 * c + 4 * lane + j;
        if (e < a.E && !((keep >> (e / size)) & 1u)) r[4 * c + j] = none;
      }
  }

  // top_k times the warp's largest rank, at its lowest index.
  const uint32_t live = rank_of(-kInf);
  int my_id[2] = {0, 0};
  float my_w[2] = {0.0f, 0.0f};
  float total = 0.0f;
  for (int n = 0; n < a.top_k; ++n) {
    uint32_t best = 0;
    int at = 0;
#pragma unroll
    for (int i = 0; i < kVals; ++i)
      if (r[i] > best) {
        best = r[i];
        at = i;
      }
    const uint32_t top = __reduce_max_sync(kFullMask, best);
    const int e = 128 * (at >> 2) + 4 * lane + (at & 3);
    const int id = (int)__reduce_min_sync(kFullMask, best == top ? (uint32_t)e : 0xffffffffu);
    float w = 0.0f;
    if (best == top && e == id) {
#pragma unroll
      for (int i = 0; i < kVals; ++i)
        if (i == at) {
          w = top > live ? s[i] : 0.0f;
          r[i] = 0;
        }
    }
    w = __shfl_sync(kFullMask, w, (id >> 2) & 31);
    total = __fadd_rn(total, w);
    if (lane == n) {
      my_id[0] = id;
      my_w[0] = w;
    } else if (lane == n - 32) {
      my_id[1] = id;
      my_w[1] = w;
    }
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int n = 32 * h + lane;
    if (n < a.top_k) {
      float w = my_w[h];
      if (a.renormalize) w = total > 0.0f ? __fdiv_rn(w, total) : 0.0f;
      a.ids[t * a.top_k + n] = my_id[h];
      a.gate_w[t * a.top_k + n] = __fmul_rn(w, a.scale);
    }
  }
}

template <typename T>
cudaError_t launch_route(const RouteArgs& a, cudaStream_t stream) {
  const dim3 grid((unsigned)((a.T + kRouteWarps - 1) / kRouteWarps)), block(kRouteWarps * 32);
  const size_t smem = a.n_groups > 1 ? sizeof(float) * kRouteWarps * a.E : 0;
  const int chunks = (a.E + 127) / 128;
  if (chunks <= 1) return launch_kernel(route_kernel<1, T>, grid, block, smem, stream, a);
  if (chunks <= 2) return launch_kernel(route_kernel<2, T>, grid, block, smem, stream, a);
  if (chunks <= 4) return launch_kernel(route_kernel<4, T>, grid, block, smem, stream, a);
  return launch_kernel(route_kernel<8, T>, grid, block, smem, stream, a);
}

}  // namespace
}  // namespace memra

using namespace memra;

extern "C" memra_status memra_moe_route(const void* logits, int32_t dtype, int64_t T, int64_t E,
                                        int64_t stride_t, const float* bias, int32_t score,
                                        int64_t n_groups, int64_t topk_groups, int64_t group_top,
                                        int64_t top_k, int32_t renormalize, float route_scale,
                                        int32_t* ids, float* gate_w, cudaStream_t stream) {
  if (T < 0 || E < 1 || top_k < 1 || stride_t < 0) return MEMRA_ERR_INVALID_ARG;
  if (dtype != MEMRA_BF16 && dtype != MEMRA_F32) return MEMRA_ERR_INVALID_ARG;
  if (score != MEMRA_SCORE_SOFTMAX && score != MEMRA_SCORE_SIGMOID) return MEMRA_ERR_INVALID_ARG;
  if (renormalize != 0 && renormalize != 1) return MEMRA_ERR_INVALID_ARG;
  if (n_groups < 1 || topk_groups < 1 || topk_groups > n_groups || E % n_groups != 0)
    return MEMRA_ERR_INVALID_ARG;
  if ((group_top != 1 && group_top != 2) || group_top > E / n_groups) return MEMRA_ERR_INVALID_ARG;
  if (top_k > topk_groups * (E / n_groups)) return MEMRA_ERR_INVALID_ARG;
  if (E > MEMRA_MAX_EXPERTS || top_k > MEMRA_MAX_TOP_K || n_groups > MEMRA_MAX_EXPERT_GROUPS)
    return MEMRA_ERR_UNSUPPORTED;
  if (T > (int64_t)INT32_MAX) return MEMRA_ERR_UNSUPPORTED;
  if (T == 0) return MEMRA_OK;
  if (!logits || !ids || !gate_w) return MEMRA_ERR_INVALID_ARG;
  const int es = dtype == MEMRA_BF16 ? 2 : 4;
  if (!aligned(logits, es) || !aligned(ids, 4) || !aligned(gate_w, 4) || !aligned(bias, 4))
    return MEMRA_ERR_ALIGNMENT;
  RouteArgs a;
  a.logits = logits;
  a.T = T;
  a.stride_t = stride_t;
  a.E = (int)E;
  a.bias = bias;
  a.score = score;
  a.n_groups = (int)n_groups;
  a.topk_groups = (int)topk_groups;
  a.group_top = (int)group_top;
  a.top_k = (int)top_k;
  a.renormalize = renormalize;
  a.scale = route_scale;
  a.ids = ids;
  a.gate_w = gate_w;
  a.vec = E % 4 == 0 && stride_t % 4 == 0 && aligned(logits, 4 * es) ? 1 : 0;
  const cudaError_t e = dtype == MEMRA_BF16 ? launch_route<uint16_t>(a, stream)
                                            : launch_route<float>(a, stream);
  if (e != cudaSuccess) return cuda_fail(e);
  return MEMRA_OK;
}
