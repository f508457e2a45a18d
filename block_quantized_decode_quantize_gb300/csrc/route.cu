// Routing to experts: scores, balance bias, groups, top-k and renormalised weights.
//
// One warp takes a token.  Lane i holds experts 128c + 4i + j (c < kChunks, j < 4) in
// registers, so a row of logits is read once in 16-byte (bf16: 8-byte) pieces; scores,
// ranks and choice never leave the warp.  A rank is kept as an order-preserving uint32 of
// its fp32 value.  The choice: the top_k-th largest of the 32 lanes' own maxima is a bound
// that top_k experts reach, so only the few at or above it are sorted, by counting for
// each how many come before it.  8191 tokens of 256 experts in 8 groups, bf16, take 13.5 us
// (0.35 TB/s): 7 us are instruction issue (1181 a token, about a third of them the
// exponentials), the rest dependent latency at 43 % of the warps and a second, partly empty
// round of tokens (1216 CTAs of 4 warps).  Small batches are bound by the chain of exchanges
// between lanes: 16 tokens 4.0 us, one of 128 experts 2.4 us, where a kernel that does
// nothing takes 2.2.
#include "common.cuh"

namespace memra {
namespace {

constexpr int kRouteWarps = 4;

// Bits of v in an order that compares as unsigned; 0 lies below every value (taken).
__device__ __forceinline__ uint32_t rank_of(float v) {
  const uint32_t u = __float_as_uint(v);
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t r) {
  return __uint_as_float((r & 0x80000000u) ? (r & 0x7fffffffu) : ~r);
}

// exp_cody_waite, operation for operation; the nearest integer comes from adding
// 1.5 * 2^23, whose low bits then hold it for the exponent.
__device__ __forceinline__ float exp_score(float x) {
  constexpr float kMagic = 12582912.0f;
  x = fminf(fmaxf(x, -87.0f), 88.0f);
  const float z = __fadd_rn(__fmul_rn(x, 1.44269504088896341f), kMagic);
  const float kf = __fsub_rn(z, kMagic);
  float r = __fsub_rn(x, __fmul_rn(kf, 0.693359375f));
  r = __fsub_rn(r, __fmul_rn(kf, -2.12194440e-4f));
  float p = 1.0f / 5040.0f;
  p = __fadd_rn(__fmul_rn(p, r), 1.0f / 720.0f);
  p = __fadd_rn(__fmul_rn(p, r), 1.0f / 120.0f);
  p = __fadd_rn(__fmul_rn(p, r), 1.0f / 24.0f);
  p = __fadd_rn(__fmul_rn(p, r), 1.0f / 6.0f);
  p = __fadd_rn(__fmul_rn(p, r), 0.5f);
  p = __fadd_rn(__fmul_rn(p, r), 1.0f);
  p = __fadd_rn(__fmul_rn(p, r), 1.0f);
  return __fmul_rn(p, __uint_as_float(__float_as_uint(z) * 8388608u + 1065353216u));
}

struct RouteArgs {
  const void* logits;
  int64_t T, stride_t;
  int E;
  const float* bias;
  int score, n_groups, topk_groups, group_top, top_k, renormalize, vec;
  uint32_t group_magic;  // ceil(2^20 / (E / n_groups)): group of e = e * magic >> 20, e < 1024
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

// A warp's candidates and choice.
struct Picks {
  uint32_t rank[32];
  int id[32];
  float score[32];
  int chosen[32];
  float weight[32];
};

template <int kChunks, typename T>
__global__ void __launch_bounds__(kRouteWarps * 32) route_kernel(RouteArgs a) {
  constexpr int kVals = 4 * kChunks;
  extern __shared__ float rows[];  // [kRouteWarps][E], with groups only
  __shared__ Picks all_picks[kRouteWarps];
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const float kInf = __int_as_float(0x7f800000);
  Picks& picks = all_picks[warp];
  for (int64_t t = (int64_t)blockIdx.x * kRouteWarps + warp; t < a.T; t += (int64_t)gridDim.x * kRouteWarps) {
    const T* row = static_cast<const T*>(a.logits) + t * a.stride_t;

    float s[kVals], lowest = kInf;
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      const int e = 128 * c + 4 * lane;
      if (a.vec & 1) {
        if (e < a.E) logits4(row + e, s + 4 * c);
        else s[4 * c] = s[4 * c + 1] = s[4 * c + 2] = s[4 * c + 3] = -kInf;
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) s[4 * c + j] = e + j < a.E ? logit_at<T>(row + e + j) : -kInf;
      }
    }
#pragma unroll
    for (int i = 0; i < kVals; ++i) {  // NaN -> -inf (fmaxf drops it), +inf -> the largest finite value
      s[i] = fminf(fmaxf(s[i], -kInf), 3.402823466e38f);
      lowest = fminf(lowest, s[i]);
    }
    uint32_t masked = 0;  // bit i: value i is a masked expert or none
    const bool any_masked = __any_sync(kFullMask, lowest == -kInf);
    if (any_masked) {
#pragma unroll
      for (int i = 0; i < kVals; ++i) masked |= (s[i] == -kInf ? 1u : 0u) << i;
    }
    if (a.score == MEMRA_SCORE_SOFTMAX) {
      float m = s[0];
#pragma unroll
      for (int i = 1; i < kVals; ++i) m = fmaxf(m, s[i]);
      m = value_of(__reduce_max_sync(kFullMask, rank_of(m)));
      float z = 0.0f;
#pragma unroll
      for (int i = 0; i < kVals; ++i) {
        s[i] = exp_score(__fsub_rn(s[i], m));
        if (any_masked && ((masked >> i) & 1u)) s[i] = 0.0f;
        z = __fadd_rn(z, s[i]);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) z = __fadd_rn(z, __shfl_xor_sync(kFullMask, z, o));
      if (z == 0.0f) z = 1.0f;  // every expert masked
#pragma unroll
      for (int i = 0; i < kVals; ++i) s[i] = __fdiv_rn(s[i], z);
    } else {
#pragma unroll
      for (int i = 0; i < kVals; ++i) {
        s[i] = __frcp_rn(__fadd_rn(1.0f, exp_score(-s[i])));
        if (any_masked && ((masked >> i) & 1u)) s[i] = 0.0f;
      }
    }

    // Ranks: what the experts are chosen by (-inf for a masked one; kept in v while groups
    // are scored).
    float v[kVals];
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      const int e = 128 * c + 4 * lane;
      float bias[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      if (a.bias != nullptr) {
        if (a.vec & 2) {
          if (e < a.E) logits4(a.bias + e, bias);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (e + j < a.E) bias[j] = a.bias[e + j];
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int i = 4 * c + j;
        v[i] = a.bias != nullptr ? __fadd_rn(s[i], bias[j]) : s[i];
        if (any_masked && ((masked >> i) & 1u)) v[i] = -kInf;
      }
    }

    uint32_t keep = 0xffffffffu;  // bit g: group g stays
    if (a.n_groups > 1) {
      const int size = a.E / a.n_groups, lanes = size >> 2;
      float g1 = -kInf, g2 = -kInf;  // the two largest of group `lane`
      if (size <= 128 && (size & 3) == 0 && (lanes & (lanes - 1)) == 0) {
        // A group is the four values of 2^k neighbouring lanes: its two largest by exchange.
        const int per_chunk = 128 / size;
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
          const float h1 = fmaxf(v[4 * c], v[4 * c + 1]), l1 = fminf(v[4 * c], v[4 * c + 1]);
          const float h2 = fmaxf(v[4 * c + 2], v[4 * c + 3]), l2 = fminf(v[4 * c + 2], v[4 * c + 3]);
          float x1 = fmaxf(h1, h2), x2 = fmaxf(fminf(h1, h2), fmaxf(l1, l2));
          for (int o = 1; o < lanes; o <<= 1) {
            const float y1 = __shfl_xor_sync(kFullMask, x1, o), y2 = __shfl_xor_sync(kFullMask, x2, o);
            x2 = fmaxf(fminf(x1, y1), fmaxf(x2, y2));
            x1 = fmaxf(x1, y1);
          }
          const int from = (lane % per_chunk) * lanes;
          const float z1 = __shfl_sync(kFullMask, x1, from), z2 = __shfl_sync(kFullMask, x2, from);
          if (lane / per_chunk == c) {
            g1 = z1;
            g2 = z2;
          }
        }
      } else {
        // Any other size: lane g reads group g's values from shared memory, each lane
        // starting elsewhere in its group so that they do not meet in one bank.
        float* mine = rows + warp * a.E;
#pragma unroll
        for (int i = 0; i < kVals; ++i) {
          const int e = 128 * (i >> 2) + 4 * lane + (i & 3);
          if (e < a.E) mine[e] = v[i];
        }
        __syncwarp();
        if (lane < a.n_groups) {
          int at = lane % size;
          for (int i = 0; i < size; ++i) {
            const float x = mine[lane * size + at];
            g2 = fmaxf(g2, fminf(g1, x));
            g1 = fmaxf(g1, x);
            at = at + 1 == size ? 0 : at + 1;
          }
        }
        __syncwarp();
      }
      const float g = a.group_top == 1 ? g1 : __fadd_rn(g1, g2);
      int before = 0;
      for (int o = 0; o < a.n_groups; ++o) {
        const float other = __shfl_sync(kFullMask, g, o);
        before += (other > g || (other == g && o < lane)) ? 1 : 0;
      }
      keep = __ballot_sync(kFullMask, lane < a.n_groups && before < a.topk_groups);
    }
    uint32_t r[kVals];
#pragma unroll
    for (int i = 0; i < kVals; ++i) r[i] = rank_of(v[i]);
    if (a.n_groups > 1) {
#pragma unroll
      for (int i = 0; i < kVals; ++i) {
        const uint32_t e = 128 * (i >> 2) + 4 * lane + (i & 3);
        if (!((keep >> (((e * a.group_magic) >> 20) & 31)) & 1u)) r[i] = rank_of(-kInf);
      }
    }
    if (128 * kChunks != a.E) {
#pragma unroll
      for (int i = 0; i < kVals; ++i)
        if (128 * (i >> 2) + 4 * lane + (i & 3) >= a.E) r[i] = 0;
    }

    // The bound: after top_k rounds that each strike out the lanes with the largest maximum
    // left, what was largest in the last round (0 if none was left).
    uint32_t best = r[0];
#pragma unroll
    for (int i = 1; i < kVals; ++i) best = max(best, r[i]);
    uint32_t bound = 0;
    if (a.top_k <= 32)
      for (int n = 0; n < a.top_k; ++n) {
        bound = __reduce_max_sync(kFullMask, best);
        if (best == bound) best = 0;
      }
    bound = max(bound, 1u);
    uint32_t at_bound = 0;
#pragma unroll
    for (int i = 0; i < kVals; ++i) at_bound |= (r[i] >= bound ? 1u : 0u) << i;
    int upto = __popc(at_bound);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(kFullMask, upto, o);
      if (lane >= o) upto += u;
    }
    const int candidates = __shfl_sync(kFullMask, upto, 31);
    const uint32_t none = rank_of(-kInf);
    int my_id[2] = {0, 0};
    float my_w[2] = {0.0f, 0.0f};
    float total = 0.0f;
    if (candidates <= 32) {
      int to = upto - __popc(at_bound);
#pragma unroll
      for (int i = 0; i < kVals; ++i)
        if ((at_bound >> i) & 1u) {
          picks.rank[to] = r[i];
          picks.id[to] = 128 * (i >> 2) + 4 * lane + (i & 3);
          picks.score[to] = r[i] > none ? s[i] : 0.0f;
          ++to;
        }
      __syncwarp();
      const uint32_t my_rank = lane < candidates ? picks.rank[lane] : 0;
      const int id = lane < candidates ? picks.id[lane] : 0;
      int before = 0;
      for (int j = 0; j < candidates; ++j) {
        const uint32_t other = picks.rank[j];
        before += other > my_rank || (other == my_rank && picks.id[j] < id) ? 1 : 0;
      }
      if (lane < candidates && before < a.top_k) {
        picks.chosen[before] = id;
        picks.weight[before] = picks.score[lane];
      }
      __syncwarp();
      for (int n = 0; n < a.top_k; ++n) total = __fadd_rn(total, picks.weight[n]);
      if (lane < a.top_k) {
        my_id[0] = picks.chosen[lane];
        my_w[0] = picks.weight[lane];
      }
      __syncwarp();  // read before the next token's are written
    } else {
      // Many equal ranks, or more than 32 to choose: one after another, the warp's largest
      // rank at its lowest index.
      for (int n = 0; n < a.top_k; ++n) {
        uint32_t most = r[0];
#pragma unroll
        for (int i = 1; i < kVals; ++i) most = max(most, r[i]);
        const uint32_t top = __reduce_max_sync(kFullMask, most);
        uint32_t e = 0xffffffffu;
        if (most == top) {
#pragma unroll
          for (int i = kVals - 1; i >= 0; --i)
            if (r[i] == top) e = 128 * (i >> 2) + 4 * lane + (i & 3);
        }
        const int id = (int)__reduce_min_sync(kFullMask, e);
        float w = 0.0f;
        if ((int)e == id) {
#pragma unroll
          for (int i = 0; i < kVals; ++i)
            if (128 * (i >> 2) + 4 * lane + (i & 3) == id) {
              w = top > none ? s[i] : 0.0f;
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
}

template <typename T>
cudaError_t launch_route(const RouteArgs& a, int sms, cudaStream_t stream) {
  // CTAs for one resident wave at most (8 an SM at 64 registers, two chunks); each takes
  // tokens in turn
  const int64_t ctas = (a.T + kRouteWarps - 1) / kRouteWarps, wave = (int64_t)sms * 8;
  const dim3 grid((unsigned)(ctas < wave ? ctas : wave)), block(kRouteWarps * 32);
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
  DeviceInfo info;
  if (!device_info(&info)) return MEMRA_ERR_CUDA;
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
  // rows (bit 0), the bias (bit 1) four at a time
  a.vec = (E % 4 == 0 && stride_t % 4 == 0 && aligned(logits, 4 * es) ? 1 : 0) |
          (E % 4 == 0 && aligned(bias, 16) ? 2 : 0);
  a.group_magic = (uint32_t)(((1 << 20) + E / n_groups - 1) / (E / n_groups));
  const cudaError_t e = dtype == MEMRA_BF16 ? launch_route<uint16_t>(a, info.sms, stream)
                                            : launch_route<float>(a, info.sms, stream);
  if (e != cudaSuccess) return cuda_fail(e);
  return MEMRA_OK;
}
