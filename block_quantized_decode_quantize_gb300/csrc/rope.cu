// Norm of queries and keys for each head and their rotation by position, in one pass.
//
// n = x * w / sqrt(mean x^2 + eps), then (a, b) -> (a cos - b sin, b cos + a sin).  A head's
// row of D values lies on D / 8 lanes, so the sum of squares takes 3 to 5 exchanges, and each
// lane holds two pieces of four values that are each other's partners in the rotation:
// nothing else passes between lanes, and a row is read and written once.  A warp takes 32 lanes'
// worth of heads (a group) of a set of one, two or four tokens, all of whose loads are on their way
// before the first is worked on.  A CTA's threads compute the R / 2 angles of a token once, for
// all of its heads, and leave cos and sin in shared memory meanwhile.
//
// Angles: F = inv_freq / 2 pi as a fraction of a turn in 64-bit fixed point, and
// position * F modulo 2^64 is the angle of any position, exact to the bits of F.
//
// 8191 tokens of 48 heads of 128 in bf16 (201 MB) take 37.5 us, 79 % of the copy rate: each further
// 2432 tokens (a CTA more for every place on the SMs) take 9.4 us, 94 % of it, so 4 us are the launch, the
// first CTAs' angles and the last stores, and the rest the last, half-filled round of CTAs.  In fp32
// (403 MB) 63.2 us, 94 %; its instances of four tokens with halves spill 4 to 24 bytes.  One
// token takes 2.1 us, as a kernel that does nothing.  Measured and not kept: one token's loads at a
// time (51.7 us), fp64 conversion of the frequencies by every thread (+1 us), two tokens a CTA (48.0), eight (47.4), and 16 bytes to a load (37.0; but 128 tokens of
// interleaved pairs 2.9 -> 3.6, 2000 of them 12.8 -> 13.8).
#include <cuda_bf16.h>

#include "common.cuh"

namespace memra {
namespace {

constexpr int kRopeWarps = 8;
constexpr int kMaxPairs = 128;   // R / 2, at most
constexpr int kMaxSets = 4;     // of four tokens, that a CTA takes

struct Rows {
  void* at;
  int64_t stride_t, stride_h;
  int bf16;
};

struct RopeArgs {
  Rows q, k, q_out, k_out;
  int64_t T;
  int Hq, heads, R, pairs, tokens;
  int sets, groups;  // what a CTA takes: sets of so many tokens, groups of heads
  const float *q_weight, *k_weight;
  float eps;
  const int32_t* positions;
  const double* inv_freq;
  Divider by_pairs, by_groups;
};

// Four values of a row.
template <typename T>
struct Piece;
template <>
struct Piece<float> {
  uint4 u;
  __device__ __forceinline__ void load(const void* p) { u = __ldcg(static_cast<const uint4*>(p)); }
  __device__ __forceinline__ void zero() { u = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void unpack(float2* v) const {
    v[0] = make_float2(__uint_as_float(u.x), __uint_as_float(u.y));
    v[1] = make_float2(__uint_as_float(u.z), __uint_as_float(u.w));
  }
};
template <>
struct Piece<uint16_t> {
  uint2 u;
  __device__ __forceinline__ void load(const void* p) { u = __ldcg(static_cast<const uint2*>(p)); }
  __device__ __forceinline__ void zero() { u = make_uint2(0, 0); }
  __device__ __forceinline__ void unpack(float2* v) const {
    v[0] = make_float2(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u));
    v[1] = make_float2(__uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u));
  }
};

__device__ __forceinline__ uint2 bf16x4(const float2* v) {
  const __nv_bfloat162 a = __float22bfloat162_rn(v[0]), b = __float22bfloat162_rn(v[1]);
  return make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

// The angle's sine and cosine of a position: F is the frequency in turns, 64 bits behind the point.
__device__ __forceinline__ uint64_t turns_of(double inv_freq) {
  double u = inv_freq * 0.15915494309189533577;  // 1 / 2 pi
  u -= floor(u);
  return __double2ull_rn(u * 18446744073709551616.0);
}

template <typename T, int kD, bool kPairs, int kTokens, bool kSets>
__global__ void __launch_bounds__(kRopeWarps * 32, 4) rope_kernel(RopeArgs a) {
  constexpr int kLanes = kD / 8;         // of a head
  constexpr int kHeads = 32 / kLanes;    // that a warp takes at once: a group
  constexpr int kAll = kTokens * (kSets ? kMaxSets : 1);
  __shared__ __align__(16) float cos_of[kAll][kMaxPairs], sin_of[kAll][kMaxPairs];
  __shared__ __align__(16) float weight_of[2][kD];
  __shared__ uint64_t turn_of[kMaxPairs];
  __shared__ int32_t pos_of[kAll];
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t0 = (int64_t)blockIdx.x * (kSets ? a.sets : 1) * kTokens;
  const int tokens = (int)min((int64_t)(kSets ? a.sets : 1) * kTokens, a.T - t0);
  const int end = kSets ? (tokens + kTokens - 1) / kTokens * a.groups
                        : min((int)(blockIdx.y + 1) * a.groups, (a.heads + kHeads - 1) / kHeads);

  // The values that the lane takes of a head: two pieces of four, from off_a and off_b.
  const int l = lane % kLanes;
  const bool turned = l < a.R / 8, halves = turned && !kPairs;
  const int off_a = halves ? 4 * l : 8 * l, off_b = halves ? a.R / 2 + 4 * l : 8 * l + 4;

  const int half = a.R / 2;
  // Weights, and the angles of all tokens: each frequency's conversion, which takes slow fp64
  // instructions, once.
  auto prepare = [&]() {
    for (int i = threadIdx.x; i < 2 * kD; i += kRopeWarps * 32) {
      const float* from = i < kD ? a.q_weight : a.k_weight;
      weight_of[i / kD][i % kD] = from != nullptr ? from[i % kD] : 1.0f;
    }
    if (threadIdx.x < half) turn_of[threadIdx.x] = turns_of(a.inv_freq[threadIdx.x]);
    if (threadIdx.x < kAll)
      pos_of[threadIdx.x] = a.positions != nullptr && threadIdx.x < tokens ? a.positions[t0 + threadIdx.x] : 0;
    __syncthreads();
    for (int i = threadIdx.x; i < tokens * half; i += kRopeWarps * 32) {
      const int t = (int)a.by_pairs((uint32_t)i), j = i - t * half;
      const uint64_t turn = turn_of[j] * (uint64_t)(uint32_t)pos_of[t];
      // the upper 32 bits as half turns in [-1, 1)
      sincospif((float)(int32_t)(uint32_t)(turn >> 32) * 4.6566128730773926e-10f, &sin_of[t][j], &cos_of[t][j]);
    }
    __syncthreads();
  };

  bool first = true;
  for (int i = (kSets ? 0 : blockIdx.y * a.groups) + warp; i < end || first; i += kRopeWarps) {
    const int set = kSets ? (int)a.by_groups((uint32_t)i) : 0, first_t = set * kTokens;
    const int head = (i - set * a.groups) * kHeads + lane / kLanes;
    const bool mine = i < end && head < a.heads, is_q = head < a.Hq;
    const Rows &in = is_q ? a.q : a.k, &out = is_q ? a.q_out : a.k_out;
    const int h = is_q ? head : head - a.Hq;
    // all tokens' values are on their way before the first is worked on
    Piece<T> pa[kTokens], pb[kTokens];
    const T* p = static_cast<const T*>(in.at) + (t0 + first_t) * in.stride_t + h * in.stride_h + off_a;
#pragma unroll
    for (int t = 0; t < kTokens; ++t, p += in.stride_t) {
      pa[t].zero();
      pb[t].zero();
      if (mine && first_t + t < tokens) {
        pa[t].load(p);
        pb[t].load(p + (off_b - off_a));
      }
    }
    if (first) prepare();
    first = false;
    if (i >= end) break;
    const int64_t es = out.bf16 ? 2 : 4, step = out.stride_t * es;
    char* to = static_cast<char*>(out.at) + ((t0 + first_t) * out.stride_t + h * out.stride_h + off_a) * es;
    const int64_t second = (off_b - off_a) * es;
#pragma unroll
    for (int t = 0; t < kTokens; ++t, to += step) {
      float2 v[4];  // off_a's four values, then off_b's
      pa[t].unpack(v);
      pb[t].unpack(v + 2);
      float2 q = __fmul2_rn(v[0], v[0]);
#pragma unroll
      for (int j = 1; j < 4; ++j) q = __ffma2_rn(v[j], v[j], q);
      // (half of the squares with 256 of them: 2^60 in all of these would sum to 2^128)
      constexpr float kPart = kD == 256 ? 0.5f : 1.0f;
      float s = kPart * (q.x + q.y);
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1) s += __shfl_xor_sync(kFullMask, s, o);
      s = fmaf(s, 1.0f / (kPart * kD), a.eps);
      // (2 ulp; without a norm, weights are ones too)
      const float r = a.eps >= 0.0f ? (s == 0.0f ? 0.0f : rsqrtf(s)) : 1.0f;
      const float4 wa = *reinterpret_cast<const float4*>(&weight_of[is_q ? 0 : 1][off_a]);
      const float4 wb = *reinterpret_cast<const float4*>(&weight_of[is_q ? 0 : 1][off_b]);
      const float2 w[4] = {{wa.x, wa.y}, {wa.z, wa.w}, {wb.x, wb.y}, {wb.z, wb.w}};
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = __fmul2_rn(__fmul2_rn(v[j], make_float2(r, r)), w[j]);
      if (turned) {
        const float4 c4 = *reinterpret_cast<const float4*>(&cos_of[first_t + t][4 * l]);
        const float4 s4 = *reinterpret_cast<const float4*>(&sin_of[first_t + t][4 * l]);
        if (kPairs) {
          const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
          for (int j = 0; j < 4; ++j)
            v[j] = __ffma2_rn(make_float2(-v[j].y, v[j].x), make_float2(s[j], s[j]), __fmul2_rn(v[j], make_float2(c[j], c[j])));
        } else {
          const float2 c[2] = {{c4.x, c4.y}, {c4.z, c4.w}}, s[2] = {{s4.x, s4.y}, {s4.z, s4.w}};
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float2 x = v[j], y = v[j + 2];
            v[j] = __ffma2_rn(make_float2(-y.x, -y.y), s[j], __fmul2_rn(x, c[j]));
            v[j + 2] = __ffma2_rn(x, s[j], __fmul2_rn(y, c[j]));
          }
        }
      }
      if (pos_of[first_t + t] < 0) {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = make_float2(0.0f, 0.0f);
      }
      if (mine && first_t + t < tokens) {
        if (out.bf16) {
          *reinterpret_cast<uint2*>(to) = bf16x4(v);
          *reinterpret_cast<uint2*>(to + second) = bf16x4(v + 2);
        } else {
          *reinterpret_cast<float4*>(to) = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
          *reinterpret_cast<float4*>(to + second) = make_float4(v[2].x, v[2].y, v[3].x, v[3].y);
        }
      }
    }
  }
}

template <typename T, int kD>
cudaError_t launch_rope(RopeArgs a, int sms, cudaStream_t stream) {
  constexpr int kHeads = 32 / (kD / 8);
  const int groups = (a.heads + kHeads - 1) / kHeads;
  // One, two or four tokens to a CTA, whose angles keep its threads busy, and all of their heads, so
  // that angles are computed once; but eight groups of heads, one a warp, where that makes fewer
  // than three CTAs an SM (us of 48 heads of 128 in bf16, so and with all heads: 1 token 2.1 and 3.0, 128
  // 3.0 and 3.4, 400 5.0 and 4.6, 1500 9.9 and 11.1; where it makes more, 8191 tokens, 38.8 and 37.3).
  const int64_t spread = a.T / (2 * (int64_t)sms);
  a.tokens = spread < 2 ? 1 : (spread < 4 ? 2 : 4);
  a.groups = (a.T + a.tokens - 1) / a.tokens < 3 * (int64_t)sms && groups > kRopeWarps ? kRopeWarps : groups;
  a.by_pairs = Divider((uint32_t)(a.R > 0 ? a.R / 2 : 1));
  a.by_groups = Divider((uint32_t)a.groups);
  // Few heads, or a number of groups that leaves warps idle: two or four sets of four tokens to a
  // CTA where that leaves fewer idle, with two CTAs an SM at least (8000 tokens of 2 heads of 128
  // 4.8 us for 9.6, of 24 of 64 12.7 for 14.1; four CTAs an SM at least 6.5 and 14.2).
  a.sets = 1;
  const auto idle = [&](int sets) { return (sets * a.groups + kRopeWarps - 1) / kRopeWarps * (kMaxSets / sets); };
  for (int sets = 2; sets <= kMaxSets && a.tokens == 4 && a.groups == groups; sets *= 2)
    if (idle(sets) < idle(a.sets) && a.T >= sets * 4 * 2 * (int64_t)sms) a.sets = sets;
  const int of_cta = a.sets * a.tokens;
  const dim3 grid((unsigned)((a.T + of_cta - 1) / of_cta), (unsigned)((groups + a.groups - 1) / a.groups));
  const auto run = [&](void (*pairs)(RopeArgs), void (*halves)(RopeArgs)) {
    return launch_kernel(a.pairs ? pairs : halves, grid, dim3(kRopeWarps * 32), 0, stream, a);
  };
  if (a.tokens == 1) return run(rope_kernel<T, kD, true, 1, false>, rope_kernel<T, kD, false, 1, false>);
  if (a.tokens == 2) return run(rope_kernel<T, kD, true, 2, false>, rope_kernel<T, kD, false, 2, false>);
  if (a.sets == 1) return run(rope_kernel<T, kD, true, 4, false>, rope_kernel<T, kD, false, 4, false>);
  return run(rope_kernel<T, kD, true, 4, true>, rope_kernel<T, kD, false, 4, true>);
}

template <typename T>
cudaError_t launch_rope(const RopeArgs& a, int64_t D, int sms, cudaStream_t stream) {
  if (D == 64) return launch_rope<T, 64>(a, sms, stream);
  if (D == 128) return launch_rope<T, 128>(a, sms, stream);
  return launch_rope<T, 256>(a, sms, stream);
}

// Whether no two rows that are written share a value: heads side by side within a token's row,
// or tokens side by side within a head's.
bool apart(const Rows& r, int64_t T, int64_t H, int64_t D) {
  if (T == 0 || H == 0) return true;
  if (T == 1) return H == 1 || r.stride_h >= D;
  if (H == 1) return r.stride_t >= D;
  return (r.stride_h >= D && r.stride_t >= (H - 1) * r.stride_h + D) ||
         (r.stride_t >= D && r.stride_h >= (T - 1) * r.stride_t + D);
}

// Bytes that rows of heads take: from `at`, T rows `row` bytes apart whose heads lie within `width`.
struct Extent {
  uintptr_t at;
  uint64_t row, width, all;
  Extent(const Rows& r, int64_t T, int64_t H, int64_t D) : at((uintptr_t)r.at), row(0), width(0), all(0) {
    if (T == 0 || H == 0) return;
    const uint64_t es = r.bf16 ? 2 : 4;
    row = (uint64_t)r.stride_t * es;
    width = ((uint64_t)(H - 1) * r.stride_h + D) * es;
    all = (uint64_t)(T - 1) * row + width;
  }
  Extent(const void* p, uint64_t bytes) : at((uintptr_t)p), row(0), width(bytes), all(p != nullptr ? bytes : 0) {}
  bool meets(const Extent& o) const {
    if (all == 0 || o.all == 0 || at >= o.at + o.all || o.at >= at + all) return false;
    if (row == 0 || row != o.row || width > row || o.width > row) return true;
    // rows side by side: where the other's begin, seen from this one's, modulo a row
    const uint64_t d = o.at >= at ? (o.at - at) % row : (row - (at - o.at) % row) % row;
    return d < width || d + o.width > row;
  }
};

}  // namespace
}  // namespace memra

using namespace memra;

extern "C" memra_status memra_qk_norm_rope(
    const void* q, const void* k, int32_t dtype, int64_t T, int64_t Hq, int64_t Hkv, int64_t D,
    int64_t q_stride_t, int64_t q_stride_h, int64_t k_stride_t, int64_t k_stride_h,
    const float* q_weight, const float* k_weight, float eps, const int32_t* positions,
    const double* inv_freq, int64_t R, int32_t layout, void* q_out, int32_t q_out_dtype,
    int64_t q_out_stride_t, int64_t q_out_stride_h, void* k_out, int32_t k_out_dtype,
    int64_t k_out_stride_t, int64_t k_out_stride_h, cudaStream_t stream) {
  if (T < 0 || Hq < 0 || Hkv < 0 || R < 0 || R % 8 != 0) return MEMRA_ERR_INVALID_ARG;
  for (const int32_t t : {dtype, q_out_dtype, k_out_dtype})
    if (t != MEMRA_BF16 && t != MEMRA_F32) return MEMRA_ERR_INVALID_ARG;
  for (const int64_t s : {q_stride_t, q_stride_h, k_stride_t, k_stride_h, q_out_stride_t,
                          q_out_stride_h, k_out_stride_t, k_out_stride_h})
    if (s < 0) return MEMRA_ERR_INVALID_ARG;
  if (layout != MEMRA_ROPE_HALVES && layout != MEMRA_ROPE_PAIRS) return MEMRA_ERR_INVALID_ARG;
  if (!(eps >= 0.0f || eps < 0.0f) || eps > 3e38f) return MEMRA_ERR_INVALID_ARG;
  if (eps < 0.0f && (q_weight || k_weight)) return MEMRA_ERR_INVALID_ARG;
  if (D != 64 && D != 128 && D != 256) return MEMRA_ERR_UNSUPPORTED;
  if (R > D) return MEMRA_ERR_INVALID_ARG;
  if (T > INT32_MAX || Hq > 65535 || Hkv > 65535 || Hq + Hkv > 65535) return MEMRA_ERR_UNSUPPORTED;
  // every offset in bytes stays far inside an int64
  for (const int64_t s : {q_stride_t, k_stride_t, q_out_stride_t, k_out_stride_t})
    if (s > ((int64_t)1 << 56) / (T + 1)) return MEMRA_ERR_UNSUPPORTED;
  for (const int64_t s : {q_stride_h, k_stride_h, q_out_stride_h, k_out_stride_h})
    if (s > ((int64_t)1 << 56) / 65536) return MEMRA_ERR_UNSUPPORTED;
  if (T == 0 || Hq + Hkv == 0) return MEMRA_OK;
  if ((Hq > 0 && (!q || !q_out)) || (Hkv > 0 && (!k || !k_out))) return MEMRA_ERR_INVALID_ARG;
  if (R > 0 && (!positions || !inv_freq)) return MEMRA_ERR_INVALID_ARG;
  RopeArgs a;
  a.q = {const_cast<void*>(q), q_stride_t, q_stride_h, dtype == MEMRA_BF16};
  a.k = {const_cast<void*>(k), k_stride_t, k_stride_h, dtype == MEMRA_BF16};
  a.q_out = {q_out, q_out_stride_t, q_out_stride_h, q_out_dtype == MEMRA_BF16};
  a.k_out = {k_out, k_out_stride_t, k_out_stride_h, k_out_dtype == MEMRA_BF16};
  const Rows* rows[] = {&a.q, &a.k, &a.q_out, &a.k_out};
  const int64_t heads[] = {Hq, Hkv, Hq, Hkv};
  for (int i = 0; i < 4; ++i) {
    const int64_t per16 = rows[i]->bf16 ? 8 : 4;
    if (heads[i] > 0 && (!aligned(rows[i]->at, 16) || rows[i]->stride_t % per16 != 0 || rows[i]->stride_h % per16 != 0))
      return MEMRA_ERR_ALIGNMENT;
  }
  if (!aligned(q_weight, 4) || !aligned(k_weight, 4) || !aligned(positions, 4) || !aligned(inv_freq, 8))
    return MEMRA_ERR_ALIGNMENT;
  if (!apart(a.q_out, T, Hq, D) || !apart(a.k_out, T, Hkv, D)) return MEMRA_ERR_INVALID_ARG;
  const Extent in[] = {Extent(a.q, T, Hq, D), Extent(a.k, T, Hkv, D), Extent(q_weight, 4 * D), Extent(k_weight, 4 * D),
                       Extent(positions, 4 * T), Extent(inv_freq, 4 * R)};
  const Extent out[] = {Extent(a.q_out, T, Hq, D), Extent(a.k_out, T, Hkv, D)};
  for (int i = 0; i < 2; ++i) {
    for (int j = 0; j < 6; ++j) {
      const Rows &x = *rows[i], &y = *rows[2 + i];
      const bool in_place = i == j && x.at == y.at && x.stride_t == y.stride_t && x.stride_h == y.stride_h && x.bf16 == y.bf16;
      if (!in_place && out[i].meets(in[j])) return MEMRA_ERR_INVALID_ARG;
    }
  }
  if (out[0].meets(out[1])) return MEMRA_ERR_INVALID_ARG;
  DeviceInfo info;
  if (!device_info(&info)) return MEMRA_ERR_CUDA;
  a.T = T;
  a.Hq = (int)Hq;
  a.heads = (int)(Hq + Hkv);
  a.R = (int)R;
  a.pairs = layout == MEMRA_ROPE_PAIRS;
  a.q_weight = q_weight;
  a.k_weight = k_weight;
  a.eps = eps;
  a.positions = positions;
  a.inv_freq = inv_freq;
  const cudaError_t e = dtype == MEMRA_BF16 ? launch_rope<uint16_t>(a, D, info.sms, stream)
                                            : launch_rope<float>(a, D, info.sms, stream);
  if (e != cudaSuccess) return cuda_fail(e);
  return MEMRA_OK;
}
