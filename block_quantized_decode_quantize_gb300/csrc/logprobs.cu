// Log probabilities of tokens from a row of logits, its entropy and its largest entries.
//
// One pass over the logits.  Each lane sums z = sum 2^u and s = sum 2^u u over its elements, with
// u = x log2 e - M, M a whole number next to the maximum of its warp's first blocks, so that u is
// one rounding and the sums of other warps differ by a power of two.  What exceeds that maximum
// makes terms above 1, which fp32 holds up to 2^127; a warp whose sums are not finite, or whose
// maximum lies more than 2^60 above, takes its blocks again, with care.  The row is cut into
// segments whose maxima go to shared memory as the pass goes by.
//
// Then the row's sums are joined, and a number is found that the maxima of top_n groups of
// segments reach, a bound that top_n elements reach: only segments whose maximum reaches it are
// read again (from L2), and the few elements at or above it are ranked by counting.  Relative to
// its largest term, Z is 1 + rest.  Where the rest is below a quarter, the elements of the lane
// that met the largest are summed again without it, so that ln Z = log1p(rest) keeps the digits
// of log probabilities near 0.
//
// A row is taken by one CTA, or, with few rows, by the CTAs of a cluster, which leave maxima and
// sums in the first one's shared memory.
//
// A masked token (-inf, NaN) is found at the end of a warp's share, or in its first batch, and the
// share is then summed again with a clamp: with a few of them in a row, most of it is read twice.
//
// 2047 rows of 151,936 bf16 logits (622 MB) take 106 us, 87 % of the copy rate: memory, with 0.54
// instructions a cycle beside it (about 6.5 for 32 elements, the exponential's unit 40 % busy) and
// 5 us of choosing (with 1, 16 and 152 masked tokens a row 151, 194 and 164 us, with half of them 114);
// 640 rows in fp32 (389 MB) 66.8 us, 86 %.  All instances take 64 registers, the most that 1024 threads
// an SM leave, and spill 12 to 28 bytes.  One row takes 7.4 us: launch 2.1, the read
// and sums 3.2, the choice 2.1, each a chain of latencies.  Measured and not kept: rescaling sums
// at every new maximum and keeping it out of them (14 instructions an element, 123 to 169 us);
// asynchronous copies into a ring of each warp, with the next row's on their way (142 to 198: the
// ring's own instructions and registers); a second launch for the choice (149 to 196: it reads
// from DRAM again what L2 no longer holds); maxima stored to the first CTA block by block
// (addresses of another CTA's memory take four more instructions each).
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include <type_traits>

#include "common.cuh"

namespace memra {
namespace {

namespace cg = cooperative_groups;

constexpr int kBlock = 256;         // elements a warp looks at together: 8 a lane
constexpr int kMost = 512;          // candidates that are ranked by counting
constexpr int kFineBytes = 65536;   // of a row with fine segments, at most
constexpr int kMaxWarps = 256;      // of a row: 16 CTAs of 16 (of smaller CTAs, one has a row)
constexpr float kLog2e = 1.44269504088896341f, kLn2 = 0.693147180559945309f;
constexpr float kLargest = 3.402823466e38f;
constexpr float kFloor = -160.0f;   // 2^u is 0 in fp32 below
constexpr float kRise = 60.0f;      // of a share's largest term over what its sums refer to, log2

struct alignas(16) Part {  // of a warp
  float m, of;        // its maximum, and what its sums refer to: Reference(of)
  float z, s;         // of all lanes but one
  float z_lane, s_lane;
  int lane;           // that one, which has met m
  int pad;
};

struct LogprobArgs {
  const void* logits;
  int64_t T, stride_t;
  int V, top_n;
  int segments;             // of a row, at most
  bool fine;                // they are pieces of 16 bytes
  const int32_t* tokens;
  float *logprobs, *entropy, *top_logprobs;
  int32_t *top_ids, *status;
};

__device__ __forceinline__ float inf() { return __int_as_float(0x7f800000); }

__device__ __forceinline__ float warp_max(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Bits of v in an order that compares as unsigned (-0 as 0); -inf is the lowest number's.
__device__ __forceinline__ uint32_t order_of(float v) {
  const uint32_t u = __float_as_uint(v + 0.0f);
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t r) {
  return __uint_as_float((r & 0x80000000u) ? (r & 0x7fffffffu) : ~r);
}

// A masked token's logit is -inf or no number; +inf counts as the largest finite value.
__device__ __forceinline__ float sane(float v) { return fminf(fmaxf(v, -inf()), kLargest); }

// A load of the one pass; kOnce: of what will hardly be read again.  Its lines are not put into L1, and
// volatile statements keep their order; which of the two makes the rows of 151,936 logits 2 to 4 % faster
// was not told apart (volatile was needed).
template <bool kOnce>
__device__ __forceinline__ uint4 load(const uint4* p) {
  if (!kOnce) return __ldcg(p);
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
  return r;
}

template <typename T>
__device__ __forceinline__ float element(const T* p);
template <>
__device__ __forceinline__ float element<float>(const float* p) { return *p; }
template <>
__device__ __forceinline__ float element<uint16_t>(const uint16_t* p) { return __uint_as_float((uint32_t)*p << 16); }

// An address in the shared memory of the cluster's first CTA, and a store there.
__device__ __forceinline__ uint32_t mapped(const void* p) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(smem_addr(p)));
  return r;
}
__device__ __forceinline__ void put(uint32_t at, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at), "f"(v) : "memory");
}

// A row seen from the 16-byte boundary at or before it: element i of the row is place
// i + shift, and block b holds places 256 b ..  A lane's 8 of them: bf16 16 bytes, fp32 twice
// 16 bytes, 512 apart.
template <typename T>
struct Row {
  const T* base;   // place 0
  int shift, end;  // places of the row: shift .. end - 1
  static constexpr bool kWide = sizeof(T) == 4;
  static constexpr int kPieces = kWide ? 2 : 1, kPer = 8 / kPieces;  // 16 bytes each
  __device__ __forceinline__ Row(const T* p, int V) {
    shift = (int)(((uintptr_t)p & 15) / sizeof(T));
    base = p - shift;
    end = V + shift;
  }
  __device__ __forceinline__ int blocks() const { return (end + kBlock - 1) / kBlock; }
  // blocks that lie within the row: first_whole .. end_whole - 1
  __device__ __forceinline__ int first_whole() const { return shift > 0 ? 1 : 0; }
  __device__ __forceinline__ int end_whole() const { return end / kBlock; }
  // place of the lane's value i of a block
  static __device__ __forceinline__ int place(int b, int lane, int i) {
    return b * kBlock + (kWide ? 4 * lane + (i & 3) + 32 * (i & 4) : 8 * lane + i);
  }
  __device__ __forceinline__ const uint4* at(int b, int lane) const {
    return reinterpret_cast<const uint4*>(base + (int64_t)b * kBlock) + lane;
  }
  struct Raw {
    uint4 u[kPieces];
  };
  __device__ __forceinline__ Raw fetch_whole(int b, int lane) const {
    Raw r;
#pragma unroll
    for (int h = 0; h < kPieces; ++h) r.u[h] = __ldcg(at(b, lane) + 32 * h);
    return r;
  }
  // any block's values, -inf for places outside the row
  __device__ __forceinline__ Raw fetch(int b, int lane) const {
    if (b >= first_whole() && b < end_whole()) return fetch_whole(b, lane);
    Raw r;
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int p = place(b, lane, i);
      w[i] = __float_as_uint(p >= shift && p < end ? element<T>(base + p) : -inf());
    }
    if (kWide) {
      r.u[0] = make_uint4(w[0], w[1], w[2], w[3]);
      r.u[kPieces - 1] = make_uint4(w[4], w[5], w[6], w[7]);
    } else {
      r.u[0] = make_uint4((w[0] >> 16) | w[1], (w[2] >> 16) | w[3], (w[4] >> 16) | w[5], (w[6] >> 16) | w[7]);
    }
    return r;
  }
  static __device__ __forceinline__ void unpack(const Raw& r, float* v) {
#pragma unroll
    for (int h = 0; h < kPieces; ++h) {
      const uint32_t w[4] = {r.u[h].x, r.u[h].y, r.u[h].z, r.u[h].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (kWide) {
          v[4 * h + i] = __uint_as_float(w[i]);
        } else {
          v[2 * i] = __uint_as_float(w[i] << 16);
          v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
      }
    }
  }
  // the largest of 16 bytes' values, exactly (NaN only where nothing else is there)
  static __device__ __forceinline__ float largest_of(const uint4& u) {
    if (kWide) return fmaxf(fmaxf(__uint_as_float(u.x), __uint_as_float(u.y)), fmaxf(__uint_as_float(u.z), __uint_as_float(u.w)));
    const uint32_t m = most2(most2(u.x, u.y), most2(u.z, u.w));
    return fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
  }
  static __device__ __forceinline__ float largest(const Raw& r) {
    return kWide ? fmaxf(largest_of(r.u[0]), largest_of(r.u[kPieces - 1])) : largest_of(r.u[0]);
  }
  static __device__ __forceinline__ uint32_t most2(uint32_t a, uint32_t b) {
    const __nv_bfloat162 x = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&x);
  }
};

// What a maximum's sums refer to: 2^(m log2 e - delta), m log2 e - delta a whole number M, or
// m log2 e itself (delta 0) where that is too large to have neighbours next to it.
struct Reference {
  float m, delta, M;
  bool far;
  __device__ __forceinline__ explicit Reference(float max) : m(max) {
    far = !(fabsf(m) < 1048576.0f);
    M = ceilf(m * kLog2e);
    delta = far ? 0.0f : fmaf(m, kLog2e, -M);
  }
  // log2 of x's term; clamped where it is 0
  __device__ __forceinline__ float term(float x) const {
    return fmaxf(far ? (x - m) * kLog2e : fmaf(x, kLog2e, -M), kFloor);
  }
  // log2 of what relates sums of another reference to this one
  __device__ __forceinline__ float from(const Reference& o) const {
    return fmaxf(far || o.far ? (o.m - m) * kLog2e - o.delta + delta : o.M - M, kFloor);
  }
};

// The lane's part of a warp's sums, in two halves.
struct Sums {
  float2 z = {0.0f, 0.0f}, s = {0.0f, 0.0f};
  // 8 values, M as in Reference.  What is infinite, no number or too large to be a term makes s no
  // finite number; with kClamp, only what is too large does.
  template <bool kClamp>
  __device__ __forceinline__ void add(const float* v, float M) {
    const float2 minus = {-M, -M}, scale = {kLog2e, kLog2e};
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      float2 u = __ffma2_rn(make_float2(v[i], v[i + 1]), scale, minus);
      if (kClamp) u = make_float2(fmaxf(u.x, kFloor), fmaxf(u.y, kFloor));
      const float2 e = {exp2_approx(u.x), exp2_approx(u.y)};
      z = __fadd2_rn(z, e);
      s = __ffma2_rn(e, u, s);
    }
  }
  __device__ __forceinline__ void add_one(float u) {
    const float e = exp2_approx(u);
    z.x += e;
    s.x = fmaf(e, u, s.x);
  }
  __device__ __forceinline__ bool sound() const { return fabsf(s.x + s.y) < inf(); }
};

// The bound: a number that the maxima of top_n segments reach, by bisection between the least
// and the largest of the maxima of 128 groups of segments, until at most 1.25 top_n + 1 of
// these reach it: of the values, a few steps for logits as they are, and of their bits, which
// ends for any.  -inf: fewer than top_n groups have a token left.
__device__ __forceinline__ float bound_of(const float* seg_max, int segments, int top_n, int lane) {
  float g[4] = {-inf(), -inf(), -inf(), -inf()};
  for (int i = lane; i < segments; i += 128) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (i + 32 * j < segments) g[j] = fmaxf(g[j], seg_max[i + 32 * j]);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) g[j] = sane(g[j]);  // what equals +inf may lie in segments without one
  float least = inf(), over = -inf();
  int numbers = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (g[j] == -inf()) continue;
    least = fminf(least, g[j]);
    over = fmaxf(over, g[j]);
    ++numbers;
  }
  if ((int)__reduce_add_sync(kFullMask, numbers) < top_n) return -inf();
  float bound = -warp_max(-least);
  over = warp_max(over);
  for (int n = 0; n < 44; ++n) {
    const uint32_t lo = order_of(bound), hi = order_of(over);
    const float mid = n < 12 ? 0.5f * bound + 0.5f * over : value_of(lo + (hi - lo) / 2);
    if (!(mid > bound && mid < over)) {
      if (n < 12) continue;
      break;
    }
    int reach = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) reach += g[j] >= mid ? 1 : 0;
    reach = (int)__reduce_add_sync(kFullMask, reach);
    if (reach < top_n) {
      over = mid;
    } else {
      bound = mid;
      if (4 * reach <= 5 * top_n + 4) break;
    }
  }
  return bound;
}

// Which blocks a warp takes: the whole ones, kAhead neighbours (a batch) at a time, batch after
// batch in turn with the other warps; those that are left at the ends one by one, the last warps
// first.
template <typename T>
struct Share {
  static constexpr int kAhead = sizeof(T) == 4 ? 2 : 4;  // 64 bytes a lane
  int f, batches, mine, left, first_left, warp, warps;
  __device__ __forceinline__ Share(const Row<T>& row, int w, int n) : warp(w), warps(n) {
    f = row.first_whole();
    batches = max(row.end_whole() - f, 0) / kAhead;
    mine = batches > w ? (batches - w - 1) / n + 1 : 0;
    const int all_left = row.blocks() - kAhead * batches;
    first_left = n - 1 - w;
    left = all_left > first_left ? (all_left - first_left - 1) / n + 1 : 0;
  }
  __device__ __forceinline__ int count() const { return mine * kAhead + left; }
  __device__ __forceinline__ int block(int i) const {  // the warp's i-th
    if (i < mine * kAhead) return f + kAhead * (warp + i / kAhead * warps) + i % kAhead;
    const int e = first_left + (i - mine * kAhead) * warps;
    return e < f ? 0 : kAhead * batches + e;
  }
};

// The batches of a warp's share.  Two are under way: one arrives while the other is summed.
template <typename T, bool kOnce, bool kClamp>
__device__ __forceinline__ void sum_batches(const LogprobArgs& a, const Row<T>& row, const Share<T>& share, int lane, bool fine, float* seg_max,
                                            Sums& sums, float& of, float& lane_top) {
  using R = Row<T>;
  constexpr int kAhead = Share<T>::kAhead;
  typename R::Raw raw[kAhead], next[kAhead];
  const uint4* p = row.at(share.f + kAhead * share.warp, lane);
  const int64_t step = share.warps * (kAhead * R::kPieces * 32);
  float M = 0.0f;
  auto fetch = [&](typename R::Raw* r) {
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
#pragma unroll
      for (int h = 0; h < R::kPieces; ++h) r[j].u[h] = load<kOnce>(p + (j * R::kPieces + h) * 32);
    p += step;
  };
  auto add = [&](const typename R::Raw* r, int i) {
    float block_most[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const float mine = R::largest(r[j]);
      lane_top = fmaxf(lane_top, mine);
      block_most[j] = warp_max(mine);
    }
    const int b0 = share.f + kAhead * (share.warp + i * share.warps);
    if (fine) {
#pragma unroll
      for (int j = 0; j < kAhead; ++j)
#pragma unroll
        for (int h = 0; h < R::kPieces; ++h) seg_max[((b0 + j) * R::kPieces + h) * 32 + lane] = R::largest_of(r[j].u[h]);
    } else if (a.top_n > 0) {
      float v = block_most[0];
#pragma unroll
      for (int j = 1; j < kAhead; ++j) v = lane == j ? block_most[j] : v;
      if (lane < kAhead) seg_max[b0 + lane] = v;
    }
    // Sums refer to the first batch that has a token left: batches without one add nothing with the
    // clamp (M is -inf there, u no number), and without it make sums that are not finite.
    if (kClamp || i == 0) {
      float most = block_most[0];
#pragma unroll
      for (int j = 1; j < kAhead; ++j) most = fmaxf(most, block_most[j]);
      if (kClamp) of = of == -inf() ? sane(most) : of;
      else of = fabsf(most) < inf() ? most : 0.0f;
      M = Reference(of).M;
    }
    // a batch's terms among themselves first, so that long sums of small terms lose less
    Sums part;
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      float x[8];
      R::unpack(r[j], x);
      part.template add<kClamp>(x, M);
    }
    sums.z = __fadd2_rn(sums.z, part.z);
    sums.s = __fadd2_rn(sums.s, part.s);
  };
  fetch(raw);
#pragma unroll 1
  for (int i = 0; i < share.mine; i += 2) {
    if (i + 1 < share.mine) fetch(next);
    add(raw, i);
    if (!kClamp && i == 0 && __any_sync(kFullMask, !sums.sound())) return;  // masked tokens
    if (i + 1 == share.mine) break;
    if (i + 2 < share.mine) fetch(raw);
    add(next, i + 1);
  }
}

// The warp's share of a row: its sums, and its segments' maxima.
template <typename T, bool kOnce>
__device__ __forceinline__ Part sum_share(const LogprobArgs& a, const Row<T>& row, int warp, int warps, int lane, bool fine, float* seg_max) {
  using R = Row<T>;
  constexpr int kAhead = Share<T>::kAhead;
  const Share<T> share(row, warp, warps);
  float lane_top = -inf(), top = -inf(), of = -inf();
  Sums sums;
  // Whether the sums are what they should be: finite, and of terms that are not too small.  What they
  // refer to is an element of the share, so the largest does not lie below it.  It may lie 2^kRise
  // above: with the row's largest 2^d above the share's, the join multiplies sums by
  // 2^-(kRise + d), which fp32 holds (to 2^-149) for d up to 89, and so 60 below the largest logit.
  auto good = [&]() {
    const Reference ref(of);
    top = warp_max(sane(lane_top));
    return (top == -inf() || (!ref.far && fmaf(top, kLog2e, -ref.M) <= kRise)) && __all_sync(kFullMask, sums.sound());
  };
  if (share.mine > 0) {
    sum_batches<T, kOnce, false>(a, row, share, lane, fine, seg_max, sums, of, lane_top);
    if (!good()) {
      sums = Sums();
      of = -inf();
      sum_batches<T, kOnce, true>(a, row, share, lane, fine, seg_max, sums, of, lane_top);
    }
  }
  // One block after another: those at the ends; and where sums have nothing to refer to yet, or the
  // quick ones did not take a value, first for the maximum, then for the sums.
  const int count = share.count();
  const int ends = share.mine * kAhead, start = of == -inf() ? ends : 0;  // (there are no batches, or no token is left in them)
  enum { kEnds, kMaximum, kAll } pass = of == -inf() ? kMaximum : kEnds;
  for (;;) {
    const Reference ref(pass == kMaximum ? -inf() : of);
    if (pass != kEnds) {
      sums = Sums();
      lane_top = -inf();
    }
#pragma unroll 1
    for (int i = pass == kEnds ? ends : start; i < count; ++i) {
      const int b = share.block(i);
      const typename R::Raw raw = row.fetch(b, lane);
      const float mine = R::largest(raw);
      lane_top = fmaxf(lane_top, mine);
      if (fine) {
#pragma unroll
        for (int h = 0; h < R::kPieces; ++h) seg_max[(b * R::kPieces + h) * 32 + lane] = R::largest_of(raw.u[h]);
      } else if (a.top_n > 0) {
        const float most = warp_max(mine);
        if (lane == 0) seg_max[b] = most;
      }
      if (pass != kMaximum) {
        float v[8];
        R::unpack(raw, v);
#pragma unroll
        for (int k = 0; k < 8; ++k) sums.add_one(ref.term(sane(v[k])));
      }
    }
    const bool done = good();
    if (pass == kAll || (pass == kEnds && done)) break;
    if (pass == kMaximum) {
      of = top;
      if (of == -inf()) break;
      pass = kAll;
    } else {
      pass = kMaximum;
    }
  }
  Part part;
  part.m = top;
  part.of = of;
  part.lane = __ffs(__ballot_sync(kFullMask, sane(lane_top) == top)) - 1;
  float z = sums.z.x + sums.z.y, s = sums.s.x + sums.s.y;
  part.z_lane = __shfl_sync(kFullMask, z, part.lane);
  part.s_lane = __shfl_sync(kFullMask, s, part.lane);
  if (lane == part.lane) z = s = 0.0f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    z += __shfl_xor_sync(kFullMask, z, o);
    s += __shfl_xor_sync(kFullMask, s, o);
  }
  part.z = z;
  part.s = s;
  part.pad = 0;
  return part;
}

template <int kParts>
struct Shared {
  Part part[kParts];
  unsigned long long candidate[kMost];
  int count;
  float bound, top, log_z;
  uint32_t taken[MEMRA_MAX_TOP_LOGPROBS];
};

template <typename T, int kThreads, bool kOnce>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads) logprob_kernel(LogprobArgs a) {
  constexpr int kWarps = kThreads / 32;
  using R = Row<T>;
  extern __shared__ float seg_max[];  // the row's first CTA
  __shared__ Shared<kThreads == 512 ? kMaxWarps : kWarps> sh;
  pdl_launch_dependents();
  cg::cluster_group cluster = cg::this_cluster();
  const int ranks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  // so that the row's first CTA has begun, and its shared memory can be written, when sums are done
  if (ranks > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int warps = ranks * kWarps, my_warp = warp * ranks + rank;
  const int64_t t = blockIdx.x / ranks;
  const R row(static_cast<const T*>(a.logits) + t * a.stride_t, a.V);
  // Segments: blocks, or, where these are too few to tell top_n elements apart, pieces of 16 bytes.
  const bool fine = a.fine;
  const int blocks = row.blocks(), segments = fine ? blocks * 32 * R::kPieces : blocks;
  if (threadIdx.x == 0) sh.count = 0;
  pdl_wait();
  const int32_t token = a.logprobs != nullptr && threadIdx.x == 0 && rank == 0 ? a.tokens[t] : -1;
  const Part mine = sum_share<T, kOnce>(a, row, my_warp, warps, lane, fine, seg_max);
  const bool known = token >= 0 && token < a.V;
  const float token_x = known ? element<T>(row.base + row.shift + token) : -inf();
  if (ranks == 1) {
    if (lane == 0) sh.part[my_warp] = mine;
    __syncthreads();
  } else {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    const float words[8] = {mine.m, mine.of, mine.z, mine.s, mine.z_lane, mine.s_lane, __int_as_float(mine.lane), 0.0f};
    const uint32_t at = mapped(&sh.part[my_warp]);
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (lane == i) put(at + 4 * i, words[i]);
    if (a.top_n > 0 && rank != 0) {
      const Share<T> share(row, my_warp, warps);
      const int per = fine ? 32 * R::kPieces : 1, count = share.count() * per;  // per: segments of a block
      __syncwarp();
      for (int i = lane; i < count; i += 32) {
        const int seg = share.block(i / per) * per + i % per;
        put(mapped(seg_max + seg), seg_max[seg]);
      }
    }
    cluster.sync();
    if (rank != 0) return;
  }

  // ---- the row's first CTA ----
  if (warp == 0) {
    float top = -inf();
    int special = 0x7fffffff;
    for (int i = lane; i < warps; i += 32)
      if (sh.part[i].m > top) {
        top = sh.part[i].m;
        special = i;
      }
    const float most = warp_max(top);
    special = __reduce_min_sync(kFullMask, top == most ? special : 0x7fffffff);
    top = most;
    const Reference ref(top);
    const float largest = exp2f(ref.delta);  // the largest element's term
    float z = 0.0f, s = 0.0f, z_lane = 0.0f, s_lane = 0.0f;
    for (int i = lane; i < warps; i += 32) {
      const Part& p = sh.part[i];
      if (p.m == -inf()) continue;
      const float up = ref.from(Reference(p.of)), e = exp2f(up);
      z = fmaf(e, p.z, z);
      s = fmaf(e, fmaf(up, p.z, p.s), s);
      const float zl = e * p.z_lane, sl = e * fmaf(up, p.z_lane, p.s_lane);
      if (i == special) {
        z_lane = zl;
        s_lane = sl;
      } else {
        z += zl;
        s += sl;
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      z += __shfl_xor_sync(kFullMask, z, o);
      s += __shfl_xor_sync(kFullMask, s, o);
      z_lane += __shfl_xor_sync(kFullMask, z_lane, o);
      s_lane += __shfl_xor_sync(kFullMask, s_lane, o);
    }
    const bool again = top > -inf() && !(z + z_lane - largest >= 0.25f * largest);
    if (again) {
      // the elements of the lane that met the largest, without it
      const Share<T> share(row, special, warps);
      const int its_lane = sh.part[special].lane;
      Sums sums;
      int equals = 0;
      for (int i = lane; i < share.count(); i += 32) {
        float v[8];
        R::unpack(row.fetch(share.block(i), its_lane), v);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float x = sane(v[k]);
          equals += x == top ? 1 : 0;
          sums.add_one(x == top ? kFloor : ref.term(x));
        }
      }
      z_lane = sums.z.x;
      s_lane = sums.s.x;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        z_lane += __shfl_xor_sync(kFullMask, z_lane, o);
        s_lane += __shfl_xor_sync(kFullMask, s_lane, o);
      }
      const float others = (float)((int)__reduce_add_sync(kFullMask, equals) - 1) * largest;
      z += z_lane + others;
      s += s_lane + others * ref.delta;
    } else {
      z += z_lane - largest;
      s += s_lane - largest * ref.delta;
    }
    if (lane == 0) {
      // relative to the largest element
      const float up = exp2f(-ref.delta), log_z = log1pf(up * z);
      const bool none_left = top == -inf();
      sh.top = top;
      sh.log_z = log_z;
      if (a.entropy != nullptr) {
        const float terms = kLn2 * up * (s - ref.delta * z);
        a.entropy[t] = none_left ? 0.0f : log_z - terms / (1.0f + up * z);
      }
      if (a.logprobs != nullptr) {
        float lp = -inf();
        if (known) {
          if (!none_left) lp = (sane(token_x) - top) - log_z;
        } else if (token == -1) {
          lp = 0.0f;
        } else if (a.status != nullptr) {
          atomicOr(a.status, 1);
        }
        a.logprobs[t] = lp;
      }
    }
  }
  if (a.top_n == 0) return;
  if (warp != 0) {
    constexpr int kLook = kWarps - 1;  // warps that look through the row again
    if (warp == 1) {
      const float b = bound_of(seg_max, segments, a.top_n, lane);
      if (lane == 0) sh.bound = b;
    }
    asm volatile("barrier.sync 1, %0;" ::"n"(kThreads - 32) : "memory");
    // Segments that reach the bound are read again, and their elements that do so become candidates.
    const float bound = fmaxf(sh.bound, -kLargest);  // (what is -inf or no number reaches no bound)
    const int f = row.first_whole();
    auto take = [&](float v, int at) {
      const int n = atomicAdd(&sh.count, 1);
      if (n < kMost) sh.candidate[n] = ((unsigned long long)order_of(sane(v)) << 32) | (uint32_t)~(uint32_t)(at - row.shift);
    };
    // kN values that reach the bound or not; place_of: where the j-th lies
    auto consider = [&](const auto& v, auto n, auto place_of) {
      constexpr int kN = decltype(n)::value;
      uint32_t reach = 0;
#pragma unroll
      for (int j = 0; j < kN; ++j) reach |= v[j] >= bound ? 1u << j : 0u;
#pragma unroll 1
      for (; reach != 0; reach &= reach - 1) {
        const int j = __ffs(reach) - 1;
        float x = v[0];
#pragma unroll
        for (int k = 1; k < kN; ++k) x = j == k ? v[k] : x;
        take(x, place_of(j));
      }
    };
    auto consider_block = [&](const typename R::Raw& raw, int seg) {
      float v[8];
      R::unpack(raw, v);
      consider(v, std::integral_constant<int, 8>(), [&](int j) { return R::place(seg, lane, j); });
    };
    if (fine) {
      // each lane notes which of its segments reach the bound, up to 32 of them, then reads those
      for (int i0 = lane * kLook + warp - 1; i0 < segments; i0 += 32 * 32 * kLook) {
        uint32_t reach = 0;
        for (int n = 0; n < 32 && i0 + n * 32 * kLook < segments; ++n) reach |= seg_max[i0 + n * 32 * kLook] >= bound ? 1u << n : 0u;
#pragma unroll 1
        for (; reach != 0; reach &= reach - 1) {
          const int first = (i0 + (__ffs(reach) - 1) * 32 * kLook) * R::kPer;
          float v[R::kPer];
#pragma unroll
          for (int j = 0; j < R::kPer; ++j) {
            const int p = first + j;
            v[j] = p >= row.shift && p < row.end ? element<T>(row.base + p) : -inf();
          }
          consider(v, std::integral_constant<int, R::kPer>(), [&](int j) { return first + j; });
        }
      }
    } else {
      for (int i0 = 0; i0 < segments; i0 += 32 * kLook) {  // neighbouring segments to different warps
        const int mine = i0 + lane * kLook + warp - 1;
        const bool reaches = mine < segments && seg_max[mine] >= bound;
        const bool whole = mine >= f && mine < row.end_whole();
        uint32_t hits = __ballot_sync(kFullMask, reaches && whole);
        while (hits != 0) {
          constexpr int kTogether = R::kWide && kThreads < 512 ? 4 : 2;  // (1 to 3 % each)
          int seg[kTogether];
          typename R::Raw raw[kTogether];
#pragma unroll
          for (int j = 0; j < kTogether; ++j) {
            seg[j] = hits != 0 ? i0 + (__ffs(hits) - 1) * kLook + warp - 1 : -1;
            hits &= hits - 1;
            if (seg[j] >= 0) raw[j] = row.fetch_whole(seg[j], lane);
          }
#pragma unroll
          for (int j = 0; j < kTogether; ++j)
            if (seg[j] >= 0) consider_block(raw[j], seg[j]);
        }
#pragma unroll 1
        for (hits = __ballot_sync(kFullMask, reaches && !whole); hits != 0; hits &= hits - 1) {
          const int seg = i0 + (__ffs(hits) - 1) * kLook + warp - 1;
          consider_block(row.fetch(seg, lane), seg);
        }
      }
    }
  }
  __syncthreads();
  const float top = sh.top, log_z = sh.log_z;
  const int count = sh.count;
  int32_t* ids = a.top_ids + t * a.top_n;
  float* out = a.top_logprobs + t * a.top_n;
  const int chosen = min(count, a.top_n);
  if (count <= kMost) {
    for (int i = threadIdx.x; i < count; i += kThreads) {
      const unsigned long long mine = sh.candidate[i];
      int before = 0;
      for (int j = 0; j < count; ++j) before += sh.candidate[j] > mine ? 1 : 0;
      if (before < a.top_n) {
        const uint32_t id = ~(uint32_t)mine;
        ids[before] = (int32_t)id;
        out[before] = (value_of((uint32_t)(mine >> 32)) - top) - log_z;
        sh.taken[before] = id;
      }
    }
  } else if (warp == 0) {
    // Many equal elements, or many large ones in a few groups: one after another, the largest
    // that is left.  Segments lie in the order of the row, so the first that holds it has its
    // lowest index; a segment's maximum is kept over what is left of it.
    using Key = unsigned long long;
    Key last = ~0ull;
    for (int n = 0; n < a.top_n; ++n) {
      float best = -inf();
      int seg = 0x7fffffff;
      for (int i = lane; i < segments; i += 32) {
        const float v = sane(seg_max[i]);  // as the keys: +inf ties with the largest finite value
        if (v > best) {
          best = v;
          seg = i;
        }
      }
      const float most = warp_max(best);
      seg = __reduce_min_sync(kFullMask, best == most ? seg : 0x7fffffff);
      Key one = 0, two = 0;  // the lane's two largest of those that are left
      auto look = [&](float v, int at) {
        const Key key = ((Key)order_of(sane(v)) << 32) | (uint32_t)~(uint32_t)(at - row.shift);
        if (key >= last) return;
        two = key > one ? one : (key > two ? key : two);
        one = key > one ? key : one;
      };
      if (fine) {
        const int at = seg * R::kPer + lane;
        if (lane < R::kPer && at >= row.shift && at < row.end) look(element<T>(row.base + at), at);
      } else {
#pragma unroll 1
        for (int j = 0; j < 8; ++j) {
          const int at = R::place(seg, lane, j);
          if (at >= row.shift && at < row.end) look(element<T>(row.base + at), at);
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const Key p1 = __shfl_xor_sync(kFullMask, one, o), p2 = __shfl_xor_sync(kFullMask, two, o);
        two = p1 > one ? (one > p2 ? one : p2) : (p1 > two ? p1 : two);
        one = p1 > one ? p1 : one;
      }
      last = one;
      if (lane == 0) {
        const uint32_t id = ~(uint32_t)one;
        seg_max[seg] = two != 0 ? value_of((uint32_t)(two >> 32)) : -inf();
        ids[n] = (int32_t)id;
        out[n] = (value_of((uint32_t)(one >> 32)) - top) - log_z;
        sh.taken[n] = id;
      }
      __syncwarp();
    }
  }
  // too few: the lowest indexes not taken, of which there are enough below top_n
  if (chosen == a.top_n) return;
  __syncthreads();
  if (warp == 0) {
    bool free = lane < a.top_n;
    for (int j = 0; j < chosen; ++j) free = free && sh.taken[j] != (uint32_t)lane;
    const uint32_t left_over = __ballot_sync(kFullMask, free);
    const int to = chosen + __popc(left_over & ((1u << lane) - 1));
    if (free && to < a.top_n) {
      ids[to] = lane;
      out[to] = -inf();
    }
  }
}

template <typename T, int kThreads, bool kOnce>
cudaError_t launch_logprobs(const LogprobArgs& a, int ranks, cudaStream_t stream) {
  void (*kernel)(LogprobArgs) = logprob_kernel<T, kThreads, kOnce>;
  if (ranks > 8) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.T * ranks));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = a.top_n > 0 ? 4 * (size_t)a.segments : 0;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)ranks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <typename T>
cudaError_t launch_logprobs(const LogprobArgs& a, const DeviceInfo& info, cudaStream_t stream) {
  // 1024 threads an SM.  Up to two rows an SM, CTAs of 512 threads, clusters of them where rows are
  // fewer (with four blocks a warp at least); up to four, CTAs of 256; CTAs of 128 beyond, which
  // leave the fewest threads waiting while a row's choice is made.  us for 301 rows of 32,003 bf16
  // logits, 553 of 114,789 fp32 and 2047 of 151,936 bf16: 512 threads 8.3, 49.4, 112.8; 256 9.1,
  // 46.3, 112.3; 128 11.2, 57.9, 105.9.
  if (a.T <= 2 * info.sms) {
    int ranks = 1;
    while (ranks < 16 && a.T * ranks * 2 <= 2 * info.sms && (int64_t)ranks * 2 * 16 * 4 * kBlock <= a.V) ranks *= 2;
    return launch_logprobs<T, 512, true>(a, ranks, stream);
  }
  // Loads of what is hardly read again where less than a twelfth of the row's blocks are (2047 rows of
  // 151,936 in bf16, 5 alternatives: 105.9 us for 108.1; 4000 of 30,121 with 32: 71.2 for 70.2).
  const bool once = (int64_t)a.top_n * 12 * kBlock <= a.V;
  if (a.T <= 4 * info.sms) return once ? launch_logprobs<T, 256, true>(a, 1, stream) : launch_logprobs<T, 256, false>(a, 1, stream);
  return once ? launch_logprobs<T, 128, true>(a, 1, stream) : launch_logprobs<T, 128, false>(a, 1, stream);
}

// Bytes at an address: T rows of `width`, `row` apart.
struct Extent {
  uintptr_t at;
  uint64_t row, width, all;
  Extent(const void* p, uint64_t T, uint64_t row_bytes, uint64_t width_bytes)
      : at((uintptr_t)p), row(row_bytes), width(width_bytes), all(p != nullptr && T > 0 && width_bytes > 0 ? (T - 1) * row_bytes + width_bytes : 0) {}
  // o without gaps, which may lie in one of this one's
  bool meets(const Extent& o) const {
    if (all == 0 || o.all == 0 || at >= o.at + o.all || o.at >= at + all) return false;
    if (o.at < at || width >= row) return true;
    const uint64_t d = (o.at - at) % row;
    return d < width || d + o.all > row;
  }
};

}  // namespace
}  // namespace memra

using namespace memra;

extern "C" memra_status memra_token_logprobs(const void* logits, int32_t dtype, int64_t T, int64_t V,
                                             int64_t stride_t, const int32_t* tokens, int64_t top_n,
                                             float* logprobs, float* entropy, int32_t* top_ids,
                                             float* top_logprobs, int32_t* dev_status,
                                             cudaStream_t stream) {
  if (T < 0 || V < 1 || stride_t < 0 || top_n < 0 || top_n > V) return MEMRA_ERR_INVALID_ARG;
  if (dtype != MEMRA_BF16 && dtype != MEMRA_F32) return MEMRA_ERR_INVALID_ARG;
  if (V > MEMRA_MAX_VOCAB || top_n > MEMRA_MAX_TOP_LOGPROBS || T > INT32_MAX / 16 ||
      stride_t > ((int64_t)1 << 56) / (T + 1))
    return MEMRA_ERR_UNSUPPORTED;
  if (T == 0) return MEMRA_OK;
  if (!logits || (tokens == nullptr) != (logprobs == nullptr)) return MEMRA_ERR_INVALID_ARG;
  if (top_n > 0 && (!top_ids || !top_logprobs)) return MEMRA_ERR_INVALID_ARG;
  const int es = dtype == MEMRA_BF16 ? 2 : 4;
  if (!aligned(logits, es)) return MEMRA_ERR_ALIGNMENT;
  const void* words[] = {tokens, logprobs, entropy, top_ids, top_logprobs, dev_status};
  for (const void* p : words)
    if (!aligned(p, 4)) return MEMRA_ERR_ALIGNMENT;
  const auto list = [](const void* p, int64_t n) { return Extent(p, 1, 0, 4 * (uint64_t)n); };
  const Extent in[] = {Extent(logits, (uint64_t)T, (uint64_t)stride_t * es, (uint64_t)V * es), list(tokens, T)};
  const Extent out[] = {list(logprobs, T), list(entropy, T), list(top_ids, T * top_n), list(top_logprobs, T * top_n), list(dev_status, 1)};
  for (const Extent& o : out) {
    if (in[0].meets(o) || in[1].meets(o)) return MEMRA_ERR_INVALID_ARG;
    for (const Extent* p = out; p != &o; ++p)
      if (p->meets(o)) return MEMRA_ERR_INVALID_ARG;
  }
  DeviceInfo info;
  if (!device_info(&info)) return MEMRA_ERR_CUDA;
  LogprobArgs a;
  a.logits = logits;
  a.T = T;
  a.stride_t = stride_t;
  a.V = (int)V;
  a.top_n = (int)top_n;
  const int64_t blocks = (V + 16 / es - 1 + kBlock - 1) / kBlock;
  // Fine segments where a sixth of the blocks or more would be read again, as far as shared memory
  // goes.  us with blocks and with pieces, bf16: 7820 rows of 6885 with 5 alternatives 53 and 52, 4000
  // of 30,121 with 32 74 and 70, with 5 55 and 63; 301 of 32,003 with 10 8.3 and 8.6.
  a.fine = V * es <= kFineBytes && V < 6 * kBlock * top_n;
  a.segments = (int)(a.fine ? blocks * kBlock * es / 16 : blocks);
  a.tokens = tokens;
  a.logprobs = logprobs;
  a.entropy = entropy;
  a.top_logprobs = top_logprobs;
  a.top_ids = top_ids;
  a.status = dev_status;
  const cudaError_t e = dtype == MEMRA_BF16 ? launch_logprobs<uint16_t>(a, info, stream)
                                            : launch_logprobs<float>(a, info, stream);
  if (e != cudaSuccess) return cuda_fail(e);
  return MEMRA_OK;
}
