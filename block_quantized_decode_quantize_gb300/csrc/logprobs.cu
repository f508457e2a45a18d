// Log probabilities of tokens from a row of logits, its entropy and its largest entries.
//
// One pass over the logits: each warp keeps a running maximum m, its lanes z = sum e^(x - m)
// and s = sum e^(x - m) (x - m), and rescales them when m grows.  The largest element itself
// stays outside the sums (its term is 1 and 0), so that ln Z = log1p(z) and log probabilities
// near 0 keep their digits.  The vocabulary is cut into segments; a segment's maximum goes to
// shared memory as the pass goes by.  The top_n-th largest of 32 groups of these maxima is a
// bound that top_n elements reach, so only segments whose maximum reaches it are read once
// more (from L2), and the few elements at or above it are ranked by counting.
//
// A row is taken by the CTAs of a cluster, which leave maxima and sums in the first one's
// shared memory: with few rows many SMs share the read of one.
#include <cooperative_groups.h>

#include "common.cuh"

namespace memra {
namespace {

namespace cg = cooperative_groups;

constexpr int kBlock = 256;         // elements a warp looks at together: 8 a lane
constexpr int kMost = 512;          // candidates that are ranked by counting
constexpr int kFineVocab = 16384; // see memra_token_logprobs
constexpr int kMaxWarps = 512;      // of a row: 16 CTAs of 32
constexpr float kLog2e = 1.44269504088896341f;
constexpr float kLargest = 3.402823466e38f;
constexpr float kFloor = -150.0f;   // e^x is 0 in fp32 below

struct LogprobArgs {
  const void* logits;
  int64_t T, stride_t;
  int V, top_n, fine, segments;     // fine: a segment is 16 bytes of the row, else a block; at most so many
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

template <typename T>
__device__ __forceinline__ float element(const T* p);
template <>
__device__ __forceinline__ float element<float>(const float* p) { return *p; }
template <>
__device__ __forceinline__ float element<uint16_t>(const uint16_t* p) { return __uint_as_float((uint32_t)*p << 16); }

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
  // place of the lane's value i of a block
  static __device__ __forceinline__ int place(int b, int lane, int i) {
    return b * kBlock + (kWide ? 4 * lane + (i & 3) + 32 * (i & 4) : 8 * lane + i);
  }
  __device__ __forceinline__ bool whole(int b) const { return b * kBlock >= shift && (b + 1) * kBlock <= end; }
  struct Raw {
    uint4 u[kWide ? 2 : 1];
  };
  __device__ __forceinline__ Raw fetch(int b, int lane) const {  // of a whole block
    Raw r;
    const uint4* p = reinterpret_cast<const uint4*>(base + (int64_t)b * kBlock) + lane;
    r.u[0] = __ldcs(p);
    if (kWide) r.u[kWide ? 1 : 0] = __ldcs(p + 32);
    return r;
  }
  static __device__ __forceinline__ void unpack(const Raw& r, float* v) {
    if (kWide) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint4& u = r.u[kWide ? h : 0];
        v[4 * h] = __uint_as_float(u.x); v[4 * h + 1] = __uint_as_float(u.y);
        v[4 * h + 2] = __uint_as_float(u.z); v[4 * h + 3] = __uint_as_float(u.w);
      }
    } else {
      const uint32_t w[4] = {r.u[0].x, r.u[0].y, r.u[0].z, r.u[0].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      }
    }
  }
  // any block, -inf for places outside the row
  __device__ __forceinline__ void load(int b, int lane, float* v) const {
    if (whole(b)) {
      unpack(fetch(b, lane), v);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int at = place(b, lane, i);
        v[i] = at >= shift && at < end ? element<T>(base + at) : -inf();
      }
    }
  }
};

struct Part {  // of a warp: the row's terms but its largest one, relative to m
  float m, z, s;
};

struct Shared {
  Part part[kMaxWarps];
  unsigned long long candidate[kMost];
  int count, listed;
  float bound, m, log_z;
  uint32_t taken[MEMRA_MAX_TOP_LOGPROBS];
};

// The warp's sums take in the 8 values of each lane.  m: the warp's maximum so far, over these too.
__device__ __forceinline__ void add8(const float* v, float m, float& z, float& s) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float d = fmaxf(v[i] - m, kFloor), e = exp2_approx(d * kLog2e);
    z += e;
    s = fmaf(e, d, s);
  }
}

template <typename T, int kThreads>
__global__ void __launch_bounds__(kThreads) logprob_kernel(LogprobArgs a) {
  constexpr int kWarps = kThreads / 32;
  constexpr int kAhead = sizeof(T) == 4 ? 2 : 4;  // blocks that a warp has under way
  extern __shared__ float seg_max[];              // [segments], the row's first CTA; then the list of segments to read again
  __shared__ Shared sh;
  pdl_launch_dependents();
  cg::cluster_group cluster = cg::this_cluster();
  const int ranks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = blockIdx.x / ranks;
  pdl_wait();
  const Row<T> row(static_cast<const T*>(a.logits) + t * a.stride_t, a.V);
  const int blocks = row.blocks();
  Shared* first = cluster.map_shared_rank(&sh, 0);
  float* first_max = cluster.map_shared_rank(seg_max, 0);

  float m = -inf(), z = 0.0f, s = 0.0f;
  bool met = false;  // the row's first CTA has begun, so its shared memory can be written
  for (int b0 = rank * kWarps + warp; b0 < blocks; b0 += ranks * kWarps * kAhead) {
    float v[kAhead][8];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int b = b0 + j * ranks * kWarps;
      if (b < blocks) {
        row.load(b, lane, v[j]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[j][i] = -inf();
      }
    }
    if (!met) {
      asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
      met = true;
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int b = b0 + j * ranks * kWarps;
      if (b >= blocks) break;
      float most = -inf();
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[j][i] = sane(v[j][i]);
        most = fmaxf(most, v[j][i]);
      }
      const float block_most = warp_max(most);
      if (a.top_n > 0) {
        if (a.fine) {
#pragma unroll
          for (int h = 0; h < Row<T>::kPieces; ++h) {
            float piece = v[j][h * Row<T>::kPer];
#pragma unroll
            for (int i = 1; i < Row<T>::kPer; ++i) piece = fmaxf(piece, v[j][h * Row<T>::kPer + i]);
            first_max[(b * Row<T>::kPieces + h) * 32 + lane] = piece;
          }
        } else if (lane == 0) {
          first_max[b] = block_most;
        }
      }
      if (block_most > m) {
        // A new largest element: what was the largest becomes a term, and the new one, in the
        // first lane that holds it, is none.
        const float down = fmaxf(m - block_most, kFloor), f = exp2_approx(down * kLog2e);
        if (m > -inf()) {
          s = f * fmaf(down, z, s);
          z *= f;
          if (lane == 0) {
            z += f;
            s = fmaf(f, down, s);
          }
        }
        m = block_most;
        const int holder = __ffs(__ballot_sync(kFullMask, most == m)) - 1;
        if (lane == holder) {
          bool out = false;
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (!out && v[j][i] == m) {
              v[j][i] = -inf();
              out = true;
            }
        }
      }
      if (m > -inf()) add8(v[j], m, z, s);
    }
  }
  if (!met) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    z += __shfl_xor_sync(kFullMask, z, o);
    s += __shfl_xor_sync(kFullMask, s, o);
  }
  if (lane == 0) first->part[rank * kWarps + warp] = {m, z, s};
  cluster.sync();
  if (rank != 0) return;

  // ---- the row's first CTA ----
  const int segments = a.fine ? blocks * 32 * Row<T>::kPieces : blocks;
  if (warp == 0) {
    float top = -inf();
    for (int i = lane; i < ranks * kWarps; i += 32) top = fmaxf(top, sh.part[i].m);
    top = warp_max(top);
    // the largest element is the first such part's; of others it is a term
    int own = 0x7fffffff;
    for (int i = ranks * kWarps - 1 - lane; i >= 0; i -= 32)
      if (sh.part[i].m == top) own = i;
    own = __reduce_min_sync(kFullMask, own);
    float zz = 0.0f, ss = 0.0f;
    for (int i = lane; i < ranks * kWarps; i += 32) {
      const Part p = sh.part[i];
      if (p.m == -inf()) continue;
      const float down = fmaxf(p.m - top, kFloor), f = exp2_approx(down * kLog2e);
      const float terms = i == own ? p.z : p.z + 1.0f;
      zz = fmaf(f, terms, zz);
      ss = fmaf(f, fmaf(down, terms, p.s), ss);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      zz += __shfl_xor_sync(kFullMask, zz, o);
      ss += __shfl_xor_sync(kFullMask, ss, o);
    }
    if (lane == 0) {
      const bool none = top == -inf();
      const float log_z = log1pf(zz);
      sh.m = top;
      sh.log_z = log_z;
      if (a.entropy != nullptr) a.entropy[t] = none ? 0.0f : log_z - ss / (1.0f + zz);
      if (a.logprobs != nullptr) {
        const int32_t token = a.tokens[t];
        float lp = -inf();
        if (token >= 0 && token < a.V) {
          const float x = sane(element<T>(row.base + row.shift + token));
          if (!none) lp = (x - top) - log_z;
        } else if (token == -1) {
          lp = 0.0f;
        } else if (a.status != nullptr) {
          atomicOr(a.status, 1);
        }
        a.logprobs[t] = lp;
      }
    }
  } else if (warp == 1 && a.top_n > 0) {
    // the bound, as the top_n-th largest of the maxima of 32 groups of segments
    float best = -inf();
    for (int i = lane; i < segments; i += 32) {
      best = fmaxf(best, seg_max[i]);
    }
    // one lane at a time is struck out, so that equal maxima count each
    float bound = -inf();
    for (int n = 0; n < a.top_n; ++n) {
      bound = warp_max(best);
      const uint32_t at = __ballot_sync(kFullMask, best == bound);
      if (lane == __ffs(at) - 1) best = -inf();
    }
    if (lane == 0) {
      sh.bound = bound;
      sh.count = sh.listed = 0;
    }
  }
  if (a.top_n == 0) return;
  __syncthreads();
  const float bound = sh.bound, top = sh.m, log_z = sh.log_z;
  const float kMasked = -inf();
  // the segments to read again, and their elements at or above the bound
  uint32_t* list = reinterpret_cast<uint32_t*>(seg_max + a.segments);
  for (int i = threadIdx.x; i < segments; i += kThreads)
    if (seg_max[i] >= bound && seg_max[i] > kMasked) list[atomicAdd(&sh.listed, 1)] = i;
  __syncthreads();
  const int listed = sh.listed;
  auto consider = [&](float v, int at) {
    v = sane(v);
    if (v >= bound && v > kMasked) {
      const int n = atomicAdd(&sh.count, 1);
      if (n < kMost)
        sh.candidate[n] = ((unsigned long long)order_of(v) << 32) | (uint32_t)~(uint32_t)(at - row.shift);
    }
  };
  if (a.fine) {
    for (int i = threadIdx.x; i < listed * Row<T>::kPer; i += kThreads) {
      const int at = list[i / Row<T>::kPer] * Row<T>::kPer + i % Row<T>::kPer;
      if (at >= row.shift && at < row.end) consider(element<T>(row.base + at), at);
    }
  } else {
    for (int i = warp; i < listed; i += kWarps) {
      float v[8];
      row.load(list[i], lane, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) consider(v[j], Row<T>::place(list[i], lane, j));
    }
  }
  __syncthreads();
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
      for (int i = lane; i < segments; i += 32)
        if (seg_max[i] > best) {
          best = seg_max[i];
          seg = i;
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
      if (a.fine) {
        const int at = seg * Row<T>::kPer + lane;
        if (lane < Row<T>::kPer && at >= row.shift && at < row.end) look(element<T>(row.base + at), at);
      } else {
        float v[8];
        row.load(seg, lane, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int at = Row<T>::place(seg, lane, j);
          if (at >= row.shift && at < row.end) look(v[j], at);
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
  if (chosen == a.top_n) return;
  __syncthreads();
  // too few: the lowest indexes not taken, of which there are enough below top_n
  if (warp == 0) {
    bool free = lane < a.top_n;
    for (int j = 0; j < chosen; ++j) free = free && sh.taken[j] != (uint32_t)lane;
    const uint32_t left = __ballot_sync(kFullMask, free);
    const int to = chosen + __popc(left & ((1u << lane) - 1));
    if (free && to < a.top_n) {
      ids[to] = lane;
      out[to] = -inf();
    }
  }
}

template <typename T, int kThreads>
cudaError_t launch_logprobs(const LogprobArgs& a, int ranks, cudaStream_t stream) {
  void (*kernel)(LogprobArgs) = logprob_kernel<T, kThreads>;
  if (ranks > 8) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.T * ranks));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = a.top_n > 0 ? (size_t)a.segments * 8 : 0;
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
cudaError_t launch_logprobs(const LogprobArgs& a, int sms, cudaStream_t stream) {
  // CTAs to a row: as many as keep the SMs busy, and no more than have four blocks a warp to look at
  int ranks = 1;
  while (ranks < 16 && a.T * ranks * 2 <= 2 * sms && (int64_t)ranks * 2 * 16 * 4 * kBlock <= a.V) ranks *= 2;
  return launch_logprobs<T, 512>(a, ranks, stream);
}

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
  DeviceInfo info;
  if (!device_info(&info)) return MEMRA_ERR_CUDA;
  LogprobArgs a;
  a.logits = logits;
  a.T = T;
  a.stride_t = stride_t;
  a.V = (int)V;
  a.top_n = (int)top_n;
  // Segments of 16 bytes where the vocabulary is small, so that there are many more of them
  // than top_n; 256 elements else.
  a.fine = V <= kFineVocab;
  const int64_t blocks = (V + 16 / es - 1 + kBlock - 1) / kBlock;
  a.segments = (int)(a.fine ? blocks * kBlock * es / 16 : blocks);
  a.tokens = tokens;
  a.logprobs = logprobs;
  a.entropy = entropy;
  a.top_logprobs = top_logprobs;
  a.top_ids = top_ids;
  a.status = dev_status;
  const cudaError_t e = dtype == MEMRA_BF16 ? launch_logprobs<uint16_t>(a, info.sms, stream)
                                            : launch_logprobs<float>(a, info.sms, stream);
  if (e != cudaSuccess) return cuda_fail(e);
  return MEMRA_OK;
}
