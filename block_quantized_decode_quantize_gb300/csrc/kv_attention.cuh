// What the attention kernels over the paged 8-bit cache share: their arguments, the work
// list and how a CTA finds its part of it.
//
// A unit is (request, cached head, group of kRows query rows); a row is a (query, query
// head) pair that reads this cached head, so grouped heads share every byte.  A unit takes
// kCost entries of the list for its fixed time and one for each tile of kTile keys; the
// list is cut into equal parts for the CTAs of one resident wave, so every CTA streams
// about the same number of bytes whatever the lengths are.
#pragma once

#include <cuda_bf16.h>

#include "common.cuh"

namespace memra {

constexpr int kStrip = 16;      // keys that share a page at least (a page is a multiple)
constexpr int kTile = 128;      // keys of an entry of the list
constexpr int kMaxCtas = 512;   // arrival counters at the workspace's start

// A weight enters the second product as p * (vd / ref) * 2^8 in fp16, ref a running maximum
// of vd kept within a factor 4, p = 2^(s - m) with m within 5 of the running maximum: at
// most 2^(5 + 2 + 8) = 2^15, and down to 2^-33 of the largest before it rounds to zero.
constexpr float kMaxSlack = 5.0f;
constexpr float kRefSlack = 4.0f;
constexpr float kWeightScale = 256.0f;

struct AttnArgs {
  const void* q;
  int64_t T, stride_t, stride_h;
  const int8_t *kq, *vq;
  const float *kd, *vd;
  const int32_t *table, *kv_lens, *cu_q;
  int64_t B, max_pages, window;
  int32_t n_pages;
  int Hq, Hkv, G, page, block;
  Divider by_page, by_block;
  uint32_t page_bytes, page_scales;  // of one page in a plane, all heads
  int step_pages, step_off;          // kTile = step_pages * page + step_off
  float scale;
  void* out;
  float* lse;
  int* arrived;   // [kMaxCtas], zero between calls
  float* parts;   // [2][CTAs][rows * (D + 2)]
  int32_t* status;
  long long wait_limit;  // of the wide kernel's waits (cycles), and the test hook's stall
  int stall_after;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Copies to shared memory that this thread waits for by groups.
__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// 16 bytes, or zeros where `there` is false.
__device__ __forceinline__ void cp16_or_zeros(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kN>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kN) : "memory");
}

__device__ __forceinline__ float value(const float* p) { return *p; }
__device__ __forceinline__ float value(const uint16_t* p) {
  return __uint_as_float((uint32_t)*p << 16);
}
__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void store4(uint16_t* p, float4 v) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
  uint2 u;
  u.x = *reinterpret_cast<const uint32_t*>(&a);
  u.y = *reinterpret_cast<const uint32_t*>(&b);
  *reinterpret_cast<uint2*>(p) = u;
}

// Where a request's part of the list lies, from its lengths.
struct Request {
  int len, n;        // tokens in the cache, queries
  int row;           // the first query's row of q
  int lo;            // first key tile's start
  int tiles, groups;
  bool over;         // longer than its row of the block table
};

template <int kRows>
__device__ __forceinline__ Request request_of(const AttnArgs& a, int64_t b) {
  Request r;
  const int64_t cap = a.max_pages * a.page;
  int64_t len = a.kv_lens[b];
  const int row = a.cu_q[b];
  r.over = len > cap;
  len = len < 0 ? 0 : (len > cap ? cap : len);
  int64_t n = (int64_t)a.cu_q[b + 1] - row;
  n = n < 0 ? 0 : (n > a.T ? a.T : n);
  r.len = (int)len;
  r.n = (int)n;
  r.row = row;
  int64_t lo = a.window > 0 ? len - n + 1 - a.window : 0;
  lo = lo < 0 ? 0 : lo / kStrip * kStrip;
  r.lo = (int)lo;
  r.tiles = n > 0 && len > lo ? (int)((len - lo + kTile - 1) / kTile) : 0;
  r.groups = (int)((n * a.G + kRows - 1) / kRows);
  return r;
}

// total entries in ctas equal parts (the first ones one longer): where part c begins, and
// which part holds entry x.
struct Cut {
  int64_t total, q, r;
  static __device__ __forceinline__ int64_t divide(int64_t a, int64_t b) {
    return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
  }
  __device__ __forceinline__ Cut(int64_t t, int ctas) : total(t), q(divide(t, ctas)), r(t - q * ctas) {}
  __device__ __forceinline__ int64_t begin(int c) const { return c * q + min((int64_t)c, r); }
  __device__ __forceinline__ int part_of(int64_t x) const {
    const int64_t longer = r * (q + 1);
    return (int)(x < longer ? divide(x, q + 1) : r + divide(x - longer, q));
  }
};

// A unit takes kCost entries and one for each tile.
template <int kCost>
__device__ __forceinline__ int64_t entries_of(const AttnArgs& a, const Request& r) {
  return r.tiles > 0 ? (int64_t)(r.tiles + kCost) * r.groups * a.Hkv : (int64_t)0;
}

// Where a CTA stands in the list: entry x of [.., stop), in request b whose first entry is at.
struct Walk {
  int64_t x, at, stop;
  int b;
  Request req;
};
template <typename T, int kD>
__device__ __forceinline__ void write_nothing(const AttnArgs& a, int64_t row0, int64_t row1,
                                              int thread, int threads) {
  T* out = static_cast<T*>(a.out);
  row0 = row0 < 0 ? 0 : row0;
  row1 = row1 > a.T ? a.T : row1;
  for (int64_t i = row0 * a.Hq * kD / 4 + thread; i < row1 * a.Hq * kD / 4; i += threads)
    store4(out + i * 4, make_float4(0.0f, 0.0f, 0.0f, 0.0f));
  if (a.lse != nullptr)
    for (int64_t i = row0 * a.Hq + thread; i < row1 * a.Hq; i += threads)
      a.lse[i] = __int_as_float(0xff800000);
}

// The kernel for many bf16 rows (kv_attention_wide.cu), D 64 or 128; rows: an average unit's.
cudaError_t launch_wide_attention(const AttnArgs& a, int D, int64_t rows, const DeviceInfo& info,
                                  int64_t max_tiles, cudaStream_t stream);

// Sums every request's entries and finds this CTA's part of the list, into *walk (all
// threads of the CTA call it; ends with a barrier).  Returns the number of CTAs that have a
// part and the list's length in *ctas and *total; false where this one has none.  Rows that
// see nothing because their request has no keys, and rows that no request owns, are
// written here, each by one CTA.
template <typename T, int kD, int kRows, int kCost, int kThreads>
__device__ __forceinline__ bool locate(const AttnArgs& a, Walk* walk, int* ctas, int64_t* total) {
  constexpr int kWarps = kThreads / 32;
  __shared__ int64_t warp_sum[kWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, cta = blockIdx.x;
  auto entries = [&](const Request& r) { return entries_of<kCost>(a, r); };
  int64_t w = 0, sum = 0;
  Request r{};
  int64_t no_row = a.B > 0 ? a.cu_q[a.B] : 0;
  // Rows that no request owns: below the first one's, and from the last one's end on.
  auto rest = [&](int64_t owned) {
    *ctas = (int)min((int64_t)gridDim.x, *total);
    for (int64_t i = cta; i < owned && i < a.T; i += gridDim.x) write_nothing<T, kD>(a, i, i + 1, tid, kThreads);
    for (no_row += cta; no_row < a.T; no_row += gridDim.x)
      write_nothing<T, kD>(a, no_row, no_row + 1, tid, kThreads);
  };
  if (a.B <= 32) {
    // a lane to a request, every warp for itself: no barrier but the last
    if (lane < a.B) {
      r = request_of<kRows>(a, lane);
      w = entries(r);
      if (cta == 0 && warp == 0 && r.over && a.status != nullptr) atomicOr(a.status, 1);
    }
    sum = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t u = __shfl_up_sync(kFullMask, sum, o);
      if (lane >= o) sum += u;
    }
    *total = __shfl_sync(kFullMask, sum, 31);
    for (uint32_t todo = __ballot_sync(kFullMask, w == 0 && r.n > 0); todo != 0; todo &= todo - 1) {
      const int e = __ffs(todo) - 1;
      if (e % gridDim.x == cta) write_nothing<T, kD>(a, a.cu_q[e], a.cu_q[e + 1], tid, kThreads);
    }
    rest(__shfl_sync(kFullMask, r.row, 0));
    if (cta >= *ctas) return false;
    const Cut cut(*total, *ctas);
    const int64_t first = cut.begin(cta);
    if (warp == 0 && w > 0 && sum - w <= first && first < sum) *walk = {first, sum - w, cut.begin(cta + 1), lane, r};
    __syncthreads();
    return true;
  }
  int64_t first = 0;
  for (int pass = 0; pass < 2; ++pass) {
    int64_t before = 0;
    for (int64_t base = 0; base < a.B; base += kThreads) {
      const int64_t b = base + tid;
      if (pass == 0 || a.B > kThreads) {  // one chunk's sums stay in registers
        w = 0;
        bool empty = false;
        if (b < a.B) {
          r = request_of<kRows>(a, b);
          w = entries(r);
          empty = w == 0 && r.n > 0;
          if (pass == 0 && cta == 0 && r.over && a.status != nullptr) atomicOr(a.status, 1);
        }
        if (pass == 0) {
          uint32_t todo = __ballot_sync(kFullMask, empty && b % gridDim.x == cta);
          while (todo != 0) {
            const int64_t e = base + warp * 32 + (__ffs(todo) - 1);
            todo &= todo - 1;
            write_nothing<T, kD>(a, a.cu_q[e], a.cu_q[e + 1], lane, 32);
          }
        }
        sum = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int64_t u = __shfl_up_sync(kFullMask, sum, o);
          if (lane >= o) sum += u;
        }
        if (lane == 31) warp_sum[warp] = sum;
        __syncthreads();
        int64_t chunk = 0;
        for (int i = 0; i < kWarps; ++i) {
          if (i < warp) sum += warp_sum[i];
          chunk += warp_sum[i];
        }
        sum += before;
        before += chunk;
      }
      if (pass == 1 && w > 0 && sum - w <= first && first < sum)
        *walk = {first, sum - w, Cut(*total, *ctas).begin(cta + 1), (int)b, r};
      __syncthreads();
    }
    if (pass == 0) {
      *total = before;
      rest(a.cu_q[0]);
      if (cta >= *ctas) return false;
      first = Cut(*total, *ctas).begin(cta);
    }
  }
  return true;
}

}  // namespace memra
