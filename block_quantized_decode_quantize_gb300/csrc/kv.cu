// The paged 8-bit KV cache: the page plan of a step, the write of its tokens and their
// read-back.  Layouts and arithmetic are stated in memra.h.
#include <cuda_bf16.h>

#include "common.cuh"

namespace memra {
namespace {

// ---------------------------------------------------------------------------
// The page plan.  One CTA scans the requests in chunks of its size (tokens and pages
// before each request), writes the per-request outputs and the chunk's new table entries,
// and, when the step is small, the rows' slots too; a second kernel over the whole GPU
// fills the rows of a large step by searching cu_q.
// ---------------------------------------------------------------------------
constexpr int kPlanThreads = 1024;

struct PlanArgs {
  const int32_t *ctx, *add;
  int64_t B, n_free, max_pages, T;
  int page;
  const int32_t *free_pages, *free_head;
  int32_t *table, *kv_lens, *cu_q, *slots, *positions, *free_head_out, *status;
};

// Inclusive sums of a and b over the CTA's threads; *ta, *tb receive the totals.
__device__ __forceinline__ void scan2(int64_t& a, int64_t& b, int64_t* sa, int64_t* sb,
                                      int64_t* ta, int64_t* tb) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t ua = __shfl_up_sync(kFullMask, a, o), ub = __shfl_up_sync(kFullMask, b, o);
    if (lane >= o) {
      a += ua;
      b += ub;
    }
  }
  if (lane == 31) {
    sa[warp] = a;
    sb[warp] = b;
  }
  __syncthreads();
  if (warp == 0) {
    int64_t wa = sa[lane], wb = sb[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t ua = __shfl_up_sync(kFullMask, wa, o), ub = __shfl_up_sync(kFullMask, wb, o);
      if (lane >= o) {
        wa += ua;
        wb += ub;
      }
    }
    sa[lane] = wa;
    sb[lane] = wb;
  }
  __syncthreads();
  if (warp > 0) {
    a += sa[warp - 1];
    b += sb[warp - 1];
  }
  *ta = sa[31];
  *tb = sb[31];
}

// Last i in [lo, hi) with a[i] <= x, given a[lo] <= x (a ascending).
template <typename V>
__device__ __forceinline__ int last_at_most(const V* a, int lo, int hi, V x) {
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

template <bool kFill>
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(PlanArgs a) {
  __shared__ int64_t sa[32], sb[32];
  __shared__ int64_t first_row[kPlanThreads], first_page[kPlanThreads];
  __shared__ int32_t have_of[kPlanThreads], ctx_of[kPlanThreads];
  pdl_launch_dependents();
  pdl_wait();
  const int tid = threadIdx.x;
  int64_t head = a.free_head != nullptr ? *a.free_head : 0;
  if (head < 0) head = 0;
  const int64_t head0 = head;
  int64_t row0 = 0, taken = 0;
  int bits = 0;
  if (tid == 0) a.cu_q[0] = 0;
  for (int64_t base = 0; base < a.B; base += kPlanThreads) {
    const int64_t b = base + tid;
    const int count = (int)min((int64_t)kPlanThreads, a.B - base);
    int64_t ctx = 0, add = 0;
    bool fits = b < a.B;
    if (fits) {
      ctx = a.ctx[b];
      add = a.add[b];
      if (ctx < 0 || add < 0) {
        fits = false;
        ctx = ctx < 0 ? 0 : ctx;
        add = add < 0 ? 0 : add;
      }
    }
    const int64_t have = (ctx + a.page - 1) / a.page, after = (ctx + add + a.page - 1) / a.page;
    int64_t rows = add, unused = 0, total_rows, total_pages, total_unused;
    // The rows decide who fits, so they are summed before the pages.
    scan2(rows, unused, sa, sb, &total_rows, &total_unused);
    const int64_t upto = row0 + rows;
    const bool counted = b < a.B;
    fits = fits && after <= a.max_pages && ctx + add <= INT32_MAX && upto <= a.T;
    if (counted && !fits) bits |= 1;
    __syncthreads();
    const int64_t need = fits ? after - have : 0;
    int64_t pages = need;
    scan2(pages, unused, sa, sb, &total_pages, &total_unused);
    const int64_t end = head + pages;
    const bool ok = fits && (need == 0 || end <= a.n_free);
    if (fits && !ok) bits |= 4;
    const int64_t got = ok ? need : 0;
    first_row[tid] = min(upto - add, a.T);
    first_page[tid] = ok ? pages - need : -1;
    have_of[tid] = (int32_t)have;
    ctx_of[tid] = (int32_t)ctx;
    if (counted) {
      a.kv_lens[b] = ok ? (int32_t)(ctx + add) : 0;
      a.cu_q[b + 1] = (int32_t)min(upto, a.T);
    }
    __syncthreads();
    // New table entries, a warp to a request: its lanes take neighbouring pages.
    for (int r = tid >> 5; r < count; r += kPlanThreads / 32) {
      const int64_t f = first_page[r];
      if (f < 0) continue;
      const int64_t c = ctx_of[r], h = have_of[r];
      const int64_t n = a.add[base + r];
      const int64_t m = (c + n + a.page - 1) / a.page - h;
      for (int64_t i = tid & 31; i < m; i += 32)
        a.table[(base + r) * a.max_pages + h + i] = a.free_pages[head + f + i];
    }
    if (kFill) {
      const int64_t stop = min(row0 + total_rows, a.T);
      for (int64_t t = min(row0, a.T) + tid; t < stop; t += kPlanThreads) {
        const int r = last_at_most(first_row, 0, count, t);
        const int64_t pos = ctx_of[r] + t - first_row[r];
        int32_t slot = -1;
        if (first_page[r] >= 0) {
          const int64_t p = pos / a.page;
          const int64_t page = p < have_of[r]
                                   ? a.table[(base + r) * a.max_pages + p]
                                   : a.free_pages[head + first_page[r] + p - have_of[r]];
          slot = (int32_t)(page * a.page + pos % a.page);
        }
        a.slots[t] = slot;
        a.positions[t] = (int32_t)pos;
      }
    }
    __syncthreads();
    // Pages granted in this chunk (the requests that were refused took none).
    int64_t granted = got, total_granted;
    scan2(granted, unused, sa, sb, &total_granted, &total_unused);
    taken += total_granted;
    head += total_pages;
    row0 += total_rows;
    __syncthreads();
  }
  if (kFill) {
    for (int64_t t = min(row0, a.T) + tid; t < a.T; t += kPlanThreads) {
      a.slots[t] = -1;
      a.positions[t] = -1;
    }
  }
  if (tid == 0) *a.free_head_out = (int32_t)(head0 + taken);
  if (bits != 0 && a.status != nullptr) atomicOr(a.status, bits);
}

// Rows of a large step: thread by thread four consecutive rows, the request found in cu_q.
// kv_lens tells a refused request (it has rows and kv_lens 0).
__global__ void __launch_bounds__(256) plan_fill_kernel(PlanArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  const int64_t t0 = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) * 4;
  if (t0 >= a.T) return;
  int r = last_at_most(a.cu_q, 0, (int)a.B + 1, (int32_t)t0);
  int32_t slot[4], posn[4];
  int32_t next = r < a.B ? a.cu_q[r + 1] : INT32_MAX;
  int32_t first = r < a.B ? a.cu_q[r] : 0, ctx = r < a.B ? max(a.ctx[r], 0) : 0;
  bool ok = r < a.B && a.kv_lens[r] > 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int32_t t = (int32_t)(t0 + i);
    while (t >= next) {
      ++r;
      next = r < a.B ? a.cu_q[r + 1] : INT32_MAX;
      first = r < a.B ? a.cu_q[r] : 0;
      ctx = r < a.B ? max(a.ctx[r], 0) : 0;
      ok = r < a.B && a.kv_lens[r] > 0;
    }
    const int32_t pos = r < a.B ? ctx + (t - first) : -1;
    posn[i] = pos;
    slot[i] = -1;
    if (ok && t < a.T)
      slot[i] = (int32_t)((int64_t)a.table[(int64_t)r * a.max_pages + pos / a.page] * a.page +
                          pos % a.page);
  }
  if (t0 + 4 <= a.T && (((uintptr_t)a.slots | (uintptr_t)a.positions) & 15) == 0) {
    *reinterpret_cast<int4*>(a.slots + t0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
    *reinterpret_cast<int4*>(a.positions + t0) = make_int4(posn[0], posn[1], posn[2], posn[3]);
  } else {
    for (int i = 0; i < 4 && t0 + i < a.T; ++i) {
      a.slots[t0 + i] = slot[i];
      a.positions[t0 + i] = posn[i];
    }
  }
}

// Steps up to this many rows are filled by the scanning CTA itself.
constexpr int64_t kPlanFillRows = 4096;

// ---------------------------------------------------------------------------
// The write.  A warp takes one run of tokens (one scale block) of one head and plane: the
// run's largest magnitude first, then the older tokens' codes if the scale grew, then the
// run's own codes.  A lane holds 16 bytes of input at a time.
// ---------------------------------------------------------------------------
constexpr int kAppendWarps = 4;

struct CacheArgs {
  int8_t *kq, *vq;
  float *kd, *vd;
  int64_t slots_in_pool;
  int Hkv, page, D, block;
};

struct AppendArgs {
  CacheArgs c;
  const void *k, *v;
  const int32_t* slots;
  int64_t T, stride_t, stride_h;
  int tile;
  int32_t* status;
};

// Place of a slot's codes (of head h) and of its scale.
__device__ __forceinline__ int64_t code_at(const CacheArgs& c, int64_t slot, int h) {
  const int64_t page = slot / c.page, off = slot % c.page;
  return ((page * c.Hkv + h) * c.page + off) * c.D;
}
__device__ __forceinline__ int64_t scale_at(const CacheArgs& c, int64_t slot, int h) {
  const int64_t page = slot / c.page, off = slot % c.page;
  return (page * c.Hkv + h) * (c.page / c.block) + off / c.block;
}

template <typename T>
struct Vec;  // 16 bytes of input
template <>
struct Vec<float> {
  static constexpr int kN = 4;
  static __device__ __forceinline__ void load(const float* p, float v[4]) {
    const float4 x = *reinterpret_cast<const float4*>(p);
    v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
  }
};
template <>
struct Vec<uint16_t> {
  static constexpr int kN = 8;
  static __device__ __forceinline__ void load(const uint16_t* p, float v[8]) { load8_bf16(p, v); }
};

template <typename T>
__global__ void __launch_bounds__(kAppendWarps * 32) append_kernel(AppendArgs a) {
  constexpr int kN = Vec<T>::kN;
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t item = (int64_t)blockIdx.x * kAppendWarps + (threadIdx.x >> 5);
  const int planes = 2 * a.c.Hkv;
  const int64_t tiles = (a.T + a.tile - 1) / a.tile;
  if (item >= tiles * planes) return;
  const int plane = (int)(item % planes);
  const int h = plane >> 1;
  const bool is_v = plane & 1;
  const T* x = static_cast<const T*>(is_v ? a.v : a.k) + h * a.stride_h;
  int8_t* codes = is_v ? a.c.vq : a.c.kq;
  float* scales = is_v ? a.c.vd : a.c.kd;
  const int D = a.c.D, S = a.c.block;
  const int per_row = D / kN;            // lanes to a row (8 .. 64)
  const int64_t t_end = min((item / planes + 1) * a.tile, a.T);
  for (int64_t t = item / planes * a.tile; t < t_end; ++t) {
    const int64_t slot = a.slots[t];
    if (slot < 0) continue;
    if (slot >= a.c.slots_in_pool) {
      if (a.status != nullptr && plane == 0 && lane == 0) atomicOr(a.status, 1);
      continue;
    }
    const int64_t blk = slot / S;
    if (t > 0) {
      const int64_t before = a.slots[t - 1];
      if (before >= 0 && before / S == blk) continue;  // not the run's first token
    }
    const int first = (int)(slot - blk * S);
    int n = 1;
    while (first + n < S && t + n < a.T) {
      const int64_t next = a.slots[t + n];
      if (next < 0 || next / S != blk) break;
      ++n;
    }
    const T* rows = x + t * a.stride_t;
    const int total = n * per_row;
    float amax = 0.0f;
    for (int i = lane; i < total; i += 32) {
      float v[kN];
      Vec<T>::load(rows + (int64_t)(i / per_row) * a.stride_t + (i % per_row) * kN, v);
#pragma unroll
      for (int j = 0; j < kN; ++j) amax = fmaxf(amax, fabsf(v[j]));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(kFullMask, amax, o));
    float* scale = scales + scale_at(a.c, slot, h);
    const float d_old = first > 0 ? *scale : 0.0f;
    const float d = fmaxf(d_old, amax / 127.0f);
    int8_t* block_codes = codes + code_at(a.c, blk * S, h);
    if (first > 0 && d > d_old) {
      const float ratio = d_old / d;
      for (int i = lane * 4; i < first * D; i += 128) {
        const char4 q = *reinterpret_cast<const char4*>(block_codes + i);
        char4 r;
        r.x = (signed char)(int)roundf(__fmul_rn((float)q.x, ratio));
        r.y = (signed char)(int)roundf(__fmul_rn((float)q.y, ratio));
        r.z = (signed char)(int)roundf(__fmul_rn((float)q.z, ratio));
        r.w = (signed char)(int)roundf(__fmul_rn((float)q.w, ratio));
        *reinterpret_cast<char4*>(block_codes + i) = r;
      }
    }
    for (int i = lane; i < total; i += 32) {
      float v[kN];
      Vec<T>::load(rows + (int64_t)(i / per_row) * a.stride_t + (i % per_row) * kN, v);
      int8_t* to = block_codes + (int64_t)(first + i / per_row) * D + (i % per_row) * kN;
#pragma unroll
      for (int j = 0; j < kN; j += 4)
        *reinterpret_cast<uint32_t*>(to + j) =
            pack4(quant_value(v[j], d), quant_value(v[j + 1], d), quant_value(v[j + 2], d),
                  quant_value(v[j + 3], d));
    }
    __syncwarp();
    if (lane == 0) *scale = d;
  }
}

// ---------------------------------------------------------------------------
// The read-back: a thread takes 16 bytes of output.
// ---------------------------------------------------------------------------
struct ReadArgs {
  CacheArgs c;
  const int32_t* slots;
  int64_t N;
  void *k, *v;
  int32_t* status;
};

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}

template <typename T>
__global__ void __launch_bounds__(256) read_kernel(ReadArgs a) {
  constexpr int kN = Vec<T>::kN;
  pdl_launch_dependents();
  pdl_wait();
  const int per_row = a.c.D / kN;
  const int64_t per_token = (int64_t)a.c.Hkv * per_row, total = 2 * a.N * per_token;
  const int64_t stride = (int64_t)gridDim.x * blockDim.x;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += stride) {
    const bool is_v = i >= a.N * per_token;
    const int64_t j = is_v ? i - a.N * per_token : i;
    const int64_t n = j / per_token;
    const int at = (int)(j % per_token), h = at / per_row, e = at % per_row * kN;
    const int64_t slot = a.slots[n];
    T* out = static_cast<T*>(is_v ? a.v : a.k) + j * kN;
    const bool have = slot >= 0 && slot < a.c.slots_in_pool;
    if (slot >= a.c.slots_in_pool && a.status != nullptr && at == 0 && !is_v)
      atomicOr(a.status, 1);
    float d = 0.0f;
    uint32_t w[kN / 4] = {};
    if (have) {
      d = (is_v ? a.c.vd : a.c.kd)[scale_at(a.c, slot, h)];
      const int8_t* q = (is_v ? a.c.vq : a.c.kq) + code_at(a.c, slot, h) + e;
#pragma unroll
      for (int x = 0; x < kN / 4; ++x) w[x] = *reinterpret_cast<const uint32_t*>(q + 4 * x);
    }
    float v[kN];
#pragma unroll
    for (int x = 0; x < kN; ++x)
      v[x] = __fmul_rn((float)(int8_t)(w[x / 4] >> (8 * (x % 4))), d);
    uint4 o;
    if (kN == 4) {
      o = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                     __float_as_uint(v[3]));
    } else {
      uint32_t p[4];
#pragma unroll
      for (int x = 0; x < 4; ++x)
        p[x] = bf16_pair(v[(2 * x) % kN], v[(2 * x + 1) % kN]);
      o = make_uint4(p[0], p[1], p[2], p[3]);
    }
    *reinterpret_cast<uint4*>(out) = o;
  }
}

}  // namespace
}  // namespace memra

using namespace memra;

extern "C" memra_status memra_kv_plan(const int32_t* ctx_lens, const int32_t* new_lens, int64_t B,
                                      int64_t page_size, const int32_t* free_pages,
                                      int64_t n_free, const int32_t* free_head,
                                      int32_t* block_table, int64_t max_pages, int64_t T,
                                      int32_t* kv_lens, int32_t* cu_q, int32_t* slots,
                                      int32_t* positions, int32_t* free_head_out,
                                      int32_t* dev_status, cudaStream_t stream) {
  if (B < 0 || n_free < 0 || max_pages < 0 || T < 0) return MEMRA_ERR_INVALID_ARG;
  if (page_size < 16 || page_size % 16 != 0) return MEMRA_ERR_INVALID_ARG;
  if (page_size > MEMRA_MAX_KV_PAGE || T > INT32_MAX - 4 || B > (1 << 24) || n_free > INT32_MAX)
    return MEMRA_ERR_UNSUPPORTED;
  if (!cu_q || !free_head_out) return MEMRA_ERR_INVALID_ARG;
  if (B > 0 && (!ctx_lens || !new_lens || !kv_lens || (max_pages > 0 && !block_table)))
    return MEMRA_ERR_INVALID_ARG;
  if ((n_free > 0 && !free_pages) || (T > 0 && (!slots || !positions)))
    return MEMRA_ERR_INVALID_ARG;
  const void* all[] = {ctx_lens, new_lens, free_pages, free_head, block_table, kv_lens, cu_q,
                       slots, positions, free_head_out, dev_status};
  for (const void* p : all)
    if (!aligned(p, 4)) return MEMRA_ERR_ALIGNMENT;
  PlanArgs a;
  a.ctx = ctx_lens;
  a.add = new_lens;
  a.B = B;
  a.n_free = n_free;
  a.max_pages = max_pages;
  a.T = T;
  a.page = (int)page_size;
  a.free_pages = free_pages;
  a.free_head = free_head;
  a.table = block_table;
  a.kv_lens = kv_lens;
  a.cu_q = cu_q;
  a.slots = slots;
  a.positions = positions;
  a.free_head_out = free_head_out;
  a.status = dev_status;
  cudaError_t e;
  if (T <= kPlanFillRows) {
    e = launch_kernel(plan_kernel<true>, dim3(1), dim3(kPlanThreads), 0, stream, a);
    if (e != cudaSuccess) return cuda_fail(e);
    return MEMRA_OK;
  }
  e = launch_kernel(plan_kernel<false>, dim3(1), dim3(kPlanThreads), 0, stream, a);
  if (e != cudaSuccess) return cuda_fail(e);
  const int64_t blocks = (T + 1023) / 1024;
  e = launch_kernel(plan_fill_kernel, dim3((unsigned)blocks), dim3(256), 0, stream, a);
  if (e != cudaSuccess) return cuda_fail(e);
  return MEMRA_OK;
}

// Shared checks of the cache's sizes and planes.
static memra_status cache_args(int8_t* kq, float* kd, int8_t* vq, float* vd, int64_t n_pages,
                               int64_t Hkv, int64_t page_size, int64_t D, int64_t block,
                               CacheArgs* c) {
  if (n_pages < 0 || Hkv < 1) return MEMRA_ERR_INVALID_ARG;
  if (page_size < 16 || page_size % 16 != 0 || block < 1 || page_size % block != 0)
    return MEMRA_ERR_INVALID_ARG;
  if (D != 64 && D != 128 && D != 256) return MEMRA_ERR_UNSUPPORTED;
  if (page_size > MEMRA_MAX_KV_PAGE || Hkv > 65535 || n_pages > INT32_MAX / page_size)
    return MEMRA_ERR_UNSUPPORTED;
  if (n_pages > 0 && (!kq || !kd || !vq || !vd)) return MEMRA_ERR_INVALID_ARG;
  if (!aligned(kq, 16) || !aligned(vq, 16) || !aligned(kd, 4) || !aligned(vd, 4))
    return MEMRA_ERR_ALIGNMENT;
  c->kq = kq;
  c->vq = vq;
  c->kd = kd;
  c->vd = vd;
  c->slots_in_pool = n_pages * page_size;
  c->Hkv = (int)Hkv;
  c->page = (int)page_size;
  c->D = (int)D;
  c->block = (int)block;
  return MEMRA_OK;
}

extern "C" memra_status memra_kv_append_q8(const void* k, const void* v, int32_t dtype, int64_t T,
                                           int64_t stride_t, int64_t stride_h,
                                           const int32_t* slots, int8_t* kq, float* kd,
                                           int8_t* vq, float* vd, int64_t n_pages, int64_t Hkv,
                                           int64_t page_size, int64_t D, int64_t block,
                                           int32_t* dev_status, cudaStream_t stream) {
  if (T < 0 || stride_t < 0 || stride_h < 0) return MEMRA_ERR_INVALID_ARG;
  if (dtype != MEMRA_BF16 && dtype != MEMRA_F32) return MEMRA_ERR_INVALID_ARG;
  AppendArgs a;
  const memra_status st = cache_args(kq, kd, vq, vd, n_pages, Hkv, page_size, D, block, &a.c);
  if (st != MEMRA_OK) return st;
  if (T > INT32_MAX) return MEMRA_ERR_UNSUPPORTED;
  if (T == 0) return MEMRA_OK;
  if (!k || !v || !slots) return MEMRA_ERR_INVALID_ARG;
  const int per16 = dtype == MEMRA_BF16 ? 8 : 4;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 4) || !aligned(dev_status, 4) ||
      stride_t % per16 != 0 || stride_h % per16 != 0)
    return MEMRA_ERR_ALIGNMENT;
  DeviceInfo info;
  if (!device_info(&info)) return MEMRA_ERR_CUDA;
  a.k = k;
  a.v = v;
  a.slots = slots;
  a.T = T;
  a.stride_t = stride_t;
  a.stride_h = stride_h;
  a.status = dev_status;
  // A warp looks at one row where the rows leave warps to spare, at 16 of them otherwise
  // (most rows of a long run begin none).
  a.tile = T * 2 * Hkv <= (int64_t)info.sms * 64 ? 1 : 16;
  const int64_t items = (T + a.tile - 1) / a.tile * 2 * Hkv;
  const int64_t blocks = (items + kAppendWarps - 1) / kAppendWarps;
  if (blocks > INT32_MAX) return MEMRA_ERR_UNSUPPORTED;
  const dim3 grid((unsigned)blocks), threads(kAppendWarps * 32);
  const cudaError_t e = dtype == MEMRA_BF16
                            ? launch_kernel(append_kernel<uint16_t>, grid, threads, 0, stream, a)
                            : launch_kernel(append_kernel<float>, grid, threads, 0, stream, a);
  if (e != cudaSuccess) return cuda_fail(e);
  return MEMRA_OK;
}

extern "C" memra_status memra_kv_read_q8(const int32_t* slots, int64_t N, const int8_t* kq,
                                         const float* kd, const int8_t* vq, const float* vd,
                                         int64_t n_pages, int64_t Hkv, int64_t page_size,
                                         int64_t D, int64_t block, int32_t dtype, void* k, void* v,
                                         int32_t* dev_status, cudaStream_t stream) {
  if (N < 0) return MEMRA_ERR_INVALID_ARG;
  if (dtype != MEMRA_BF16 && dtype != MEMRA_F32) return MEMRA_ERR_INVALID_ARG;
  ReadArgs a;
  const memra_status st =
      cache_args(const_cast<int8_t*>(kq), const_cast<float*>(kd), const_cast<int8_t*>(vq),
                 const_cast<float*>(vd), n_pages, Hkv, page_size, D, block, &a.c);
  if (st != MEMRA_OK) return st;
  if (N > INT32_MAX) return MEMRA_ERR_UNSUPPORTED;
  if (N == 0) return MEMRA_OK;
  if (!slots || !k || !v) return MEMRA_ERR_INVALID_ARG;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 4) || !aligned(dev_status, 4))
    return MEMRA_ERR_ALIGNMENT;
  DeviceInfo info;
  if (!device_info(&info)) return MEMRA_ERR_CUDA;
  a.slots = slots;
  a.N = N;
  a.k = k;
  a.v = v;
  a.status = dev_status;
  const int64_t items = 2 * N * Hkv * (D / (dtype == MEMRA_BF16 ? 8 : 4));
  int64_t blocks = (items + 255) / 256;
  if (blocks > (int64_t)info.sms * 8) blocks = (int64_t)info.sms * 8;
  const dim3 grid((unsigned)blocks), threads(256);
  const cudaError_t e = dtype == MEMRA_BF16
                            ? launch_kernel(read_kernel<uint16_t>, grid, threads, 0, stream, a)
                            : launch_kernel(read_kernel<float>, grid, threads, 0, stream, a);
  if (e != cudaSuccess) return cuda_fail(e);
  return MEMRA_OK;
}
