// The paged 8-bit KV cache: the page plan of a step, the write of its tokens and their
// read-back.  Layouts and arithmetic are stated in memra.h.
#include <cuda_bf16.h>

#include "common.cuh"

namespace memra {
namespace {

// ---------------------------------------------------------------------------
// The page plan.  Every CTA sums the requests' rows and pages for itself, a chunk of its
// size at a time (two scans; the lengths come from L2, 8 bytes a request), and then fills
// its own share of the chunk's table entries and rows: a thread finds the request of its
// entry, or of its four rows, by bisection in shared memory.  Nothing passes between CTAs,
// so one launch does for any size, and what bounds it is latency: launch, one read of the
// lengths, two scans, one read of pages, one write.  4.3 us for 16 sequences of one token
// (a kernel that does nothing: 2.2), 8.2 us for 512 prompts, 328,486 slots (81 CTAs, the
// arithmetic pipe 56 % busy).
// ---------------------------------------------------------------------------
constexpr int kPlanThreads = 1024;

struct PlanArgs {
  const int32_t *ctx, *add;
  int64_t B, n_free, max_pages, T;
  int page;
  uint32_t pages_named;  // pages whose every slot is an int32
  const int32_t *free_pages, *free_head;
  int32_t *table, *kv_lens, *cu_q, *slots, *positions, *free_head_out, *status;
};

// Inclusive sum of v over the CTA's threads; *total receives the CTA's.
__device__ __forceinline__ int64_t scan(int64_t v, int64_t* warp_sum, int64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(kFullMask, v, o);
    if (lane >= o) v += u;
  }
  if (lane == 31) warp_sum[warp] = v;
  __syncthreads();
  // every warp sums the warps' totals for itself
  int64_t w = lane < warps ? warp_sum[lane] : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(kFullMask, w, o);
    if (lane >= o) w += u;
  }
  *total = __shfl_sync(kFullMask, w, 31);
  const int64_t before = __shfl_sync(kFullMask, w, (warp + 31) & 31);
  return warp > 0 ? v + before : v;
}

// Last i in [0, n) with a[i] <= x, given a[0] <= x (a ascending).
__device__ __forceinline__ int last_at_most(const int64_t* a, int n, int64_t x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

// kLater: *free_head_out and kv_lens alone, where they are the plan's own inputs and it has
// several CTAs (none of which may write what another still reads).  One CTA: a thread
// reads a request's lengths before it writes its new one.
template <bool kLater>
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(PlanArgs a) {
  __shared__ int64_t sum_a[32], sum_b[32];
  __shared__ int64_t first_row[kPlanThreads], first_page[kPlanThreads];
  __shared__ int32_t have_of[kPlanThreads], ctx_of[kPlanThreads];
  __shared__ uint32_t refused[kPlanThreads / 32];
  pdl_launch_dependents();
  pdl_wait();
  const int tid = threadIdx.x, threads = blockDim.x;
  const int cta = blockIdx.x, ctas = gridDim.x;
  int64_t head = a.free_head != nullptr ? *a.free_head : 0;
  if (head < 0) head = 0;
  int64_t row0 = 0, last_end = head;
  int bits = 0;
  bool no_page = false;
  if (!kLater && cta == 0 && tid == 0) a.cu_q[0] = 0;
  const bool wide = (((uintptr_t)a.slots | (uintptr_t)a.positions) & 15) == 0;
  for (int64_t base = 0; base < a.B; base += threads) {
    const int64_t b = base + tid;
    const int count = (int)min((int64_t)threads, a.B - base);
    const bool mine = b < a.B;
    int64_t ctx = mine ? a.ctx[b] : 0, add = mine ? a.add[b] : 0;
    bool fits = mine && ctx >= 0 && add >= 0;
    ctx = ctx < 0 ? 0 : ctx;
    add = add < 0 ? 0 : add;
    const int have = (int)((uint32_t)(ctx + a.page - 1) / (uint32_t)a.page);
    const int after = (int)((uint32_t)(ctx + add + a.page - 1) / (uint32_t)a.page);
    int64_t rows, pages;
    const int64_t upto = row0 + scan(add, sum_a, &rows);
    fits = fits && after <= a.max_pages && ctx + add <= INT32_MAX && upto <= a.T;
    const int64_t need = fits ? after - have : 0;
    const int64_t end = head + scan(need, sum_b, &pages);
    const bool ok = fits && (need == 0 || end <= a.n_free);
    if (ok && need > 0) last_end = end;  // those that take pages come before those refused them
    if (mine && !fits) bits |= 1;
    if (fits && !ok) bits |= 4;
    if (mine && cta == 0 && a.kv_lens != nullptr) a.kv_lens[b] = ok ? (int32_t)(ctx + add) : 0;
    if (!kLater) {
      first_row[tid] = min(upto - add, a.T);
      first_page[tid] = end - need;
      have_of[tid] = have;
      ctx_of[tid] = (int32_t)ctx;
      const uint32_t no = __ballot_sync(kFullMask, !ok);
      if ((tid & 31) == 0) refused[tid >> 5] = no;
      if (mine && cta == 0) a.cu_q[b + 1] = (int32_t)min(upto, a.T);
      __syncthreads();
      // new table entries: pages head .. of the chunk that the free list holds
      const int64_t last = min(head + pages, a.n_free);
      for (int64_t p = head + (int64_t)cta * threads + tid; p < last; p += (int64_t)ctas * threads) {
        const int r = last_at_most(first_page, count, p);
        if (!((refused[r >> 5] >> (r & 31)) & 1u))
          a.table[(base + r) * a.max_pages + have_of[r] + (p - first_page[r])] = a.free_pages[p];
      }
      // rows, four neighbours to a thread
      const int64_t from = min(row0, a.T), to = min(row0 + rows, a.T);
      for (int64_t t0 = from / 4 * 4 + ((int64_t)cta * threads + tid) * 4; t0 < to;
           t0 += (int64_t)ctas * threads * 4) {
        const int64_t lo = max(t0, from), hi = min(t0 + 4, to);
        int r = last_at_most(first_row, count, lo);
        int32_t slot[4], pos[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int64_t t = t0 + i;
          slot[i] = pos[i] = -1;
          if (t < lo || t >= hi) continue;
          while (r + 1 < count && first_row[r + 1] <= t) ++r;
          const uint32_t at = (uint32_t)ctx_of[r] + (uint32_t)(t - first_row[r]);
          pos[i] = (int32_t)at;
          if ((refused[r >> 5] >> (r & 31)) & 1u) continue;
          const int p = (int)(at / (uint32_t)a.page);
          const uint32_t page = p < have_of[r] ? a.table[(base + r) * a.max_pages + p]
                                              : a.free_pages[first_page[r] + (p - have_of[r])];
          const bool named = page < a.pages_named;
          no_page |= !named;
          slot[i] = named ? (int32_t)(page * (uint32_t)a.page + (at - (uint32_t)p * (uint32_t)a.page)) : -1;
        }
        if (wide && hi - lo == 4) {
          *reinterpret_cast<int4*>(a.slots + t0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
          *reinterpret_cast<int4*>(a.positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (t0 + i >= lo && t0 + i < hi) {
              a.slots[t0 + i] = slot[i];
              a.positions[t0 + i] = pos[i];
            }
        }
      }
    }
    head += pages;
    row0 += rows;
    __syncthreads();
  }
  if (!kLater)
    for (int64_t t = min(row0, a.T) + (int64_t)cta * threads + tid; t < a.T; t += (int64_t)ctas * threads) {
      a.slots[t] = -1;
      a.positions[t] = -1;
    }
  if (cta == 0 && a.free_head_out != nullptr) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) last_end = max(last_end, (int64_t)__shfl_xor_sync(kFullMask, last_end, o));
    if ((tid & 31) == 0) sum_a[tid >> 5] = last_end;
    __syncthreads();
    if (tid == 0) {
      for (int w = 1; w < threads / 32; ++w) last_end = max(last_end, sum_a[w]);
      *a.free_head_out = (int32_t)last_end;
    }
  }
  if (cta != 0) bits = 0;
  if (no_page) bits |= 1;
  if (!kLater && bits != 0 && a.status != nullptr) atomicOr(a.status, bits);
}

// ---------------------------------------------------------------------------
// The write.  A warp takes one run of tokens (one scale block) of one head and plane: the
// run's largest magnitude first, then the older tokens' codes if the scale grew, then the
// run's own codes.  A lane holds 16 bytes of input at a time, and a run of up to eight
// such pieces a lane (16 tokens of 128 bf16) stays in registers between the two passes.
// Latency bounds the small calls (one token of 8 heads and its read-back: 3.8 us).  8191 bf16
// tokens of 8 heads (34 MB in, 17 out) take 12.2 us, where their bytes need 7.4 and their
// instructions 6.2: neither is at its rate in so short a call.  32000 take 34.3, 85 % of the
// copy rate; in fp32 19.7 us (12.4) and 62.1 (48.3).
// ---------------------------------------------------------------------------
constexpr int kAppendWarps = 4;

struct CacheArgs {
  int8_t *kq, *vq;
  float *kd, *vd;
  int64_t slots_in_pool;
  int Hkv, page, D, block;
  Divider by_page, by_block;
};

struct AppendArgs {
  CacheArgs c;
  const void *k, *v;
  const int32_t* slots;
  int64_t T, stride_t, stride_h;
  int tile;
  int32_t* status;
};

template <typename T>
struct Vec;  // 16 bytes of input
template <>
struct Vec<float> {
  static constexpr int kN = 4;
  static __device__ __forceinline__ void unpack(const uint4& u, float* v) {
    v[0] = __uint_as_float(u.x); v[1] = __uint_as_float(u.y);
    v[2] = __uint_as_float(u.z); v[3] = __uint_as_float(u.w);
  }
  struct Largest {  // the largest magnitude of the pieces taken
    float m = 0.0f;
    __device__ __forceinline__ void take(const uint4& u) {
      m = fmaxf(fmaxf(m, fmaxf(fabsf(__uint_as_float(u.x)), fabsf(__uint_as_float(u.y)))),
                fmaxf(fabsf(__uint_as_float(u.z)), fabsf(__uint_as_float(u.w))));
    }
    __device__ __forceinline__ float value() const { return m; }
  };
};
template <>
struct Vec<uint16_t> {
  static constexpr int kN = 8;
  static __device__ __forceinline__ void unpack(const uint4& u, float* v) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  struct Largest {
    uint32_t m = 0;  // two bf16
    __device__ __forceinline__ void take(const uint4& u) {
      m = most(m, most(most(u.x & 0x7fff7fffu, u.y & 0x7fff7fffu), most(u.z & 0x7fff7fffu, u.w & 0x7fff7fffu)));
    }
    static __device__ __forceinline__ uint32_t most(uint32_t a, uint32_t b) {
      const __nv_bfloat162 x = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&a),
                                       *reinterpret_cast<const __nv_bfloat162*>(&b));
      return *reinterpret_cast<const uint32_t*>(&x);
    }
    __device__ __forceinline__ float value() const {
      return fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
    }
  };
};

// Codes of kN values with scale d, the integers of quant_value: v * inv with inv = 1 / d
// rounded, corrected once by its remainder, is the IEEE quotient (Markstein, "Computation
// of elementary functions on the IBM RISC System/6000 processor", 1990; no underflow for
// d above 1e-30 but where the code is 0 anyway), and a half added towards its sign and cut
// off rounds halves away from zero.  A bf16 value is often an exact half of its block's
// scale, so a shortcut that leaves halves to a division would take it all the time.
template <int kN>
__device__ __forceinline__ void codes_of(const float* v, float d, float inv, uint32_t* out) {
  uint32_t y[kN];
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    float q = __fmul_rn(v[i], inv);
    q = __fmaf_rn(__fmaf_rn(-q, d, v[i]), inv, q);
    y[i] = (uint32_t)__float2int_rz(__fadd_rz(q, copysignf(0.5f, q)));
  }
#pragma unroll
  for (int i = 0; i < kN; i += 4)
    out[i / 4] = __byte_perm(__byte_perm(y[i], y[i + 1], 0x0040), __byte_perm(y[i + 2], y[i + 3], 0x0040), 0x5410);
}

template <typename T, int kD>
__global__ void __launch_bounds__(kAppendWarps * 32, 8) append_kernel(AppendArgs a) {
  constexpr int kN = Vec<T>::kN;
  constexpr int kLanes = kD / kN;                       // 16-byte pieces of a row
  constexpr int kStepRows = kLanes < 32 ? 32 / kLanes : 1;
  constexpr int kPieces = kLanes < 32 ? 1 : kLanes / 32;
  constexpr int kHeld = 8 / kPieces;                    // steps of a run that stay in registers
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  // grid: x tiles of rows, y planes
  const int64_t t0 = ((int64_t)blockIdx.x * kAppendWarps + (threadIdx.x >> 5)) * a.tile;
  if (t0 >= a.T) return;
  const bool is_v = blockIdx.y & 1;
  const int h = (int)(blockIdx.y >> 1);
  // Slots of rows t0 - 1 .. t0 + 30, one a lane; blk: which scale block, -1 for none.
  const uint32_t S = a.c.block;
  const int64_t row = t0 - 1 + lane;
  const int32_t slot = row >= 0 && row < a.T ? a.slots[row] : -1;
  const bool beyond = slot >= a.c.slots_in_pool;
  int32_t blk = slot >= 0 && !beyond ? (int32_t)a.c.by_block((uint32_t)slot) : -1;
  const int32_t blk_before = __shfl_up_sync(kFullMask, blk, 1);
  const bool in_tile = lane >= 1 && lane <= a.tile;
  if (beyond && in_tile && blockIdx.y == 0 && a.status != nullptr) atomicOr(a.status, 1);
  uint32_t leaders = __ballot_sync(kFullMask, in_tile && blk >= 0 && blk != blk_before);

  const int lane_row = kLanes < 32 ? lane / kLanes : 0;
  const T* x = static_cast<const T*>(is_v ? a.v : a.k) + (lane % kLanes) * kN;
  int8_t* planes_codes = is_v ? a.c.vq : a.c.kq;
  float* planes_scales = is_v ? a.c.vd : a.c.kd;
  for (; leaders != 0; leaders &= leaders - 1) {
    const int lead = __ffs(leaders) - 1;
    const int32_t my_blk = __shfl_sync(kFullMask, blk, lead);
    const uint32_t my_slot = (uint32_t)__shfl_sync(kFullMask, slot, lead);
    const int first = (int)(my_slot - (uint32_t)my_blk * S);
    const int64_t t = t0 - 1 + lead;
    // the run: rows of the same block that follow, at most to the block's end
    const uint32_t same = __ballot_sync(kFullMask, blk == my_blk) >> lead;
    int n = __ffs(~same) - 1;
    n = n < 0 ? 32 : n;
    if (n == 32 - lead)  // it reaches the last row looked at
      while (t + n < a.T && first + n < (int)S) {
        const int64_t next = a.slots[t + n];
        if (next < 0 || next >= a.c.slots_in_pool || a.c.by_block((uint32_t)next) != (uint32_t)my_blk) break;
        ++n;
      }
    n = min(n, (int)S - first);
    const uint32_t page = a.c.by_page(my_slot);
    const uint32_t off = my_slot - page * (uint32_t)a.c.page;
    const uint32_t block_in_page = a.c.by_block(off);
    const T* rows = x + t * a.stride_t + h * a.stride_h;
    const int64_t head = (int64_t)page * a.c.Hkv + h;
    float* scale = planes_scales + head * (a.c.page / (int)S) + block_in_page;
    int8_t* block_codes = planes_codes + (head * a.c.page + off - first) * kD;
    const float d_old = first > 0 ? *scale : 0.0f;

    uint4 held[kHeld][kPieces];
    typename Vec<T>::Largest largest;
#pragma unroll
    for (int s = 0; s < kHeld; ++s)
#pragma unroll
      for (int p = 0; p < kPieces; ++p) {
        const int r = s * kStepRows + lane_row;
        held[s][p] = r < n ? *reinterpret_cast<const uint4*>(rows + r * a.stride_t + p * 32 * kN)
                           : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
    for (int s = 0; s < kHeld; ++s)
#pragma unroll
      for (int p = 0; p < kPieces; ++p) largest.take(held[s][p]);
    for (int r = kHeld * kStepRows + lane_row; r < n; r += kStepRows)
#pragma unroll
      for (int p = 0; p < kPieces; ++p)
        largest.take(*reinterpret_cast<const uint4*>(rows + r * a.stride_t + p * 32 * kN));
    float amax = largest.value();
    amax = __uint_as_float(__reduce_max_sync(kFullMask, __float_as_uint(amax)));
    // a scale of either sign stays until its magnitude has to grow (one that is no number is
    // replaced)
    const float least = amax / 127.0f;
    const bool grows = !(least <= fabsf(d_old));
    const float d = grows ? least : d_old;

    if (first > 0 && grows) {
      const float ratio = d_old / d;
      for (int i = lane * 4; i < first * kD; i += 128) {
        const char4 q = *reinterpret_cast<const char4*>(block_codes + i);
        char4 r;
        r.x = (signed char)(int)roundf(__fmul_rn((float)q.x, ratio));
        r.y = (signed char)(int)roundf(__fmul_rn((float)q.y, ratio));
        r.z = (signed char)(int)roundf(__fmul_rn((float)q.z, ratio));
        r.w = (signed char)(int)roundf(__fmul_rn((float)q.w, ratio));
        *reinterpret_cast<char4*>(block_codes + i) = r;
      }
    }
    int8_t* to = block_codes + (int64_t)first * kD + (lane % kLanes) * kN;
    auto write = [&](int r, int p, const uint32_t* w) {
      int8_t* dst = to + (int64_t)r * kD + p * 32 * kN;
      if (kN == 8) *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[kN / 4 - 1]);
      else *reinterpret_cast<uint32_t*>(dst) = w[0];
    };
    float v[kN];
    uint32_t w[kN / 4];
    if (fabsf(d) > 1e-30f) {
      const float inv = 1.0f / d;
#pragma unroll
      for (int s = 0; s < kHeld; ++s) {
        const int r = s * kStepRows + lane_row;
#pragma unroll
        for (int p = 0; p < kPieces; ++p)
          if (r < n) {
            Vec<T>::unpack(held[s][p], v);
            codes_of<kN>(v, d, inv, w);
            write(r, p, w);
          }
      }
#pragma unroll 1
      for (int r = kHeld * kStepRows + lane_row; r < n; r += kStepRows)
#pragma unroll
        for (int p = 0; p < kPieces; ++p) {
          Vec<T>::unpack(*reinterpret_cast<const uint4*>(rows + r * a.stride_t + p * 32 * kN), v);
          codes_of<kN>(v, d, inv, w);
          write(r, p, w);
        }
    } else {  // zeros, or next to nothing: divide
#pragma unroll 1
      for (int r = lane_row; r < n; r += kStepRows)
#pragma unroll 1
        for (int p = 0; p < kPieces; ++p) {
          Vec<T>::unpack(*reinterpret_cast<const uint4*>(rows + r * a.stride_t + p * 32 * kN), v);
#pragma unroll
          for (int j = 0; j < kN; j += 4)
            w[j / 4] = pack4(quant_value(v[j], d), quant_value(v[j + 1], d), quant_value(v[j + 2], d),
                             quant_value(v[j + 3], d));
          write(r, p, w);
        }
    }
    if (lane == 0) *scale = d;
  }
}

// ---------------------------------------------------------------------------
// The read-back: a lane takes 16 bytes of output at a time.  Its bytes bound it, or the wait for
// them: 8191 bf16 tokens of 8 heads take 8.8 us (bytes alone 7.4), 32000 37.9 (29.0), in fp32
// 16.7 (12.4) and 63.4 (48.3).
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

constexpr int kReadWarps = 8;
constexpr int kReadPieces = 4;  // 16-byte pieces of output a lane

// A warp takes 128 pieces of the K or V rows of one token (all heads lie one after another in
// the output).  Several tokens to a warp are slower at every size (4 x 8000 tokens of 8
// heads, with their write: 70.6 us, with two a warp 79.7, with four 89.8).
template <typename T>
__global__ void __launch_bounds__(kReadWarps * 32) read_kernel(ReadArgs a, int head_bits) {
  constexpr int kN = Vec<T>::kN;
  pdl_launch_dependents();
  pdl_wait();
  // grid: x tokens, y K or V, z 128 pieces
  const int64_t n = (int64_t)blockIdx.x * kReadWarps + (threadIdx.x >> 5);
  if (n >= a.N) return;
  const bool is_v = blockIdx.y;
  const int lane = threadIdx.x & 31;
  const int total = a.c.Hkv << head_bits;  // pieces of a row, 2^head_bits of a head
  const int blocks = (int)a.c.by_block((uint32_t)a.c.page);
  const int32_t slot = a.slots[n];
  const bool have = slot >= 0 && slot < a.c.slots_in_pool;
  if (slot >= a.c.slots_in_pool && a.status != nullptr && lane == 0) atomicOr(a.status, 1);
  const uint32_t page = have ? a.c.by_page((uint32_t)slot) : 0;
  const uint32_t off = have ? (uint32_t)slot - page * (uint32_t)a.c.page : 0;
  const int64_t head0 = (int64_t)page * a.c.Hkv;
  const int8_t* q0 = (is_v ? a.c.vq : a.c.kq) + (head0 * a.c.page + off) * a.c.D;
  const float* d0 = (is_v ? a.c.vd : a.c.kd) + head0 * blocks + a.c.by_block(off);
  float d[kReadPieces];
  uint2 w[kReadPieces];
#pragma unroll
  for (int i = 0; i < kReadPieces; ++i) {
    const int piece = (int)blockIdx.z * (32 * kReadPieces) + i * 32 + lane;
    d[i] = 0.0f;
    w[i] = make_uint2(0, 0);
    if (have && piece < total) {
      const int h = piece >> head_bits, e = (piece & ((1 << head_bits) - 1)) * kN;
      const int8_t* q = q0 + (int64_t)h * a.c.page * a.c.D + e;
      d[i] = d0[h * blocks];
      if (kN == 8) w[i] = *reinterpret_cast<const uint2*>(q);
      else w[i].x = *reinterpret_cast<const uint32_t*>(q);
    }
  }
  T* out = static_cast<T*>(is_v ? a.v : a.k);
#pragma unroll
  for (int i = 0; i < kReadPieces; ++i) {
    const int piece = (int)blockIdx.z * (32 * kReadPieces) + i * 32 + lane;
    if (piece >= total) continue;
    // a code q as the float 2^23 + 128 + q (its byte under that exponent), less 2^23 + 128
    const uint32_t raised[2] = {w[i].x ^ 0x80808080u, w[i].y ^ 0x80808080u};
    float v[8];
#pragma unroll
    for (int x = 0; x < kN; ++x)
      v[x] = __fmul_rn(__fsub_rn(__uint_as_float(__byte_perm(raised[x / 4], 0x4b000000u, 0x7440 | (x % 4))),
                                 8388736.0f), d[i]);
    uint4 o;
    if (kN == 4)
      o = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                     __float_as_uint(v[3]));
    else
      o = make_uint4(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[4], v[5]),
                     bf16_pair(v[6], v[7]));
    *reinterpret_cast<uint4*>(out + (n * total + piece) * kN) = o;
  }
}

template <typename T>
cudaError_t launch_read(const ReadArgs& a, int head_bits, unsigned groups, cudaStream_t stream) {
  const dim3 grid((unsigned)((a.N + kReadWarps - 1) / kReadWarps), 2, groups);
  return launch_kernel(read_kernel<T>, grid, dim3(kReadWarps * 32), 0, stream, a, head_bits);
}

template <typename T>
cudaError_t launch_append(const AppendArgs& a, dim3 grid, cudaStream_t stream) {
  const dim3 block(kAppendWarps * 32);
  if (a.c.D == 64) return launch_kernel(append_kernel<T, 64>, grid, block, 0, stream, a);
  if (a.c.D == 128) return launch_kernel(append_kernel<T, 128>, grid, block, 0, stream, a);
  return launch_kernel(append_kernel<T, 256>, grid, block, 0, stream, a);
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
  // What is written lies apart from all else, but for lengths and the free list's position
  // that advance in place.
  struct Span {
    const int32_t* at;
    int64_t words;
    bool meets(const Span& o) const {
      const uintptr_t a = (uintptr_t)at, b = (uintptr_t)o.at;
      return words > 0 && o.words > 0 && a < b + 4 * (uint64_t)o.words && b < a + 4 * (uint64_t)words;
    }
  };
  const int64_t row = max_pages < INT32_MAX ? max_pages : INT32_MAX;
  const Span in[] = {{ctx_lens, B}, {new_lens, B}, {free_head, free_head != nullptr}, {free_pages, n_free}};
  const Span out[] = {{kv_lens, B}, {free_head_out, 1}, {cu_q, B + 1}, {slots, T}, {positions, T},
                      {block_table, B * row}, {dev_status, dev_status != nullptr}};
  const bool lens_in_place = B > 0 && (kv_lens == ctx_lens || kv_lens == new_lens);
  const bool head_in_place = free_head == free_head_out;
  for (int i = 0; i < 7; ++i) {
    for (int j = 0; j < 4; ++j) {
      const bool in_place = out[i].at == in[j].at && ((i == 0 && j < 2) || (i == 1 && j == 2));
      if (!in_place && out[i].meets(in[j])) return MEMRA_ERR_INVALID_ARG;
    }
    for (int j = 0; j < i; ++j)
      if (out[i].meets(out[j])) return MEMRA_ERR_INVALID_ARG;
  }
  PlanArgs a;
  a.ctx = ctx_lens;
  a.add = new_lens;
  a.B = B;
  a.n_free = n_free;
  a.max_pages = max_pages;
  a.T = T;
  a.page = (int)page_size;
  a.pages_named = (uint32_t)(INT32_MAX / page_size);
  a.free_pages = free_pages;
  a.free_head = free_head;
  a.table = block_table;
  a.kv_lens = kv_lens;
  a.cu_q = cu_q;
  a.slots = slots;
  a.positions = positions;
  a.free_head_out = free_head_out;
  a.status = dev_status;
  DeviceInfo info;
  if (!device_info(&info)) return MEMRA_ERR_CUDA;
  // A CTA for every 4096 rows, up to one an SM; small plans take a small CTA, whose barriers
  // cost less.
  const bool small = B <= 256 && T <= 1024;
  int64_t ctas = (T + 4 * kPlanThreads - 1) / (4 * kPlanThreads);
  ctas = ctas < 1 ? 1 : (ctas > info.sms ? info.sms : ctas);
  const bool later = ctas > 1 && (lens_in_place || head_in_place);
  if (later && lens_in_place) a.kv_lens = nullptr;
  if (later && head_in_place) a.free_head_out = nullptr;
  cudaError_t e = launch_kernel(plan_kernel<false>, dim3((unsigned)ctas),
                                dim3(small ? 256 : kPlanThreads), 0, stream, a);
  if (e == cudaSuccess && later) {
    a.kv_lens = lens_in_place ? kv_lens : nullptr;
    a.free_head_out = head_in_place ? free_head_out : nullptr;
    e = launch_kernel(plan_kernel<true>, dim3(1), dim3(kPlanThreads), 0, stream, a);
  }
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
  if (page_size > MEMRA_MAX_KV_PAGE || Hkv > 32767 || n_pages > INT32_MAX / page_size)
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
  c->by_page = Divider((uint32_t)page_size);
  c->by_block = Divider((uint32_t)block);
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
  // (most rows of a long run begin none).  Taking several heads in one warp, to look at the
  // slots once, was slower (8191 rows: 31 us with four heads, 30 with one).
  a.tile = T * 2 * Hkv <= (int64_t)info.sms * 64 ? 1 : 16;
  const int64_t tiles = (T + a.tile - 1) / a.tile;
  const dim3 grid((unsigned)((tiles + kAppendWarps - 1) / kAppendWarps), (unsigned)(2 * Hkv));
  const cudaError_t e = dtype == MEMRA_BF16 ? launch_append<uint16_t>(a, grid, stream)
                                            : launch_append<float>(a, grid, stream);
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
  a.slots = slots;
  a.N = N;
  a.k = k;
  a.v = v;
  a.status = dev_status;
  int head_bits = 0;
  while ((1 << head_bits) < D / (dtype == MEMRA_BF16 ? 8 : 4)) ++head_bits;
  const int64_t pieces = Hkv << head_bits;
  const int64_t groups = (pieces + 32 * kReadPieces - 1) / (32 * kReadPieces);
  if (groups > 65535) return MEMRA_ERR_UNSUPPORTED;
  const cudaError_t e = dtype == MEMRA_BF16
                            ? launch_read<uint16_t>(a, head_bits, (unsigned)groups, stream)
                            : launch_read<float>(a, head_bits, (unsigned)groups, stream);
  if (e != cudaSuccess) return cuda_fail(e);
  return MEMRA_OK;
}
