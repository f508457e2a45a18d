// Attention over the paged 8-bit KV cache (layouts and arithmetic in memra.h).
//
// The work list is that of kv_attention.cuh.  The cut ends of a unit leave (maximum, sum,
// weighted values) in the workspace, and the CTA that arrives last at the unit joins them
// in the order of the keys, so results do not depend on timing.
//
// A CTA's eight warps take strips of 16 keys in turn, each with its own ring of
// cp.async stages and its own running statistics; nothing in the loop crosses warps.
// A strip is two products on the tensor cores with the keys (dims) in the 16-row operand,
// so that 8 query rows waste nothing:
//   S^T [16 keys x 8 rows]  = K [16 x D] * Q^T,   O^T [D x 8 rows] += V^T [D x 16] * P^T.
// An int8 code c becomes an fp16 operand exactly: the byte c + 128 (one xor) under the
// exponent of 1024 is 1024 + 128 + c, and an fp16 subtraction leaves c.  (Taking the byte
// as it is, for the subnormal (c + 128) * 2^-24, and the 128 out of the sums saves the
// subtraction but no time (130k keys 52.1 us so, 52.1 with it), and leaves an error of the
// 128's own size: ten times as much in the log-sum, 2^-14 of the scale in the result.)
// Scales never meet the codes: kd multiplies the score, vd the weight.
//
// The tensor cores cut their fp32 sums off, so a sum over V that stayed in them would lose
// up to 2^-23 of itself with each product, always to the same side (7e-5 after the 1024
// strips that a warp has of 131072 keys).  A strip's products therefore start from zero,
// and its sums are added to the running ones in registers, rounded to nearest: no loss
// for 8 bf16 rows (52.1 us for 52.2 at 130k), 31.4 us for 29.2 of the 16 fp32 sequences.
//
// One token of one sequence of 130k (40 heads on 8, D 128) takes 52.0 us, 5.1 TB/s of codes
// and scales: about 10 us are fixed (launch, the list, first copies, the join of a unit's
// parts), and the strips keep the arithmetic pipe 50 % busy beside memory's 55 %.  16
// sequences of 37 to 16000 tokens, fp32: 31.4 us, 3.2 TB/s (twice the products); nothing is
// near its rate there (memory 35 %, arithmetic pipe 36 %, tensor pipe 17 %), and the first
// reason why a warp waits is that its next instruction has not been fetched.
#include <atomic>

#include "kv_attention.cuh"

namespace memra {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
static_assert(kWarps * kStrip == kTile, "a CTA's step is an entry of the list");
constexpr int kUnitCost = 3;   // entries of the list for a unit's fixed time (1: 36.8 us, 3: 31.5, 6:
                               // 33.1 for 16 sequences of 37 to 16000 tokens, fp32)
// Above this many rows to a unit, and with at least so many in all (rows times heads), the
// tcgen05 kernel takes bf16 queries: below, its larger parts and ends of units cost more than
// its products save.  8 cached heads of 128, us here / there: 32 rows, 16 requests of 500 to
// 8000 tokens 64 / 69, 64 of 500 to 3000 121 / 141; 48 rows, 16 requests 104 / 70; 64 rows, 8
// requests (4096 in all) 64 / 44, 4 (2048) 41 / 35, 2 (1024) 32 / 31, one of 8000 (512) 31 / 33;
// 128 rows, one of 16000 (1024) 64 / 55; 256 rows, one of 8000 (2048) 62 / 45; 64 rows, 32
// requests of 100 to 500 56 / 36.  Heads of 64, in the same order: 46 / 49, 88 / 101, 74 / 50,
// 46 / 32, 30 / 26, 24 / 24, 23 / 25, 44 / 41, 44 / 34, 40 / 28.
constexpr int kWideRows = 32, kWideAll = 1024;
// Where the reference for scales of V starts: 2^8 over it is an fp32 number, which 2^8 over
// a scale below 7.6e-37 is not.  Smaller scales are next to nothing.
constexpr float kLeastRef = 0x1p-115f;
constexpr int kMaxParts = 64;  // CTAs to a unit, on average (32: 57.0 us, 64 and 128: 52.0 for one
                               // sequence of 130k)

__device__ __forceinline__ void mma_16816(float c[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same from zero: c is written only.
__device__ __forceinline__ void mma_16816_zero(float c[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                               uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

__device__ __forceinline__ void add4(float c[4], const float a[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] += a[i];
}

// Codes 0 and 2 (1 and 3) of w as two fp16: the byte under the exponent of 1024 is 1024 + 128 + code.
__device__ __forceinline__ uint32_t minus_1152(uint32_t h) {
  const __half2 v = __hsub2(*reinterpret_cast<const __half2*>(&h), __half2half2(__ushort_as_half(0x6480)));
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t even_bytes(uint32_t w) {
  return minus_1152((w & 0x00ff00ffu) ^ 0x64806480u);
}
__device__ __forceinline__ uint32_t odd_bytes(uint32_t w) {
  return minus_1152(((w >> 8) & 0x00ff00ffu) ^ 0x64806480u);
}

__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float2 unpack_half(uint32_t h) {
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

// Which key of 8 sits in operand row i.  With 128-byte rows and more, keys i and i + 1 of a
// 16-byte load's quarter-warp have to differ in bit 2 for the swizzle below to part them.
template <int kD>
__device__ __forceinline__ int key_of(int i) {
  return kD == 64 ? i : (i >> 1) | ((i & 1) << 2);
}
// Byte offset of 16-byte chunk c of key k (0..15) in a stage's K or V part.
template <int kD>
__device__ __forceinline__ uint32_t k_place(int k, int c) {
  if (kD == 64) return k * 64 + c * 16;
  return k * kD + ((c ^ (k & 7)) << 4);
}
template <int kD>
__device__ __forceinline__ uint32_t v_place(int k, int c) {
  if (kD == 64)  // two keys to a 128-byte line
    return (k >> 1) * 128 + (((((k & 1) << 2) | c) ^ (((k >> 1) & 3) << 1)) << 4);
  return k * kD + ((c ^ (((k & 3) << 1) | ((k >> 2) & 1))) << 4);
}

template <typename T>
struct Row;  // 16 bytes of a query row
template <>
struct Row<uint16_t> {
  static constexpr bool kPair = false;  // bf16 has 8 significant bits: one fp16 holds them
};
template <>
struct Row<float> {
  static constexpr bool kPair = true;   // fp32: two fp16, 22 bits
};
template <typename T, int kD, int kNT>
struct Shape {
  static constexpr int kRows = 8 * kNT;
  static constexpr bool kPair = Row<T>::kPair;
  // CTAs of an SM: two where 128 registers hold the rows' sums, else one with 255 (16
  // sequences of 500 to 8000 tokens, two CTAs / one: 16 bf16 rows of 128 32.8 / 26.4 us, fp32
  // 37.7 / 28.4; 32 bf16 rows of 64 40.1 / 28.0; but 8 fp32 rows of 128 31.2 / 33.4).
  static constexpr int kCtas = kNT * kD <= 128 ? 2 : 1;
  static constexpr int kStage = 2 * kStrip * kD + 8 * kStrip;  // K, V, 16 kd, 16 vd
  static constexpr int kStages = kD == 64 ? 5 : (kCtas == 2 ? 3 : (kD == 128 ? 6 : 3));
  static constexpr int kRing = kWarps * kStages * kStage;
  static constexpr int kJoin = kWarps * kRows * kD * 4;  // reuses the ring
  static constexpr int kBig = kRing > kJoin ? kRing : kJoin;
  static constexpr int kQ = (kPair ? 2 : 1) * (kD / 16) * kNT * 32 * 8;
  static constexpr int kStats = (2 * kWarps + 4) * kRows * 4;
  static constexpr int kSmem = kBig + kQ + kStats;
};

// What a CTA keeps in shared memory while its strips want the registers: where it stands in
// the list, and the unit at hand.
struct Unit {
  int h, row0, rows, token0;
  int first_cta, parts;  // CTAs that hold a part of it
  int begins, whole;
};

template <typename T, int kD, int kNT>
__global__ void __launch_bounds__(kThreads, (Shape<T, kD, kNT>::kCtas)) attention_kernel(AttnArgs a) {
  using Sh = Shape<T, kD, kNT>;
  constexpr int kRows = Sh::kRows;
  constexpr bool kPair = Sh::kPair;
  constexpr int kSteps = kD / 16;          // k16 steps of S, m16 tiles of O
  const float kInf = __int_as_float(0x7f800000);
  extern __shared__ __align__(128) uint8_t smem[];
  uint8_t* ring = smem;
  uint2* q_frag = reinterpret_cast<uint2*>(smem + Sh::kBig);  // [hi, lo][step][tile][lane]
  float* stats = reinterpret_cast<float*>(smem + Sh::kBig + Sh::kQ);
  float* warp_m = stats;                       // [kWarps][kRows]
  float* warp_l = warp_m + kWarps * kRows;     // [kWarps][kRows]
  float* row_m = warp_l + kWarps * kRows;      // [kRows]
  float* row_l = row_m + kRows;
  float* row_scale = row_l + kRows;
  int* row_limit = reinterpret_cast<int*>(row_scale + kRows);
  __shared__ int last_part;
  __shared__ Walk walk;
  __shared__ Unit unit_at_hand;

  pdl_launch_dependents();
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t4 = lane & 3;
  const int cta = blockIdx.x;

  int ctas;
  int64_t total;
  if (!locate<T, kD, kRows, kUnitCost, kThreads>(a, &walk, &ctas, &total)) return;

  const uint32_t my_ring = smem_addr(ring) + warp * Sh::kStages * Sh::kStage;
  // Lane constants of the ring: where this lane's 16 bytes of a copy go (row i * 512 bytes
  // further on differs by a constant exclusive-or in bits 4..6), and where it reads.
  constexpr int kChunks = kD / 16;
  const uint32_t k_dst = k_place<kD>(lane / kChunks, lane % kChunks);
  const uint32_t v_dst = kStrip * kD + v_place<kD>(lane / kChunks, lane % kChunks);
  const int ka = key_of<kD>(g), kb = 8 + ka;
  const uint32_t k_src = k_place<kD>(ka, t4);
  const int vk0 = key_of<kD>(2 * t4), vk1 = key_of<kD>(2 * t4 + 1);
  const uint32_t v_src0 = kStrip * kD + (kD == 64 ? v_place<kD>(vk0, g >> 1) + (g & 1) * 8 : v_place<kD>(vk0, g));
  const uint32_t v_src1 = kStrip * kD + (kD == 64 ? v_place<kD>(vk1, g >> 1) + (g & 1) * 8 : v_place<kD>(vk1, g));
  const int64_t v_minus_k = a.vq - a.kq;

  for (;;) {
    __syncthreads();  // the ring, the queries and the statistics are free again
    const int64_t x = walk.x, stop = walk.stop;
    if (x >= stop) break;
    int64_t at = walk.at;
    int b = walk.b;
    Request req = walk.req;
    int64_t w = entries_of<kUnitCost>(a, req);
    while (x >= at + w) {
      at += w;
      req = request_of<kRows>(a, ++b);
      w = entries_of<kUnitCost>(a, req);
    }
    // ---- this unit: cached head h, rows [row0, row0 + kRows) of the request's n * G ----
    const int unit_size = req.tiles + kUnitCost;
    const int unit = (int)Cut::divide(x - at, unit_size);
    const int64_t unit_at = at + (int64_t)unit * unit_size;
    const int64_t unit_stop = unit_at + unit_size;
    const int64_t x_stop = unit_stop < stop ? unit_stop : stop;
    const int tile0 = max((int)(x - unit_at) - kUnitCost, 0);
    const int tile1 = (int)(x_stop - unit_at) - kUnitCost;
    if (tile1 <= 0) break;  // this part ends within the unit's fixed entries
    const bool begins = tile0 == 0;
    const int h = unit / req.groups, row0 = unit % req.groups * kRows;
    const int rows = min(kRows, req.n * a.G - row0);
    const int token0 = req.row;
    // Keys that the first and the last row see end here; those below low_max are hidden
    // from the last row (window).
    const int limit_min = min(req.len, req.len - req.n + row0 / a.G + 1);
    const int limit_max = min(req.len, req.len - req.n + (row0 + rows - 1) / a.G + 1);
    const int low_max = a.window > 0 ? (int)max((int64_t)0, limit_max - a.window) : 0;

    // This warp's query rows (row r = warp + 8 j) on their way to registers.
    constexpr int kPer = kD / 32;
    float qv[kNT][kPer];
#pragma unroll
    for (int j = 0; j < kNT; ++j) {
      const int r = warp + kWarps * j;
      const int64_t token = token0 + (row0 + r) / a.G;
      const bool real = r < rows && token >= 0 && token < a.T;
      const T* src = static_cast<const T*>(a.q) +
                     (real ? token * a.stride_t + (h * a.G + (row0 + r) % a.G) * a.stride_h : 0);
#pragma unroll
      for (int k = 0; k < kPer; ++k) qv[j][k] = real ? value(src + k * 32 + lane) : 0.0f;
    }

    // ---- the warp's strips: keys key, key + kTile, ... below key_stop ----
    int key = req.lo + tile0 * kTile + warp * kStrip;
    const int key_stop = min(req.lo + tile1 * kTile, limit_max);
    const int strips = key < key_stop ? (key_stop - key + kTile - 1) / kTile : 0;
    const int32_t* pages = a.table + (int64_t)b * a.max_pages;
    const int8_t* k_head = a.kq + (int64_t)h * a.page * kD + lane * 16;
    const float* scale_head = (lane < 16 ? a.kd : a.vd) + (int64_t)h * (a.page / a.block);
    uint32_t hidden = 0;  // bit i: stage i's strip has no page
    // The page of a strip is looked up one strip before its copies are issued (those of the
    // first strips at once).
    int look = 0, look_at = (int)a.by_page((uint32_t)key), look_off = key - look_at * a.page;
    int issued = 0, write_slot = 0;
    uint32_t write_at = my_ring;

    auto look_up = [&](int32_t& page, int& off) {
      off = look_off;
      page = look < strips ? pages[look_at] : 0;
      ++look;
      look_at += a.step_pages;
      look_off += a.step_off;
      if (look_off >= a.page) {
        look_off -= a.page;
        ++look_at;
      }
    };
    auto issue = [&](int32_t page, int off) {
      if (issued++ < strips) {
        if ((uint32_t)page < (uint32_t)a.n_pages) {
          const int8_t* src = k_head + (uint64_t)(uint32_t)page * a.page_bytes + off * kD;
          const int8_t* src_v = src + v_minus_k;
          const uint32_t kd0 = write_at + k_dst, vd0 = write_at + v_dst;
#pragma unroll
          for (int i = 0; i < kStrip * kChunks / 32; ++i) {
            constexpr uint32_t kNone = 0;
            const uint32_t xk = kD == 64 ? kNone : kD == 128 ? (i & 1) * 64u : (i & 3) * 32u;
            const uint32_t xv = kD == 64 ? kNone
                                         : kD == 128 ? (i & 1) * 16u
                                                     : ((i & 1) * 4u + ((i >> 1) & 1)) * 16u;
            cp16((kd0 ^ xk) + i * 512, src + i * 512);
            cp16((vd0 ^ xv) + i * 512, src_v + i * 512);
          }
          cp4(write_at + 2 * kStrip * kD + lane * 4,
              scale_head + (uint64_t)(uint32_t)page * a.page_scales +
                  a.by_block((uint32_t)(off + (lane & 15))));
        } else {
          hidden |= 1u << write_slot;
          if (lane == 0 && a.status != nullptr) atomicOr(a.status, 1);
        }
      }
      cp_commit();
      write_at += Sh::kStage;
      if (++write_slot == Sh::kStages) {
        write_slot = 0;
        write_at = my_ring;
      }
    };

    int32_t page[Sh::kStages];
    int off[Sh::kStages];
#pragma unroll
    for (int s = 0; s < Sh::kStages; ++s) look_up(page[s], off[s]);
#pragma unroll
    for (int s = 0; s < Sh::kStages - 1; ++s) issue(page[s], off[s]);
    int32_t next_page = page[Sh::kStages - 1];
    int next_off = off[Sh::kStages - 1];

    // Queries to shared memory as B operands: row r of tile r / 8 is operand column r % 8;
    // k index (2i, 2i+1, 2i+8, 2i+9) of step 4c+w is dim 64c + 16i + 4w + (0, 2, 1, 3).
    // Each row is scaled by a power of two that brings its largest value to [2^13, 2^14).
#pragma unroll
    for (int row_step = 0; row_step < kNT; ++row_step) {
      const int r = warp + kWarps * row_step, i = (row0 + r) / a.G;
      const float* v = qv[row_step];
      float amax = 0.0f;
#pragma unroll
      for (int j = 0; j < kPer; ++j) amax = fmaxf(amax, fabsf(v[j]));
      amax = __uint_as_float(__reduce_max_sync(kFullMask, __float_as_uint(amax)));
      int e = (int)(__float_as_uint(amax) >> 23) - 127;
      e = e < -100 ? -100 : e;
      const float up = __int_as_float((13 - e + 127) << 23);  // 2^(13 - e), e in [-100, 128]
      if (lane == 0) {
        row_scale[r] = amax > 0.0f ? a.scale * 1.44269504088896341f * __int_as_float((e - 13 + 127) << 23) : 0.0f;
        row_limit[r] = min(req.len, req.len - req.n + i + 1);
      }
      __half* frag = reinterpret_cast<__half*>(q_frag);
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const int d = j * 32 + lane;
        const int step = (d >> 6) * 4 + ((d >> 2) & 3), t = (d >> 4) & 3, y = d & 3;
        // y 0, 2 -> register 0 halves 0, 1; y 1, 3 -> register 1 halves 0, 1
        const int half = ((y & 1) << 1) | (y >> 1);
        const int idx = (((step * kNT + (r >> 3)) * 32 + (r & 7) * 4 + t) << 2) + half;
        const float s = v[j] * up;
        const __half hi = __float2half_rn(s);
        frag[idx] = hi;
        if (kPair) frag[idx + kSteps * kNT * 32 * 4] = __float2half_rn(s - __half2float(hi));
      }
    }
    __syncthreads();
    if (tid == 0) {
      const Cut cut(total, ctas);
      const bool whole = begins && x_stop == unit_stop;
      const int c0 = whole ? cta : cut.part_of(unit_at + kUnitCost);
      const int c1 = whole ? cta : cut.part_of(unit_stop - 1);
      unit_at_hand = {h, row0, rows, token0, c0, c1 - c0 + 1, begins, whole};
      walk.x = x_stop;
      walk.at = at;
      walk.b = b;
      walk.req = req;
    }
    float qs[kNT][2];
    int limit[kNT][2];
#pragma unroll
    for (int n = 0; n < kNT; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        qs[n][c] = row_scale[8 * n + 2 * t4 + c];
        limit[n][c] = row_limit[8 * n + 2 * t4 + c];
      }

    // m: the reference that weights are taken against (0 while a row has seen no key);
    // bar: m + kMaxSlack (-inf then).
    float o[kSteps][kNT][4];
    float m[kNT][2], bar[kNT][2], l[kNT][2], ref = kLeastRef, inv_ref = kWeightScale / kLeastRef;
#pragma unroll
    for (int n = 0; n < kNT; ++n) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        m[n][c] = 0.0f;
        bar[n][c] = -kInf;
        l[n][c] = 0.0f;
      }
#pragma unroll
      for (int i = 0; i < kSteps; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) o[i][n][c] = 0.0f;
    }

    uint32_t read_at = my_ring;
    int read_slot = 0;
    for (int s = 0; s < strips; ++s) {
      cp_wait<Sh::kStages - 2>();
      __syncwarp();
      float c[kNT][4];
#pragma unroll
      for (int n = 0; n < kNT; ++n) c[n][0] = c[n][1] = c[n][2] = c[n][3] = 0.0f;
      // with one tile of rows, odd steps sum apart: two chains of products instead of one
      float c2[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int q = 0; q < kD / 64; ++q) {
        const uint32_t from = ((read_at + k_src) ^ (kD == 64 ? 0u : (q & 1) * 64u)) + (q >> 1) * 128;
        const uint4 xa = lds_v4(from), xb = lds_v4(from + 8 * kD);
        const uint32_t wa[4] = {xa.x, xa.y, xa.z, xa.w}, wb[4] = {xb.x, xb.y, xb.z, xb.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int step = 4 * q + i;
          const uint32_t a0 = even_bytes(wa[i]), a1 = even_bytes(wb[i]);
          const uint32_t a2 = odd_bytes(wa[i]), a3 = odd_bytes(wb[i]);
#pragma unroll
          for (int n = 0; n < kNT; ++n) {
            const uint2 f = q_frag[(step * kNT + n) * 32 + lane];
            float* to = kNT == 1 && (i & 1) ? c2 : c[n];
            mma_16816(to, a0, a1, a2, a3, f.x, f.y);
            if (kPair) {
              const uint2 lo = q_frag[((kSteps + step) * kNT + n) * 32 + lane];
              mma_16816(to, a0, a1, a2, a3, lo.x, lo.y);
            }
          }
        }
      }

      if (kNT == 1) {
#pragma unroll
        for (int i = 0; i < 4; ++i) c[0][i] += c2[i];
      }

      // c[n]: (key a, row 2t), (key a, row 2t+1), (key b, row 2t), (key b, row 2t+1)
      const uint32_t d_at = read_at + 2 * kStrip * kD + ka * 4;
      const float kda = lds_f32(d_at), kdb = lds_f32(d_at + 32);
      float vda = lds_f32(d_at + 64), vdb = lds_f32(d_at + 96);
#pragma unroll
      for (int n = 0; n < kNT; ++n) {
        c[n][0] *= kda * qs[n][0];
        c[n][1] *= kda * qs[n][1];
        c[n][2] *= kdb * qs[n][0];
        c[n][3] *= kdb * qs[n][1];
      }
      const bool no_page = (hidden >> read_slot) & 1u;
      if (key + kStrip > limit_min || key < low_max || no_page) {
        hidden &= ~(1u << read_slot);
#pragma unroll
        for (int n = 0; n < kNT; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int k = key + (i < 2 ? ka : kb), lim = limit[n][i & 1];
            const bool seen = k < lim && (a.window == 0 || k >= lim - a.window) && !no_page;
            c[n][i] = seen ? c[n][i] : -kInf;
          }
        vda = key + ka < limit_max && !no_page ? vda : 0.0f;
        vdb = key + kb < limit_max && !no_page ? vdb : 0.0f;
      }

      // The references move only when a score (a scale) passes them by more than the slack.
      const float v_top = fmaxf(fabsf(vda), fabsf(vdb));
      bool move = v_top > kRefSlack * ref;
#pragma unroll
      for (int n = 0; n < kNT; ++n) {
        move |= fmaxf(c[n][0], c[n][2]) > bar[n][0];
        move |= fmaxf(c[n][1], c[n][3]) > bar[n][1];
      }
      if (__any_sync(kFullMask, move)) {
        const float top = __uint_as_float(__reduce_max_sync(kFullMask, __float_as_uint(v_top)));
        const float new_ref = fmaxf(ref, top);
        const float rescale = ref / new_ref;
        ref = new_ref;
        inv_ref = kWeightScale / ref;
#pragma unroll
        for (int n = 0; n < kNT; ++n)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float y = fmaxf(c[n][i], c[n][2 + i]);
#pragma unroll
            for (int w2 = 4; w2 < 32; w2 <<= 1) y = fmaxf(y, __shfl_xor_sync(kFullMask, y, w2));
            float f = 1.0f;
            if (y > bar[n][i] - kMaxSlack) {  // new maximum (bar - slack is -inf at first)
              f = bar[n][i] == -kInf ? 0.0f : ex2(m[n][i] - y);
              m[n][i] = y;
              bar[n][i] = y + kMaxSlack;
            }
            l[n][i] *= f;
#pragma unroll
            for (int j = 0; j < kSteps; ++j) {
              o[j][n][i] *= f * rescale;
              o[j][n][2 + i] *= f * rescale;
            }
          }
      }
      const float wa2 = vda * inv_ref, wb2 = vdb * inv_ref;
      uint32_t p0[kNT], p1[kNT], e0[kNT], e1[kNT];
#pragma unroll
      for (int n = 0; n < kNT; ++n) {
        const float x0 = ex2(c[n][0] - m[n][0]), x1 = ex2(c[n][1] - m[n][1]);
        const float x2 = ex2(c[n][2] - m[n][0]), x3 = ex2(c[n][3] - m[n][1]);
        l[n][0] += x0 + x2;
        l[n][1] += x1 + x3;
        const float y0 = x0 * wa2, y1 = x1 * wa2, y2 = x2 * wb2, y3 = x3 * wb2;
        const uint32_t h0 = pack_half(y0, y1), h1 = pack_half(y2, y3);
        p0[n] = transpose_8x8(h0);
        p1[n] = transpose_8x8(h1);
        if (kPair) {
          const float2 r0 = unpack_half(h0), r1 = unpack_half(h1);
          e0[n] = transpose_8x8(pack_half(y0 - r0.x, y1 - r0.y));
          e1[n] = transpose_8x8(pack_half(y2 - r1.x, y3 - r1.y));
        }
      }

      // O^T: operand rows g, g + 8 of tile 2w (2w + 1) are dims 4w, 4w+1 (4w+2, 4w+3) of this
      // lane's run of dims; keys 2t, 2t+1 of the operand are key_of(2t), key_of(2t+1).
#pragma unroll
      for (int q = 0; q < (kD + 127) / 128; ++q) {
        constexpr int kWords = kD == 64 ? 2 : 4;
        uint32_t v[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t from = read_at + (i & 1 ? v_src1 : v_src0) + (i & 2 ? 8 * kD : 0) + q * 128;
          if (kD == 64) {
            asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v[i][0]), "=r"(v[i][1]) : "r"(from));
          } else {
            const uint4 y = lds_v4(from);
            v[i][0] = y.x; v[i][1] = y.y; v[i][2] = y.z; v[i][3] = y.w;
          }
        }
#pragma unroll
        for (int w2 = 0; w2 < kWords; ++w2) {
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const uint32_t sel = half ? 0x7632u : 0x5410u;
            const uint32_t z0 = __byte_perm(v[0][w2], v[1][w2], sel);
            const uint32_t z1 = __byte_perm(v[2][w2], v[3][w2], sel);
            const int tile = (q * kWords + w2) * 2 + half;
            const uint32_t a0 = even_bytes(z0), a1 = odd_bytes(z0);
            const uint32_t a2 = even_bytes(z1), a3 = odd_bytes(z1);
#pragma unroll
            for (int n = 0; n < kNT; ++n) {
              float strip[4];
              mma_16816_zero(strip, a0, a1, a2, a3, p0[n], p1[n]);
              if (kPair) mma_16816(strip, a0, a1, a2, a3, e0[n], e1[n]);
              add4(o[tile][n], strip);
            }
          }
        }
      }
      __syncwarp();
      issue(next_page, next_off);
      look_up(next_page, next_off);
      key += kTile;
      read_at += Sh::kStage;
      if (++read_slot == Sh::kStages) {
        read_slot = 0;
        read_at = my_ring;
      }
    }
    cp_wait<0>();

    // ---- join the warps ----
#pragma unroll
    for (int n = 0; n < kNT; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int w2 = 4; w2 < 32; w2 <<= 1) l[n][i] += __shfl_xor_sync(kFullMask, l[n][i], w2);
        if (g == 0) {
          warp_m[warp * kRows + 8 * n + 2 * t4 + i] = bar[n][i] == -kInf ? -kInf : m[n][i];
          warp_l[warp * kRows + 8 * n + 2 * t4 + i] = l[n][i];
        }
      }
    __syncthreads();  // also: every warp is done with its ring
    for (int r = tid; r < kRows; r += kThreads) {
      float top = -kInf, sum = 0.0f;
      for (int i = 0; i < kWarps; ++i) top = fmaxf(top, warp_m[i * kRows + r]);
      for (int i = 0; i < kWarps; ++i)
        if (warp_m[i * kRows + r] > -kInf) sum += warp_l[i * kRows + r] * ex2(warp_m[i * kRows + r] - top);
      row_m[r] = top;
      row_l[r] = sum;
    }
    float* join = reinterpret_cast<float*>(ring) + warp * kRows * kD;
#pragma unroll
    for (int n = 0; n < kNT; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = 8 * n + 2 * t4 + i;
        float top = -kInf;
        for (int k = 0; k < kWarps; ++k) top = fmaxf(top, warp_m[k * kRows + r]);
        const float f = bar[n][i] == -kInf ? 0.0f
                                            : ex2(m[n][i] - top) * ref * (1.0f / kWeightScale);
        constexpr int kRun = kD == 64 ? 8 : 16;  // consecutive dims of a lane
#pragma unroll
        for (int j = 0; j < kSteps / 2; ++j) {
          const float4 v = make_float4(o[2 * j][n][i] * f, o[2 * j][n][2 + i] * f,
                                       o[2 * j + 1][n][i] * f, o[2 * j + 1][n][2 + i] * f);
          const int d = (j / (kRun / 4)) * 128 + g * kRun + (j % (kRun / 4)) * 4;
          *reinterpret_cast<float4*>(join + r * kD + d) = v;
        }
      }
    __syncthreads();

    const Unit u = unit_at_hand;
    // Values 4i .. 4i+3 of the unit's rows, divided by their sums, to their place.
    auto finish = [&](int i, float4 v) {
      const int r = i * 4 / kD, d = i * 4 % kD;
      const int64_t token = u.token0 + (u.row0 + r) / a.G;
      if (r >= u.rows || token < 0 || token >= a.T) return;
      const float sum_l = row_l[r], f = sum_l > 0.0f ? 1.0f / sum_l : 0.0f;
      const int64_t row = token * a.Hq + u.h * a.G + (u.row0 + r) % a.G;
      store4(static_cast<T*>(a.out) + row * kD + d, make_float4(v.x * f, v.y * f, v.z * f, v.w * f));
      if (a.lse != nullptr && d == 0)
        a.lse[row] = sum_l > 0.0f ? (row_m[r] + log2f(sum_l)) * 0.693147180559945309f : -kInf;
    };
    constexpr int kItems = kRows * kD / 4;
    constexpr int kPart = kRows * (kD + 2);  // m, l, values
    float* mine = a.parts + (int64_t)((u.begins ? gridDim.x : 0) + cta) * kPart;
    for (int i = tid; i < kItems; i += kThreads) {
      float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int k = 0; k < kWarps; ++k) {
        const float4 y = reinterpret_cast<const float4*>(ring)[k * kItems + i];
        v.x += y.x; v.y += y.y; v.z += y.z; v.w += y.w;
      }
      if (u.whole) finish(i, v);
      else __stcg(reinterpret_cast<float4*>(mine + 2 * kRows) + i, v);
    }
    if (!u.whole) {
      if (tid < kRows) {
        __stcg(mine + tid, row_m[tid]);
        __stcg(mine + kRows + tid, row_l[tid]);
      }
      __syncthreads();
      if (tid == 0) {
        // releases the CTA's part (ordered before by the barrier), acquires the others'
        int n;
        asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;"
                     : "=r"(n) : "l"(a.arrived + u.first_cta) : "memory");
        last_part = n == u.parts - 1;
        if (last_part) a.arrived[u.first_cta] = 0;
      }
      __syncthreads();
      if (last_part) {
        // ---- join the unit's parts, in the order of the keys ----
        // Part 0 is the second one of its CTA, the others are the first ones of theirs.
        const int parts = u.parts;
        const float* part0 = a.parts + (int64_t)(gridDim.x + u.first_cta) * kPart;
        const float* part1 = a.parts + (int64_t)u.first_cta * kPart;
        float* fac = reinterpret_cast<float*>(ring);  // [parts][kRows]: m, then the factor
        float* sum_of = fac + parts * kRows;          // [parts][kRows]: l
        // The values follow through shared memory, each thread's own ones, as many parts at a
        // time as fit; the first are on their way while the factors are made.
        float4* values = reinterpret_cast<float4*>(fac + (2 * parts * kRows + 3) / 4 * 4);
        const int batch = (Sh::kBig - (2 * parts * kRows + 3) / 4 * 16) / (kItems * 16);
        auto fetch = [&](int first_part) {
          const int n = min(batch, parts - first_part);
          for (int i = tid; i < kItems; i += kThreads) {
            const uint32_t dst = smem_addr(values + i);
            const float* src = part1 + 2 * kRows + i * 4;
            for (int k = 0; k < n; ++k)
              cp16(dst + k * kItems * 16,
                   first_part + k == 0 ? part0 + 2 * kRows + i * 4 : src + (int64_t)(first_part + k) * kPart);
          }
          cp_commit();
        };
        fetch(0);
        for (int i = tid; i < parts * kRows; i += kThreads) {
          const float* src = (i < kRows ? part0 : part1 + (int64_t)(i / kRows) * kPart) + i % kRows;
          fac[i] = __ldcg(src);
          sum_of[i] = __ldcg(src + kRows);
        }
        __syncthreads();
        for (int r = warp; r < kRows; r += kWarps) {
          float top = -kInf, total_l = 0.0f;
          for (int i = lane; i < parts; i += 32) top = fmaxf(top, fac[i * kRows + r]);
#pragma unroll
          for (int w2 = 16; w2 > 0; w2 >>= 1) top = fmaxf(top, __shfl_xor_sync(kFullMask, top, w2));
          for (int i = lane; i < parts; i += 32) {
            const float pm = fac[i * kRows + r];
            const float f = pm > -kInf ? ex2(pm - top) : 0.0f;
            fac[i * kRows + r] = f;
            total_l += f * sum_of[i * kRows + r];
          }
#pragma unroll
          for (int w2 = 16; w2 > 0; w2 >>= 1) total_l += __shfl_xor_sync(kFullMask, total_l, w2);
          if (lane == 0) {
            row_m[r] = top;
            row_l[r] = total_l;
          }
        }
        __syncthreads();
        float4 v[(kItems + kThreads - 1) / kThreads] = {};
        for (int first_part = 0; first_part < parts; first_part += batch) {
          if (first_part > 0) fetch(first_part);
          cp_wait<0>();
          const int n = min(batch, parts - first_part);
#pragma unroll
          for (int j = 0; j < (kItems + kThreads - 1) / kThreads; ++j) {
            const int i = tid + j * kThreads;
            if (i >= kItems) continue;
#pragma unroll 2
            for (int k = 0; k < n; ++k) {
              const float4 y = values[k * kItems + i];
              const float f = fac[(first_part + k) * kRows + i * 4 / kD];
              v[j].x += y.x * f; v[j].y += y.y * f; v[j].z += y.z * f; v[j].w += y.w * f;
            }
          }
        }
#pragma unroll
        for (int j = 0; j < (kItems + kThreads - 1) / kThreads; ++j)
          if (tid + j * kThreads < kItems) finish(tid + j * kThreads, v[j]);
      }
    }
  }
}

template <typename T, int kD, int kNT>
cudaError_t launch_shape(const AttnArgs& a, const DeviceInfo& info, int64_t max_tiles,
                         cudaStream_t stream) {
  using Sh = Shape<T, kD, kNT>;
  static_assert(Sh::kSmem * Sh::kCtas <= 226 * 1024, "shared memory of the CTAs of an SM");
  // The attribute is set once for each device: it stays with the function, whose size is
  // always the same.
  static std::atomic<uint64_t> ready{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !((ready.load() >> dev) & 1u)) {
    e = cudaFuncSetAttribute(attention_kernel<T, kD, kNT>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::kSmem);
    if (e != cudaSuccess) return e;
    if (dev < 64) ready.fetch_or(1ull << dev);
  }
  int64_t ctas = (int64_t)info.sms * Sh::kCtas;
  const int64_t fit = (MEMRA_KV_ATTENTION_WORKSPACE_BYTES - kMaxCtas * 4) /
                      (2 * Sh::kRows * (kD + 2) * (int64_t)sizeof(float));
  if (ctas > fit) ctas = fit;
  if (ctas > kMaxCtas) ctas = kMaxCtas;
  // a unit may have as many parts: their factors and one part's values at a time fit the ring
  constexpr int kMost = (Sh::kBig - Sh::kRows * kD * 4 - 16) / (Sh::kRows * 8);
  static_assert(kMost >= 64, "parts that can be joined");
  if (ctas > kMost) ctas = kMost;
  // One CTA joins a unit's parts at the rate of one SM, so few units are cut less finely.
  const int64_t batch_rows = (a.B > 0 ? a.B : 1) * Sh::kRows;
  const int64_t units = batch_rows / Sh::kRows * a.Hkv * ((a.T * a.G + batch_rows - 1) / batch_rows);
  if (ctas > units * kMaxParts) ctas = units * kMaxParts;
  const int64_t groups = (a.T * a.G + Sh::kRows - 1) / Sh::kRows + a.B;
  const int64_t tiles = (max_tiles + 1) * groups * a.Hkv;  // what the list can hold at most
  if (ctas > tiles) ctas = tiles;
  if (ctas < 1) ctas = 1;
  return launch_kernel(attention_kernel<T, kD, kNT>, dim3((unsigned)ctas), dim3(kThreads),
                       (size_t)Sh::kSmem, stream, a);
}

// Query rows of a step: 8, 16 or 32, the fewest that hold an average request's (its keys
// are read once for each step).
template <typename T>
cudaError_t launch_attention(const AttnArgs& a, int D, const DeviceInfo& info, cudaStream_t stream) {
  const int64_t rows = a.B > 0 ? (a.T * a.G + a.B - 1) / a.B : 1;
  const int64_t max_tiles = a.max_pages * a.page / kTile + 1 + kUnitCost;
  if (sizeof(T) == 2 && D <= 128 && rows > kWideRows && a.T * a.Hq >= kWideAll)
    return launch_wide_attention(a, D, rows, info, max_tiles, stream);
  if (D == 64) {
    if (rows <= 8) return launch_shape<T, 64, 1>(a, info, max_tiles, stream);
    if (rows <= 16) return launch_shape<T, 64, 2>(a, info, max_tiles, stream);
    return launch_shape<T, 64, 4>(a, info, max_tiles, stream);
  }
  if (D == 128) {
    if (rows <= 8) return launch_shape<T, 128, 1>(a, info, max_tiles, stream);
    if (rows <= 16) return launch_shape<T, 128, 2>(a, info, max_tiles, stream);
    return launch_shape<T, 128, 4>(a, info, max_tiles, stream);
  }
  if (rows <= 8) return launch_shape<T, 256, 1>(a, info, max_tiles, stream);
  return launch_shape<T, 256, 2>(a, info, max_tiles, stream);
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
      max_pages > (INT32_MAX - kTile) / page_size || T > INT32_MAX / Hq || B > (1 << 24))
    return MEMRA_ERR_UNSUPPORTED;
  // (a sequence's last tile of keys ends below 2^31)
  if (Hkv * page_size * D > (int64_t)UINT32_MAX) return MEMRA_ERR_UNSUPPORTED;
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
  DeviceInfo info;
  if (!device_info(&info)) return MEMRA_ERR_CUDA;
  AttnArgs a;
  a.q = q;
  a.T = T;
  a.stride_t = stride_t;
  a.stride_h = stride_h;
  a.kq = kq;
  a.vq = vq;
  a.kd = kd;
  a.vd = vd;
  a.table = block_table;
  a.kv_lens = kv_lens;
  a.cu_q = cu_q;
  a.B = B;
  a.max_pages = max_pages;
  a.window = window;
  a.n_pages = (int32_t)n_pages;
  a.Hq = (int)Hq;
  a.Hkv = (int)Hkv;
  a.G = (int)(Hq / Hkv);
  a.page = (int)page_size;
  a.block = (int)block;
  a.by_page = Divider((uint32_t)page_size);
  a.by_block = Divider((uint32_t)block);
  a.page_bytes = (uint32_t)(Hkv * page_size * D);
  a.page_scales = (uint32_t)(Hkv * (page_size / block));
  a.step_pages = kTile / (int)page_size;
  a.step_off = kTile % (int)page_size;
  a.scale = scale;
  a.out = out;
  a.lse = lse;
  a.arrived = static_cast<int*>(workspace);
  a.parts = reinterpret_cast<float*>(static_cast<char*>(workspace) + kMaxCtas * 4);
  a.status = dev_status;
  wait_settings(&a.wait_limit, &a.stall_after);
  const cudaError_t e = dtype == MEMRA_BF16 ? launch_attention<uint16_t>(a, (int)D, info, stream)
                                            : launch_attention<float>(a, (int)D, info, stream);
  if (e != cudaSuccess) return cuda_fail(e);
  return MEMRA_OK;
}
