// Attention over the paged 8-bit KV cache for many query rows: speculative verify, chunks
// of a prompt, wide groups of heads.  bf16 queries, D 64 or 128; kv_attention.cu has the
// rest.
//
// With tens of rows to a cached head, the work is two matrix products and goes to the
// tcgen05 tensor cores: S [128 rows x 128 keys] = Q K^T and O [128 rows x D] += P V, both in
// fp16 (exact for bf16 queries and 8-bit codes) with fp32 accumulators in tensor memory.
// Weights as bf16 would need no scaling against the scales of V, but round at 2^-8, which
// doubles the result's own rounding.  Warps of one CTA an SM have three tasks:
//   11 warps bring a tile of codes from the cache (a tile ahead, each thread its own), turn them
//     into fp16 exactly and lay K and V out in shared memory as the products read them
//     (rows of 64 dims, 128-byte swizzle; two stages);
//   1 thread issues the products: S of the next tile before O of this one;
//   8 warps turn scores into weights, four to every other tile, each group with its own
//     statistics and its own accumulators, so that neither waits for the other; a thread
//     has a row and its keys, and the weights go back to tensor memory, over the scores,
//     as the second product's operand.
// Units of up to 64 rows put every row into the product twice, and each copy's lane takes
// half of the keys (the products write the lanes of one copy at a time): that spreads the
// exponentials, 16 a cycle on an SM, over all of its quarters.
// Every wait is bounded: when one runs out the CTA's other warps are released too, its rows
// become NaN and status bit 2 is set.
// Accumulators stay in tensor memory for up to 512 tiles; they are rescaled only when a
// maximum moves by more than the slack, and the two groups' (and copies') are joined at the
// end.  Scales never meet the codes: kd multiplies a score, vd a weight.
//
// A verify step of 16 sequences (8 tokens each, contexts of 500 to 8000, 32 heads on 4, D 128)
// takes 43.1 to 44.4 us; bytes and operations alone need 7.1.  A CTA has some ten tiles.  About half
// of the time is a unit's two ends (list, queries, first tile: 8 us; last products, parts,
// arrival, join: 10), the rest the tiles, 3000 cycles each: the operands' way through shared
// memory (codes in and out, fp16 in, read by the products: some 2000 cycles of it) and the
// waits between the tasks.  Neither the exponentials nor the products are the bound: with
// half of either the time changes by under 5 %.
#include <atomic>

#include "kv_attention.cuh"

namespace memra {
namespace {

constexpr int kLanes = 128;  // rows of a product
constexpr int kSoftWarps = 8, kFeedWarps = 11;  // and one: 20 warps may have 96 registers
constexpr int kSoftThreads = kSoftWarps * 32, kFeedThreads = kFeedWarps * 32;
constexpr int kThreads = kSoftThreads + kFeedThreads + 32;
// Keeps 2^8 / ref times a row's sum in range; blocks of smaller scales are next to nothing.
constexpr float kLeastRef = 1e-25f;
constexpr int kCost = 5;  // entries of the list for a unit's fixed time (3: 45.9 us, 4: 45.8, 5: 43.6, 6:
                          // 44.1 for the verify step above; 32 requests of 100 to 500: 41.7, 36.5, 36.1, 35.5)

// Tiles after which a range's sums leave tensor memory: the tensor cores cut their fp32 sums
// off at every product, to one side (of V of one sign 1.7e-4 over 131072 keys with units of 64
// rows, 3.6e-4 with 128, and so on with the length).  With 512 tiles it is 1e-4 and 2.2e-4 at
// any length.  An end and a new beginning cost about 22 us (512 queries on 130k keys: 1629 us
// without, 1666 so, 1783 with 128 tiles).
constexpr int kRun = 512;

// Tensor memory columns: scores of two or three tiles and each group's weights (two fp16 a
// column), then each group's accumulators.
constexpr uint32_t kTmemColumns = 512, kTmemO = 256, kTmemGroup = 128;
constexpr int kTurns = 8;  // tiles whose scales of K and V are kept

// kRows: a unit's rows, 64 (two lanes to a row) or 128.
template <int kD, int kRows>
struct Shape {
  static constexpr int kOperand = kTile * kD * 2;       // K or V of a tile in fp16
  static constexpr int kQ = kLanes * kD * 2;
  static constexpr int kQAt = 4 * kOperand;             // after two stages of K, V
  static constexpr int kScalesAt = kQAt + kQ;           // kd, then vd: [kTurns][128]
  static constexpr int kUnitAt = kScalesAt + 2 * kTurns * kTile * 4;  // amax [group][lane], [2 units][m, l][group][lane]
  static constexpr int kMiscAt = kUnitAt + 10 * kLanes * 4;      // vd maxima [kTurns][4], hidden strips [kTurns][8]
  static constexpr int kHiddenAt = kMiscAt + kTurns * 16;
  static constexpr int kRawAt = kHiddenAt + kTurns * 8;  // the feeding threads' pieces of the next tile
  static constexpr int kRaw = 2 * ((kTile * kD / 16 + kFeedThreads - 1) / kFeedThreads) * kFeedThreads * 16;
  static constexpr int kHeldAt = kRawAt + kRaw;         // m and l of a range so far, a soft thread's own
  static constexpr int kBarsAt = kHeldAt + kSoftThreads * 8;
  static constexpr int kSmem = kBarsAt + 18 * 8 + 1024;          // and room to align to 1024
  static constexpr int kPart = 2 * kRows + kRows * kD;           // m, l, values: floats
  // Scores run kStages - 1 tiles ahead of the values: two where a lane has half of the keys,
  // so that a group finds its next scores when it has made its weights (a tile took 3500
  // cycles with one tile); with all keys the columns are full, and the weights lie over the
  // last half of the scores.
  static constexpr int kCopies = kLanes / kRows, kKeys = kTile / kCopies;  // of a tile, a lane
  static constexpr int kStages = kCopies == 2 ? 3 : 2;
  static __device__ __forceinline__ uint32_t scores_at(uint32_t tile) { return tile % kStages * kKeys; }
  static __device__ __forceinline__ uint32_t scores_phase(uint32_t tile) { return tile / kStages & 1; }
  static __device__ __forceinline__ uint32_t weights_at(uint32_t group) {
    return kCopies == 2 ? kStages * kKeys + group * (kKeys / 2) : group * kTile + kTile / 2;
  }
};

// ---- tcgen05 ----
__device__ __forceinline__ void tmem_alloc(uint32_t dst, uint32_t columns) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst), "r"(columns)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
__device__ __forceinline__ void tmem_free(uint32_t at, uint32_t columns) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(columns));
}
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
// D [128 x N] (+)= A [128 x 16] B [N x 16]^T, A from shared or tensor memory; lanes whose bit
// of `skip` (of each 32) is set keep their D.
__device__ __forceinline__ void tc_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t what, uint32_t skip, bool add) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, {%5, %5, %5, %5}, p;\n}" ::"r"(d), "l"(a), "l"(b),
      "r"(what), "r"((uint32_t)add), "r"(skip)
      : "memory");
}
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t what, uint32_t skip, bool add) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, {%5, %5, %5, %5}, p;\n}" ::"r"(d), "r"(a), "l"(b),
      "r"(what), "r"((uint32_t)add), "r"(skip)
      : "memory");
}
// 32 columns of this warp's 32 lanes.
__device__ __forceinline__ void tmem_load32(uint32_t at, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
        "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
        "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
        "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(at));
}
__device__ __forceinline__ void tmem_store32(uint32_t at, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(at),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]),
      "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]),
      "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_store16(uint32_t at, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16};" ::"r"(at),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// Waits for this thread's loads; r: what they loaded, which nothing may use before.
template <int kN>
__device__ __forceinline__ void tmem_wait_loads(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < kN; ++i) asm volatile("" : "+r"(r[i]));
}
__device__ __forceinline__ void tmem_wait_stores() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// Plain shared-memory writes that happened before become visible to the products.  The
// thread that issues those makes this fence, after its waits: in the feeding warps it
// would also wait for their loads of the next tile (a tile took 4500 cycles then).
__device__ __forceinline__ void async_proxy_fence() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Shared-memory operand: rows of 64 fp16 under the 128-byte swizzle, eight rows (1024
// bytes) after one another; `lead` parts neighbouring blocks of 64 columns where those are
// the product's rows.
__device__ __forceinline__ uint64_t operand(uint32_t at, uint32_t lead) {
  return (uint64_t)((at >> 4) & 0x3fff) | (uint64_t)(lead >> 4) << 16 | (uint64_t)(1024 >> 4) << 32 |
         1ull << 46 | 2ull << 61;
}
// kind::f16 with fp16 operands and fp32 sums, 128 rows, N columns; values: B's rows (the
// keys) lie one after another, contiguous along N.
template <int N, bool values>
constexpr uint32_t kProduct = 1u << 4 | (values ? 1u << 16 : 0u) | (uint32_t)(N >> 3) << 17 |
                              (uint32_t)(kLanes >> 4) << 24;

// A value cached in L2 only, or 0: one piece of code without a branch, so that nothing waits
// for the load here.
__device__ __forceinline__ float load_or_zero(const float* p, bool there) {
  float r;
  asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %2, 0;\n mov.b32 %0, 0;\n @p ld.global.cg.f32 %0, [%1];\n}"
               : "=&f"(r) : "l"(p), "r"((uint32_t)there));
  return r;
}
__device__ __forceinline__ int32_t load_or_none(const int32_t* p, bool there) {  // -1
  int32_t r;
  asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %2, 0;\n mov.b32 %0, -1;\n @p ld.global.cg.s32 %0, [%1];\n}"
               : "=&r"(r) : "l"(p), "r"((uint32_t)there));
  return r;
}

// Pairs of fp32 in one instruction.
using Pair = unsigned long long;
__device__ __forceinline__ Pair pair_of(uint32_t lo, uint32_t hi) {
  Pair p;
  asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "r"(lo), "r"(hi));
  return p;
}
__device__ __forceinline__ Pair pair_of(float lo, float hi) { return pair_of(__float_as_uint(lo), __float_as_uint(hi)); }
__device__ __forceinline__ float2 parts_of(Pair p) {
  uint32_t lo, hi;
  asm("mov.b64 {%0, %1}, %2;" : "=r"(lo), "=r"(hi) : "l"(p));
  return make_float2(__uint_as_float(lo), __uint_as_float(hi));
}
__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
  Pair d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ Pair add2(Pair a, Pair b) {
  Pair d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
  Pair d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}

// One CTA's range of one unit, or kRun tiles of it.
struct Segment {
  int b, h, row0, rows, token0;
  int key0, key_stop, tiles;             // its keys, in tiles of kTile
  int limit_min, limit_max, low_max;     // what the first and the last row see
  int len, n;
  bool begins, whole;                    // the CTA has the unit's first keys, all of them
  bool continues, ends;                  // not the range's first keys; its last ones
  int64_t unit_at, unit_stop;
};

template <int kRows>
struct Walker {
  Walk w;
  bool begins, inside;  // of the range that w.x is inside of
  __device__ __forceinline__ bool next(const AttnArgs& a, Segment* s) {
    if (w.x >= w.stop) return false;
    int64_t entries = entries_of<kCost>(a, w.req);
    while (w.x >= w.at + entries) {
      w.at += entries;
      w.req = request_of<kRows>(a, ++w.b);
      entries = entries_of<kCost>(a, w.req);
    }
    const Request& req = w.req;
    const int size = req.tiles + kCost;
    const int unit = (int)Cut::divide(w.x - w.at, size);
    s->unit_at = w.at + (int64_t)unit * size;
    s->unit_stop = s->unit_at + size;
    const int64_t x_stop = s->unit_stop < w.stop ? s->unit_stop : w.stop;
    const int tile0 = max((int)(w.x - s->unit_at) - kCost, 0);
    const int tile1 = (int)(x_stop - s->unit_at) - kCost;
    w.x = x_stop;
    if (tile1 <= 0) return false;  // the part ends within the unit's fixed entries
    s->continues = inside;
    if (!inside) begins = tile0 == 0;
    s->begins = begins;
    s->whole = begins && x_stop == s->unit_stop;
    s->b = w.b;
    s->h = unit / req.groups;
    s->row0 = unit % req.groups * kRows;
    s->rows = min(kRows, req.n * a.G - s->row0);
    s->token0 = req.row;
    s->len = req.len;
    s->n = req.n;
    s->limit_min = min(req.len, req.len - req.n + s->row0 / a.G + 1);
    s->limit_max = min(req.len, req.len - req.n + (s->row0 + s->rows - 1) / a.G + 1);
    s->low_max = a.window > 0 ? (int)max((int64_t)0, s->limit_max - a.window) : 0;
    s->key0 = req.lo + tile0 * kTile;
    s->key_stop = min(req.lo + tile1 * kTile, s->limit_max);
    s->tiles = s->key0 < s->key_stop ? (s->key_stop - s->key0 + kTile - 1) / kTile : 0;
    inside = s->tiles > kRun;
    s->ends = !inside;
    if (inside) {
      s->tiles = kRun;
      s->key_stop = s->key0 + kRun * kTile;
      w.x = s->unit_at + kCost + tile0 + kRun;
    }
    return true;
  }
};

// Each warp goes over the CTA's part of the list by itself; where it stands lies in shared
// memory (registers hold the tile on its way).
template <int kRows>
struct Way {
  Walker<kRows> walker;
  Segment seg;
};
// The next unit, for a whole warp.
template <int kRows>
__device__ __forceinline__ bool next_unit(const AttnArgs& a, Way<kRows>* way) {
  __syncwarp();
  bool more = false;
  if ((threadIdx.x & 31) == 0) more = way->walker.next(a, &way->seg);
  __syncwarp();  // orders lane 0's writes before the other lanes' reads (an exchange does not)
  return __shfl_sync(kFullMask, (int)more, 0) != 0;
}

// A whole warp's bounded wait, with one answer for all its lanes.
__device__ __forceinline__ bool warp_wait(const AttnArgs& a, uint32_t bar, uint32_t parity, volatile int* abort) {
  return __all_sync(kFullMask, mbar_wait(bar, parity, abort, a.wait_limit));
}

struct Bars {  // shared-memory addresses
  uint32_t k_full[2], v_full[2], empty[2], scores[3], weights[2], q, pair[4], soft, done;
};

// ---- 11 warps: codes from the cache to fp16 operands ----
template <int kD, int kRows>
__device__ __forceinline__ void feed(const AttnArgs& a, Way<kRows>* way, uint8_t* smem, const Bars& bars,
                                     volatile int* abort) {
  using Sh = Shape<kD, kRows>;
  constexpr int kChunks = kD / 16;  // 16-code pieces of a row
  constexpr int kLoads = (kTile * kChunks + kFeedThreads - 1) / kFeedThreads;  // of K, and of V, a thread
  constexpr int kStep = kFeedThreads / kChunks;  // rows from one of a thread's pieces to the next
  static_assert(kFeedThreads % kChunks == 0 && kFeedThreads >= 2 * kTile, "pieces and scales");
  const int tid = threadIdx.x - kSoftThreads, lane = tid & 31, warp = tid >> 5;
  // Eight neighbouring lanes write pieces of two rows' same block of 64 dims: the rows'
  // swizzles differ in the lowest bit, so they meet in no bank.
  const int row = kD == 64 ? tid >> 2 : (tid >> 4) * 2 + ((tid >> 2) & 1);
  const int chunk = kD == 64 ? tid & 3 : (tid & 3) + ((tid >> 3) & 1) * 4;
  // Scales: kd of key tid (warps 0 .. 3), vd of key tid - 128 (4 .. 7).
  const bool scale_v = tid >= kTile, has_scale = tid < 2 * kTile;
  const int scale_key = tid & (kTile - 1);
  // A tile's scales stay until its weights are made.  They are written after the scores two
  // tiles back, which follow the weights of three more tiles back at least.
  float* scales = reinterpret_cast<float*>(smem + Sh::kScalesAt);  // [kd, vd][turn][key]
  float* v_most = reinterpret_cast<float*>(smem + Sh::kMiscAt);    // [turn][4]
  uint8_t* hidden = smem + Sh::kHiddenAt;                          // [turn][8]
  const int blocks = (int)a.by_block((uint32_t)a.page);

  int tile = 0, tiles = 0;
  bool more = true;
  // A tile: its first key, the end of the keys that are there, its head; the pages of strip
  // lane & 7 and of this thread's scales (-1: not there).
  struct Ref {
    int key, stop, h;
    int32_t page, scale_page;
  };
  auto next_ref = [&](Ref& r) {
    r.page = r.scale_page = -1;
    while (more && tile >= tiles) {
      more = next_unit(a, way);
      tiles = way->seg.tiles;
      tile = 0;
    }
    if (!more) return false;
    const Segment& seg = way->seg;
    r.key = seg.key0 + tile * kTile;
    r.stop = seg.key_stop;
    r.h = seg.h;
    ++tile;
    const int32_t* pages = a.table + (int64_t)seg.b * a.max_pages;
    const int there = (r.stop + kStrip - 1) / kStrip * kStrip;
    const int k0 = r.key + (lane & 7) * kStrip, k = r.key + scale_key;
    r.page = load_or_none(pages + a.by_page((uint32_t)k0), k0 < there);
    r.scale_page = load_or_none(pages + a.by_page((uint32_t)k), has_scale && k < there);
    return true;
  };
  // Where strip lane & 7 of the tile lies in a plane (-1: nowhere).
  auto strip_of = [&](const Ref& r) {
    const int k0 = r.key + (lane & 7) * kStrip, off = k0 - (int)a.by_page((uint32_t)k0) * a.page;
    return (uint32_t)r.page < (uint32_t)a.n_pages
               ? (int64_t)((uint64_t)(uint32_t)r.page * a.page_bytes + (uint32_t)((r.h * a.page + off) * kD))
               : (int64_t)-1;
  };
  float scale = 0.0f;
  bool gone = false;  // the strip of scale_key has no page
  const int8_t* k_lane = a.kq + chunk * 16;
  const int8_t* v_lane = a.vq + chunk * 16;
  // This thread's own places for its pieces: the j-th of K, then of V.
  const uint32_t raw = smem_addr(smem + Sh::kRawAt) + tid * 16;
  constexpr uint32_t kPlace = kFeedThreads * 16;
  auto load_pieces = [&](const int8_t* plane, int64_t strip, int v) {
    const int8_t* from[kLoads];
    bool there[kLoads];
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {  // a warp's rows of a piece lie in one strip
      const int64_t at = __shfl_sync(kFullMask, strip, ((j * kStep + row) / kStrip) & 7);
      there[j] = at >= 0 && j * kStep + row < kTile;
      from[j] = there[j] ? plane + at + (j * kStep + row) % kStrip * kD : plane;
    }
#pragma unroll
    for (int j = 0; j < kLoads; ++j) cp16_or_zeros(raw + (v * kLoads + j) * kPlace, from[j], there[j]);
    cp_commit();
  };
  auto scale_of = [&](const float* plane, const Ref& r, int key, int32_t page) {
    const int k = r.key + key;
    const int off = k - (int)a.by_page((uint32_t)k) * a.page;
    const bool there = (uint32_t)page < (uint32_t)a.n_pages && k < r.stop;
    return load_or_zero(plane + (there ? (int64_t)(uint32_t)page * a.page_scales + (int64_t)r.h * blocks +
                                             a.by_block((uint32_t)off) : 0), there);
  };
  auto load_scales = [&](const Ref& r, bool ahead) {
    gone = ahead && (uint32_t)r.scale_page >= (uint32_t)a.n_pages && r.key + scale_key < r.stop;
    scale = scale_of(scale_v ? a.vd : a.kd, r, scale_key, r.scale_page);
  };
  // 16 codes as fp16 (the byte code + 128 under the exponent of 1024 is 1024 + 128 + code) to
  // two neighbouring 16-byte units of their row.
  auto put = [&](uint8_t* base, int key, const uint4& x) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t h[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t y = w[i] ^ 0x80808080u;
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const uint32_t z = __byte_perm(y, 0x64646464u, p ? 0x4342u : 0x4140u);
        const __half2 v = __hsub2(*reinterpret_cast<const __half2*>(&z), __half2half2(__ushort_as_half(0x6480)));
        h[2 * i + p] = *reinterpret_cast<const uint32_t*>(&v);
      }
    }
    uint8_t* line = base + (chunk >> 2) * (kTile * 128) + key * 128;
    const int at = ((2 * (chunk & 3)) ^ (key & 7)) << 4;
    *reinterpret_cast<uint4*>(line + at) = make_uint4(h[0], h[1], h[2], h[3]);
    *reinterpret_cast<uint4*>(line + (at ^ 16)) = make_uint4(h[4], h[5], h[6], h[7]);
  };

  auto convert = [&](uint8_t* base, int v) {
    uint4 x[kLoads];
#pragma unroll
    for (int j = 0; j < kLoads; ++j) x[j] = lds_v4(raw + (v * kLoads + j) * kPlace);
#pragma unroll
    for (int j = 0; j < kLoads; ++j)
      if (j * kStep + row < kTile) put(base, j * kStep + row, x[j]);
  };

  // Each piece's place takes the next tile's as soon as it is read; K goes a tile ahead of V,
  // so that no scores wait for the values of a tile before.
  Ref next{};
  auto put_k = [&](uint32_t g, int wait_for) {  // tile g: scales and K, once the scores two tiles back are made
    const int stage = g & 1, turn = g & (kTurns - 1);
    if (g >= 2 && !warp_wait(a, bars.scores[(g - 2) % Sh::kStages], Sh::scores_phase(g - 2), abort)) return false;
    if (has_scale) {
      scales[(scale_v ? kTurns + turn : turn) * kTile + scale_key] = scale;
      if (scale_v) {
        const uint32_t most = __reduce_max_sync(kFullMask, __float_as_uint(fabsf(scale)));
        if (lane == 0) v_most[turn * 4 + (warp & 3)] = __uint_as_float(most);
      } else if ((lane & 15) == 0) {
        hidden[turn * 8 + scale_key / kStrip] = gone ? 1 : 0;
        if (gone && a.status != nullptr) atomicOr(a.status, 1);
      }
    }
    if (wait_for == 0) cp_wait<0>();
    else cp_wait<1>();  // V's pieces may be under way
    convert(smem + stage * 2 * Sh::kOperand, 0);
    __syncwarp();
    if (lane == 0) mbar_arrive(bars.k_full[stage]);
    return true;
  };
  bool have = a.stall_after != 0 && next_ref(next);  // tile g, then g + 1 and g + 2
  int64_t strip = -1;
  if (have) {
    strip = strip_of(next);
    load_pieces(k_lane, strip, 0);
    load_pieces(v_lane, strip, 1);
    load_scales(next, true);
  }
  bool ahead = have && next_ref(next);
  if (have) {
    put_k(0, 1);
    strip = strip_of(next);
    load_pieces(k_lane, strip, 0);
    load_scales(next, ahead);
  }
  for (uint32_t g = 0; have && (int)g != a.stall_after; ++g) {
    // at this point: V of tile g and K of g + 1 are under way, strip is tile g + 1's
    const bool beyond = ahead && next_ref(next);  // tile g + 2: its pages are there when K of g + 1 is done
    if (!beyond) next.page = next.scale_page = -1;
    if (ahead && !put_k(g + 1, g == 0 ? 0 : 1)) break;
    const int64_t strip2 = strip_of(next);
    load_pieces(k_lane, strip2, 0);
    load_scales(next, beyond);
    // V, once the values two tiles back are summed
    const int stage = g & 1;
    if (g >= 2 && !warp_wait(a, bars.empty[stage], ((g >> 1) & 1) ^ 1, abort)) break;
    cp_wait<1>();
    convert(smem + stage * 2 * Sh::kOperand + Sh::kOperand, 1);
    __syncwarp();
    if (lane == 0) mbar_arrive(bars.v_full[stage]);
    load_pieces(v_lane, strip, 1);
    strip = strip2;
    have = ahead;
    ahead = beyond;
  }
  cp_wait<0>();
}

// ---- one thread: the products ----
template <int kD, int kRows>
__device__ __forceinline__ void multiply(const AttnArgs& a, Walker<kRows>* walker, uint32_t smem, uint32_t tmem,
                                         const Bars& bars, volatile int* abort) {
  using Sh = Shape<kD, kRows>;
  constexpr int kCopies = Sh::kCopies, kKeys = Sh::kKeys;
  constexpr uint32_t kScores = kProduct<kKeys, false>, kValues = kProduct<kD, true>;
  Segment seg;
  uint32_t g = 0, unit = 0;
  auto skip = [](int copy) { return kCopies == 1 ? 0u : copy ? 0x0000ffffu : 0xffff0000u; };
  auto scores = [&](uint32_t t) {
    const uint32_t k = smem + (t & 1) * 2 * Sh::kOperand, q = smem + Sh::kQAt;
#pragma unroll
    for (int c = 0; c < kCopies; ++c)
#pragma unroll
      for (int s = 0; s < kD / 16; ++s)
        tc_mma_ss(tmem + Sh::scores_at(t), operand(q + (s >> 2) * (kLanes * 128) + (s & 3) * 32, 16),
                  operand(k + c * (kKeys * 128) + (s >> 2) * (kTile * 128) + (s & 3) * 32, 16), kScores, skip(c), s > 0);
    mbar_arrive(bars.scores[t % Sh::kStages]);  // passes on what the feeding warps wrote (the scales)
    tc_commit(bars.scores[t % Sh::kStages]);
  };
  auto scores_when_there = [&](uint32_t t) {
    if (!mbar_wait(bars.k_full[t & 1], (t >> 1) & 1, abort, a.wait_limit)) return false;
    async_proxy_fence();
    tc_after();
    scores(t);
    return true;
  };
  while (walker->next(a, &seg)) {
    if (seg.tiles == 0) continue;
    if (!mbar_wait(bars.q, unit & 1, abort, a.wait_limit)) return;
    ++unit;
    for (int t = 0; t < Sh::kStages - 1 && t < seg.tiles; ++t)
      if (!scores_when_there(g + t)) return;
    for (int t = 0; t < seg.tiles; ++t, ++g) {
      if (t + Sh::kStages - 1 < seg.tiles && !scores_when_there(g + Sh::kStages - 1)) return;
      if (!mbar_wait(bars.v_full[g & 1], (g >> 1) & 1, abort, a.wait_limit)) return;
      if (!mbar_wait(bars.weights[g & 1], (g >> 1) & 1, abort, a.wait_limit)) return;
      async_proxy_fence();
      tc_after();
      const uint32_t v = smem + (g & 1) * 2 * Sh::kOperand + Sh::kOperand;
#pragma unroll
      for (int c = 0; c < kCopies; ++c)
#pragma unroll
        for (int s = 0; s < kKeys / 16; ++s)  // 16 keys are two groups of eight rows
          tc_mma_ts(tmem + kTmemO + (g & 1) * kTmemGroup, tmem + Sh::weights_at(g & 1) + s * 8,
                    operand(v + c * (kKeys * 128) + s * 2048, kTile * 128), kValues, skip(c), t > 1 || s > 0);
      tc_commit(bars.empty[g & 1]);
    }
  }
}

// ---- 8 warps: scores to weights, results ----
template <int kD, int kRows>
__device__ __forceinline__ void soften(const AttnArgs& a, Way<kRows>* way, uint8_t* smem, uint32_t tmem,
                                       const Bars& bars, volatile int* abort, int64_t total, int ctas,
                                       int* last_part) {
  using Sh = Shape<kD, kRows>;
  constexpr int kCopies = Sh::kCopies, kKeys = Sh::kKeys;
  constexpr int kStepKeys = 32;           // of these, at a time in registers
  constexpr int kDims = kD / 2;           // of a row, a thread, at a unit's two ends
  const float kInf = __int_as_float(0x7f800000);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int quarter = warp & 3, group = warp >> 2, at_lane = quarter * 32 + lane;
  const int row = quarter * (kRows / 4) + lane % (kRows / 4), copy = lane / (kRows / 4);
  const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
  const uint32_t w_at = lanes + Sh::weights_at(group), o_at = lanes + kTmemO + group * kTmemGroup;
  const ulonglong2* scales = reinterpret_cast<const ulonglong2*>(smem + Sh::kScalesAt) + copy * kKeys / 4;
  const float4* v_most = reinterpret_cast<const float4*>(smem + Sh::kMiscAt);
  const uint2* hidden = reinterpret_cast<const uint2*>(smem + Sh::kHiddenAt);
  float* unit_x = reinterpret_cast<float*>(smem + Sh::kUnitAt);
  float2* held = reinterpret_cast<float2*>(smem + Sh::kHeldAt) + tid;
  uint32_t pair_phase = 0, soft_phase = 0, units = 0, g0 = 0;  // g0: the CTA's tiles before this unit
  // With the other group's warp of the same lanes; false when a wait ran out somewhere.
  auto pair_sync = [&]() {
    __syncwarp();
    if (lane == 0) mbar_arrive(bars.pair[quarter]);
    const bool ok = warp_wait(a, bars.pair[quarter], pair_phase, abort);
    pair_phase ^= 1;
    return ok;
  };
  auto soft_sync = [&]() {
    __syncwarp();
    if (lane == 0) mbar_arrive(bars.soft);
    const bool ok = warp_wait(a, bars.soft, soft_phase, abort);
    soft_phase ^= 1;
    return ok;
  };

  const Segment& seg = way->seg;
  for (; next_unit(a, way); g0 += seg.tiles) {
    const bool active = quarter * (kRows / 4) < seg.rows;  // the warp has rows
    const int i = (seg.row0 + row) / a.G, hq = seg.h * a.G + (seg.row0 + row) % a.G;
    const int64_t token = (int64_t)seg.token0 + i;
    const bool real = row < seg.rows && token >= 0 && token < a.T;
    const int limit = min(seg.len, seg.len - seg.n + i + 1);
    float qs = 1.0f;
    if (seg.tiles > 0) {
      // This thread's half of its query, scaled by a power of two that brings the row's
      // largest value to [2^13, 2^14) (bf16's eight bits fit fp16 then), |scale| kept apart.
      uint4 raw[kDims / 8];
      float amax = 0.0f;
      const uint16_t* src = static_cast<const uint16_t*>(a.q) + (real ? token * a.stride_t + hq * a.stride_h : 0) + group * kDims;
#pragma unroll
      for (int k = 0; k < kDims / 8; ++k) {
        raw[k] = real && active ? *reinterpret_cast<const uint4*>(src + 8 * k) : make_uint4(0, 0, 0, 0);
        const uint32_t w[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
          amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(w[j] << 16)), fabsf(__uint_as_float(w[j] & 0xffff0000u))));
      }
      unit_x[group * kLanes + at_lane] = amax;
      if (!pair_sync()) return;
      amax = fmaxf(amax, unit_x[(group ^ 1) * kLanes + at_lane]);
      int e = (int)(__float_as_uint(amax) >> 23) - 127;
      e = e < -100 ? -100 : e;
      float up = __int_as_float((13 - e + 127) << 23);
      if (amax > 0.0f && a.scale != 0.0f) qs = fabsf(a.scale) * 1.44269504088896341f * __int_as_float((e - 13 + 127) << 23);
      up = a.scale == 0.0f ? 0.0f : copysignf(up, a.scale);
      uint8_t* q_at = smem + Sh::kQAt + at_lane * 128;
#pragma unroll
      for (int k = 0; k < kDims / 8; ++k) {
        const uint32_t w[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
        uint32_t h[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const __half2 v = __floats2half2_rn(__uint_as_float(w[j] << 16) * up, __uint_as_float(w[j] & 0xffff0000u) * up);
          h[j] = *reinterpret_cast<const uint32_t*>(&v);
        }
        const int unit = group * (kDims / 8) + k;  // of the row's units of eight dims
        *reinterpret_cast<uint4*>(q_at + (unit >> 3) * (kLanes * 128) + (((unit & 7) ^ (lane & 7)) << 4)) =
            make_uint4(h[0], h[1], h[2], h[3]);
      }
    }
    if (seg.tiles > 0) {
      __syncwarp();
      if (lane == 0) mbar_arrive(bars.q);
    }

    // Weights are taken as 2^(x - m) with the scales' reference in m = most - log2(2^8 / ref),
    // most the reference of the row's maximum (bar: most + kMaxSlack, -inf until there is
    // one), so that l and O are in the same units.
    float most = 0.0f, bar = -kInf, m = 0.0f, l = 0.0f, ref = 0.0f, shift = 0.0f;
    const int t0 = (int)((g0 ^ group) & 1);  // the group's first tile
    for (int t = t0; t < seg.tiles; t += 2) {
      const uint32_t phase = ((g0 + t) >> 1) & 1, turn = (g0 + t) & (kTurns - 1);
      const uint32_t s_at = lanes + Sh::scores_at(g0 + t);
      const ulonglong2* kd = scales + turn * (kTile / 4);
      const ulonglong2* vd = kd + kTurns * (kTile / 4);
      if (!warp_wait(a, bars.scores[(g0 + t) % Sh::kStages], Sh::scores_phase(g0 + t), abort)) return;
      if (active) {
        tc_after();
        const int key = seg.key0 + t * kTile + copy * kKeys;
        const uint2 gone = hidden[turn];  // a byte to a strip
        const bool plain = seg.key0 + (t + 1) * kTile <= seg.limit_min && seg.key0 + t * kTile >= seg.low_max &&
                           (gone.x | gone.y) == 0;
        Pair s[kStepKeys / 2];
        // Scores of kStepKeys keys from `first` on (of this thread's), without the row's scale.
        auto fetch = [&](int first) {
          uint32_t bits[kStepKeys];
          tmem_load32(s_at + first, bits);
          tmem_wait_loads<kStepKeys>(bits);
#pragma unroll
          for (int j = 0; j < kStepKeys; j += 4) {
            const ulonglong2 d = kd[(first + j) / 4];
            s[j / 2] = mul2(pair_of(bits[j], bits[j + 1]), d.x);
            s[j / 2 + 1] = mul2(pair_of(bits[j + 2], bits[j + 3]), d.y);
          }
          if (!plain) {
#pragma unroll
            for (int j = 0; j < kStepKeys; j += 2) {
              const float2 x = parts_of(s[j / 2]);
              const int k = key + first + j, strip = (copy * kKeys + first + j) / kStrip;
              const bool there = (((strip & 4 ? gone.y : gone.x) >> (8 * (strip & 3))) & 1u) == 0;
              const bool s0 = k < limit && (a.window == 0 || k >= limit - a.window) && there;
              const bool s1 = k + 1 < limit && (a.window == 0 || k + 1 >= limit - a.window) && there;
              s[j / 2] = pair_of(s0 ? x.x : -kInf, s1 ? x.y : -kInf);
            }
          }
        };
        float top = -kInf;
#pragma unroll 1
        for (int first = 0; first < kKeys; first += kStepKeys) {
          fetch(first);
          float y0 = -kInf, y1 = -kInf;
#pragma unroll
          for (int j = 0; j < kStepKeys / 2; j += 2) {
            const float2 u = parts_of(s[j]), w = parts_of(s[j + 1]);
            y0 = fmaxf(fmaxf(y0, u.x), u.y);
            y1 = fmaxf(fmaxf(y1, w.x), w.y);
          }
          top = fmaxf(top, fmaxf(y0, y1));
        }
        if (kCopies == 2) top = fmaxf(top, __shfl_xor_sync(kFullMask, top, 16));
        top *= qs;
        const float4 vm = v_most[turn];
        const float v_top = fmaxf(fmaxf(vm.x, vm.y), fmaxf(vm.z, vm.w));
        if (__any_sync(kFullMask, top > bar) || v_top > kRefSlack * ref) {
          float f = 1.0f;
          if (v_top > ref) {
            ref = v_top;
            const float new_shift = 8.0f - log2f(fmaxf(ref, kLeastRef));
            f = ex2(new_shift - shift);
            shift = new_shift;
          }
          if (bar == -kInf ? top > bar : top > most) {  // a new maximum
            f = bar == -kInf ? 0.0f : f * ex2(most - top);
            most = top;
            bar = most + kMaxSlack;
          }
          m = most - shift;
          l *= f;
          if (t > 1) {  // the accumulators, once the group's last product is done
            if (!warp_wait(a, bars.empty[group], phase ^ 1, abort)) return;
            tc_after();
#pragma unroll 1
            for (int c = 0; c < kD; c += 32) {
              uint32_t o[32];
              tmem_load32(o_at + c, o);
              tmem_wait_loads<32>(o);
#pragma unroll
              for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
              tmem_store32(o_at + c, o);
            }
          }
        }
        // The group's last weights are read when its last product is done; with two stages that
        // came before these scores.
        if (Sh::kStages == 3 && t > 1) {
          if (!warp_wait(a, bars.empty[group], phase ^ 1, abort)) return;
          tc_after();
        }
        // Weights: where a lane has all keys they lie over the last half of the scores, so the
        // last keys come first, whose scores are read by then.
        Pair sum0 = pair_of(0.0f, 0.0f), sum1 = sum0;
        const Pair qs2 = pair_of(qs, qs), m2 = pair_of(-m, -m);
#pragma unroll 1
        for (int first = kKeys - kStepKeys; first >= 0; first -= kStepKeys) {
          fetch(first);
          uint32_t p[kStepKeys / 2];
#pragma unroll
          for (int j = 0; j < kStepKeys; j += 4) {
            const ulonglong2 d = vd[(first + j) / 4];
            const float2 x0 = parts_of(fma2(s[j / 2], qs2, m2)), x1 = parts_of(fma2(s[j / 2 + 1], qs2, m2));
            const Pair p0 = pair_of(ex2(x0.x), ex2(x0.y)), p1 = pair_of(ex2(x1.x), ex2(x1.y));
            sum0 = add2(sum0, p0);
            sum1 = add2(sum1, p1);
            const float2 w0 = parts_of(mul2(p0, d.x)), w1 = parts_of(mul2(p1, d.y));
            const __half2 lo = __floats2half2_rn(w0.x, w0.y), hi = __floats2half2_rn(w1.x, w1.y);
            p[j / 2] = *reinterpret_cast<const uint32_t*>(&lo);
            p[j / 2 + 1] = *reinterpret_cast<const uint32_t*>(&hi);
          }
          tmem_store16(w_at + first / 2, p);
        }
        const float2 sums = parts_of(add2(sum0, sum1));
        l += sums.x + sums.y;
        tmem_wait_stores();
        tc_before();
      } else if (Sh::kStages == 3 && t > 1 && !warp_wait(a, bars.empty[group], phase ^ 1, abort)) {
        // A warp without rows waits for the group's last product too: with scores two tiles ahead
        // it would else arrive for this tile before the others have for that one, and stand in
        // for one of them.
        return;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bars.weights[group]);
    }

    // ---- the unit's end, or the run's: both groups' sums, and the copies', and those of the
    // range's runs before (each thread's own part of them lies where it will put the sum) ----
    const bool finished = seg.whole && seg.ends;
    const bool has[2] = {seg.tiles > (int)(g0 & 1), seg.tiles > (int)((g0 ^ 1) & 1)};  // group 0's, 1's tiles
    for (int k = 0; k < 2; ++k) {
      const uint32_t last = g0 + seg.tiles - 1;  // the last tile of stage k is this or the one before
      if (has[k] && !warp_wait(a, bars.empty[k], ((last - ((last ^ k) & 1)) >> 1) & 1, abort)) return;
    }
    tc_after();
    float* mine = a.parts + (int64_t)((seg.begins ? gridDim.x : 0) + blockIdx.x) * Sh::kPart;
    if (kCopies == 2) l += __shfl_xor_sync(kFullMask, l, 16);
    float* ends = unit_x + (2 + 4 * (units++ & 1)) * kLanes + at_lane;
    ends[group * kLanes] = bar == -kInf ? -kInf : m;
    ends[(2 + group) * kLanes] = l;
    if (!pair_sync()) return;
    if (active) {
      const float m0 = ends[0], m1 = ends[kLanes];
      m = fmaxf(m0, m1);
      float f0 = m0 > -kInf ? ex2(m0 - m) : 0.0f, f1 = m1 > -kInf ? ex2(m1 - m) : 0.0f;
      l = f0 * ends[2 * kLanes] + f1 * ends[3 * kLanes];
      float before = 0.0f;
      if (seg.continues) {
        const float2 h = *held;
        const float to = fmaxf(m, h.x), f = m > -kInf ? ex2(m - to) : 0.0f;
        before = h.x > -kInf ? ex2(h.x - to) : 0.0f;
        f0 *= f;
        f1 *= f;
        l = l * f + h.y * before;
        m = to;
      }
      *held = make_float2(m, l);
      if (finished) {
        const float f = l > 0.0f ? 1.0f / l : 0.0f;
        f0 *= f;
        f1 *= f;
        before *= f;
      }
      uint16_t* out = static_cast<uint16_t*>(a.out) + (token * a.Hq + hq) * kD + group * kDims;
#pragma unroll 1
      for (int c = 0; c < kDims; c += 32) {
        float v[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = 0.0f;
        for (int k = 0; k < 2; ++k) {
          if (!has[k]) continue;
          uint32_t o[32];
          tmem_load32(lanes + kTmemO + k * kTmemGroup + group * kDims + c, o);
          tmem_wait_loads<32>(o);
          const float f = k ? f1 : f0;
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] += f != 0.0f ? __uint_as_float(o[j]) * f : 0.0f;
        }
        if (kCopies == 2)
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] += __shfl_xor_sync(kFullMask, v[j], 16);
        if (real)  // each copy its share
#pragma unroll
          for (int j = 0; j < 32 / kCopies; j += 4) {
            float x[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) x[k] = kCopies == 2 && copy ? v[(j + k + 16) & 31] : v[j + k];
            const int d = c + j + copy * (32 / kCopies);
            float4 y = make_float4(x[0], x[1], x[2], x[3]);
            float4* part = reinterpret_cast<float4*>(mine + 2 * kRows + row * kD + group * kDims + d);
            if (before != 0.0f) {
              const float4 z = __ldcg(part);
              y = make_float4(y.x + z.x * before, y.y + z.y * before, y.z + z.z * before, y.w + z.w * before);
            }
            if (finished) store4(out + d, y);
            else __stcg(part, y);
          }
      }
      if (group == 0 && copy == 0) {
        if (!finished) {
          __stcg(mine + row, m);
          __stcg(mine + kRows + row, l);
        } else if (real && a.lse != nullptr) {
          a.lse[token * a.Hq + hq] = l > 0.0f ? (m + log2f(l)) * 0.693147180559945309f : -kInf;
        }
      }
    }
    tc_before();
    if (seg.ends && !seg.whole) {
      const Cut cut(total, ctas);
      const int c0 = cut.part_of(seg.unit_at + kCost), parts = cut.part_of(seg.unit_stop - 1) - c0 + 1;
      if (!soft_sync()) return;
      if (tid == 0) {
        // releases the CTA's part (ordered before by the barrier), acquires the others'
        int n;
        asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;" : "=r"(n) : "l"(a.arrived + c0) : "memory");
        *last_part = n == parts - 1;
        if (n == parts - 1) a.arrived[c0] = 0;
      }
      if (!soft_sync()) return;
      if (*last_part) {  // joins the unit's parts, in the order of the keys
        const float* part0 = a.parts + (int64_t)(gridDim.x + c0) * Sh::kPart;
        const float* part1 = a.parts + (int64_t)c0 * Sh::kPart;
        // Four threads to a row.  Every other part comes through the queries' place in shared
        // memory, so that a thread has two parts on the way.
        constexpr int kItems = kD / 16;  // four values each
        const int sub = tid & 3;
        uint4* second = reinterpret_cast<uint4*>(smem + Sh::kQAt) + tid;
        for (int r = tid >> 2; r < seg.rows; r += kSoftThreads / 4) {
          float4 v[kItems];
          float high = -kInf, sum = 0.0f;
#pragma unroll
          for (int j = 0; j < kItems; ++j) v[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          auto values_of = [&](int k) { return (k == 0 ? part0 : part1 + (int64_t)k * Sh::kPart) + 2 * kRows + r * kD + sub * 4; };
          auto fold = [&](float pm, float pl, const float4* y) {
            if (pm == -kInf) return;
            const float to = fmaxf(high, pm);
            const float f0 = high > -kInf ? ex2(high - to) : 0.0f, f1 = ex2(pm - to);
            high = to;
            sum = sum * f0 + pl * f1;
#pragma unroll
            for (int j = 0; j < kItems; ++j) {
              v[j].x = v[j].x * f0 + y[j].x * f1;
              v[j].y = v[j].y * f0 + y[j].y * f1;
              v[j].z = v[j].z * f0 + y[j].z * f1;
              v[j].w = v[j].w * f0 + y[j].w * f1;
            }
          };
          for (int k = 0; k < parts; k += 2) {
            const float* p = values_of(k);
            const float* p2 = values_of(min(k + 1, parts - 1));
            float4 y[kItems];
#pragma unroll
            for (int j = 0; j < kItems; ++j) cp16(smem_addr(second + j * kSoftThreads), p2 + j * 16);
            cp_commit();
#pragma unroll
            for (int j = 0; j < kItems; ++j) y[j] = __ldcg(reinterpret_cast<const float4*>(p + j * 16));
            const int back = -2 * kRows - r * kD - sub * 4 + r;  // from a row's values to its m
            const float pm = __ldcg(p + back), pl = __ldcg(p + back + kRows);
            const float pm2 = __ldcg(p2 + back), pl2 = __ldcg(p2 + back + kRows);
            fold(pm, pl, y);
            cp_wait<0>();
            if (k + 1 < parts) {
#pragma unroll
              for (int j = 0; j < kItems; ++j) y[j] = *reinterpret_cast<const float4*>(second + j * kSoftThreads);
              fold(pm2, pl2, y);
            }
          }
          const int64_t tok = (int64_t)seg.token0 + (seg.row0 + r) / a.G;
          if (tok < 0 || tok >= a.T) continue;
          const float f = sum > 0.0f ? 1.0f / sum : 0.0f;
          const int64_t at = tok * a.Hq + seg.h * a.G + (seg.row0 + r) % a.G;
#pragma unroll
          for (int j = 0; j < kItems; ++j)
            store4(static_cast<uint16_t*>(a.out) + at * kD + j * 16 + sub * 4,
                   make_float4(v[j].x * f, v[j].y * f, v[j].z * f, v[j].w * f));
          if (sub == 0 && a.lse != nullptr)
            a.lse[at] = sum > 0.0f ? (high + log2f(sum)) * 0.693147180559945309f : -kInf;
        }
        if (!soft_sync()) return;  // before *last_part is written again
      }
    }
  }
}

template <int kD, int kRows>
__global__ void __launch_bounds__(kThreads, 1) wide_attention_kernel(AttnArgs a) {
  using Sh = Shape<kD, kRows>;
  extern __shared__ uint8_t raw[];
  uint8_t* smem = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);
  __shared__ Walk walk;
  __shared__ Way<kRows> ways[kThreads / 32];
  __shared__ uint32_t tmem_at;
  __shared__ int last_part, abort, late;
  pdl_launch_dependents();
  const int tid = threadIdx.x, warp = tid >> 5;
  if (warp == kThreads / 32 - 1) tmem_alloc(smem_addr(&tmem_at), kTmemColumns);
  const uint32_t base = smem_addr(smem) + Sh::kBarsAt;
  Bars bars;
  for (int i = 0; i < 2; ++i) {
    bars.k_full[i] = base + 8 * i;
    bars.v_full[i] = base + 16 + 8 * i;
    bars.empty[i] = base + 32 + 8 * i;
    bars.weights[i] = base + 64 + 8 * i;
  }
  for (int i = 0; i < 2; ++i) bars.scores[i] = base + 48 + 8 * i;
  bars.scores[2] = base + 136;
  bars.q = base + 80;
  for (int i = 0; i < 4; ++i) bars.pair[i] = base + 88 + 8 * i;
  bars.soft = base + 120;
  bars.done = base + 128;
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(bars.k_full[i], kFeedWarps);
      mbar_init(bars.v_full[i], kFeedWarps);
      mbar_init(bars.empty[i], 1);
      mbar_init(bars.weights[i], kSoftWarps / 2);
    }
    for (int i = 0; i < 3; ++i) mbar_init(bars.scores[i], 2);
    mbar_init(bars.q, kSoftWarps);
    for (int i = 0; i < 4; ++i) mbar_init(bars.pair[i], 2);
    mbar_init(bars.soft, kSoftWarps);
    mbar_init(bars.done, 1);
    mbar_init_fence();
    abort = late = 0;
  }
  pdl_wait();
  int ctas;
  int64_t total;
  const bool busy = locate<uint16_t, kD, kRows, kCost, kThreads>(a, &walk, &ctas, &total);
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = tmem_at;
  Way<kRows>* way = ways + warp;
  if ((tid & 31) == 0) way->walker = {walk, false, false};
  if (!busy) {
  } else if (warp < kSoftWarps) {
    soften<kD, kRows>(a, way, smem, tmem, bars, &abort, total, ctas, &last_part);
  } else if (warp < kSoftWarps + kFeedWarps) {
    feed<kD, kRows>(a, way, smem, bars, &abort);
  } else if ((tid & 31) == 0) {
    multiply<kD, kRows>(a, &way->walker, smem_addr(smem), tmem, bars, &abort);
    tc_commit(bars.done);  // nothing is in flight when the memory is given back
    mbar_wait(bars.done, 0, &late);
  }
  tc_before();
  __syncthreads();
  tc_after();
  __syncwarp();
  if (warp == kThreads / 32 - 1) tmem_free(tmem, kTmemColumns);
  if (abort != 0) {  // a wait ran out: the CTA's rows are not to be taken for results
    if (tid == 0 && a.status != nullptr) atomicOr(a.status, 2);
    const float nan = __int_as_float(0x7fffffff);
    Walker<kRows> walker{walk, false, false};
    Segment seg;
    while (walker.next(a, &seg))
      for (int i = tid; i < seg.rows * (kD / 4); i += kThreads) {
        const int r = seg.row0 + i / (kD / 4), d = i % (kD / 4) * 4;
        const int64_t token = (int64_t)seg.token0 + r / a.G, at = token * a.Hq + seg.h * a.G + r % a.G;
        if (token < 0 || token >= a.T) continue;
        store4(static_cast<uint16_t*>(a.out) + at * kD + d, make_float4(nan, nan, nan, nan));
        if (d == 0 && a.lse != nullptr) a.lse[at] = nan;
      }
  }
}

template <int kD, int kRows>
cudaError_t launch(const AttnArgs& a, const DeviceInfo& info, int64_t max_tiles, cudaStream_t stream) {
  using Sh = Shape<kD, kRows>;
  static std::atomic<uint64_t> ready{0};  // devices whose attribute is set (it stays with the function)
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !((ready.load() >> dev) & 1u)) {
    e = cudaFuncSetAttribute(wide_attention_kernel<kD, kRows>, cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::kSmem);
    if (e != cudaSuccess) return e;
    if (dev < 64) ready.fetch_or(1ull << dev);
  }
  int64_t ctas = info.sms;
  const int64_t fit = (MEMRA_KV_ATTENTION_WORKSPACE_BYTES - kMaxCtas * 4) / (2 * Sh::kPart * (int64_t)sizeof(float));
  if (ctas > fit) ctas = fit;
  if (ctas > kMaxCtas) ctas = kMaxCtas;
  const int64_t groups = (a.T * a.G + kRows - 1) / kRows + a.B;
  const int64_t entries = (max_tiles + kCost) * groups * a.Hkv;  // what the list can hold at most
  if (ctas > entries) ctas = entries;
  if (ctas < 1) ctas = 1;
  return launch_kernel(wide_attention_kernel<kD, kRows>, dim3((unsigned)ctas), dim3(kThreads), (size_t)Sh::kSmem, stream, a);
}

}  // namespace

cudaError_t launch_wide_attention(const AttnArgs& a, int D, int64_t rows, const DeviceInfo& info,
                                  int64_t max_tiles, cudaStream_t stream) {
  if (rows <= 64)
    return D == 64 ? launch<64, 64>(a, info, max_tiles, stream) : launch<128, 64>(a, info, max_tiles, stream);
  return D == 64 ? launch<64, 128>(a, info, max_tiles, stream) : launch<128, 128>(a, info, max_tiles, stream);
}

}  // namespace memra
