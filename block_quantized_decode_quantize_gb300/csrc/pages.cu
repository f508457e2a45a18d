// Pages of the cache after they are taken: sequences that share them, copies on write, their
// return and their compaction.  Rules and orders are stated in memra.h.
//
// All but the copy are whole numbers on block tables, 4 bytes an entry, and bound by latency: one
// launch each.  Where a result depends on all entries (which holder is a page's last, how many
// pages go before this one) either one CTA has the table in its registers and what it counts of
// each page in its shared memory, or, with more than that, the CTAs of one cluster count in
// global memory and meet at the cluster's barrier; counts are atomic, but nothing written depends
// on their order.  For 256 forks of 32 sequences (36,608 cells): fork 1.9 us, copy on write 4,
// release 12.3 (19.5 of as many random pages); for 4 forks of one 1.5, 1.7, 3.1.  Compaction of
// 256 pages 3.1, of 6000 pages and 6048 cells 6.8.  Measured and not kept: for a large release
// 16 CTAs (14.1 for 12.3), counts in the shared memories of the cluster (13.7).
#include <cooperative_groups.h>

#include "common.cuh"

namespace memra {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxRanks = 8;  // CTAs of a cluster

// Cells that a lane looks at together, so that their loads wait for each other once.  A table of
// one such tile a lane (8192 cells, 65,536 with eight CTAs) is read once and stays in registers.
constexpr int kTile = 8;

// A table cell's place and what it holds.
struct Table {
  const int32_t* lens;
  const int32_t* entries;
  int64_t B, max_pages, n_pages;
  int page;
  Divider by_row, by_page;
  // pages of a sequence of `len` tokens; *bad: the length is none
  __device__ __forceinline__ int pages_of(int32_t len, bool* bad) const {
    if (len < 0) {
      *bad = true;
      return 0;
    }
    const uint32_t whole = by_page((uint32_t)len), n = whole + (whole * (uint32_t)page != (uint32_t)len ? 1 : 0);
    if (n > (uint64_t)max_pages) {
      *bad = true;
      return (int)max_pages;
    }
    return (int)n;
  }
  __device__ __forceinline__ bool is_page(int32_t p) const { return p >= 0 && p < n_pages; }
};

// All threads of the cluster, which may be one CTA.
__device__ __forceinline__ void meet(cg::cluster_group& cluster, int ranks) {
  if (ranks > 1) cluster.sync();
  else __syncthreads();
}

// Exclusive place of this warp's `count` among the counts of all warps of the cluster, and their
// sum.  Every thread of the cluster calls it; `slots` is a CTA's own.
struct Counts {
  int32_t of_warp[kWarps];
};
__device__ __forceinline__ void place_of(cg::cluster_group& cluster, Counts& mine, int32_t count, int32_t* before, int32_t* all) {
  const int ranks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (lane == 0) mine.of_warp[warp] = count;
  meet(cluster, ranks);
  int32_t b = 0, n = 0;
  if (ranks == 1) {
    n = mine.of_warp[lane];
    b = lane < warp ? n : 0;
  } else {
    int32_t c[kMaxRanks];
#pragma unroll
    for (int r = 0; r < kMaxRanks; ++r) c[r] = r < ranks ? cluster.map_shared_rank(&mine, r)->of_warp[lane] : 0;
#pragma unroll
    for (int r = 0; r < kMaxRanks; ++r) {
      n += c[r];
      if (r < rank || (r == rank && lane < warp)) b += c[r];
    }
  }
  *before = __reduce_add_sync(kFullMask, b);
  *all = __reduce_add_sync(kFullMask, n);
}

__device__ __forceinline__ void tell(int bits, int32_t* status) {
  if (status == nullptr) return;
  bits = __reduce_or_sync(kFullMask, bits);
  if ((threadIdx.x & 31) == 0 && bits != 0) atomicOr(status, bits);
}

// ---------------------------------------------------------------------------
// Fork: a CTA to a new row.
// ---------------------------------------------------------------------------
struct ForkArgs {
  Table t;
  const int32_t *parents, *prefix;
  int32_t *refs, *lens_out, *table_out, *status;
};

constexpr int kForkThreads = 128;

__global__ void __launch_bounds__(kForkThreads) fork_kernel(ForkArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  const int64_t r = blockIdx.x;
  const int64_t parent = a.parents[r];
  const bool real = parent >= 0 && parent < a.t.B;
  bool bad = !real && parent != -1;
  int32_t len = real ? a.t.lens[parent] : 0;
  (void)a.t.pages_of(len, &bad);  // whether it is a length
  len = (int32_t)max((int64_t)0, min((int64_t)len, a.t.max_pages * a.t.page));
  if (a.prefix != nullptr) len = min(len, max(a.prefix[r], 0));
  const int pages = a.t.pages_of(len, &bad);
  for (int64_t i = threadIdx.x; i < a.t.max_pages; i += kForkThreads) {
    int32_t p = -1;
    if (i < pages) {
      p = a.t.entries[parent * a.t.max_pages + i];
      if (a.t.is_page(p)) {
        atomicAdd(a.refs + p, 1);
      } else {
        p = -1;
        bad = true;
      }
    }
    a.table_out[r * a.t.max_pages + i] = p;
  }
  if (threadIdx.x == 0) a.lens_out[r] = len;
  tell(bad ? 1 : 0, a.status);
}

// ---------------------------------------------------------------------------
// Copy on write: one CTA, 1024 sequences at a time.  Those of a chunk that stand in a shared
// page are listed in shared memory, and each counts those before it in the same page.
// ---------------------------------------------------------------------------
struct UnshareArgs {
  Table t;
  const int32_t *new_lens, *free_pages, *free_head;
  int64_t n_free;
  int32_t *refs, *table, *new_out, *src, *dst, *tokens, *free_head_out, *status;
};

__global__ void __launch_bounds__(kThreads) unshare_kernel(UnshareArgs a) {
  __shared__ __align__(16) int32_t page_of[kThreads];  // of the sharers listed
  __shared__ int32_t warp_sum[kWarps];
  __shared__ uint32_t refused_of[kThreads / 32];
  pdl_launch_dependents();
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
  int64_t head = a.free_head != nullptr ? *a.free_head : 0;
  if (head < 0) head = 0;
  int bits = 0;
  // sum of `flag` over the threads before this one, and over all
  auto place = [&](bool flag, int* all) {
    const uint32_t ballot = __ballot_sync(kFullMask, flag);
    __syncthreads();
    if (lane == 0) warp_sum[warp] = __popc(ballot);
    __syncthreads();
    const int v = lane < warps ? warp_sum[lane] : 0;
    *all = (int)__reduce_add_sync(kFullMask, v);
    return (int)__reduce_add_sync(kFullMask, lane < warp ? v : 0) + __popc(ballot & ((1u << lane) - 1));
  };
  for (int64_t base = 0; base < a.t.B; base += blockDim.x) {
    const int64_t b = base + tid;
    const bool mine = b < a.t.B;
    const int32_t len = mine ? a.t.lens[b] : 0;
    int32_t add = mine ? a.new_lens[b] : 0;
    bool bad = add < 0;
    add = max(add, 0);
    const int pages = a.t.pages_of(len, &bad);
    const int inside = len > 0 ? (int)((uint32_t)len - a.t.by_page((uint32_t)len) * (uint32_t)a.t.page) : 0;
    int64_t cell = 0;
    int32_t p = -1, holders = 0;
    // a length beyond the table has no last page there
    if (mine && add > 0 && inside > 0 && pages == (int64_t)a.t.by_page((uint32_t)len) + 1) {
      cell = b * a.t.max_pages + pages - 1;
      p = a.t.entries[cell];
      if (a.t.is_page(p)) holders = __ldcg(a.refs + p);
      else bad = true;
    }
    const bool shares = holders > 0;
    int sharers;
    const int at = place(shares, &sharers);
    if (sharers == 0) {  // the same in all threads
      if (mine) {
        a.new_out[b] = add;
        a.src[b] = a.dst[b] = -1;
        a.tokens[b] = 0;
      }
      if (bad) bits |= 1;
      continue;
    }
    if (shares) page_of[at] = p;
    __syncthreads();
    int before = 0, latest = -1;  // sharers of the same page before this one, and the last of them
    if (shares)
      for (int i = 0; i < at; i += 4) {
        const int4 q = *reinterpret_cast<const int4*>(page_of + i);
        const int32_t other[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (other[j] == p && i + j < at) {
            ++before;
            latest = i + j;
          }
      }
    const bool takes = shares && before < holders;
    int takers;
    const int turn = place(takes, &takers);
    const bool fits = takes && head + turn < a.n_free;
    // a page's last holder keeps it, unless one before it could not leave
    if (tid < kThreads / 32) refused_of[tid] = 0;
    __syncthreads();
    if (takes && !fits) atomicOr(&refused_of[at >> 5], 1u << (at & 31));
    __syncthreads();
    bool refused = takes && !fits;
    if (shares && !takes && latest >= 0) {
      // the one before it is a taker, or kept the page as it does
      int i = latest;
      refused = (refused_of[i >> 5] >> (i & 31)) & 1u;
      while (!refused && --i >= 0)
        if (page_of[i] == p) refused = (refused_of[i >> 5] >> (i & 31)) & 1u;
    }
    int32_t f = -1;
    if (fits) {
      f = a.free_pages[head + turn];
      atomicSub(a.refs + p, 1);
      a.table[cell] = f;
      if (!a.t.is_page(f)) bad = true;
    }
    if (mine) {
      a.new_out[b] = refused ? 0 : add;
      a.src[b] = fits ? p : -1;
      a.dst[b] = f;
      a.tokens[b] = fits ? inside : 0;
    }
    if (bad) bits |= 1;
    if (refused) bits |= 4;
    head += min((int64_t)takers, max((int64_t)0, a.n_free - head));
    __syncthreads();
  }
  if (tid == 0) *a.free_head_out = (int32_t)head;
  tell(bits, a.status);
}

// ---------------------------------------------------------------------------
// Copies.  A warp takes 8 KB of one head's rows of a page in one plane, 4 KB of loads at a time.
// Memory bounds it: 1331 whole pages in 2 layers of 8 heads of 128 (698 MB in and out) 106.3 us,
// 97 % of the copy rate; the parts of 256 pages, of 32 sources, in 16 layers (276 MB) 49.5 us, 82 %.
// ---------------------------------------------------------------------------
constexpr int kCopyWarps = 8;
constexpr int kCopyLayers = 64;           // of a launch
constexpr int kCopyPiece = 8192;          // bytes

struct CopyArgs {
  memra_kv_layer layer[kCopyLayers];
  const int32_t *src, *dst, *tokens;
  int64_t N, n_pages;
  int Hkv, page, D, block, pieces;        // pieces of a head's page
  int32_t* status;
};

__global__ void __launch_bounds__(kCopyWarps * 32) copy_kernel(const __grid_constant__ CopyArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t per_entry = 2ll * a.Hkv * a.pieces;
  const int64_t item = (int64_t)blockIdx.x * kCopyWarps + (threadIdx.x >> 5);
  const int64_t i = item / per_entry;
  if (i >= a.N) return;
  const int rest = (int)(item - i * per_entry), piece = rest % a.pieces;
  const int h = (rest / a.pieces) >> 1, is_v = (rest / a.pieces) & 1;
  const int32_t from = a.src[i], to = a.dst[i];
  int32_t n = a.tokens != nullptr ? a.tokens[i] : a.page;
  if (from == -1 || to == -1 || from == to) return;
  if (from < 0 || to < 0 || from >= a.n_pages || to >= a.n_pages || n < 0 || n > a.page) {
    if (rest == 0 && lane == 0 && blockIdx.y == 0 && a.status != nullptr) atomicOr(a.status, 1);
    return;
  }
  const memra_kv_layer& layer = a.layer[blockIdx.y];
  int8_t* codes = is_v ? layer.vq : layer.kq;
  const int64_t head_bytes = (int64_t)a.page * a.D;
  const int64_t first = (int64_t)piece * kCopyPiece;
  const int bytes = (int)max((int64_t)0, min((int64_t)n * a.D - first, (int64_t)kCopyPiece));
  const uint4* s = reinterpret_cast<const uint4*>(codes + ((int64_t)from * a.Hkv + h) * head_bytes + first);
  uint4* d = reinterpret_cast<uint4*>(codes + ((int64_t)to * a.Hkv + h) * head_bytes + first);
  const int words = bytes / 16;
  for (int w = lane; w < words; w += 256) {
    uint4 v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (w + 32 * j < words) v[j] = __ldcs(s + w + 32 * j);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (w + 32 * j < words) __stcs(d + w + 32 * j, v[j]);
  }
  if (piece == 0) {
    float* scales = is_v ? layer.vd : layer.kd;
    const int per_page = a.page / a.block, count = (n + a.block - 1) / a.block;
    const float* ss = scales + ((int64_t)from * a.Hkv + h) * per_page;
    float* ds = scales + ((int64_t)to * a.Hkv + h) * per_page;
    for (int j = lane; j < count; j += 32) ds[j] = ss[j];
  }
}

// ---------------------------------------------------------------------------
// Release.  Cells of the table in order, cut evenly over the cluster's warps:
//   count   refs falls by one for each entry given up;
//   last    a page whose refs is below 0 goes, and its word then holds the least code of its
//           entries: code(e) = INT32_MIN + (cells - 1 - e), so the last entry's;
//   place   how many entries of each warp let a page go, and where each warp's begin;
//   write   the free list, and refs back to 0.
// Counts of any table that fits (2^30 cells) stay above all codes.
// ---------------------------------------------------------------------------
struct ReleaseArgs {
  Table t;
  const int32_t *keep, *free_head;
  int64_t n_free;
  int32_t *refs, *free_pages, *lens_out, *free_head_out, *status;
};

__global__ void __launch_bounds__(kThreads) release_kernel(ReleaseArgs a) {
  __shared__ Counts counts;
  pdl_launch_dependents();
  pdl_wait();
  cg::cluster_group cluster = cg::this_cluster();
  const int lane = threadIdx.x & 31, ranks = (int)cluster.num_blocks();
  const int64_t warps = (int64_t)ranks * kWarps;
  const int64_t my_warp = (int64_t)cluster.block_rank() * kWarps + (threadIdx.x >> 5);
  const int64_t cells = a.t.B * a.t.max_pages;
  const int64_t chunks = (cells + 31) / 32;
  const int64_t c0 = chunks * my_warp / warps, c1 = chunks * (my_warp + 1) / warps;
  const int64_t head = *a.free_head;
  bool bad = false;

  // the pages that the lane's cells of a tile give up, -1 for none
  int32_t page[kTile];
  auto look = [&](int64_t c, bool check) {
    int32_t len[kTile], keep[kTile];
#pragma unroll
    for (int j = 0; j < kTile; ++j) {
      const int64_t e = (c + j) * 32 + lane;
      const bool in = c + j < c1 && e < cells;
      const uint32_t b = in ? a.t.by_row((uint32_t)e) : 0;
      page[j] = in ? a.t.entries[e] : -1;
      len[j] = in ? a.t.lens[b] : 0;
      keep[j] = in && a.keep != nullptr ? a.keep[b] : 0;
    }
#pragma unroll
    for (int j = 0; j < kTile; ++j) {
      const int64_t e = (c + j) * 32 + lane;
      const bool in = c + j < c1 && e < cells;
      const int i = in ? (int)((uint32_t)e - a.t.by_row((uint32_t)e) * (uint32_t)a.t.max_pages) : 0;
      bool odd = false;
      const bool given = in && i < a.t.pages_of(len[j], &odd) && i >= a.t.pages_of(max(keep[j], 0), &odd);
      if (given && check && !a.t.is_page(page[j])) bad = true;
      if (!given || !a.t.is_page(page[j])) page[j] = -1;
    }
  };
  const bool one = c1 - c0 <= kTile;
  auto code = [&](int64_t c, int j) { return (int32_t)(INT32_MIN + (cells - 1 - ((c + j) * 32 + lane))); };

  for (int64_t c = c0; c < c1; c += kTile) {
    look(c, true);
#pragma unroll
    for (int j = 0; j < kTile; ++j)
      if (page[j] >= 0) atomicSub(a.refs + page[j], 1);
  }
  meet(cluster, ranks);
  for (int64_t c = c0; c < c1; c += kTile) {
    if (!one) look(c, false);
    int32_t r[kTile];
#pragma unroll
    for (int j = 0; j < kTile; ++j) r[j] = page[j] >= 0 ? __ldcg(a.refs + page[j]) : 0;
#pragma unroll
    for (int j = 0; j < kTile; ++j)
      if (r[j] < 0) {
        if (r[j] < -1 && r[j] > INT32_MIN / 2) bad = true;  // more often than it was held
        atomicMin(a.refs + page[j], code(c, j));
      } else {
        page[j] = -1;  // others hold it
      }
  }
  meet(cluster, ranks);
  uint32_t goes = 0;  // of one tile
  int32_t mine = 0;
  for (int64_t c = c0; c < c1; c += kTile) {
    if (!one) look(c, false);
    int32_t r[kTile];
#pragma unroll
    for (int j = 0; j < kTile; ++j) r[j] = page[j] >= 0 ? __ldcg(a.refs + page[j]) : 0;
#pragma unroll
    for (int j = 0; j < kTile; ++j) {
      const bool go = page[j] >= 0 && r[j] == code(c, j);
      goes |= (go ? 1u : 0u) << j;
      mine += __popc(__ballot_sync(kFullMask, go));
    }
  }
  int32_t before, all;
  place_of(cluster, counts, mine, &before, &all);
  int64_t to = head - all + before;
  for (int64_t c = c0; c < c1 && mine > 0; c += kTile) {
    if (!one) {
      look(c, false);
      goes = 0;
#pragma unroll
      for (int j = 0; j < kTile; ++j) goes |= (page[j] >= 0 && __ldcg(a.refs + page[j]) == code(c, j) ? 1u : 0u) << j;
    }
#pragma unroll
    for (int j = 0; j < kTile; ++j) {
      const bool go = (goes >> j) & 1u;
      const uint32_t going = __ballot_sync(kFullMask, go);
      if (go) {
        const int64_t at = to + __popc(going & ((1u << lane) - 1));
        if (at >= 0 && at < a.n_free) a.free_pages[at] = page[j];
        a.refs[page[j]] = 0;
      }
      to += __popc(going);
    }
  }
  // lengths have been read by all, in one tile even before the counts were
  int bits = bad ? 1 : 0;
  if (ranks > 1) cluster.sync();  // (and counts by the other CTAs)
  for (int64_t b = (int64_t)cluster.block_rank() * kThreads + threadIdx.x; b < a.t.B; b += (int64_t)ranks * kThreads) {
    bool odd = false;
    const int32_t len = a.t.lens[b], keep = a.keep != nullptr ? a.keep[b] : 0;
    (void)a.t.pages_of(len, &odd);
    if (odd || keep < 0) bits |= 1;
    const int32_t most = (int32_t)max((int64_t)0, min((int64_t)len, a.t.max_pages * a.t.page));
    a.lens_out[b] = min(most, max(keep, 0));
  }
  if (my_warp == 0 && lane == 0) {
    if (head - all < 0 || head > a.n_free) bits |= 4;
    *a.free_head_out = (int32_t)max((int64_t)0, head - all);
  }
  tell(bits, a.status);
}

// ---------------------------------------------------------------------------
// Compaction.  Cells and pages in order, cut evenly over the cluster's warps: the larger tables.
// ---------------------------------------------------------------------------
struct CompactArgs {
  Table t;
  int32_t *table_out, *refs, *free_out, *src, *dst, *free_head_out, *status;
};

__global__ void __launch_bounds__(kThreads) compact_kernel(CompactArgs a) {
  __shared__ Counts counts;
  pdl_launch_dependents();
  pdl_wait();
  cg::cluster_group cluster = cg::this_cluster();
  const int lane = threadIdx.x & 31;
  constexpr int64_t all_threads = kMaxRanks * kThreads;
  const int64_t me = (int64_t)cluster.block_rank() * kThreads + threadIdx.x;
  const int64_t cells = a.t.B * a.t.max_pages, n = a.t.n_pages, moves = n / 2;
  // the pages of the thread's cells, kTile at a time; of one such tile they stay in registers
  int32_t page[kTile];
  auto look = [&](int64_t e0) {
    int32_t len[kTile];
#pragma unroll
    for (int j = 0; j < kTile; ++j) {
      const int64_t e = e0 + j * all_threads;
      page[j] = e < cells ? a.t.entries[e] : -1;
      len[j] = e < cells ? a.t.lens[a.t.by_row((uint32_t)e)] : 0;
    }
    bool none = true;
#pragma unroll
    for (int j = 0; j < kTile; ++j) {
      const int64_t e = e0 + j * all_threads;
      const int i = e < cells ? (int)((uint32_t)e - a.t.by_row((uint32_t)e) * (uint32_t)a.t.max_pages) : 0;
      bool odd = false;  // told of below
      const bool held = e < cells && i < a.t.pages_of(len[j], &odd);
      if (held && !a.t.is_page(page[j])) none = false;
      if (!held || !a.t.is_page(page[j])) page[j] = -1;
    }
    return !none;
  };
  const int64_t tile = all_threads * kTile;
  const bool one = cells <= tile;
  bool bad = false;
  for (int64_t p = me; p < n; p += all_threads) a.refs[p] = 0;
  for (int64_t k = me; k < moves; k += all_threads) a.src[k] = a.dst[k] = -1;
  for (int64_t b = me; b < a.t.B; b += all_threads) (void)a.t.pages_of(a.t.lens[b], &bad);
  if (one) bad |= look(me);
  cluster.sync();
  for (int64_t e0 = me; e0 < cells; e0 += tile) {
    if (!one) bad |= look(e0);
#pragma unroll
    for (int j = 0; j < kTile; ++j)
      if (page[j] >= 0) atomicAdd(a.refs + page[j], 1);
  }
  cluster.sync();
  const int64_t warps = all_threads / 32, my_warp = me / 32, chunks = (n + 31) / 32;
  const int64_t c0 = chunks * my_warp / warps, c1 = chunks * (my_warp + 1) / warps;
  int32_t mine = 0;
  for (int64_t c = c0; c < c1; ++c) {
    const int64_t p = c * 32 + lane;
    mine += __popc(__ballot_sync(kFullMask, p < n && __ldcg(a.refs + p) > 0));
  }
  int32_t before, used;
  place_of(cluster, counts, mine, &before, &used);
  // a page below `used` that nobody holds is a hole; one from there on that is held moves: the
  // k-th hole from below takes the k-th such page from above
  for (int64_t c = c0; c < c1; ++c) {
    const int64_t p = c * 32 + lane;
    const int32_t count = p < n ? __ldcg(a.refs + p) : 0;
    const uint32_t in_use = __ballot_sync(kFullMask, count > 0);
    const int32_t below = before + __popc(in_use & ((1u << lane) - 1));
    before += __popc(in_use);
    if (p >= n) continue;
    if (p < used) {
      if (count > 0) a.refs[p] = count - 1;
      else a.dst[p - below] = (int32_t)p;
    } else if (count > 0) {
      a.src[used - 1 - below] = (int32_t)p;
      a.free_out[p] = used - 1 - below;  // for now: its move
    }
  }
  cluster.sync();
  for (int64_t e0 = me; e0 < cells; e0 += tile) {
    if (!one) (void)look(e0);
    int32_t to[kTile];
#pragma unroll
    for (int j = 0; j < kTile; ++j) to[j] = page[j] >= used ? __ldcg(a.free_out + page[j]) : -1;
#pragma unroll
    for (int j = 0; j < kTile; ++j)
      if (to[j] >= 0) page[j] = __ldcg(a.dst + to[j]);
#pragma unroll
    for (int j = 0; j < kTile; ++j)
      if (e0 + j * all_threads < cells) a.table_out[e0 + j * all_threads] = page[j];
  }
  for (int64_t p = used + me; p < n; p += all_threads) {
    const int32_t count = __ldcg(a.refs + p);
    if (count > 0) {
      a.refs[__ldcg(a.dst + __ldcg(a.free_out + p))] = count - 1;
      a.refs[p] = 0;
    }
  }
  cluster.sync();
  for (int64_t p = me; p < n; p += all_threads) a.free_out[p] = (int32_t)p;
  if (me == 0) *a.free_head_out = used;
  tell(bad ? 1 : 0, a.status);
}

// ---------------------------------------------------------------------------
// Release and compaction of a table of one tile (8192 cells) over a pool of up to 16,384 pages: one
// CTA, whose shared memory holds what is counted of each page, so that global memory is waited for
// once or twice instead of at every step.  us, so and with the steps in global memory: a release of
// all of 1024 pages 3.7 and 7.0 (by one CTA; a cluster 8.2), of 8000 8.2 and 10.6 (by a cluster; one CTA
// 25.1); compaction of 256 pages 2.9 and 8.6 (by a cluster, as the others), of 8000 7.6 and 10.0, of
// 16,384 11.3 and 11.9.
// ---------------------------------------------------------------------------
constexpr int kSmallCells = kTile * kThreads, kSmallPages = 16384;

// What the thread's cells of a small table hold: cell tid + 1024 j, -1 for nothing.  `given` says of
// a cell in use, from its row and place there, whether it counts.
template <typename Given>
__device__ __forceinline__ bool cells_of(const Table& t, int32_t* page, Given given) {
  const int cells = (int)(t.B * t.max_pages);
  int32_t len[kTile];
  uint32_t row[kTile];
#pragma unroll
  for (int j = 0; j < kTile; ++j) page[j] = -1;
#pragma unroll
  for (int j = 0; j < kTile; ++j) {
    if (j * kThreads >= cells) break;
    const int e = threadIdx.x + j * kThreads;
    row[j] = e < cells ? t.by_row((uint32_t)e) : 0;
    page[j] = e < cells ? t.entries[e] : -1;
    len[j] = e < cells ? t.lens[row[j]] : 0;
  }
  bool bad = false;
#pragma unroll
  for (int j = 0; j < kTile; ++j) {
    if (j * kThreads >= cells) break;
    const int e = threadIdx.x + j * kThreads;
    const int i = e - (int)row[j] * (int)t.max_pages;
    bool odd = false;  // lengths are told of elsewhere
    const bool counts = e < cells && i < t.pages_of(len[j], &odd) && given(row[j], i);
    if (counts && !t.is_page(page[j])) bad = true;
    if (!counts || !t.is_page(page[j])) page[j] = -1;
  }
  return bad;
}

__global__ void __launch_bounds__(kThreads) small_release_kernel(ReleaseArgs a) {
  extern __shared__ int32_t pool[];
  int32_t *left = pool, *last = pool + a.t.n_pages;  // of a page: its refs, the last cell that gives it up
  __shared__ int32_t goes_of[kTile][kWarps];
  pdl_launch_dependents();
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n = (int)a.t.n_pages;
  const int tiles = ((int)(a.t.B * a.t.max_pages) + kThreads - 1) / kThreads;  // of a thread's cells, that are any
  const int64_t head = *a.free_head;
  int32_t page[kTile];
  for (int p = tid; p < n; p += kThreads) {
    left[p] = __ldcg(a.refs + p);
    last[p] = -1;
  }
  bool bad = cells_of(a.t, page, [&](uint32_t b, int i) {
    bool odd = false;
    return a.keep == nullptr || i >= a.t.pages_of(max(a.keep[b], 0), &odd);
  });
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kTile; ++j)
    if (page[j] >= 0) {
      atomicSub(left + page[j], 1);
      atomicMax(last + page[j], tid + j * kThreads);
    }
  __syncthreads();
  uint32_t goes = 0;
#pragma unroll
  for (int j = 0; j < kTile; ++j) {
    if (j >= tiles) break;
    const bool go = page[j] >= 0 && last[page[j]] == tid + j * kThreads && left[page[j]] < 0;
    const uint32_t going = __ballot_sync(kFullMask, go);
    goes |= (go ? 1u : 0u) << j;
    if (lane == 0) goes_of[j][warp] = __popc(going);
  }
  for (int p = tid; p < n; p += kThreads) {
    if (last[p] < 0) continue;
    if (left[p] < -1) bad = true;  // more often than it was held
    a.refs[p] = max(left[p], 0);
  }
  __syncthreads();
  // cells lie in the order (j, warp, lane)
  int32_t all = 0;
  int32_t to[kTile];
#pragma unroll
  for (int j = 0; j < kTile; ++j) {
    if (j >= tiles) break;
    const int32_t v = goes_of[j][lane];
    to[j] = all + (int)__reduce_add_sync(kFullMask, lane < warp ? v : 0) +
            __popc(__ballot_sync(kFullMask, (goes >> j) & 1u) & ((1u << lane) - 1));
    all += (int)__reduce_add_sync(kFullMask, v);
  }
#pragma unroll
  for (int j = 0; j < kTile; ++j) {
    const int64_t at = head - all + to[j];
    if (((goes >> j) & 1u) && at >= 0 && at < a.n_free) a.free_pages[at] = page[j];
  }
  int bits = bad ? 1 : 0;
  for (int64_t b = tid; b < a.t.B; b += kThreads) {
    bool odd = false;
    const int32_t len = a.t.lens[b], keep = a.keep != nullptr ? a.keep[b] : 0;
    (void)a.t.pages_of(len, &odd);
    if (odd || keep < 0) bits |= 1;
    const int32_t most = (int32_t)max((int64_t)0, min((int64_t)len, a.t.max_pages * a.t.page));
    a.lens_out[b] = min(most, max(keep, 0));
  }
  if (tid == 0) {
    if (head - all < 0 || head > a.n_free) bits |= 4;
    *a.free_head_out = (int32_t)max((int64_t)0, head - all);
  }
  tell(bits, a.status);
}

__global__ void __launch_bounds__(kThreads) small_compact_kernel(CompactArgs a) {
  extern __shared__ int32_t pool[];
  const int n = (int)a.t.n_pages, cells = (int)(a.t.B * a.t.max_pages);
  int32_t *count = pool, *move = pool + n, *hole = pool + 2 * n;  // entries and the move of a page, holes from below
  __shared__ int32_t used_of[kWarps], moved;
  pdl_launch_dependents();
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int32_t page[kTile];
  bool bad = cells_of(a.t, page, [](uint32_t, int) { return true; });
  for (int64_t b = tid; b < a.t.B; b += kThreads) (void)a.t.pages_of(a.t.lens[b], &bad);
  for (int p = tid; p < n; p += kThreads) {
    count[p] = 0;
    a.free_out[p] = p;
  }
  if (tid == 0) moved = 0;
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kTile; ++j)
    if (page[j] >= 0) atomicAdd(count + page[j], 1);
  __syncthreads();
  const int chunks = (n + 31) / 32, c0 = chunks * warp / kWarps, c1 = chunks * (warp + 1) / kWarps;
  int32_t mine = 0;
  for (int c = c0; c < c1; ++c) mine += __popc(__ballot_sync(kFullMask, c * 32 + lane < n && count[c * 32 + lane] > 0));
  if (lane == 0) used_of[warp] = mine;
  __syncthreads();
  const int32_t used = (int)__reduce_add_sync(kFullMask, used_of[lane]);
  int32_t before = (int)__reduce_add_sync(kFullMask, lane < warp ? used_of[lane] : 0);
  for (int c = c0; c < c1; ++c) {
    const int p = c * 32 + lane;
    const bool held = p < n && count[p] > 0;
    const uint32_t in_use = __ballot_sync(kFullMask, held);
    const int32_t below = before + __popc(in_use & ((1u << lane) - 1));
    before += __popc(in_use);
    if (p == used) moved = used - below;
    if (p >= used) {
      if (held) {
        move[p] = used - 1 - below;
        a.src[used - 1 - below] = p;
      }
    } else if (!held) {
      hole[p - below] = p;
    }
  }
  __syncthreads();
  const int moves = moved;
  for (int k = tid; k < n / 2; k += kThreads) {
    if (k >= moves) a.src[k] = -1;
    a.dst[k] = k < moves ? hole[k] : -1;
  }
  for (int p = tid; p < n; p += kThreads) {
    const int32_t c = count[p];
    if (p < used) {
      if (c > 0) a.refs[p] = c - 1;
    } else {
      a.refs[p] = 0;
      if (c > 0) a.refs[hole[move[p]]] = c - 1;
    }
  }
#pragma unroll
  for (int j = 0; j < kTile; ++j) {
    const int e = tid + j * kThreads;
    if (e < cells) a.table_out[e] = page[j] >= used ? hole[move[page[j]]] : page[j];
  }
  if (tid == 0) *a.free_head_out = used;
  tell(bad ? 1 : 0, a.status);
}

// ---------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------

// Bytes at an address.
struct Span {
  const void* at;
  int64_t words;  // of 4 bytes
  bool meets(const Span& o) const {
    const uintptr_t a = (uintptr_t)at, b = (uintptr_t)o.at;
    return at != nullptr && o.at != nullptr && words > 0 && o.words > 0 && a < b + 4 * (uint64_t)o.words &&
           b < a + 4 * (uint64_t)words;
  }
};

// Outputs lie apart from each other and from the inputs; `same` lists pairs (output, input) that
// may be one array.
struct Pair {
  const void *out, *in;
};
bool lie_apart(std::initializer_list<Span> outs, std::initializer_list<Span> ins, std::initializer_list<Pair> same) {
  for (const Span* o = outs.begin(); o != outs.end(); ++o) {
    for (const Span* p = outs.begin(); p != o; ++p)
      if (o->meets(*p)) return false;
    for (const Span& i : ins) {
      bool in_place = false;
      for (const Pair& s : same) in_place |= s.out == o->at && s.in == i.at && s.out == s.in;
      if (!in_place && o->meets(i)) return false;
    }
  }
  return true;
}

memra_status table_args(const int32_t* lens, const int32_t* entries, int64_t B, int64_t max_pages, int64_t page_size,
                        int64_t n_pages, Table* t) {
  if (B < 0 || max_pages < 0 || n_pages < 0) return MEMRA_ERR_INVALID_ARG;
  if (page_size < 16 || page_size % 16 != 0) return MEMRA_ERR_INVALID_ARG;
  if (page_size > MEMRA_MAX_KV_PAGE || n_pages > INT32_MAX / page_size || B > (1 << 24) || max_pages > (1 << 30) ||
      B * max_pages > (1 << 30))
    return MEMRA_ERR_UNSUPPORTED;
  if (B > 0 && (!lens || (max_pages > 0 && !entries))) return MEMRA_ERR_INVALID_ARG;
  if (!aligned(lens, 4) || !aligned(entries, 4)) return MEMRA_ERR_ALIGNMENT;
  t->lens = lens;
  t->entries = entries;
  t->B = B;
  t->max_pages = max_pages;
  t->n_pages = n_pages;
  t->page = (int)page_size;
  t->by_page = Divider((uint32_t)page_size);
  t->by_row = Divider((uint32_t)(max_pages > 0 ? max_pages : 1));
  return MEMRA_OK;
}

bool words_aligned(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (!aligned(p, 4)) return false;
  return true;
}

// One cluster of so many CTAs.
template <typename Args>
cudaError_t launch_cluster(void (*kernel)(Args), unsigned ranks, cudaStream_t stream, const Args& a) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ranks);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ranks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

// The one CTA of a small table, with so many bytes of shared memory to a page.
template <typename Args>
cudaError_t launch_small(void (*kernel)(Args), int bytes, cudaStream_t stream, const Args& a) {
  const int smem = bytes * (int)a.t.n_pages;
  if (smem > 32 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes * kSmallPages);
    if (e != cudaSuccess) return e;
  }
  return launch_kernel(kernel, dim3(1), dim3(kThreads), (size_t)smem, stream, a);
}

bool is_small(const Table& t) { return t.B * t.max_pages <= kSmallCells && t.n_pages <= kSmallPages; }

}  // namespace
}  // namespace memra

using namespace memra;

extern "C" memra_status memra_kv_fork(const int32_t* parents, const int32_t* prefix_lens, int64_t C,
                                      const int32_t* lens, const int32_t* block_table, int64_t B,
                                      int64_t max_pages, int64_t page_size, int32_t* refs,
                                      int64_t n_pages, int32_t* lens_out, int32_t* table_out,
                                      int32_t* dev_status, cudaStream_t stream) {
  ForkArgs a;
  const memra_status st = table_args(lens, block_table, B, max_pages, page_size, n_pages, &a.t);
  if (st != MEMRA_OK) return st;
  if (C < 0) return MEMRA_ERR_INVALID_ARG;
  if (C > (1 << 24) || C * max_pages > (1 << 30)) return MEMRA_ERR_UNSUPPORTED;
  if (C == 0) return MEMRA_OK;
  if (!parents || !lens_out || (max_pages > 0 && !table_out) || (n_pages > 0 && !refs)) return MEMRA_ERR_INVALID_ARG;
  if (!words_aligned({parents, prefix_lens, refs, lens_out, table_out, dev_status})) return MEMRA_ERR_ALIGNMENT;
  if (!lie_apart({{lens_out, C}, {table_out, C * max_pages}, {refs, n_pages}, {dev_status, 1}},
                 {{parents, C}, {prefix_lens, C}, {lens, B}, {block_table, B * max_pages}}, {}))
    return MEMRA_ERR_INVALID_ARG;
  a.parents = parents;
  a.prefix = prefix_lens;
  a.refs = refs;
  a.lens_out = lens_out;
  a.table_out = table_out;
  a.status = dev_status;
  const cudaError_t e = launch_kernel(fork_kernel, dim3((unsigned)C), dim3(kForkThreads), 0, stream, a);
  if (e != cudaSuccess) return cuda_fail(e);
  return MEMRA_OK;
}

extern "C" memra_status memra_kv_unshare(const int32_t* lens, const int32_t* new_lens, int64_t B,
                                         int64_t page_size, int32_t* refs, int64_t n_pages,
                                         const int32_t* free_pages, int64_t n_free,
                                         const int32_t* free_head, int32_t* block_table,
                                         int64_t max_pages, int32_t* new_lens_out, int32_t* src,
                                         int32_t* dst, int32_t* tokens, int32_t* free_head_out,
                                         int32_t* dev_status, cudaStream_t stream) {
  UnshareArgs a;
  const memra_status st = table_args(lens, block_table, B, max_pages, page_size, n_pages, &a.t);
  if (st != MEMRA_OK) return st;
  if (n_free < 0) return MEMRA_ERR_INVALID_ARG;
  if (n_free > INT32_MAX) return MEMRA_ERR_UNSUPPORTED;
  if (!free_head_out || (n_free > 0 && !free_pages) || (n_pages > 0 && !refs)) return MEMRA_ERR_INVALID_ARG;
  if (B > 0 && (!new_lens || !new_lens_out || !src || !dst || !tokens)) return MEMRA_ERR_INVALID_ARG;
  if (!words_aligned({new_lens, refs, free_pages, free_head, new_lens_out, src, dst, tokens, free_head_out, dev_status}))
    return MEMRA_ERR_ALIGNMENT;
  if (!lie_apart({{block_table, B * max_pages}, {refs, n_pages}, {new_lens_out, B}, {src, B}, {dst, B}, {tokens, B},
                  {free_head_out, 1}, {dev_status, 1}},
                 {{lens, B}, {new_lens, B}, {free_pages, n_free}, {free_head, 1}},
                 {{new_lens_out, new_lens}, {free_head_out, free_head}}))
    return MEMRA_ERR_INVALID_ARG;
  a.new_lens = new_lens;
  a.free_pages = free_pages;
  a.free_head = free_head;
  a.n_free = n_free;
  a.refs = refs;
  a.table = block_table;
  a.new_out = new_lens_out;
  a.src = src;
  a.dst = dst;
  a.tokens = tokens;
  a.free_head_out = free_head_out;
  a.status = dev_status;
  const int threads = B >= kThreads ? kThreads : (int)((B + 31) / 32 * 32);
  const cudaError_t e = launch_kernel(unshare_kernel, dim3(1), dim3(threads > 0 ? threads : 32), 0, stream, a);
  if (e != cudaSuccess) return cuda_fail(e);
  return MEMRA_OK;
}

extern "C" memra_status memra_kv_copy_pages(const int32_t* src, const int32_t* dst, const int32_t* tokens,
                                            int64_t N, const memra_kv_layer* layers, int64_t n_layers,
                                            int64_t n_pages, int64_t Hkv, int64_t page_size, int64_t D,
                                            int64_t block, int32_t* dev_status, cudaStream_t stream) {
  if (N < 0 || n_layers < 0 || n_pages < 0 || Hkv < 1) return MEMRA_ERR_INVALID_ARG;
  if (page_size < 16 || page_size % 16 != 0 || block < 1 || page_size % block != 0) return MEMRA_ERR_INVALID_ARG;
  if (D != 64 && D != 128 && D != 256) return MEMRA_ERR_UNSUPPORTED;
  if (page_size > MEMRA_MAX_KV_PAGE || Hkv > 32767 || n_pages > INT32_MAX / page_size) return MEMRA_ERR_UNSUPPORTED;
  if (N == 0 || n_layers == 0) return MEMRA_OK;
  if (!src || !dst || !layers) return MEMRA_ERR_INVALID_ARG;
  if (!words_aligned({src, dst, tokens, dev_status})) return MEMRA_ERR_ALIGNMENT;
  for (int64_t l = 0; l < n_layers; ++l) {
    const memra_kv_layer& x = layers[l];
    if (n_pages > 0 && (!x.kq || !x.kd || !x.vq || !x.vd)) return MEMRA_ERR_INVALID_ARG;
    if (!aligned(x.kq, 16) || !aligned(x.vq, 16) || !aligned(x.kd, 4) || !aligned(x.vd, 4)) return MEMRA_ERR_ALIGNMENT;
    const int64_t codes = n_pages * Hkv * page_size * D / 4, scales = n_pages * Hkv * (page_size / block);
    for (const Span& plane : {Span{x.kq, codes}, Span{x.vq, codes}, Span{x.kd, scales}, Span{x.vd, scales}})
      for (const Span& list : {Span{src, N}, Span{dst, N}, Span{tokens, N}, Span{dev_status, 1}})
        if (plane.meets(list)) return MEMRA_ERR_INVALID_ARG;
  }
  CopyArgs a;
  a.src = src;
  a.dst = dst;
  a.tokens = tokens;
  a.N = N;
  a.n_pages = n_pages;
  a.Hkv = (int)Hkv;
  a.page = (int)page_size;
  a.D = (int)D;
  a.block = (int)block;
  a.pieces = (int)((page_size * D + kCopyPiece - 1) / kCopyPiece);
  a.status = dev_status;
  const int64_t per_entry = 2 * Hkv * a.pieces;
  if (N > ((int64_t)INT32_MAX - 1) * kCopyWarps / per_entry) return MEMRA_ERR_UNSUPPORTED;
  const int64_t ctas = (N * per_entry + kCopyWarps - 1) / kCopyWarps;
  for (int64_t l = 0; l < n_layers; l += kCopyLayers) {
    const int count = (int)(n_layers - l < kCopyLayers ? n_layers - l : kCopyLayers);
    for (int i = 0; i < count; ++i) a.layer[i] = layers[l + i];
    const cudaError_t e = launch_kernel(copy_kernel, dim3((unsigned)ctas, (unsigned)count), dim3(kCopyWarps * 32), 0, stream, a);
    if (e != cudaSuccess) return cuda_fail(e);
  }
  return MEMRA_OK;
}

extern "C" memra_status memra_kv_release(const int32_t* lens, const int32_t* keep_lens, int64_t B,
                                         int64_t page_size, const int32_t* block_table,
                                         int64_t max_pages, int32_t* refs, int64_t n_pages,
                                         int32_t* free_pages, int64_t n_free,
                                         const int32_t* free_head, int32_t* lens_out,
                                         int32_t* free_head_out, int32_t* dev_status,
                                         cudaStream_t stream) {
  ReleaseArgs a;
  const memra_status st = table_args(lens, block_table, B, max_pages, page_size, n_pages, &a.t);
  if (st != MEMRA_OK) return st;
  if (n_free < 0) return MEMRA_ERR_INVALID_ARG;
  if (n_free > INT32_MAX) return MEMRA_ERR_UNSUPPORTED;
  if (!free_head || !free_head_out || (n_free > 0 && !free_pages) || (n_pages > 0 && !refs) || (B > 0 && !lens_out))
    return MEMRA_ERR_INVALID_ARG;
  if (!words_aligned({keep_lens, refs, free_pages, free_head, lens_out, free_head_out, dev_status})) return MEMRA_ERR_ALIGNMENT;
  if (!lie_apart({{refs, n_pages}, {free_pages, n_free}, {lens_out, B}, {free_head_out, 1}, {dev_status, 1}},
                 {{lens, B}, {keep_lens, B}, {block_table, B * max_pages}, {free_head, 1}},
                 {{lens_out, lens}, {free_head_out, free_head}}))
    return MEMRA_ERR_INVALID_ARG;
  a.keep = keep_lens;
  a.free_head = free_head;
  a.n_free = n_free;
  a.refs = refs;
  a.free_pages = free_pages;
  a.lens_out = lens_out;
  a.free_head_out = free_head_out;
  a.status = dev_status;
  const cudaError_t e = is_small(a.t) ? launch_small(small_release_kernel, 8, stream, a)
                                      : launch_cluster(release_kernel, B * max_pages <= kSmallCells ? 1 : kMaxRanks, stream, a);
  if (e != cudaSuccess) return cuda_fail(e);
  return MEMRA_OK;
}

extern "C" memra_status memra_kv_compact(const int32_t* lens, const int32_t* block_table, int64_t B,
                                         int64_t max_pages, int64_t page_size, int64_t n_pages,
                                         int32_t* table_out, int32_t* refs_out, int32_t* free_out,
                                         int32_t* src, int32_t* dst, int32_t* free_head_out,
                                         int32_t* dev_status, cudaStream_t stream) {
  CompactArgs a;
  const memra_status st = table_args(lens, block_table, B, max_pages, page_size, n_pages, &a.t);
  if (st != MEMRA_OK) return st;
  if (!free_head_out || (n_pages > 0 && (!refs_out || !free_out)) || (n_pages > 1 && (!src || !dst)) ||
      (B * max_pages > 0 && !table_out))
    return MEMRA_ERR_INVALID_ARG;
  if (!words_aligned({table_out, refs_out, free_out, src, dst, free_head_out, dev_status})) return MEMRA_ERR_ALIGNMENT;
  if (!lie_apart({{table_out, B * max_pages}, {refs_out, n_pages}, {free_out, n_pages}, {src, n_pages / 2},
                  {dst, n_pages / 2}, {free_head_out, 1}, {dev_status, 1}},
                 {{lens, B}, {block_table, B * max_pages}}, {{table_out, block_table}}))
    return MEMRA_ERR_INVALID_ARG;
  a.table_out = table_out;
  a.refs = refs_out;
  a.free_out = free_out;
  a.src = src;
  a.dst = dst;
  a.free_head_out = free_head_out;
  a.status = dev_status;
  const cudaError_t e = is_small(a.t) ? launch_small(small_compact_kernel, 10, stream, a)
                                      : launch_cluster(compact_kernel, kMaxRanks, stream, a);
  if (e != cudaSuccess) return cuda_fail(e);
  return MEMRA_OK;
}
