// pages.cu -- the pages of the resident tier: grow, fork, free and compact
// (hisparse_pages_* of include/hisparse.h).
//
// Two launches at most.  A plan kernel (one cluster of kPlanCtas CTAs) settles which
// pages go where: each CTA scans a slice of the reference counts, the slices' totals
// meet in distributed shared memory, and every rank below is the exact rank in
// page order or list order, so results depend on no timing.  Then a copy kernel
// over the whole GPU moves the bytes of the pages in the plan.
#include <cooperative_groups.h>

#include <algorithm>
#include <climits>

#include "common.cuh"

namespace cg = cooperative_groups;

namespace {

constexpr int kPlanCtas = 8;
constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;

// d_work: word 0 the number of copies, word 1 the pages in use; then three arrays of `span`
// = max(num_pages, num_requests) words: the pages copied from, the pages copied to,
// and the rows of each copy (fork) or which move is each page's (compact).  With
// grow and fork the third array first holds the list's demands, and the second the free
// pages by rank.
constexpr int kWorkHead = 16;

struct PoolArgs {
  int32_t pages, R, blocks, page_tokens, layers;
  int64_t row_bytes, layer_stride, page_stride;
  char *store;
  int32_t *tables, *refs, *work;
  uint32_t *status;
  int32_t span, n;
  const int32_t *src, *dst, *want;  // fork: tokens in want; grow: blocks in want
};

__device__ __forceinline__ void report(const PoolArgs &a, uint32_t bit) {
  if (a.status) atomicOr(a.status, bit);
}

// Sum over the CTA and this thread's exclusive prefix; all threads call it.
__device__ __forceinline__ int block_scan(int v, int *warp_sums, int &total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) warp_sums[w] = x;
  __syncthreads();
  const int s = warp_sums[lane];  // kPlanWarps == 32
  int t = s;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, t, o);
    if (lane >= o) t += y;
  }
  total = __shfl_sync(0xffffffffu, t, 31);
  const int before = __shfl_sync(0xffffffffu, t - s, w);
  return before + x - v;
}
// The same of values up to `most` (at most 2^30 + 1) whose sums stay at it once they reach it.
__device__ __forceinline__ uint32_t block_scan_to(uint32_t v, uint32_t most, int *warp_sums, uint32_t &total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  uint32_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x = min(x + y, most);
  }
  __syncthreads();
  if (lane == 31) warp_sums[w] = x;
  __syncthreads();
  uint32_t t = warp_sums[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, t, o);
    if (lane >= o) t = min(t + y, most);
  }
  total = __shfl_sync(0xffffffffu, t, 31);
  const uint32_t before = __shfl_sync(0xffffffffu, t, max(w - 1, 0)), left = __shfl_up_sync(0xffffffffu, x, 1);
  return min((w > 0 ? before : 0) + (lane > 0 ? left : 0), most);
}

// Every CTA of the cluster learns the totals of all CTAs: `tell`, a cluster barrier, `learn`, which
// returns the sum of the lower ranks' and, in `all`, of all.
__device__ __forceinline__ void tell(int mine, int *slot) {
  cg::cluster_group c = cg::this_cluster();
  if (threadIdx.x < kPlanCtas) *c.map_shared_rank(slot + c.block_rank(), threadIdx.x) = mine;
}
__device__ __forceinline__ int learn(const int *slot, int &all) {
  const int rank = cg::this_cluster().block_rank();
  int before = 0;
  all = 0;
  for (int i = 0; i < kPlanCtas; ++i) {
    if (i < rank) before += slot[i];
    all += slot[i];
  }
  return before;
}

struct Slice {
  int lo, hi;
};
__device__ __forceinline__ Slice slice_of(int total, int rank) {
  const int per = ((total + kPlanCtas - 1) / kPlanCtas + 31) & ~31;
  const int lo = min(total, rank * per);
  return {lo, min(total, lo + per)};
}

// A slice in words of 32 pages: a warp takes `words` words in a row, at most 32, and lane j keeps
// word j as bits, so that ranks are exclusive sums over threads and a word's pages are read and
// listed side by side.  A CTA's round is at most 32 K pages: the pools of a GPU's memory take one or a few.
struct Words {
  int words, round;  // of a warp; pages of the CTA
  __device__ explicit Words(const Slice &s)
      : words(min(32, max(1, (s.hi - s.lo + 1023) / 1024))), round(words * 1024) {}
  __device__ int first(int p0) const { return p0 + (threadIdx.x >> 5) * words * 32; }  // of the warp
};
// The warp's words from page p on: pages in use, or free ones.
template <bool kFree>
__device__ __forceinline__ uint32_t page_bits(const PoolArgs &a, int p, int hi, int words) {
  const int lane = threadIdx.x & 31;
  uint32_t mine = 0;
  for (int w0 = 0; w0 < words; w0 += 8) {
    int v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int q = p + 32 * (w0 + u) + lane;
      v[u] = w0 + u < words && q < hi ? a.refs[q] : -1;
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const uint32_t bits = __ballot_sync(0xffffffffu, kFree ? v[u] == 0 : v[u] > 0);
      if (lane == w0 + u) mine = bits;
    }
  }
  return mine;
}

// The free pages of the slice: their number (the thread's of the first round in `bits`).
__device__ int count_free(const PoolArgs &a, const Slice &s, const Words &w, uint32_t &bits) {
  int count = 0;
  for (int p0 = s.lo; p0 < s.hi; p0 += w.round) {
    const uint32_t b = page_bits<true>(a, w.first(p0), s.hi, w.words);
    if (p0 == s.lo) bits = b;
    count += __popc(b);
  }
  return count;
}
// The slice's free pages into list[base ...], as far as list[need - 1].
__device__ void list_free(const PoolArgs &a, const Slice &s, const Words &w, uint32_t bits, int base, int need,
                          int *list, int *warp_sums) {
  const int lane = threadIdx.x & 31;
  for (int p0 = s.lo; p0 < s.hi && base < need; p0 += w.round) {
    const int p = w.first(p0);
    if (p0 != s.lo) bits = page_bits<true>(a, p, s.hi, w.words);
    int total;
    const int k = base + block_scan(__popc(bits), warp_sums, total);
    for (int j = 0; j < w.words; ++j) {
      const uint32_t b = __shfl_sync(0xffffffffu, bits, j);
      const int at = __shfl_sync(0xffffffffu, k, j) + __popc(b & ((1u << lane) - 1));
      if ((b >> lane & 1) && at < need) list[at] = p + 32 * j + lane;
    }
    base += total;
  }
}

// ---------------------------------------------------------------------------
// Grow and fork.  Demands of the list's entries -> ranks -> free pages -> tables.  Bound by the
// latency of about eight dependent reads of L2 and three cluster barriers: a fork of 32 in a pool of 4096 pages takes
// 12 us with its copy; 40 requests freed and 40 grown by up to 1024 blocks in 200,003 pages 18 us (21
// with one warp to a request, 33 with 32 pages to a thread in place of a word of 32 to a warp too).
// ---------------------------------------------------------------------------
struct ForkNeed {
  bool ok;
  int full, part, last;  // shared blocks, rows of the part-filled one, its page (-1: none)
};
__device__ __forceinline__ ForkNeed fork_need(const PoolArgs &a, int i) {
  ForkNeed f = {false, 0, 0, -1};
  const int s = a.src[i], d = a.dst[i], t = a.want[i];
  if (s < 0 || s >= a.R || d < 0 || d >= a.R || t < 0) return f;
  f.full = t / a.page_tokens;
  f.part = t - f.full * a.page_tokens;
  if (f.full > a.blocks || (f.full == a.blocks && f.part)) return f;
  f.ok = true;
  if (f.part) f.last = a.tables[static_cast<int64_t>(s) * a.blocks + f.full];
  return f;
}

// Blocks [lo, hi) of `total` for warp `part` of the `parts` of an entry.
__device__ __forceinline__ Slice part_of(int total, int part, int parts) {
  const int per = ((total + parts - 1) / parts + 31) & ~31;
  const int lo = min(total, part * per);
  return {lo, min(total, lo + per)};
}
// What entry i asks for, as far as this warp's part of it goes; INT_MIN: it is skipped.
template <bool kFork>
__device__ int demand_of(const PoolArgs &a, int i, int part, int parts) {
  const int lane = threadIdx.x & 31;
  if (kFork) {
    const ForkNeed f = fork_need(a, i);
    bool empty = f.ok;
    if (f.ok) {
      const int32_t *row = a.tables + static_cast<int64_t>(a.dst[i]) * a.blocks;
      const Slice s = part_of(a.blocks, part, parts);
#pragma unroll 8
      for (int b = s.lo + lane; b < s.hi; b += 32) empty &= row[b] == -1;
    }
    if (!__all_sync(0xffffffffu, empty)) return INT_MIN;
    return part == 0 && f.last >= 0 ? 1 : 0;
  }
  const int r = a.src[i], w = a.want[i];
  if (r < 0 || r >= a.R || w < 0 || w > a.blocks) return INT_MIN;
  const int32_t *row = a.tables + static_cast<int64_t>(r) * a.blocks;
  const Slice s = part_of(w, part, parts);
  int k = 0;
#pragma unroll 8
  for (int b = s.lo + lane; b < s.hi; b += 32) k += row[b] == -1;
  return __reduce_add_sync(0xffffffffu, k);
}
// A fork's shared blocks, as far as this part goes; part 0 gives it the new last page, if it needs
// one, and notes the rows to copy.
__device__ void fork_entry(const PoolArgs &a, int i, int part, int parts, int need, int r0, const int32_t *to,
                           int32_t *from, int32_t *rows_of) {
  const int lane = threadIdx.x & 31;
  int rows = 0, last = -1;
  if (need >= 0 && r0 >= 0) {
    const ForkNeed f = fork_need(a, i);
    const int32_t *src = a.tables + static_cast<int64_t>(a.src[i]) * a.blocks;
    int32_t *dst = a.tables + static_cast<int64_t>(a.dst[i]) * a.blocks;
    const Slice s = part_of(f.full, part, parts);
    for (int b = s.lo + lane; b < s.hi; b += 32) {
      const int p = src[b];
      if (p >= 0 && p < a.pages) {
        dst[b] = p;
        atomicAdd(a.refs + p, 1);
      } else if (p != -1) {
        report(a, HISPARSE_ERR_RANGE);
      }
    }
    if (part == 0 && need && f.last >= a.pages) {
      report(a, HISPARSE_ERR_RANGE);
    } else if (part == 0 && need) {
      rows = f.part;
      last = f.last;
      if (lane == 0) {
        dst[f.full] = to[r0];
        a.refs[to[r0]] = 1;
      }
    }
  } else if (need >= 0 && part == 0 && lane == 0) {
    report(a, HISPARSE_ERR_FULL);
  }
  // copy i: `rows` rows (0: none) of page `last`, in the places that the warp's lanes have read
  // this entry's demand and rank from
  __syncwarp();
  if (part == 0 && lane == 0) {
    rows_of[i] = rows;
    from[i] = last;
  }
}
// The pages of rank r ... for the holes of this part of a request's blocks.
__device__ void grow_entry(const PoolArgs &a, int i, int part, int parts, int r, const int32_t *to) {
  const int lane = threadIdx.x & 31;
  int32_t *row = a.tables + static_cast<int64_t>(a.src[i]) * a.blocks;
  const Slice s = part_of(a.want[i], part, parts);
  for (int b0 = s.lo; b0 < s.hi; b0 += 8 * 32) {
    bool hole[8];
    int at[8], page[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int b = b0 + 32 * u + lane;
      hole[u] = b < s.hi && row[b] == -1;
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const unsigned m = __ballot_sync(0xffffffffu, hole[u]);
      at[u] = r + __popc(m & ((1u << lane) - 1));
      r += __popc(m);
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) page[u] = hole[u] ? to[at[u]] : 0;
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (hole[u]) {
        row[b0 + 32 * u + lane] = page[u];
        a.refs[page[u]] = 1;
      }
  }
}

template <bool kFork>
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const PoolArgs a) {
  __shared__ int warp_sums[32], slot[kPlanCtas], s_part[kPlanWarps];
  pdl_wait();
  pdl_launch();
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = cluster.block_rank(), lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int kGWarps = kPlanCtas * kPlanWarps;
  int32_t *from = a.work + kWorkHead, *to = from + a.span, *third = to + a.span;
  // An entry has `parts` warps of one CTA, where its blocks give each four for a lane and the whole
  // list has warps at once; the list goes over all CTAs.
  int parts = 8;
  while (parts > 1 && (a.n * parts > kGWarps || 128 * parts > a.blocks)) parts >>= 1;
  const int first = warp / parts * kPlanCtas + rank, part = warp % parts;

  cluster.barrier_arrive();  // (every CTA runs before another writes its shared memory)
  const Slice slice = slice_of(a.pages, rank);
  const Words words(slice);
  uint32_t bits = 0;
  int total;
  block_scan(count_free(a, slice, words, bits), warp_sums, total);
  // demand of each entry; INT_MIN marks one that is skipped
  for (int i = first; i < a.n; i += kGWarps) {
    const int need = demand_of<kFork>(a, i, part, parts);
    if (lane == 0) s_part[warp] = need;
    if (parts == 1 && lane == 0) {
      third[i] = need;
      if (need == INT_MIN) report(a, HISPARSE_ERR_RANGE);
    }
  }
  if (parts > 1) {  // (one turn of the loop above)
    __syncthreads();
    if (lane == 0 && part == 0 && first < a.n) {
      int need = 0;
      for (int p = 0; p < parts; ++p) need = need == INT_MIN || s_part[warp + p] == INT_MIN ? INT_MIN : need + s_part[warp + p];
      third[first] = need;
      if (need == INT_MIN) report(a, HISPARSE_ERR_RANGE);
    }
  }
  cluster.barrier_wait();
  tell(total, slot);
  cluster.sync();
  // every CTA ranks the whole list: thread t takes a run of entries.  (The list may ask for more than
  // 2^31 pages, and its first entries still get theirs: one more than there are pages is all that counts.)
  const int run = (a.n + kPlanThreads - 1) / kPlanThreads;
  const int i0 = min(a.n, static_cast<int>(threadIdx.x) * run), i1 = min(a.n, i0 + run);
  const uint32_t most = a.pages + 1u;
  uint32_t mine = 0, demand;
  for (int i = i0; i < i1; ++i) mine = min(mine + min(static_cast<uint32_t>(max(0, third[i])), most), most);
  uint32_t at = block_scan_to(mine, most, warp_sums, demand);
  int free_pages;
  const int before = learn(slot, free_pages);
  list_free(a, slice, words, bits, before, static_cast<int>(min(demand, most - 1)), to, warp_sums);
  // the demands that fit are a prefix of the list; `from` keeps each entry's first rank
  for (int i = i0; i < i1; ++i) {
    const uint32_t need = min(static_cast<uint32_t>(max(0, third[i])), most);
    if (rank == 0) from[i] = need > 0 && at + need > static_cast<uint32_t>(free_pages) ? -1 : static_cast<int>(at);
    at = min(at + need, most);
  }
  cluster.sync();  // the free list, the ranks; everyone has read every demand
  if (kFork) {
    int need = first < a.n ? third[first] : 0, r0 = first < a.n ? from[first] : 0;
    if (parts > 1) __syncthreads();  // part 0 writes over what the others have read here
    for (int i = first; i < a.n; i += kGWarps) {
      if (i != first) need = third[i], r0 = from[i];
      fork_entry(a, i, part, parts, need, r0, to, from, third);
    }
  } else {
    for (int i = first; i < a.n; i += kGWarps) {
      const int need = third[i];
      int r = from[i];
      if (need <= 0) continue;
      if (r < 0) {
        if (lane == 0 && part == 0) report(a, HISPARSE_ERR_FULL);
        continue;
      }
      for (int p = 0; p < part; ++p) r += s_part[warp - part + p];
      grow_entry(a, i, part, parts, r, to);
    }
  }
}

// ---------------------------------------------------------------------------
// Compact: with m pages in use, the j-th page in use at or above m moves to
// the j-th free page below m.  Rank of a free page p < m: p - used before p;
// of a mover p >= m: used before p - used before m.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(kPlanThreads) compact_plan_kernel(const PoolArgs a) {
  __shared__ int warp_sums[32], slot[kPlanCtas], slot2[kPlanCtas];
  pdl_wait();
  pdl_launch();
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = cluster.block_rank();
  int32_t *from = a.work + kWorkHead, *to = from + a.span, *moved = to + a.span;
  const int lane = threadIdx.x & 31;
  const Slice s = slice_of(a.pages, rank);
  const Words words(s);
  int total, m, low;
  cluster.barrier_arrive();  // (every CTA runs before another writes its shared memory)
  uint32_t bits = 0;
  int count = 0;
  for (int p0 = s.lo; p0 < s.hi; p0 += words.round) {
    const uint32_t b = page_bits<false>(a, words.first(p0), s.hi, words.words);
    if (p0 == s.lo) bits = b;
    count += __popc(b);
  }
  block_scan(count, warp_sums, total);
  cluster.barrier_wait();
  tell(total, slot);
  cluster.sync();
  const int before = learn(slot, m);
  // used pages below m
  count = 0;
  for (int p0 = s.lo; p0 < min(s.hi, m); p0 += words.round) {
    const int p = words.first(p0), below = m - (p + 32 * lane);  // of this lane's word
    const uint32_t b = p0 == s.lo ? bits : page_bits<false>(a, p, s.hi, words.words);
    count += __popc(b & (below >= 32 ? ~0u : below > 0 ? (1u << below) - 1 : 0u));
  }
  block_scan(count, warp_sums, total);
  tell(total, slot2);
  cluster.sync();
  learn(slot2, low);
  int base = before;
  for (int p0 = s.lo; p0 < s.hi; p0 += words.round) {
    const int p = words.first(p0);
    if (p0 != s.lo) bits = page_bits<false>(a, p, s.hi, words.words);
    const int k = base + block_scan(__popc(bits), warp_sums, total);
    for (int j = 0; j < words.words; ++j) {
      const uint32_t b = __shfl_sync(0xffffffffu, bits, j);
      const int used = __shfl_sync(0xffffffffu, k, j) + __popc(b & ((1u << lane) - 1));
      const int q = p + 32 * j + lane;
      if (q >= s.hi) continue;
      if (b >> lane & 1) {
        if (q >= m) from[used - low] = q;
      } else if (q < m) {
        to[q - used] = q;
      }
    }
    base += total;
  }
  cluster.sync();
  const int movers = m - low;
  for (int j = rank * kPlanThreads + threadIdx.x; j < movers; j += kPlanCtas * kPlanThreads) {
    const int f = from[j], t = to[j];
    moved[f] = j;
    a.refs[t] = a.refs[f];
    a.refs[f] = 0;
  }
  if (rank == 0 && threadIdx.x == 0) {
    a.work[0] = movers;
    a.work[1] = m;
  }
}

// ---------------------------------------------------------------------------
// page_copy_kernel: the bytes of the plan's pages in every layer, in 16-byte
// chunks over the whole grid, kCopyUnroll reads of a thread in flight.  For a
// fork, copy i goes to the part-filled block of its destination's table row.  For a
// compaction the table entries above the used pages follow their pages too.  Bound by one
// read and one write of the pages: 1.7 thousand pages of 36 KB in 4 layers (512 MB of traffic) take 88 us with
// their plan, 5.8 TB/s.
// ---------------------------------------------------------------------------
constexpr int kCopyThreads = 512;
constexpr int kCopyUnroll = 4;
constexpr int kCopyCtas = 152 * 4;
constexpr int kPiece = 1024;  // 16-byte chunks

template <bool kFork>
__global__ void __launch_bounds__(kCopyThreads) page_copy_kernel(const PoolArgs a) {
  pdl_wait();
  pdl_launch();
  const int32_t *from = a.work + kWorkHead, *to = from + a.span, *third = to + a.span;
  const int copies = kFork ? a.n : a.work[0];
  const int64_t tid = static_cast<int64_t>(blockIdx.x) * kCopyThreads + threadIdx.x;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kCopyThreads;
  if (!kFork) {
    const int m = a.work[1];
    for (int64_t e = tid; e < static_cast<int64_t>(a.R) * a.blocks; e += step) {
      const int p = a.tables[e];
      if (p < m) continue;
      // Its move, if the list of moves says so too: a page that no count stands for has none, and an
      // earlier call's word in the place of it.
      const int j = p < a.pages ? third[p] : -1;
      if (j >= 0 && j < copies && from[j] == p) {
        a.tables[e] = to[j];
      } else {
        report(a, HISPARSE_ERR_RANGE);
      }
    }
  }
  // Pieces of 16 KB (or a page, where it is smaller) of every copy in every layer, a half CTA to a
  // piece in turn; pages under 1 KB a warp to a page.
  const int64_t page = static_cast<int64_t>(a.page_tokens) * a.row_bytes / 16;  // chunks of 16 bytes
  const int pieces = static_cast<int>((page + kPiece - 1) / kPiece);
  const int team = page <= 64 ? 32 : 256;  // threads to a piece
  const int64_t items = static_cast<int64_t>(copies) * a.layers * pieces;
  const int in = threadIdx.x & (team - 1);
  for (int64_t it = tid / team; it < items; it += step / team) {
    const int64_t cl = it / pieces;
    const int64_t first = (it - cl * pieces) * kPiece;
    const int c = static_cast<int>(cl / a.layers), l = static_cast<int>(cl - static_cast<int64_t>(c) * a.layers);
    int64_t chunks = page;
    int dst;
    if (kFork) {
      chunks = third[c] * a.row_bytes / 16;
      if (chunks <= first) continue;
      dst = a.tables[static_cast<int64_t>(a.dst[c]) * a.blocks + a.want[c] / a.page_tokens];
      if (dst < 0 || dst >= a.pages) continue;
    } else {
      dst = to[c];
    }
    const uint4 *s = reinterpret_cast<const uint4 *>(a.store + l * a.layer_stride +
                                                     static_cast<int64_t>(from[c]) * a.page_stride) + first;
    uint4 *d = reinterpret_cast<uint4 *>(a.store + l * a.layer_stride +
                                         static_cast<int64_t>(dst) * a.page_stride) + first;
    const int n = static_cast<int>(min(static_cast<int64_t>(kPiece), chunks - first));
    for (int i = in; i < n; i += team * kCopyUnroll) {
      uint4 v[kCopyUnroll];
#pragma unroll
      for (int u = 0; u < kCopyUnroll; ++u)
        if (i + u * team < n) v[u] = __ldcs(s + i + u * team);
#pragma unroll
      for (int u = 0; u < kCopyUnroll; ++u)
        if (i + u * team < n) __stcs(d + i + u * team, v[u]);
    }
  }
}

// Each entry of the listed rows is taken out once, whatever the list repeats.
__global__ void __launch_bounds__(256) free_kernel(const PoolArgs a) {
  pdl_wait();
  pdl_launch();
  const int r = a.src[blockIdx.x];
  if (r < 0 || r >= a.R) {
    if (threadIdx.x == 0 && blockIdx.y == 0) report(a, HISPARSE_ERR_RANGE);
    return;
  }
  int32_t *row = a.tables + static_cast<int64_t>(r) * a.blocks;
  for (int b = blockIdx.y * 256 + threadIdx.x; b < a.blocks; b += gridDim.y * 256) {
    if (row[b] == -1) continue;
    const int p = atomicExch(row + b, -1);
    if (p == -1) continue;
    if (p < 0 || p >= a.pages) {
      report(a, HISPARSE_ERR_RANGE);
    } else {
      atomicSub(a.refs + p, 1);
    }
  }
}

int pool_args(const hisparse_page_pool *p, PoolArgs &a) {
  if (!p || p->num_pages < 1 || p->num_requests < 1 || p->max_blocks < 1 || p->page_tokens < 1 ||
      p->layers < 1 || p->row_bytes < 16 || p->row_bytes % 16)
    return HISPARSE_EINVAL;
  if (!p->store || !p->d_tables || !p->d_refs || !p->d_work || !aligned16(p->store) ||
      !aligned16(p->d_refs) || p->layer_stride % 16 || p->page_stride % 16 ||
      p->page_stride < p->row_bytes * p->page_tokens || p->layer_stride < 0)
    return HISPARSE_EINVAL;
  // (loops over a table row step by up to 2048 blocks in 32 bits)
  if (p->num_pages > (1 << 30) || p->num_requests > 8192 || p->max_blocks > (1 << 30)) return HISPARSE_EBOUND;
  a = {};
  a.pages = p->num_pages; a.R = p->num_requests; a.blocks = p->max_blocks;
  a.page_tokens = p->page_tokens; a.layers = p->layers;
  a.row_bytes = p->row_bytes; a.layer_stride = p->layer_stride; a.page_stride = p->page_stride;
  a.store = static_cast<char *>(p->store);
  a.tables = p->d_tables; a.refs = p->d_refs; a.work = p->d_work; a.status = p->d_status;
  a.span = std::max(a.pages, a.R);
  return HISPARSE_OK;
}

}  // namespace

extern "C" {

int64_t hisparse_pages_work_ints(int32_t num_pages, int32_t num_requests) {
  if (num_pages < 1 || num_requests < 1 || num_pages > (1 << 30) || num_requests > 8192) return -1;
  return kWorkHead + 3 * static_cast<int64_t>(std::max(num_pages, num_requests));
}

int hisparse_pages_grow(const hisparse_page_pool *p, const int32_t *d_reqs,
                        const int32_t *d_blocks, int32_t n, void *stream) {
  PoolArgs a;
  if (const int rc = pool_args(p, a)) return rc;
  if (n < 0 || (n > 0 && (!d_reqs || !d_blocks))) return HISPARSE_EINVAL;
  if (n > a.R) return HISPARSE_EBOUND;
  if (n == 0) return HISPARSE_OK;
  a.n = n; a.src = d_reqs; a.want = d_blocks;
  return launch_pdl(plan_kernel<false>, dim3(kPlanCtas), dim3(kPlanThreads), 0, stream, kPlanCtas, a);
}

int hisparse_pages_fork(const hisparse_page_pool *p, const int32_t *d_src, const int32_t *d_dst,
                        const int32_t *d_tokens, int32_t n, void *stream) {
  PoolArgs a;
  if (const int rc = pool_args(p, a)) return rc;
  if (n < 0 || (n > 0 && (!d_src || !d_dst || !d_tokens))) return HISPARSE_EINVAL;
  if (n > a.R) return HISPARSE_EBOUND;
  if (n == 0) return HISPARSE_OK;
  a.n = n; a.src = d_src; a.dst = d_dst; a.want = d_tokens;
  if (const int rc = launch_pdl(plan_kernel<true>, dim3(kPlanCtas), dim3(kPlanThreads), 0, stream,
                                kPlanCtas, a))
    return rc;
  const int64_t page = static_cast<int64_t>(a.page_tokens) * a.row_bytes / 16;
  const int64_t threads = static_cast<int64_t>(n) * a.layers * ((page + kPiece - 1) / kPiece) * (page <= 64 ? 32 : 256);
  const int64_t ctas = std::min<int64_t>(kCopyCtas, (threads + kCopyThreads - 1) / kCopyThreads);
  return launch_pdl(page_copy_kernel<true>, dim3(static_cast<unsigned>(ctas)), dim3(kCopyThreads), 0, stream, 1, a);
}

int hisparse_pages_free(const hisparse_page_pool *p, const int32_t *d_reqs, int32_t n,
                        void *stream) {
  PoolArgs a;
  if (const int rc = pool_args(p, a)) return rc;
  if (n < 0 || (n > 0 && !d_reqs)) return HISPARSE_EINVAL;
  if (n == 0) return HISPARSE_OK;
  a.n = n; a.src = d_reqs;
  const int parts = std::min(8, (a.blocks + 255) / 256);
  return launch_pdl(free_kernel, dim3(n, parts), dim3(256), 0, stream, 1, a);
}

int hisparse_pages_compact(const hisparse_page_pool *p, void *stream) {
  PoolArgs a;
  if (const int rc = pool_args(p, a)) return rc;
  if (const int rc = launch_pdl(compact_plan_kernel, dim3(kPlanCtas), dim3(kPlanThreads), 0, stream,
                                kPlanCtas, a))
    return rc;
  return launch_pdl(page_copy_kernel<false>, dim3(kCopyCtas), dim3(kCopyThreads), 0, stream, 1, a);
}

}  // extern "C"
