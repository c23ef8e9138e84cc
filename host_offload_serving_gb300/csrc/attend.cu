// attend.cu -- sparse attention over 8-bit records (hisparse_attend of include/hisparse.h).
//
// One thread-block cluster works on one query row, KV head and group of N query
// heads; its CTAs split the row's tokens and join through distributed shared memory.
// A CTA turns the problem so that tokens are the long side of both products:
//
//   S^T [tokens x N]  = K  [tokens x k_dim] . Q^T        (K-major K rows, as they are stored)
//   O^T [v_dim x N]  += V^T [v_dim x tokens] . P^T       (the same rows, read transposed)
//
// Both run on the tensor cores (tcgen05.mma kind::f8f6f4, M = 128) with the
// records' e4m3 bytes as they are: nothing is dequantised, and a latent record's K tile
// serves as V without a second copy.  What is not 8 bits becomes a sum of 8-bit terms:
// q, scaled by a power of two for each head to below 2^8, is t1 + t2 (+ t3 for f16), each the e4m3
// rounding of what the ones before leave.  That is exact down to 2^-9 (f16: 2^-6) of the head's largest
// value; e4m3 ends at 2^-9, so smaller ones are within 2^-17 of the largest.
// The scale of K enters the scores in 32 bits; the scale of V enters the probabilities
// (p_j sV_j is what multiplies the raw bytes of V), through the exponent, so the
// running maximum is over s_j + log2(sV_j) and no product leaves the range.
// The p_j sV_j are three e5m2 terms, four for f16: each leaves 2^-4 of what it rounds, so together
// 2^-11 (2^-15), as far down as the last reaches, 2^-17 where the largest is 2^15.  Their range is what
// counts where one token has nearly all of the weight and a small V: the output is then made
// of the others, which lie 2^-20 below.  (e4m3 and e5m2, with the largest at 2^2 so that it could grow,
// lost them: 3 % from 64 bits beside a token of weight 0.9, 40 % at 0.997; now 0.0017, which is the
// rounding to bf16, up to 0.9999.)  All sums are in 32 bits.
//
// Warps: four softmax warps (a lane a token, TMEM lane = token) for each 32 columns; six (four for
// 64 columns) that gather (16-byte cp.async into the 128-byte-swizzled tiles that the tensor cores
// read, as many tiles ahead as there are stages); four (two) that turn slots and positions into
// addresses and scales, further ahead; and two that issue the products.  S is double buffered in
// TMEM, so the scores of tile i+1 are computed while the softmax of tile i runs.  A column's offset
// moves (with its sums and O) only where a probability would exceed 2^15.75, the range of e5m2.  It is set
// so that 2^12 of that are left above the largest of the warp that lies lowest, and the largest is 2^15 at most
// and 2^8 at least: in rows of normal scores the largest of later tiles seldom passes that, a dominant token
// gets the whole range below it, and several of them, one in each warp, what lies below 2^8.  16 requests of
// 2048 tokens take 22.1 us; 21.6 without the least, 22.5 with 2^10 for it, 21.4 where nothing ever moves.
//
// What bounds it, and what it measured.  64 requests of 2048 tokens, 128 heads on one latent head of
// 576 + 512 (two groups of 64 heads read each row, one from L2): 76 us, where 75 MB of rows would allow 14
// and the products (two terms with K, three with V) 26.  A CTA turns a tile of 96 tokens in 5100 cycles: its shared
// memory has room for two tiles beside the 80 KB of q, so a tile's copy (2000 cycles at the
// 27 B/cycle that 16-byte copies reach on an SM), scores (1150), softmax (2000) and values (1730) overlap
// only with one other tile's.  (The third product with V is 6 us of it.)  With few rows the fixed parts count: 8
// requests and 64 heads take 16 us, 6 of them before the first scores (launch, look-up, first rows, cold
// instructions) and 2 joining clusters; one request of 64 tokens 8.2 us.  16 requests of 8 heads of 128, 32
// query heads, 2048 tokens (67 MB): 22.1 us, 3.1 TB/s; there a tile's softmax is a chain of waits of one
// warp a scheduler, 1300 cycles.
// Not kept: rows gathered by the copy engine, four an instruction (100 us where the copies by threads
// took 100 too); rows prefetched into L2 by the look-up warps (10,000 cycles a tile there); a barrier
// for each 128 columns of a tile (116 us against 86); two softmax groups on alternate tiles (20 warps of
// 96 registers spill, 27 us for the last case; 16 warps leave two to look rows up, 26 us); values before
// scores, or scores before values, by a flag between the two warps (78 and 81 us).
#include <algorithm>
#include <atomic>
#include <climits>

#include "common.cuh"
#include "waits.cuh"

namespace {

constexpr int kMaxStages = 6;
constexpr int kMaxCluster = 16;
constexpr float kNone = -1e30f; // a CTA's offset where it had no token
constexpr int32_t kMasked = 0x7fffffff;  // in place of K's scale: a token that does not count
// log2 of a column's largest probability when its offset is set, at the most and at the least; of what it
// may grow to before the offset moves again (the largest e5m2 is 57344 = 2^15.8); and the room that is left
// above the warp whose tokens lie lowest.
constexpr float kTop = 15.f, kLeast = 8.f, kSlack = 15.75f, kRoom = 12.f;
// Sums of probabilities are kept 2^-kFold of what they are: a token whose scale of V is 2^-100 adds
// 2^115 at the most, and a few thousand of them would leave the range.
constexpr float kFold = 16.f;

struct AttendArgs {
  int32_t rows, entries, heads, kv_heads, k_dim, v_dim, latent, B;
  int32_t columns, group, hgroups;
  FastDiv rec_tokens, sel_block, S;
  float scale_log2;
  const void *q;
  int64_t q_row, q_head;
  void *out;
  int64_t out_row, out_head;
  float *lse;
  const int32_t *sel, *slots;
  const char *hot;
  int64_t hot_req;
  uint32_t hot_row, res_row, res_rows, row_bytes;  // row_bytes: a token's part of a record
  const char *resident;
  const float *scales;
  int64_t scales_req;
  uint32_t scale_blocks;
  const int32_t *seq_lens, *num_reqs;
  uint32_t *status;
  // the launch's plan
  int32_t cluster, per_cta, tile, stages, k_chunks, v_chunks, v_tiles, tmem_cols;
  int32_t sums;  // of a column: one, or one for each term of the probabilities
  FastDiv quads;  // v_dim / 4
  uint32_t stage_bytes, off_q, off_p, off_meta, off_rows;
};

// ---- PTX ---------------------------------------------------------------------
__device__ __forceinline__ void fence_async() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
__device__ __forceinline__ void tc_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(r)::"memory");
  return r;
}
// This lane's mbarrier arrival once its products so far are done.
__device__ __forceinline__ void tc_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
               : "memory");
}
// Shared-memory descriptor of a 128-byte-swizzled operand whose groups of 8 rows are 1024
// bytes apart (either major-ness: the other offset is not used).  Its lower word; the
// upper one is the same for all.
constexpr uint32_t kDescHi = 64u | 1u << 14 | 2u << 29;
// The same of one with 64-byte swizzle, whose groups of 8 rows are 512 bytes apart.
constexpr uint32_t kDescHi64 = 32u | 1u << 14 | 4u << 29;
__device__ __forceinline__ uint32_t smem_desc(uint32_t addr) { return addr >> 4 | 1u << 16; }
// Instruction descriptor: f32 accumulator, A e4m3, B e4m3 or e5m2, M = 128.
__device__ __forceinline__ uint32_t mma_desc(int n, bool b_e5m2, bool transposed) {
  return (1u << 4) | (b_e5m2 ? 1u << 10 : 0u) | (transposed ? 3u << 15 : 0u) |
         (static_cast<uint32_t>(n) >> 3 << 17) | (128u >> 4 << 24);
}
// Products are issued by one lane, in unrolled runs of constant offsets: the operands go through
// uniform registers, and a run of any length keeps the tensor cores fed (39 cycles an
// instruction for 16 columns, 64 for 128), where a loop around one took 100.
template <uint32_t kHiB = kDescHi>
__device__ __forceinline__ void mma_f8(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 da, db;\n"
      " setp.ne.b32 p, %4, 0;\n"
      " mov.b64 da, {%1, %5};\n mov.b64 db, {%2, %6};\n"
      " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], da, db, %3, p;\n}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "r"(kDescHi), "r"(kHiB)
      : "memory");
}
__device__ __forceinline__ void tc_ld16(uint32_t addr, uint32_t *r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(addr));
}
__device__ __forceinline__ void tc_st16(uint32_t addr, const uint32_t *r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::"r"(r[0]), "r"(r[1]),
      "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(addr)
      : "memory");
}
// Waits for the loads before it; the values pass through it, so nothing that uses them moves
// ahead of the wait.
__device__ __forceinline__ void tc_wait_ld16(uint32_t *r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]),
                 "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]),
                 "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}
__device__ __forceinline__ void tc_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, uint64_t src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// What a masked token's row reads: zeros, as its probability is 0 and 0 * NaN is not.
__device__ uint4 g_zeros[640 / 16];
// Arrives once this thread's copies so far are complete.  Their bytes are then seen by whoever
// waited for the barrier, and by that thread's tensor-core reads after its proxy fence.
__device__ __forceinline__ void cp_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ float warp_max(float x) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float lg2(float x) {
  float r;
  asm("lg2.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// OR over a group of four softmax warps, and their barrier (1 or 2: constants, as a CTA
// takes all 16 hardware barriers for one that is not, and two such CTAs do not fit an SM).
template <int kId>
__device__ __forceinline__ bool any_of_128(bool x) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %1, 0;\n"
      " barrier.cta.red.or.pred q, %2, 128, p;\n selp.u32 %0, 1, 0, q;\n}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(x)), "n"(kId)
      : "memory");
  return r != 0;
}
template <int kGroups>
__device__ __forceinline__ bool soft_any(int group, bool x) {
  if (kGroups == 1 || group == 0) return any_of_128<1>(x);
  return any_of_128<2>(x);
}
template <int kGroups>
__device__ __forceinline__ void soft_sync(int group) {
  if (kGroups == 1 || group == 0) {
    asm volatile("barrier.cta.sync 1, 128;" ::: "memory");
  } else {
    asm volatile("barrier.cta.sync 2, 128;" ::: "memory");
  }
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}
__device__ __forceinline__ uint32_t peer(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ float4 ld_peer4(uint32_t addr) {
  float4 r;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(r.x), "=f"(r.y), "=f"(r.z), "=f"(r.w)
               : "r"(addr)
               : "memory");
  return r;
}
__device__ __forceinline__ float4 ld_shared4(uint32_t addr) {
  float4 r;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(r.x), "=f"(r.y), "=f"(r.z), "=f"(r.w)
               : "r"(addr)
               : "memory");
  return r;
}
__device__ __forceinline__ void st_shared4(uint32_t addr, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(x), "r"(y), "r"(z), "r"(w)
               : "memory");
}

// Two values to e4m3 with rounding to nearest; *x and *y keep what the rounding leaves.
__device__ __forceinline__ uint32_t take_term(float &x, float &y) {
  uint16_t p;
  uint32_t h;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(p) : "f"(y), "f"(x));
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(p));
  const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
  x -= f.x;
  y -= f.y;
  return p;
}
// Two values to e5m2, the upper byte of f16, with rounding to nearest; they keep what the rounding leaves,
// exactly.
__device__ __forceinline__ uint32_t take_e5m2(float &x, float &y) {
  uint16_t p;
  asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(p) : "f"(y), "f"(x));
  const uint32_t back = __byte_perm(p, 0, 0x1404);
  const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&back));
  x -= f.x;
  y -= f.y;
  return p;
}
__device__ __forceinline__ uint32_t take_e5m2(__half2 &h) {
  uint16_t p;
  asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(p) : "r"(*reinterpret_cast<const uint32_t *>(&h)));
  const uint32_t back = __byte_perm(p, 0, 0x1404);
  h = __hsub2(h, *reinterpret_cast<const __half2 *>(&back));
  return p;
}

// The largest magnitude of 24 values (NaN left out).
template <class T>
__device__ __forceinline__ float abs_max(const uint4 (&v)[3]);
template <>
__device__ __forceinline__ float abs_max<__nv_bfloat16>(const uint4 (&v)[3]) {
  __nv_bfloat162 m = __float2bfloat162_rn(0.f);
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    const __nv_bfloat162 *e = reinterpret_cast<const __nv_bfloat162 *>(&v[i]);
#pragma unroll
    for (int j = 0; j < 4; ++j) m = __hmax2(m, __habs2(e[j]));
  }
  return fmaxf(__low2float(m), __high2float(m));
}
template <>
__device__ __forceinline__ float abs_max<__half>(const uint4 (&v)[3]) {
  __half2 m = __float2half2_rn(0.f);
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    const __half2 *e = reinterpret_cast<const __half2 *>(&v[i]);
#pragma unroll
    for (int j = 0; j < 4; ++j) m = __hmax2(m, __habs2(e[j]));
  }
  return fmaxf(__low2float(m), __high2float(m));
}
// 8 values times `up` as e4m3 terms; word 0 holds the terms of the first four.
// (Out of line: unrolled into its callers it would be a sixth of the kernel, which does not fit the
// instruction cache as it is.)
template <int kTerms>
struct Split {
  uint32_t w0[kTerms], w1[kTerms];
};
template <class T, int kTerms>
__device__ __noinline__ Split<kTerms> split8(uint4 v, float up) {
  const T *e = reinterpret_cast<const T *>(&v);
  Split<kTerms> s;
  uint32_t (&w0)[kTerms] = s.w0, (&w1)[kTerms] = s.w1;
  if constexpr (kTerms == 2) {
    // |x| < 256: in f16, 11 significant bits against the 8 of the values, and as far down as
    // the second term reaches.
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float x = to_f32<T>(e[2 * j]) * up, y = to_f32<T>(e[2 * j + 1]) * up;
      uint32_t h, back;
      uint16_t p, r;
      asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(y), "f"(x));
      asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(p) : "r"(h));
      asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(back) : "h"(p));
      const __half2 left = __hsub2(*reinterpret_cast<__half2 *>(&h), *reinterpret_cast<__half2 *>(&back));
      asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(*reinterpret_cast<const uint32_t *>(&left)));
      hi[j] = p;
      lo[j] = r;
    }
    w0[0] = hi[0] | hi[1] << 16;
    w1[0] = hi[2] | hi[3] << 16;
    w0[1] = lo[0] | lo[1] << 16;
    w1[1] = lo[2] | lo[3] << 16;
  } else {
    float x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = to_f32<T>(e[j]) * up;
#pragma unroll
    for (int t = 0; t < kTerms; ++t) {
      w0[t] = take_term(x[0], x[1]);
      w0[t] |= take_term(x[2], x[3]) << 16;
      w1[t] = take_term(x[4], x[5]);
      w1[t] |= take_term(x[6], x[7]) << 16;
    }
  }
  return s;
}

// 2^kLw columns of 16-byte chunks of a warp's share of the rows: lane t * 2^kLw + c copies
// chunk c of row t of a turn.  The rows' addresses are a table in shared memory (8 bytes a
// row); `dst` is the lane's place in row 0 of a 128-byte-swizzled tile, whose 16-byte
// chunk is XORed with the row's lowest 3 bits.  A warp takes every kWarps-th group of 8 rows.
template <int kLw, int kWarps>
__device__ __forceinline__ void gather_columns(uint32_t table, uint32_t off, uint32_t dst, int groups, int warp,
                                               int lane) {
  constexpr int kDt = 32 >> kLw;                  // rows in one turn of the warp
  constexpr int kTurns = kDt < 8 ? 8 / kDt : 1;   // turns in a group of 8 rows
  constexpr int kAtOnce = kDt <= 8 ? 1 : kDt / 8; // groups in one turn
  const int tl = lane >> kLw;
  const int sub = kAtOnce > 1 ? tl >> 3 : 0;      // the group of a turn that the lane is in
  const int row = kAtOnce > 1 ? tl & 7 : tl;
  constexpr int kBatch = kTurns >= 4 ? 2 : 3;  // turns of groups whose addresses are read together
#pragma unroll 1
  for (int g = warp; g < groups; g += kBatch * kWarps * kAtOnce) {
    uint64_t p[kBatch][kTurns];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int mine = g + (b * kAtOnce + sub) * kWarps;
      if (mine < groups) {
#pragma unroll
        for (int u = 0; u < kTurns; ++u)
          asm volatile("ld.shared.b64 %0, [%1];" : "=l"(p[b][u]) : "r"(table + (mine * 8 + row + u * kDt) * 8));
      }
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int mine = g + (b * kAtOnce + sub) * kWarps;
      const uint32_t to = (dst ^ ((row & 7) << 4)) + (mine * 8 + row) * 128;
      if (mine < groups) {
#pragma unroll
        for (int u = 0; u < kTurns; ++u) cp_async16((to ^ (u * kDt << 4)) + u * kDt * 128, p[b][u] + off);
      }
    }
  }
}

// A tile's columns come, are multiplied and go in two halves: the chunks of K and of V, or those
// of a latent record in two of about as many 16-byte columns (16 and 20 of 36: 66 us for the largest case
// with two terms of the probabilities, 24 and 12 68).  Chunks [c0, c1) of K or V; the values read [v0, v1)
// of them.
struct Half {
  int c0, c1, v0, v1;
  bool is_v;
};
__device__ __forceinline__ Half half_of(const AttendArgs &a, int u) {
  if (!a.latent) return {0, u ? a.v_chunks : a.k_chunks, 0, u ? a.v_chunks : 0, u == 1};
  const int mid = max(1, ((a.k_dim >> 4) + 8) >> 4), c0 = u ? mid : 0, c1 = u ? a.k_chunks : mid;
  return {c0, c1, min(c0, a.v_tiles), min(c1, a.v_tiles), false};
}

// ---- tokens ------------------------------------------------------------------
// A load, or a constant without one; nothing waits here for the load.
__device__ __forceinline__ int32_t ld_if(const int32_t *p, bool take, int32_t other) {
  int32_t r;
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %2, 0;\n mov.b32 %0, %3;\n @p ld.global.b32 %0, [%1];\n}"
      : "=&r"(r)
      : "l"(p), "r"(static_cast<int>(take)), "r"(other));
  return r;
}
struct Raw {
  int32_t slot, sel, entry;
};
struct Token {
  uint64_t row;  // address; 0: nothing to read
  const float *scales;
};

// e4m3 terms of q, and e5m2 terms of a probability: each of these leaves 2^-4 of what it rounds, so that
// three give 2^-11 and four as much as the f16 that they are taken from.
template <class T>
struct Terms;
template <>
struct Terms<__nv_bfloat16> {
  static constexpr int n = 2, p = 3;
};
template <>
struct Terms<__half> {
  static constexpr int n = 3, p = 4;
};

// Sums of l[0 .. N) over the warp's lanes: at each step a lane hands over half of its
// columns and keeps the others.  Column c ends at l[c % per] of lanes whose upper bits
// spell c / per, per = max(1, N / 32).
template <int N, int O, int kHalf>
__device__ __forceinline__ void column_sums(float (&l)[N], int lane) {
  if constexpr (kHalf >= 1) {
    const bool up = lane & O;
#pragma unroll
    for (int c = 0; c < kHalf; ++c) {
      const float send = up ? l[c] : l[c + kHalf], keep = up ? l[c + kHalf] : l[c];
      l[c] = keep + __shfl_xor_sync(0xffffffffu, send, O);
    }
  } else {
    l[0] += __shfl_xor_sync(0xffffffffu, l[0], O);
  }
  if constexpr (O > 1) column_sums<N, O / 2, kHalf / 2>(l, lane);
}

template <int N>
struct Shape {
  static constexpr int groups = N > 32 ? N / 32 : 1;  // of four softmax warps
  static constexpr int cols = N / groups;             // columns of a softmax thread
  static constexpr int soft = 4 * groups;             // softmax warps
  static constexpr int gather = N > 32 ? 4 : 6;       // warps that copy rows
  static constexpr int mma = soft + gather;           // two warps that issue products: scores, values
  static constexpr int look = mma + 2;                // warps that look rows up
  static constexpr int looks = N > 32 ? 2 : 4;
  static constexpr int tables = N > 32 ? 3 : 8;      // tiles that are looked up ahead
  static constexpr int threads = 32 * (look + looks);
};

template <class T, int N>
__global__ void __launch_bounds__(Shape<N>::threads, 1)
    attend_kernel(const AttendArgs a) {
  constexpr int kTerms = Terms<T>::n, kP = Terms<T>::p;
  // Terms of the probabilities that a token's row of 128 bytes takes; what is left (the third of 64 heads)
  // has a tile of rows of 64 bytes behind it.
  constexpr int kP0 = kP * N > 128 ? 128 / N : kP;
  static_assert(kP * N <= 128 || (kP - kP0) * N == 64);
  // Where the tensor memory has room, all terms are one product with sums of their own, which are added
  // at the end: 44 cycles for three of 16 columns, where one after another took 120.
  constexpr bool kMerge = kP0 == kP;
  constexpr int NC = Shape<N>::cols, kSoft = Shape<N>::soft, kGather = Shape<N>::gather, kTables = Shape<N>::tables;
  constexpr int kThreads = Shape<N>::threads;
  constexpr int kQ = kTerms * N;  // rows of Q: the terms of a head are N rows apart
  extern __shared__ char smem_raw[];
  __shared__ uint64_t s_bars[4 * kMaxStages + 3 * kTables + 9];
  __shared__ uint32_t s_tmem;
  __shared__ int s_fail;
  __shared__ float s_l[N], s_d[N], s_wmax[4][N], s_w[N];
  __shared__ float2 s_pair[N];
  __shared__ __align__(16) float s_qf[N], s_m[N], s_f[N];
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t bars = smem_u32(s_bars);
  const uint32_t b_full = bars, b_empty = bars + 16 * kMaxStages;  // [stage][half]
  const uint32_t b_s = bars + 32 * kMaxStages;
  const uint32_t b_p = b_s + 16, b_pv = b_s + 24, b_q = b_s + 32;
  const uint32_t b_read = b_s + 40;  // a score buffer has been read
  const uint32_t b_tab = b_s + 56, b_meta = b_tab + 8 * kTables,
                 b_used = b_meta + 8 * kTables;  // addresses and scales: written; done with
  const uint32_t b_done = b_used + 8 * kTables;  // after a wait that ran out: the products issued so far
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const uint32_t rank = a.cluster > 1 ? blockIdx.x % a.cluster : 0;
  const uint32_t unit = blockIdx.x / a.cluster;
  const uint32_t hg = unit % a.hgroups, kvh = unit / a.hgroups % a.kv_heads;
  const int64_t qrow = unit / a.hgroups / a.kv_heads;
  const int req = static_cast<int>(qrow / a.rows);

  if (tid == 0) {
    bar_init(b_s, 1);
    bar_init(b_s + 8, 1);
    bar_init(b_read, 32 * kSoft);
    bar_init(b_read + 8, 32 * kSoft);
    bar_init(b_p, 32 * kSoft);
    bar_init(b_pv, 1);
    bar_init(b_q, 32 * (kSoft + 2));
    for (int t = 0; t < kTables; ++t) {
      bar_init(b_tab + 8 * t, 32 * Shape<N>::looks);
      bar_init(b_meta + 8 * t, 32 * Shape<N>::looks);
      bar_init(b_used + 8 * t, 1);
    }
    bar_init(b_done, 1);
    bar_init(b_done + 8, 1);
    s_fail = 0;
  }
  for (int i = tid; i < 2 * a.stages; i += kThreads) {
    bar_init(b_full + 8 * i, 32 * kGather / 2);
    bar_init(b_empty + 8 * i, 1);
  }
  for (int c = tid; c < N; c += kThreads) s_m[c] = 0.f;
  // The last 16 of 32 K columns that a product reads beyond k_dim: zero in every
  // stage (the copies never write them) and in Q.
  if (a.k_dim & 16) {
    const int c = a.k_dim >> 7, j = (a.k_dim & 127) >> 4;
    for (int i = tid; i < a.stages * a.tile; i += kThreads) {
      const int s = i / a.tile, t = i - s * a.tile;
      st_shared4(base + s * a.stage_bytes + (c * a.tile + t) * 128 + ((j ^ (t & 7)) << 4), 0, 0, 0, 0);
    }
    for (int i = tid; i < kQ; i += kThreads) {
      st_shared4(base + a.off_q + (c * kQ + i) * 128 + ((j ^ (i & 7)) << 4), 0, 0, 0, 0);
    }
    fence_async();
  }
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  pdl_wait();
  if (a.num_reqs && req >= *a.num_reqs) return;  // the whole cluster
  if (a.cluster > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  if (warp == Shape<N>::mma) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)),
                 "r"(a.tmem_cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_before();
  __syncthreads();
  tc_after();
  pdl_launch();
  const uint32_t tmem = s_tmem;
  const uint32_t t_o = tmem + 2 * kQ;

  const int ntok = a.entries * static_cast<int>(a.rec_tokens.d);
  const int t0 = min(ntok, static_cast<int>(rank) * a.per_cta), t1 = min(ntok, t0 + a.per_cta);
  const int tiles = (t1 - t0 + a.tile - 1) / a.tile;
  const int64_t entry0 = qrow * a.entries;
  volatile int *fail = &s_fail;

  // Query heads of this group into e4m3 terms, by the softmax and product warps while the first
  // rows come.
  auto make_q = [&](int w) {
    const int vecs = a.k_dim >> 3;
    const T *q0 = static_cast<const T *>(a.q) + qrow * a.q_row;
    constexpr int kWarps = kSoft + 2, kBatch = (N + kWarps - 1) / kWarps;
    {
      const int n0 = w;
      uint4 v[kBatch][3];  // all of a warp's heads in flight together
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int n = n0 + kWarps * b, h = static_cast<int>(hg) * N + n;
        const uint4 *src = reinterpret_cast<const uint4 *>(q0 + static_cast<int64_t>(kvh * a.group + h) * a.q_head);
#pragma unroll
        for (int i = 0; i < 3; ++i)
          v[b][i] = n < N && h < a.group && lane + 32 * i < vecs ? src[lane + 32 * i] : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int n = n0 + kWarps * b;
        if (n >= N) break;
        const float m = warp_max(abs_max<T>(v[b]));
        // q * 2^sh has its largest in [128, 256)
        const int ex = static_cast<int>(__float_as_uint(m) >> 23) - 127;
        const int sh = m > 0.f ? min(7 - ex, 120) : 0;
        const float up = __uint_as_float(static_cast<uint32_t>(127 + sh) << 23);
        if (lane == 0)  // infinities do not fit a term: they make the scores NaN
          s_qf[n] = m < INFINITY ? a.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 - sh) << 23)
                                 : NAN;
#pragma unroll
        for (int i = 0; i < 3; ++i) {
          if (32 * i >= vecs) break;
          if (lane + 32 * i >= vecs) continue;
          const int d = (lane + 32 * i) * 8;
          const uint32_t at = base + a.off_q + ((d >> 7) * kQ + n) * 128 + (((d & 127) >> 4 ^ (n & 7)) << 4) + (d & 15);
          const Split<kTerms> w = split8<T, kTerms>(v[b][i], up);
#pragma unroll
          for (int t = 0; t < kTerms; ++t)
            asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(at + t * N * 128), "r"(w.w0[t]), "r"(w.w1[t])
                         : "memory");
        }
      }
    }
    fence_async();
    bar_arrive(b_q);
  };

  if (warp < kSoft || (warp >= Shape<N>::mma && warp < Shape<N>::look)) make_q(warp < kSoft ? warp : warp - kGather);

  if (warp < kSoft) {
    // ---- softmax ---------------------------------------------------------------
    bar_wait(b_q, 0, fail);  // the factors of all heads
    const int grp = warp >> 2, wl = warp & 3, c0 = grp * NC, gt = tid & 127;
    float l[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) l[c] = 0.f;
    const uint32_t lanes = static_cast<uint32_t>(wl * 32) << 16;
    const int tk = wl * 32 + lane;
    const uint32_t p_row = base + a.off_p + tk * 128, p_row2 = base + a.off_p + a.tile * 128 + tk * 64;
    bool open = true;   // some column has had no token that counts, and no offset
    bool set = false;   // whether column c0 + gt has one
    constexpr bool kHeld = NC == 16;  // factors and offsets fit in registers
    float qf[kHeld ? NC : 1], off[kHeld ? NC : 1];
    if (kHeld) {
#pragma unroll
      for (int c = 0; c < NC; ++c) qf[kHeld ? c : 0] = s_qf[c0 + c], off[kHeld ? c : 0] = 0.f;
    }
    // This lane's token of a tile: its scale of K, and of V as log2 and inverse.
    // A scale of V that is no number leaves the softmax as it is and spoils the token's probabilities.
    float ks, lv, iv;
    bool use, spoilt;
    auto scales_of = [&](int i) {
      bar_wait(b_meta + 8 * (i % kTables), (i / kTables) & 1, fail);
      ks = 0.f, lv = 0.f, iv = 1.f;
      use = spoilt = false;
      if (tk < min(a.tile, t1 - t0 - i * a.tile)) {
        float2 meta;
        asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];"
                     : "=f"(meta.x), "=f"(meta.y)
                     : "r"(base + a.off_meta + (i % kTables * a.tile + tk) * 8)
                     : "memory");
        use = __float_as_int(meta.x) != kMasked;
        if (use) {
          ks = meta.x;
          spoilt = !(meta.y < INFINITY);
          // (approximate to 2^-21, and the inverse of the very same)
          if (!spoilt) lv = lg2(fmaxf(meta.y, 0x1p-100f));
          iv = ex2(-kFold - lv);
        }
      }
    };
    if (tiles > 0) scales_of(0);
    for (int i = 0; i < tiles; ++i) {
      const int cn = min(a.tile, t1 - t0 - i * a.tile);
      bar_wait(b_s + 8 * (i & 1), (i >> 1) & 1, fail);
      __syncwarp();
      tc_after();
      float x[NC];
      {
        const uint32_t at = tmem + lanes + (i & 1) * kQ + c0;
#pragma unroll
        for (int c = 0; c < NC; c += 16) {
          float y[kTerms][16];
#pragma unroll
          for (int t = 0; t < kTerms; ++t) tc_ld16(at + t * N + c, reinterpret_cast<uint32_t *>(y[t]));
#pragma unroll
          for (int t = 0; t < kTerms; ++t) tc_wait_ld16(reinterpret_cast<uint32_t *>(y[t]));
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            x[c + e] = y[0][e] + y[1][e];
            if (kTerms == 3) x[c + e] += y[kTerms - 1][e];
          }
        }
      }
      tc_before();
      bar_arrive(b_read + 8 * (i & 1));
      // scores in powers of two, the V scale in them, above their column's offset
      float most = -INFINITY;
#pragma unroll
      for (int c = 0; c < NC; c += 4) {
        float4 f, m;
        if (kHeld) {
          f = make_float4(qf[kHeld ? c : 0], qf[kHeld ? c + 1 : 0], qf[kHeld ? c + 2 : 0], qf[kHeld ? c + 3 : 0]);
          m = make_float4(off[kHeld ? c : 0], off[kHeld ? c + 1 : 0], off[kHeld ? c + 2 : 0], off[kHeld ? c + 3 : 0]);
        } else {
          f = ld_shared4(smem_u32(s_qf + c0 + c)), m = ld_shared4(smem_u32(s_m + c0 + c));
        }
        const float g[4] = {f.x, f.y, f.z, f.w}, o[4] = {m.x, m.y, m.z, m.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[c + e] = use ? fmaf(x[c + e] * ks, g[e], lv - o[e]) : -INFINITY;
          most = fmaxf(most, x[c + e]);
        }
      }
      const bool moved = soft_any<Shape<N>::groups>(grp, most > kSlack || (open && most > -INFINITY));
      auto previous = [&] {  // O and the probabilities' buffer are free
        if (i > 0) {
          bar_wait(b_pv, (i - 1) & 1, fail);
          __syncwarp();
          tc_after();
        }
      };
      if (moved) {  // some columns outgrew their offset: new offsets, and their sums follow
        float mine = -INFINITY;  // lane c keeps the maximum of column c
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          const float m = warp_max(x[c]);
          if (lane == c) mine = m;
        }
        if (lane < NC) s_wmax[wl][c0 + lane] = mine;
        soft_sync<Shape<N>::groups>(grp);
        if (gt < NC) {
          const int c = c0 + gt;
          // The largest of the column goes to 2^kTop, or as far below (to 2^kLeast) as leaves kRoom above the
          // largest of the warp that lies lowest: a token far above the others leaves them their bits, and
          // is not outgrown; one among others leaves room for those that come.
          float m = -INFINITY, low = INFINITY;
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const float x = s_wmax[w][c];
            m = fmaxf(m, x);
            if (x > -INFINITY) low = fminf(low, x);
          }
          const float top = tiles == 1 ? kTop : fminf(kTop, fmaxf(kLeast, kSlack - kRoom + (m - low)));
          const bool fresh = !set && m > -INFINITY;
          const float d = m > kSlack || fresh ? m - top : 0.f;
          s_d[c] = d;
          s_f[c] = fresh ? 1.f : ex2(-d);  // (the sums of one without an offset are 0)
          s_m[c] += d;
          set |= fresh;
        }
        open = soft_any<Shape<N>::groups>(grp, gt < NC && !set);
        previous();
        if (i > 0) {
#pragma unroll 1
          for (int c = 0; c < NC; c += 16) {
            if (!__any_sync(0xffffffffu, s_f[c0 + c + (lane & 15)] != 1.f)) continue;
#pragma unroll 1
            for (int j = 0; j < a.v_tiles * a.sums; ++j) {
              uint32_t o[16];
              const uint32_t at = t_o + lanes + j * N + c0 + c;
              tc_ld16(at, o);
              tc_wait_ld16(o);
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * s_f[c0 + c + e]);
              tc_st16(at, o);
            }
          }
          tc_wait_st();
#pragma unroll
          for (int c = 0; c < NC; ++c) l[c] *= s_f[c0 + c];
        }
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          const float d = s_d[c0 + c];
          x[c] -= d;
          if (kHeld) off[kHeld ? c : 0] += d;
        }
      }
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        x[c] = ex2(x[c]);
        l[c] = fmaf(x[c], iv, l[c]);
        if (spoilt) x[c] = NAN;
      }
      if (i + 1 < tiles) scales_of(i + 1);  // while the products before are still under way
      if (!moved) previous();
      if (tk < ((cn + 31) & ~31)) {
#pragma unroll
        for (int c = 0; c < NC; c += 16) {
          uint32_t w[kP][4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float *y = x + c + 4 * e;
            // (in f16 behind the first term; for bf16, whose terms end above it, from the start)
            if (kP > 3) w[0][e] = take_e5m2(y[0], y[1]) | take_e5m2(y[2], y[3]) << 16;
            __half2 g = __floats2half2_rn(y[0], y[1]), h = __floats2half2_rn(y[2], y[3]);
#pragma unroll
            for (int t = kP > 3 ? 1 : 0; t < kP; ++t) {
              w[t][e] = take_e5m2(g);
              w[t][e] |= take_e5m2(h) << 16;
            }
          }
#pragma unroll
          for (int t = 0; t < kP; ++t) {
            const int at = t * N + c0 + c;
            st_shared4(t < kP0 ? p_row + ((at >> 4 ^ (tk & 7)) << 4) : p_row2 + (((at - kP0 * N) >> 4 ^ (tk >> 1 & 3)) << 4),
                       w[t][0], w[t][1], w[t][2], w[t][3]);
          }
        }
      }
      fence_async();
      tc_before();
      bar_arrive(b_p);
    }
    column_sums<NC, 16, NC / 2>(l, lane);
    soft_sync<Shape<N>::groups>(grp);  // s_wmax is free
    if (NC == 32) {
      s_wmax[wl][c0 + lane] = l[0];
    } else if ((lane & 1) == 0) {
      s_wmax[wl][c0 + (lane >> 1)] = l[0];
    }
    soft_sync<Shape<N>::groups>(grp);
    if (gt < NC) {
      const int c = c0 + gt;
      const float z = (s_wmax[0][c] + s_wmax[1][c]) + (s_wmax[2][c] + s_wmax[3][c]);
      s_l[c] = z;
      if (!set) s_m[c] = kNone;
      s_f[c] = z > 0.f || z != z ? exp2f(-kFold) / z : 0.f;
    }
    if (tiles > 0) {
      bar_wait(b_pv, (tiles - 1) & 1, fail);
      tc_after();
    }
    __syncwarp();
  } else if (warp < Shape<N>::mma) {
    // ---- gather ------------------------------------------------------------------
    // A tile comes in halves, each as soon as its place is free and with its own arrival and its own
    // half of the warps, as a half is mostly latency; a warp takes every kShare-th group of 8 rows.
    constexpr int kShare = kGather / 2;
    const int u = (warp - kSoft) & 1, gw = (warp - kSoft) >> 1;
    const Half half = half_of(a, u);
    const int cols = min(8 * half.c1, (half.is_v ? a.v_dim : a.k_dim) >> 4);
    const uint32_t table = base + a.off_rows + (half.is_v ? kTables * a.tile * 8 : 0);
    uint32_t st = base + (half.is_v ? a.k_chunks * a.tile * 128 : 0);
    int s = 0, turn = 0;  // the tile's stage, and how often the stages went round
    bool good = true;     // every table so far was written
    for (int i = 0; i < tiles; ++i) {
      const int groups = (min(a.tile, t1 - t0 - i * a.tile) + 31) >> 5 << 2;
      const uint32_t rows = table + i % kTables * a.tile * 8;
      good = bar_wait(b_tab + 8 * (i % kTables), (i / kTables) & 1, fail) && good;
      if (turn > 0) good = bar_wait(b_empty + 16 * s + 8 * u, (turn - 1) & 1, fail) && good;
      for (int col0 = good ? 8 * half.c0 : cols; col0 < cols;) {
        const int left = cols - col0, lw = left >= 32 ? 5 : 31 - __clz(left);
        const int j = col0 + (lane & ((1 << lw) - 1));
        const uint32_t dst = st + (j >> 3) * a.tile * 128 + ((j & 7) << 4);
        switch (lw) {
          case 5: gather_columns<5, kShare>(rows, 16 * j, dst, groups, gw, lane); break;
          case 4: gather_columns<4, kShare>(rows, 16 * j, dst, groups, gw, lane); break;
          case 3: gather_columns<3, kShare>(rows, 16 * j, dst, groups, gw, lane); break;
          case 2: gather_columns<2, kShare>(rows, 16 * j, dst, groups, gw, lane); break;
          case 1: gather_columns<1, kShare>(rows, 16 * j, dst, groups, gw, lane); break;
          default: gather_columns<0, kShare>(rows, 16 * j, dst, groups, gw, lane); break;
        }
        col0 += 1 << lw;
      }
      cp_arrive(b_full + 16 * s + 8 * u);
      st += a.stage_bytes;
      if (++s == a.stages) {
        s = 0, ++turn;
        st -= a.stages * a.stage_bytes;
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp >= Shape<N>::look) {
    // ---- rows: slot -> address, position -> scales, tiles ahead of their copies --------
    const uint32_t k_at = kvh * a.k_dim, v_at = a.kv_heads * a.k_dim + kvh * a.v_dim;
    const uint32_t seq = a.seq_lens ? max(0, a.seq_lens[req]) : 0x80000000u;
    const float *scales = a.scales + req * a.scales_req + kvh;
    const char *hot = a.hot + req * a.hot_req;
    const int v_col = a.latent ? 0 : a.kv_heads;
    const int32_t *slots = a.slots + entry0, *sels = a.sel + entry0 / a.sel_block.d;
    const uint64_t zeros = reinterpret_cast<uint64_t>(g_zeros);
    const bool plain = a.rec_tokens.d == 1 && a.sel_block.d == 1;  // an entry is a token
    auto raw = [&](int t) {
      Raw r;
      r.entry = plain ? t : static_cast<int>(a.rec_tokens.div(t));
      r.slot = ld_if(slots + r.entry, t < t1, -1);
      r.sel = ld_if(sels + (plain ? t : static_cast<int>(a.sel_block.div(r.entry))), t < t1, -1);
      return r;
    };
    auto token = [&](const Raw &r, int t) {
      Token k = {0, nullptr};
      uint32_t pos = r.sel, sub = 0;  // a position past 2^31 - 1 (one below 0) is in no block
      if (!plain) {
        const uint32_t block = a.sel_block.div(r.entry);
        sub = t - r.entry * a.rec_tokens.d;
        const int64_t rec = static_cast<int64_t>(r.sel) * a.sel_block.d + (r.entry - block * a.sel_block.d);
        const int64_t p = rec * a.rec_tokens.d + sub;  // (below 2^63: sel_block and rec_tokens are below 2^16)
        pos = r.sel < 0 || p > INT32_MAX ? 0x80000000u : static_cast<uint32_t>(p);
      }
      const uint32_t blk = a.S.div(pos & 0x7fffffffu), near = r.slot, far = r.slot - a.B - 1;
      const bool is_near = near <= static_cast<uint32_t>(a.B), is_far = r.slot > a.B && far < a.res_rows;
      const bool inside = pos < 0x80000000u && blk < a.scale_blocks;
      if (r.slot != -1) {
        if (inside && pos < seq && (is_near || is_far)) {
          const uint64_t base0 = reinterpret_cast<uint64_t>(is_near ? hot : a.resident);
          k.row = base0 + static_cast<uint64_t>(is_near ? near : far) * (is_near ? a.hot_row : a.res_row);
          if (!plain) k.row += static_cast<uint64_t>(sub) * a.row_bytes;
          k.scales = scales + blk * a.columns;
        } else if (a.status && !(pos < 0x80000000u && pos >= seq)) {  // (beyond seq the table may end)
          atomicOr(a.status, HISPARSE_ERR_RANGE);
        }
      }
      return k;
    };
    // In steps of a token a lane, `per` of them a tile.  Loads are kAhead steps ahead of their
    // use: of slots and positions, and of the scales after the addresses are out; each of kAhead
    // steps in turn has its own registers, so that none waits for another's load.
    constexpr int kLooks = Shape<N>::looks, kAhead = 2;
    const int per = (a.tile + 32 * kLooks - 1) / (32 * kLooks), steps = tiles * per;
    const int mine = (warp - Shape<N>::look) * 32 + lane;
    struct Step {
      Raw r;
      int32_t k, v;
      bool use;
    };
    auto fetch = [&](Step &x, int tile, int sub) {
      const int j = mine + 32 * kLooks * sub;
      x.r = raw(j < a.tile ? t0 + tile * a.tile + j : t1);
    };
    auto put_scales = [&](const Step &x, int tile, int sub) {
      const int j = mine + 32 * kLooks * sub;
      // a NaN scale of K may have the masked tokens' bits: it gets others
      const int32_t k = !x.use ? kMasked : (x.k & 0x7fffffff) > 0x7f800000 ? 0x7fc00000 : x.k;
      if (j < a.tile)
        asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(base + a.off_meta + (tile % kTables * a.tile + j) * 8),
                     "r"(k), "r"(x.v)
                     : "memory");
      if (sub == per - 1) bar_arrive(b_meta + 8 * (tile % kTables));
    };
    // Steps kAhead behind, now, and kAhead ahead: (tile, sub) of each.
    int bt = 0, bs = 0, nt = 0, ns = 0, at = 0, as = 0;
    auto advance = [&](int &tile, int &sub) {
      if (++sub == per) {
        sub = 0;
        ++tile;
      }
    };
    auto step = [&](Step &x, int n) {
      if (n >= steps) return;
      const int slot = nt % kTables, j = mine + 32 * kLooks * ns;
      const Token now = token(x.r, t0 + nt * a.tile + j);
      fetch(x, at, as);
      advance(at, as);
      bool put = n >= kAhead;  // the scales of the step before the last
      if (ns == 0 && nt >= kTables) {
        if (put) put_scales(x, bt, bs), advance(bt, bs);
        put = false;
        bar_wait(b_used + 8 * slot, (nt / kTables - 1) & 1, fail);
      }
      if (j < a.tile) {
        const uint32_t to = base + a.off_rows + (slot * a.tile + j) * 8;
        asm volatile("st.shared.b64 [%0], %1;" ::"r"(to), "l"(now.row ? now.row + k_at : zeros) : "memory");
        if (!a.latent)
          asm volatile("st.shared.b64 [%0], %1;" ::"r"(to + kTables * a.tile * 8), "l"(now.row ? now.row + v_at : zeros)
                       : "memory");
      }
      if (ns == per - 1) bar_arrive(b_tab + 8 * slot);
      advance(nt, ns);
      if (put) put_scales(x, bt, bs), advance(bt, bs);
      const int32_t *sc = reinterpret_cast<const int32_t *>(now.scales);
      x.use = now.row != 0;
      x.k = ld_if(sc, x.use, 0);
      x.v = ld_if(sc + v_col, x.use, 0);
    };
    Step x0, x1;
    fetch(x0, at, as), advance(at, as);
    fetch(x1, at, as), advance(at, as);
#pragma unroll 1
    for (int n = 0; n < steps; n += kAhead) {
      step(x0, n);
      step(x1, n + 1);
    }
    // the last two steps' scales, in order
    if (steps > 1) {
      put_scales(steps & 1 ? x1 : x0, bt, bs);
      advance(bt, bs);
    }
    if (steps > 0) put_scales(steps & 1 ? x0 : x1, bt, bs);
  } else {
    // ---- products: a warp for the scores and one for the values; one lane issues -----------
    const uint32_t d_qk = mma_desc(kQ, false, false);
    const uint32_t d_pv = mma_desc(N, true, true), d_pvs = mma_desc(kP * N, true, true);
    const int k_steps = (a.k_dim + 31) >> 5;
    const bool elected = elect_one();
    const uint32_t q_desc = smem_desc(base + a.off_q), p_desc = smem_desc(base + a.off_p);
    // A half's part of tile i's scores.
    int s = 0, turn = 0;  // the tile's stage, and how often the stages went round
    auto scores = [&](int i, int u) {
      const Half half = half_of(a, u);
      const uint32_t d = tmem + (i & 1) * kQ;
      uint32_t q = q_desc + half.c0 * kQ * 8, k = smem_desc(base + s * a.stage_bytes) + half.c0 * a.tile * 8;
      if (elected) {
        int left = k_steps - 4 * half.c0;
        for (int c = half.c0; c < half.c1; ++c, left -= 4, k += a.tile * 8, q += kQ * 8) {
          if (left >= 4) {
#pragma unroll
            for (int e = 0; e < 4; ++e) mma_f8(d, k + 2 * e, q + 2 * e, d_qk, e > 0 ? 1 : c > 0);
          } else {
            for (int e = 0; e < left; ++e) mma_f8(d, k + 2 * e, q + 2 * e, d_qk, c > 0 || e > 0);
          }
        }
        if (half.v0 == half.v1) tc_commit(b_empty + 16 * s + 8 * u);
        if (u == 1 || !a.latent) tc_commit(b_s + 8 * (i & 1));
      }
      __syncwarp();
    };
    // ... and of its products with the probabilities.
    auto values = [&](int i, int u) {
      const Half half = half_of(a, u);
      const int steps = (min(a.tile, t1 - t0 - i * a.tile) + 31) >> 5;
      uint32_t v = smem_desc(base + s * a.stage_bytes) + ((half.is_v ? a.k_chunks : 0) + half.v0) * a.tile * 8;
      if (elected) {
        for (int j = half.v0; j < half.v1; ++j, v += a.tile * 8) {
          const uint32_t d = t_o + j * a.sums * N;
          if (kMerge && a.sums > 1) {
            uint32_t p = p_desc, w = v;
#pragma unroll 2
            for (int k = 0; k < steps; ++k, p += 256, w += 256) mma_f8(d, w, p, d_pvs, i > 0 || k > 0);
            continue;
          }
          uint32_t p = p_desc, p2 = p_desc + a.tile * 8, w = v;
#pragma unroll 2
          for (int k = 0; k < steps; ++k, p += 256, p2 += 128, w += 256) {
#pragma unroll
            for (int t = 0; t < kP0; ++t) mma_f8(d, w, p + t * N / 16, d_pv, t > 0 ? 1 : i > 0 || k > 0);
            if (kP0 < kP) mma_f8<kDescHi64>(d, w, p2, d_pv, 1);
          }
        }
        if (half.v0 < half.v1) tc_commit(b_empty + 16 * s + 8 * u);
        if (u == 1) {
          tc_commit(b_used + 8 * (i % kTables));
          tc_commit(b_pv);
        }
      }
      __syncwarp();
    };
    // Scores run at most one tile ahead of the softmax (two buffers); each half starts as it
    // arrives.
    if (warp == Shape<N>::mma) {
      bar_wait(b_q, 0, fail);
      for (int i = 0; i < tiles; ++i) {
        if (i > 1) bar_wait(b_read + 8 * (i & 1), (i / 2 - 1) & 1, fail);
#pragma unroll 1
        for (int u = 0; u < (a.latent ? 2 : 1); ++u) {
          bar_wait(b_full + 16 * s + 8 * u, turn & 1, fail);
          fence_async();
          __syncwarp();
          tc_after();
          scores(i, u);
        }
        if (++s == a.stages) s = 0, ++turn;
      }
    } else {
      for (int i = 0; i < tiles; ++i) {
        // V's half is waited for, and made visible to the tensor cores, before the probabilities come.
        // A latent record's halves were, by the warp that issued the scores that led to them.
        if (!a.latent) {
          bar_wait(b_full + 16 * s + 8, turn & 1, fail);
          fence_async();
          __syncwarp();
        }
        bar_wait(b_p, i & 1, fail);
        __syncwarp();
        tc_after();
#pragma unroll 1
        for (int u = a.latent ? 0 : 1; u < 2; ++u) values(i, u);
        if (++s == a.stages) s = 0, ++turn;
      }
    }
  }
  // ---- join ----------------------------------------------------------------------
  // Every product is done (the softmax warps' last wait), so the stages and Q hold
  // nothing any more.  A lone CTA's results pass through them in their type; in a cluster they
  // take the CTA's sums [N][v_dim] for the others to read, and each CTA joins a share of the heads.
  // (Loops rather than unrolled runs: this is executed once, at the instruction cache's pace.)
  __syncwarp();
  const bool lone = a.cluster == 1;
  const int share = N / a.cluster, n0 = static_cast<int>(rank) * share;
  if (!lone) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");  // all CTAs run
  __syncthreads();
  if (s_fail) {  // (no wait follows that sets it)  Nothing here is a result; the products end before TMEM goes.
    if (tid < N) s_l[tid] = s_f[tid] = NAN;
    if (warp == Shape<N>::mma || warp == Shape<N>::mma + 1) {
      const uint32_t bar = b_done + 8 * (warp - Shape<N>::mma);
      if (elect_one()) tc_commit(bar);
      __syncwarp();
      const long long start = clock64();
      while (!bar_try(bar, 0) && clock64() - start < kWaitCycles) {
      }
    }
    __syncthreads();
  }
  T *out = static_cast<T *>(a.out) + qrow * a.out_row;
  const int h0 = kvh * a.group + hg * N, heads = min(N, a.group - static_cast<int>(hg) * N);
  if (!lone && tid < N) {  // a column's offset and sum to the CTA that joins it
    const uint32_t to = peer(smem_u32(&s_pair[rank * share + tid % share]), tid / share);
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(to), "f"(s_m[tid]), "f"(s_l[tid]) : "memory");
  }
  if (warp < kSoft) {
    tc_after();
    const int wl = warp & 3;
    const uint32_t lanes = static_cast<uint32_t>(wl * 32) << 16;
#pragma unroll 1
    for (int c = (warp >> 2) * NC; c < ((warp >> 2) + 1) * NC; c += 16) {
      float f[16];
#pragma unroll
      for (int e = 0; e < 16; e += 4) {
        const float4 x = ld_shared4(smem_u32(s_f + c + e));
        f[e] = x.x, f[e + 1] = x.y, f[e + 2] = x.z, f[e + 3] = x.w;
      }
#pragma unroll 1
      for (int j = 0; j < a.v_tiles; ++j) {
        const int d = j * 128 + wl * 32 + lane;
        uint32_t o[16];
        if (tiles > 0) {
          const uint32_t at = t_o + lanes + j * a.sums * N + c;
          tc_ld16(at, o);
          if (kMerge && a.sums > 1) {
            uint32_t y[kP - 1][16];
#pragma unroll
            for (int t = 1; t < kP; ++t) tc_ld16(at + t * N, y[t - 1]);
            tc_wait_ld16(o);
#pragma unroll
            for (int t = 1; t < kP; ++t) {
              tc_wait_ld16(y[t - 1]);
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) + __uint_as_float(y[t - 1][e]));
            }
          } else {
            tc_wait_ld16(o);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] = 0;
        }
        if (d >= a.v_dim) continue;
        if (lone) {
          const uint32_t to = base + (c * a.v_dim + d) * static_cast<uint32_t>(sizeof(T));
          uint16_t h[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const T x = from_f32<T>(f[e] != 0.f ? __uint_as_float(o[e]) * f[e] : 0.f);
            h[e] = *reinterpret_cast<const uint16_t *>(&x);
          }
#pragma unroll
          for (int e = 0; e < 16; ++e)
            asm volatile("st.shared.b16 [%0], %1;" ::"r"(to + e * a.v_dim * static_cast<uint32_t>(sizeof(T))), "h"(h[e]) : "memory");
        } else {
          const uint32_t to = base + (c * a.v_dim + d) * 4;
#pragma unroll
          for (int e = 0; e < 16; ++e)
            asm volatile("st.shared.b32 [%0], %1;" ::"r"(to + e * a.v_dim * 4), "r"(o[e]) : "memory");
        }
      }
    }
    __syncwarp();
    tc_before();
  }
  __syncwarp();
  if (lone) {
    __syncthreads();
  } else {
    cluster_sync();
  }
  if (warp == Shape<N>::mma) {
    tc_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(a.tmem_cols));
  }
  if (tid == 0 && s_fail && a.status) atomicOr(a.status, HISPARSE_ERR_WAIT);
  if (!lone) {
    // weights 2^(m_r - max m) of the CTAs' sums
    if (tid < share) {
      float m = kNone, z = 0.f;
#pragma unroll 1
      for (int r = 0; r < a.cluster; ++r) m = fmaxf(m, s_pair[r * share + tid].x);
#pragma unroll 1
      for (int r = 0; r < a.cluster; ++r) {
        const float2 x = s_pair[r * share + tid];
        const float w = ex2(x.x - m);
        s_w[r * share + tid] = w;
        z = fmaf(w, x.y, z);
      }
      s_m[tid] = m;
      s_l[tid] = z;
      s_f[tid] = z > 0.f || z != z ? exp2f(-kFold) / z : 0.f;
    }
    __syncthreads();
  }
  const int mine = lone ? heads : min(share, heads - n0), first = lone ? 0 : n0;
  if (a.lse && tid < mine) {
    const float z = s_l[tid];
    a.lse[qrow * a.heads + h0 + first + tid] =
        z > 0.f || z != z ? (s_m[tid] + (kFold + log2f(z))) * 0.6931471805599453f : -INFINITY;
  }
  if (lone) {
    const uint32_t total = heads * (a.quads.d >> 1);
    for (uint32_t i = tid; i < total; i += kThreads) {
      uint32_t n, d;
      a.quads.divmod(2 * i, n, d);
      const float4 v = ld_shared4(base + (n * a.v_dim + 4 * d) * sizeof(T));
      *reinterpret_cast<float4 *>(out + static_cast<int64_t>(h0 + n) * a.out_head + 4 * d) = v;
    }
    return;
  }
#pragma unroll 1
  for (int i = tid; i < mine * static_cast<int>(a.quads.d); i += kThreads) {
    uint32_t nn, d;
    a.quads.divmod(i, nn, d);
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    const uint32_t at = base + ((n0 + nn) * a.v_dim + 4 * d) * 4;
#pragma unroll 1
    for (int r0 = 0; r0 < a.cluster; r0 += 4) {
      float4 v[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) v[r] = ld_peer4(peer(at, min(r0 + r, a.cluster - 1)));
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float w = r0 + r < a.cluster ? s_w[(r0 + r) * share + nn] : 0.f;
        acc[0] = fmaf(w, v[r].x, acc[0]);
        acc[1] = fmaf(w, v[r].y, acc[1]);
        acc[2] = fmaf(w, v[r].z, acc[2]);
        acc[3] = fmaf(w, v[r].w, acc[3]);
      }
    }
    const float inv = s_f[nn];
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[e] = inv != 0.f ? acc[e] * inv : 0.f;
    Vec<T, 4> o;
    o.set_pair(0, acc[0], acc[1]);
    o.set_pair(1, acc[2], acc[3]);
    *reinterpret_cast<Vec<T, 4> *>(out + static_cast<int64_t>(h0 + n0 + nn) * a.out_head + 4 * d) = o;
  }
  __syncwarp();
  cluster_sync();  // peers have read this CTA's shared memory
}

constexpr uint32_t kSmemSm = 233472;     // of an SM; a CTA takes its own and 1 KB more
constexpr uint32_t kSmemCta = 232448;    // at most, static and dynamic

// Tile, stages and offsets for N heads; false where they do not fit in `limit` bytes.
bool plan_smem(AttendArgs &a, int N, int terms, int p_terms, int tables, int tile, uint32_t limit, uint32_t &bytes) {
  a.tile = tile;
  a.k_chunks = (a.k_dim + 127) / 128;
  a.v_tiles = (a.v_dim + 127) / 128;
  a.v_chunks = a.latent ? 0 : a.v_tiles;
  // (a latent record whose V is wider than its K's chunks cannot be: v_dim <= k_dim)
  a.stage_bytes = static_cast<uint32_t>(a.k_chunks + a.v_chunks) * tile * 128;
  const uint32_t q = static_cast<uint32_t>(terms) * a.k_chunks * N * 128;
  const uint32_t p = tile * (p_terms * N > 128 ? 192 : 128);
  // rows beyond a tile that the 128-row products read stay inside: Q and P follow
  const uint32_t over = (128 - tile) * 128;
  const uint32_t rest = q + p + (q + p < over ? over - q - p : 0);
  // tables: two scales a token, and a row or its address (two with a V part)
  const uint32_t meta = tables * tile * (a.latent ? 16 : 24);
  const uint32_t sums = static_cast<uint32_t>(N) * a.v_dim * 4;
  const uint32_t fixed = rest + meta + 1024;
  if (fixed + 2 * a.stage_bytes > limit) return false;
  a.stages = std::min<uint32_t>(kMaxStages, (limit - fixed) / a.stage_bytes);
  a.off_q = a.stages * a.stage_bytes;
  a.off_p = a.off_q + q;
  a.off_meta = a.off_q + rest;
  a.off_rows = a.off_meta + tables * tile * 8;
  bytes = std::max(a.off_meta + meta, sums) + 1024;
  return bytes <= limit;
}

// Clusters of c CTAs that the GPU runs at once (asked once for each of the few
// combinations that a program uses).
int active_clusters(const void *fn, int threads, uint32_t bytes, int c, int dev) {
  struct Known {
    const void *fn;
    uint32_t bytes;
    int c, dev, n;
  };
  thread_local Known known[64];
  thread_local int count = 0;
  for (int i = 0; i < std::min(count, 64); ++i)
    if (known[i].fn == fn && known[i].bytes == bytes && known[i].c == c && known[i].dev == dev) return known[i].n;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3(c);
  lc.blockDim = dim3(threads);
  lc.dynamicSmemBytes = bytes;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = c;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  lc.attrs = at;
  lc.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, fn, &lc) != cudaSuccess) {
    cudaGetLastError();
    n = 0;
  }
  known[count++ % 64] = {fn, bytes, c, dev, n};
  return n;
}

struct Plan {
  AttendArgs a;
  int64_t units;
  double cycles;
  uint32_t bytes;
};

// How N heads a CTA and a cluster of how many CTAs would do, in estimated cycles.
//
// A wave of CTAs costs its start (11,000 cycles to the first scores, 90 for each head's q),
// a turn for every tile, and the join of a cluster (N * v_dim sums a CTA at the 14 B/cycle of
// distributed shared memory).  A tile's turn is the largest of: its copies, at 27 B/cycle; its
// products, 32 cycles for the rows and a quarter for each column, 40 at least; the softmax;
// and the 7,400 cycles from a free stage to the next over the number of stages.  Wider groups read a row
// fewer times, narrower ones make more CTAs.  What that reads at 1.92 GHz, against what was measured (us,
// 2048 tokens a row):
//   8 requests, 64 latent heads: 16 heads by 4 CTAs 16 (16), 32 by 4 22 (22), 64 by 8 20 (22), 16 by 1 37 (35),
//     16 by 8 38 (36), 32 by 8 33 (34);
//   32 requests, 32 latent heads: 32 by 4 22 (25), 16 by 2 24 (25), 32 by 2 31 (36), 16 by 1 37 (38), 32 by 1 50 (56);
//   64 requests, 128 latent heads: 64 by 1 51 (76), 64 by 2 67 (95), 32 by 1 99 (111), 16 by 1 149 (147);
//   16, 24 and 64 requests, 32 heads on 8 of 128: 16 by 1 20 (22), 40 (42) and 80 (82), by 2 29 (29), 44 (45) and
//     103 (103), by 4 46 (43) and 68 (65).
// 64 heads take longer than it says, as two stages are not enough to overlap what a tile goes through; the
// order is right in each row.
template <class T, int N>
int plan_attend(const AttendArgs &args, int64_t pairs, Plan &best) {
  AttendArgs a = args;
  a.hgroups = (a.group + N - 1) / N;
  const int64_t units = pairs * a.hgroups;
  constexpr int kTerms = Terms<T>::n;
  // TMEM: two score buffers and the sums, those of each term where there is room, a power of two of columns.
  constexpr int kP = Terms<T>::p;
  int cols = 32;
  a.v_tiles = (a.v_dim + 127) / 128;
  a.sums = kP * N <= 128 && 2 * kTerms * N + a.v_tiles * kP * N <= 512 ? kP : 1;
  while (cols < 2 * kTerms * N + a.v_tiles * a.sums * N) cols *= 2;
  a.tmem_cols = cols;
  const int64_t tokens = static_cast<int64_t>(a.entries) * a.rec_tokens.d;
  auto fn = attend_kernel<T, N>;
  static std::atomic<uint64_t> ready{0};
  static std::atomic<uint32_t> fixed{0};
  int dev = 0;
  HS_CUDA(cudaGetDevice(&dev));
  if (!(ready.load() >> (dev & 63) & 1)) {
    cudaFuncAttributes fa;
    HS_CUDA(cudaFuncGetAttributes(&fa, fn));
    fixed.store(static_cast<uint32_t>(fa.sharedSizeBytes));
    HS_CUDA(cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kSmemCta - static_cast<uint32_t>(fa.sharedSizeBytes)));
    HS_CUDA(cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1));
    ready.fetch_or(1ull << (dev & 63));
  }
  // CTAs that share an SM would share its TMEM: each takes at least as large a part of
  // the SM's shared memory as of its TMEM, so that no CTA of a cluster waits for columns that
  // a CTA of another cluster holds.
  const uint32_t whole = kSmemCta - fixed.load();
  const uint32_t least = std::min(whole, kSmemSm / 512 * cols - 1024);
  uint32_t bytes = 0;
  bool ok = false;
  for (int tile = 128; tile >= 64 && !ok; tile -= 32) ok = plan_smem(a, N, kTerms, Terms<T>::p, Shape<N>::tables, tile, whole, bytes);
  if (!ok) return HISPARSE_OK;  // the widest rows leave no room for two tiles of so many heads
  bytes = std::max(bytes, least);
  const double copy = 400 + a.tile * (a.k_dim + (a.latent ? 0 : a.v_dim)) / 27.0;
  const double products = (a.k_dim + 31) / 32 * std::max(40.0, 32 + kTerms * N / 4.0) +
                          a.v_tiles * (a.tile / 32) * (a.sums > 1 ? std::max(40.0, 32 + kP * N / 4.0) : kP * std::max(40.0, 32 + N / 4.0));
  const double turn = std::max({copy, products, N > 32 ? 2000.0 : 1200.0, 7400.0 / a.stages});
  for (int c = 1; c <= kMaxCluster; c *= 2) {
    if (c > 1 && tokens < 64 * c) break;
    const int at_once = active_clusters(reinterpret_cast<const void *>(fn), Shape<N>::threads, bytes, c, dev);
    if (at_once < 1) continue;
    const int64_t waves = (units + at_once - 1) / at_once;
    const int64_t per = ((tokens + c - 1) / c + 31) / 32 * 32;
    const double join = c > 1 ? 2500 + N * a.v_dim * 4.0 * (c - 1) / c / 14 : 0;
    const double cycles = waves * (11000 + 90.0 * N + turn * ((per + a.tile - 1) / a.tile) + join);
    if (cycles < best.cycles) {
      a.cluster = c;
      a.per_cta = static_cast<int>(per);
      best = {a, units, cycles, bytes};
    }
  }
  return HISPARSE_OK;
}

template <class T, int N>
int launch_attend(const Plan &p, void *stream) {
  const int64_t ctas = p.units * p.a.cluster;
  if (ctas > 0x7fffffff) return HISPARSE_EBOUND;
  return launch_pdl(attend_kernel<T, N>, dim3(static_cast<unsigned>(ctas)), dim3(Shape<N>::threads), p.bytes, stream,
                    p.a.cluster, p.a);
}

template <class T>
int pick_attend(const AttendArgs &a, int64_t pairs, void *stream) {
  Plan best = {};
  best.cycles = 1e300;
  int n = 0;
  // 64 heads with two terms at most: three of 64 do not fit a 128-byte row of probabilities.
  double before = best.cycles;
  auto took = [&](int heads) {
    if (best.cycles < before) n = heads;
    before = best.cycles;
  };
  if (const int rc = plan_attend<T, 16>(a, pairs, best)) return rc;
  took(16);
  if (a.group > 16) {
    if (const int rc = plan_attend<T, 32>(a, pairs, best)) return rc;
    took(32);
  }
  if constexpr (Terms<T>::n == 2) {
    if (a.group > 32) {
      if (const int rc = plan_attend<T, 64>(a, pairs, best)) return rc;
      took(64);
    }
    if (n == 64) return launch_attend<T, 64>(best, stream);
  }
  if (n == 32) return launch_attend<T, 32>(best, stream);
  if (n == 16) return launch_attend<T, 16>(best, stream);
  return HISPARSE_EBOUND;
}

}  // namespace

extern "C" {

int hisparse_attend(const hisparse_attend_args *g, void *stream) {
  if (!g) return HISPARSE_EINVAL;
  const hisparse_records &r = g->rec;
  if (const int rc = records_ok(r)) return rc;
  if (g->dtype != HISPARSE_BF16 && g->dtype != HISPARSE_F16) return HISPARSE_EINVAL;
  if (g->num_requests < 0 || g->rows < 1 || g->entries < 0 || g->heads < 1 ||
      g->heads % r.kv_heads || g->buffer_slots < 0 || g->record_tokens < 1 ||
      g->sel_block_tokens < 0 || g->scale_blocks < 1 || g->resident_rows < 0)
    return HISPARSE_EINVAL;
  if (g->sel_block_tokens > 1 && g->entries % g->sel_block_tokens) return HISPARSE_EINVAL;
  if (g->num_requests == 0) return HISPARSE_OK;
  if (!g->q || !g->out || !g->hot || !g->scales) return HISPARSE_EINVAL;
  if (g->entries > 0 && (!g->d_slots || !g->d_sel)) return HISPARSE_EINVAL;
  if (!aligned16(g->q) || !aligned16(g->out) || !aligned16(g->hot) || g->q_row_stride % 8 ||
      g->q_head_stride % 8 || g->out_row_stride % 8 || g->out_head_stride % 8 ||
      g->hot_req_stride % 16 || g->hot_row_stride % 16)
    return HISPARSE_EINVAL;
  const int64_t row = record_row_bytes(r);
  if (g->hot_row_stride < row * g->record_tokens) return HISPARSE_EINVAL;
  if (g->resident && (!aligned16(g->resident) || g->resident_row_stride % 16 ||
                      g->resident_row_stride < row * g->record_tokens))
    return HISPARSE_EINVAL;
  if (g->hot_row_stride > UINT32_MAX || (g->resident && g->resident_row_stride > UINT32_MAX) ||
      static_cast<int64_t>(g->scale_blocks) * record_columns(r) > INT32_MAX || g->sel_block_tokens > 65535)
    return HISPARSE_EBOUND;
  if (g->record_tokens > 65535 || g->heads > 65535 ||
      static_cast<int64_t>(g->num_requests) * g->rows > (1 << 28) ||
      static_cast<int64_t>(g->entries) * g->record_tokens > (1 << 30))
    return HISPARSE_EBOUND;
  AttendArgs a = {};
  a.rows = g->rows; a.entries = g->entries; a.heads = g->heads;
  a.kv_heads = r.kv_heads; a.k_dim = r.k_dim; a.v_dim = r.v_dim; a.latent = r.latent;
  a.group = g->heads / r.kv_heads;
  a.B = g->buffer_slots; a.columns = record_columns(r);
  a.S = FastDiv(r.block_tokens);
  a.rec_tokens = FastDiv(g->record_tokens);
  a.sel_block = FastDiv(std::max(1, g->sel_block_tokens));
  a.scale_log2 = g->softmax_scale * 1.4426950408889634f;
  a.q = g->q; a.q_row = g->q_row_stride; a.q_head = g->q_head_stride;
  a.out = g->out; a.out_row = g->out_row_stride; a.out_head = g->out_head_stride;
  a.lse = g->lse; a.sel = g->d_sel; a.slots = g->d_slots;
  a.hot = static_cast<const char *>(g->hot);
  a.hot_req = g->hot_req_stride; a.hot_row = static_cast<uint32_t>(g->hot_row_stride);
  a.resident = static_cast<const char *>(g->resident);
  a.res_rows = g->resident ? static_cast<uint32_t>(std::min<int64_t>(g->resident_rows, INT32_MAX)) : 0;
  a.res_row = g->resident ? static_cast<uint32_t>(g->resident_row_stride) : 0;
  a.scales = g->scales; a.scales_req = g->scales_req_stride; a.scale_blocks = g->scale_blocks;
  a.seq_lens = g->d_seq_lens; a.num_reqs = g->d_num_reqs; a.status = g->d_status;
  a.row_bytes = static_cast<uint32_t>(row);
  a.quads = FastDiv(r.v_dim / 4);
  const int64_t pairs = static_cast<int64_t>(g->num_requests) * g->rows * r.kv_heads;
  return g->dtype == HISPARSE_BF16 ? pick_attend<__nv_bfloat16>(a, pairs, stream)
                                   : pick_attend<__half>(a, pairs, stream);
}

}  // extern "C"
