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
// q, scaled by a power of two for each head, is t1 + t2 (+ t3 for f16), each the e4m3
// rounding of what the ones before leave; bf16's 8 significant bits are two such terms
// exactly.  The probabilities are e4m3 + e5m2 (f16: e4m3 + e4m3 + e5m2), the last one in
// e5m2 for its range: with 64 as the largest, what falls below is 2^-22 of it.
// The scale of K enters the scores in 32 bits; the scale of V enters the probabilities
// (p_j sV_j is what multiplies the raw bytes of V), through the exponent, so the
// running maximum is over s_j + log2(sV_j) and no product leaves the range.
//
// Warps: four softmax warps (a lane a token, TMEM lane = token) for each 32 columns, four that
// gather (16-byte cp.async into the 128-byte-swizzled tiles the tensor cores read,
// several tiles ahead), and one that issues the products.  S is double buffered in TMEM, so the scores of tile i+1
// are computed while the softmax of tile i runs.  O is rescaled only where a column's
// maximum has grown by more than 2^2.75 since it was last set.
#include <algorithm>
#include <atomic>

#include "common.cuh"

namespace {

constexpr int kGather = 4;  // warps that gather
constexpr int kMaxStages = 6;
constexpr int kMaxCluster = 16;
constexpr float kTop = 6.f;     // log2 of a column's largest probability when its offset is set
constexpr float kSlack = 8.75f; // ... and what it may grow to before the offset moves (448 = 2^8.8)

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
  int64_t hot_req, hot_row;
  const char *resident;
  int64_t res_rows, res_row;
  const float *scales;
  int64_t scales_req;
  int32_t scale_blocks;
  const int32_t *seq_lens, *num_reqs;
  uint32_t *status;
  int64_t row_bytes;  // a token's part of a record
  // the launch's plan
  int32_t cluster, per_cta, tile, stages, k_chunks, v_chunks, v_tiles, tmem_cols;
  FastDiv quads;  // v_dim / 4
  uint32_t stage_bytes, off_q, off_p, off_meta, off_misc;
};

// ---- PTX ---------------------------------------------------------------------
__device__ __forceinline__ uint32_t smem_u32(const void *p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool bar_test(uint32_t bar, uint32_t parity) {  // never suspends
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n"
      " mbarrier.test_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n"
      " mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// Waits have a limit (seconds, against microseconds in use).  One that runs out sets
// *fail, after which no wait of the CTA waits any more: every loop still makes
// its turns, so barriers stay matched, TMEM is freed and the kernel ends, with
// HISPARSE_ERR_WAIT in the status.
__device__ __noinline__ void bar_wait_slow(uint32_t bar, uint32_t parity, volatile int *fail) {
  const long long start = clock64();
  while (clock64() - start < (1ll << 32)) {
    if (bar_try(bar, parity) || *fail) return;
  }
  *fail = 1;
}
__device__ __forceinline__ void bar_wait(uint32_t bar, uint32_t parity, volatile int *fail) {
#pragma unroll 1
  for (int i = 0; i < 64; ++i)
    if (bar_try(bar, parity)) return;
  bar_wait_slow(bar, parity, fail);
}
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
// The elected lane's mbarrier arrival once its products so far are done.
__device__ __forceinline__ void tc_commit(uint32_t bar, uint32_t elected) {
  asm volatile(
      "{\n .reg .pred e;\n setp.ne.b32 e, %1, 0;\n"
      " @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}" ::"r"(bar),
      "r"(elected)
      : "memory");
}
// Shared-memory descriptor of a 128-byte-swizzled operand whose groups of 8 rows are 1024
// bytes apart (either major-ness: the other offset is not used).  Its lower word; the
// upper one is the same for all.
constexpr uint32_t kDescHi = 64u | 1u << 14 | 2u << 29;
__device__ __forceinline__ uint32_t smem_desc(uint32_t addr) { return addr >> 4 | 1u << 16; }
// Instruction descriptor: f32 accumulator, A e4m3, B e4m3 or e5m2, M = 128.
__device__ __forceinline__ uint32_t mma_desc(int n, bool b_e5m2, bool transposed) {
  return (1u << 4) | (b_e5m2 ? 1u << 10 : 0u) | (transposed ? 3u << 15 : 0u) |
         (static_cast<uint32_t>(n) >> 3 << 17) | (128u >> 4 << 24);
}
__device__ __forceinline__ void mma_f8(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc,
                                       uint32_t accumulate, uint32_t elected) {
  asm volatile(
      "{\n .reg .pred p, e;\n .reg .b64 da, db;\n"
      " setp.ne.b32 p, %4, 0;\n setp.ne.b32 e, %5, 0;\n"
      " mov.b64 da, {%1, %6};\n mov.b64 db, {%2, %6};\n"
      " @e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], da, db, %3, p;\n}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "r"(elected), "r"(kDescHi)
      : "memory");
}
#define TC_REGS16(r)                                                                        \
  "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),   \
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),     \
      "r"(r[15])
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
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::TC_REGS16(r),
      "r"(addr)
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
// 16 bytes of global memory into shared memory, or 16 zeros where `bytes` is 0.
__device__ __forceinline__ void cp_async16(uint32_t dst, const char *src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void cp_wait(int pending) {
  switch (pending) {
    case 0: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
    case 1: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
    case 2: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
    case 3: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
    case 4: asm volatile("cp.async.wait_group 4;" ::: "memory"); break;
    default: asm volatile("cp.async.wait_group 5;" ::: "memory"); break;
  }
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
// OR over a group of four softmax warps, and their barrier.
__device__ __forceinline__ bool soft_any(int group, bool x) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %1, 0;\n"
      " barrier.cta.red.or.pred q, %2, 128, p;\n selp.u32 %0, 1, 0, q;\n}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(x)), "r"(group + 1)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void soft_sync(int group) {
  asm volatile("barrier.cta.sync %0, 128;" ::"r"(group + 1) : "memory");
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
__device__ __forceinline__ float ld_peer(uint32_t addr) {
  float r;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(r) : "r"(addr) : "memory");
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
__device__ __forceinline__ void st_shared4(uint32_t addr, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(x), "r"(y), "r"(z), "r"(w)
               : "memory");
}

// Two values to e4m3 (or e5m2) with rounding to nearest; *x and *y keep what the rounding
// leaves.
template <bool kE5M2>
__device__ __forceinline__ uint32_t take_term(float &x, float &y) {
  uint16_t p;
  uint32_t h;
  if (kE5M2) {
    asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(p) : "f"(y), "f"(x));
    return p;
  }
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(p) : "f"(y), "f"(x));
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(p));
  const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
  x -= f.x;
  y -= f.y;
  return p;
}

// ---- tokens ------------------------------------------------------------------
struct Raw {
  int32_t slot, sel, entry;
};
struct Token {
  const char *row;  // NULL: nothing to read
  float k, v;       // the scales
};

template <class T>
struct Terms;
template <>
struct Terms<__nv_bfloat16> {
  static constexpr int n = 2;
};
template <>
struct Terms<__half> {
  static constexpr int n = 3;
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
  static constexpr int workers = soft + kGather;
  static constexpr int threads = 32 * (workers + 1);
};

template <class T, int N>
__global__ void __launch_bounds__(Shape<N>::threads, N == 16 ? 2 : 1) attend_kernel(const AttendArgs a) {
  constexpr int kTerms = Terms<T>::n;
  constexpr int NC = Shape<N>::cols, kSoft = Shape<N>::soft, kWorkers = Shape<N>::workers;
  constexpr int kThreads = Shape<N>::threads;
  extern __shared__ char smem_raw[];
  __shared__ uint64_t s_bars[2 * kMaxStages + 5];
  __shared__ uint32_t s_tmem;
  __shared__ int s_fail;
  __shared__ float s_m[N], s_l[N], s_f[N], s_wmax[4][N], s_w[kMaxCluster * N];
  __shared__ __align__(16) float s_qf[N];
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t bars = smem_u32(s_bars);
  const uint32_t b_full = bars, b_empty = bars + 8 * kMaxStages, b_s = bars + 16 * kMaxStages;
  const uint32_t b_p = b_s + 16, b_pv = b_s + 24, b_q = b_s + 32;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const uint32_t rank = a.cluster > 1 ? blockIdx.x % a.cluster : 0;
  const uint32_t unit = blockIdx.x / a.cluster;
  const uint32_t hg = unit % a.hgroups, kvh = unit / a.hgroups % a.kv_heads;
  const int64_t qrow = unit / a.hgroups / a.kv_heads;
  const int req = static_cast<int>(qrow / a.rows);

  if (tid == 0) {
    for (int s = 0; s < a.stages; ++s) {
      bar_init(b_full + 8 * s, 32 * kGather);
      bar_init(b_empty + 8 * s, 1);
    }
    bar_init(b_s, 1);
    bar_init(b_s + 8, 1);
    bar_init(b_p, 32 * kSoft);
    bar_init(b_pv, 1);
    bar_init(b_q, 32 * kWorkers);
    s_fail = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  for (int c = tid; c < N; c += kThreads) s_m[c] = -INFINITY;
  // The last 16 of 32 K columns that a product reads beyond k_dim: zero in every
  // stage (the gather never writes them) and in Q.
  if (a.k_dim & 16) {
    const int c = a.k_dim >> 7, j = (a.k_dim & 127) >> 4;
    for (int i = tid; i < a.stages * a.tile; i += kThreads) {
      const int s = i / a.tile, t = i - s * a.tile;
      st_shared4(base + s * a.stage_bytes + (c * a.tile + t) * 128 + ((j ^ (t & 7)) << 4), 0, 0, 0, 0);
    }
    for (int i = tid; i < kTerms * N; i += kThreads) {
      const int n = i % N, term = i / N;
      st_shared4(base + a.off_q + ((term * a.k_chunks + c) * N + n) * 128 + ((j ^ (n & 7)) << 4), 0, 0, 0, 0);
    }
    fence_async();
  }
  pdl_wait();
  if (a.num_reqs && req >= *a.num_reqs) return;  // the whole cluster
  if (warp == kWorkers) {
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
  const uint32_t t_o = tmem + 2 * N;

  const int ntok = a.entries * static_cast<int>(a.rec_tokens.d);
  const int t0 = min(ntok, static_cast<int>(rank) * a.per_cta), t1 = min(ntok, t0 + a.per_cta);
  const int tiles = (t1 - t0 + a.tile - 1) / a.tile;
  const int64_t entry0 = qrow * a.entries;
  volatile int *fail = &s_fail;

  // Query heads of this group into e4m3 terms, a warp a head in turn of the workers.
  auto make_q = [&](int w) {
    const int vecs = a.k_dim >> 3;
    const T *q0 = static_cast<const T *>(a.q) + qrow * a.q_row;
    constexpr int kTurns = (N + kWorkers - 1) / kWorkers;
    constexpr int kBatch = kTurns < 3 ? kTurns : kTurns == 4 ? 4 : 3;
#pragma unroll 1
    for (int n0 = w; n0 < N; n0 += kWorkers * kBatch) {
      uint4 v[kBatch][3];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int n = n0 + kWorkers * b, h = static_cast<int>(hg) * N + n;
        const uint4 *src = reinterpret_cast<const uint4 *>(q0 + static_cast<int64_t>(kvh * a.group + h) * a.q_head);
#pragma unroll
        for (int i = 0; i < 3; ++i)
          v[b][i] = n < N && h < a.group && lane + 32 * i < vecs ? src[lane + 32 * i] : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int n = n0 + kWorkers * b;
        if (n >= N) break;
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < 3; ++i) {
          const T *e = reinterpret_cast<const T *>(&v[b][i]);
#pragma unroll
          for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(to_f32<T>(e[j])));
        }
        m = warp_max(m);
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
          const T *e = reinterpret_cast<const T *>(&v[b][i]);
          float x[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) x[j] = to_f32<T>(e[j]) * up;
          const int d = (lane + 32 * i) * 8;
          const uint32_t at = ((d >> 7) * N + n) * 128 + (((d & 127) >> 4 ^ (n & 7)) << 4) + (d & 15);
#pragma unroll
          for (int t = 0; t < kTerms; ++t) {
            uint32_t w0 = take_term<false>(x[0], x[1]);
            w0 |= take_term<false>(x[2], x[3]) << 16;
            uint32_t w1 = take_term<false>(x[4], x[5]);
            w1 |= take_term<false>(x[6], x[7]) << 16;
            asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(base + a.off_q + t * a.k_chunks * N * 128 + at),
                         "r"(w0), "r"(w1)
                         : "memory");
          }
        }
      }
    }
    fence_async();
    bar_arrive(b_q);
  };

  if (warp < kSoft) {
    // ---- softmax ---------------------------------------------------------------
    make_q(warp);
    bar_wait(b_q, 0, fail);  // the factors of all heads
    const int grp = warp >> 2, wl = warp & 3, c0 = grp * NC, gt = tid & 127;
    float l[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) l[c] = 0.f;
    const uint32_t lanes = static_cast<uint32_t>(wl * 32) << 16;
    const int tk = wl * 32 + lane;
    const uint32_t p_row = base + a.off_p + tk * 128;
    for (int i = 0; i < tiles; ++i) {
      const int s = i % a.stages, cn = min(a.tile, t1 - t0 - i * a.tile);
      bar_wait(b_full + 8 * s, (i / a.stages) & 1, fail);
      float ks = 0.f, lv = 0.f, iv = 1.f;
      bool use = false;
      if (tk < cn) {
        float2 meta;
        asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];"
                     : "=f"(meta.x), "=f"(meta.y)
                     : "r"(base + a.off_meta + (s * a.tile + tk) * 8)
                     : "memory");
        use = __float_as_int(meta.x) != 0x7fffffff;
        if (use) {
          ks = meta.x;
          const float v = fmaxf(meta.y, 0x1p-100f);
          lv = log2f(v);
          iv = 1.f / v;
        }
      }
      bar_wait(b_s + 8 * (i & 1), (i >> 1) & 1, fail);
      __syncwarp();
      tc_after();
      float x[NC];
#pragma unroll
      for (int c = 0; c < NC; c += 16)
        tc_ld16(tmem + lanes + (i & 1) * N + c0 + c, reinterpret_cast<uint32_t *>(x + c));
#pragma unroll
      for (int c = 0; c < NC; c += 16) tc_wait_ld16(reinterpret_cast<uint32_t *>(x + c));
      // scores in powers of two, the V scale in them
      float mine = -INFINITY;  // lane c keeps the maximum of column c
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        x[c] = use ? fmaf(x[c] * ks, s_qf[c0 + c], lv) : -INFINITY;
        const float m = warp_max(x[c]);
        if (lane == c) mine = m;
      }
      if (lane < NC) s_wmax[wl][c0 + lane] = mine;
      soft_sync(grp);
      bool moved = false;
      if (gt < NC) {
        const int c = c0 + gt;
        const float m = fmaxf(fmaxf(s_wmax[0][c], s_wmax[1][c]), fmaxf(s_wmax[2][c], s_wmax[3][c]));
        const float old = s_m[c];
        float f = 1.f;
        if (m > -INFINITY && !(m - old <= kSlack)) {
          f = old > -INFINITY ? ex2(old - (m - kTop)) : 0.f;
          s_m[c] = m - kTop;
          moved = true;
        }
        s_f[c] = f;
      }
      moved = soft_any(grp, moved);
      if (i > 0) {
        bar_wait(b_pv, (i - 1) & 1, fail);  // O and the probabilities' buffer are free
        __syncwarp();
        tc_after();
      }
      if (moved) {
#pragma unroll
        for (int c = 0; c < NC; ++c) l[c] *= s_f[c0 + c];
        if (i > 0) {
          for (int j = 0; j < a.v_tiles; ++j)
#pragma unroll
            for (int c = 0; c < NC; c += 16) {
              uint32_t o[16];
              const uint32_t at = t_o + lanes + j * N + c0 + c;
              tc_ld16(at, o);
              tc_wait_ld16(o);
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * s_f[c0 + c + e]);
              tc_st16(at, o);
            }
          tc_wait_st();
        }
      }
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const float m = s_m[c0 + c];
        x[c] = ex2(x[c] - (m > -INFINITY ? m : 0.f));
        l[c] = fmaf(x[c], iv, l[c]);
      }
      if (tk < ((cn + 31) & ~31)) {
#pragma unroll
        for (int t = 0; t < kTerms; ++t)
#pragma unroll
          for (int c = 0; c < NC; c += 16) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float *y = x + c + 4 * e;
              if (t + 1 < kTerms) {
                w[e] = take_term<false>(y[0], y[1]);
                w[e] |= take_term<false>(y[2], y[3]) << 16;
              } else {
                w[e] = take_term<true>(y[0], y[1]);
                w[e] |= take_term<true>(y[2], y[3]) << 16;
              }
            }
            st_shared4(p_row + (((t * N + c0 + c) >> 4 ^ (tk & 7)) << 4), w[0], w[1], w[2], w[3]);
          }
      }
      fence_async();
      tc_before();
      bar_arrive(b_p);
    }
    column_sums<NC, 16, NC / 2>(l, lane);
    soft_sync(grp);  // s_wmax is free
    if (NC == 32) {
      s_wmax[wl][c0 + lane] = l[0];
    } else if ((lane & 1) == 0) {
      s_wmax[wl][c0 + (lane >> 1)] = l[0];
    }
    soft_sync(grp);
    if (gt < NC) {
      const int c = c0 + gt;
      const float z = (s_wmax[0][c] + s_wmax[1][c]) + (s_wmax[2][c] + s_wmax[3][c]);
      s_l[c] = z;
      s_f[c] = z > 0.f || z != z ? 1.f / z : 0.f;
    }
    if (tiles > 0) {
      bar_wait(b_pv, (tiles - 1) & 1, fail);
      tc_after();
    }
    __syncwarp();
  } else if (warp < kWorkers) {
    // ---- gather ------------------------------------------------------------------
    const int pw = warp - kSoft, per = a.tile / kGather;
    const int kc = a.k_dim >> 4, cpr = kc + (a.latent ? 0 : a.v_dim >> 4);
    const int64_t k_at = static_cast<int64_t>(kvh) * a.k_dim;
    // from a K head's first byte to where its V head would begin 16 * kc bytes earlier
    const int64_t v_at = static_cast<int64_t>(a.kv_heads) * a.k_dim + static_cast<int64_t>(kvh) * a.v_dim - 16 * kc - k_at;
    const int seq = a.seq_lens ? a.seq_lens[req] : INT32_MAX;
    const float *scales = a.scales + req * a.scales_req + kvh;
    const char *hot = a.hot + req * a.hot_req;
    const int v_col = a.latent ? 0 : a.kv_heads;
    auto raw = [&](int i) {
      Raw r = {-1, -1, 0};
      const int t = t0 + i * a.tile + pw * per + lane;
      if (lane < per && i < tiles && t < t1) {
        r.entry = static_cast<int>(a.rec_tokens.div(t));
        r.slot = a.slots[entry0 + r.entry];
        r.sel = a.sel_block.d > 1 ? a.sel[entry0 / a.sel_block.d + a.sel_block.div(r.entry)]
                                  : a.sel[entry0 + r.entry];
      }
      return r;
    };
    auto token = [&](const Raw &r, int i) {
      Token k = {nullptr, 0.f, 0.f};
      if (r.slot == -1) return k;
      const int t = t0 + i * a.tile + pw * per + lane;
      const int sub = t - r.entry * static_cast<int>(a.rec_tokens.d);
      int64_t pos = r.sel;
      if (a.sel_block.d > 1 && pos >= 0)
        pos = pos * a.sel_block.d + (r.entry - a.sel_block.div(r.entry) * a.sel_block.d);
      pos = pos < 0 ? -1 : pos * a.rec_tokens.d + sub;
      const int64_t blk = pos <= INT32_MAX ? a.S.div(static_cast<uint32_t>(max(pos, int64_t(0)))) : pos / a.S.d;
      if (pos >= 0 && blk < a.scale_blocks) {
        if (pos >= seq) return k;
        if (r.slot >= 0 && r.slot <= a.B) {
          k.row = hot + r.slot * a.hot_row;
        } else if (r.slot > a.B && r.slot - a.B - 1 < a.res_rows) {
          k.row = a.resident + (static_cast<int64_t>(r.slot) - a.B - 1) * a.res_row;
        }
      }
      if (!k.row) {
        if (a.status) atomicOr(a.status, HISPARSE_ERR_RANGE);
        return k;
      }
      k.row += sub * a.row_bytes;
      const float *sc = scales + blk * a.columns;
      k.k = sc[0];
      k.v = sc[v_col];
      return k;
    };
    int issued = 0, signalled = 0;
    Token cur = token(raw(0), 0);
    Raw next = raw(1);
    // A tile's rows, `per` of them this warp's: 16-byte chunks in passes of a power of two of
    // columns, so that a lane's column, and with it all but the row, is fixed in a pass.
    auto issue = [&]() {
      const int i = issued, s = i % a.stages;
      const int cn = min(a.tile, t1 - t0 - i * a.tile);
      const Token ahead = token(next, i + 1);
      next = raw(i + 2);
      if (lane < per)
        asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(base + a.off_meta + (s * a.tile + pw * per + lane) * 8),
                     "f"(cur.row ? cur.k : __int_as_float(0x7fffffff)), "f"(cur.v)
                     : "memory");
      const uint32_t have = __ballot_sync(0xffffffffu, cur.row != nullptr);
      const uint64_t row = reinterpret_cast<uint64_t>(cur.row ? cur.row + k_at : a.hot);
      const int rows = min(per, max(0, ((cn + 31) & ~31) - pw * per));
      const uint32_t st = base + s * a.stage_bytes + pw * per * 128;
      for (int col0 = 0; col0 < cpr;) {
        const int left = cpr - col0, lw = left >= 32 ? 5 : 31 - __clz(left);
        const int tl = lane >> lw, col = col0 + (lane & ((1 << lw) - 1));
        const bool is_k = col < kc;
        const int j = is_k ? col : col - kc;
        const int64_t src_off = 16 * col + (is_k ? 0 : v_at);
        const uint32_t dst_off = st + ((is_k ? 0 : a.k_chunks) + (j >> 3)) * a.tile * 128;
#pragma unroll 4
        for (int tb = 0; tb < rows; tb += 32 >> lw) {
          const int t = tb + tl;
          const uint64_t src = __shfl_sync(0xffffffffu, row, t & 31);
          const bool ok = have >> (t & 31) & 1;
          if (t < rows)
            cp_async16(dst_off + t * 128 + ((j & 7 ^ (t & 7)) << 4),
                       reinterpret_cast<const char *>(src) + (ok ? src_off : 0), ok ? 16 : 0);
        }
        col0 += 1 << lw;
      }
      cp_commit();
      cur = ahead;
      ++issued;
    };
    auto signal = [&]() {
      cp_wait(issued - signalled - 1);
      fence_async();
      bar_arrive(b_full + 8 * (signalled % a.stages));
      ++signalled;
    };
    while (issued < min(tiles, a.stages)) issue();
    make_q(kSoft + pw);
    while (signalled < tiles) {
      bool go = false;
      if (issued < tiles) {
        const uint32_t bar = b_empty + 8 * (issued % a.stages), parity = (issued / a.stages - 1) & 1;
        if (issued == signalled) bar_wait(bar, parity, fail);
        go = issued == signalled || __all_sync(0xffffffffu, bar_test(bar, parity));
      }
      if (go) {
        issue();
      } else {
        signal();
      }
    }
  } else {
    // ---- products: the whole warp walks the loops, one lane issues -------------------
    const uint32_t d_qk = mma_desc(N, false, false);
    const uint32_t d_pv = mma_desc(N, false, true), d_pv5 = mma_desc(N, true, true);
    const int k_steps = (a.k_dim + 31) >> 5;
    const uint32_t elected = elect_one();
    const uint32_t q_desc = smem_desc(base + a.off_q), p_desc = smem_desc(base + a.off_p);
    bar_wait(b_q, 0, fail);
    auto scores = [&](int i) {
      const int s = i % a.stages;
      bar_wait(b_full + 8 * s, (i / a.stages) & 1, fail);
      __syncwarp();
      tc_after();
      const uint32_t d = tmem + (i & 1) * N;
      uint32_t q = q_desc;
      for (int t = 0; t < kTerms; ++t) {
        uint32_t k = smem_desc(base + s * a.stage_bytes);
        for (int left = k_steps; left > 0; left -= 4) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (e < left) mma_f8(d, k + 2 * e, q + 2 * e, d_qk, t > 0 || left < k_steps || e > 0, elected);
          k += a.tile * 8;
          q += N * 8;
        }
      }
      tc_commit(b_s + 8 * (i & 1), elected);
    };
    if (tiles > 0) scores(0);
    for (int i = 0; i < tiles; ++i) {
      if (i + 1 < tiles) scores(i + 1);
      const int s = i % a.stages, cn = min(a.tile, t1 - t0 - i * a.tile);
      bar_wait(b_p, i & 1, fail);
      __syncwarp();
      tc_after();
      uint32_t v = smem_desc(base + s * a.stage_bytes + (a.latent ? 0 : a.k_chunks * a.tile * 128));
      const int steps = (cn + 31) >> 5;
      for (int j = 0; j < a.v_tiles; ++j) {
        for (int k = 0; k < steps; ++k)
#pragma unroll
          for (int t = 0; t < kTerms; ++t)
            mma_f8(t_o + j * N, v + k * 256, p_desc + k * 256 + t * N / 16,
                   t + 1 < kTerms ? d_pv : d_pv5, i > 0 || k > 0 || t > 0, elected);
        v += a.tile * 8;
      }
      tc_commit(b_empty + 8 * s, elected);
      tc_commit(b_pv, elected);
    }
  }
  // ---- join ----------------------------------------------------------------------
  // Every product is done (the softmax warps' last wait), so the stages and Q hold
  // nothing any more.  A lone CTA writes its results from TMEM; in a cluster they take the
  // CTA's sums [N][v_dim] for the others to read.
  __syncwarp();
  __syncthreads();
  T *out = static_cast<T *>(a.out) + qrow * a.out_row;
  const int h0 = kvh * a.group + hg * N, heads = min(N, a.group - static_cast<int>(hg) * N);
  if (warp < kSoft) {
    tc_after();
    const int grp = warp >> 2, wl = warp & 3, c0 = grp * NC;
    const uint32_t lanes = static_cast<uint32_t>(wl * 32) << 16;
    for (int j = 0; j < a.v_tiles; ++j) {
      const int d = j * 128 + wl * 32 + lane;
      float o[NC];
      if (tiles > 0) {
#pragma unroll
        for (int c = 0; c < NC; c += 16)
          tc_ld16(t_o + lanes + j * N + c0 + c, reinterpret_cast<uint32_t *>(o + c));
#pragma unroll
        for (int c = 0; c < NC; c += 16) tc_wait_ld16(reinterpret_cast<uint32_t *>(o + c));
      } else {
#pragma unroll
        for (int c = 0; c < NC; ++c) o[c] = 0.f;
      }
      if (d >= a.v_dim) continue;
      if (a.cluster == 1) {
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          const float f = s_f[c0 + c];
          if (c0 + c < heads)
            out[static_cast<int64_t>(h0 + c0 + c) * a.out_head + d] = from_f32<T>(f != 0.f ? o[c] * f : 0.f);
        }
      } else {
#pragma unroll
        for (int c = 0; c < NC; ++c)
          asm volatile("st.shared.f32 [%0], %1;" ::"r"(base + ((c0 + c) * a.v_dim + d) * 4), "f"(o[c]) : "memory");
      }
    }
    __syncwarp();
    tc_before();
  }
  if (a.cluster == 1) {
    if (a.lse && tid < heads) {
      const float z = s_l[tid];
      a.lse[qrow * a.heads + h0 + tid] =
          z > 0.f || z != z ? (s_m[tid] + log2f(z)) * 0.6931471805599453f : -INFINITY;
    }
    __syncthreads();
  } else {
    __syncwarp();
    cluster_sync();
  }
  if (warp == kWorkers) {
    tc_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(a.tmem_cols));
  }
  if (tid == 0 && s_fail && a.status) atomicOr(a.status, HISPARSE_ERR_WAIT);
  if (a.cluster == 1) return;
  // Each CTA joins a share of the heads: weights 2^(m_r - max m) of the CTAs' sums.
  const int share = N / a.cluster, n0 = static_cast<int>(rank) * share;
  if (tid < share) {
    const int n = n0 + tid;
    float m = -INFINITY, z = 0.f;
#pragma unroll 4
    for (int r = 0; r < a.cluster; ++r) {
      const float x = ld_peer(peer(smem_u32(&s_m[n]), r));
      s_w[r * N + tid] = x;
      m = fmaxf(m, x);
    }
#pragma unroll 4
    for (int r = 0; r < a.cluster; ++r) {
      const float x = s_w[r * N + tid], y = ld_peer(peer(smem_u32(&s_l[n]), r));
      const float w = x > -INFINITY ? ex2(x - m) : 0.f;
      s_w[r * N + tid] = w;
      z = fmaf(w, y, z);
    }
    s_qf[tid] = z > 0.f || z != z ? 1.f / z : 0.f;
    if (a.lse && n < heads)
      a.lse[qrow * a.heads + h0 + n] = z > 0.f || z != z ? (m + log2f(z)) * 0.6931471805599453f : -INFINITY;
  }
  __syncthreads();
  for (uint32_t i = tid; i < share * a.quads.d; i += kThreads) {
    uint32_t nn, d;
    a.quads.divmod(i, nn, d);
    if (n0 + static_cast<int>(nn) >= heads) continue;
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    const uint32_t at = base + ((n0 + nn) * a.v_dim + 4 * d) * 4;
#pragma unroll 1
    for (int r0 = 0; r0 < a.cluster; r0 += 4) {
      float4 v[4];
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (r0 + r < a.cluster) v[r] = ld_peer4(peer(at, r0 + r));
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        if (r0 + r >= a.cluster) break;
        const float w = s_w[(r0 + r) * N + nn];
        acc[0] = fmaf(w, v[r].x, acc[0]);
        acc[1] = fmaf(w, v[r].y, acc[1]);
        acc[2] = fmaf(w, v[r].z, acc[2]);
        acc[3] = fmaf(w, v[r].w, acc[3]);
      }
    }
    const float inv = s_qf[nn];
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[e] = inv != 0.f ? acc[e] * inv : 0.f;
    store_vec<T, 4>(out + static_cast<int64_t>(h0 + n0 + nn) * a.out_head + 4 * d, acc);
  }
  cluster_sync();  // peers have read this CTA's shared memory
}

constexpr uint32_t kSmemSm = 233472;     // of an SM; a CTA takes its own and 1 KB more
constexpr uint32_t kSmemCta = 232448;    // at most, static and dynamic

// Tile, stages and offsets for N heads; false where they do not fit in `limit` bytes.
bool plan_smem(AttendArgs &a, int N, int terms, int tile, uint32_t limit, uint32_t &bytes) {
  a.tile = tile;
  a.k_chunks = (a.k_dim + 127) / 128;
  a.v_tiles = (a.v_dim + 127) / 128;
  a.v_chunks = a.latent ? 0 : a.v_tiles;
  // (a latent record whose V is wider than its K's chunks cannot be: v_dim <= k_dim)
  a.stage_bytes = static_cast<uint32_t>(a.k_chunks + a.v_chunks) * tile * 128;
  const uint32_t q = static_cast<uint32_t>(terms) * a.k_chunks * N * 128;
  const uint32_t p = tile * 128;
  // rows beyond a tile that the 128-row products read stay inside: Q and P follow
  const uint32_t over = (128 - tile) * 128;
  const uint32_t rest = q + p + (q + p < over ? over - q - p : 0);
  const uint32_t meta = tile * 8;
  const uint32_t sums = static_cast<uint32_t>(N) * a.v_dim * 4;
  const uint32_t fixed = rest + 1024;
  if (fixed + 2 * (a.stage_bytes + meta) > limit) return false;
  a.stages = std::min<uint32_t>(kMaxStages, (limit - fixed) / (a.stage_bytes + meta));
  a.off_q = a.stages * a.stage_bytes;
  a.off_p = a.off_q + q;
  a.off_meta = a.off_q + rest;
  bytes = std::max(a.off_meta + a.stages * meta, sums) + 1024;
  return bytes <= limit;
}

template <class T, int N>
int launch_attend(AttendArgs a, int64_t units, void *stream) {
  // TMEM: two score buffers and the sums, a power of two of columns.
  int cols = 32;
  a.v_tiles = (a.v_dim + 127) / 128;
  while (cols < 2 * N + a.v_tiles * N) cols *= 2;
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
  // CTAs that share an SM share its TMEM: each takes at least as large a part of
  // the SM's shared memory as of its TMEM, so that no CTA of a cluster waits for columns that
  // a CTA of another cluster holds.
  const uint32_t whole = kSmemCta - fixed.load();
  const uint32_t least = std::min(whole, kSmemSm / 512 * cols - 1024);
  uint32_t bytes = 0;
  bool ok = false;
  const uint32_t limits[2] = {std::max(least, kSmemSm / 2 - 1024 - fixed.load()), whole};
  for (int l = N == 16 ? 0 : 1; l < 2 && !ok; ++l)
    for (int tile = 128; tile >= 64 && !ok; tile -= 32)
      ok = plan_smem(a, N, Terms<T>::n, tile, limits[l], bytes);
  if (!ok) return HISPARSE_EBOUND;
  bytes = std::max(bytes, least);
  const int per_sm = 2 * (bytes + fixed.load() + 1024) <= kSmemSm ? 2 : 1;
  // Split the tokens while there are SMs without work and a CTA keeps 64 tokens or more.
  int c = 1;
  while (c < kMaxCluster && units * c * 2 <= 152 * per_sm && tokens >= static_cast<int64_t>(c) * 2 * 64) c *= 2;
  a.cluster = c;
  a.per_cta = static_cast<int>(((tokens + c - 1) / c + 31) / 32 * 32);
  if (units * c > 0x7fffffff) return HISPARSE_EBOUND;
  return launch_pdl(fn, dim3(static_cast<unsigned>(units * c)), dim3(Shape<N>::threads), bytes, stream, c, a);
}

template <class T>
int pick_attend(AttendArgs a, int64_t pairs, void *stream) {
  // Heads of a KV head that one CTA takes: enough for the group, at most 64 (32 with
  // three terms, whose probabilities fill a 128-byte row).
  int n = a.group <= 16 ? 16 : a.group <= 32 || Terms<T>::n == 3 ? 32 : 64;
  a.hgroups = (a.group + n - 1) / n;
  const int64_t units = pairs * a.hgroups;
  if (n == 16) return launch_attend<T, 16>(a, units, stream);
  if (n == 32) return launch_attend<T, 32>(a, units, stream);
  if constexpr (Terms<T>::n == 2) return launch_attend<T, 64>(a, units, stream);
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
  if (g->record_tokens > 65536 || g->heads > 65535 ||
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
  a.hot_req = g->hot_req_stride; a.hot_row = g->hot_row_stride;
  a.resident = static_cast<const char *>(g->resident);
  a.res_rows = g->resident ? g->resident_rows : 0;
  a.res_row = g->resident_row_stride;
  a.scales = g->scales; a.scales_req = g->scales_req_stride; a.scale_blocks = g->scale_blocks;
  a.seq_lens = g->d_seq_lens; a.num_reqs = g->d_num_reqs; a.status = g->d_status;
  a.row_bytes = row;
  a.quads = FastDiv(r.v_dim / 4);
  const int64_t pairs = static_cast<int64_t>(g->num_requests) * g->rows * r.kv_heads;
  return g->dtype == HISPARSE_BF16 ? pick_attend<__nv_bfloat16>(a, pairs, stream)
                                   : pick_attend<__half>(a, pairs, stream);
}

}  // extern "C"
