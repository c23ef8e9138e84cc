// rotary.cu -- rotary positions, and the packing of K and V into 8-bit records
// (hisparse_rotary and hisparse_pack of include/hisparse.h).
#include <algorithm>

#include "common.cuh"

namespace {

// Cosines and sines of `tokens` tokens in shared memory, P pairs to a unit: laid out so that lanes
// whose units, then tokens, follow one another read 16 bytes each side by side.  (Pairs in their
// own order cost four times the reads.)
template <int P>
__device__ __forceinline__ int table_at(int pair, int token, int tokens, int units) {
  if (P == 1) return token * units + pair;
  const int u = pair / P, e = pair % P;
  return ((e >> 1) * tokens + token) * 2 * units + 2 * u + (e & 1);
}
template <int P>
__device__ __forceinline__ void table_read(const float2 *cs, int unit, int token, int tokens, int units,
                                           float2 (&w)[P]) {
  if constexpr (P == 1) {
    w[0] = cs[token * units + unit];
  } else {
#pragma unroll
    for (int e = 0; e < P; e += 2) {
      const float4 x = *reinterpret_cast<const float4 *>(cs + ((e >> 1) * tokens + token) * 2 * units + 2 * unit);
      w[e] = make_float2(x.x, x.y);
      w[e + 1] = make_float2(x.z, x.w);
    }
  }
}

constexpr int kRotThreads = 384;  // two CTAs of 80 registers a thread to an SM
constexpr int kRotTable = 48 * 1024;  // bytes of cosines and sines a CTA may hold

struct RotTensor {
  const void *x;
  void *y;
  int64_t xt, xh, yt, yh;
  FastDiv units;      // per head: the rotating ones, then those only copied
  uint32_t per_token; // units of a token: heads * units per head
};
struct RotArgs {
  RotTensor t[2];
  const int32_t *pos;
  const int64_t *turns;
  int64_t tokens;
  int32_t offset, rot;
  FastDiv half;
  uint32_t rot_units;   // of a head
  uint32_t token_units; // both tensors
  FastDiv span;         // units of a token that one CTA does (grid.y parts)
  int32_t abreast;      // tokens side by side in a CTA
  int32_t tokens_per_cta;
  float amplitude, sign;
};
// Vectors, pairs and tokens in flight of a thread: neighbours that turn together lie in one vector,
// halves that do in two.
template <class T, int V, bool I>
struct RotShape {
  static constexpr int vecs = I && V > 1 ? 1 : 2;
  static constexpr int pairs = I && V > 1 ? V / 2 : V;
  static constexpr int batch = V == 1 ? 4 : 128 / (vecs * V * static_cast<int>(sizeof(T))) > 8 ? 8 : 128 / (vecs * V * static_cast<int>(sizeof(T)));
};

// ---------------------------------------------------------------------------
// rotary_kernel<T, V, I>: a unit is V values of one head and their partners (for interleaved
// pairs these are among them), or V values outside the rotated part, which are only copied.
// A thread keeps its unit (which tensor, head and pairs) for `batch` tokens; all its loads are under
// way before the cosines and sines of the CTA's tokens are computed, once into shared
// memory for every head of q and k.  Bound by one read and one write of the tensors: 8191 tokens of
// 32 + 8 heads of 128 (168 MB) take 26 us, 6.4 TB/s; with the loads behind the sines 44 us.
// ---------------------------------------------------------------------------
template <class T, int V, bool I>
__global__ void __launch_bounds__(kRotThreads, 2) rotary_kernel(const RotArgs a) {
  using Sh = RotShape<T, V, I>;
  extern __shared__ __align__(16) float2 cs[];
  pdl_wait();
  pdl_launch();
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * a.tokens_per_cta;
  const int nt = static_cast<int>(min(static_cast<int64_t>(a.tokens_per_cta), a.tokens - t0));
  uint32_t lane_t, u;  // which of the tokens abreast; the unit of the token
  a.span.divmod(threadIdx.x, lane_t, u);
  u += blockIdx.y * a.span.d;
  const bool mine = lane_t < static_cast<uint32_t>(a.abreast) && u < a.token_units;
  const int which = u >= a.t[0].per_token;
  const RotTensor &x = a.t[which];
  if (which) u -= a.t[0].per_token;
  uint32_t head, unit;
  x.units.divmod(u, head, unit);
  const bool rotates = unit < a.rot_units;
  const int far = I ? 1 : a.rot / 2;
  int d;
  if (rotates) {
    d = a.offset + static_cast<int>(unit) * (I ? 2 * Sh::pairs : V);
  } else {
    d = static_cast<int>(unit - a.rot_units) * V;
    if (d >= a.offset) d += a.rot;
  }
  using Vt = Vec<T, V>;
  Vt lo[Sh::batch], hi[Sh::vecs == 2 ? Sh::batch : 1];
  const T *src = static_cast<const T *>(x.x) + (t0 + lane_t) * x.xt + head * x.xh + d;
  const int64_t xs = a.abreast * x.xt;
#pragma unroll
  for (int b = 0; b < Sh::batch; ++b)
    if (mine && lane_t + b * a.abreast < nt) {
      lo[b] = *reinterpret_cast<const Vt *>(src + b * xs);
      if (Sh::vecs == 2 && rotates) hi[Sh::vecs == 2 ? b : 0] = *reinterpret_cast<const Vt *>(src + b * xs + far);
    }
  const int half = a.half.d;
  for (uint32_t i = threadIdx.x; i < nt * half; i += blockDim.x) {
    uint32_t t, p;
    a.half.divmod(i, t, p);
    cs[table_at<Sh::pairs>(p, t, nt, a.rot_units)] =
        rotary_cos_sin(a.pos[t0 + t], a.turns[p], a.amplitude, a.sign);
  }
  __syncthreads();
  if (!mine) return;
  T *dst = static_cast<T *>(x.y) + (t0 + lane_t) * x.yt + head * x.yh + d;
  const int64_t ys = a.abreast * x.yt;
#pragma unroll
  for (int b = 0; b < Sh::batch; ++b) {
    const int t = lane_t + b * a.abreast;
    if (t >= nt) break;
    Vt na = lo[b];
    if (rotates) {
      float2 w[Sh::pairs];
      table_read<Sh::pairs>(cs, unit, t, nt, a.rot_units, w);
      if constexpr (V == 1) {
        Vt nb;
        const float p = to_f32<T>(lo[b].e), q = to_f32<T>(hi[b].e);
        na.e = from_f32<T>(p * w[0].x - q * w[0].y);
        nb.e = from_f32<T>(p * w[0].y + q * w[0].x);
        *reinterpret_cast<Vt *>(dst + b * ys + far) = nb;
      } else if constexpr (Sh::vecs == 1) {
#pragma unroll
        for (int i = 0; i < Sh::pairs; ++i) {
          const float2 p = lo[b].pair(i);
          na.set_pair(i, p.x * w[i].x - p.y * w[i].y, p.x * w[i].y + p.y * w[i].x);
        }
      } else {
        Vt nb;
#pragma unroll
        for (int i = 0; i < V; i += 2) {
          const float2 p = lo[b].pair(i / 2), q = hi[b].pair(i / 2);
          na.set_pair(i / 2, p.x * w[i].x - q.x * w[i].y, p.y * w[i + 1].x - q.y * w[i + 1].y);
          nb.set_pair(i / 2, p.x * w[i].y + q.x * w[i].x, p.y * w[i + 1].y + q.y * w[i + 1].x);
        }
        *reinterpret_cast<Vt *>(dst + b * ys + far) = nb;
      }
    }
    *reinterpret_cast<Vt *>(dst + b * ys) = na;
  }
}

template <class T, int V, bool I>
int launch_rotary(const hisparse_rotary_args &g, void *stream) {
  using Sh = RotShape<T, V, I>;
  RotArgs a = {};
  a.pos = g.d_positions;
  a.turns = g.d_turns;
  a.tokens = g.tokens;
  a.rot = g.rot_dim;
  a.half = FastDiv(g.rot_dim / 2);
  a.offset = g.offset;
  a.rot_units = g.rot_dim / 2 / Sh::pairs;
  a.amplitude = g.amplitude;
  a.sign = (g.flags & HISPARSE_ROTARY_INVERSE) ? -1.f : 1.f;
  for (int j = 0; j < 2; ++j) {
    const hisparse_rotary_tensor &t = g.t[j];
    if (t.heads == 0) {
      a.t[j].units = FastDiv(1);
      continue;
    }
    const uint32_t per = a.rot_units + (t.x != t.y ? (t.dim - g.rot_dim) / V : 0);
    a.t[j] = {t.x, t.y, t.x_token_stride, t.x_head_stride, t.y_token_stride, t.y_head_stride,
              FastDiv(per), per * static_cast<uint32_t>(t.heads)};
    a.token_units += a.t[j].per_token;
  }
  // A token's units over CTAs of nearly equal share; several tokens abreast where they are few.
  uint32_t parts = (a.token_units + kRotThreads - 1) / kRotThreads;
  const uint32_t span = (a.token_units + parts - 1) / parts;
  parts = (a.token_units + span - 1) / span;
  if (parts > 65535) return HISPARSE_EBOUND;
  a.span = FastDiv(span);
  const int64_t row = static_cast<int64_t>(g.rot_dim) / 2 * static_cast<int>(sizeof(float2));
  const int64_t fit = std::max<int64_t>(1, kRotTable / row);  // (rot_dim is at most 8192: 32 KB)
  a.abreast = static_cast<int>(std::min<int64_t>({kRotThreads / span, g.tokens, fit}));
  // Tokens in a row: enough to have `batch` loads in flight, unless SMs would be left without.
  const int64_t turns = std::max<int64_t>(1, std::min<int64_t>(Sh::batch, g.tokens * parts / (a.abreast * 304)));
  a.tokens_per_cta = static_cast<int>(std::min({turns * a.abreast, fit, g.tokens}));
  const int64_t gx = (g.tokens + a.tokens_per_cta - 1) / a.tokens_per_cta;
  if (gx > 0x7fffffff) return HISPARSE_EBOUND;
  const int threads = (a.abreast * static_cast<int>(span) + 31) / 32 * 32;
  return launch_pdl(rotary_kernel<T, V, I>, dim3(static_cast<unsigned>(gx), parts), dim3(threads),
                    a.tokens_per_cta * row, stream, 1, a);
}

template <class T>
int pick_rotary(const hisparse_rotary_args &g, void *stream) {
  // The widest vector that every address and extent allows: 16 bytes of 16-bit
  // values (two loads of 16 of 32-bit ones), then 4 values, else one.
  auto fits = [&](int v) {
    const size_t bytes = std::min<size_t>(16, v * sizeof(T));
    if (g.rot_dim / 2 % v || g.offset % v) return false;
    for (int j = 0; j < 2; ++j) {
      const hisparse_rotary_tensor &t = g.t[j];
      if (t.heads == 0) continue;
      if (reinterpret_cast<uintptr_t>(t.x) % bytes || reinterpret_cast<uintptr_t>(t.y) % bytes)
        return false;
      if (t.dim % v || t.x_token_stride % v || t.x_head_stride % v || t.y_token_stride % v ||
          t.y_head_stride % v)
        return false;
    }
    return true;
  };
  const bool i = (g.flags & HISPARSE_ROTARY_INTERLEAVED) != 0;
  if (fits(8)) return i ? launch_rotary<T, 8, true>(g, stream) : launch_rotary<T, 8, false>(g, stream);
  if (fits(4)) return i ? launch_rotary<T, 4, true>(g, stream) : launch_rotary<T, 4, false>(g, stream);
  return i ? launch_rotary<T, 1, true>(g, stream) : launch_rotary<T, 1, false>(g, stream);
}

// ---------------------------------------------------------------------------
// Packing
// ---------------------------------------------------------------------------
constexpr int kLow = 8;  // tokens of the low table of angles

struct PackSide {
  const void *x;
  int64_t ts, hs;  // elements between tokens, heads
  int32_t dim, row_at;
  FastDiv upt;     // units of 16 values in a token's head
  int32_t abreast; // tokens side by side in a team
};
struct PackArgs {
  PackSide side[2];
  const int32_t *cu, *start, *reqs;
  int64_t tokens;
  float *scales;
  int64_t scales_req;
  int32_t n, max_len, R, scale_blocks, S;
  int32_t kv_heads, columns;
  int32_t team;                // threads to a block's head: a power of two, or whole warps
  int32_t heads, blocks_cta;   // teams of a CTA: heads of each of its blocks
  int32_t k_groups;            // CTAs for the K heads
  float headroom;
  char *dst;
  int64_t dst_rows, dst_row, dst_req;
  const int32_t *pages;
  int32_t max_blocks, page_tokens;
  int32_t rot, rot_offset, interleaved;
  FastDiv half, by_S, by_team, by_heads;
  float amplitude, sign;
  const int64_t *turns;
  uint32_t *status;
};

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 turned(float2 a, float2 b) {  // a * b as complex numbers
  return make_float2(a.x * b.x - a.y * b.y, a.x * b.y + a.y * b.x);
}

// ---------------------------------------------------------------------------
// pack_kernel<T, PU, THREADS, WALK>: one CTA per (block of the sequence or several small ones,
// sequence, group of heads), a team of threads to a head of a block.  A unit is two runs of 8 values: partners of a rotation, or
// two stretches that are only packed.  A thread keeps its unit for PU tokens of the block:
// it reads them, turns them, holds them in 32 bits, and once the largest magnitude of the head is
// known writes their e4m3 bytes.  Blocks with more tokens than the CTA's registers hold are
// walked twice (WALK; the second read comes from L2).
// A token's angle is the sum of one of 8 low tokens' and one of the eighths': nt / 8 + 8 sines a pair
// in place of nt, and the product of the two costs a thread 4 multiplies a pair (one more rounding of
// 32 bits than the sine's own).
// Its bytes, 2 (or 4) read and 1 written a value, would allow half the time; what binds is the
// instructions (about 20 a value, 2.6 issued a cycle) and the wait of each CTA for its one round of
// loads.  8 ragged prompts of up to 4096 tokens, 8 + 8 heads of 128 (151 MB) take 44 us, 3.4 TB/s: with
// 4 units a thread and 3 CTAs of 256 threads to an SM (80 registers); 2 units and 2 CTAs of 512 took
// 53, 1 unit 79, 4 units and 6 CTAs of 128 49.  A sine for every token and pair, and the rotation
// done twice in place of held, took 105.
// ---------------------------------------------------------------------------
template <class T, int PU, int THREADS, bool WALK>
__global__ void __launch_bounds__(THREADS, 768 / THREADS) pack_kernel(const PackArgs a) {
  extern __shared__ __align__(16) float2 angles[];  // low: kLow tokens, then one for each kLow of a chunk
  __shared__ uint32_t s_max[20];
  pdl_wait();
  pdl_launch();
  const int seq = blockIdx.y;
  const int64_t cu0 = a.cu ? a.cu[seq] : static_cast<int64_t>(seq) * a.max_len;
  const int64_t len = (a.cu ? a.cu[seq + 1] : cu0 + a.max_len) - cu0;
  const int32_t p0 = a.start[seq];
  const int req = a.reqs ? a.reqs[seq] : seq;
  if (len <= 0) return;
  if (len > a.max_len || cu0 < 0 || cu0 + len > a.tokens || p0 < 0 || len > INT32_MAX - p0 || req < 0 ||
      req >= a.R) {
    if (blockIdx.x == 0 && blockIdx.z == 0 && threadIdx.x == 0 && a.status)
      atomicOr(a.status, HISPARSE_ERR_RANGE);
    return;
  }
  // The CTA's blocks and tokens, then this thread's team's.
  const uint32_t blk0 = a.by_S.div(p0) + blockIdx.x * a.blocks_cta;
  const int64_t stop = p0 + len;
  const int64_t cta_base = static_cast<int64_t>(blk0) * a.S;
  const int64_t cta_first = max(cta_base, static_cast<int64_t>(p0));
  if (cta_first >= stop) return;
  const int cta_tokens = static_cast<int>(min(cta_base + static_cast<int64_t>(a.blocks_cta) * a.S, stop) - cta_first);
  const int team = a.by_team.div(threadIdx.x), tid = threadIdx.x - team * a.team;
  const int group = a.by_heads.div(team);
  const bool is_v = static_cast<int>(blockIdx.z) >= a.k_groups;
  const int head = (is_v ? blockIdx.z - a.k_groups : blockIdx.z) * a.heads + (team - group * a.heads);
  const uint32_t blk = blk0 + group;
  const int64_t base = cta_base + static_cast<int64_t>(group) * a.S;
  const int32_t first = static_cast<int32_t>(min(max(base, cta_first), stop));
  int nt = group < a.blocks_cta ? static_cast<int>(min(base + a.S, stop) - first) : 0;
  const bool has_first = first == base, has_last = nt > 0 && first + static_cast<int64_t>(nt) == base + a.S;
  if (nt > 0 && blk >= static_cast<uint32_t>(a.scale_blocks)) {
    if (tid == 0 && a.status) atomicOr(a.status, HISPARSE_ERR_RANGE);
    nt = 0;
  }
  const int64_t tok0 = cu0 + (first - p0);  // the call's token of position `first`
  const int off = static_cast<int>(first - cta_first);

  // this thread's tokens and unit; a CTA has K heads or V heads
  const PackSide &sd = a.side[is_v];
  uint32_t lane_t, unit;
  sd.upt.divmod(tid, lane_t, unit);
  const bool mine = nt > 0 && head < a.kv_heads && lane_t < static_cast<uint32_t>(sd.abreast);
  const bool rot = !is_v && a.rot > 0;
  const int half = a.half.d, units = half >> 3;  // rotating units
  const bool turns = rot && unit < static_cast<uint32_t>(units);
  int d0, d1;
  if (turns) {
    d0 = a.rot_offset + (a.interleaved ? 16 : 8) * static_cast<int>(unit);
    d1 = d0 + (a.interleaved ? 8 : half);
  } else {
    const int skip = rot ? a.rot : 0;
    d0 = 8 * static_cast<int>(rot ? unit - units : unit);
    d1 = d0 + (sd.dim - skip) / 2;
    if (rot && d0 >= a.rot_offset) d0 += skip;
    if (rot && d1 >= a.rot_offset) d1 += skip;
  }
  const T *src = static_cast<const T *>(sd.x) + (tok0 + lane_t) * sd.ts + head * sd.hs;
  float *scale_p = a.scales + req * a.scales_req + static_cast<int64_t>(blk) * a.columns + (is_v ? a.kv_heads + head : head);
  const float old = mine ? *scale_p : 0.f;
  const int chunk = sd.abreast * PU, chunks = WALK ? (cta_tokens + chunk - 1) / chunk : 1;
  float2 *const low = angles, *const high = angles + kLow * half;
  using Vt = Vec<T, 8>;
  float m = 0.f, inv = 0.f;
  if (threadIdx.x < 20) s_max[threadIdx.x] = 0;

  for (int step = 0; step < (chunks == 1 ? 1 : 2 * chunks); ++step) {
    const int c0 = WALK ? (step < chunks ? step : step - chunks) * chunk : 0;
    Vt raw[PU][2];
#pragma unroll
    for (int j = 0; j < PU; ++j) {
      const int t = c0 + lane_t + j * sd.abreast;
      if (mine && t < nt) {
        const T *p = src + static_cast<int64_t>(c0 + j * sd.abreast) * sd.ts;
        raw[j][0] = *reinterpret_cast<const Vt *>(p + d0);
        raw[j][1] = *reinterpret_cast<const Vt *>(p + d1);
      } else {
        raw[j][0] = raw[j][1] = Vt{};
      }
    }
    const int n_table = WALK ? min(chunk, cta_tokens - c0) : cta_tokens;
    const int n_high = (n_table + kLow - 1) / kLow;
    if (rot) {
      if (step) __syncthreads();
      const int n_low = min(kLow, n_table);
      for (uint32_t i = threadIdx.x; i < (n_low + n_high) * half; i += blockDim.x) {
        uint32_t t, p;
        a.half.divmod(i, t, p);
        const bool lo = t < n_low;
        if (!lo) t -= n_low;
        const float2 w = rotary_cos_sin(lo ? static_cast<uint32_t>(cta_first) + c0 + t : t * kLow, a.turns[p], lo ? a.amplitude : 1.f, a.sign);
        (lo ? low : high)[table_at<8>(p, t, lo ? kLow : n_high, units)] = w;
      }
    }
    __syncthreads();
    float x[PU][16];
#pragma unroll
    for (int j = 0; j < PU; ++j) {
#pragma unroll
      for (int e = 0; e < 16; e += 2) {
        const float2 p = raw[j][e >> 3].pair((e & 7) / 2);
        x[j][e] = p.x;
        x[j][e + 1] = p.y;
      }
      const int t = off + lane_t + j * sd.abreast;
      // (threads left over beside the last unit have tokens past their chunk's table)
      if (turns && mine && t - off + c0 < nt) {
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          const float4 l = *reinterpret_cast<const float4 *>(low + ((e >> 1) * kLow + (t & (kLow - 1))) * 2 * units + 2 * unit);
          const float4 h = *reinterpret_cast<const float4 *>(high + ((e >> 1) * n_high + t / kLow) * 2 * units + 2 * unit);
          const float2 w[2] = {turned(make_float2(l.x, l.y), make_float2(h.x, h.y)),
                               turned(make_float2(l.z, l.w), make_float2(h.z, h.w))};
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float &p = a.interleaved ? x[j][2 * (e + i)] : x[j][e + i];
            float &q = a.interleaved ? x[j][2 * (e + i) + 1] : x[j][8 + e + i];
            const float np = p * w[i].x - q * w[i].y;
            q = p * w[i].y + q * w[i].x;
            p = np;
          }
        }
      }
    }
    if (step < chunks) {
      // The largest finite magnitude.  fmaxf leaves NaN out; infinities are rare, and looked for only
      // where the plain maximum is one.
      float top = 0.f;
#pragma unroll
      for (int j = 0; j < PU; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) top = fmaxf(top, fabsf(x[j][e]));
      if (top == INFINITY) {
        top = 0.f;
#pragma unroll
        for (int j = 0; j < PU; ++j)
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float y = fabsf(x[j][e]);
            top = fmaxf(top, y < INFINITY ? y : 0.f);
          }
      }
      m = fmaxf(m, top);
    }
    if (step == chunks - 1) {
      // Magnitudes are not negative: their bits compare as they do.
      uint32_t w = __float_as_uint(m);
      if (a.team >= 32) {
        w = __reduce_max_sync(0xffffffffu, w);
        if ((threadIdx.x & 31) == 0) atomicMax(&s_max[team], w);
        __syncthreads();  // (every thread has read `old`)
        w = s_max[team];
      } else {
        for (int o = a.team >> 1; o; o >>= 1) w = max(w, __shfl_xor_sync(0xffffffffu, w, o));
        __syncwarp();
      }
      m = __uint_as_float(w);
      float s = old;
      if ((has_first || old == 0.f) && m > 0.f) {
        s = fmaxf(m * ((has_last ? 1.f : a.headroom) / 448.f), 0x1p-100f);
        if (tid == 0 && mine) *scale_p = s;
      }
      // (without a scale all finite values are 0, and the others stay what they are)
      inv = s > 0.f ? 1.f / s : s == 0.f ? 1.f : 0.f;
    }
    if (step < chunks && chunks > 1) continue;
#pragma unroll
    for (int j = 0; j < PU; ++j) {
      const int t = c0 + lane_t + j * sd.abreast;
      if (!mine || t >= nt) break;
      int64_t row = a.dst_req ? first + t : tok0 + t;
      if (a.pages) {
        const uint32_t pos = first + t, b = pos / a.page_tokens;
        const int32_t page = b < static_cast<uint32_t>(a.max_blocks) ? a.pages[static_cast<int64_t>(req) * a.max_blocks + b] : -1;
        if (page == -1) continue;  // no resident copy of this token
        row = static_cast<int64_t>(page) * a.page_tokens + (pos - b * a.page_tokens);
      }
      if (row < 0 || row >= a.dst_rows) {
        if (a.status) atomicOr(a.status, HISPARSE_ERR_RANGE);
        continue;
      }
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        w[e] = e4m3x2(x[j][4 * e] * inv, x[j][4 * e + 1] * inv) | e4m3x2(x[j][4 * e + 2] * inv, x[j][4 * e + 3] * inv) << 16;
      char *out = a.dst + req * a.dst_req + row * a.dst_row + sd.row_at + head * sd.dim;
      *reinterpret_cast<uint2 *>(out + d0) = make_uint2(w[0], w[1]);
      *reinterpret_cast<uint2 *>(out + d1) = make_uint2(w[2], w[3]);
    }
  }
}

template <class T, int PU, int THREADS, bool WALK>
int launch_pack(PackArgs a, int span, int most, void *stream) {
  // Tokens abreast so that a team holds a block's tokens, within a CTA; then heads to a CTA (they
  // share the angles), then blocks, while there are CTAs for every SM.
  const int sides = a.columns > a.kv_heads ? 2 : 1;
  const int upt = std::max(a.side[0].dim, sides > 1 ? a.side[1].dim : 0) / 16;
  const int want = upt * ((most + PU - 1) / PU);
  a.team = std::min(THREADS, (want + 31) / 32 * 32);
  if (want < 32)
    for (a.team = 1; a.team < want;) a.team *= 2;
  const int64_t all = static_cast<int64_t>(span) * a.n * a.columns;
  const int teams = static_cast<int>(std::min<int64_t>(THREADS / a.team, std::max<int64_t>(1, all / 304)));
  a.heads = std::min(teams, a.kv_heads);
  a.blocks_cta = WALK ? 1 : std::min(teams / a.heads, span);
  for (int i = 0; i < sides; ++i) {
    a.side[i].upt = FastDiv(a.side[i].dim / 16);
    a.side[i].abreast = std::min(a.team / (a.side[i].dim / 16), most);
  }
  const int tokens = a.blocks_cta > 1 ? std::min(a.blocks_cta * a.S, a.max_len) : std::min(a.side[0].abreast * PU, most);
  const int table = a.rot ? (kLow + (tokens + kLow - 1) / kLow) * (a.rot / 2) * static_cast<int>(sizeof(float2)) : 0;
  a.by_S = FastDiv(a.S);
  a.by_team = FastDiv(a.team);
  a.by_heads = FastDiv(a.heads);
  a.k_groups = (a.kv_heads + a.heads - 1) / a.heads;
  return launch_pdl(pack_kernel<T, PU, THREADS, WALK>, dim3((span + a.blocks_cta - 1) / a.blocks_cta, a.n, a.k_groups * sides),
                    dim3((a.team * a.heads * a.blocks_cta + 31) / 32 * 32), table, stream, 1, a);
}

template <class T>
int pick_pack(const PackArgs &a, int span, void *stream) {
  // Four units a thread where there is work for every SM, one where there is not (or a block has no
  // four tokens); a CTA of 640 threads where 256 would have to walk a block twice.
  const int most = std::min(a.S, a.max_len);
  const int upt = std::max(a.side[0].dim, a.side[1].dim) / 16;
  const int64_t all = static_cast<int64_t>(span) * a.n * a.columns * upt * most;
  if (upt * most <= 256 && (most < 4 || all <= 304 * 256)) return launch_pack<T, 1, 256, false>(a, span, most, stream);
  if (upt * ((most + 3) / 4) <= 256) return launch_pack<T, 4, 256, false>(a, span, most, stream);
  return launch_pack<T, 4, 640, true>(a, span, most, stream);
}

}  // namespace

extern "C" {

int hisparse_rotary(const hisparse_rotary_args *g, void *stream) {
  if (!g || g->tokens < 0 || g->rot_dim < 2 || g->rot_dim % 2 || g->offset < 0) return HISPARSE_EINVAL;
  if (g->dtype < HISPARSE_BF16 || g->dtype > HISPARSE_F32) return HISPARSE_EINVAL;
  if (g->flags & ~(HISPARSE_ROTARY_INTERLEAVED | HISPARSE_ROTARY_INVERSE)) return HISPARSE_EINVAL;
  if (g->t[0].heads < 0 || g->t[1].heads < 0) return HISPARSE_EINVAL;
  if (g->rot_dim > 8192) return HISPARSE_EBOUND;
  const int size = g->dtype == HISPARSE_F32 ? 4 : 2;
  int64_t units = 0;
  for (int j = 0; j < 2; ++j) {
    const hisparse_rotary_tensor &t = g->t[j];
    if (t.heads == 0) continue;
    if (t.dim < 1 || g->offset > t.dim - g->rot_dim) return HISPARSE_EINVAL;
    units += static_cast<int64_t>(t.heads) * t.dim;
    if (g->tokens == 0) continue;
    if (!t.x || !t.y || reinterpret_cast<uintptr_t>(t.x) % size ||
        reinterpret_cast<uintptr_t>(t.y) % size)
      return HISPARSE_EINVAL;
    if (t.x == t.y && (t.x_token_stride != t.y_token_stride || t.x_head_stride != t.y_head_stride))
      return HISPARSE_EINVAL;
  }
  if (units > 0x3fffffff) return HISPARSE_EBOUND;
  if (g->tokens == 0 || units == 0) return HISPARSE_OK;
  if (!g->d_positions || !g->d_turns) return HISPARSE_EINVAL;
  switch (g->dtype) {
    case HISPARSE_BF16: return pick_rotary<__nv_bfloat16>(*g, stream);
    case HISPARSE_F16: return pick_rotary<__half>(*g, stream);
    default: return pick_rotary<float>(*g, stream);
  }
}

int hisparse_pack(const hisparse_pack_args *g, void *stream) {
  if (!g) return HISPARSE_EINVAL;
  const hisparse_records &r = g->rec;
  if (const int rc = records_ok(r)) return rc;
  if (g->dtype < HISPARSE_BF16 || g->dtype > HISPARSE_F32) return HISPARSE_EINVAL;
  if (g->n < 0 || g->max_len < 1 || g->num_requests < 1 || g->scale_blocks < 1 || g->tokens < 0)
    return HISPARSE_EINVAL;
  if (!(g->headroom >= 1.f)) return HISPARSE_EINVAL;
  if (g->n == 0 || g->tokens == 0) return HISPARSE_OK;
  if (g->n > 65535) return HISPARSE_EBOUND;
  if (!g->d_start || !g->k || !g->scales || !g->dst || (!r.latent && !g->v)) return HISPARSE_EINVAL;
  if (!g->d_cu_lens && g->tokens < static_cast<int64_t>(g->n) * g->max_len) return HISPARSE_EINVAL;
  if (!aligned16(g->k) || g->k_token_stride % 8 || g->k_head_stride % 8) return HISPARSE_EINVAL;
  if (!r.latent && (!aligned16(g->v) || g->v_token_stride % 8 || g->v_head_stride % 8))
    return HISPARSE_EINVAL;
  if (!aligned16(g->dst) || g->dst_row_stride % 16 || g->dst_req_stride % 16 ||
      g->dst_row_stride < record_row_bytes(r) || g->dst_rows < 0 || g->dst_req_stride < 0)
    return HISPARSE_EINVAL;
  if (g->d_blocks && (g->max_blocks < 1 || g->page_tokens < 1 || g->dst_req_stride))
    return HISPARSE_EINVAL;
  if (!g->d_blocks && !g->dst_req_stride && g->dst_rows < g->tokens) return HISPARSE_EINVAL;
  if (g->rot_dim) {
    if (g->rot_dim < 0 || g->rot_dim % 16 || g->rot_offset < 0 || g->rot_offset % 8 ||
        g->rot_offset > r.k_dim - g->rot_dim || !g->d_turns ||
        (g->rot_flags & ~(HISPARSE_ROTARY_INTERLEAVED | HISPARSE_ROTARY_INVERSE)))
      return HISPARSE_EINVAL;
  }
  PackArgs a = {};
  a.cu = g->d_cu_lens; a.start = g->d_start; a.reqs = g->d_reqs;
  a.tokens = g->tokens;
  a.side[0] = {g->k, g->k_token_stride, g->k_head_stride, r.k_dim, 0};
  if (!r.latent)
    a.side[1] = {g->v, g->v_token_stride, g->v_head_stride, r.v_dim, r.kv_heads * r.k_dim};
  a.scales = g->scales; a.scales_req = g->scales_req_stride;
  a.n = g->n; a.max_len = g->max_len; a.R = g->num_requests; a.scale_blocks = g->scale_blocks;
  a.S = r.block_tokens;
  a.kv_heads = r.kv_heads; a.columns = record_columns(r);
  a.headroom = g->headroom;
  a.dst = static_cast<char *>(g->dst);
  a.dst_rows = g->dst_rows; a.dst_row = g->dst_row_stride; a.dst_req = g->dst_req_stride;
  a.pages = g->d_blocks; a.max_blocks = g->max_blocks; a.page_tokens = g->page_tokens;
  a.rot = g->rot_dim; a.half = FastDiv(std::max(1, g->rot_dim / 2)); a.rot_offset = g->rot_offset;
  a.interleaved = (g->rot_flags & HISPARSE_ROTARY_INTERLEAVED) != 0;
  a.sign = (g->rot_flags & HISPARSE_ROTARY_INVERSE) ? -1.f : 1.f;
  a.amplitude = g->amplitude;
  a.turns = g->d_turns;
  a.status = g->d_status;
  // A sequence of max_len tokens touches at most this many blocks, whatever its start.
  const int64_t span = (static_cast<int64_t>(g->max_len) + a.S - 2) / a.S + 1;
  if (span > 0x7fffffff) return HISPARSE_EBOUND;
  switch (g->dtype) {
    case HISPARSE_BF16: return pick_pack<__nv_bfloat16>(a, static_cast<int>(span), stream);
    case HISPARSE_F16: return pick_pack<__half>(a, static_cast<int>(span), stream);
    default: return pick_pack<float>(a, static_cast<int>(span), stream);
  }
}

}  // extern "C"
