// rotary.cu -- rotary positions, and the packing of K and V into 8-bit records
// (hisparse_rotary and hisparse_pack of include/hisparse.h).
#include <algorithm>

#include "common.cuh"

namespace {

constexpr int kRotThreads = 256;
constexpr int kRotBatch = 2;  // units a thread reads before it writes the first

struct RotTensor {
  const void *x;
  void *y;
  int64_t xt, xh, yt, yh;
  FastDiv units;      // per head: half / V rotating ones, then those only copied
  uint32_t per_token; // units of a token: heads * units per head
};
struct RotArgs {
  RotTensor t[2];
  const int32_t *pos;
  const int64_t *turns;
  int64_t tokens;
  int32_t half, offset, rot;
  uint32_t rot_units;     // half / V
  uint32_t token_units;   // both tensors
  uint32_t unit_span;     // units of a token that one CTA does (grid.y parts)
  int32_t tokens_per_cta;
  int32_t interleaved;
  float amplitude, sign;
};

// ---------------------------------------------------------------------------
// rotary_kernel<T, V>: a unit is V pairs of one head (2V values), or V values
// outside the rotated part, which are only copied.  A CTA does the units of
// tokens_per_cta tokens (or a part of one token's, grid.y); the cosines and
// sines of its tokens are computed once into shared memory and serve every
// head of q and k.  The work is one read and one write of the tensors; the
// instructions per unit (two divisions by multiplication, 4 FMA a pair) stay
// below what hides under them.
// ---------------------------------------------------------------------------
template <class T, int V>
__global__ void __launch_bounds__(kRotThreads) rotary_kernel(const RotArgs a) {
  extern __shared__ float2 cs[];  // [tokens_per_cta][half]
  pdl_wait();
  pdl_launch();
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * a.tokens_per_cta;
  const int nt = static_cast<int>(min(static_cast<int64_t>(a.tokens_per_cta), a.tokens - t0));
  for (int i = threadIdx.x; i < nt * a.half; i += kRotThreads) {
    const int t = i / a.half, p = i - t * a.half;
    cs[i] = rotary_cos_sin(a.pos[t0 + t], a.turns[p], a.amplitude, a.sign);
  }
  __syncthreads();
  const uint32_t u0 = blockIdx.y * a.unit_span;
  const uint32_t span = min(a.unit_span, a.token_units - u0);
  const uint32_t total = span * nt;
  for (uint32_t base = threadIdx.x; base < total; base += kRotThreads * kRotBatch) {
    float lo[kRotBatch][V], hi[kRotBatch][V];
    T *out[kRotBatch];
    int cs_at[kRotBatch];  // -1: copied, -2: nothing
#pragma unroll
    for (int j = 0; j < kRotBatch; ++j) {
      uint32_t i = base + j * kRotThreads;
      cs_at[j] = -2;
      if (i >= total) continue;
      uint32_t tok = 0;
      if (nt > 1) {
        tok = i / span;
        i -= tok * span;
      }
      uint32_t u = u0 + i;
      const int which = u >= a.t[0].per_token;
      const RotTensor &x = a.t[which];
      if (which) u -= a.t[0].per_token;
      uint32_t head, unit;
      x.units.divmod(u, head, unit);
      const T *src = static_cast<const T *>(x.x) + (t0 + tok) * x.xt + head * x.xh;
      T *dst = static_cast<T *>(x.y) + (t0 + tok) * x.yt + head * x.yh;
      if (unit < a.rot_units) {
        const int p = unit * V;
        cs_at[j] = static_cast<int>(tok) * a.half + p;
        const int d = a.offset + (a.interleaved ? 2 * p : p);
        out[j] = dst + d;
        load_vec<T, V>(src + d, lo[j]);
        load_vec<T, V>(src + d + (a.interleaved ? V : a.half), hi[j]);
      } else {
        int d = static_cast<int>(unit - a.rot_units) * V;
        if (d >= a.offset) d += a.rot;
        cs_at[j] = -1;
        out[j] = dst + d;
        load_vec<T, V>(src + d, lo[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < kRotBatch; ++j) {
      if (cs_at[j] == -2) continue;
      if (cs_at[j] >= 0) {
        float na[V], nb[V];
        const float2 *c = cs + cs_at[j];
        if (a.interleaved) {
#pragma unroll
          for (int i = 0; i < 2 * V; i += 2) {  // pair i/2 of the 2V values [lo | hi]
            const float x = i < V ? lo[j][i % V] : hi[j][i % V];
            const float y = i + 1 < V ? lo[j][(i + 1) % V] : hi[j][(i + 1) % V];
            const float2 w = c[i / 2];
            const float r0 = x * w.x - y * w.y, r1 = x * w.y + y * w.x;
            if (i < V) na[i % V] = r0; else nb[i % V] = r0;
            if (i + 1 < V) na[(i + 1) % V] = r1; else nb[(i + 1) % V] = r1;
          }
        } else {
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const float2 w = c[i];
            na[i] = lo[j][i] * w.x - hi[j][i] * w.y;
            nb[i] = lo[j][i] * w.y + hi[j][i] * w.x;
          }
        }
        store_vec<T, V>(out[j], na);
        store_vec<T, V>(out[j] + (a.interleaved ? V : a.half), nb);
      } else {
        store_vec<T, V>(out[j], lo[j]);
      }
    }
  }
}

template <class T, int V>
int launch_rotary(const hisparse_rotary_args &g, bool copies, void *stream) {
  RotArgs a = {};
  a.pos = g.d_positions;
  a.turns = g.d_turns;
  a.tokens = g.tokens;
  a.rot = g.rot_dim;
  a.half = g.rot_dim / 2;
  a.offset = g.offset;
  a.rot_units = a.half / V;
  a.interleaved = (g.flags & HISPARSE_ROTARY_INTERLEAVED) != 0;
  a.amplitude = g.amplitude;
  a.sign = (g.flags & HISPARSE_ROTARY_INVERSE) ? -1.f : 1.f;
  for (int j = 0; j < 2; ++j) {
    const hisparse_rotary_tensor &t = g.t[j];
    if (t.heads == 0) {
      a.t[j].units = FastDiv(1);
      continue;
    }
    const uint32_t per = a.rot_units + (copies && t.x != t.y ? (t.dim - g.rot_dim) / V : 0);
    a.t[j] = {t.x, t.y, t.x_token_stride, t.x_head_stride, t.y_token_stride, t.y_head_stride,
              FastDiv(per), per * static_cast<uint32_t>(t.heads)};
    a.token_units += a.t[j].per_token;
  }
  // About two batches of units a thread; few tokens are split over several CTAs.
  const uint32_t want = kRotThreads * kRotBatch * 2;
  const int64_t all = static_cast<int64_t>(a.token_units) * g.tokens;
  const uint32_t share = static_cast<uint32_t>(
      std::min<int64_t>(want, std::max<int64_t>(kRotThreads, all / 304)));
  const int max_tokens = std::max(1, 32768 / (a.half * 8));  // 32 KB of cosines and sines
  a.tokens_per_cta = std::min<int64_t>(
      std::min<int64_t>(max_tokens, g.tokens), std::max<uint32_t>(1, share / a.token_units));
  uint32_t parts = (a.token_units + share - 1) / share;
  if (a.tokens_per_cta > 1) parts = 1;
  parts = std::min<uint32_t>(parts, 65535);
  a.unit_span = (a.token_units + parts - 1) / parts;
  parts = (a.token_units + a.unit_span - 1) / a.unit_span;
  const int64_t gx = (g.tokens + a.tokens_per_cta - 1) / a.tokens_per_cta;
  if (gx > 0x7fffffff) return HISPARSE_EBOUND;
  const size_t smem = static_cast<size_t>(a.tokens_per_cta) * a.half * sizeof(float2);
  return launch_pdl(rotary_kernel<T, V>, dim3(static_cast<unsigned>(gx), parts), dim3(kRotThreads),
                    smem, stream, 1, a);
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
  if (fits(8)) return launch_rotary<T, 8>(g, true, stream);
  if (fits(4)) return launch_rotary<T, 4>(g, true, stream);
  return launch_rotary<T, 1>(g, true, stream);
}

// ---------------------------------------------------------------------------
// Packing
// ---------------------------------------------------------------------------
constexpr int kPackThreads = 256;
constexpr int kPackTable = 48 * 1024;  // bytes of cosines and sines a CTA may hold

struct PackArgs {
  const int32_t *cu, *start, *reqs;
  const void *k, *v;
  int64_t tokens, kt, kh, vt, vh;
  float *scales;
  int64_t scales_req;
  int32_t n, max_len, R, scale_blocks, S;
  int32_t kv_heads, k_dim, v_dim, columns, cols_per_cta;
  float headroom;
  char *dst;
  int64_t dst_rows, dst_row, dst_req;
  const int32_t *blocks;
  int32_t max_blocks, page_tokens;
  int32_t rot, half, rot_offset, interleaved;
  float amplitude, sign;
  const int64_t *turns;
  uint32_t *status;
  int32_t chunk_k, chunk_v;  // tokens whose values a CTA's registers hold
};

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint2 e4m3x8(const float (&v)[8], float inv) {
  uint2 r;
  r.x = e4m3x2(v[0] * inv, v[1] * inv) | e4m3x2(v[2] * inv, v[3] * inv) << 16;
  r.y = e4m3x2(v[4] * inv, v[5] * inv) | e4m3x2(v[6] * inv, v[7] * inv) << 16;
  return r;
}
__device__ __forceinline__ float finite_max(float m, float x) {
  x = fabsf(x);
  return x < INFINITY ? fmaxf(m, x) : m;
}

// Unit u of a head: two runs of 8 values, at d0 and d1.  The first rot / 16 units are
// the rotating ones; the rest walk the values outside the rotated part.
struct Unit {
  int d0, d1, pair;  // pair: first of its 8 pairs, -1: not rotated
};
__device__ __forceinline__ Unit unit_at(const PackArgs &a, int u, bool rotates) {
  Unit r;
  const int ru = rotates ? a.rot >> 4 : 0;
  if (u < ru) {
    r.pair = u * 8;
    r.d0 = a.rot_offset + (a.interleaved ? 16 * u : 8 * u);
    r.d1 = r.d0 + (a.interleaved ? 8 : a.half);
  } else {
    r.pair = -1;
    const int e = (u - ru) * 16;
    r.d0 = rotates && e >= a.rot_offset ? e + a.rot : e;
    r.d1 = rotates && e + 8 >= a.rot_offset ? e + 8 + a.rot : e + 8;
  }
  return r;
}

// ---------------------------------------------------------------------------
// pack_kernel<T, PU>: one CTA per (block of the sequence, sequence, group of
// heads).  For each head it reads the block's tokens once into registers (PU units
// of 16 values a thread), rotates them, reduces their largest magnitude over
// the CTA, fixes the scale, and writes the e4m3 bytes.  Blocks with more
// tokens than the registers hold are walked twice in chunks (the second
// read comes from L2).  The cosines and sines of the tokens are computed once
// into shared memory and serve all heads of the CTA.  Bound by its bytes:
// 2 (or 4) read and 1 written a value.
// ---------------------------------------------------------------------------
template <class T, int PU>
__global__ void __launch_bounds__(kPackThreads) pack_kernel(const PackArgs a) {
  extern __shared__ float2 cs[];  // [chunk_k][half]
  __shared__ float s_max[kPackThreads / 32];
  __shared__ float s_scale;
  pdl_wait();
  pdl_launch();
  const int seq = blockIdx.y, tid = threadIdx.x;
  const int64_t cu0 = a.cu ? a.cu[seq] : static_cast<int64_t>(seq) * a.max_len;
  const int64_t len = (a.cu ? a.cu[seq + 1] : cu0 + a.max_len) - cu0;
  const int64_t p0 = a.start[seq];
  const int req = a.reqs ? a.reqs[seq] : seq;
  if (len <= 0) return;
  if (len > a.max_len || cu0 < 0 || cu0 + len > a.tokens || p0 < 0 || req < 0 || req >= a.R) {
    if (blockIdx.x == 0 && blockIdx.z == 0 && tid == 0 && a.status)
      atomicOr(a.status, HISPARSE_ERR_RANGE);
    return;
  }
  const int64_t blk = p0 / a.S + blockIdx.x;
  const int64_t first = max(blk * a.S, p0), end = min(blk * a.S + a.S, p0 + len);
  if (first >= end) return;
  if (blk >= a.scale_blocks) {
    if (tid == 0 && a.status) atomicOr(a.status, HISPARSE_ERR_RANGE);
    return;
  }
  const int nt = static_cast<int>(end - first);
  const int64_t tok0 = cu0 + (first - p0);  // the call's token of position `first`
  const bool has_first = first == blk * a.S, has_last = end == blk * a.S + a.S;

  const int col_end = min(a.columns, static_cast<int>(blockIdx.z + 1) * a.cols_per_cta);
  int table_at = -1;  // first token of the chunk whose table is in shared memory
  for (int col = blockIdx.z * a.cols_per_cta; col < col_end; ++col) {
    const bool is_k = col < a.kv_heads;
    const int head = is_k ? col : col - a.kv_heads;
    const int dim = is_k ? a.k_dim : a.v_dim;
    const int upt = dim >> 4;
    const int chunk = is_k ? a.chunk_k : a.chunk_v;
    const bool rot = is_k && a.rot > 0;
    const T *src = static_cast<const T *>(is_k ? a.k : a.v) + head * (is_k ? a.kh : a.vh);
    const int64_t ts = is_k ? a.kt : a.vt;
    const int64_t row_at = is_k ? static_cast<int64_t>(head) * a.k_dim
                                : static_cast<int64_t>(a.kv_heads) * a.k_dim +
                                      static_cast<int64_t>(head) * a.v_dim;
    float *scale_p = a.scales + req * a.scales_req + blk * a.columns + col;
    float x[PU][16];
    auto fetch = [&](int c0, int cn) {
      if (rot && table_at != c0) {
        __syncthreads();
        for (int i = tid; i < cn * a.half; i += kPackThreads) {
          const int t = i / a.half, p = i - t * a.half;
          cs[i] = rotary_cos_sin(static_cast<int32_t>(first + c0 + t), a.turns[p], a.amplitude,
                                 a.sign);
        }
        table_at = c0;
        __syncthreads();
      }
#pragma unroll
      for (int j = 0; j < PU; ++j) {
        const int i = tid + j * kPackThreads;
        if (i < cn * upt) {
          const int t = i / upt;
          const Unit u = unit_at(a, i - t * upt, rot);
          const T *p = src + (tok0 + c0 + t) * ts;
          load_vec<T, 8>(p + u.d0, *reinterpret_cast<float(*)[8]>(&x[j][0]));
          load_vec<T, 8>(p + u.d1, *reinterpret_cast<float(*)[8]>(&x[j][8]));
        }
      }
      if (!rot) return;
#pragma unroll
      for (int j = 0; j < PU; ++j) {
        const int i = tid + j * kPackThreads;
        if (i >= cn * upt) continue;
        const int t = i / upt;
        const Unit u = unit_at(a, i - t * upt, rot);
        if (u.pair < 0) continue;
        const float2 *c = cs + t * a.half + u.pair;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float2 w = c[e];
          float &p = a.interleaved ? x[j][2 * e] : x[j][e];
          float &q = a.interleaved ? x[j][2 * e + 1] : x[j][8 + e];
          const float np = p * w.x - q * w.y;
          q = p * w.y + q * w.x;
          p = np;
        }
      }
    };
    float m = 0.f;
    const float old = *scale_p;
    const bool fresh = has_first || old == 0.f;
    for (int c0 = 0; c0 < nt; c0 += chunk) {
      const int cn = min(chunk, nt - c0);
      if (!fresh && nt > chunk) break;  // the scale stands and the values are read below
      fetch(c0, cn);
#pragma unroll
      for (int j = 0; j < PU; ++j)
        if (tid + j * kPackThreads < cn * upt) {
#pragma unroll
          for (int e = 0; e < 16; ++e) m = finite_max(m, x[j][e]);
        }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    __syncthreads();  // every thread has read `old`, and s_max and s_scale are free
    if ((tid & 31) == 0) s_max[tid >> 5] = m;
    __syncthreads();
    if (tid == 0) {
      for (int w = 0; w < kPackThreads / 32; ++w) m = fmaxf(m, s_max[w]);
      float s = old;
      if (fresh && m > 0.f) {
        s = fmaxf(m * ((has_last ? 1.f : a.headroom) / 448.f), 0x1p-100f);
        *scale_p = s;
      }
      s_scale = s;
    }
    __syncthreads();
    const float inv = s_scale > 0.f ? 1.f / s_scale : 0.f;
    for (int c0 = 0; c0 < nt; c0 += chunk) {
      const int cn = min(chunk, nt - c0);
      if (nt > chunk) fetch(c0, cn);
#pragma unroll
      for (int j = 0; j < PU; ++j) {
        const int i = tid + j * kPackThreads;
        if (i >= cn * upt) continue;
        const int t = i / upt;
        const Unit u = unit_at(a, i - t * upt, rot);
        const int64_t pos = first + c0 + t;
        int64_t row = a.dst_req ? pos : tok0 + c0 + t;
        if (a.blocks) {
          const int64_t b = pos / a.page_tokens;
          const int32_t page = b < a.max_blocks
                                   ? a.blocks[static_cast<int64_t>(req) * a.max_blocks + b]
                                   : -1;
          if (page == -1) continue;  // no resident copy of this token
          row = static_cast<int64_t>(page) * a.page_tokens + pos % a.page_tokens;
        }
        if (row < 0 || row >= a.dst_rows) {
          if (a.status) atomicOr(a.status, HISPARSE_ERR_RANGE);
          continue;
        }
        char *out = a.dst + req * a.dst_req + row * a.dst_row + row_at;
        *reinterpret_cast<uint2 *>(out + u.d0) =
            e4m3x8(*reinterpret_cast<float(*)[8]>(&x[j][0]), inv);
        *reinterpret_cast<uint2 *>(out + u.d1) =
            e4m3x8(*reinterpret_cast<float(*)[8]>(&x[j][8]), inv);
      }
    }
  }
}

template <class T, int PU>
int launch_pack(PackArgs a, int span, int groups, void *stream) {
  const int cap = kPackThreads * PU;
  a.chunk_k = std::max(1, cap / (a.k_dim / 16));
  a.chunk_v = std::max(1, cap / (a.v_dim / 16));
  int table = 0;
  if (a.rot) {
    a.chunk_k = std::min(a.chunk_k, kPackTable / (a.half * 8));
    table = std::min({a.chunk_k, a.S, a.max_len}) * a.half * 8;
  }
  return launch_pdl(pack_kernel<T, PU>, dim3(span, a.n, groups), dim3(kPackThreads), table, stream,
                    1, a);
}

template <class T>
int pick_pack(const PackArgs &a, int span, int groups, void *stream) {
  const int tokens = std::min(a.S, a.max_len);
  const int units = tokens * std::max(a.k_dim, a.v_dim) / 16;
  if (units <= kPackThreads) return launch_pack<T, 1>(a, span, groups, stream);
  if (units <= kPackThreads * 2) return launch_pack<T, 2>(a, span, groups, stream);
  return launch_pack<T, 5>(a, span, groups, stream);
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
  a.k = g->k; a.v = g->v; a.tokens = g->tokens;
  a.kt = g->k_token_stride; a.kh = g->k_head_stride;
  a.vt = g->v_token_stride; a.vh = g->v_head_stride;
  a.scales = g->scales; a.scales_req = g->scales_req_stride;
  a.n = g->n; a.max_len = g->max_len; a.R = g->num_requests; a.scale_blocks = g->scale_blocks;
  a.S = r.block_tokens;
  a.kv_heads = r.kv_heads; a.k_dim = r.k_dim; a.v_dim = r.v_dim; a.columns = record_columns(r);
  a.headroom = g->headroom;
  a.dst = static_cast<char *>(g->dst);
  a.dst_rows = g->dst_rows; a.dst_row = g->dst_row_stride; a.dst_req = g->dst_req_stride;
  a.blocks = g->d_blocks; a.max_blocks = g->max_blocks; a.page_tokens = g->page_tokens;
  a.rot = g->rot_dim; a.half = g->rot_dim / 2; a.rot_offset = g->rot_offset;
  a.interleaved = (g->rot_flags & HISPARSE_ROTARY_INTERLEAVED) != 0;
  a.sign = (g->rot_flags & HISPARSE_ROTARY_INVERSE) ? -1.f : 1.f;
  a.amplitude = g->amplitude;
  a.turns = g->d_turns;
  a.status = g->d_status;
  // A sequence of max_len tokens touches at most this many blocks, whatever its start.
  const int64_t span = (static_cast<int64_t>(g->max_len) + a.S - 2) / a.S + 1;
  // Heads share the rotation's table: as many to a CTA as still leave some
  // CTAs for every SM.
  const int64_t ctas = span * g->n;
  a.cols_per_cta = static_cast<int>(std::min<int64_t>(
      a.columns, std::max<int64_t>(1, ctas * a.columns / (152 * 8))));
  const int groups = (a.columns + a.cols_per_cta - 1) / a.cols_per_cta;
  if (span > 0x7fffffff) return HISPARSE_EBOUND;
  switch (g->dtype) {
    case HISPARSE_BF16: return pick_pack<__nv_bfloat16>(a, static_cast<int>(span), groups, stream);
    case HISPARSE_F16: return pick_pack<__half>(a, static_cast<int>(span), groups, stream);
    default: return pick_pack<float>(a, static_cast<int>(span), groups, stream);
  }
}

}  // extern "C"
