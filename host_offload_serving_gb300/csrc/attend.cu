// attend.cu -- sparse attention over 8-bit records (hisparse_attend of include/hisparse.h).
#include <cuda_fp8.h>

#include <algorithm>

#include "common.cuh"

namespace {

struct AttendArgs {
  int32_t R, rows, entries, heads, kv_heads, k_dim, v_dim, latent, S, B;
  int32_t rec_tokens, sel_block, columns;
  float scale;
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
};

struct Token {
  const char *row;  // NULL: nothing to read
  int64_t block;
};
// Token i of a query row: entry i / rec_tokens, its sub-th token.
__device__ __forceinline__ Token token_at(const AttendArgs &a, int req, int64_t entry0, int64_t i) {
  const int64_t e = i / a.rec_tokens, sub = i - e * a.rec_tokens;
  const int32_t slot = a.slots[entry0 + e];
  if (slot == -1) return {nullptr, 0};
  int64_t pos;
  if (a.sel_block > 1) {
    const int64_t j = entry0 + e;  // entries is a multiple of sel_block
    const int32_t b = a.sel[j / a.sel_block];
    pos = b < 0 ? -1 : static_cast<int64_t>(b) * a.sel_block + j % a.sel_block;
  } else {
    pos = a.sel[entry0 + e];
  }
  pos = pos < 0 ? -1 : pos * a.rec_tokens + sub;
  const int64_t block = pos / a.S;
  const char *row = nullptr;
  if (pos >= 0 && block < a.scale_blocks) {
    if (a.seq_lens && pos >= a.seq_lens[req]) return {nullptr, 0};
    if (slot >= 0 && slot <= a.B) {
      row = a.hot + req * a.hot_req + slot * a.hot_row;
    } else if (slot > a.B && a.resident && slot - a.B - 1 < a.res_rows) {
      row = a.resident + (static_cast<int64_t>(slot) - a.B - 1) * a.res_row;
    }
  }
  if (!row) {
    if (a.status) atomicOr(a.status, HISPARSE_ERR_RANGE);
    return {nullptr, 0};
  }
  return {row + sub * a.row_bytes, block};
}

__device__ __forceinline__ float e4m3(const char *p) {
  __nv_fp8_e4m3 x;
  x.__x = static_cast<__nv_fp8_storage_t>(*p);
  return static_cast<float>(x);
}

// One CTA per (query row, head); chunks of kChunk tokens with a running maximum and sum.
constexpr int kThreads = 256, kChunk = 64;

template <class T>
__global__ void __launch_bounds__(kThreads) attend_kernel(const AttendArgs a) {
  __shared__ float q[640], s[kChunk];
  __shared__ Token tok[kChunk];
  pdl_wait();
  pdl_launch();
  const int64_t qrow = blockIdx.x;
  const int req = static_cast<int>(qrow / a.rows), head = blockIdx.y;
  if (a.num_reqs && req >= *a.num_reqs) return;
  const int kvh = head / (a.heads / a.kv_heads);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const T *qp = static_cast<const T *>(a.q) + qrow * a.q_row + head * a.q_head;
  for (int d = tid; d < a.k_dim; d += kThreads) q[d] = to_f32<T>(qp[d]);
  const int64_t n = static_cast<int64_t>(a.entries) * a.rec_tokens;
  const int64_t k_at = static_cast<int64_t>(kvh) * a.k_dim;
  const int64_t v_at = a.latent ? k_at
                                : static_cast<int64_t>(a.kv_heads) * a.k_dim +
                                      static_cast<int64_t>(kvh) * a.v_dim;
  const int v_col = a.latent ? kvh : a.kv_heads + kvh;
  float m = -INFINITY, l = 0.f, o[2] = {0.f, 0.f};
  for (int64_t c0 = 0; c0 < n; c0 += kChunk) {
    const int cn = static_cast<int>(min(static_cast<int64_t>(kChunk), n - c0));
    __syncthreads();
    if (tid < cn) tok[tid] = token_at(a, req, qrow * a.entries, c0 + tid);
    __syncthreads();
    for (int j = warp; j < cn; j += kThreads / 32) {
      const Token t = tok[j];
      float x = 0.f;
      if (t.row)
        for (int d = lane; d < a.k_dim; d += 32) x += q[d] * e4m3(t.row + k_at + d);
#pragma unroll
      for (int w = 16; w; w >>= 1) x += __shfl_xor_sync(0xffffffffu, x, w);
      if (lane == 0)
        s[j] = t.row ? x * a.scale * a.scales[req * a.scales_req + t.block * a.columns + kvh]
                     : -INFINITY;
    }
    __syncthreads();
    float mc = m;
    for (int j = 0; j < cn; ++j) mc = fmaxf(mc, s[j]);
    if (mc == -INFINITY) continue;
    const float f = __expf(m - mc);
    l *= f;
    o[0] *= f;
    o[1] *= f;
    m = mc;
    for (int j = 0; j < cn; ++j) {
      if (!tok[j].row) continue;
      const float p = __expf(s[j] - m);
      l += p;
      const float pv = p * a.scales[req * a.scales_req + tok[j].block * a.columns + v_col];
      if (tid < a.v_dim) o[0] += pv * e4m3(tok[j].row + v_at + tid);
      if (tid + kThreads < a.v_dim) o[1] += pv * e4m3(tok[j].row + v_at + tid + kThreads);
    }
  }
  T *op = static_cast<T *>(a.out) + qrow * a.out_row + head * a.out_head;
  const float inv = l > 0.f ? 1.f / l : 0.f;
  if (tid < a.v_dim) op[tid] = from_f32<T>(l > 0.f ? o[0] * inv : 0.f);
  if (tid + kThreads < a.v_dim) op[tid + kThreads] = from_f32<T>(l > 0.f ? o[1] * inv : 0.f);
  if (a.lse && tid == 0) a.lse[qrow * a.heads + head] = l > 0.f ? m + logf(l) : -INFINITY;
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
  a.R = g->num_requests; a.rows = g->rows; a.entries = g->entries; a.heads = g->heads;
  a.kv_heads = r.kv_heads; a.k_dim = r.k_dim; a.v_dim = r.v_dim; a.latent = r.latent;
  a.S = r.block_tokens; a.B = g->buffer_slots; a.rec_tokens = g->record_tokens;
  a.sel_block = g->sel_block_tokens; a.columns = record_columns(r);
  a.scale = g->softmax_scale;
  a.q = g->q; a.q_row = g->q_row_stride; a.q_head = g->q_head_stride;
  a.out = g->out; a.out_row = g->out_row_stride; a.out_head = g->out_head_stride;
  a.lse = g->lse; a.sel = g->d_sel; a.slots = g->d_slots;
  a.hot = static_cast<const char *>(g->hot);
  a.hot_req = g->hot_req_stride; a.hot_row = g->hot_row_stride;
  a.resident = static_cast<const char *>(g->resident);
  a.res_rows = g->resident_rows; a.res_row = g->resident_row_stride;
  a.scales = g->scales; a.scales_req = g->scales_req_stride; a.scale_blocks = g->scale_blocks;
  a.seq_lens = g->d_seq_lens; a.num_reqs = g->d_num_reqs; a.status = g->d_status;
  a.row_bytes = row;
  const dim3 grid(static_cast<unsigned>(a.R) * a.rows, a.heads);
  return g->dtype == HISPARSE_BF16
             ? launch_pdl(attend_kernel<__nv_bfloat16>, grid, dim3(kThreads), 0, stream, 1, a)
             : launch_pdl(attend_kernel<__half>, grid, dim3(kThreads), 0, stream, 1, a);
}

}  // extern "C"
