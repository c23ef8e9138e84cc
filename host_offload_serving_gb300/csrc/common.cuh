// common.cuh -- what the translation units of the library share: the error of
// the last failed CUDA call, and small helpers.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "hisparse.h"

extern thread_local int g_last_cuda_error;

inline int cuda_fail(cudaError_t e) {
  g_last_cuda_error = static_cast<int>(e);
  return HISPARSE_ECUDA;
}
#define HS_CUDA(call)                              \
  do {                                             \
    cudaError_t e_ = (call);                       \
    if (e_ != cudaSuccess) return cuda_fail(e_);   \
  } while (0)

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// The sizes of a record that every call accepts.
inline int records_ok(const hisparse_records &r) {
  if (r.kv_heads < 1 || r.k_dim < 16 || r.v_dim < 16 || r.block_tokens < 1) return HISPARSE_EINVAL;
  if (r.k_dim % 16 || r.v_dim % 16 || (r.latent != 0 && r.latent != 1)) return HISPARSE_EINVAL;
  if (r.latent && r.v_dim > r.k_dim) return HISPARSE_EINVAL;
  if (r.k_dim > 640 || r.v_dim > 512 || r.block_tokens > 4096 || r.kv_heads > 1024)
    return HISPARSE_EBOUND;
  return HISPARSE_OK;
}
inline int64_t record_row_bytes(const hisparse_records &r) {
  return static_cast<int64_t>(r.kv_heads) * (r.k_dim + (r.latent ? 0 : r.v_dim));
}
inline int record_columns(const hisparse_records &r) { return r.kv_heads * (r.latent ? 1 : 2); }

// Launch on `stream` with programmatic dependent launch: the grid may be set up
// while the previous kernel of the stream finishes.  Every kernel launched so
// begins with griddepcontrol.wait and reads and writes no memory before it.
template <class... P, class... A>
inline int launch_pdl(void (*fn)(P...), dim3 grid, dim3 block, size_t smem, void *stream,
                      int cluster, A... args) {
  cudaLaunchConfig_t lc = {};
  lc.gridDim = grid;
  lc.blockDim = block;
  lc.dynamicSmemBytes = smem;
  lc.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = at;
  lc.numAttrs = 1;
  if (cluster > 1) {
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = cluster;
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    lc.numAttrs = 2;
  }
  const cudaError_t e = cudaLaunchKernelEx(&lc, fn, static_cast<P>(args)...);
  return e == cudaSuccess ? HISPARSE_OK : cuda_fail(e);
}

// ---- device ----
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_launch() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// x / d for 0 <= x < 2^31 by a multiply (round-up method; exact for these x).
struct FastDiv {
  uint32_t d, mul, shift;
  FastDiv() = default;
  __host__ __device__ explicit FastDiv(uint32_t div) : d(div) {
    shift = 0;
    while ((1ull << shift) < div) ++shift;
    mul = static_cast<uint32_t>(((1ull << 32) * ((1ull << shift) - div)) / div + 1);
  }
  __device__ __forceinline__ uint32_t div(uint32_t x) const {
    return (__umulhi(x, mul) + x) >> shift;
  }
  __device__ __forceinline__ void divmod(uint32_t x, uint32_t &q, uint32_t &r) const {
    q = div(x);
    r = x - q * d;
  }
};

template <class T>
__device__ __forceinline__ float to_f32(T x);
template <>
__device__ __forceinline__ float to_f32(float x) { return x; }
template <>
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
template <>
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
template <class T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ __half from_f32(float x) { return __float2half_rn(x); }

// N contiguous elements, kept in the words they are loaded as (N * sizeof(T) bytes, naturally
// aligned up to 16), so that they cost no more registers than that until they are used.
template <class T, int N>
struct alignas(sizeof(T) * N > 16 ? 16 : sizeof(T) * N) Vec {
  static constexpr int words = sizeof(T) * N / 4;
  uint32_t w[words];
  __device__ __forceinline__ float2 pair(int i) const;          // elements 2i, 2i + 1 in 32 bits
  __device__ __forceinline__ void set_pair(int i, float x, float y);  // rounded to T
};
template <class T>
struct alignas(sizeof(T)) Vec<T, 1> {
  T e;
};
template <class T, int N>
__device__ __forceinline__ float2 Vec<T, N>::pair(int i) const {
  if constexpr (sizeof(T) == 4) {
    return make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
  } else if constexpr (std::is_same_v<T, __half>) {
    return __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
  } else {  // the upper 16 bits of a float
    return make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  }
}
template <class T, int N>
__device__ __forceinline__ void Vec<T, N>::set_pair(int i, float x, float y) {
  if constexpr (sizeof(T) == 4) {
    w[2 * i] = __float_as_uint(x);
    w[2 * i + 1] = __float_as_uint(y);
  } else if constexpr (std::is_same_v<T, __half>) {
    const __half2 h = __floats2half2_rn(x, y);
    w[i] = *reinterpret_cast<const uint32_t *>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    w[i] = *reinterpret_cast<const uint32_t *>(&h);
  }
}

// cos and sin of the phase position * turns, a 64-bit fraction of a turn that
// wraps: the multiplication is exact, so the angle is as good at a million
// positions as at one.
__device__ __forceinline__ float2 rotary_cos_sin(int32_t position, int64_t turns, float amplitude,
                                                 float sign) {
  const int64_t phase = static_cast<int64_t>(static_cast<uint64_t>(static_cast<int64_t>(position)) *
                                             static_cast<uint64_t>(turns));
  float s, c;
  // Half turns in [-1, 1], rounded to 32 bits from all 64: the sine of an angle far below a turn (slow
  // pairs, small positions) is as fine as any.  By two conversions of 32 bits, as one of 64 is slow.
  const uint64_t mag = phase < 0 ? 0 - static_cast<uint64_t>(phase) : static_cast<uint64_t>(phase);
  const float half_turns = fmaf(__uint2float_rn(static_cast<uint32_t>(mag)), 0x1p-63f,
                                __uint2float_rn(static_cast<uint32_t>(mag >> 32)) * 0x1p-31f);
  sincospif(phase < 0 ? -half_turns : half_turns, &s, &c);
  return make_float2(c * amplitude, s * amplitude * sign);
}
