// Element access shared by the row kernels (norm, rotary positions, cache append): bf16, fp16 and
// fp32 tensors read and written as fp32, one element or eight at a time.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "sm100.cuh"

namespace dsa {
namespace elem {

__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(float v) { return v; }

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }

// Eight consecutive elements as loaded (16 or 32 bytes), so that loads can be issued ahead of
// their use at the cost of the raw registers only.  The pointer is 16-byte aligned.
template <typename T>
struct Raw8 {
  uint4 v[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) v[i] = reinterpret_cast<const uint4*>(p)[i];
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) v[i] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void store(T* p) const {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) reinterpret_cast<uint4*>(p)[i] = v[i];
  }
  __device__ __forceinline__ void get(float* f) const;
  __device__ __forceinline__ void set(const float* f);
};

template <>
__device__ __forceinline__ void Raw8<__nv_bfloat16>::get(float* f) const {
  const uint32_t w[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {  // a bf16 is the upper half of an fp32
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
template <>
__device__ __forceinline__ void Raw8<__nv_bfloat16>::set(const float* f) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  v[0] = make_uint4(w[0], w[1], w[2], w[3]);
}
template <>
__device__ __forceinline__ void Raw8<__half>::get(float* f) const {
  const uint32_t w[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    f[2 * i] = t.x;
    f[2 * i + 1] = t.y;
  }
}
template <>
__device__ __forceinline__ void Raw8<__half>::set(const float* f) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  v[0] = make_uint4(w[0], w[1], w[2], w[3]);
}
template <>
__device__ __forceinline__ void Raw8<float>::get(float* f) const {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    f[4 * i] = __uint_as_float(v[i].x);
    f[4 * i + 1] = __uint_as_float(v[i].y);
    f[4 * i + 2] = __uint_as_float(v[i].z);
    f[4 * i + 3] = __uint_as_float(v[i].w);
  }
}
template <>
__device__ __forceinline__ void Raw8<float>::set(const float* f) {
#pragma unroll
  for (int i = 0; i < 2; ++i)
    v[i] = make_uint4(__float_as_uint(f[4 * i]), __float_as_uint(f[4 * i + 1]), __float_as_uint(f[4 * i + 2]),
                      __float_as_uint(f[4 * i + 3]));
}

// V = 8, 4, 2 or 1 consecutive elements of a row, at a multiple of their size (8: of 16 bytes).
template <typename T, int V>
struct alignas(V * sizeof(T)) Piece {
  T v[V];
  __device__ __forceinline__ void load(const T* p) { *this = *reinterpret_cast<const Piece*>(p); }
  __device__ __forceinline__ void store(T* p) const { *reinterpret_cast<Piece*>(p) = *this; }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = from_f32<T>(0.f);
  }
  __device__ __forceinline__ void get(float* f) const {
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = to_f32(v[i]);
  }
  __device__ __forceinline__ void set(const float* f) {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = from_f32<T>(f[i]);
  }
};
template <typename T>
struct Piece<T, 8> : Raw8<T> {};

// Bulk copy of `bytes` (a multiple of 16, both addresses 16-byte aligned) from global to this CTA's
// shared memory; its bytes count towards the barrier's phase.
__device__ __forceinline__ void bulk_load(void* dst_smem, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   dev::smem_addr(dst_smem)),
               "l"(src), "r"(bytes), "r"(dev::smem_addr(bar))
               : "memory");
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

}  // namespace elem
}  // namespace dsa
