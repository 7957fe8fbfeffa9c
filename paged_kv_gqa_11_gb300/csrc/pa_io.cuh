// Rows of fp32, binary16 or bfloat16 values in global memory, and rows of the
// pools read as fp32: eight values at a time, rounded once (to nearest even) on
// the way out.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "pa.h"
#include "pa_layout.cuh"

namespace pa_dev {

// Pairs of floats in 64 bits, for the paired fp32 instructions.

__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}


// Bytes of one value of a pa_dtype; 0 if there is no such type.
inline int dtype_bytes(int32_t t) {
  return t == PA_DT_F32 ? 4 : t == PA_DT_F16 || t == PA_DT_BF16 ? 2 : 0;
}

// Eight values from the 16 (32 for fp32) bytes that hold them.
template <typename T>
__device__ __forceinline__ void unpack8(const uint4* v, float (&x)[8]);

template <>
__device__ __forceinline__ void unpack8<float>(const uint4* v, float (&x)[8]) {
  const uint32_t w[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(w[i]);
}

template <>
__device__ __forceinline__ void unpack8<__half>(const uint4* v, float (&x)[8]) {
  const uint32_t w[4] = {v->x, v->y, v->z, v->w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

template <>
__device__ __forceinline__ void unpack8<__nv_bfloat16>(const uint4* v, float (&x)[8]) {
  const uint32_t w[4] = {v->x, v->y, v->z, v->w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

// src 16-byte aligned.  Plain loads, not the read-only path: the rows may be
// overwritten in place by the same kernel.
template <typename T>
__device__ __forceinline__ void load8(const uint8_t* src, float (&x)[8]) {
  uint4 v[sizeof(T) / 2];
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) v[i] = reinterpret_cast<const uint4*>(src)[i];
  unpack8<T>(v, x);
}

// Eight values packed in 16 bytes.
template <typename T>
__device__ __forceinline__ uint4 pack8(const float (&x)[8]);

template <>
__device__ __forceinline__ uint4 pack8<__half>(const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <>
__device__ __forceinline__ uint4 pack8<__nv_bfloat16>(const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <typename T>
__device__ __forceinline__ void store8(uint8_t* dst, const float (&x)[8]) {
  *reinterpret_cast<uint4*>(dst) = pack8<T>(x);
}

template <>
__device__ __forceinline__ void store8<float>(uint8_t* dst, const float (&x)[8]) {
  reinterpret_cast<float4*>(dst)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(dst)[1] = make_float4(x[4], x[5], x[6], x[7]);
}

__host__ __device__ constexpr int row_bytes_of(int type) {
  return type == PA_F16 ? pa_layout::Fmt<PA_F16>::kRow : type == PA_Q8_0 ? pa_layout::Fmt<PA_Q8_0>::kRow : pa_layout::Fmt<PA_Q4_0>::kRow;
}

}  // namespace pa_dev
