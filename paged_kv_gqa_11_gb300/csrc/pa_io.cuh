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

// Bytes of one value of a pa_dtype; 0 if there is no such type.
inline int dtype_bytes(int32_t t) {
  return t == PA_DT_F32 ? 4 : t == PA_DT_F16 || t == PA_DT_BF16 ? 2 : 0;
}

// src 16-byte aligned.  Plain loads, not the read-only path: the rows may be
// overwritten in place by the same kernel.
template <typename T>
__device__ __forceinline__ void load8(const uint8_t* src, float (&x)[8]);

template <>
__device__ __forceinline__ void load8<float>(const uint8_t* src, float (&x)[8]) {
  const float4 a = reinterpret_cast<const float4*>(src)[0], b = reinterpret_cast<const float4*>(src)[1];
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}

template <>
__device__ __forceinline__ void load8<__half>(const uint8_t* src, float (&x)[8]) {
  const uint4 v = *reinterpret_cast<const uint4*>(src);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const uint8_t* src, float (&x)[8]) {
  const uint4 v = *reinterpret_cast<const uint4*>(src);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
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

// Values 8 lane .. 8 lane + 7 of row r of the group at grp.
__device__ __forceinline__ void read_row(int type, bool is_v, const uint8_t* grp, int r, int lane, float (&x)[8]) {
  if (type == PA_F16) {
    load8<__half>(grp + pa_layout::chunk_offset(0, pa_layout::Fmt<PA_F16>::kRowQ, r, lane), x);
    return;
  }
  const int b = lane >> 2;
  const float d = __half2float(
      *reinterpret_cast<const __half*>(grp + (is_v ? pa_layout::v_scale_offset(r, b) : pa_layout::k_scale_offset(r, b))));
  if (type == PA_Q8_0) {
    const uint2 w = *reinterpret_cast<const uint2*>(grp + pa_layout::chunk_offset(256, pa_layout::Fmt<PA_Q8_0>::kRowQ, r, lane >> 1) +
                                                    8 * (lane & 1));
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = (float)(int8_t)(((i < 4 ? w.x : w.y) >> (8 * (i & 3))) & 0xffu) * d;
  } else {
    const uint2 w = *reinterpret_cast<const uint2*>(grp + pa_layout::chunk_offset(256, pa_layout::Fmt<PA_Q4_0>::kRowQ, r, b) + 8 * (lane & 1));
    const int sh = lane & 2 ? 4 : 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = (float)((int)(((i < 4 ? w.x : w.y) >> (8 * (i & 3) + sh)) & 15u) - 8) * d;
  }
}

}  // namespace pa_dev
