// What the kernels that work on single rows of a cache share: where a row lies, how it is
// stored and read, the angles of a rotation, and the host's checks and launches.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <type_traits>

#include "pa.h"
#include "pa_device.cuh"
#include "pa_io.cuh"
#include "pa_layout.cuh"

namespace pa_rows_io {

using namespace pa_dev;
using namespace pa_layout;

constexpr int kD = 256;
constexpr int kWarps = 4;  // per CTA
constexpr int kMaxPairs = kD / 2;

// ------------------------------------------------------------------ cache rows

// Where (seq, pos) sits: the first row of its group in head 0's page, counted
// in rows of the pool, and its row in the group; false for a row outside the
// batch, the table or the pool.
struct Place {
  long long grp_row;
  int r;
};

__device__ __forceinline__ bool place_of(const int32_t* table, int table_stride, int n_seq, int n_blocks, int page_size,
                                         int n_heads, int s, int pos, Place* out) {
  if (s < 0 || s >= n_seq || pos < 0) return false;
  const uint32_t page = (uint32_t)pos / (uint32_t)page_size;
  if (page >= (uint32_t)table_stride) return false;
  const int blk = __ldg(table + (long long)s * table_stride + page);
  if (blk < 0 || blk >= n_blocks) return false;
  const int slot = (int)((uint32_t)pos - page * (uint32_t)page_size);
  out->grp_row = (long long)blk * n_heads * page_size + (slot & ~(kGroup - 1));
  out->r = slot & (kGroup - 1);
  return true;
}

// Four whole numbers -128 .. 255 as bytes.
__device__ __forceinline__ uint32_t bytes4(int a, int b, int c, int d) {
  return prmt(prmt((uint32_t)a, (uint32_t)b, 0x0040), prmt((uint32_t)c, (uint32_t)d, 0x0040), 0x5410);
}

// The quantisers are ggml's reference rule in fp32, every operation rounded on its
// own, a block of 32 values being four neighbouring lanes (lane l: values 8l .. 8l+7):
//   Q8_0: d = max|x| / 127, id = d ? 1/d : 0, q = round-half-away(x * id);
//   Q4_0: m = the x of largest |x| (the first on ties), d = m / -8,
//         q = min(15, trunc(x * id + 8.5)).
// round-half-away(y) is trunc(y + copysign(1/2 - 2^-25, y)): the sum of a tie k +
// 1/2 rounds up to k + 1, the one of the largest float below it stays below.
// Both return the 8 bytes at the lane's place in its block (Q4_0: in lanes 0 and 1 of four).
__device__ __forceinline__ uint2 quantise_q8(const float (&x)[8], float* d) {
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(x[i]));
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  *d = __fdiv_rn(amax, 127.f);
  const float id = *d != 0.f ? __fdiv_rn(1.f, *d) : 0.f;
  int q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float y = __fmul_rn(x[i], id);
    q[i] = __float2int_rz(__fadd_rn(y, copysignf(0.49999997f, y)));
  }
  return make_uint2(bytes4(q[0], q[1], q[2], q[3]), bytes4(q[4], q[5], q[6], q[7]));
}

__device__ __forceinline__ uint2 quantise_q4(const float (&x)[8], int lane, float* d) {
  float amax = 0.f, m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (fabsf(x[i]) > amax) {
      amax = fabsf(x[i]);
      m = x[i];
    }
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {  // the first of equals: the lower lane's
    const float om = __shfl_xor_sync(0xffffffffu, m, o);
    if (fabsf(om) > fabsf(m) || (fabsf(om) == fabsf(m) && (lane & o))) m = om;
  }
  *d = __fdiv_rn(m, -8.f);
  const float id = *d != 0.f ? __fdiv_rn(1.f, *d) : 0.f;
  int q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = min(__float2int_rz(__fadd_rn(__fmul_rn(x[i], id), 8.5f)), 15);
  const uint32_t w0 = bytes4(q[0], q[1], q[2], q[3]), w1 = bytes4(q[4], q[5], q[6], q[7]);
  // lanes 0, 1 of a block hold its low nibbles, lanes 2, 3 the high ones
  const uint32_t h0 = __shfl_xor_sync(0xffffffffu, w0, 2), h1 = __shfl_xor_sync(0xffffffffu, w1, 2);
  return make_uint2(w0 | (h0 << 4), w1 | (h1 << 4));
}

// What a lane stores of a row: an F16 row's 16 bytes; of a quantised row the 8 bytes at
// its place in its block, and the block's scale.
struct Packed {
  uint4 w;
  uint32_t d;
};

__device__ __forceinline__ Packed quantised(int type, const float (&x)[8], int lane) {
  if (type == PA_F16) return Packed{pack8<__half>(x), 0u};
  float d;
  const uint2 w = type == PA_Q8_0 ? quantise_q8(x, &d) : quantise_q4(x, lane, &d);
  return Packed{make_uint4(w.x, w.y, 0u, 0u), (uint32_t)__half_as_ushort(__float2half_rn(d))};
}

// Where a lane's bytes and its block's scale lie in row r of a group.
struct Lane {
  int body, scale;
};

__device__ __forceinline__ Lane lane_of(int type, bool is_v, int r, int lane) {
  const int b = lane >> 2;
  if (type == PA_F16) return Lane{chunk_offset(0, Fmt<PA_F16>::kRowQ, r, lane), 0};
  const int chunk = type == PA_Q8_0 ? chunk_offset(256, Fmt<PA_Q8_0>::kRowQ, r, lane >> 1) : chunk_offset(256, Fmt<PA_Q4_0>::kRowQ, r, b);
  return Lane{chunk + 8 * (lane & 1), is_v ? v_scale_offset(r, b) : k_scale_offset(r, b)};
}

__device__ __forceinline__ void put(int type, const Packed& x, uint8_t* row, const Lane& at, int lane) {
  if (type == PA_F16) {
    *reinterpret_cast<uint4*>(row + at.body) = x.w;
    return;
  }
  if (type == PA_Q8_0 || !(lane & 2)) *reinterpret_cast<uint2*>(row + at.body) = make_uint2(x.w.x, x.w.y);
  if ((lane & 3) == 0) *reinterpret_cast<uint16_t*>(row + at.scale) = (uint16_t)x.d;
}

// Store a head's values as row r of the group at grp.  (Not by quantised and put: one branch
// on the type, with the stores inside; 777 rows of Q8_0 appended and read 13.8 us against 15.3.)
__device__ __forceinline__ void store_row(int type, bool is_v, const float (&x)[8], uint8_t* grp, int r, int lane) {
  if (type == PA_F16) {
    *reinterpret_cast<uint4*>(grp + chunk_offset(0, Fmt<PA_F16>::kRowQ, r, lane)) = pack8<__half>(x);
    return;
  }
  const int b = lane >> 2;
  float d;
  if (type == PA_Q8_0) {
    *reinterpret_cast<uint2*>(grp + chunk_offset(256, Fmt<PA_Q8_0>::kRowQ, r, lane >> 1) + 8 * (lane & 1)) = quantise_q8(x, &d);
  } else {
    const uint2 w = quantise_q4(x, lane, &d);
    if (!(lane & 2)) *reinterpret_cast<uint2*>(grp + chunk_offset(256, Fmt<PA_Q4_0>::kRowQ, r, b) + 8 * (lane & 1)) = w;
  }
  if ((lane & 3) == 0)
    *reinterpret_cast<uint16_t*>(grp + (is_v ? v_scale_offset(r, b) : k_scale_offset(r, b))) = __half_as_ushort(__float2half_rn(d));
}

// ------------------------------------------------------------------ angles

// cos and sin of `phase` / 2^32 revolutions: the nearest quarter turn apart, the
// rest (at most pi / 4) by Taylor's series.  Off by less than 5 u (u = 2^-24): the phase
// cut to 32 bits 2^-29 = u / 32 and the angle t three roundings (to fp32, the constant, the
// product), 3 u |t| < 2.4 u; the series' next terms, t^10 / 10! and t^11 / 11!, are below
// 2^-25 = u / 2; its evaluation: t^2 and the coefficients are off by 2 u of terms of at most
// 0.31 and 0.08 together, the last sum by half a step, u / 2: below 1.5 u.
__device__ __forceinline__ void cos_sin(uint32_t phase, float* c, float* s) {
  const uint32_t near = phase + 0x20000000u, quarter = near >> 30;
  const float t = (float)((int32_t)(near & 0x3fffffffu) - 0x20000000) * 1.4629180792671596e-9f;  // 2 pi / 2^32
  const float u = t * t;
  float a = fmaf(u, 2.7557319e-6f, -1.9841270e-4f);
  a = fmaf(u, a, 8.3333333e-3f);
  a = fmaf(u, a, -1.6666667e-1f);
  a = fmaf(t * u, a, t);
  float b = fmaf(u, 2.4801587e-5f, -1.3888889e-3f);
  b = fmaf(u, b, 4.1666667e-2f);
  b = fmaf(u, b, -0.5f);
  b = fmaf(u, b, 1.f);
  const float x = (quarter & 1) ? a : b, y = (quarter & 1) ? b : a;
  *c = __uint_as_float(__float_as_uint(x) ^ (((quarter + 1) & 2) << 30));
  *s = __uint_as_float(__float_as_uint(y) ^ ((quarter & 2) << 30));
}

// What a lane multiplies its values and their partners by: the cosines and
// (signed) sines of its row, times the weights of one kind of head; two values
// to an element, for the paired fp32 instructions.
struct Turn {
  uint64_t c[4], s[4];
};

// Values from rot_dim on have no partner: theirs is read as a zero and their sine is one
// of the other sign, so that x c + partner s is x c - 0, which is x c for infinities and
// zeros of either sign too.  Whole lanes are turned or not (rot_dim is a multiple of 16).
__device__ __forceinline__ bool is_turned(int rot, int lane) { return 8 * lane < rot; }

// The lane that holds the partners of this lane's values (itself when they are
// its own, or when there is nothing to turn).
__device__ __forceinline__ int partner_lane(int rot, int interleaved, int lane) {
  const int h = rot >> 4;  // lanes of half a rotation
  return interleaved || lane >= 2 * h ? lane : lane < h ? lane + h : lane - h;
}

// A lane computes four of the angles of its row: its own four pairs, or half of
// the eight that it shares with its partner lane.  phase_of: of a pair, in 2^64ths of a
// revolution.
template <class PhaseOf>
__device__ __forceinline__ Turn make_turn(int rot, int interleaved, float factor, PhaseOf&& phase_of, int lane, int from) {
  float c[8], s[8];
  const bool turned = is_turned(rot, lane), second = from < lane;
  float ac[4], as[4];
  const int pair0 = interleaved ? 4 * lane : second ? 8 * from + 4 : 8 * lane;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    ac[j] = 1.f;
    as[j] = 0.f;
    if (turned) {
      const uint64_t phase = phase_of(pair0 + j);
      cos_sin((uint32_t)(phase >> 32), &ac[j], &as[j]);
      ac[j] *= factor;
      as[j] *= factor;
    }
  }
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      c[i] = ac[i >> 1];
      s[i] = (i & 1) ? as[i >> 1] : -as[i >> 1];  // the first of a pair takes -sin; not turned: -0, +0
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float oc = __shfl_sync(0xffffffffu, ac[j], from), os = __shfl_sync(0xffffffffu, as[j], from);
      c[j] = second ? oc : ac[j];
      c[j + 4] = second ? ac[j] : oc;
      s[j] = second ? os : -as[j];
      s[j + 4] = second ? as[j] : -os;
    }
  }
  Turn t;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    t.c[i] = pack2(c[2 * i], c[2 * i + 1]);
    t.s[i] = pack2(s[2 * i], s[2 * i + 1]);
  }
  return t;
}

// ------------------------------------------------------------------ stored rows

// A lane's eight values of a stored row: the quants as exact binary16 pairs and
// their scale, or binary16 values.
template <int T>
struct Stored {
  uint32_t h[4];
  uint32_t d;  // the scale twice

  uint4 raw;
  __device__ __forceinline__ void load(const uint8_t* grp, int r, int lane, bool is_v) {
    if (T == PA_F16) {
      raw = *reinterpret_cast<const uint4*>(grp + chunk_offset(0, Fmt<T>::kRowQ, r, lane));
      return;
    }
    const int b = lane >> 2;
    const uint2 w = *reinterpret_cast<const uint2*>(
        grp + chunk_offset(256, Fmt<T>::kRowQ, r, T == PA_Q8_0 ? lane >> 1 : b) + 8 * (lane & 1));
    raw = make_uint4(w.x, w.y, 0u, 0u);
    d = *reinterpret_cast<const uint16_t*>(grp + (is_v ? v_scale_offset(r, b) : k_scale_offset(r, b)));
  }
  // The values as Out, the exact products rounded once.
  template <typename Out>
  __device__ __forceinline__ void store(uint8_t* dst, int lane) {
    float x[8];
    if (T == PA_F16) {
      if (sizeof(Out) == 2 && std::is_same<Out, __half>::value) {
        *reinterpret_cast<uint4*>(dst) = raw;
        return;
      }
      unpack8<__half>(&raw, x);
      store8<Out>(dst, x);
      return;
    }
    // bytes 0 .. 255 under 0x64 are the binary16 numbers 1024 + byte
    const uint32_t bias = T == PA_Q8_0 ? 0xe480e480u : 0xe408e408u;  // -1152, -1032
    uint32_t w[2] = {raw.x, raw.y};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      w[i] = T == PA_Q8_0 ? w[i] ^ 0x80808080u : (w[i] >> ((lane & 2) << 1)) & 0x0f0f0f0fu;
      h[2 * i] = hadd2(prmt(w[i], 0x64646464u, 0x4140), bias);
      h[2 * i + 1] = hadd2(prmt(w[i], 0x64646464u, 0x4342), bias);
    }
    const uint32_t d2 = d | (d << 16);
    if (std::is_same<Out, __half>::value) {
      *reinterpret_cast<uint4*>(dst) = make_uint4(hmul2(h[0], d2), hmul2(h[1], d2), hmul2(h[2], d2), hmul2(h[3], d2));
      return;
    }
    const float df = __half2float(__ushort_as_half((unsigned short)d));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
      x[2 * i] = f.x * df;
      x[2 * i + 1] = f.y * df;
    }
    store8<Out>(dst, x);
  }
};

// ------------------------------------------------------------------ host side

// Revolutions per position in 64-bit fixed point, modulo one revolution.
inline uint64_t turns_of(double radians) {
  double t = radians / 6.283185307179586476925286766559;
  t -= std::floor(t);
  t = std::ldexp(t, 64);
  return t >= 18446744073709551616.0 ? 0 : (uint64_t)t;
}

inline pa_status check_rope(const pa_rope_desc* r) {
  if (!r) return PA_ERR_INVALID;
  if (r->rot_dim > (uint32_t)kD || r->rot_dim % 16) return PA_ERR_UNSUPPORTED;
  if (r->interleaved != 0 && r->interleaved != 1) return PA_ERR_INVALID;
  if (!(r->eps >= 0.f) || !std::isfinite(r->eps) || !std::isfinite(r->weight_offset) || !std::isfinite(r->attn_factor))
    return PA_ERR_INVALID;
  for (uint32_t i = 0; i < r->rot_dim / 2; ++i)
    if (!std::isfinite(r->inv_freq[i])) return PA_ERR_INVALID;
  return PA_OK;
}

inline bool aligned16(const void* a) { return ((uintptr_t)a & 15) == 0; }

inline pa_status sm_count(int* sms) {
  int device = 0;
  if (cudaGetDevice(&device) != cudaSuccess) return PA_ERR_CUDA;
  return cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, device) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

// As a programmatic dependent of what runs before it on the stream: its set-up
// overlaps the other's tail (one token normalised and rotated, call after call:
// 2.1 us instead of 2.8).
template <typename P>
pa_status launch(void (*kernel)(P), const P& p, unsigned grid, cudaStream_t cs) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(32 * kWarps);
  cfg.stream = cs;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace pa_rows_io
