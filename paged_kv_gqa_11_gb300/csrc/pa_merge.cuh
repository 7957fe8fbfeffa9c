// The merge of a row's pieces (pa_prefix_impl.cuh): what the shared-prefix decode and the
// windowed attention have in common.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "pa_io.cuh"
#include "pa_prefix_impl.cuh"

namespace pa_prefix {

// One CTA per output row: G groups of 64 threads (a float4 of the dims each) take
// every G-th piece of the row, kAhead pieces' loads at once;
// then the groups' states are joined.  With M the largest reference maximum and
// w_i = 2^(m_i - M): out = sum w_i O_i / sum w_i l_i, lse = (M + log2 sum w_i l_i)
// ln 2.  The order is fixed, so the result does not depend on timing.
//
// G by the rows: the more there are, the fewer threads for each, so that all of
// them are resident at once (merge_groups).  Whole calls with 1, 2, 4 and 8
// groups, us: 192 rows 31.9, 28.2, 25.7, 25.0; 408 rows 25.1, 23.7, 22.5, 22.8;
// 768 rows 36.6, 35.0, 35.9, 37.4; 1536 rows 40.8, 42.1, 44.5, 47.3.  Pieces at once:
// 192 rows of 34 pieces 25.2 us with two, 23.7 with five, 25.7 with eight; 768 rows of
// 15 35.5 with four, 34.1 with eight.
inline int merge_groups(int64_t rows, int sms) {
  int g = 8;
  while (g > 1 && rows * g * 64 > (int64_t)sms * 768) g /= 2;
  return g;
}

struct Merged {
  float M, W;  // the largest reference, the sum of weights
  float4 O;    // their sum of V, four dims
};

// The pieces 0 .. np - 1 of a row, whose slot rows row_of gives; true for the threads that
// have the result (group 0: thread col has the dims 4 col .. + 3).
// kRowsPerCta: rows that the CTA's threads merge at once, this thread's being in_cta.
template <int G, int kRowsPerCta = 1, class RowOf>
__device__ __forceinline__ bool merge_pieces(const float2* part_ml, const float* part_o, int np, RowOf&& row_of, int grp, int col,
                                             Merged* out, int in_cta = 0) {
  constexpr int kAhead = kRowsPerCta > 1 && G == 1 ? 2 : G <= 2 ? 8 : 5;
  __shared__ float sms[kRowsPerCta][G], sws[kRowsPerCta][G];
  __shared__ float4 sos[kRowsPerCta][G][64];
  float* sm = sms[in_cta];
  float* sw = sws[in_cta];
  float4(*so)[64] = sos[in_cta];
  float M = -INFINITY, W = 0.f;
  float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = grp; i0 < np; i0 += G * kAhead) {
    float2 ml[kAhead];
    float4 x[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int i = i0 + G * k;
      ml[k] = make_float2(-INFINITY, 0.f);
      x[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i < np) {
        const long long row = row_of(i);
        ml[k] = __ldcg(part_ml + row);
        x[k] = __ldcg(reinterpret_cast<const float4*>(part_o + row * kD) + col);
      }
    }
    float mr = M;
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (ml[k].y != 0.f) mr = fmaxf(mr, ml[k].x);
    const float f0 = W != 0.f ? exp2f(M - mr) : 0.f;
    W *= f0;
    O = make_float4(O.x * f0, O.y * f0, O.z * f0, O.w * f0);
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      // a piece in which the row sees nothing (a sum of 0, not one that is NaN) carries no
      // weight, whatever its reference
      const float f = ml[k].y != 0.f ? exp2f(ml[k].x - mr) : 0.f;
      W = fmaf(f, ml[k].y, W);
      if (ml[k].y != 0.f)
        O = make_float4(fmaf(f, x[k].x, O.x), fmaf(f, x[k].y, O.y), fmaf(f, x[k].z, O.z), fmaf(f, x[k].w, O.w));
    }
    M = mr;
  }
  if (G == 1) {
    *out = Merged{M, W, O};
    return true;
  }
  if (col == 0) {
    sm[grp] = M;
    sw[grp] = W;
  }
  so[grp][col] = O;
  __syncthreads();
  if (grp != 0) return false;
  float Mr = -INFINITY;
#pragma unroll
  for (int i = 0; i < G; ++i) Mr = fmaxf(Mr, sm[i]);
  W = 0.f;
  O = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int i = 0; i < G; ++i) {
    const float f = sw[i] != 0.f ? exp2f(sm[i] - Mr) : 0.f;
    W = fmaf(f, sw[i], W);
    const float4 v = so[i][col];
    O = make_float4(fmaf(f, v.x, O.x), fmaf(f, v.y, O.y), fmaf(f, v.z, O.z), fmaf(f, v.w, O.w));
  }
  *out = Merged{Mr, W, O};
  return true;
}

// A merged row to the values at `at` of out (of out_type) and its lse; zeros and -inf where
// the sequence's length on the device is another.
__device__ __forceinline__ void store_merged(Merged m, bool other, uint8_t* out, int out_type, long long at, int col, float* lse) {
  if (other) {
    m.W = 0.f;
    m.O = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  const float inv = m.W != 0.f ? 1.f / m.W : 0.f;  // NaN where a sum of weights is
  const float4 O = make_float4(m.O.x * inv, m.O.y * inv, m.O.z * inv, m.O.w * inv);
  if (out_type == PA_DT_F32) {
    reinterpret_cast<float4*>(out)[at / 4 + col] = O;
  } else if (out_type == PA_DT_F16) {
    reinterpret_cast<uint2*>(out)[at / 4 + col] = make_uint2(pack_half2(O.x, O.y), pack_half2(O.z, O.w));
  } else {
    const __nv_bfloat162 u = __floats2bfloat162_rn(O.x, O.y), v = __floats2bfloat162_rn(O.z, O.w);
    reinterpret_cast<uint2*>(out)[at / 4 + col] =
        make_uint2(*reinterpret_cast<const uint32_t*>(&u), *reinterpret_cast<const uint32_t*>(&v));
  }
  if (col == 0 && lse) *lse = m.W != 0.f ? (m.M + log2f(m.W)) * pa_split::kLn2 : -INFINITY;
}

}  // namespace pa_prefix
