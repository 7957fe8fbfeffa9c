// Row kernels around the decode: the norm and position rotation of query and
// key heads (pa_norm_rope), the same on the way into a paged cache
// (pa_append_rows_rope), and rows of a paged cache as floating values
// (pa_read_rows).
//
// Mathematics, per head of 256 values x with weight w at position p:
//   norm      y_i = x_i (w_i + offset) / sqrt(mean(x^2) + eps)
//   rotation  (y_a, y_b) -> (y_a c - y_b s, y_b c + y_a s) for the pair i of
//             the first rot_dim values, c = f cos(p w_i), s = f sin(p w_i).
// An angle p w_i of a far position loses its fraction in 32 bits, and 64-bit
// floating arithmetic is slow on this part, so the host turns every frequency
// into 64-bit fixed-point turns (2^64 = one revolution): p times that, modulo
// 2^64, is the phase, exact to p * 2^-53 revolutions; its top 32 bits go
// through sincospif.
//
// One warp works on one head at a time: lane l holds values 8l .. 8l+7 (16
// bytes of a 16-bit row), the sum of squares is a shuffle reduction in fp32,
// the rotation partner half a rotation away comes by shuffles, and the cosines
// stay in registers for all the heads of the row that the warp walks.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "pa.h"
#include "pa_device.cuh"
#include "pa_io.cuh"
#include "pa_layout.cuh"

using namespace pa_dev;
using namespace pa_layout;

namespace {

constexpr int kD = 256;
constexpr int kWarps = 4;  // per CTA
constexpr int kMaxPairs = kD / 2;

struct RopeParams {
  const uint8_t* q;
  const uint8_t* k;
  const uint8_t* v;
  const void* wq;
  const void* wk;
  uint8_t* q_out;
  uint8_t* k_out;
  const int32_t* row_pos;
  long long q_stride, k_stride, v_stride, q_out_stride, k_out_stride;  // bytes per row
  long long n_rows;
  int hq, hk, hv;      // heads per row
  int chunks, per;     // warps per row, heads per warp
  int w_type;
  int rot, interleaved;
  float eps, w_offset, factor;
  // append only
  uint8_t* k_pool;
  uint8_t* v_pool;
  const int32_t* row_seq;
  const int32_t* table;
  int32_t* err;
  int page_size, table_stride, n_seq, n_blocks, k_type, v_type;
  uint64_t turns[kMaxPairs];
};

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

// Store a head's values (lane l: 8l .. 8l+7) as row r of the group at grp.  The
// quantisers are ggml's reference rule in fp32, every operation rounded on its
// own, a block of 32 values being four neighbouring lanes:
//   Q8_0: d = max|x| / 127, id = d ? 1/d : 0, q = round-half-away(x * id);
//   Q4_0: m = the x of largest |x| (the first on ties), d = m / -8,
//         q = min(15, trunc(x * id + 8.5)).
__device__ __forceinline__ void store_row(int type, bool is_v, const float (&x)[8], uint8_t* grp, int r, int lane) {
  if (type == PA_F16) {
    *reinterpret_cast<uint4*>(grp + chunk_offset(0, Fmt<PA_F16>::kRowQ, r, lane)) = pack8<__half>(x);
    return;
  }
  const int b = lane >> 2;
  float amax = 0.f, m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (fabsf(x[i]) > amax) {
      amax = fabsf(x[i]);
      m = x[i];
    }
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {  // the first of equals: the lower lane's
    const float oa = __shfl_xor_sync(0xffffffffu, amax, o), om = __shfl_xor_sync(0xffffffffu, m, o);
    if (oa > amax || (oa == amax && (lane & o))) {
      amax = oa;
      m = om;
    }
  }
  float d;
  if (type == PA_Q8_0) {
    d = __fdiv_rn(amax, 127.f);
    const float id = d != 0.f ? __fdiv_rn(1.f, d) : 0.f;
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; ++i)
      w[i >> 2] |= ((uint32_t)(uint8_t)(int8_t)(int)roundf(__fmul_rn(x[i], id))) << (8 * (i & 3));
    *reinterpret_cast<uint2*>(grp + chunk_offset(256, Fmt<PA_Q8_0>::kRowQ, r, lane >> 1) + 8 * (lane & 1)) =
        make_uint2(w[0], w[1]);
  } else {
    d = __fdiv_rn(m, -8.f);
    const float id = d != 0.f ? __fdiv_rn(1.f, d) : 0.f;
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; ++i)
      w[i >> 2] |= (uint32_t)min((int)truncf(__fadd_rn(__fmul_rn(x[i], id), 8.5f)), 15) << (8 * (i & 3));
    // lanes 0, 1 of a block hold its low nibbles, lanes 2, 3 the high ones
    const uint32_t h0 = __shfl_xor_sync(0xffffffffu, w[0], 2), h1 = __shfl_xor_sync(0xffffffffu, w[1], 2);
    if (!(lane & 2))
      *reinterpret_cast<uint2*>(grp + chunk_offset(256, Fmt<PA_Q4_0>::kRowQ, r, b) + 8 * (lane & 1)) =
          make_uint2(w[0] | (h0 << 4), w[1] | (h1 << 4));
  }
  if ((lane & 3) == 0)
    *reinterpret_cast<uint16_t*>(grp + (is_v ? v_scale_offset(r, b) : k_scale_offset(r, b))) =
        __half_as_ushort(__float2half_rn(d));
}

// ------------------------------------------------------------------ norm and rotation

// A row's cosines and sines for this lane's values.
struct Turn {
  float c[8], s[8];
};

__device__ __forceinline__ void make_turn(const RopeParams& p, const uint64_t* turns, int pos, int lane, Turn* t) {
  const int half = p.rot >> 1;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int d = 8 * lane + i;
    float c = 1.f, s = 0.f;
    if (d < p.rot) {
      const int pair = p.interleaved ? d >> 1 : d < half ? d : d - half;
      const uint64_t phase = (uint64_t)(int64_t)pos * turns[pair];
      const float x = (float)(int32_t)(uint32_t)(phase >> 32) * (1.f / 2147483648.f);  // half-turns
      sincospif(x, &s, &c);
      c *= p.factor;
      s *= p.factor;
      if (p.interleaved ? !(d & 1) : d < half) s = -s;  // the first of a pair takes -sin
    }
    t->c[i] = c;
    t->s[i] = s;
  }
}

__device__ __forceinline__ void norm_turn(const RopeParams& p, float (&x)[8], const float (&w)[8], bool norm,
                                          const Turn& t, int lane) {
  if (norm) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const float r = rsqrtf(ss * (1.f / kD) + p.eps);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = x[i] * r * w[i];
  }
  if (p.rot == 0) return;
  if (p.interleaved) {
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const float a = x[i], b = x[i + 1];
      x[i] = fmaf(a, t.c[i], b * t.s[i]);
      x[i + 1] = fmaf(b, t.c[i + 1], a * t.s[i + 1]);
    }
  } else {
    const int h = p.rot >> 4;  // lanes of half a rotation
    const int from = lane < h ? lane + h : lane < 2 * h ? lane - h : lane;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float o = __shfl_sync(0xffffffffu, x[i], from);
      x[i] = fmaf(x[i], t.c[i], o * t.s[i]);
    }
  }
}

__device__ __forceinline__ void load_weight(const RopeParams& p, const void* w, int lane, float (&out)[8]) {
  if (!w) return;
  if (p.w_type == PA_DT_F32) load8<float>(static_cast<const uint8_t*>(w) + 32 * lane, out);
  else if (p.w_type == PA_DT_F16) load8<__half>(static_cast<const uint8_t*>(w) + 16 * lane, out);
  else load8<__nv_bfloat16>(static_cast<const uint8_t*>(w) + 16 * lane, out);
#pragma unroll
  for (int i = 0; i < 8; ++i) out[i] += p.w_offset;
}

// kAppend: keys and values go into the pools; else keys go to k_out.
template <typename In, typename Out, bool kAppend>
__global__ void __launch_bounds__(32 * kWarps) pa_rope_kernel(const __grid_constant__ RopeParams p) {
  if (threadIdx.x == 0) asm volatile("griddepcontrol.launch_dependents;");
  __shared__ uint64_t turns[kMaxPairs];
  const int lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < p.rot / 2; i += 32 * kWarps) turns[i] = p.turns[i];
  __syncthreads();
  const long long item = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const long long row = item / p.chunks;
  if (row >= p.n_rows) return;
  const int chunk = (int)(item - row * p.chunks);
  const int h0 = chunk * p.per, h1 = min(h0 + p.per, p.hq + p.hk + p.hv);
  const int pos = __ldg(p.row_pos + row);
  Turn t;
  if (h0 < p.hq + p.hk) make_turn(p, turns, pos, lane, &t);
  float wq[8], wk[8];
  if (h0 < p.hq) load_weight(p, p.wq, lane, wq);
  if (h0 < p.hq + p.hk && h1 > p.hq) load_weight(p, p.wk, lane, wk);
  Place at{};
  bool placed = false;
  if (kAppend && h1 > p.hq) {
    placed = place_of(p.table, p.table_stride, p.n_seq, p.n_blocks, p.page_size, p.hk, __ldg(p.row_seq + row), pos, &at);
    if (!placed && lane == 0) record_error(p.err, PA_ERR_BOUNDS);
  }
  for (int h = h0; h < h1; ++h) {
    float x[8];
    if (h < p.hq) {
      load8<In>(p.q + row * p.q_stride + (long long)h * kD * sizeof(In) + 8 * sizeof(In) * lane, x);
      norm_turn(p, x, wq, p.wq != nullptr, t, lane);
      store8<Out>(p.q_out + row * p.q_out_stride + (long long)h * kD * sizeof(Out) + 8 * sizeof(Out) * lane, x);
    } else if (h < p.hq + p.hk) {
      const int hh = h - p.hq;
      load8<In>(p.k + row * p.k_stride + (long long)hh * kD * sizeof(In) + 8 * sizeof(In) * lane, x);
      norm_turn(p, x, wk, p.wk != nullptr, t, lane);
      if constexpr (kAppend) {
        if (placed)
          store_row(p.k_type, false, x, p.k_pool + (at.grp_row + (long long)hh * p.page_size) * row_bytes_of(p.k_type),
                    at.r, lane);
      } else {
        store8<Out>(p.k_out + row * p.k_out_stride + (long long)hh * kD * sizeof(Out) + 8 * sizeof(Out) * lane, x);
      }
    } else if constexpr (kAppend) {
      const int hh = h - p.hq - p.hk;
      load8<In>(p.v + row * p.v_stride + (long long)hh * kD * sizeof(In) + 8 * sizeof(In) * lane, x);
      if (placed)
        store_row(p.v_type, true, x, p.v_pool + (at.grp_row + (long long)hh * p.page_size) * row_bytes_of(p.v_type),
                  at.r, lane);
    }
  }
}

// ------------------------------------------------------------------ reading rows back

struct ReadParams {
  const uint8_t* k_pool;
  const uint8_t* v_pool;
  uint8_t* k_out;
  uint8_t* v_out;
  const int32_t* row_seq;
  const int32_t* row_pos;
  const int32_t* table;
  int32_t* err;
  long long n_rows;
  int n_heads, page_size, table_stride, n_seq, n_blocks, k_type, v_type;
};

// One warp per (row, head): its K row, then its V row.
template <typename Out>
__global__ void __launch_bounds__(32 * kWarps) pa_read_kernel(const __grid_constant__ ReadParams p) {
  if (threadIdx.x == 0) asm volatile("griddepcontrol.launch_dependents;");
  const int lane = threadIdx.x & 31;
  const long long item = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const long long row = item / p.n_heads;
  if (row >= p.n_rows) return;
  const int head = (int)(item - row * p.n_heads);
  Place at{};
  const bool placed = place_of(p.table, p.table_stride, p.n_seq, p.n_blocks, p.page_size, p.n_heads,
                               __ldg(p.row_seq + row), __ldg(p.row_pos + row), &at);
  if (!placed && lane == 0) record_error(p.err, PA_ERR_BOUNDS);
  const long long gr = at.grp_row + (long long)head * p.page_size, o = (item * kD + 8 * lane) * (long long)sizeof(Out);
  float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (p.k_out) {
    if (placed) read_row(p.k_type, false, p.k_pool + gr * row_bytes_of(p.k_type), at.r, lane, x);
    store8<Out>(p.k_out + o, x);
  }
  if (p.v_out) {
    if (placed) read_row(p.v_type, true, p.v_pool + gr * row_bytes_of(p.v_type), at.r, lane, x);
    store8<Out>(p.v_out + o, x);
  }
}

// ------------------------------------------------------------------ host side

// Revolutions per position in 64-bit fixed point, modulo one revolution.
uint64_t turns_of(double radians) {
  double t = radians / 6.283185307179586476925286766559;
  t -= std::floor(t);
  t = std::ldexp(t, 64);
  return t >= 18446744073709551616.0 ? 0 : (uint64_t)t;
}

pa_status check_rope(const pa_rope_desc* r) {
  if (!r) return PA_ERR_INVALID;
  if (r->rot_dim > (uint32_t)kD || r->rot_dim % 16) return PA_ERR_UNSUPPORTED;
  if (r->interleaved != 0 && r->interleaved != 1) return PA_ERR_INVALID;
  if (!(r->eps >= 0.f) || !std::isfinite(r->eps) || !std::isfinite(r->weight_offset) || !std::isfinite(r->attn_factor))
    return PA_ERR_INVALID;
  for (uint32_t i = 0; i < r->rot_dim / 2; ++i)
    if (!std::isfinite(r->inv_freq[i])) return PA_ERR_INVALID;
  return PA_OK;
}

void fill_rope(const pa_rope_desc* r, RopeParams* p) {
  p->rot = (int)r->rot_dim;
  p->interleaved = r->interleaved;
  p->eps = r->eps;
  p->w_offset = r->weight_offset;
  p->factor = r->attn_factor;
  for (int i = 0; i < p->rot / 2; ++i) p->turns[i] = turns_of(r->inv_freq[i]);
}

bool aligned16(const void* a) { return ((uintptr_t)a & 15) == 0; }

// A row stride in elements: every row 16-byte aligned, and no row inside
// another's heads.
bool stride_ok(int64_t stride, uint32_t heads, int type) {
  return stride >= (int64_t)heads * kD && (stride * dtype_bytes(type)) % 16 == 0 && stride <= (int64_t(1) << 40);
}

pa_status sm_count(int* sms) {
  int device = 0;
  if (cudaGetDevice(&device) != cudaSuccess) return PA_ERR_CUDA;
  return cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, device) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

template <typename In, typename Out, bool kAppend>
pa_status launch_rope(RopeParams& p, cudaStream_t cs) {
  int sms = 0;
  const pa_status st = sm_count(&sms);
  if (st != PA_OK) return st;
  // Few rows: a warp per head, so that a step of one token spreads over the
  // SMs; many rows: a warp walks more heads of its row and computes the row's
  // angles once for them.
  const int heads = p.hq + p.hk + p.hv;
  const long long want = (32ll * sms + p.n_rows - 1) / p.n_rows;
  p.per = (int)((heads + (want < heads ? want : heads) - 1) / (want < heads ? want : heads));
  p.chunks = (heads + p.per - 1) / p.per;
  const long long items = p.n_rows * p.chunks, grid = (items + kWarps - 1) / kWarps;
  if (grid > 0x7fffffffll) return PA_ERR_UNSUPPORTED;
  pa_rope_kernel<In, Out, kAppend><<<(unsigned)grid, 32 * kWarps, 0, cs>>>(p);
  return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

template <typename In, bool kAppend>
pa_status launch_rope_out(RopeParams& p, int out_type, cudaStream_t cs) {
  if (out_type == PA_DT_F32) return launch_rope<In, float, kAppend>(p, cs);
  if (out_type == PA_DT_F16) return launch_rope<In, __half, kAppend>(p, cs);
  return launch_rope<In, __nv_bfloat16, kAppend>(p, cs);
}

template <bool kAppend>
pa_status launch_rope_in(RopeParams& p, int in_type, int out_type, cudaStream_t cs) {
  if (in_type == PA_DT_F32) return launch_rope_out<float, kAppend>(p, out_type, cs);
  if (in_type == PA_DT_F16) return launch_rope_out<__half, kAppend>(p, out_type, cs);
  return launch_rope_out<__nv_bfloat16, kAppend>(p, out_type, cs);
}

// Checks of one set of heads: present with sound strides and alignment, or
// absent altogether.
pa_status check_heads(const void* x, int64_t stride, uint32_t heads, int in_type, const void* w, const void* out,
                      int64_t out_stride, int out_type) {
  if (heads == 0) return x || out ? PA_ERR_INVALID : PA_OK;
  if (!x || !out || heads > 4096) return PA_ERR_INVALID;
  if (!aligned16(x) || !aligned16(out) || (w && !aligned16(w))) return PA_ERR_INVALID;
  if (!stride_ok(stride, heads, in_type) || !stride_ok(out_stride, heads, out_type)) return PA_ERR_INVALID;
  // in place only when every head lands on itself
  if (x == out && (in_type != out_type || stride != out_stride)) return PA_ERR_INVALID;
  return PA_OK;
}

}  // namespace

extern "C" pa_status pa_norm_rope(const pa_rope_desc* rope, const void* q, int64_t q_stride, uint32_t n_q_heads,
                                  const void* k, int64_t k_stride, uint32_t n_kv_heads, int32_t in_type,
                                  const void* q_weight, const void* k_weight, int32_t w_type, const int32_t* row_pos,
                                  uint32_t n_rows, void* q_out, int64_t q_out_stride, void* k_out,
                                  int64_t k_out_stride, int32_t out_type, pa_stream_t stream) {
  pa_status st = check_rope(rope);
  if (st != PA_OK) return st;
  if (!dtype_bytes(in_type) || !dtype_bytes(out_type) || !dtype_bytes(w_type)) return PA_ERR_UNSUPPORTED;
  if (n_q_heads + n_kv_heads == 0) return PA_ERR_INVALID;
  if (n_rows == 0) return PA_OK;
  if (!row_pos) return PA_ERR_INVALID;
  st = check_heads(q, q_stride, n_q_heads, in_type, q_weight, q_out, q_out_stride, out_type);
  if (st != PA_OK) return st;
  st = check_heads(k, k_stride, n_kv_heads, in_type, k_weight, k_out, k_out_stride, out_type);
  if (st != PA_OK) return st;
  RopeParams p{};
  fill_rope(rope, &p);
  p.q = static_cast<const uint8_t*>(q);
  p.k = static_cast<const uint8_t*>(k);
  p.wq = q_weight;
  p.wk = k_weight;
  p.w_type = w_type;
  p.q_out = static_cast<uint8_t*>(q_out);
  p.k_out = static_cast<uint8_t*>(k_out);
  p.q_stride = q_stride * dtype_bytes(in_type);
  p.k_stride = k_stride * dtype_bytes(in_type);
  p.q_out_stride = q_out_stride * dtype_bytes(out_type);
  p.k_out_stride = k_out_stride * dtype_bytes(out_type);
  p.row_pos = row_pos;
  p.n_rows = n_rows;
  p.hq = (int)n_q_heads;
  p.hk = (int)n_kv_heads;
  return launch_rope_in<false>(p, in_type, out_type, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" pa_status pa_append_rows_rope(const pa_pool* pool, void* k_pool, void* v_pool, const pa_rope_desc* rope,
                                         const void* k_rows, int64_t k_stride, const void* v_rows, int64_t v_stride,
                                         int32_t in_type, const void* k_weight, int32_t w_type, const void* q,
                                         int64_t q_stride, uint32_t n_q_heads, const void* q_weight, void* q_out,
                                         int64_t q_out_stride, int32_t q_out_type, const int32_t* row_seq,
                                         const int32_t* row_pos, uint32_t n_rows, const int32_t* block_table,
                                         uint32_t table_stride, uint32_t n_seq, int32_t* err, pa_stream_t stream) {
  pa_pool_desc d;
  if (pa_pool_get_desc(pool, &d) != PA_OK) return PA_ERR_INVALID;
  pa_status st = check_rope(rope);
  if (st != PA_OK) return st;
  if (d.head_dim != (uint32_t)kD) return PA_ERR_UNSUPPORTED;
  if (!dtype_bytes(in_type) || !dtype_bytes(w_type) || !dtype_bytes(q_out_type)) return PA_ERR_UNSUPPORTED;
  if (n_rows == 0) return PA_OK;
  if (!k_pool || !v_pool || !k_rows || !v_rows || !row_seq || !row_pos || !block_table || !err || table_stride == 0 ||
      n_seq == 0)
    return PA_ERR_INVALID;
  if (!aligned16(k_pool) || !aligned16(v_pool) || !aligned16(k_rows) || !aligned16(v_rows) ||
      (k_weight && !aligned16(k_weight)) || !stride_ok(k_stride, d.n_kv_heads, in_type) ||
      !stride_ok(v_stride, d.n_kv_heads, in_type))
    return PA_ERR_INVALID;
  st = check_heads(q, q_stride, n_q_heads, in_type, q_weight, q_out, q_out_stride, q_out_type);
  if (st != PA_OK) return st;
  RopeParams p{};
  fill_rope(rope, &p);
  p.q = static_cast<const uint8_t*>(q);
  p.k = static_cast<const uint8_t*>(k_rows);
  p.v = static_cast<const uint8_t*>(v_rows);
  p.wq = q_weight;
  p.wk = k_weight;
  p.w_type = w_type;
  p.q_out = static_cast<uint8_t*>(q_out);
  p.q_stride = q_stride * dtype_bytes(in_type);
  p.k_stride = k_stride * dtype_bytes(in_type);
  p.v_stride = v_stride * dtype_bytes(in_type);
  p.q_out_stride = q_out_stride * dtype_bytes(q_out_type);
  p.row_pos = row_pos;
  p.row_seq = row_seq;
  p.n_rows = n_rows;
  p.hq = (int)n_q_heads;
  p.hk = p.hv = (int)d.n_kv_heads;
  p.k_pool = static_cast<uint8_t*>(k_pool);
  p.v_pool = static_cast<uint8_t*>(v_pool);
  p.table = block_table;
  p.err = err;
  p.page_size = (int)d.page_size;
  p.table_stride = (int)table_stride;
  p.n_seq = (int)n_seq;
  p.n_blocks = (int)d.n_blocks;
  p.k_type = d.k_type;
  p.v_type = d.v_type;
  return launch_rope_in<true>(p, in_type, q_out_type, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" pa_status pa_read_rows(const pa_pool* pool, const void* k_pool, const void* v_pool, const int32_t* row_seq,
                                  const int32_t* row_pos, uint32_t n_rows, const int32_t* block_table,
                                  uint32_t table_stride, uint32_t n_seq, void* k_out, void* v_out, int32_t out_type,
                                  int32_t* err, pa_stream_t stream) {
  pa_pool_desc d;
  if (pa_pool_get_desc(pool, &d) != PA_OK) return PA_ERR_INVALID;
  if (d.head_dim != (uint32_t)kD || !dtype_bytes(out_type)) return PA_ERR_UNSUPPORTED;
  if (n_rows == 0) return PA_OK;
  if ((!k_out && !v_out) || (k_out && !k_pool) || (v_out && !v_pool) || !row_seq || !row_pos || !block_table || !err ||
      table_stride == 0 || n_seq == 0)
    return PA_ERR_INVALID;
  if (!aligned16(k_pool) || !aligned16(v_pool) || !aligned16(k_out) || !aligned16(v_out)) return PA_ERR_INVALID;
  ReadParams p{};
  p.k_pool = static_cast<const uint8_t*>(k_pool);
  p.v_pool = static_cast<const uint8_t*>(v_pool);
  p.k_out = static_cast<uint8_t*>(k_out);
  p.v_out = static_cast<uint8_t*>(v_out);
  p.row_seq = row_seq;
  p.row_pos = row_pos;
  p.table = block_table;
  p.err = err;
  p.n_rows = n_rows;
  p.n_heads = (int)d.n_kv_heads;
  p.page_size = (int)d.page_size;
  p.table_stride = (int)table_stride;
  p.n_seq = (int)n_seq;
  p.n_blocks = (int)d.n_blocks;
  p.k_type = d.k_type;
  p.v_type = d.v_type;
  const long long grid = ((long long)n_rows * d.n_kv_heads + kWarps - 1) / kWarps;
  if (grid > 0x7fffffffll) return PA_ERR_UNSUPPORTED;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  if (out_type == PA_DT_F32) pa_read_kernel<float><<<(unsigned)grid, 32 * kWarps, 0, cs>>>(p);
  else if (out_type == PA_DT_F16) pa_read_kernel<__half><<<(unsigned)grid, 32 * kWarps, 0, cs>>>(p);
  else pa_read_kernel<__nv_bfloat16><<<(unsigned)grid, 32 * kWarps, 0, cs>>>(p);
  return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
