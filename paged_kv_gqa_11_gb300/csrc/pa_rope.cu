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
// 2^64, is the phase, exact to p * 2^-53 revolutions.
//
// One warp works on a few heads at a time: lane l holds values 8l .. 8l+7 (16
// bytes of a 16-bit row), the sum of squares is a shuffle reduction in fp32,
// the rotation partner half a rotation away comes by shuffles of the loaded words,
// and the cosines and sines, times the weights, stay in registers for all the
// heads of the row that the warp walks.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "pa.h"
#include "pa_device.cuh"
#include "pa_io.cuh"
#include "pa_layout.cuh"
#include "pa_row_ops.cuh"

using namespace pa_dev;
using namespace pa_layout;
using namespace pa_rows_io;

namespace {


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

// ------------------------------------------------------------------ norm and rotation

// The turn times a weight vector (value i's own, and its partner's).
__device__ __forceinline__ Turn weighted(const RopeParams& p, const Turn& t, const void* w, int lane, int from) {
  if (!w) return t;
  float x[8];
  if (p.w_type == PA_DT_F32) load8<float>(static_cast<const uint8_t*>(w) + 32 * lane, x);
  else if (p.w_type == PA_DT_F16) load8<__half>(static_cast<const uint8_t*>(w) + 16 * lane, x);
  else load8<__nv_bfloat16>(static_cast<const uint8_t*>(w) + 16 * lane, x);
  Turn r;
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] += p.w_offset;
  float o[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    o[i] = p.interleaved ? x[i ^ 1] : __shfl_sync(0xffffffffu, x[i], from);
    if (!is_turned(p.rot, lane)) o[i] = 1.f;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r.c[i] = mul2(t.c[i], pack2(x[2 * i], x[2 * i + 1]));
    r.s[i] = mul2(t.s[i], pack2(o[2 * i], o[2 * i + 1]));
  }
  return r;
}

// A lane's eight values as loaded.
template <typename T>
struct Raw {
  uint4 v[sizeof(T) / 2];

  __device__ __forceinline__ void load(const uint8_t* src) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) v[i] = reinterpret_cast<const uint4*>(src)[i];
  }
  __device__ __forceinline__ Raw from_lane(int l) const {
    Raw r;
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i)
      r.v[i] = make_uint4(__shfl_sync(0xffffffffu, v[i].x, l), __shfl_sync(0xffffffffu, v[i].y, l),
                          __shfl_sync(0xffffffffu, v[i].z, l), __shfl_sync(0xffffffffu, v[i].w, l));
    return r;
  }
  __device__ __forceinline__ Raw masked(uint32_t m) const {
    Raw r;
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.v[i] = make_uint4(v[i].x & m, v[i].y & m, v[i].z & m, v[i].w & m);
    return r;
  }
  __device__ __forceinline__ void get(float (&x)[8]) const { unpack8<T>(v, x); }
  __device__ __forceinline__ void get(uint64_t (&x)[4]) const {
    float f[8];
    get(f);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = pack2(f[2 * i], f[2 * i + 1]);
  }
};

// 1 / sqrt(mean(x^2) + eps) of N heads; the heads' shuffles interleave, so that
// their latencies overlap.
template <typename T, int N>
__device__ __forceinline__ void inverse_norms(const RopeParams& p, const Raw<T> (&raw)[N], float (&r)[N]) {
#pragma unroll
  for (int k = 0; k < N; ++k) {
    uint64_t x[4];
    raw[k].get(x);
    uint64_t sq = mul2(x[0], x[0]);
#pragma unroll
    for (int i = 1; i < 4; ++i) sq = fma2(x[i], x[i], sq);
    const float2 h = unpack2(sq);
    r[k] = h.x + h.y;
  }
#pragma unroll
  for (int m = 16; m > 0; m >>= 1)
#pragma unroll
    for (int k = 0; k < N; ++k) r[k] += __shfl_xor_sync(0xffffffffu, r[k], m);
#pragma unroll
  for (int k = 0; k < N; ++k) r[k] = rsqrtf(r[k] * (1.f / kD) + p.eps);
}

// y = r (x c + partner s), the weights inside c and s; mask: all ones in a lane that is
// turned, else 0.
template <typename T>
__device__ __forceinline__ void turn_head(const RopeParams& p, const Raw<T>& raw, const Turn& t, float r, int from, uint32_t mask,
                                          float (&y)[8]) {
  uint64_t x[4], o[4];
  raw.get(x);
  if (p.interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 v = unpack2(x[i]);
      o[i] = pack2(__uint_as_float(__float_as_uint(v.y) & mask),
                   __uint_as_float((__float_as_uint(v.x) & mask) | (~mask & 0x80000000u)));
    }
  } else {
    raw.from_lane(from).masked(mask).get(o);
  }
  const uint64_t rr = pack2(r, r);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = unpack2(mul2(fma2(x[i], t.c[i], mul2(o[i], t.s[i])), rr));
    y[2 * i] = v.x;
    y[2 * i + 1] = v.y;
  }
}

// Heads that are loaded at once (the next ones are prefetched meanwhile), warps
// that few rows are split into, and resident CTAs that the registers allow: 28
// warps an SM, 20 for the append, whose quantisers would spill more.  4096 rows of
// bf16, one launch after another: 22.8 us with 28 warps and the prefetch, 23.3 with 20,
// 27.0 without the prefetch (20.9 us, 5.6 TB/s, as programmatic dependents); 8192
// rows appended as Q8_0 and Q4_0 and read back: 61.9 us, 64.5 and more with over 20
// warps, 68.0 without the prefetch (60.4 as dependents); batches of two or eight
// heads are slower.  At 72 registers 16-bit rows spill 76 to 116 bytes a thread, fp32
// rows 240 to 328; the append spills with fp32 rows only (38 to 64).  28 warps was
// chosen with bf16 rows; 4096 of fp32 take 43.8 us, 0.79 of what their bytes need.
constexpr int kBatch = 4, kWarpsPerSm = 48;

// kAppend: keys and values go into the pools; else keys go to k_out.
template <typename In, typename Out, bool kAppend>
__global__ void __launch_bounds__(32 * kWarps, kAppend ? 5 : 7) pa_rope_kernel(const __grid_constant__ RopeParams p) {
  if (threadIdx.x == 0) asm volatile("griddepcontrol.launch_dependents;");
  __shared__ uint64_t turns[kMaxPairs];
  const int lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < p.rot / 2; i += 32 * kWarps) turns[i] = p.turns[i];
  __syncthreads();
  const long long item = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const long long row = item / p.chunks;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // nothing that another kernel wrote is read before this
  if (row >= p.n_rows) return;
  const int chunk = (int)(item - row * p.chunks);
  const int h0 = chunk * p.per, h1 = min(h0 + p.per, p.hq + p.hk + p.hv);
  const int pos = __ldg(p.row_pos + row), from = partner_lane(p.rot, p.interleaved, lane);
  const uint32_t mask = is_turned(p.rot, lane) ? ~0u : 0u;
  if (p.per > kBatch) {  // many rows: the first heads are on their way before the position is known
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int h = h0 + i;
      if (h >= h1) break;
      const uint8_t* src = h < p.hq          ? p.q + row * p.q_stride + h * kD * (int)sizeof(In)
                           : h < p.hq + p.hk ? p.k + row * p.k_stride + (h - p.hq) * kD * (int)sizeof(In)
                                             : p.v + row * p.v_stride + (h - p.hq - p.hk) * kD * (int)sizeof(In);
      asm volatile("prefetch.global.L1 [%0];" ::"l"(src + 8 * (int)sizeof(In) * lane));
    }
  }
  Place at{};
  bool placed = false;
  if (kAppend && h1 > p.hq) {
    placed = place_of(p.table, p.table_stride, p.n_seq, p.n_blocks, p.page_size, p.hk, __ldg(p.row_seq + row), pos, &at);
    if (!placed && lane == 0) record_error(p.err, PA_ERR_BOUNDS);
  }
  // Heads a .. b - 1 of one kind, kBatch at a time: normalised (norm) and turned
  // by t, or as they are (no t), to `put` with their number.
  auto heads = [&](const uint8_t* src, int a, int b, const Turn* t, bool norm, auto&& put) {
    constexpr int kHead = kD * (int)sizeof(In);
    src += a * kHead + 8 * (int)sizeof(In) * lane;
    auto batch = [&](auto count) {
      constexpr int N = decltype(count)::value;
      Raw<In> raw[N];
      float r[N], y[8];
#pragma unroll
      for (int i = 0; i < N; ++i) {
        raw[i].load(src + i * kHead);
        r[i] = 1.f;
      }
      if (N == kBatch) {  // the next batch is on its way while this one is worked on
#pragma unroll
        for (int i = 0; i < N; ++i)
          if (a + N + i < b) asm volatile("prefetch.global.L1 [%0];" ::"l"(src + (N + i) * kHead));
      }
      if (norm) inverse_norms<In, N>(p, raw, r);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        if (t) turn_head<In>(p, raw[i], *t, r[i], from, mask, y);
        else raw[i].get(y);
        put(a + i, y);
      }
      a += N;
      src += N * kHead;
    };
    while (a + kBatch <= b) batch(std::integral_constant<int, kBatch>());
    while (a < b) batch(std::integral_constant<int, 1>());
  };
  const int qk = p.hq + p.hk;
  if (h0 < qk) {
    const Turn t = make_turn(p.rot, p.interleaved, p.factor, [&](int i) { return (uint64_t)(int64_t)pos * turns[i]; }, lane, from);
    if (h0 < p.hq) {
      const Turn tq = weighted(p, t, p.wq, lane, from);
      uint8_t* out = p.q_out + row * p.q_out_stride + 8 * (int)sizeof(Out) * lane;
      heads(p.q + row * p.q_stride, h0, min(h1, p.hq), &tq, p.wq != nullptr,
            [&](int h, const float (&y)[8]) { store8<Out>(out + h * kD * (int)sizeof(Out), y); });
    }
    if (h1 > p.hq) {
      const Turn tk = weighted(p, t, p.wk, lane, from);
      heads(p.k + row * p.k_stride, max(h0, p.hq) - p.hq, min(h1, qk) - p.hq, &tk, p.wk != nullptr,
            [&](int h, const float (&y)[8]) {
              if constexpr (kAppend) {
                if (placed)
                  store_row(p.k_type, false, y, p.k_pool + (at.grp_row + (long long)h * p.page_size) * row_bytes_of(p.k_type),
                            at.r, lane);
              } else {
                store8<Out>(p.k_out + row * p.k_out_stride + (h * kD + 8 * lane) * (int)sizeof(Out), y);
              }
            });
    }
  }
  if constexpr (kAppend) {
    if (h1 > qk && placed)
      heads(p.v + row * p.v_stride, max(h0, qk) - qk, h1 - qk, nullptr, false, [&](int h, const float (&y)[8]) {
        store_row(p.v_type, true, y, p.v_pool + (at.grp_row + (long long)h * p.page_size) * row_bytes_of(p.v_type), at.r, lane);
      });
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
  int pools, rows;  // pools read; rows of a warp
};

constexpr int kReadRows = 8;  // rows of a warp, looked up by a lane each

// The heads of one row of one pool, four in flight at a time.
template <int T, typename Out>
__device__ __forceinline__ void read_heads(const uint8_t* pool, bool is_v, long long grp_row, int r, bool placed, int n_heads,
                                           int page_size, uint8_t* dst, int lane) {
  const uint8_t* grp = pool + grp_row * Fmt<T>::kRow;
  const long long step = (long long)page_size * Fmt<T>::kRow;
  dst += 8 * lane * (int)sizeof(Out);
  if (!placed) {
    const float zero[8] = {};
    for (int h = 0; h < n_heads; ++h) store8<Out>(dst + h * kD * (int)sizeof(Out), zero);
    return;
  }
  for (int h = 0; h < n_heads; h += 4) {
    Stored<T> s[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (h + i < n_heads) s[i].load(grp + (h + i) * step, r, lane, is_v);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (h + i < n_heads) s[i].template store<Out>(dst + (h + i) * kD * (int)sizeof(Out), lane);
  }
}

// A warp per kRows rows of K or of V; their places are looked up at once, a lane
// for each: the three dependent loads of a lookup take longer than a row's copy.
template <int T, typename Out>
__device__ __forceinline__ void read_warp(const ReadParams& p, bool is_v, long long row0, int rows, int lane) {
  Place at{};
  bool placed = false;
  if (lane < rows)
    placed = place_of(p.table, p.table_stride, p.n_seq, p.n_blocks, p.page_size, p.n_heads, __ldg(p.row_seq + row0 + lane),
                      __ldg(p.row_pos + row0 + lane), &at);
  if (lane < rows && !placed) record_error(p.err, PA_ERR_BOUNDS);
  for (int i = 0; i < rows; ++i)
    read_heads<T, Out>(is_v ? p.v_pool : p.k_pool, is_v, __shfl_sync(0xffffffffu, at.grp_row, i), __shfl_sync(0xffffffffu, at.r, i),
                       __shfl_sync(0xffffffffu, (int)placed, i) != 0, p.n_heads, p.page_size,
                       (is_v ? p.v_out : p.k_out) + (row0 + i) * p.n_heads * kD * (long long)sizeof(Out), lane);
}

template <typename Out>
__global__ void __launch_bounds__(32 * kWarps) pa_read_kernel(const __grid_constant__ ReadParams p) {
  if (threadIdx.x == 0) asm volatile("griddepcontrol.launch_dependents;");
  const int lane = threadIdx.x & 31;
  const long long item = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const long long batch = item / p.pools;
  const long long row0 = batch * p.rows;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // nothing that another kernel wrote is read before this
  if (row0 >= p.n_rows) return;
  const bool is_v = p.pools == 1 ? p.k_out == nullptr : item - batch * p.pools != 0;
  const int rows = (int)min((long long)p.rows, p.n_rows - row0), type = is_v ? p.v_type : p.k_type;
  if (type == PA_F16) read_warp<PA_F16, Out>(p, is_v, row0, rows, lane);
  else if (type == PA_Q8_0) read_warp<PA_Q8_0, Out>(p, is_v, row0, rows, lane);
  else read_warp<PA_Q4_0, Out>(p, is_v, row0, rows, lane);
}

// ------------------------------------------------------------------ host side

void fill_rope(const pa_rope_desc* r, RopeParams* p) {
  p->rot = (int)r->rot_dim;
  p->interleaved = r->interleaved;
  p->eps = r->eps;
  p->w_offset = r->weight_offset;
  p->factor = r->attn_factor;
  for (int i = 0; i < p->rot / 2; ++i) p->turns[i] = turns_of(r->inv_freq[i]);
}

// A row stride in elements: every row 16-byte aligned, and no row inside
// another's heads.
bool stride_ok(int64_t stride, uint32_t heads, int type) {
  return stride >= (int64_t)heads * kD && (stride * dtype_bytes(type)) % 16 == 0 && stride <= (int64_t(1) << 40);
}

// Few rows: a warp per head, so that a step of one token spreads over the SMs;
// many rows: a warp walks more heads of its row and computes the row's angles
// once for them.
void split_heads(int heads, long long rows, int sms, int* chunks, int* per) {
  long long want = (kWarpsPerSm * (long long)sms + rows - 1) / rows;
  if (want > heads) want = heads;
  *per = (int)((heads + want - 1) / want);
  if (*per > kBatch) *per = (*per + kBatch - 1) / kBatch * kBatch;  // whole batches of loads
  *chunks = (heads + *per - 1) / *per;
}

template <typename In, typename Out, bool kAppend>
pa_status launch_rope(RopeParams& p, cudaStream_t cs) {
  int sms = 0;
  const pa_status st = sm_count(&sms);
  if (st != PA_OK) return st;
  split_heads(p.hq + p.hk + p.hv, p.n_rows, sms, &p.chunks, &p.per);
  const long long items = p.n_rows * p.chunks, grid = (items + kWarps - 1) / kWarps;
  if (grid > 0x7fffffffll) return PA_ERR_UNSUPPORTED;
  return launch(pa_rope_kernel<In, Out, kAppend>, p, (unsigned)grid, cs);
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
  int sms = 0;
  const pa_status st = sm_count(&sms);
  if (st != PA_OK) return st;
  p.pools = (k_out != nullptr) + (v_out != nullptr);
  p.rows = (int)std::min<long long>(kReadRows, ((long long)n_rows * p.pools + 32ll * sms - 1) / (32ll * sms));  // 1 while warps are few
  const long long grid = (((long long)n_rows + p.rows - 1) / p.rows * p.pools + kWarps - 1) / kWarps;
  if (grid > 0x7fffffffll) return PA_ERR_UNSUPPORTED;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  if (out_type == PA_DT_F32) return launch(pa_read_kernel<float>, p, (unsigned)grid, cs);
  if (out_type == PA_DT_F16) return launch(pa_read_kernel<__half>, p, (unsigned)grid, cs);
  return launch(pa_read_kernel<__nv_bfloat16>, p, (unsigned)grid, cs);
}
