// Decode of sequences that share prefixes (pa_decode_prefix).
//
// One CTA per (sequence, query token, KV head): each of its eight warps takes
// every eighth key, a lane holding eight of the 256 dims, for the six query
// heads at once; an online softmax in fp32 per warp, and the warps' states
// joined at the end.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "pa.h"
#include "pa_device.cuh"
#include "pa_io.cuh"
#include "pa_layout.cuh"

using namespace pa_dev;

namespace {

constexpr int kD = 256, kGqa = 6, kWarps = 8;
constexpr uint32_t kMaxQTok = 96;

struct PrefixParams {
  const uint8_t* q;
  const uint8_t* k_pool;
  const uint8_t* v_pool;
  const int32_t* table;
  const int32_t* seq_lens;
  uint8_t* out;
  float* lse;
  int32_t* err;
  int n_qtok, n_kv_heads, n_q_heads, page_size, table_stride, n_blocks, k_type, v_type, q_type, out_type;
  float scale;
  int first_seq;
  int32_t lens[256];
};

__device__ __forceinline__ void load_any(int type, const uint8_t* base, long long i, float (&x)[8]) {
  if (type == PA_DT_F32) load8<float>(base + 4 * i, x);
  else if (type == PA_DT_F16) load8<__half>(base + 2 * i, x);
  else load8<__nv_bfloat16>(base + 2 * i, x);
}
__device__ __forceinline__ void store_any(int type, uint8_t* base, long long i, const float (&x)[8]) {
  if (type == PA_DT_F32) store8<float>(base + 4 * i, x);
  else if (type == PA_DT_F16) store8<__half>(base + 2 * i, x);
  else store8<__nv_bfloat16>(base + 2 * i, x);
}

__global__ void __launch_bounds__(32 * kWarps) pa_prefix_kernel(const __grid_constant__ PrefixParams p) {
  __shared__ float sm[kWarps][kGqa], sl[kWarps][kGqa];
  __shared__ float so[kWarps][kGqa][kD];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int head = blockIdx.x % p.n_kv_heads, t = (blockIdx.x / p.n_kv_heads) % p.n_qtok,
            s = blockIdx.x / p.n_kv_heads / p.n_qtok;
  const int L = p.lens[s];
  const bool len_ok = __ldg(p.seq_lens + s) == L;
  if (!len_ok && threadIdx.x == 0) record_error(p.err, PA_ERR_BOUNDS);
  const long long qrow = ((long long)(p.first_seq + s) * p.n_qtok + t) * p.n_q_heads + head * kGqa;
  float q[kGqa][8], o[kGqa][8], m[kGqa], l[kGqa];
  for (int h = 0; h < kGqa; ++h) {
    load_any(p.q_type, p.q, (qrow + h) * kD + 8 * lane, q[h]);
    m[h] = -INFINITY;
    l[h] = 0.f;
    for (int i = 0; i < 8; ++i) o[h][i] = 0.f;
  }
  const int n = len_ok ? L - p.n_qtok + t + 1 : 0;
  for (int j = w; j < n; j += kWarps) {
    const int blk = __ldg(p.table + (long long)s * p.table_stride + j / p.page_size);
    float k[8] = {}, v[8] = {};
    if (blk >= 0 && blk < p.n_blocks) {
      const int slot = j % p.page_size;
      const long long row = ((long long)blk * p.n_kv_heads + head) * p.page_size + (slot & ~15);
      read_row(p.k_type, false, p.k_pool + row * row_bytes_of(p.k_type), slot & 15, lane, k);
      read_row(p.v_type, true, p.v_pool + row * row_bytes_of(p.v_type), slot & 15, lane, v);
    } else if (lane == 0) {
      record_error(p.err, PA_ERR_BOUNDS);
    }
    for (int h = 0; h < kGqa; ++h) {
      float z = 0.f;
      for (int i = 0; i < 8; ++i) z = fmaf(q[h][i], k[i], z);
      for (int x = 16; x > 0; x >>= 1) z += __shfl_xor_sync(0xffffffffu, z, x);
      z *= p.scale;
      const float mn = fmaxf(m[h], z), a = expf(m[h] - mn), e = expf(z - mn);
      m[h] = mn;
      l[h] = l[h] * a + e;
      for (int i = 0; i < 8; ++i) o[h][i] = o[h][i] * a + e * v[i];
    }
  }
  for (int h = 0; h < kGqa; ++h) {
    if (lane == 0) {
      sm[w][h] = m[h];
      sl[w][h] = l[h];
    }
    for (int i = 0; i < 8; ++i) so[w][h][8 * lane + i] = o[h][i];
  }
  __syncthreads();
  if (w >= kGqa) return;
  float M = -INFINITY, W = 0.f, y[8] = {};
  for (int c = 0; c < kWarps; ++c) M = fmaxf(M, sm[c][w]);
  for (int c = 0; c < kWarps; ++c) {
    const float a = sl[c][w] > 0.f ? expf(sm[c][w] - M) : 0.f;
    W += a * sl[c][w];
    for (int i = 0; i < 8; ++i) y[i] += a * so[c][w][8 * lane + i];
  }
  for (int i = 0; i < 8; ++i) y[i] = W > 0.f ? y[i] / W : 0.f;
  store_any(p.out_type, p.out, (qrow + w) * kD + 8 * lane, y);
  if (lane == 0 && p.lse) p.lse[qrow + w] = W > 0.f ? M + logf(W) : -INFINITY;
}

pa_status check_shape(const pa_pool* pool, uint32_t n_qtok, uint32_t n_q_heads, pa_pool_desc* d) {
  if (pa_pool_get_desc(pool, d) != PA_OK) return PA_ERR_INVALID;
  if (d->head_dim != (uint32_t)kD || n_q_heads != d->n_kv_heads * kGqa || n_qtok < 1 || n_qtok > kMaxQTok)
    return PA_ERR_UNSUPPORTED;
  return PA_OK;
}

}  // namespace

extern "C" size_t pa_decode_prefix_workspace_size(const pa_pool* pool, uint32_t n_seq, uint32_t n_groups,
                                                  uint32_t n_qtok, int device) {
  pa_pool_desc d;
  (void)n_groups;
  (void)device;
  if (pa_pool_get_desc(pool, &d) != PA_OK || check_shape(pool, n_qtok, d.n_kv_heads * kGqa, &d) != PA_OK || n_seq == 0)
    return 0;
  return 256;
}

extern "C" pa_status pa_decode_prefix(const pa_pool* pool, const void* q, int32_t q_type, const void* k_pool,
                                      const void* v_pool, const int32_t* block_table, uint32_t table_stride,
                                      const int32_t* seq_lens_dev, const int32_t* seq_lens_host, uint32_t n_seq,
                                      const uint32_t* group_sizes, const int32_t* prefix_lens, uint32_t n_groups,
                                      uint32_t n_qtok, uint32_t n_q_heads, float scale, void* out, int32_t out_type,
                                      float* lse, void* workspace, size_t ws_bytes, int32_t* err,
                                      pa_stream_t stream) {
  pa_pool_desc d;
  pa_status st = check_shape(pool, n_qtok, n_q_heads, &d);
  if (st != PA_OK) return st;
  if (!dtype_bytes(q_type) || !dtype_bytes(out_type)) return PA_ERR_UNSUPPORTED;
  if (n_seq == 0) return n_groups == 0 ? PA_OK : PA_ERR_INVALID;
  if (!q || !k_pool || !v_pool || !block_table || !seq_lens_dev || !seq_lens_host || !group_sizes || !prefix_lens ||
      !out || !workspace || !err || table_stride == 0 || n_groups == 0 || n_groups > n_seq)
    return PA_ERR_INVALID;
  if (((uintptr_t)q | (uintptr_t)out | (uintptr_t)k_pool | (uintptr_t)v_pool) & 15) return PA_ERR_INVALID;
  if ((uintptr_t)workspace & 255) return PA_ERR_INVALID;
  if (!(scale > 0.f) || !std::isfinite(scale)) return PA_ERR_INVALID;
  uint64_t at = 0;
  for (uint32_t g = 0; g < n_groups; ++g) {
    const uint64_t end = at + group_sizes[g];
    if (group_sizes[g] == 0 || end > n_seq || prefix_lens[g] < 0) return PA_ERR_INVALID;
    for (; at < end; ++at) {
      const int64_t L = seq_lens_host[at];
      if (L < (int64_t)n_qtok || L > (int64_t)table_stride * d.page_size || prefix_lens[g] > L - (int64_t)n_qtok)
        return PA_ERR_INVALID;
    }
  }
  if (at != n_seq) return PA_ERR_INVALID;
  if (ws_bytes < 256) return PA_ERR_INVALID;
  for (uint32_t c0 = 0; c0 < n_seq; c0 += 256) {
    PrefixParams p{};
    const uint32_t cn = std::min<uint32_t>(256, n_seq - c0);
    p.q = static_cast<const uint8_t*>(q);
    p.k_pool = static_cast<const uint8_t*>(k_pool);
    p.v_pool = static_cast<const uint8_t*>(v_pool);
    p.table = block_table + (size_t)c0 * table_stride;
    p.seq_lens = seq_lens_dev + c0;
    p.out = static_cast<uint8_t*>(out);
    p.lse = lse;
    p.err = err;
    p.n_qtok = (int)n_qtok;
    p.n_kv_heads = (int)d.n_kv_heads;
    p.n_q_heads = (int)n_q_heads;
    p.page_size = (int)d.page_size;
    p.table_stride = (int)table_stride;
    p.n_blocks = (int)d.n_blocks;
    p.k_type = d.k_type;
    p.v_type = d.v_type;
    p.q_type = q_type;
    p.out_type = out_type;
    p.scale = scale;
    p.first_seq = (int)c0;
    for (uint32_t i = 0; i < cn; ++i) p.lens[i] = seq_lens_host[c0 + i];
    pa_prefix_kernel<<<cn * n_qtok * d.n_kv_heads, 32 * kWarps, 0, reinterpret_cast<cudaStream_t>(stream)>>>(p);
    if (cudaGetLastError() != cudaSuccess) return PA_ERR_CUDA;
  }
  return PA_OK;
}
