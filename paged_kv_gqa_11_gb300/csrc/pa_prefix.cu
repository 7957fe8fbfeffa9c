// Decode with shared prefixes: the plan, the merge of the pieces, and the host
// side of pa_decode_prefix.  The kernel over the keys is in pa_prefix_impl.cuh,
// compiled once per (K format, V format) pair.
//
// The plan, from the host copy of the lengths: a group's prefix is cut to whole
// row groups (16 keys; the rest joins the suffixes, so a suffix's row groups
// are whole too), and read as a shared prefix when that takes fewer key tiles
// than leaving it in every sequence's own keys.  The tiles, prefixes first, are
// cut into contiguous ranges of equal cost, one CTA per SM (cost_of).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "pa_io.cuh"
#include "pa_merge.cuh"
#include "pa_prefix_impl.cuh"

using namespace pa_dev;
using namespace pa_prefix;
using pa_split::kLn2;
using pa_split::kLog2e;

namespace {

constexpr uint32_t kMaxQTok = 96;
constexpr int64_t kMaxLen = 0x7fffffff - 2 * kKeys;  // a tile past the last key is still a 32-bit number

// ------------------------------------------------------------------ merge

struct MergeParams {
  const float2* part_ml;
  const float* part_o;
  const int32_t* seq_lens;  // device lengths, only compared
  uint8_t* out;
  float* lse;
  int32_t* err;
  int out_type, n_qtok, n_kv_heads, n_q_heads, n_ctas;
  uint64_t len_inv;  // 2^64 / total_len, rounded up
  int weigh, prefix_len, total_len, suffix_row_tiles, suffix_rows, suffix_base;
  int32_t len[kMaxSeqs], start[kMaxSeqs], seq_at[kMaxSeqs];
  int16_t group[kMaxSeqs];  // a sequence's group, or -1
  int32_t group_first[kMaxGroups], group_seqs[kMaxGroups], group_keys[kMaxGroups], group_at[kMaxGroups],
      group_seg[kMaxGroups];
};

// The pieces of one segment: slot rows of one query row, `step` apart.
struct Pieces {
  long long row;
  int n, step;
};

// The CTA of place x, by a reciprocal: a 64-bit division per row and thread costs
// more than the row's sums.  The reciprocal is less than 1 too large, so the quotient
// is by less than num / 2^64: at most one.
__device__ __forceinline__ int cta_of(const MergeParams& p, int x) {
  const uint64_t num = ((uint64_t)x + 1) * (uint32_t)p.n_ctas - 1, q = __umul64hi(num, p.len_inv);
  return (int)q - (q * (uint32_t)p.total_len > num);
}

__device__ __forceinline__ Pieces pieces_of(const MergeParams& p, int at, int unit_rows, int in_unit, int nt, int seg,
                                            int step, int base, int r) {
  const Cost c = cost_of(p.weigh, unit_rows);
  at += in_unit * (c.lead + nt * c.tile) + c.lead;
  const int c0 = cta_of(p, at), c1 = cta_of(p, at + (nt - 1) * c.tile);
  return Pieces{base + (long long)(c0 + seg) * step + r, c1 - c0 + 1, step};
}

// One CTA per output row (pa_merge.cuh).
template <int G>
__global__ void __launch_bounds__(64 * G) pa_prefix_merge_kernel(const __grid_constant__ MergeParams p) {
  const int col = threadIdx.x & 63, grp = threadIdx.x >> 6;
  const int h = blockIdx.x, t = blockIdx.y, s = blockIdx.z;
  const int head = h / kGqa, hl = h % kGqa;
  Pieces a, b{0, 0, 0};
  {
    const int nt = ceil_div(p.len[s] - p.start[s], kKeys), rg = t * kGqa + hl, rt = rg / kRows;
    const int seg = (s * p.n_kv_heads + head) * p.suffix_row_tiles + rt;
    a = pieces_of(p, p.prefix_len + p.seq_at[s], kGqa * p.n_qtok, head * p.suffix_row_tiles + rt, nt, seg, p.suffix_rows,
                  p.suffix_base, rg % kRows);
  }
  const int g = p.group[s];
  if (g >= 0) {
    const int nt = ceil_div(p.group_keys[g], kKeys), rows = kGqa * p.n_qtok * p.group_seqs[g], nrt = ceil_div(rows, kRows);
    const int rg = ((s - p.group_first[g]) * p.n_qtok + t) * kGqa + hl, rt = rg / kRows;
    b = pieces_of(p, p.group_at[g], rows, head * nrt + rt, nt, p.group_seg[g] + head * nrt + rt, kRows, 0, rg % kRows);
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (threadIdx.x == 0) asm volatile("griddepcontrol.launch_dependents;");
  const int len_dev = __ldg(p.seq_lens + s);  // compared once the pieces are on their way
  Merged m;
  if (!merge_pieces<G>(p.part_ml, p.part_o, a.n + b.n,
                       [&](int i) { return i < a.n ? a.row + (long long)i * a.step : b.row + (long long)(i - a.n) * b.step; }, grp, col,
                       &m))
    return;
  const bool other = len_dev != p.len[s];
  if (other && threadIdx.x == 0) record_error(p.err, PA_ERR_BOUNDS);
  const long long row = ((long long)s * p.n_qtok + t) * p.n_q_heads + h;
  store_merged(m, other, p.out, p.out_type, row * kD, col, p.lse ? p.lse + row : nullptr);
}

// ------------------------------------------------------------------ host side

bool lookup_kernel(int kt, int vt, KernelInfo* out) {
#define PA_PAIR(k, v) \
  if (kt == k && vt == v) return lookup_prefix_kernel_##k##_##v(out);
  PA_PAIR(1, 1) PA_PAIR(1, 2) PA_PAIR(1, 8)
  PA_PAIR(2, 1) PA_PAIR(2, 2) PA_PAIR(2, 8)
  PA_PAIR(8, 1) PA_PAIR(8, 2) PA_PAIR(8, 8)
#undef PA_PAIR
  return false;
}

int type_slot(int t) { return t == PA_F16 ? 0 : t == PA_Q4_0 ? 1 : 2; }

constexpr int kMaxDevices = 64;
std::mutex g_mu;
int g_sms[kMaxDevices];
bool g_ready[kMaxDevices][3][3];  // the kernel's shared-memory limit is raised

// SM count of the device, and, with a kernel, its limit raised there (the
// device must be current for that).
pa_status device_ready(int device, int kt, int vt, const KernelInfo* ki, int* sms) {
  if (device < 0 || device >= kMaxDevices) return PA_ERR_INVALID;
  std::lock_guard<std::mutex> lk(g_mu);
  if (g_sms[device] == 0) {
    int v = 0;
    if (cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, device) != cudaSuccess) return PA_ERR_CUDA;
    g_sms[device] = v;
  }
  *sms = g_sms[device];
  if (ki) {
    bool& r = g_ready[device][type_slot(kt)][type_slot(vt)];
    if (!r && cudaFuncSetAttribute(ki->fn, cudaFuncAttributeMaxDynamicSharedMemorySize, ki->smem) != cudaSuccess)
      return PA_ERR_CUDA;
    r = true;
  }
  return PA_OK;
}

pa_status check_shape(const pa_pool* pool, uint32_t n_qtok, uint32_t n_q_heads, pa_pool_desc* d) {
  if (!pool || pa_pool_get_desc(pool, d) != PA_OK) return PA_ERR_INVALID;
  if (d->head_dim != (uint32_t)kD || n_qtok < 1 || n_qtok > kMaxQTok ||
      (uint64_t)n_q_heads != (uint64_t)d->n_kv_heads * kGqa)
    return PA_ERR_UNSUPPORTED;
  KernelInfo ki;
  return lookup_kernel(d->k_type, d->v_type, &ki) ? PA_OK : PA_ERR_UNSUPPORTED;
}

// Rows of a suffix segment's slot, and its row tiles.
int suffix_rows_of(uint32_t n_qtok) { return std::min<int>(kRows, kGqa * (int)n_qtok); }
int suffix_row_tiles_of(uint32_t n_qtok) { return ceil_div(kGqa * (int)n_qtok, kRows); }

struct WsLayout {
  size_t o, total;  // (m, l) at 0, O at o
};

WsLayout layout_of(int64_t slot_rows) {
  WsLayout w;
  w.o = ((size_t)slot_rows * sizeof(float2) + 255) & ~size_t(255);
  w.total = w.o + (size_t)slot_rows * kD * sizeof(float);
  return w;
}

// Slot rows for any batch of n_seq sequences in n_groups groups: a piece's slot
// is numbered CTA + segment, first the prefixes', then the suffixes'.
int64_t max_slot_rows(int sms, int64_t heads, uint32_t n_seq, uint32_t n_groups, uint32_t n_qtok) {
  const int64_t n = std::min<uint32_t>(n_seq, kMaxSeqs), g = std::min<int64_t>(n_groups, n);
  const int64_t prefix_segs = heads * ((int64_t)kGqa * n_qtok * n / kRows + g);
  const int64_t suffix_segs = heads * n * suffix_row_tiles_of(n_qtok);
  return (sms + prefix_segs) * kRows + (sms + suffix_segs) * suffix_rows_of(n_qtok);
}

struct Batch {  // what a call's sub-batches share
  pa_pool_desc d;
  const uint8_t* q;
  const void* k_pool;
  const void* v_pool;
  const int32_t* table;
  const int32_t* lens_dev;
  const int32_t* lens;
  uint8_t* out;
  float* lse;
  uint8_t* ws;
  size_t ws_bytes;
  int32_t* err;
  uint32_t table_stride, n_qtok;
  int q_type, out_type, sms;
  float scale;
};

// One launch pair over sequences c0 .. c0 + cn - 1; groups: (first sequence of
// the sub-batch, sequences in it, prefix length).
struct Group {
  int first, n, keys;
};

pa_status run_chunk(const Batch& b, uint32_t c0, uint32_t cn, const Group* groups, int n_groups, const KernelInfo& ki,
                    cudaStream_t cs) {
  static thread_local Params p;  // kept off the stack
  static thread_local MergeParams m;
  const int heads = (int)b.d.n_kv_heads, T = (int)b.n_qtok, srt = suffix_row_tiles_of(b.n_qtok);
  int64_t tiles = 0, segs = 0;
  int ng = 0;
  for (uint32_t i = 0; i < cn; ++i) {
    p.len[i] = m.len[i] = b.lens[c0 + i];
    p.start[i] = m.start[i] = 0;
    m.group[i] = -1;
  }
  for (int k = 0; k < n_groups; ++k) {
    const Group& g = groups[k];
    const int keys = g.keys & ~(kGroup - 1);
    if (g.n < 2 || keys == 0) continue;
    const int nrt = ceil_div(kGqa * T * g.n, kRows);
    int64_t with = (int64_t)nrt * ceil_div(keys, kKeys), without = 0;
    for (int i = g.first; i < g.first + g.n; ++i) {
      with += (int64_t)srt * ceil_div(p.len[i] - keys, kKeys);
      without += (int64_t)srt * ceil_div(p.len[i], kKeys);
    }
    if (with >= without) continue;
    for (int i = g.first; i < g.first + g.n; ++i) {
      p.start[i] = m.start[i] = keys;
      m.group[i] = (int16_t)ng;
    }
    p.group_first[ng] = m.group_first[ng] = g.first;
    p.group_seqs[ng] = m.group_seqs[ng] = g.n;
    p.group_keys[ng] = m.group_keys[ng] = keys;
    p.group_tile[ng] = (int32_t)tiles;
    p.group_seg[ng] = m.group_seg[ng] = (int32_t)segs;
    tiles += (int64_t)heads * nrt * ceil_div(keys, kKeys);
    segs += (int64_t)heads * nrt;
    if (tiles >= (1ll << 27)) return PA_ERR_UNSUPPORTED;
    ++ng;
  }
  for (uint32_t i = 0; i < cn; ++i) {
    p.seq_tile[i] = (int32_t)tiles;
    tiles += (int64_t)heads * srt * ceil_div(p.len[i] - p.start[i], kKeys);
    if (tiles >= (1ll << 27)) return PA_ERR_UNSUPPORTED;
  }
  const int ctas = (int)std::min<int64_t>(tiles, b.sms);
  // every CTA must have a tile: with weights its range is longer than a lead and
  // a tile
  const int weigh = tiles > 3 * ctas;
  int64_t at = 0;
  for (int k = 0; k < ng; ++k) {
    const int rows = kGqa * T * p.group_seqs[k];
    const Cost c = cost_of(weigh, rows);
    p.group_at[k] = m.group_at[k] = (int32_t)at;
    at += (int64_t)heads * ceil_div(rows, kRows) * (c.lead + ceil_div(p.group_keys[k], kKeys) * c.tile);
  }
  const int64_t prefix_len = at;
  const Cost c = cost_of(weigh, kGqa * T);
  for (uint32_t i = 0; i < cn; ++i) {
    p.seq_at[i] = m.seq_at[i] = (int32_t)(at - prefix_len);
    at += (int64_t)heads * srt * (c.lead + ceil_div(p.len[i] - p.start[i], kKeys) * c.tile);
  }
  if (at >= (1ll << 30)) return PA_ERR_UNSUPPORTED;
  const int64_t base = (ctas + segs) * kRows,
                rows = base + (ctas + (int64_t)heads * cn * srt) * suffix_rows_of(b.n_qtok);
  const WsLayout lay = layout_of(rows);
  if (lay.total > b.ws_bytes) return PA_ERR_INVALID;
  const size_t q_row = (size_t)T * heads * kGqa * kD;  // values of a sequence
  p.q = b.q + c0 * q_row * dtype_bytes(b.q_type);
  p.k_pool = static_cast<const uint8_t*>(b.k_pool);
  p.v_pool = static_cast<const uint8_t*>(b.v_pool);
  p.table = b.table + (size_t)c0 * b.table_stride;
  p.err = m.err = b.err;
  p.part_ml = reinterpret_cast<float2*>(b.ws);
  p.part_o = reinterpret_cast<float*>(b.ws + lay.o);
  p.q_type = b.q_type;
  p.n_qtok = m.n_qtok = T;
  p.n_kv_heads = m.n_kv_heads = heads;
  p.n_q_heads = m.n_q_heads = heads * kGqa;
  p.page_size = (int)b.d.page_size;
  p.page_shift = -1;
  for (int i = 4; i < 31; ++i)
    if (b.d.page_size == 1u << i) p.page_shift = i;
  p.table_stride = (int)b.table_stride;
  p.n_blocks = (int)b.d.n_blocks;
  p.n_seq = (int)cn;
  p.n_groups = ng;
  p.n_ctas = m.n_ctas = ctas;
  p.weigh = m.weigh = weigh;
  p.total_tiles = (int)tiles;
  m.len_inv = ~0ull / (uint64_t)at + 1;
  p.prefix_len = m.prefix_len = (int32_t)prefix_len;
  p.total_len = m.total_len = (int32_t)at;
  p.suffix_row_tiles = m.suffix_row_tiles = srt;
  p.suffix_rows = m.suffix_rows = suffix_rows_of(b.n_qtok);
  p.suffix_base = m.suffix_base = (int32_t)base;
  p.scale_log2 = b.scale * kLog2e;
  m.part_ml = p.part_ml;
  m.part_o = p.part_o;
  m.seq_lens = b.lens_dev + c0;
  m.out = b.out + c0 * q_row * dtype_bytes(b.out_type);
  m.lse = b.lse ? b.lse + (size_t)c0 * T * heads * kGqa : nullptr;
  m.out_type = b.out_type;
  // Both are programmatic dependents of what runs before them on the stream:
  // their set-up overlaps its tail, and they wait for it before they read.
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = (size_t)ki.smem;
  cfg.stream = cs;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, ki.fn, p) != cudaSuccess) return PA_ERR_CUDA;
  cfg.gridDim = dim3((unsigned)(heads * kGqa), (unsigned)T, cn);
  const int wide = merge_groups((int64_t)cn * T * heads * kGqa, b.sms);
  cfg.blockDim = dim3(64 * wide);
  cfg.dynamicSmemBytes = 0;
  const auto merge = wide == 8   ? pa_prefix_merge_kernel<8>
                     : wide == 4 ? pa_prefix_merge_kernel<4>
                     : wide == 2 ? pa_prefix_merge_kernel<2>
                                   : pa_prefix_merge_kernel<1>;
  return cudaLaunchKernelEx(&cfg, merge, m) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace

extern "C" size_t pa_decode_prefix_workspace_size(const pa_pool* pool, uint32_t n_seq, uint32_t n_groups,
                                                  uint32_t n_qtok, int device) {
  pa_pool_desc d;
  if (!pool || pa_pool_get_desc(pool, &d) != PA_OK) return 0;
  if (check_shape(pool, n_qtok, d.n_kv_heads * kGqa, &d) != PA_OK) return 0;
  int sms = 0;
  if (device_ready(device, d.k_type, d.v_type, nullptr, &sms) != PA_OK) return 0;
  return layout_of(max_slot_rows(sms, d.n_kv_heads, n_seq, n_groups, n_qtok)).total;
}

extern "C" pa_status pa_decode_prefix(const pa_pool* pool, const void* q, int32_t q_type, const void* k_pool,
                                      const void* v_pool, const int32_t* block_table, uint32_t table_stride,
                                      const int32_t* seq_lens_dev, const int32_t* seq_lens_host, uint32_t n_seq,
                                      const uint32_t* group_sizes, const int32_t* prefix_lens, uint32_t n_groups,
                                      uint32_t n_qtok, uint32_t n_q_heads, float scale, void* out, int32_t out_type,
                                      float* lse, void* workspace, size_t ws_bytes, int32_t* err,
                                      pa_stream_t stream) {
  Batch b;
  pa_status st = check_shape(pool, n_qtok, n_q_heads, &b.d);
  if (st != PA_OK) return st;
  if (!dtype_bytes(q_type) || !dtype_bytes(out_type)) return PA_ERR_UNSUPPORTED;
  if (n_seq == 0) return n_groups == 0 ? PA_OK : PA_ERR_INVALID;
  if (!q || !k_pool || !v_pool || !block_table || !seq_lens_dev || !seq_lens_host || !group_sizes || !prefix_lens ||
      !out || !workspace || !err || table_stride == 0 || table_stride > 0x7fffffffu || n_groups == 0 || n_groups > n_seq)
    return PA_ERR_INVALID;
  if (((uintptr_t)q | (uintptr_t)out | (uintptr_t)k_pool | (uintptr_t)v_pool) & 15) return PA_ERR_INVALID;
  if ((uintptr_t)workspace & 255) return PA_ERR_INVALID;
  if (!(scale > 0.f) || !std::isfinite(scale)) return PA_ERR_INVALID;
  // every length and group is checked before the first launch
  uint64_t at = 0;
  for (uint32_t g = 0; g < n_groups; ++g) {
    const uint64_t end = at + group_sizes[g];
    if (group_sizes[g] == 0 || end > n_seq || prefix_lens[g] < 0) return PA_ERR_INVALID;
    for (; at < end; ++at) {
      const int64_t L = seq_lens_host[at];
      if (L > kMaxLen) return PA_ERR_UNSUPPORTED;
      if (L < (int64_t)n_qtok || L > (int64_t)table_stride * b.d.page_size || prefix_lens[g] > L - (int64_t)n_qtok)
        return PA_ERR_INVALID;
    }
  }
  if (at != n_seq) return PA_ERR_INVALID;
  int device = 0;
  if (cudaGetDevice(&device) != cudaSuccess) return PA_ERR_CUDA;
  KernelInfo ki;
  lookup_kernel(b.d.k_type, b.d.v_type, &ki);
  st = device_ready(device, b.d.k_type, b.d.v_type, &ki, &b.sms);
  if (st != PA_OK) return st;
  if (ws_bytes < layout_of(max_slot_rows(b.sms, b.d.n_kv_heads, n_seq, n_groups, n_qtok)).total) return PA_ERR_INVALID;
  b.q = static_cast<const uint8_t*>(q);
  b.k_pool = k_pool;
  b.v_pool = v_pool;
  b.table = block_table;
  b.lens_dev = seq_lens_dev;
  b.lens = seq_lens_host;
  b.out = static_cast<uint8_t*>(out);
  b.lse = lse;
  b.ws = static_cast<uint8_t*>(workspace);
  b.ws_bytes = ws_bytes;
  b.err = err;
  b.table_stride = table_stride;
  b.n_qtok = n_qtok;
  b.q_type = q_type;
  b.out_type = out_type;
  b.scale = scale;
  // Sub-batches in order on the stream, sharing the workspace: each one's first
  // kernel waits for the one before to complete.
  Group groups[kMaxSeqs];
  uint32_t g = 0, used = 0;  // the group being cut, its sequences already taken
  for (uint32_t c0 = 0; c0 < n_seq; c0 += kMaxSeqs) {
    const uint32_t cn = std::min<uint32_t>(kMaxSeqs, n_seq - c0);
    int n = 0;
    for (uint32_t i = 0; i < cn;) {
      const uint32_t take = std::min<uint32_t>(group_sizes[g] - used, cn - i);
      groups[n++] = Group{(int)i, (int)take, prefix_lens[g]};
      i += take;
      used += take;
      if (used == group_sizes[g]) {
        ++g;
        used = 0;
      }
    }
    st = run_chunk(b, c0, cn, groups, n, ki, reinterpret_cast<cudaStream_t>(stream));
    if (st != PA_OK) return st;
  }
  return PA_OK;
}
