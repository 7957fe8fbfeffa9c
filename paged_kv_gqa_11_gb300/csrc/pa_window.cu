// Attention over a sliding window and first keys: the plan, the merge of the segments that
// are cut, and the host side of pa_attend_window.  The kernel over the keys is in
// pa_window_impl.cuh and pa_prefix_impl.cuh, compiled once per (K format, V format) pair.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "pa_io.cuh"
#include "pa_merge.cuh"
#include "pa_window_impl.cuh"

using namespace pa_dev;
using namespace pa_prefix;
using pa_split::kLog2e;

namespace {

constexpr int64_t kMaxLen = 0x7fffffff - 2 * kKeys;  // a tile past the last key is still a 32-bit number
constexpr uint32_t kMaxNew = 1u << 24;               // new tokens of a sequence
constexpr int kMaxCtas = 256;
constexpr int64_t kMaxPlaces = 1ll << 30;

// ------------------------------------------------------------------ merge

struct Cut {  // a segment of several pieces: those of CTAs cta .. cta + n - 1
  int32_t seq, len, token, rows_row0, head, cta, n;
};

struct MergeParams {
  const float2* part_ml;
  const float* part_o;
  const int32_t* lens;  // device lengths, only compared
  uint8_t* out;
  float* lse;
  int32_t* err;
  long long out_stride;
  int out_type, n_q_heads, slot_rows;
  Cut cut[kMaxCtas];
};

// A CTA per row of a cut segment (pa_merge.cuh).
template <int G>
__global__ void __launch_bounds__(64 * G) pa_window_merge_kernel(const __grid_constant__ MergeParams p) {
  const int col = threadIdx.x & 63, grp = threadIdx.x >> 6;
  const Cut& c = p.cut[blockIdx.x];
  const int r = blockIdx.y;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (threadIdx.x == 0) asm volatile("griddepcontrol.launch_dependents;");
  if (r >= (c.rows_row0 & 0xff)) return;
  const bool other = __ldg(p.lens + c.seq) != c.len;
  const long long slot = 2ll * c.cta * p.slot_rows + r;
  Merged m;
  // the first piece ends its CTA's range (the second slot), the others begin theirs
  if (!merge_pieces<G>(p.part_ml, p.part_o, c.n, [&](int i) { return slot + (i == 0 ? 1ll : 2ll * i) * p.slot_rows; }, grp, col, &m))
    return;
  if (other && threadIdx.x == 0) record_error(p.err, PA_ERR_BOUNDS);
  const int rg = (c.rows_row0 >> 8) + r, h = c.head * kGqa + rg % kGqa;
  const long long token = c.token + rg / kGqa;
  store_merged(m, other, p.out, p.out_type, token * p.out_stride + h * kD, col, p.lse ? p.lse + token * p.n_q_heads + h : nullptr);
}

// ------------------------------------------------------------------ host side

bool lookup_kernel(int kt, int vt, WindowKernel* out) {
#define PA_PAIR(k, v) \
  if (kt == k && vt == v) return lookup_window_kernel_##k##_##v(out);
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

// CTAs of a launch on the device (one per SM), and, with a kernel, its limit raised there
// (the device must be current for that).
pa_status device_ready(int device, int kt, int vt, const WindowKernel* ki, int* ctas) {
  if (device < 0 || device >= kMaxDevices) return PA_ERR_INVALID;
  std::lock_guard<std::mutex> lk(g_mu);
  if (g_sms[device] == 0) {
    int v = 0;
    if (cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, device) != cudaSuccess) return PA_ERR_CUDA;
    g_sms[device] = v;
  }
  *ctas = std::min(g_sms[device], kMaxCtas);
  if (ki) {
    bool& r = g_ready[device][type_slot(kt)][type_slot(vt)];
    if (!r && cudaFuncSetAttribute(ki->fn, cudaFuncAttributeMaxDynamicSharedMemorySize, ki->smem) != cudaSuccess)
      return PA_ERR_CUDA;
    r = true;
  }
  return PA_OK;
}

struct WsLayout {
  size_t o, total;  // (m, l) at 0, O at o
};

// Two slots for each CTA, of the rows of the largest unit.
int slot_rows_of(uint32_t max_new) { return (int)std::min<uint64_t>(kRows, (uint64_t)kGqa * max_new); }

WsLayout layout_of(int ctas, uint32_t max_new) {
  const size_t rows = 2 * (size_t)ctas * slot_rows_of(max_new);
  WsLayout w;
  w.o = (rows * sizeof(float2) + 255) & ~size_t(255);
  w.total = w.o + rows * kD * sizeof(float);
  return w;
}

// The units of the batch in order: sequence s's rows 64 rt .. of 6 n.
struct Cursor {
  uint32_t seq;
  int rt;
  int token;  // of the sequence's first row
};

int tiles_of(const Unit& u, int window, int sinks) { return ceil_div(span_of(u, window, sinks).end, kKeys); }

// What a launch takes of the units from `at` on, which it moves: p's units, ranges and m's
// cuts.
struct Plan {
  int cuts, rows;  // cut segments, rows of the largest
};

Plan plan_chunk(WindowParams& p, MergeParams& m, const int32_t* lens, const int32_t* n_new, uint32_t n_seq, int max_ctas, Cursor* at) {
  const int heads = p.n_kv_heads;
  int64_t tiles = 0;
  p.n_units = 0;
  for (; at->seq < n_seq && p.n_units < kMaxUnits; at->token += n_new[at->seq++], at->rt = 0) {
    const int rows = kGqa * n_new[at->seq];
    for (; at->rt * kRows < rows && p.n_units < kMaxUnits; ++at->rt) {
      const int row = at->rt * kRows;
      Unit& u = p.unit[p.n_units];
      u.seq = (int32_t)at->seq;
      u.token = at->token + row / kGqa;
      u.len = lens[at->seq];
      u.pos = u.len - n_new[at->seq] + row / kGqa;
      u.rows_row0 = std::min(kRows, rows - row) | (row % kGqa) << 8;
      u.tile = (int32_t)tiles;
      const int64_t more = tiles + (int64_t)heads * tiles_of(u, p.window, p.sinks);
      if (p.n_units > 0 && more > (kMaxPlaces >> 5)) break;  // the next launch's
      tiles = more;
      ++p.n_units;
    }
    if (at->rt * kRows < rows) break;
  }
  if (p.n_units == 0) return Plan{0, 0};
  p.total_tiles = (int)tiles;
  p.n_ctas = (int)std::min<int64_t>(tiles, max_ctas);
  // every CTA must have a tile: with weights its range is longer than a lead and a tile
  p.weigh = tiles > 3 * p.n_ctas;
  int64_t places = 0;
  for (int i = 0; i < p.n_units; ++i) {
    Unit& u = p.unit[i];
    const Cost c = cost_of(p.weigh, unit_rows(u));
    u.at = (int32_t)places;
    places += (int64_t)heads * (c.lead + (int64_t)tiles_of(u, p.window, p.sinks) * c.tile);
  }
  p.total_len = (int)places;
  int cuts = 0, rows = 0, unit = -1, head = -1;
  for (int c = 1; c < p.n_ctas; ++c) {
    const Pos t = locate(p, (int)((long long)c * p.total_len / p.n_ctas));
    if (t.j == 0) continue;  // the range begins with a segment
    if (t.unit == unit && t.head == head) {
      ++m.cut[cuts - 1].n;
      continue;
    }
    unit = t.unit;
    head = t.head;
    const Unit& u = p.unit[unit];
    m.cut[cuts++] = Cut{u.seq, u.len, u.token, u.rows_row0, head, c - 1, 2};
    rows = std::max(rows, unit_rows(u));
  }
  return Plan{cuts, rows};
}

pa_status launch_chunk(const WindowParams& p, const MergeParams& m, const Plan& plan, const WindowKernel& ki, int max_ctas,
                       cudaStream_t cs) {
  if (p.n_units == 0) return PA_OK;
  // Both are programmatic dependents of what runs before them on the stream: their set-up
  // overlaps its tail, and they wait for it before they read.
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.n_ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = (size_t)ki.smem;
  cfg.stream = cs;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, ki.fn, p) != cudaSuccess) return PA_ERR_CUDA;
  if (plan.cuts == 0) return PA_OK;
  const int wide = merge_groups((int64_t)plan.cuts * plan.rows, max_ctas);
  cfg.gridDim = dim3((unsigned)plan.cuts, (unsigned)plan.rows);
  cfg.blockDim = dim3(64 * wide);
  cfg.dynamicSmemBytes = 0;
  const auto merge = wide == 8   ? pa_window_merge_kernel<8>
                     : wide == 4 ? pa_window_merge_kernel<4>
                     : wide == 2 ? pa_window_merge_kernel<2>
                                 : pa_window_merge_kernel<1>;
  return cudaLaunchKernelEx(&cfg, merge, m) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

pa_status check_pool(const pa_pool* pool, pa_pool_desc* d, WindowKernel* ki) {
  if (!pool || pa_pool_get_desc(pool, d) != PA_OK) return PA_ERR_INVALID;
  return d->head_dim == (uint32_t)kD && lookup_kernel(d->k_type, d->v_type, ki) ? PA_OK : PA_ERR_UNSUPPORTED;
}

}  // namespace

extern "C" size_t pa_attend_window_workspace_size(const pa_pool* pool, uint32_t max_new, int device) {
  pa_pool_desc d;
  WindowKernel ki;
  int ctas = 0;
  if (check_pool(pool, &d, &ki) != PA_OK || device_ready(device, d.k_type, d.v_type, nullptr, &ctas) != PA_OK) return 0;
  return layout_of(ctas, max_new).total;
}

extern "C" pa_status pa_attend_window(const pa_pool* pool, const void* q, int64_t q_stride, int32_t q_type, const void* k_pool,
                                      const void* v_pool, const int32_t* block_table, uint32_t table_stride,
                                      const int32_t* seq_lens_dev, const int32_t* seq_lens_host, const int32_t* n_new,
                                      uint32_t n_seq, uint32_t n_q_heads, uint32_t window, uint32_t sinks, float scale,
                                      void* out, int64_t out_stride, int32_t out_type, float* lse, void* workspace,
                                      size_t ws_bytes, int32_t* err, pa_stream_t stream) {
  pa_pool_desc d;
  WindowKernel ki;
  pa_status st = check_pool(pool, &d, &ki);
  if (st != PA_OK) return st;
  if ((uint64_t)n_q_heads != (uint64_t)d.n_kv_heads * kGqa) return PA_ERR_UNSUPPORTED;
  if (!dtype_bytes(q_type) || !dtype_bytes(out_type)) return PA_ERR_UNSUPPORTED;
  if (n_seq == 0) return PA_OK;
  if (!seq_lens_host || !n_new) return PA_ERR_INVALID;
  if (!(scale > 0.f) || !std::isfinite(scale)) return PA_ERR_INVALID;
  const int w = window == 0 ? kAllKeys : (int)std::min<uint32_t>(window, kAllKeys), s = (int)std::min<uint32_t>(sinks, kAllKeys);
  // every length is checked before the first launch
  uint64_t tokens = 0;
  uint32_t most = 0;
  for (uint32_t i = 0; i < n_seq; ++i) {
    const int64_t len = seq_lens_host[i], n = n_new[i];
    if (n < 0 || len < n || len > (int64_t)table_stride * d.page_size) return PA_ERR_INVALID;
    if (n > kMaxNew || len > kMaxLen) return PA_ERR_UNSUPPORTED;
    tokens += (uint64_t)n;
    most = std::max(most, (uint32_t)n);
    if (n > 0) {  // one unit fits a launch: its window is at most that long
      const int64_t keys = std::min<int64_t>(len, (int64_t)w + (int64_t)s + 4 * kKeys);
      if (d.n_kv_heads * (kLead + (keys / kKeys + 1) * (kTileCost + 2)) >= kMaxPlaces) return PA_ERR_UNSUPPORTED;
    }
  }
  if (tokens == 0) return PA_OK;
  if (tokens > 0x7fffffffu) return PA_ERR_UNSUPPORTED;
  if (!q || !k_pool || !v_pool || !block_table || !seq_lens_dev || !out || !workspace || !err || table_stride == 0 ||
      table_stride > 0x7fffffffu)
    return PA_ERR_INVALID;
  if (((uintptr_t)q | (uintptr_t)out | (uintptr_t)k_pool | (uintptr_t)v_pool) & 15) return PA_ERR_INVALID;
  if ((uintptr_t)workspace & 255) return PA_ERR_INVALID;
  for (int i = 0; i < 2; ++i) {  // rows 16-byte aligned, none inside another's heads
    const int64_t stride = i ? out_stride : q_stride;
    if (stride < (int64_t)n_q_heads * kD || stride > (int64_t(1) << 40) || (stride * dtype_bytes(i ? out_type : q_type)) % 16)
      return PA_ERR_INVALID;
  }
  int device = 0, ctas = 0;
  if (cudaGetDevice(&device) != cudaSuccess) return PA_ERR_CUDA;
  st = device_ready(device, d.k_type, d.v_type, &ki, &ctas);
  if (st != PA_OK) return st;
  const WsLayout lay = layout_of(ctas, most);
  if (ws_bytes < lay.total) return PA_ERR_INVALID;
  static thread_local WindowParams p;  // kept off the stack
  static thread_local MergeParams m;
  p.q = static_cast<const uint8_t*>(q);
  p.k_pool = static_cast<const uint8_t*>(k_pool);
  p.v_pool = static_cast<const uint8_t*>(v_pool);
  p.table = block_table;
  p.lens = m.lens = seq_lens_dev;
  p.err = m.err = err;
  m.part_ml = p.part_ml = static_cast<float2*>(workspace);
  m.part_o = p.part_o = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + lay.o);
  p.out = m.out = static_cast<uint8_t*>(out);
  p.lse = m.lse = lse;
  p.q_stride = q_stride;
  p.out_stride = m.out_stride = out_stride;
  p.q_type = q_type;
  p.out_type = m.out_type = out_type;
  p.n_kv_heads = (int)d.n_kv_heads;
  p.n_q_heads = m.n_q_heads = (int)n_q_heads;
  p.page_size = (int)d.page_size;
  p.page_shift = -1;
  for (int i = 4; i < 31; ++i)
    if (d.page_size == 1u << i) p.page_shift = i;
  p.table_stride = (int)table_stride;
  p.n_blocks = (int)d.n_blocks;
  p.window = w;
  p.sinks = s;
  p.slot_rows = m.slot_rows = slot_rows_of(most);
  p.scale_log2 = scale * kLog2e;
  // Launches in order on the stream, sharing the workspace: each one's kernel waits for the
  // one before to complete.
  Cursor at{0, 0, 0};
  while (at.seq < n_seq) {
    const Plan plan = plan_chunk(p, m, seq_lens_host, n_new, n_seq, ctas, &at);
    st = launch_chunk(p, m, plan, ki, ctas, reinterpret_cast<cudaStream_t>(stream));
    if (st != PA_OK) return st;
  }
  return PA_OK;
}
