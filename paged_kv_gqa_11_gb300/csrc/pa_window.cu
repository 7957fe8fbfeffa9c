// Attention over a sliding window and first keys: the plan, the merge of the segments that
// are cut, and the host side of pa_attend_window.  The kernel over the keys for sequences with few
// new tokens is in pa_window_impl.cuh and pa_prefix_impl.cuh, compiled once per (K format,
// V format) pair, that for large batches of single tokens in pa_step_impl.cuh, the kernels for
// sequences with many tokens in pa_prompt.cu.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "pa_io.cuh"
#include "pa_merge.cuh"
#include "pa_prompt.cuh"
#include "pa_step.cuh"
#include "pa_window_impl.cuh"

using namespace pa_dev;
using namespace pa_prefix;
using pa_split::kLog2e;

namespace {

constexpr int64_t kMaxLen = 0x7fffffff - 2 * kKeys;  // a tile past the last key is still a 32-bit number
constexpr uint32_t kMaxNew = 1u << 24;               // new tokens of a sequence
constexpr int64_t kMaxPlaces = 1ll << 30;
// Sequences of so many new tokens or more are the prompts' kernel's, which turns the keys into binary16 first.
// 63 tokens by the kernel of few and 64 by the prompts', us, without a window, sequences x keys:
//          1 x 512      1 x 4096     1 x 32768  1 x 131072  4 x 4096     4 x 32768  16 x 2048
//   Q4_0   13.6, 17.6   24.5, 33.2   83, 107    280, 354    58.6, 65.7   286, 388   112, 108
//   Q8_0   14.2, 18.3   31.1, 33.8   133, 118   400, 385    83.9, 74.8   409, 401   159, 121
//   F16    13.1, 17.5   23.8, 32.5   105, 96    462, 325    54.1, 61.2   468, 371   122, 99
// The two pass each other near here for Q8_0 and F16 keys; with Q4_0 keys, and over short contexts, the kernel of few is
// still up to a quarter faster at 63 tokens.  2048 tokens, window 1024: 161 us and 59.
constexpr int32_t kPromptTokens = 64;

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

// Rows of a cut segment by groups of G times 64 threads (pa_merge.cuh), kMergeRows / G of them to a
// CTA.
constexpr int kMergeRows = 8;

template <int G>
__global__ void __launch_bounds__(64 * kMergeRows) pa_window_merge_kernel(const __grid_constant__ MergeParams p) {
  const int col = threadIdx.x & 63, grp = (threadIdx.x >> 6) % G, in_cta = (threadIdx.x >> 6) / G;
  const Cut& c = p.cut[blockIdx.x];
  const int r = (int)blockIdx.y * (kMergeRows / G) + in_cta;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (threadIdx.x == 0) asm volatile("griddepcontrol.launch_dependents;");
  const bool mine = r < (c.rows_row0 & 0xffff);
  const bool other = __ldg(p.lens + c.seq) != c.len;
  const long long slot = 2ll * c.cta * p.slot_rows + r;
  Merged m;
  // the first piece ends its CTA's range (the second slot), the others begin theirs
  if (!merge_pieces<G, kMergeRows / G>(p.part_ml, p.part_o, mine ? c.n : 0,
                                       [&](int i) { return slot + (i == 0 ? 1ll : 2ll * i) * p.slot_rows; }, grp, col, &m, in_cta) ||
      !mine)
    return;
  if (other && col == 0) record_error(p.err, PA_ERR_BOUNDS);
  const int rg = (c.rows_row0 >> 16) + r, h = c.head * kGqa + rg % kGqa;
  const long long token = c.token + rg / kGqa;
  store_merged(m, other, p.out, p.out_type, token * p.out_stride + h * kD, col, p.lse ? p.lse + token * p.n_q_heads + h : nullptr);
}

// ------------------------------------------------------------------ host side

struct Kernels {  // of a (K format, V format) pair
  WindowKernel few;
  StepKernel step;
};

bool lookup_kernels(int kt, int vt, Kernels* out) {
#define PA_PAIR(k, v) \
  if (kt == k && vt == v) return lookup_window_kernel_##k##_##v(&out->few) && lookup_step_kernel_##k##_##v(&out->step);
  PA_PAIR(1, 1) PA_PAIR(1, 2) PA_PAIR(1, 8)
  PA_PAIR(2, 1) PA_PAIR(2, 2) PA_PAIR(2, 8)
  PA_PAIR(8, 1) PA_PAIR(8, 2) PA_PAIR(8, 8)
#undef PA_PAIR
  return false;
}

int type_slot(int t) { return t == PA_F16 ? 0 : t == PA_Q4_0 ? 1 : 2; }

// Every launch is a programmatic dependent of what runs before it on the stream: its set-up
// overlaps the other's tail, and it waits for it before it reads.
struct Launch {
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = {};
  explicit Launch(cudaStream_t cs) {
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.stream = cs;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
  }
};

// A launch of pa_step_kernel over `segments` clusters.
void set_steps(Launch& l, const StepKernel& ki, int cluster, int segments) {
  l.attr[1].id = cudaLaunchAttributeClusterDimension;
  l.attr[1].val.clusterDim.x = (unsigned)cluster;
  l.attr[1].val.clusterDim.y = l.attr[1].val.clusterDim.z = 1;
  l.cfg.numAttrs = 2;
  l.cfg.gridDim = dim3((unsigned)(segments * cluster));
  l.cfg.blockDim = dim3(kStepThreads);
  l.cfg.dynamicSmemBytes = (size_t)ki.smem;
}

// Clusters of pa_step_kernel that the device holds at once, of 1, 2, 4 and 8 CTAs.
struct StepFit {
  int clusters[4];
};

constexpr int kMaxDevices = 64;
std::mutex g_mu;
int g_sms[kMaxDevices];
bool g_ready[kMaxDevices][3][3];  // the kernels' shared-memory limits are raised
StepFit g_fit[kMaxDevices][3][3];

// CTAs of a launch on the device (one per SM), and, with a kernel, its limit raised there
// (the device must be current for that) and what the device holds of the step kernel.
pa_status device_ready(int device, int kt, int vt, const Kernels* ki, int* ctas, StepFit* fit = nullptr) {
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
    if (!r && (cudaFuncSetAttribute(ki->few.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, ki->few.smem) != cudaSuccess ||
               (ki->step.fn && cudaFuncSetAttribute(ki->step.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, ki->step.smem) != cudaSuccess) ||
               prompt_ready() != PA_OK))
      return PA_ERR_CUDA;
    StepFit& f = g_fit[device][type_slot(kt)][type_slot(vt)];
    for (int i = 0; i < 4 && !r && ki->step.fn; ++i) {
      Launch l(nullptr);
      set_steps(l, ki->step, 1 << i, 1);
      l.cfg.attrs = l.attr + 1;  // the cluster alone
      l.cfg.numAttrs = 1;
      if (cudaOccupancyMaxActiveClusters(&f.clusters[i], ki->step.fn, &l.cfg) != cudaSuccess) return PA_ERR_CUDA;
    }
    r = true;
    if (fit) *fit = f;
  }
  return PA_OK;
}

// What a batch needs, its lengths checked.
struct Batch {
  const int32_t* lens;
  const int32_t* n_new;
  uint32_t n_seq;
  int window, sinks, heads;
  uint64_t tokens;
  uint32_t most;        // new tokens of the largest sequence of few
  uint32_t prompts;     // sequences of many
  int64_t groups;       // row groups for their keys
  int64_t few, keys, longest;  // sequences of few, keys that they read, and the longest's
  bool many(uint32_t s) const { return is_many(n_new[s]); }
  static bool is_many(int32_t n) { return n >= kPromptTokens; }
};

pa_status check_batch(const pa_pool_desc& d, uint64_t max_len, Batch* b) {
  b->tokens = 0;
  b->most = b->prompts = 0;
  b->groups = b->few = b->keys = b->longest = 0;
  for (uint32_t i = 0; i < b->n_seq; ++i) {
    const int64_t len = b->lens[i], n = b->n_new[i];
    if (n < 0 || len < n || len > (int64_t)max_len) return PA_ERR_INVALID;
    if (n > kMaxNew || len > kMaxLen) return PA_ERR_UNSUPPORTED;
    if (n == 0) continue;
    b->tokens += (uint64_t)n;
    // one unit fits a launch: its window is at most that long
    const int64_t keys = std::min<int64_t>(len, (int64_t)b->window + (int64_t)b->sinks + 4 * kKeys);
    if (d.n_kv_heads * (kLead + (keys / kKeys + 1) * (kTileCost + 2)) >= kMaxPlaces) return PA_ERR_UNSUPPORTED;
    if (b->many(i)) {
      ++b->prompts;
      b->groups += room_for(len, n, b->window, b->sinks);
    } else {
      b->most = std::max(b->most, (uint32_t)n);
      const int64_t seen = std::min<int64_t>(len, (int64_t)b->window + (int64_t)b->sinks + n - 1);
      ++b->few;
      b->keys += seen;
      b->longest = std::max(b->longest, seen);
    }
  }
  return b->tokens > 0x7fffffffu || b->groups > 0x7fffffff / 16 ? PA_ERR_UNSUPPORTED : PA_OK;
}

// The workspace: two slots of (m, l) and O for each CTA, of the rows of the largest unit, the same for the
// kernel of few tokens and, when that and its merge are done, that of many; the many's keys, values and which
// keys are wide.  More of anything in a batch needs no less: the slots of a unit of many (256 rows for a pair of
// CTAs) are larger than those of the largest of few (64 for a CTA), and the keys' room only grows (room_for).
struct WsLayout {
  size_t o, k, v, wide, total;  // the (m, l) at 0
};

int slot_rows_of(uint32_t max_new) { return (int)std::min<uint64_t>(kRows, (uint64_t)kGqa * max_new); }

WsLayout layout_of(int ctas, const Batch& b) {
  const size_t few = 2 * (size_t)ctas * slot_rows_of(b.most), many = b.prompts ? 2 * (size_t)(ctas / 2) * kPromptRows : 0;
  const size_t rows = std::max(few, many);
  const size_t keys = (size_t)b.groups * b.heads * kGroupBytes;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t from = at;
    at += (bytes + 255) & ~size_t(255);
    return from;
  };
  WsLayout w;
  take(rows * sizeof(float2));
  w.o = take(rows * kD * sizeof(float));
  w.k = take(keys);
  w.v = take(keys);
  w.wide = take((size_t)b.groups * b.heads * 2);
  w.total = at;
  return w;
}

// The units of the batch in order: rows P::kUnitRows rt .. of the 6 n of sequence s.
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

template <class P>
Plan plan_chunk(P& p, MergeParams& m, const Batch& b, bool many, int max_ctas, Cursor* at) {
  const int32_t* const lens = b.lens;
  const int32_t* const n_new = b.n_new;
  const int heads = p.n_kv_heads;
  int64_t tiles = 0;
  p.n_units = 0;
  for (; at->seq < b.n_seq && p.n_units < P::kMaxUnits; at->token += n_new[at->seq++], at->rt = 0) {
    const int rows = b.many(at->seq) == many ? kGqa * n_new[at->seq] : 0;
    for (; at->rt * P::kUnitRows < rows && p.n_units < P::kMaxUnits; ++at->rt) {
      const int row = at->rt * P::kUnitRows;
      Unit& u = p.unit[p.n_units];
      u.seq = (int32_t)at->seq;
      u.token = at->token + row / kGqa;
      u.len = lens[at->seq];
      u.pos = u.len - n_new[at->seq] + row / kGqa;
      u.rows_row0 = std::min(P::kUnitRows, rows - row) | (row % kGqa) << 16;
      u.tile = (int32_t)tiles;
      const int64_t more = tiles + (int64_t)heads * tiles_of(u, p.window, p.sinks);
      if (p.n_units > 0 && more > (kMaxPlaces >> 5)) break;  // the next launch's
      tiles = more;
      ++p.n_units;
    }
    if (at->rt * P::kUnitRows < rows) break;
  }
  if (p.n_units == 0) return Plan{0, 0};
  p.total_tiles = (int)tiles;
  p.n_ctas = (int)std::min<int64_t>(tiles, max_ctas);
  // Every CTA must have a tile: with weights its range is at least as long as a lead and a tile.
  int64_t places = 0;
  for (p.weigh = tiles > 3 * p.n_ctas;; p.weigh = 0) {
    places = 0;
    int most = 0;
    for (int i = 0; i < p.n_units; ++i) {
      Unit& u = p.unit[i];
      const Cost c = cost_of(p, u);
      u.at = (int32_t)places;
      places += (int64_t)heads * (c.lead + (int64_t)tiles_of(u, p.window, p.sinks) * c.tile);
      most = std::max(most, c.lead + c.tile);
    }
    if (!p.weigh || places / p.n_ctas >= most) break;
  }
  p.total_len = (int)places;
  int cuts = 0, rows = 0, unit = -1, head = -1;
  p.start[p.n_ctas] = Start{0, 0, p.total_tiles};
  for (int c = 0; c < p.n_ctas; ++c) {
    const Pos t = locate(p, (int)((long long)c * p.total_len / p.n_ctas));
    p.start[c] = Start{t.unit | t.head << 16, t.j, t.tile};
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

pa_status launch_few(const WindowParams& p, const WindowKernel& ki, cudaStream_t cs) {
  Launch l(cs);
  l.cfg.gridDim = dim3((unsigned)p.n_ctas);
  l.cfg.blockDim = dim3(kThreads);
  l.cfg.dynamicSmemBytes = (size_t)ki.smem;
  return cudaLaunchKernelEx(&l.cfg, ki.fn, p) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

pa_status launch_merge(const MergeParams& m, const Plan& plan, int max_ctas, cudaStream_t cs) {
  if (plan.cuts == 0) return PA_OK;
  Launch l(cs);
  const int wide = merge_groups((int64_t)plan.cuts * plan.rows, max_ctas);
  l.cfg.gridDim = dim3((unsigned)plan.cuts, (unsigned)ceil_div(plan.rows, kMergeRows / wide));
  l.cfg.blockDim = dim3(64 * kMergeRows);
  const auto merge = wide == 8   ? pa_window_merge_kernel<8>
                     : wide == 4 ? pa_window_merge_kernel<4>
                     : wide == 2 ? pa_window_merge_kernel<2>
                                 : pa_window_merge_kernel<1>;
  return cudaLaunchKernelEx(&l.cfg, merge, m) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

// CTAs of a segment of pa_step_kernel, or 0: the sequences of few tokens are the other kernel's.  The step
// kernel is taken for single tokens where its
// CTAs, two to an SM, fill four fifths of the device in each wave, no sequence has more than 5/4 of the mean
// keys, and a segment has 128 keys for each CTA of its cluster and each wave (one wave of clusters of one: any number);
// and where, with clusters of several, the device holds all of them at once (fit; a cluster lies in one of its groups of
// SMs, so that some SMs are left over: 74 clusters of 4 go on 152 SMs, not 76, and 36 of 8, not 38, of which the last two
// wait all the same while one launch follows another).  Segments of 1024 / 4096 keys, us: 74 clusters of 4 20.1 / 36.2,
// 75 27.5 / 53.5; 34 of 8 12.9 / 23.0, 36 17.3 / 30.7.  pa_step_impl.cuh has both sides' times.
int step_cluster(const Batch& b, int sms, const StepFit* fit = nullptr) {
  if (b.most != 1) return 0;
  const int64_t slots = 2 * sms;
  if (b.longest * b.few > b.keys + b.keys / 4) return 0;
  for (int i = 3; i >= 0; --i) {
    const int64_t c = 1 << i, n = b.few * b.heads * c, waves = (n + slots - 1) / slots;
    if ((waves > 1 && c > 1) || n * 5 < waves * slots * 4) continue;
    if (fit && c > 1 && b.few * b.heads > fit->clusters[i] - (c == 8 ? 2 : 0)) continue;
    return waves * c == 1 || b.longest >= 128 * c * waves ? (int)c : 0;
  }
  return 0;
}

// One token per sequence: kMaxStepSeqs sequences to a launch, a cluster to each of their heads.
pa_status launch_steps(StepParams& p, const Batch& b, const StepKernel& ki, cudaStream_t cs) {
  for (uint32_t s = 0, token = 0; s < b.n_seq;) {
    int n = 0;
    for (; s < b.n_seq && n < kMaxStepSeqs; token += b.n_new[s++])
      if (b.n_new[s] == 1) p.seq[n++] = StepSeq{(int32_t)s, (int32_t)token, b.lens[s]};
    if (n == 0) break;
    Launch l(cs);
    set_steps(l, ki, p.cluster, n * p.n_kv_heads);
    if (cudaLaunchKernelEx(&l.cfg, ki.fn, p) != cudaSuccess) return PA_ERR_CUDA;
  }
  return PA_OK;
}

// The keys of the batch's sequences of many tokens into the workspace.
pa_status prepare_prompts(PrepareParams& r, const Batch& b, int sms, cudaStream_t cs) {
  int group0 = 0;
  for (uint32_t i = 0; i < b.n_seq;) {
    r.n_seqs = r.groups = 0;
    for (; i < b.n_seq && r.n_seqs < PrepareParams::kMaxPromptSeqs; ++i) {
      if (!b.many(i)) continue;
      const SeqSpan s = seq_span(b.lens[i], b.n_new[i], b.window, b.sinks);
      r.seq[r.n_seqs++] = PromptSeq{(int32_t)i, b.lens[i], s.lo, s.s16, s.shift, s.groups, group0, s.edge, r.groups};
      r.groups += s.groups;
      group0 += s.groups;
    }
    if (r.n_seqs == 0) break;
    const pa_status st = launch_prepare(r, sms, cs);
    if (st != PA_OK) return st;
  }
  return PA_OK;
}

// Where the units' sequences have their keys; (seq, group0): of the launches before.
void place_prompts(PromptParams& p, const Batch& b, uint32_t* seq, int* group0) {
  for (int i = 0; i < p.n_units; ++i) {
    PromptUnit& u = p.unit[i];
    for (; *seq < (uint32_t)u.seq; ++*seq)
      if (b.many(*seq)) *group0 += seq_span(b.lens[*seq], b.n_new[*seq], b.window, b.sinks).groups;
    const SeqSpan s = seq_span(u.len, b.n_new[u.seq], b.window, b.sinks);
    u.groups = s.groups;
    u.group0 = *group0;
    u.shift0 = s.shift;
    u.edge = span_of(u, b.window, b.sinks).lo >= s.s16 ? s.edge : -1;
  }
}

// Whole segments for each pair instead of p's ranges, if the longest pair's share is no longer
// than the ranges with their merge.
bool list_segments(PromptParams& p, const Plan& plan) {
  p.listed = 0;
  const int segs = p.n_units * p.n_kv_heads;
  if (segs > PromptParams::kMaxListed || segs < p.n_ctas) return false;
  struct Seg {
    int32_t cost;
    uint16_t unit;
  };
  static thread_local Seg seg[PromptParams::kMaxUnits];
  int64_t total = 0;
  for (int i = 0; i < p.n_units; ++i) {
    seg[i] = Seg{kPromptLead + kPromptTile * tiles_of(p.unit[i], p.window, p.sinks), (uint16_t)i};
    total += (int64_t)p.n_kv_heads * seg[i].cost;
  }
  std::sort(seg, seg + p.n_units, [](const Seg& a, const Seg& b) { return a.cost > b.cost || (a.cost == b.cost && a.unit < b.unit); });
  // a heap of (load, pair), the least first
  static thread_local uint64_t heap[kMaxCtas];
  static thread_local uint16_t owner[PromptParams::kMaxListed];
  for (int i = 0; i < p.n_ctas; ++i) heap[i] = (uint64_t)i;
  const auto more = [](uint64_t a, uint64_t b) { return a > b; };
  int k = 0;
  uint64_t longest = 0;
  for (int i = 0; i < p.n_units; ++i)
    for (int h = 0; h < p.n_kv_heads; ++h) {
      std::pop_heap(heap, heap + p.n_ctas, more);
      uint64_t& top = heap[p.n_ctas - 1];
      owner[k++] = (uint16_t)(top & 0xffff);
      top += (uint64_t)seg[i].cost << 16;
      longest = std::max(longest, top >> 16);
      std::push_heap(heap, heap + p.n_ctas, more);
    }
  if ((int64_t)longest > total / p.n_ctas + (plan.cuts ? kPromptMerge : 0)) return false;
  uint16_t at[kMaxCtas / 2 + 1] = {};
  for (int i = 0; i < segs; ++i) ++at[owner[i]];
  uint16_t sum = 0;
  for (int i = 0; i < p.n_ctas; ++i) {
    p.first[i] = sum;
    sum = (uint16_t)(sum + at[i]);
    at[i] = p.first[i];
  }
  p.first[p.n_ctas] = sum;
  k = 0;
  for (int i = 0; i < p.n_units; ++i)
    for (int h = 0; h < p.n_kv_heads; ++h) p.list[at[owner[k++]]++] = (uint16_t)(seg[i].unit * p.n_kv_heads + h);
  p.listed = 1;
  return true;
}

pa_status check_pool(const pa_pool* pool, pa_pool_desc* d, Kernels* ki) {
  if (!pool || pa_pool_get_desc(pool, d) != PA_OK) return PA_ERR_INVALID;
  return d->head_dim == (uint32_t)kD && d->n_kv_heads <= 0x7fff && lookup_kernels(d->k_type, d->v_type, ki) ? PA_OK : PA_ERR_UNSUPPORTED;
}

// The window as the kernels take it: at most as long as any sequence.
int clamp_keys(uint32_t n) { return (int)std::min<uint32_t>(n, kAllKeys); }

// What both kernels' parameters, and the merge's, have in common.
template <class P>
void fill(P& p, const Batch& b, const pa_pool_desc& d, const void* q, int64_t q_stride, int32_t q_type, const int32_t* lens_dev, float scale,
          void* out, int64_t out_stride, int32_t out_type, float* lse, int32_t* err) {
  p.q = static_cast<const uint8_t*>(q);
  p.lens = lens_dev;
  p.err = err;
  p.out = static_cast<uint8_t*>(out);
  p.lse = lse;
  p.q_stride = q_stride;
  p.out_stride = out_stride;
  p.q_type = q_type;
  p.out_type = out_type;
  p.n_kv_heads = (int)d.n_kv_heads;
  p.n_q_heads = (int)d.n_kv_heads * kGqa;
  p.window = b.window;
  p.sinks = b.sinks;
  p.scale_log2 = scale * kLog2e;
}

// The same with the parts of cut segments, and the merge's parameters.
template <class P>
void fill_parts(P& p, MergeParams& m, uint8_t* ws, size_t o, int slot_rows) {
  m.lens = p.lens;
  m.err = p.err;
  m.part_ml = p.part_ml = reinterpret_cast<float2*>(ws);
  m.part_o = p.part_o = reinterpret_cast<float*>(ws + o);
  m.out = p.out;
  m.lse = p.lse;
  m.out_stride = p.out_stride;
  m.out_type = p.out_type;
  m.n_q_heads = p.n_q_heads;
  m.slot_rows = p.slot_rows = slot_rows;
}

// The pools as the kernels that read them take them.
template <class P>
void fill_pools(P& p, const pa_pool_desc& d, const void* k_pool, const void* v_pool, const int32_t* table, uint32_t table_stride) {
  p.k_pool = static_cast<const uint8_t*>(k_pool);
  p.v_pool = static_cast<const uint8_t*>(v_pool);
  p.table = table;
  p.page_size = (int)d.page_size;
  p.page_shift = -1;
  for (int i = 4; i < 31; ++i)
    if (d.page_size == 1u << i) p.page_shift = i;
  p.table_stride = (int)table_stride;
  p.n_blocks = (int)d.n_blocks;
}

}  // namespace

extern "C" size_t pa_attend_window_workspace_size(const pa_pool* pool, const int32_t* seq_lens_host, const int32_t* n_new,
                                                  uint32_t n_seq, uint32_t window, uint32_t sinks, int device) {
  pa_pool_desc d;
  Kernels ki;
  int ctas = 0;
  if (check_pool(pool, &d, &ki) != PA_OK || (n_seq && (!seq_lens_host || !n_new))) return 0;
  Batch b{seq_lens_host, n_new, n_seq, clamp_keys(window ? window : ~0u), clamp_keys(sinks), (int)d.n_kv_heads};
  if (check_batch(d, ~0u, &b) != PA_OK || device_ready(device, d.k_type, d.v_type, nullptr, &ctas) != PA_OK) return 0;
  return layout_of(ctas, b).total;
}

extern "C" pa_status pa_attend_window(const pa_pool* pool, const void* q, int64_t q_stride, int32_t q_type, const void* k_pool,
                                      const void* v_pool, const int32_t* block_table, uint32_t table_stride,
                                      const int32_t* seq_lens_dev, const int32_t* seq_lens_host, const int32_t* n_new,
                                      uint32_t n_seq, uint32_t n_q_heads, uint32_t window, uint32_t sinks, float scale,
                                      void* out, int64_t out_stride, int32_t out_type, float* lse, void* workspace,
                                      size_t ws_bytes, int32_t* err, pa_stream_t stream) {
  pa_pool_desc d;
  Kernels ki;
  pa_status st = check_pool(pool, &d, &ki);
  if (st != PA_OK) return st;
  if ((uint64_t)n_q_heads != (uint64_t)d.n_kv_heads * kGqa) return PA_ERR_UNSUPPORTED;
  if (!dtype_bytes(q_type) || !dtype_bytes(out_type)) return PA_ERR_UNSUPPORTED;
  if (n_seq == 0) return PA_OK;
  if (!seq_lens_host || !n_new) return PA_ERR_INVALID;
  if (!(scale > 0.f) || !std::isfinite(scale)) return PA_ERR_INVALID;
  // every length is checked before the first launch
  Batch b{seq_lens_host, n_new, n_seq, clamp_keys(window ? window : ~0u), clamp_keys(sinks), (int)d.n_kv_heads};
  st = check_batch(d, (uint64_t)table_stride * d.page_size, &b);
  if (st != PA_OK) return st;
  if (b.tokens == 0) return PA_OK;
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
  StepFit fit = {};
  st = device_ready(device, d.k_type, d.v_type, &ki, &ctas, &fit);
  if (st != PA_OK) return st;
  const WsLayout lay = layout_of(ctas, b);
  if (ws_bytes < lay.total) return PA_ERR_INVALID;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  static thread_local MergeParams m;  // kept off the stack
  // Launches in order on the stream, sharing the workspace: each one's kernel waits for the
  // one before to complete.
  if (const int cluster = ki.step.fn ? step_cluster(b, ctas, &fit) : 0) {
    static thread_local StepParams p;
    fill(p, b, d, q, q_stride, q_type, seq_lens_dev, scale, out, out_stride, out_type, lse, err);
    fill_pools(p, d, k_pool, v_pool, block_table, table_stride);
    p.cluster = cluster;
    if ((st = launch_steps(p, b, ki.step, cs)) != PA_OK) return st;
  } else if (b.most > 0) {
    static thread_local WindowParams p;
    fill(p, b, d, q, q_stride, q_type, seq_lens_dev, scale, out, out_stride, out_type, lse, err);
    fill_parts(p, m, ws, lay.o, slot_rows_of(b.most));
    fill_pools(p, d, k_pool, v_pool, block_table, table_stride);
    for (Cursor at{0, 0, 0}; at.seq < n_seq;) {
      const Plan plan = plan_chunk(p, m, b, false, ctas, &at);
      if (p.n_units == 0) break;
      if ((st = launch_few(p, ki.few, cs)) != PA_OK || (st = launch_merge(m, plan, ctas, cs)) != PA_OK) return st;
    }
  }
  if (b.prompts > 0) {
    static thread_local PromptParams p;
    static thread_local PrepareParams r;
    fill(p, b, d, q, q_stride, q_type, seq_lens_dev, scale, out, out_stride, out_type, lse, err);
    fill_parts(p, m, ws, lay.o, kPromptRows);
    p.k = r.k = ws + lay.k;
    p.v = r.v = ws + lay.v;
    p.wide = r.wide = d.k_type == PA_F16 ? nullptr : ws + lay.wide;
    r.k_pool = static_cast<const uint8_t*>(k_pool);
    r.v_pool = static_cast<const uint8_t*>(v_pool);
    r.table = block_table;
    r.err = err;
    r.k_type = d.k_type;
    r.v_type = d.v_type;
    r.n_kv_heads = (int)d.n_kv_heads;
    r.page_size = (int)d.page_size;
    r.table_stride = (int)table_stride;
    r.n_blocks = (int)d.n_blocks;
    r.sinks = b.sinks;
    if ((st = prepare_prompts(r, b, ctas, cs)) != PA_OK) return st;
    uint32_t seq = 0;
    int group0 = 0;
    for (Cursor at{0, 0, 0}; at.seq < n_seq;) {
      Plan plan = plan_chunk(p, m, b, true, ctas / 2, &at);  // ranges of pairs of CTAs
      if (p.n_units == 0) break;
      if (list_segments(p, plan)) plan.cuts = 0;
      place_prompts(p, b, &seq, &group0);
      if ((st = launch_prompt(p, cs)) != PA_OK || (st = launch_merge(m, plan, ctas, cs)) != PA_OK) return st;
    }
  }
  return PA_OK;
}
