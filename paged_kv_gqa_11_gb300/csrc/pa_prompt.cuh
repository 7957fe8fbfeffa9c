// Windowed attention of many new tokens (chunks of prompt, whole prompts): parameters of its
// kernels (pa_prompt.cu) for the host side (pa_window.cu).
#pragma once

#include <cuda_runtime.h>

#include "pa_window_impl.cuh"

namespace pa_prefix {

constexpr int kPromptRows = 256;              // query rows of a unit: 128 for each CTA of a pair
constexpr int kGroupBytes = kGroup * kD * 2;  // a group's keys (or values) in binary16

// A unit of a prompt, and where its sequence's keys lie in the workspace: the row groups
// group0 .. group0 + groups - 1, of position v (v < s16), else v + shift0.  edge: the group that
// stands for the values of the one in which the sinks end, or -1 (SeqSpan).
struct PromptUnit : Unit {
  int32_t groups, group0, shift0, edge;
};

// The key order of all new tokens of a sequence: that of a unit from its first to its last.
//
// A value counts as a zero where no new token sees its key, but the sequence's first tokens may see
// the keys behind the last sink in the sinks' last row group, which is in the order of every unit.  A
// weight of 0 does not take an infinite or NaN value out of a product, so where some windows begin
// in that group or before it and others behind it, the sequence has the group once more, the
// last (edge), with zeros behind the last sink, for the units whose windows all begin behind it.
struct SeqSpan : Span {
  int groups, edge;
};

inline SeqSpan seq_span(int len, int n_new, int window, int sinks) {
  SeqSpan s;
  const int first = len - n_new;
  s.lo = first >= window ? first - window + 1 : 0;
  s.s16 = (sinks + kGroup - 1) & ~(kGroup - 1);
  const int group = s.lo & ~(kGroup - 1);
  s.shift = group > s.s16 ? group - s.s16 : 0;
  s.end = len - s.shift;
  s.groups = ceil_div(s.end, kGroup);
  s.edge = sinks < s.s16 && s.lo < s.s16 && len - window >= s.s16 ? s.groups++ : -1;  // len - window: the last token's first key
  return s;
}

// The workspace's row groups for such a sequence: no fewer than it has, wherever in a row group its window
// begins, and no fewer for more keys, new tokens, window or first keys.
inline int64_t room_for(int64_t len, int64_t n_new, int64_t window, int64_t sinks) {
  const int64_t all = (len + kGroup - 1) / kGroup, some = (sinks + kGroup - 1) / kGroup + (n_new + window + 2 * kGroup - 3) / kGroup;
  return (all < some ? all : some) + 1;  // and edge
}

struct PromptParams {
  static constexpr int kUnitRows = kPromptRows, kMaxUnits = 256;
  const uint8_t* q;
  const int32_t* lens;  // device lengths, only compared
  const uint8_t* k;     // the workspace's keys and values, and which keys are wide (or NULL: none can be)
  const uint8_t* v;
  const uint8_t* wide;
  int32_t* err;
  float2* part_ml;
  float* part_o;
  uint8_t* out;
  float* lse;
  long long q_stride, out_stride;
  int q_type, out_type, n_kv_heads, n_q_heads;
  int n_units, n_ctas, weigh;  // n_ctas: pairs of CTAs
  int total_len, total_tiles;
  int window, sinks;
  int slot_rows;
  float scale_log2;
  Start start[kMaxCtas / 2 + 1];
  // Or whole segments for each pair (listed): list[first[i]] .. list[first[i + 1] - 1], unit *
  // n_kv_heads + head.
  static constexpr int kMaxListed = 1024;
  int listed;
  uint16_t first[kMaxCtas / 2 + 1];
  uint16_t list[kMaxListed];
  PromptUnit unit[kMaxUnits];
};

// What a piece takes, and a tile; and the cuts of a launch (a merge, and rows in fp32 by way of the
// workspace) in the same places, 0.15 us each.  4096 tokens without a window, cut: a lead of 4 308 us, 16 237, 32 and
// 40 167, 48 176.
constexpr int kPromptLead = 40, kPromptTile = 8, kPromptMerge = 70;
__host__ __device__ __forceinline__ Cost cost_of(const PromptParams& p, const Unit&) {
  return p.weigh ? Cost{kPromptLead, kPromptTile} : Cost{0, 1};
}

// The places of a unit's order that a row sees: v <= hi with v >= lo or v < sinks (a row behind
// the unit's: none).
struct RowKeys {
  int lo, hi;
  __host__ __device__ __forceinline__ bool has(int v, int sinks) const { return v <= hi && (v >= lo || v < sinks); }
  // has(v + k, sinks) in bit k, k < 64.
  __host__ __device__ __forceinline__ uint64_t bits(int v, int sinks) const {
    return below(hi - v + 1) & (~below(lo - v) | below(sinks - v));
  }
  static __host__ __device__ __forceinline__ uint64_t below(int n) { return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1; }
};

__host__ __device__ __forceinline__ RowKeys row_keys(const Unit& u, const Span& s, int row, int window) {
  const int pos = u.pos + (unit_row0(u) + row) / kGqa;
  return RowKeys{(pos >= window ? pos - window + 1 : 0) - s.shift, row < unit_rows(u) ? pos - s.shift : -1};
}

// The group of place v of a unit's order among its sequence's.
__host__ __device__ __forceinline__ int group_of(const PromptUnit& u, const Span& s, int v) {
  return (v < s.s16 ? v : v + s.shift - u.shift0) >> 4;
}

// The run of the sequence's groups that the places v (the first of a row group) .. end - 1 begin with: up to `stop`, from
// `group` on.  One run holds them all, or two (sinks, window), or three where `edge` (of values u.edge, of keys -1)
// stands for the group in which the sinks end.
struct Run {
  int group, stop;
};
__host__ __device__ __forceinline__ Run run_of(const PromptUnit& u, const Span& s, int edge, int v, int end) {
  Run r{group_of(u, s, v), end};
  if (v < s.s16) {
    const int last = s.s16 - kGroup;
    if (edge >= 0 && v == last) r.group = edge;
    const int stop = edge >= 0 && v < last ? last : edge >= 0 || s.shift != u.shift0 ? s.s16 : end;
    r.stop = stop < end ? stop : end;
  }
  return r;
}

// A sequence's keys on their way into the workspace.
struct PromptSeq {
  int32_t seq, len;
  int32_t lo;  // first key of its first new token's window
  int32_t s16, shift, groups, group0, edge;
  int32_t at;  // groups of the launch's sequences before it
};

// The position of a group's first key.
__host__ __device__ __forceinline__ int first_key(const PromptSeq& s, int group) {
  const int v = group == s.edge ? s.s16 - kGroup : group * kGroup;
  return v < s.s16 ? v : v + s.shift;
}

// Whether a group has the value of `key`, one of its 16, or a zero in its place, whatever lies there.
__host__ __device__ __forceinline__ bool has_value(const PromptSeq& s, int group, int key, int sinks) {
  return key < s.len && (key < sinks || (key >= s.lo && group != s.edge));
}

struct PrepareParams {
  static constexpr int kMaxPromptSeqs = 128;
  const uint8_t* k_pool;
  const uint8_t* v_pool;
  const int32_t* table;
  uint8_t* k;
  uint8_t* v;
  uint8_t* wide;
  int32_t* err;
  int k_type, v_type, n_kv_heads, page_size, table_stride, n_blocks;
  int sinks;
  int n_seqs, groups;
  PromptSeq seq[kMaxPromptSeqs];
};

// Launches (programmatic dependents of what runs before them on the stream).
pa_status launch_prepare(const PrepareParams& p, int sms, cudaStream_t cs);
pa_status launch_prompt(const PromptParams& p, cudaStream_t cs);
pa_status prompt_ready();  // raises the kernel's limits on the current device

}  // namespace pa_prefix
