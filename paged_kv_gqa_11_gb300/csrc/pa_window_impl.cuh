// Attention over a sliding window of the cache and its first keys (sm_103a): the walk
// over the tiles, the copies, the masks and the results of pa_attend_window.  Everything
// else -- products, dequantisation, softmax, hand-offs -- is the kernel of
// pa_prefix_impl.cuh, compiled for these parameters.
//
// The mathematics.  Token t of a sequence, at position p_t, sees the keys x <= p_t with
// x > p_t - W or x < S (a window of W keys, S sinks).  A unit is up to 64 query rows of a
// sequence (six per token and KV head); its first row's window begins at lo = p - W + 1,
// its last row's ends at the position of its token, and what any of its rows sees lies in
// two runs of row groups (16 keys): those of the sinks, and those from lo's on.  They are
// laid end to end, the sinks' first, as the unit's key order, and cut into tiles of 128:
//   key v of the order is position v (v < s16) or v + shift.
// A segment is (unit, KV head).  The tiles of all segments, laid end to end by their cost,
// are cut into one equal range per CTA.  A segment inside one range (of a prompt nearly all)
// is finished there: the softmax warps divide by the sum of weights and write the
// result.  One that is cut leaves a piece in each range, and a merge joins them; a range
// cuts at its two ends only, so there are two slots for each CTA, whatever the batch.
//
// Masks.  In the tiles at the ends of the two runs a row's logits become -inf where it
// does not see the key; the others have no mask.  Keys that no row of the unit sees (in the
// row groups at the ends of the runs) count as zeros in V, whatever the pool holds
// there.  A key that some rows of the unit see and others do not has weight 0 for those.
//
// A row's first key (its window's, or the first sink) lies in the first tile of any
// piece in which it sees a key at all: the tokens of a unit are up to 11 apart (43 in a
// prompt's unit of 256 rows, pa_prompt.cu), so their windows begin within 26 (58) keys of the
// unit's first row group, and a tile has 128.  The softmax relies on it: a reference is set at
// a piece's first tile, and only raised later.
//
// What bounds it: latency.  Bulk copies of a row group's 2 to 8 KB take the copy engine 55
// cycles each and 36 bytes a cycle, a tile of 128 keys 1 to 2.3 us, and 7 to 8 us pass from
// launch to the merge's last row (8 tokens, window 4096, Q4_0: 20.3 us, 0.28 of what their bytes
// take; 8 x 4, window 2048, F16: 22.0 from HBM, 0.46, and 16.5 while the L2 holds the rows).  It was made for up to
// 64 query rows; a single token has six, so pa_decode, made for one, is faster over long contexts (8 x 8192 keys, Q4_0:
// 23.6 us, this kernel 30.1), and so is pa_prefix_kernel, whose walk has less to decide for a tile (28.1).
// Many tokens have pa_prompt.cu, large batches of single ones pa_step_impl.cuh.
#pragma once

#include "pa_prefix_impl.cuh"

namespace pa_prefix {

constexpr int kAllKeys = 0x7fffffff - 2 * kKeys;  // a window as long as any sequence: that of a call without one

struct Unit {
  int32_t seq;        // row of the table
  int32_t token;      // of its first row, among all queries
  int32_t pos;        // that token's position
  int32_t len;        // of the sequence
  int32_t rows_row0;  // query rows | first row among its token's six << 16
  int32_t at, tile;   // places, tiles before the unit
};

// Where a CTA's range begins: j-th tile of (unit, head), the launch's tile-th; one more for the
// end.  The host finds them: a search among the units in the kernel takes 2 us of cold loads.
struct Start {
  int32_t unit_head;  // unit | head << 16
  int32_t j, tile;
};
constexpr int kMaxCtas = 256;

struct WindowParams {
  static constexpr bool kWindow = true;
  static constexpr int kUnitRows = kRows, kMaxUnits = 448;  // query rows of a unit, units per launch
  using Live = int4;  // of a tile: its live keys are those before x and from y to z - 1
  const uint8_t* q;
  const uint8_t* k_pool;
  const uint8_t* v_pool;
  const int32_t* table;
  const int32_t* lens;  // device lengths, only compared
  int32_t* err;
  float2* part_ml;  // (reference maximum in log2 units, sum of weights) per slot row
  float* part_o;    // [slot row][256]
  uint8_t* out;
  float* lse;
  long long q_stride, out_stride;  // values per token
  int q_type, out_type, n_kv_heads, n_q_heads, page_size, table_stride, n_blocks;
  int page_shift;  // log2 of page_size, or -1
  int n_units, n_ctas, weigh;
  int total_len, total_tiles;
  int window, sinks;
  int slot_rows;  // rows of a slot
  float scale_log2;
  Start start[kMaxCtas + 1];
  Unit unit[kMaxUnits];
};

__host__ __device__ inline int unit_rows(const Unit& u) { return u.rows_row0 & 0xffff; }
__host__ __device__ inline int unit_row0(const Unit& u) { return u.rows_row0 >> 16; }

// The key order of a unit.
struct Span {
  int s16, shift;  // position of v: v, from s16 on v + shift
  int lo, end;     // first key of the first row's window, place in the order after the last key
};

__host__ __device__ inline Span span_of(const Unit& u, int window, int sinks) {
  Span s;
  const int last = u.pos + (unit_row0(u) + unit_rows(u) - 1) / kGqa;
  s.lo = u.pos >= window ? u.pos - window + 1 : 0;
  s.s16 = (sinks + kGroup - 1) & ~(kGroup - 1);
  const int group = s.lo & ~(kGroup - 1);
  s.shift = group > s.s16 ? group - s.s16 : 0;
  s.end = last + 1 - s.shift;
  return s;
}

// ------------------------------------------------------------------ the walk
//
// P: WindowParams, or those of the prompts' kernel.

__host__ __device__ __forceinline__ Cost cost_of(const WindowParams& p, const Unit& u) { return cost_of(p.weigh, unit_rows(u)); }

template <class P>
__host__ __device__ __forceinline__ void pos_sizes(const P& p, Pos& t) {
  t.nt = ceil_div(span_of(p.unit[t.unit], p.window, p.sinks).end, kKeys);
}

template <class P>
__host__ __device__ __forceinline__ void advance(const P& p, Pos& t) {
  if (++t.j < t.nt) return;
  t.j = 0;
  if (++t.head < p.n_kv_heads) return;
  t.head = 0;
  if (++t.unit >= p.n_units) return;  // past the last tile
  pos_sizes(p, t);
}

// The first tile at place x or after it.
template <class P>
__host__ __device__ __forceinline__ Pos locate(const P& p, int x) {
  Pos t;
  t.pre = false;
  t.rt = 0;
  t.nrt = 1;
  int lo = 0, hi = p.n_units - 1;  // the last unit whose first place is <= x
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.unit[mid].at <= x) lo = mid; else hi = mid - 1;
  }
  t.unit = lo;
  x -= p.unit[lo].at;
  pos_sizes(p, t);
  const Cost c = cost_of(p, p.unit[lo]);
  const int len = c.lead + t.nt * c.tile;
  t.head = x / len;
  t.j = ((x > t.head * len + c.lead ? x - t.head * len - c.lead : 0) + c.tile - 1) / c.tile;
  t.tile = p.unit[lo].tile + t.head * t.nt + t.j;
  if (t.j == t.nt) {  // past the segment's last tile
    --t.j;
    advance(p, t);
  }
  return t;
}

template <class P>
__device__ __forceinline__ Pos start_of(const P& p, int cta) {
  const Start& s = p.start[cta];
  Pos t;
  t.pre = false;
  t.rt = 0;
  t.nrt = 1;
  t.unit = s.unit_head & 0xffff;
  t.head = s.unit_head >> 16;
  t.j = s.j;
  t.tile = s.tile;
  pos_sizes(p, t);
  return t;
}

__device__ __forceinline__ int pos_rows(const WindowParams& p, const Pos& t) { return unit_rows(p.unit[t.unit]); }
__device__ __forceinline__ int pos_row0(const WindowParams& p, const Pos& t) { return unit_row0(p.unit[t.unit]); }
__device__ __forceinline__ int pos_token(const WindowParams& p, const Pos& t) { return p.unit[t.unit].token; }
__device__ __forceinline__ long long query_at(const WindowParams& p, int t, int h) { return t * p.q_stride + h * kD; }

// ------------------------------------------------------------------ tiles

// Of a window's tile: info bit 10: some row does not see some key; bit 16: the sequence's
// length on the device is another; open: the first token's position; slot_row: -1 where
// the piece is the whole segment; pad: its first key's place in the order, the shift.
constexpr uint32_t kEdge = 1u << 10, kOtherLength = 1u << 16;

__device__ __forceinline__ bool has_edge(const WindowParams&, const Tile& t) { return t.info & kEdge; }

__host__ __device__ __forceinline__ WindowKeys live_keys(const WindowParams&, int4 l, int from) { return WindowKeys{l.x - from, l.y - from, l.z - from}; }

__host__ __device__ __forceinline__ int clamp_rows(int x) { return x < 0 ? 0 : x > kRows ? kRows : x; }

// The rows x .. y - 1 that see key k of a tile (as far as they are among its own).
__host__ __device__ __forceinline__ int2 rows_that_see(const WindowParams& p, const Tile& t, int k) {
  const int v = t.pad[0] + k, s16 = (p.sinks + kGroup - 1) & ~(kGroup - 1), key = v < s16 ? v : v + t.pad[1];
  const int rel = key - t.open;  // tokens from the first one to the key
  const int first = clamp_rows(rel), last = key < p.sinks ? kRows : clamp_rows(rel + p.window);
  return make_int2(kGqa * first - t.row0, kGqa * last - t.row0);
}

// Whether every row sees every key of the tile from place key0 on: none of them after the
// first token, none before the last one's window (or all of them sinks).
__host__ __device__ __forceinline__ bool sees_all(const Span& s, int key0, int first_pos, int last_lo, int sinks) {
  const int to = key0 + kKeys - 1;
  const bool window_only = key0 >= s.s16 || s.shift == 0;
  return to + (window_only ? s.shift : 0) <= first_pos && ((window_only && key0 + s.shift >= last_lo) || to < sinks);
}

// The live keys of the tile from place key0 on: those before x and from y to z - 1.
__host__ __device__ __forceinline__ int4 live_of(const Span& s, int key0, int sinks) {
  return make_int4(sinks - key0, s.lo - s.shift - key0, s.end - key0, 0);
}

// The slot row of a tile's piece (where it is the piece's last tile): -1, the segment's only one; that of
// the CTA's first slot, if the segment began before its range, or of its second.
__host__ __device__ __forceinline__ int slot_of(bool fresh, bool ends, int cta, int slot_rows) {
  return fresh && ends ? -1 : (2 * cta + (fresh ? 1 : 0)) * slot_rows;
}

// The copies (see copy_role above), with the window's key order and what the tiles say of
// it.
__device__ __forceinline__ int copy_role(const WindowParams& p, Pos pos, int n, bool is_v, int gb, int rb, int ns, uint32_t ring,
                                         uint32_t full, uint32_t empty, Tile* tiles, int4* lives, volatile int* abort,
                                         int lane) {
  const uint8_t* pool = is_v ? p.v_pool : p.k_pool;
  const long long block_rows = (long long)p.n_kv_heads * p.page_size;
  const int half = (lane >> 2) & 1, lane_key = lane < 8 ? kGroup * lane : kKeys;  // lanes past 7 have no group
  const int page_shift = p.page_shift;
  // of the segment
  const int32_t* row = nullptr;
  Span sp{0, 0, 0, 0};
  int key0 = 0, head_row = 0, last_lo = 0, first_pos = 0;
  uint32_t info = 0;
  int token = 0, head = 0, row0 = 0;
  uint32_t odd = 1;
  int entry = -1, off = 0;
  int pair = 0;         // stages 2 pair, 2 pair + 1
  uint32_t parity = 1;  // of the wait for the stages' previous use; flips when the ring wraps
  bool last = true, fresh = true;
  for (int j = -1; j < n; ++j) {  // issues tile j, looks tile j + 1 up
    const int left = sp.end - key0, tb = entry;
    const bool mine = lane_key < min(kKeys, left), ok = mine && (uint32_t)tb < (uint32_t)p.n_blocks;
    const uint8_t* src = pool + (tb * block_rows + (head_row + off)) * rb;
    if (j >= 0) {
      last = j + 1 == n || pos.j + 1 == pos.nt;
      if (lane == 0) {
        if (is_v) {
          lives[j & (kTiles - 1)] = live_of(sp, key0, p.sinks);
        } else {
          const bool inner = sees_all(sp, key0, first_pos, last_lo, p.sinks);
          const int slot = slot_of(fresh, pos.j + 1 == pos.nt, (int)blockIdx.x, p.slot_rows);
          int4* t = reinterpret_cast<int4*>(tiles + (j & (kTiles - 1)));
          t[0] = make_int4((int)(info | (last ? 1u << 9 : 0u) | (inner ? 0u : kEdge)), first_pos, row0, slot);
          t[1] = make_int4(token, head, key0, sp.shift);
        }
      }
      info &= ~(1u << 8);
      if (last) {
        if (j + 1 < n) advance(p, pos);
      } else {
        ++pos.j;
        key0 += kKeys;
      }
    }
    if (j + 1 < n) {
      if (last) {
        odd ^= 1;
        const Unit& u = p.unit[pos.unit];
        sp = span_of(u, p.window, p.sinks);
        row = p.table + (long long)u.seq * p.table_stride;
        key0 = pos.j * kKeys;
        head = pos.head;
        head_row = head * p.page_size;
        token = u.token;
        row0 = unit_row0(u);
        first_pos = u.pos;
        const int last_pos = u.pos + (row0 + unit_rows(u) - 1) / kGqa;
        last_lo = last_pos >= p.window ? last_pos - p.window + 1 : 0;
        fresh = pos.j == 0;
        info = (uint32_t)unit_rows(u) | 1u << 8 | odd << 11;
        if (!is_v && __ldg(p.lens + u.seq) != u.len) info |= kOtherLength;
      }
      const int v = key0 + lane_key;
      entry = -1;
      if (lane_key < kKeys && v < sp.end) {
        const int k = v < sp.s16 ? v : v + sp.shift;
        const int page = page_shift >= 0 ? k >> page_shift : k / p.page_size;
        off = k - page * p.page_size;
        entry = __ldg(row + page);
      }
    }
    if (j < 0) continue;
    const uint32_t good = __ballot_sync(0xffffffffu, ok), bad = __ballot_sync(0xffffffffu, mine && !ok);
    const uint32_t stage = 2 * pair + half, fb = full + 8 * stage, dst = ring + stage * (4 * gb) + (lane & 3) * gb;
    if (j >= ns / 2 && !warp_wait(empty + 8 * stage, parity, p.err, abort)) return 2 * j;
    if (bad) {  // rows of an entry outside the pool read as zeros
      if (lane == 0) record_error(p.err, PA_ERR_BOUNDS);
#pragma unroll 1
      for (int g = 0; g < 8; ++g) {
        if (!((bad >> g) & 1)) continue;
#pragma unroll 1
        for (int i = lane; i < gb / 16; i += 32) sts128_zero(ring + (2 * pair + (g >> 2)) * (4 * gb) + (g & 3) * gb + 16 * i);
      }
      fence_proxy_async_smem();
      __syncwarp();
    }
    __syncwarp();  // the tile's record, written by lane 0, comes before lane 4's arrival too
    if (lane == 0 || lane == 4) mbar_arrive_expect_tx(fb, __popc(good & (0xfu << lane)) * gb);
    __syncwarp();
    if (ok)
      asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                   "l"(src), "r"(gb), "r"(fb)
                   : "memory");
    if (++pair == ns / 2) {
      pair = 0;
      parity ^= 1;
    }
  }
  return 2 * n;
}

// ------------------------------------------------------------------ results

__device__ __forceinline__ void store_value(uint8_t* dst, int type, float x) {
  if (type == PA_DT_F32) *reinterpret_cast<float*>(dst) = x;
  else if (type == PA_DT_F16) *reinterpret_cast<__half*>(dst) = __float2half_rn(x);
  else *reinterpret_cast<__nv_bfloat16*>(dst) = __float2bfloat16_rn(x);
}

// A finished row: its lse, and what its sums are multiplied by: 1 / l, 0 for a row of
// zeros (its sequence's length on the device is another).
__device__ __forceinline__ float finish_row(const WindowParams& p, const Tile& t, int r, float m, float l) {
  if (t.info & kOtherLength) {
    if (r == 0) record_error(p.err, PA_ERR_BOUNDS);
    l = 0.f;
  }
  const int rg = t.row0 + r;
  if (p.lse)
    p.lse[(long long)(t.token + rg / kGqa) * p.n_q_heads + t.head * kGqa + rg % kGqa] =
        l != 0.f ? (m + log2f(l)) * pa_split::kLn2 : -INFINITY;
  return l != 0.f ? 1.f / l : 0.f;
}

// Rows r .. r + 15 of O^T (of which there are `rows`), dim d.
__device__ __forceinline__ void write_out(const WindowParams& p, const Tile& t, int r, int rows, const float* inv, int d,
                                          const uint32_t (&o)[16]) {
  const int bytes = p.out_type == PA_DT_F32 ? 4 : 2;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    if (r + i >= rows) break;
    const int rg = t.row0 + r + i, tok = rg / kGqa;
    const float f = inv[r + i], x = f != 0.f ? __uint_as_float(o[i]) * f : 0.f;
    store_value(p.out + ((t.token + tok) * p.out_stride + (t.head * kGqa + rg - tok * kGqa) * kD + d) * bytes, p.out_type, x);
  }
}

using WindowKernel = KernelOf<WindowParams>;

#define PA_DECLARE_WINDOW(k, v) bool lookup_window_kernel_##k##_##v(WindowKernel* out);
PA_DECLARE_WINDOW(1, 1) PA_DECLARE_WINDOW(1, 2) PA_DECLARE_WINDOW(1, 8)
PA_DECLARE_WINDOW(2, 1) PA_DECLARE_WINDOW(2, 2) PA_DECLARE_WINDOW(2, 8)
PA_DECLARE_WINDOW(8, 1) PA_DECLARE_WINDOW(8, 2) PA_DECLARE_WINDOW(8, 8)
#undef PA_DECLARE_WINDOW

}  // namespace pa_prefix
