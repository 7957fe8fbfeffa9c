// Rows and blocks of a cache moved within its pools (pa_move_rows, pa_move_blocks,
// pa_copy_blocks).
//
// Mathematics.  A key at position p was turned by the angles p f of its pairs; at position
// p' under frequencies f' it is to be turned by p' f' - p f more.  The difference is taken
// in 64-bit fixed-point turns, like the angles themselves (pa_row_ops.cuh), so far
// positions lose nothing.  A turned block of 32 values is dequantised, turned and quantised
// again by the rule of the append; all other bytes of a row stay what they are.
//
// Rows that land where others still have to be read: all reads come before all writes.  Few
// rows (64 of 4 heads) stay in the registers of one cluster of CTAs between the two (its hardware barrier
// is the only thing between them: one launch); more go through the workspace, in the pools'
// formats, by two launches.  Where the caller vouches that no row's place is another row's
// source, one launch reads and writes at once.
//
// Bound: the memory, where keys keep their bytes or rows are many; a turned key costs 300 instructions
// a head (dequantised, turned, its maximum found, quantised), which a warp hides by having the
// next four heads' loads on their way.  K's rows and V's are in CTAs of their own, so that rows
// turned in place do not leave every second warp idle.  Measured, one GB300: 24 rows 3.4 us (one launch),
// 12000 rows of Q8_0 down by 777, 64 values turned (two launches) 31.1 (28.6 while the L2 holds them), the same rows
// to other pages (disjoint, one launch) 22.3, without a turn 15.0 (7.7 are their bytes), 65536 rows of Q8_0 keys turned in place
// (all 256 values, 2.0 TB/s read and written: the arithmetic) 71.3; with rows of both pools in one
// warp and no loads ahead 138.  Partly turned heads packed so that a warp turns only their blocks
// were slower (more registers, 154, and more shuffles than the arithmetic that they saved).
#include <cuda_runtime.h>

#include <algorithm>
#include <cstring>

#include "pa_row_ops.cuh"

using namespace pa_rows_io;

namespace {

struct MoveParams {
  uint8_t* k_pool;
  uint8_t* v_pool;
  uint8_t* ws;
  const int32_t* src_seq;
  const int32_t* src_pos;
  const int32_t* dst_seq;
  const int32_t* dst_pos;
  const int32_t* src_table;
  const int32_t* dst_table;
  int32_t* err;
  long long n_rows;
  int n_heads, page_size, src_stride, src_seqs, dst_stride, dst_seqs, n_blocks, k_type, v_type;
  int rows;         // of a warp
  int rot, interleaved;
  int still;        // a row that keeps its position is not turned
  float factor;
  uint64_t from[kMaxPairs], to[kMaxPairs];
};

// A row on its way: both places (head 0's group, in rows of the pool, and the row in it),
// and whether its key is turned.
struct Move {
  long long src, dst;
  int src_r, dst_r;
  int src_pos, dst_pos;
  bool ok, turned, same;  // same: both places are one
};

__device__ __forceinline__ Move move_of(const MoveParams& p, long long row) {
  Move m{};
  Place a{}, b{};
  m.src_pos = __ldg(p.src_pos + row);
  m.dst_pos = __ldg(p.dst_pos + row);
  const bool has = place_of(p.src_table, p.src_stride, p.src_seqs, p.n_blocks, p.page_size, p.n_heads, __ldg(p.src_seq + row), m.src_pos, &a);
  m.ok = place_of(p.dst_table, p.dst_stride, p.dst_seqs, p.n_blocks, p.page_size, p.n_heads, __ldg(p.dst_seq + row), m.dst_pos, &b) && has;
  m.src = a.grp_row;
  m.src_r = a.r;
  m.dst = b.grp_row;
  m.dst_r = b.r;
  m.same = a.grp_row == b.grp_row && a.r == b.r;
  m.turned = p.rot > 0 && !(p.still && m.src_pos == m.dst_pos);
  return m;
}

__device__ __forceinline__ Move from_lane(const Move& m, int l) {
  Move r;
  r.src = __shfl_sync(0xffffffffu, m.src, l);
  r.dst = __shfl_sync(0xffffffffu, m.dst, l);
  r.src_r = __shfl_sync(0xffffffffu, m.src_r, l);
  r.dst_r = __shfl_sync(0xffffffffu, m.dst_r, l);
  r.src_pos = __shfl_sync(0xffffffffu, m.src_pos, l);
  r.dst_pos = __shfl_sync(0xffffffffu, m.dst_pos, l);
  const int f = __shfl_sync(0xffffffffu, (int)m.ok | (int)m.turned << 1 | (int)m.same << 2, l);
  r.ok = f & 1;
  r.turned = f >> 1 & 1;
  r.same = f >> 2 & 1;
  return r;
}

template <int T>
__device__ __forceinline__ Packed get(const uint8_t* row, const Lane& at) {
  if (T == PA_F16) return Packed{*reinterpret_cast<const uint4*>(row + at.body), 0u};
  const uint2 w = *reinterpret_cast<const uint2*>(row + at.body);
  return Packed{make_uint4(w.x, w.y, 0u, 0u), *reinterpret_cast<const uint16_t*>(row + at.scale)};
}

// The eight values of lane l that x holds, in pairs.
template <int T>
__device__ __forceinline__ void values(const Packed& x, int l, uint64_t (&y)[4]) {
  if (T == PA_F16) {
    float f[8];
    unpack8<__half>(&x.w, f);
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = pack2(f[2 * i], f[2 * i + 1]);
    return;
  }
  const float d = __half2float(__ushort_as_half((unsigned short)x.d));
  const uint64_t d2 = pack2(d, d);
  // bytes 0 .. 255 under 0x4b0000 are the fp32 numbers 2^23 + byte
  const float bias = T == PA_Q8_0 ? -8388736.f : -8388616.f;  // -(2^23 + 128), -(2^23 + 8)
  const uint64_t b2 = pack2(bias, bias);
  const uint32_t w[2] = {x.w.x, x.w.y};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t u = T == PA_Q8_0 ? w[i] ^ 0x80808080u : (w[i] >> ((l & 2) << 1)) & 0x0f0f0f0fu;
#pragma unroll
    for (int k = 0; k < 2; ++k)
      y[2 * i + k] = mul2(add2(pack2(__uint_as_float(prmt(u, 0x4b000000u, k ? 0x7442 : 0x7440)),
                                     __uint_as_float(prmt(u, 0x4b000000u, k ? 0x7443 : 0x7441))),
                               b2),
                          d2);
  }
}

// A head's row turned by t: its turned blocks quantised anew, the others as they are.
template <int T>
__device__ __forceinline__ Packed turned(const MoveParams& p, const Packed& x, const Turn& t, int from, int lane) {
  uint64_t a[4], b[4];
  values<T>(x, lane, a);
  if (p.interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 v = unpack2(a[i]);
      b[i] = pack2(v.y, v.x);
    }
  } else {
    Packed o;
    o.w.x = __shfl_sync(0xffffffffu, x.w.x, from);
    o.w.y = __shfl_sync(0xffffffffu, x.w.y, from);
    o.w.z = T == PA_F16 ? __shfl_sync(0xffffffffu, x.w.z, from) : 0u;
    o.w.w = T == PA_F16 ? __shfl_sync(0xffffffffu, x.w.w, from) : 0u;
    o.d = T == PA_F16 ? 0u : __shfl_sync(0xffffffffu, x.d, from);
    values<T>(o, from, b);
  }
  float y[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = unpack2(fma2(a[i], t.c[i], mul2(b[i], t.s[i])));
    y[2 * i] = v.x;
    y[2 * i + 1] = v.y;
  }
  if ((p.rot & 16) && !is_turned(p.rot, lane)) {  // the second half of the last turned block
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 v = unpack2(a[i]);
      y[2 * i] = v.x;
      y[2 * i + 1] = v.y;
    }
  }
  __syncwarp();
  const Packed q = quantised(T, y, lane);
  return 32 * (lane >> 2) < p.rot ? q : x;
}

__device__ __forceinline__ Turn turn_of(const MoveParams& p, const uint64_t* from_turns, const uint64_t* to_turns, int src_pos, int dst_pos,
                                        int lane, int from) {
  return make_turn(
      p.rot, p.interleaved, p.factor,
      // whole products (positions are 0 and more): of one frequency the difference is that of the distance, for all rows
      // that are moved by it the same
      [&](int i) { return (uint64_t)(uint32_t)dst_pos * to_turns[i] - (uint64_t)(uint32_t)src_pos * from_turns[i]; },
      lane, from);
}

// A row between its places in the pools: at ws, heads one after the other, each its chunks,
// then its scales.
__device__ __forceinline__ Lane lane_in_ws(int type, int lane) {
  if (type == PA_F16) return Lane{16 * lane, 0};
  return type == PA_Q8_0 ? Lane{8 * lane, Fmt<PA_Q8_0>::kRowQ + 2 * (lane >> 2)}
                         : Lane{16 * (lane >> 2) + 8 * (lane & 1), Fmt<PA_Q4_0>::kRowQ + 2 * (lane >> 2)};
}

enum Phase { kDirect, kGather, kScatter };

// Four heads of a row on their way: where they come from and go to.
struct Ends {
  const uint8_t* src;
  uint8_t* dst;
  Lane a, b;
};

template <int T, int kPhase>
__device__ __forceinline__ Ends ends_of(const MoveParams& p, uint8_t* pool, bool is_v, const Move& m, uint8_t* ws, int lane) {
  Ends e;
  e.src = kPhase == kScatter ? ws : pool + m.src * Fmt<T>::kRow;
  e.dst = kPhase == kGather ? ws : pool + m.dst * Fmt<T>::kRow;
  e.a = kPhase == kScatter ? lane_in_ws(T, lane) : lane_of(T, is_v, m.src_r, lane);
  e.b = kPhase == kGather ? lane_in_ws(T, lane) : lane_of(T, is_v, m.dst_r, lane);
  return e;
}

// A warp's rows of one pool, the next four heads' loads (of the row, or of the next row) before the
// last ones are worked on.
template <int T, int kPhase>
__device__ __forceinline__ void move_rows_of(const MoveParams& p, bool is_v, const Move& moves, int rows, long long row0, const uint64_t* from_turns,
                                             const uint64_t* to_turns, int lane) {
  const long long step = (long long)p.page_size * Fmt<T>::kRow;
  const long long src_step = kPhase == kScatter ? Fmt<T>::kRow : step, dst_step = kPhase == kGather ? Fmt<T>::kRow : step;
  uint8_t* pool = is_v ? p.v_pool : p.k_pool;
  const long long k_row = (long long)p.n_heads * row_bytes_of(p.k_type), v_row = (long long)p.n_heads * row_bytes_of(p.v_type);
  const int from = partner_lane(p.rot, p.interleaved, lane);
  const int quads = (p.n_heads + 3) >> 2;
  // the rows that have something to do
  const bool turns_mine = !is_v && moves.turned;
  uint32_t todo = __ballot_sync(0xffffffffu, lane < rows && moves.ok && !(moves.same && !turns_mine));
  if (kPhase != kScatter) {  // the first eight rows' first four heads are on their way at once: lane = (row, head)
    const int r = lane >> 2, h = lane & 3;
    const long long src = __shfl_sync(0xffffffffu, moves.src, r);
    const int src_r = __shfl_sync(0xffffffffu, moves.src_r, r);
    if (todo >> r & 1 && h < p.n_heads) {
      const uint8_t* grp = pool + src * Fmt<T>::kRow + h * step;
#pragma unroll
      for (int i = 0; i < Fmt<T>::kRowQ; i += 128)
        asm volatile("prefetch.global.L1 [%0];" ::"l"(grp + Fmt<T>::kScales + src_r * Fmt<T>::kRowQ + i));
    }
  }
  Ends next{};
  Packed ahead[4] = {};
  int next_row = -1, next_quad = 0;
  Move next_move{};
  auto fetch = [&]() {  // the next four heads
    if (next_row >= 0 && ++next_quad < quads) {
    } else {
      if (todo == 0) {
        next_row = -1;
        return;
      }
      next_row = __ffs(todo) - 1;
      todo &= todo - 1;
      next_quad = 0;
      next_move = from_lane(moves, next_row);
      const long long row = row0 + next_row;
      next = ends_of<T, kPhase>(p, pool, is_v, next_move, kPhase == kDirect ? nullptr : p.ws + (is_v ? p.n_rows * k_row + row * v_row : row * k_row), lane);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (4 * next_quad + i < p.n_heads) ahead[i] = get<T>(next.src + (4 * next_quad + i) * src_step, next.a);
  };
  fetch();
  Turn t;
  int turned_row = -1, turned_by = 0;
  while (next_row >= 0) {
    Packed x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = ahead[i];
    uint8_t* dst = next.dst;
    const Lane b = next.b;
    const int row = next_row, h = 4 * next_quad;
    const bool turn = kPhase != kScatter && !is_v && next_move.turned;
    const int src_pos = next_move.src_pos, dst_pos = next_move.dst_pos;
    fetch();
    if (turn && turned_row != row) {
      const int by = dst_pos - src_pos;  // positions are 0 and more
      if (turned_row < 0 || !p.still || by != turned_by) t = turn_of(p, from_turns, to_turns, src_pos, dst_pos, lane, from);
      turned_row = row;
      turned_by = by;
    }
    // heads that are not there are turned all the same: nothing stands between the four
    if (turn) {
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = turned<T>(p, x[i], t, from, lane);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (h + i < p.n_heads) put(T, x[i], dst + (h + i) * dst_step, b, lane);
  }
}

__device__ __forceinline__ void load_turns(const MoveParams& p, uint64_t* from_turns, uint64_t* to_turns) {
  for (int i = threadIdx.x; i < p.rot / 2; i += blockDim.x) {
    from_turns[i] = p.from[i];
    to_turns[i] = p.to[i];
  }
  __syncthreads();
}

template <int kPhase>
__global__ void __launch_bounds__(32 * kWarps) pa_move_kernel(const __grid_constant__ MoveParams p) {
  if (threadIdx.x == 0) asm volatile("griddepcontrol.launch_dependents;");
  __shared__ uint64_t from_turns[kMaxPairs], to_turns[kMaxPairs];
  const int lane = threadIdx.x & 31;
  load_turns(p, from_turns, to_turns);
  // K's rows first, V's in CTAs of their own: where keys are turned in place those have nothing to do
  const long long half = gridDim.x >> 1;
  const bool is_v = blockIdx.x >= half;
  const long long row0 = ((long long)(blockIdx.x - (is_v ? half : 0)) * kWarps + (threadIdx.x >> 5)) * p.rows;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // nothing that another kernel wrote is read before this
  if (row0 >= p.n_rows) return;
  const int rows = (int)min((long long)p.rows, p.n_rows - row0);
  Move m{};
  if (lane < rows) {
    m = move_of(p, row0 + lane);
    if (!m.ok && !is_v && kPhase != kScatter) record_error(p.err, PA_ERR_BOUNDS);
  }
  const int type = is_v ? p.v_type : p.k_type;
  if (type == PA_F16) move_rows_of<PA_F16, kPhase>(p, is_v, m, rows, row0, from_turns, to_turns, lane);
  else if (type == PA_Q8_0) move_rows_of<PA_Q8_0, kPhase>(p, is_v, m, rows, row0, from_turns, to_turns, lane);
  else move_rows_of<PA_Q4_0, kPhase>(p, is_v, m, rows, row0, from_turns, to_turns, lane);
}

// Few rows: every warp of a cluster reads a (row, pool, four heads), all warps meet, every warp
// writes.  Of rows of 4 heads in Q8_0: 24 rows 5.5 us; the others' two launches 6.9.  More than one
// item to a warp, its loads one after the other, are slower than those (100 rows 9.2, 256 16.8).
constexpr int kSmallWarps = 16, kMaxCluster = 8;

template <int T>
__device__ __forceinline__ void read_item(const MoveParams& p, const uint8_t* pool, bool is_v, const Move& m, int h0, bool turns,
                                          const Turn& t, int from, int lane, Packed (&x)[4]) {
  const long long step = (long long)p.page_size * Fmt<T>::kRow;
  const uint8_t* src = pool + m.src * Fmt<T>::kRow + h0 * step;
  const Lane a = lane_of(T, is_v, m.src_r, lane);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (h0 + i < p.n_heads) x[i] = get<T>(src + i * step, a);
  if (turns) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (h0 + i < p.n_heads) x[i] = turned<T>(p, x[i], t, from, lane);
  }
}

__global__ void __launch_bounds__(32 * kSmallWarps, 1) pa_move_few_kernel(const __grid_constant__ MoveParams p) {
  if (threadIdx.x == 0) asm volatile("griddepcontrol.launch_dependents;");
  __shared__ uint64_t from_turns[kMaxPairs], to_turns[kMaxPairs];
  const int lane = threadIdx.x & 31, from = partner_lane(p.rot, p.interleaved, lane);
  load_turns(p, from_turns, to_turns);
  const int quads = (p.n_heads + 3) / 4, item = (int)blockIdx.x * kSmallWarps + (threadIdx.x >> 5);
  asm volatile("griddepcontrol.wait;" ::: "memory");  // nothing that another kernel wrote is read before this
  const int row = item / (2 * quads), rest = item - row * 2 * quads, h0 = 4 * (rest >> 1);
  const bool is_v = rest & 1;
  const int type = is_v ? p.v_type : p.k_type;
  uint8_t* const pool = is_v ? p.v_pool : p.k_pool;
  Packed x[4];
  Move m{};
  bool go = false;
  if (row < (int)p.n_rows) {
    m = move_of(p, row);
    if (!m.ok && rest == 0 && lane == 0) record_error(p.err, PA_ERR_BOUNDS);
    const bool turns = !is_v && m.turned;
    go = m.ok && (turns || !m.same);
    if (go) {
      Turn t;
      if (turns) t = turn_of(p, from_turns, to_turns, m.src_pos, m.dst_pos, lane, from);
      if (type == PA_F16) read_item<PA_F16>(p, pool, is_v, m, h0, turns, t, from, lane, x);
      else if (type == PA_Q8_0) read_item<PA_Q8_0>(p, pool, is_v, m, h0, turns, t, from, lane, x);
      else read_item<PA_Q4_0>(p, pool, is_v, m, h0, turns, t, from, lane, x);
    }
  }
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  if (!go) return;
  const long long rb = row_bytes_of(type), step = (long long)p.page_size * rb;
  uint8_t* to = pool + m.dst * rb + h0 * step;
  const Lane b = lane_of(type, is_v, m.dst_r, lane);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (h0 + i < p.n_heads) put(type, x[i], to + i * step, b, lane);
}

// ------------------------------------------------------------------ blocks

// Whole blocks (every KV head's page, K and V) from src[i] to dst[i], and the tables' entries
// src[i] as dst[i].  All blocks' 16-byte pieces, laid end to end, one to a thread at a time, then the
// tables' entries, each found in src (ascending) by bisection.  Bound: HBM (5000 blocks of 64 rows, Q8_0 /
// Q4_0: 164 us, 6.5 TB/s read and written).  2048 threads an SM have as much on its way as
// the memory takes; 2 or 4 pieces to a thread (fewer fit) took 176 and 185 us, parts of 16 KB inside a block 181.
struct BlockParams {
  uint8_t* k_pool;
  uint8_t* v_pool;
  const int32_t* src;
  const int32_t* dst;
  const int32_t* table;
  int32_t* table_out;
  int32_t* err;
  long long k_pieces, v_pieces;  // of a block
  long long entries;
  long long pieces, parts;       // of all pairs; parts of kBlockThreads
  int n, n_blocks;
  int small;                     // pieces is a 31-bit number
};

constexpr int kBlockThreads = 256;

__global__ void __launch_bounds__(kBlockThreads, 8) pa_move_blocks_kernel(const __grid_constant__ BlockParams p) {
  if (threadIdx.x == 0) asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");  // nothing that another kernel wrote is read before this
  const long long per = p.k_pieces + p.v_pieces;
  const long long parts = p.parts + (p.entries + kBlockThreads - 1) / kBlockThreads;
  for (long long part = blockIdx.x; part < parts; part += gridDim.x) {
    if (part >= p.parts) {
      const long long e = (part - p.parts) * kBlockThreads + threadIdx.x;
      if (e >= p.entries) continue;
      const int x = __ldcg(p.table + e);
      int lo = 0, hi = p.n;  // the first pair with src >= x
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(p.src + mid) < x) lo = mid + 1; else hi = mid;
      }
      int to = x;
      if (lo < p.n && __ldg(p.src + lo) == x && (uint32_t)x < (uint32_t)p.n_blocks) {
        const int d = __ldg(p.dst + lo);
        if ((uint32_t)d < (uint32_t)p.n_blocks) to = d;
      }
      p.table_out[e] = to;
      continue;
    }
    const long long i = part * kBlockThreads + threadIdx.x;
    if (i >= p.pieces) continue;
    const long long pair = p.small ? (long long)((uint32_t)i / (uint32_t)per) : i / per, c = i - pair * per;
    const int s = __ldg(p.src + pair), d = __ldg(p.dst + pair);
    if (c == 0 && p.table && pair > 0 && __ldg(p.src + pair - 1) >= s) record_error(p.err, PA_ERR_INVALID);
    if ((uint32_t)s >= (uint32_t)p.n_blocks || (uint32_t)d >= (uint32_t)p.n_blocks) {
      if (c == 0) record_error(p.err, PA_ERR_BOUNDS);
      continue;
    }
    const bool is_v = c >= p.k_pieces;
    const long long size = is_v ? p.v_pieces : p.k_pieces, at = is_v ? c - p.k_pieces : c;
    uint4* pool = reinterpret_cast<uint4*>(is_v ? p.v_pool : p.k_pool);
    pool[d * size + at] = pool[s * size + at];
  }
}

// ------------------------------------------------------------------ host side

// Rows that one cluster moves at once.
bool is_few(long long n_rows, int n_heads) { return n_rows * 2 * ((n_heads + 3) / 4) <= kSmallWarps * kMaxCluster; }

pa_status launch_few(const MoveParams& p, cudaStream_t cs) {
  const long long items = p.n_rows * 2 * ((p.n_heads + 3) / 4);
  const unsigned ctas = (unsigned)((items + kSmallWarps - 1) / kSmallWarps);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(32 * kSmallWarps);
  cfg.stream = cs;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, pa_move_few_kernel, p) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

pa_status launch_blocks(const BlockParams& p, cudaStream_t cs) {
  int sms = 0;
  const pa_status st = sm_count(&sms);
  if (st != PA_OK) return st;
  const long long parts = p.parts + (p.entries + kBlockThreads - 1) / kBlockThreads;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)std::min<long long>(parts, 8ll * sms));
  cfg.blockDim = dim3(kBlockThreads);
  cfg.stream = cs;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, pa_move_blocks_kernel, p) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

pa_status move_blocks(const pa_pool* pool, void* k_pool, void* v_pool, const int32_t* src, const int32_t* dst, uint32_t n,
                      const int32_t* table, int32_t* table_out, uint64_t entries, int32_t* err, pa_stream_t stream) {
  pa_pool_desc d;
  if (pa_pool_get_desc(pool, &d) != PA_OK) return PA_ERR_INVALID;
  if (n == 0 && entries == 0) return PA_OK;
  if (!k_pool || !v_pool || (n && (!src || !dst)) || !err || (entries && (!table || !table_out))) return PA_ERR_INVALID;
  if (!aligned16(k_pool) || !aligned16(v_pool)) return PA_ERR_INVALID;
  const size_t bk = (size_t)d.n_kv_heads * d.page_size * pa_row_bytes(d.k_type, d.head_dim);
  const size_t bv = (size_t)d.n_kv_heads * d.page_size * pa_row_bytes(d.v_type, d.head_dim);
  if (bk == 0 || bv == 0 || ((bk | bv) & 15)) return PA_ERR_UNSUPPORTED;
  if (n > 0x7fffffffu || entries > (uint64_t(1) << 40) || (bk + bv) / 16 > 0x7fffffffu) return PA_ERR_UNSUPPORTED;
  BlockParams p{};
  p.k_pool = static_cast<uint8_t*>(k_pool);
  p.v_pool = static_cast<uint8_t*>(v_pool);
  p.src = src;
  p.dst = dst;
  p.table = entries ? table : nullptr;
  p.table_out = table_out;
  p.err = err;
  p.k_pieces = (long long)(bk / 16);
  p.v_pieces = (long long)(bv / 16);
  p.entries = (long long)entries;
  p.n = (int)n;
  p.pieces = (long long)n * (p.k_pieces + p.v_pieces);
  p.parts = (p.pieces + kBlockThreads - 1) / kBlockThreads;
  p.small = p.pieces <= 0x7fffffff;
  p.n_blocks = (int)d.n_blocks;
  return launch_blocks(p, reinterpret_cast<cudaStream_t>(stream));
}

size_t move_workspace(const pa_pool_desc& d, uint64_t n_rows) {
  return (size_t)n_rows * d.n_kv_heads * (pa_row_bytes(d.k_type, d.head_dim) + pa_row_bytes(d.v_type, d.head_dim));
}

}  // namespace

extern "C" pa_status pa_copy_blocks(const pa_pool* pool, void* k_pool, void* v_pool, const int32_t* src,
                                    const int32_t* dst, uint32_t n, int32_t* err, pa_stream_t stream) {
  return move_blocks(pool, k_pool, v_pool, src, dst, n, nullptr, nullptr, 0, err, stream);
}

extern "C" pa_status pa_move_blocks(const pa_pool* pool, void* k_pool, void* v_pool, const int32_t* src,
                                    const int32_t* dst, uint32_t n, const int32_t* table, int32_t* table_out,
                                    uint64_t n_entries, int32_t* err, pa_stream_t stream) {
  return move_blocks(pool, k_pool, v_pool, src, dst, n, table, table_out, n_entries, err, stream);
}

extern "C" size_t pa_move_rows_workspace_size(const pa_pool* pool, uint32_t n_rows) {
  pa_pool_desc d;
  if (pa_pool_get_desc(pool, &d) != PA_OK || is_few(n_rows, (int)d.n_kv_heads)) return 0;
  return move_workspace(d, n_rows);
}

extern "C" pa_status pa_move_rows(const pa_pool* pool, void* k_pool, void* v_pool, const pa_rope_desc* rope,
                                  const pa_rope_desc* rope_from, const int32_t* src_seq, const int32_t* src_pos,
                                  const int32_t* dst_seq, const int32_t* dst_pos, uint32_t n_rows,
                                  const int32_t* src_table, uint32_t src_stride, uint32_t src_n_seq,
                                  const int32_t* dst_table, uint32_t dst_stride, uint32_t dst_n_seq, int32_t disjoint,
                                  void* workspace, size_t ws_bytes, int32_t* err, pa_stream_t stream) {
  pa_pool_desc d;
  if (pa_pool_get_desc(pool, &d) != PA_OK) return PA_ERR_INVALID;
  if (d.head_dim != (uint32_t)kD) return PA_ERR_UNSUPPORTED;
  if (!rope && rope_from) return PA_ERR_INVALID;
  for (const pa_rope_desc* r : {rope, rope_from}) {
    if (!r) continue;
    const pa_status st = check_rope(r);
    if (st != PA_OK) return st;
  }
  if (rope_from && (rope_from->rot_dim != rope->rot_dim || rope_from->interleaved != rope->interleaved)) return PA_ERR_INVALID;
  if (n_rows == 0) return PA_OK;
  if (!k_pool || !v_pool || !src_seq || !src_pos || !dst_seq || !dst_pos || !src_table || !dst_table || !err || src_stride == 0 ||
      dst_stride == 0 || src_n_seq == 0 || dst_n_seq == 0)
    return PA_ERR_INVALID;
  if (src_stride > 0x7fffffffu || dst_stride > 0x7fffffffu || src_n_seq > 0x7fffffffu || dst_n_seq > 0x7fffffffu) return PA_ERR_INVALID;
  if (!aligned16(k_pool) || !aligned16(v_pool)) return PA_ERR_INVALID;
  MoveParams p{};
  p.factor = 1.f;
  p.still = 1;
  if (rope) {
    const pa_rope_desc* was = rope_from ? rope_from : rope;
    const double factor = (double)rope->attn_factor / (double)was->attn_factor;
    if (!std::isfinite(factor) || !std::isfinite((float)factor)) return PA_ERR_INVALID;  // nothing brings back what a factor of 0 made
    p.rot = (int)rope->rot_dim;
    p.interleaved = rope->interleaved;
    p.factor = (float)factor;
    p.still = factor == 1.0;
    for (int i = 0; i < p.rot / 2; ++i) {
      p.from[i] = turns_of(was->inv_freq[i]);
      p.to[i] = turns_of(rope->inv_freq[i]);
      if (p.from[i] != p.to[i]) p.still = 0;
    }
  }
  p.k_pool = static_cast<uint8_t*>(k_pool);
  p.v_pool = static_cast<uint8_t*>(v_pool);
  p.src_seq = src_seq;
  p.src_pos = src_pos;
  p.dst_seq = dst_seq;
  p.dst_pos = dst_pos;
  p.src_table = src_table;
  p.dst_table = dst_table;
  p.err = err;
  p.n_rows = n_rows;
  p.n_heads = (int)d.n_kv_heads;
  p.page_size = (int)d.page_size;
  p.src_stride = (int)src_stride;
  p.src_seqs = (int)src_n_seq;
  p.dst_stride = (int)dst_stride;
  p.dst_seqs = (int)dst_n_seq;
  p.n_blocks = (int)d.n_blocks;
  p.k_type = d.k_type;
  p.v_type = d.v_type;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  if (!disjoint && is_few(n_rows, p.n_heads)) return launch_few(p, cs);
  if (!disjoint) {
    if (!workspace || !aligned16(workspace) || ws_bytes < move_workspace(d, n_rows)) return PA_ERR_INVALID;
    p.ws = static_cast<uint8_t*>(workspace);
  }
  int sms = 0;
  pa_status st = sm_count(&sms);
  if (st != PA_OK) return st;
  // as few rows to a warp as give 32 warps an SM, up to 8 (12000 rows: 2 a warp 34.2 us, these 5 28.4, 8 33.5)
  p.rows = (int)std::min<long long>(8, (2ll * n_rows + 32ll * sms - 1) / (32ll * sms));
  const long long grid = 2 * ((((long long)n_rows + p.rows - 1) / p.rows + kWarps - 1) / kWarps);
  if (grid > 0x7fffffffll) return PA_ERR_UNSUPPORTED;
  if (disjoint) return launch(pa_move_kernel<kDirect>, p, (unsigned)grid, cs);
  st = launch(pa_move_kernel<kGather>, p, (unsigned)grid, cs);
  return st == PA_OK ? launch(pa_move_kernel<kScatter>, p, (unsigned)grid, cs) : st;
}
