// Windowed attention of many new tokens, on the fifth-generation tensor core (sm_103a).
//
// The mathematics is that of pa_window_impl.cuh.  A prompt's tokens share their keys: a key
// tile meets dozens of row tiles.  So the keys and values that any new token sees are
// first turned into binary16 once, in the workspace (pa_prompt_prepare_kernel; a chunk's stay
// in L2), in the order in which the MMAs take them, and the attention is a dense one over tiles
// of 256 query rows (a unit) x 128 keys, by pairs of CTAs (clusters of two, cta_group::2):
//   S = Q K^T   tcgen05.mma M = 256 rows, N = 128 keys, K = 256 dims; Q and K in shared memory;
//   O += P V    M = 256 rows, N = 256 dims, K = keys; P in tensor memory (in its S's place), V in shared memory.
// A CTA holds 128 of the rows (Q, S, P and O), 64 of the tile's keys of K and 128 of the dims
// of V; the tensor cores read each other's half.
//
// Why pairs.  An SM takes in 30 bytes a cycle from L2 (all of them 8.9 TB/s, measured).
// A CTA of its own reads 128 KB for 128 rows x 128 keys, 4300 cycles for 2048 of MMA
// (4096 tokens, no window: 312 us); one of a pair 64 KB.  (Bulk copies to both CTAs
// at once, multicast, run at 12 bytes a cycle.)
//
// The workspace's layout, per (sequence, head); a core matrix is 8 rows x 16 bytes:
//   K   two planes of 128 dims, each [8 keys][16 slots of 8 dims] core matrices (rows = keys);
//   V   two planes of 128 dims, each [8 keys][16 slots of 8 dims] core matrices, transposed (rows = dims);
// a run of row groups of a plane is one contiguous piece, and an MMA's B operand.  The row group in which the
// first keys end may be there twice (SeqSpan), so that a value that only early tokens see meets no later ones.
//
// Tensor memory: O in columns 0-255, two buffers of S in 256-383 and 384-511; P as pairs
// of binary16 in the first 64 columns of its S.
//
// Shared memory: Q twice (64 KB each, this piece's and the next one's) and a ring of five stages
// of 16 KB: of K 64 keys x 128 dims, of V 64 keys x 128 dims, each worth 512 cycles of MMA.
//
// Warps, hand-offs on mbarriers, every wait bounded:
//   0-7    softmax: (half of the keys, lane quarter), thread = row;
//   8-11   query rows into Q (the first piece's: 0-7), and a finished piece's O to its place;
//   12     MMA issue (the pair's first CTA; the second's tells it of the second's copies);
//   13, 14 copies of K and of V.
// S of tile j + 1 is multiplied while the softmax of tile j runs, and that of j + 1 while PV of
// j and S of j + 2 are.
//
// Ranges, cuts and slots are those of pa_window_impl.cuh, with units of 256 rows and ranges of
// pairs; or, where that is no longer than with cuts and their merge, every pair has whole
// segments, the largest dealt first, each to the pair with least (4096 tokens, no window: 147 us
// against 167; 2048 tokens, window 1024: 59 against 67; both before K and V had a warp each).
//
// Measured: 4096 tokens without a window in F16 139 to 143 us replayed from a graph, 148 call by call (1393
// TFLOP/s of the 206 GFLOP that are not masked, 0.71 of cuBLAS's burst rate); 2048 tokens, window 1024, Q8_0 / Q4_0
// 61 us (58 while the L2 holds the rows), of which 6 for the keys' launch.  What bounds it: the copy engine's 32 bytes a cycle, 2040 cycles for a
// tile's 64 KB beside 2048 of MMA (each alone runs at its rate, with all other traffic around it); the
// engine and the MMAs wait for one another through a ring of five stages, 2300 cycles a tile.  A piece's end
// costs 2 us: its O is read before the next piece's first PV.  V by cp.async (65 bytes a cycle and SM by
// itself) was slower, with a proxy fence before its MMAs (154 us) or in the copying warp (170).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "pa_prompt.cuh"
#include "pa_row_ops.cuh"

namespace pa_prefix {

namespace {

using pa_rows_io::Lane;

constexpr int kPlaneGroup = kGroupBytes / 2;  // bytes of a group in a plane

// ------------------------------------------------------------------ keys and values into the workspace

// A warp takes eight rows (half a row group) of one head of one pool: lane l their dims 8 l ..
// + 7, which is one core matrix of the MMA's operand, 128 bytes.

// A lane's eight values of a row in binary16 (scale * quant, rounded once); wide: the row's
// scales as they are may overflow (dequant_k), the values are 2^-8 of what they are.
template <int T>
__device__ __forceinline__ uint4 half_values(const uint8_t* grp, int r, int lane, bool is_v, bool* wide) {
  const Lane at = pa_rows_io::lane_of(T, is_v, r, lane);
  if (T == PA_F16) return *reinterpret_cast<const uint4*>(grp + at.body);
  const uint2 raw = *reinterpret_cast<const uint2*>(grp + at.body);
  uint32_t d = *reinterpret_cast<const uint16_t*>(grp + at.scale);
  d |= d << 16;
  if (!is_v) {
    *wide = __any_sync(0xffffffffu, ((d & 0x7fffu) + (T == PA_Q8_0 ? 0x2000u : 0x1000u)) & 0x8000u);
    if (*wide) d = hmul2(d, kR256);
  }
  const uint32_t w[2] = {raw.x, raw.y};
  uint32_t h[4];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    // bytes 0 .. 255 under 0x64 are the binary16 numbers 1024 + byte
    const uint32_t u = T == PA_Q8_0 ? w[i] ^ 0x80808080u : (w[i] >> ((lane & 2) << 1)) & 0x0f0f0f0fu;
    const uint32_t bias = T == PA_Q8_0 ? 0xe480e480u : 0xe408e408u;  // -1152, -1032
    h[2 * i] = hmul2(hadd2(prmt(u, 0x64646464u, 0x4140), bias), d);
    h[2 * i + 1] = hmul2(hadd2(prmt(u, 0x64646464u, 0x4342), bias), d);
  }
  return make_uint4(h[0], h[1], h[2], h[3]);
}

template <int T>
__device__ __forceinline__ void prepare_rows(const PrepareParams& p, const PromptSeq& s, bool is_v, int head, int group, int half,
                                             const uint8_t* grp, int first, uint4* stage, int lane) {
  uint4 x[8];
  uint32_t wide_rows = 0;
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    bool wide = false;
    x[r] = grp ? half_values<T>(grp, 8 * half + r, lane, is_v, &wide) : make_uint4(0u, 0u, 0u, 0u);
    wide_rows |= (uint32_t)wide << r;
    if (is_v && !has_value(s, group, first + r, p.sinks)) x[r] = make_uint4(0u, 0u, 0u, 0u);
  }
  const long long reg = (long long)s.group0 * p.n_kv_heads + (long long)head * s.groups;
  if (is_v) {  // eight dims x eight keys, transposed
    uint32_t y[8][4];
#pragma unroll
    for (int d = 0; d < 4; ++d) {  // dims 2 d and 2 d + 1 of the lane's eight
      uint32_t w[8];
#pragma unroll
      for (int r = 0; r < 8; ++r) w[r] = d == 0 ? x[r].x : d == 1 ? x[r].y : d == 2 ? x[r].z : x[r].w;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        y[2 * d][k] = prmt(w[2 * k], w[2 * k + 1], 0x5410);
        y[2 * d + 1][k] = prmt(w[2 * k], w[2 * k + 1], 0x7632);
      }
    }
#pragma unroll
    for (int r = 0; r < 8; ++r) x[r] = make_uint4(y[r][0], y[r][1], y[r][2], y[r][3]);
  } else if (p.wide && lane == 0) {
    p.wide[(reg + group) * 2 + half] = (uint8_t)wide_rows;
  }
  // The lane's core matrix, by way of shared memory (chunk r of lane l at r ^ (l & 7)), so that a
  // store writes 512 bytes in a row: lanes 0 - 15 are the first plane's 2 KB, the others the second's.
#pragma unroll
  for (int r = 0; r < 8; ++r) stage[8 * lane + (r ^ (lane & 7))] = x[r];
  __syncwarp();
  uint8_t* to = (is_v ? p.v : p.k) + reg * kGroupBytes + (long long)(2 * group + half) * 2048;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int c = 32 * i + lane, l = c >> 3;  // chunk c of the 4 KB, of lane l
    *reinterpret_cast<uint4*>(to + (i >> 2) * (long long)s.groups * kPlaneGroup + ((c & 127) << 4)) = stage[8 * l + ((c & 7) ^ (l & 7))];
  }
  __syncwarp();
}

constexpr int kPrepareWarps = 4;

__global__ void __launch_bounds__(32 * kPrepareWarps, 8) pa_prompt_prepare_kernel(const __grid_constant__ PrepareParams p) {
  // In this order: when the attention starts, all that came before this kernel is complete,
  // and it may read its queries before it waits for this kernel's keys.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (threadIdx.x == 0) asm volatile("griddepcontrol.launch_dependents;");
  __shared__ uint4 stages[kPrepareWarps][256];
  uint4* stage = stages[threadIdx.x >> 5];
  const int lane = threadIdx.x & 31;
  const long long items = (long long)p.groups * 4 * p.n_kv_heads, step = (long long)gridDim.x * kPrepareWarps;
  for (long long i = (long long)blockIdx.x * kPrepareWarps + (threadIdx.x >> 5); i < items; i += step) {
    const int half = (int)(i & 1), is_v = (int)(i >> 1 & 1);
    const long long g = i >> 2;
    const int head = (int)(g % p.n_kv_heads), at = (int)(g / p.n_kv_heads);
    int lo = 0, hi = p.n_seqs - 1;  // the last sequence whose first group is <= at
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (p.seq[mid].at <= at) lo = mid; else hi = mid - 1;
    }
    const PromptSeq& s = p.seq[lo];
    const int group = at - s.at, first = first_key(s, group);
    if (group == s.edge && !is_v) continue;  // of values only
    const int page = first / p.page_size, off = first - page * p.page_size;
    const int entry = __ldg(p.table + (long long)s.seq * p.table_stride + page);
    const bool ok = (uint32_t)entry < (uint32_t)p.n_blocks;
    if (!ok && lane == 0) record_error(p.err, PA_ERR_BOUNDS);  // its rows read as zeros
    const int type = is_v ? p.v_type : p.k_type;
    const uint8_t* grp =
        ok ? (is_v ? p.v_pool : p.k_pool) + (((long long)entry * p.n_kv_heads + head) * p.page_size + off) * row_bytes_of(type) : nullptr;
    if (type == PA_F16) prepare_rows<PA_F16>(p, s, is_v, head, group, half, grp, first + 8 * half, stage, lane);
    else if (type == PA_Q8_0) prepare_rows<PA_Q8_0>(p, s, is_v, head, group, half, grp, first + 8 * half, stage, lane);
    else prepare_rows<PA_Q4_0>(p, s, is_v, head, group, half, grp, first + 8 * half, stage, lane);
  }
}

// ------------------------------------------------------------------ the attention

constexpr int kStageBytes = 16384, kNStages = 5;
constexpr int kCtaRows = kPromptRows / 2;  // rows of a CTA
constexpr int kPSmWarps = 8, kAuxWarp0 = 8, kMmaWarp = 12, kCopyWarp = 13, kPThreads = 15 * 32;
constexpr uint32_t kPOCol = 0, kPSCol = 256;

struct PSmem {
  static constexpr int kQBytes = kCtaRows * kD * 2;
  static constexpr int kQ = 0, kRing = 2 * kQBytes, kRed = kRing + kNStages * kStageBytes;
  static constexpr int kSum = kRed + 2 * kCtaRows * 4;        // [piece & 1][half of the keys][row]
  static constexpr int kRef = kSum + 4 * kCtaRows * 4;        // [piece & 1][row]
  static constexpr int kBar = kRef + 2 * kCtaRows * 4;
  static constexpr int kNBar = 2 * kNStages + 2 + 2 + 2 + 2 + 2 + 1 + 2 + 1;
  static constexpr int kMisc = kBar + 8 * kNBar + 8 * (kNBar & 1);  // abort, tmem base, the softmax's leave [quarter][2]
  static constexpr int kTotal = kMisc + 48;
  static constexpr int kLaunch = kTotal + 1024;
  static_assert(kLaunch <= 232448, "shared memory");
};

// ------------------------------------------------------------------ pairs of CTAs

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

// A meeting of all threads of both CTAs, in its two halves.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// An arrival at the first CTA's barrier of this address.  What it stands for -- a finished
// bulk copy, tensor memory behind a tcgen05 fence, shared memory behind a proxy fence -- is
// read by the tensor cores alone, not through this thread's own memory order, so the
// arrival has the CTA's scope (the cluster's takes about 1000 cycles in the arriving thread:
// 361 us for 4096 tokens without a window).
__device__ __forceinline__ void arrive_first(uint32_t bar, uint32_t rank) {
  if (rank == 0)
    mbar_arrive(bar);
  else
    asm volatile("{\n\t.reg .b32 r;\n\tmapa.shared::cluster.u32 r, %0, 0;\n\tmbarrier.arrive.shared::cluster.b64 _, [r];\n\t}" ::"r"(bar) : "memory");
}

// One arrival at both CTAs' barriers of this address when every MMA issued so far has
// completed.
__device__ __forceinline__ void commit_pair(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(bar),
      "h"((uint16_t)3)
      : "memory");
}

// MMAs of one stage, issued by the lane whose leader is set; one statement, so that what they
// share is moved to uniform registers once (mma8).  acc 0: the first overwrites D.
//   scores: D += Q K^T over 128 dims, eight steps of 16 (two slots of a row each);
//   values: D += P V over 64 keys, four steps of 16 (a row group each), or only the first `steps`.
#define PA_MMA(A, AOFF, BOFF, P) \
  A "\n\tadd.u64 b1, %2, " #BOFF ";\n\t@e tcgen05.mma.cta_group::2.kind::f16 [%0], " AOFF ", b1, %3, " P ";\n\t"
__device__ __forceinline__ void mma_scores(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc, uint32_t leader) {
#define PA_STEP(OFF, P) PA_MMA("add.u64 a1, %1, " #OFF ";", "a1", OFF, P)
  asm volatile("{\n\t.reg .pred p, e;\n\t.reg .b64 a1, b1;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.ne.u32 e, %5, 0;\n\t" PA_STEP(0, "p")
                   PA_STEP(16, "1") PA_STEP(32, "1") PA_STEP(48, "1") PA_STEP(64, "1") PA_STEP(80, "1") PA_STEP(96, "1") PA_STEP(112, "1") "}" ::"r"(d),
               "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(leader)
               : "memory");
#undef PA_STEP
}

__device__ __forceinline__ void mma_values(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc, int steps, uint32_t leader) {
#define PA_STEP(AOFF, BOFF, P) PA_MMA("add.u32 a1, %1, " #AOFF ";", "[a1]", BOFF, P)
  if (steps == 4) {
    asm volatile("{\n\t.reg .pred p, e;\n\t.reg .b32 a1;\n\t.reg .b64 b1;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.ne.u32 e, %5, 0;\n\t" PA_STEP(
                     0, 0, "p") PA_STEP(8, 256, "1") PA_STEP(16, 512, "1") PA_STEP(24, 768, "1") "}" ::"r"(d),
                 "r"(a), "l"(b), "r"(idesc), "r"(acc), "r"(leader)
                 : "memory");
  } else {
    for (int i = 0; i < steps; ++i)
      asm volatile("{\n\t.reg .pred p, e;\n\t.reg .b32 a1;\n\t.reg .b64 b1;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.ne.u32 e, %5, 0;\n\t" PA_STEP(
                       0, 0, "p") "}" ::"r"(d),
                   "r"(a + 8 * i), "l"(b + 256 * i), "r"(idesc), "r"(acc | (uint32_t)i), "r"(leader)
                   : "memory");
  }
#undef PA_STEP
}
#undef PA_MMA
static_assert(kPlaneGroup == 16 * 256, "a step of values in a descriptor");

// A piece of the pair's range: tiles j0 .. j1 - 1 of a (unit, head).
struct Piece {
  int unit, head, j0, j1, nt;
  bool first, last;  // of the segment's tiles
};

// The roles walk the CTA's pieces each on its own.
struct Walk {
  Pos pos;
  int left;         // tiles of the range from here on
  int item, items;  // of the list
  __device__ __forceinline__ Walk(const PromptParams& p, int pair) {
    left = item = items = 0;
    if (p.listed) {
      item = p.first[pair];
      items = p.first[pair + 1];
    } else {
      pos = start_of(p, pair);
      left = p.start[pair + 1].tile - pos.tile;  // at least 1
    }
  }
  __device__ __forceinline__ bool next(const PromptParams& p, Piece& x) {
    if (p.listed) {
      if (item == items) return false;
      const int seg = p.list[item++];
      x.unit = seg / p.n_kv_heads;
      x.head = seg - x.unit * p.n_kv_heads;
      x.j0 = 0;
      x.j1 = x.nt = ceil_div(span_of(p.unit[x.unit], p.window, p.sinks).end, kKeys);
      x.first = x.last = true;
      return true;
    }
    if (left == 0) return false;
    x.unit = pos.unit;
    x.head = pos.head;
    x.nt = pos.nt;
    x.j0 = pos.j;
    x.j1 = min(pos.nt, pos.j + left);
    x.first = pos.j == 0;
    x.last = x.j1 == pos.nt;
    left -= x.j1 - x.j0;
    pos.j = x.j1 - 1;
    if (left > 0) advance(p, pos);
    return true;
  }
};

// Keys of tile j of a unit, up to 128, and the same in whole steps of an MMA.
__device__ __forceinline__ int tile_keys(const Span& s, int j) { return min(kKeys, s.end - j * kKeys); }
__device__ __forceinline__ int whole16(int n) { return (n + 15) & ~15; }

__device__ __forceinline__ void bulk_copy(uint32_t dst, const uint8_t* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
               "r"(bytes), "r"(bar)
               : "memory");
}

// Rows r0 .. r1 - 1 (whole eights) of a CTA's query rows by one warp as binary16 into Q, rows from `rows`
// on as zeros (stage_q_begin's layout and range).  Lane: row r8 + lane % 8, slots lane / 8 + 4 i.
// 16-bit rows are copied asynchronously, all at once (begin), and bfloat16 converted where it
// lies (end).
__device__ __forceinline__ void load_queries_begin(const PromptParams& p, int token, int row0, int rows, int head, uint32_t q, int r0, int r1, int lane) {
#pragma unroll 1
  for (int r8 = r0; r8 < r1; r8 += 8) {
    const int row = r8 + (lane & 7), rg = row0 + row;
    const uint32_t to = q + canon(row, lane >> 3, kD / 8);
    const long long at = (token + rg / kGqa) * p.q_stride + (head * kGqa + rg % kGqa) * kD + 8 * (lane >> 3);
    if (row >= rows) {
#pragma unroll
      for (int i = 0; i < 8; ++i) sts128_zero(to + 512 * i);
    } else if (p.q_type == PA_DT_F32) {
      const float4* src = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p.q) + at);
      uint32_t top = 0;
#pragma unroll 4
      for (int i = 0; i < 8; ++i) {
        const float4 x = __ldg(src + 8 * i), y = __ldg(src + 8 * i + 1);
        const uint4 v = make_uint4(pack_half2(x.x, x.y), pack_half2(x.z, x.w), pack_half2(y.x, y.y), pack_half2(y.z, y.w));
        top = larger2(larger2(larger2(top, v.x), v.y), larger2(v.z, v.w));
        sts128(to + 512 * i, v);
      }
      q_range(top, to);
    } else {
      const uint8_t* src = p.q + 2 * at;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + 512 * i), "l"(src + 64 * i) : "memory");
    }
  }
}

__device__ __forceinline__ void load_queries_end(const PromptParams& p, uint32_t q, int r0, int r1, int lane) {
  if (p.q_type == PA_DT_F32) return;
  asm volatile("cp.async.wait_all;" ::: "memory");
  if (p.q_type != PA_DT_BF16) return;
#pragma unroll 1
  for (int r8 = r0; r8 < r1; r8 += 8) {
    const uint32_t to = q + canon(r8 + (lane & 7), lane >> 3, kD / 8);
    uint4 v[8];
    __nv_bfloat162 top = __floats2bfloat162_rn(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = lds128(to + 512 * i);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t u[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        top = __hmax2(top, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&u[k])));
        u[k] = pack_half2(__uint_as_float(u[k] << 16), __uint_as_float(u[k] & 0xffff0000u));
      }
      sts128(to + 512 * i, make_uint4(u[0], u[1], u[2], u[3]));
    }
    // the bfloat16 numbers from 65536 on round to binary16's infinity, those before do not (q_range)
    if (fmaxf(__low2float(top), __high2float(top)) >= 65536.f)
      asm volatile("st.shared.b16 [%0], %1;" ::"r"(to), "h"((unsigned short)0x7fff) : "memory");
  }
}

// This warp's 32 rows of O (lane = row), times f (0: zeros), to rows of global memory by way of
// shared memory at `stage` (16 KB of the warp's own), so that a store writes whole rows.
// to: where this lane's row goes (or NULL), of `type`.  done(): O has been read.  One body for
// all types, 32 columns at a time: a piece's end meets cold instruction caches as it is.
template <class Done>
__device__ __forceinline__ void write_rows(uint32_t from, float f, uint32_t stage, int lane, uint8_t* to, int type, Done&& done) {
  const bool wide = type == PA_DT_F32;
  const int passes = wide ? 2 : 1, steps = wide ? 4 : 8;  // of 512 bytes of each row, of 32 columns
  const uint32_t row = stage + 512 * lane, r7 = lane & 7;
  const uint64_t f2 = pack2(f, f);
#pragma unroll 1
  for (int pass = 0; pass < passes; ++pass) {
#pragma unroll 1
    for (int i = 0; i < steps; ++i) {
      uint32_t o[32];
      tmem_ld32(from + 32 * (steps * pass + i), o);
      tmem_ld_wait();
      loaded(o);
      if (f == 0.f) {  // whatever O holds
#pragma unroll
        for (int k = 0; k < 32; ++k) o[k] = 0u;
      }
#pragma unroll
      for (int k = 0; k < 32; k += 2) put2(o + k, mul2(get2(o + k), f2));
      // chunk x of row r lies at x ^ (r & 7)
      if (wide) {
#pragma unroll
        for (int k = 0; k < 8; ++k) sts128(row + (((8 * i + k) ^ r7) << 4), make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]));
      } else {
        uint32_t h[16];
        if (type == PA_DT_F16) {
#pragma unroll
          for (int k = 0; k < 16; ++k) h[k] = pack_half2(__uint_as_float(o[2 * k]), __uint_as_float(o[2 * k + 1]));
        } else {
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(__uint_as_float(o[2 * k]), __uint_as_float(o[2 * k + 1]));
            h[k] = *reinterpret_cast<const uint32_t*>(&b);
          }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) sts128(row + (((4 * i + k) ^ r7) << 4), make_uint4(h[4 * k], h[4 * k + 1], h[4 * k + 2], h[4 * k + 3]));
      }
    }
    __syncwarp();
    if (pass + 1 == passes) done();
    const unsigned long long mine = reinterpret_cast<unsigned long long>(to ? to + 512 * pass : nullptr);
#pragma unroll 4
    for (int r = 0; r < 32; ++r) {
      uint8_t* at = reinterpret_cast<uint8_t*>(__shfl_sync(0xffffffffu, mine, r));
      const uint4 v = lds128(stage + 512 * r + ((lane ^ (r & 7)) << 4));
      if (at) *reinterpret_cast<uint4*>(at + 16 * lane) = v;
    }
    __syncwarp();
  }
}

__global__ void __launch_bounds__(kPThreads, 1) pa_prompt_kernel(const __grid_constant__ PromptParams p) {
  using SM = PSmem;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + ((1024 - (raw & 1023)) & 1023);
  const uint32_t base = smem_u32(smem);
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_rank();
  const int pair = (int)(blockIdx.x >> 1), cta_row0 = kCtaRows * (int)rank;  // this CTA's rows of a unit
  // Hand-offs (tile j, piece i of the pair's range).  What the MMAs complete is told both
  // CTAs (commit_pair), what they wait for is told the first one:
  //   full [stage]                copies -> MMA: the first CTA's own, and the second's word of its own
  //   empty [stage]               MMA -> copies
  //   q_full / q_empty [i & 1]    query rows of piece i in Q / its last S done
  //   s_full [j & 1]              S(j) in tensor memory
  //   p_full [j & 1]              P(j) in its place
  //   pv_done [j & 1]             O holds tile j
  //   o_free                      piece i's O has been read
  // and within a CTA:
  //   l_full [i & 1]              piece i's sums and references in shared memory
  // A role whose wait expires stops: it arrives nowhere any more.
  const uint32_t full = base + SM::kBar, empty = full + 8 * kNStages, q_full = empty + 8 * kNStages, q_empty = q_full + 16,
                 s_full = q_empty + 16, p_full = s_full + 16, pv_done = p_full + 16, o_free = pv_done + 16, l_full = o_free + 8,
                 drain = l_full + 16;
  volatile int* abort = reinterpret_cast<volatile int*>(smem + SM::kMisc);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + SM::kMisc + 4);
  volatile int* leave = reinterpret_cast<volatile int*>(smem + SM::kMisc + 8) + 2 * (w & 3);  // of even, odd tiles
  if (tid < 128 && lane == 0) leave[0] = leave[1] = 0;
  if (tid == 0) {
    *abort = 0;
    for (int i = 0; i < kNStages; ++i) {
      mbar_init(full + 8 * i, rank == 0 ? 2 : 1);
      mbar_init(empty + 8 * i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(q_full + 8 * i, 8);
      mbar_init(q_empty + 8 * i, 1);
      mbar_init(s_full + 8 * i, 1);
      mbar_init(p_full + 8 * i, 2 * kPSmWarps);
      mbar_init(pv_done + 8 * i, 1);
      mbar_init(l_full + 8 * i, kPSmWarps);
    }
    mbar_init(o_free, 8);
    mbar_init(drain, 1);
    fence_mbar_init();
  }
  Walk walk(p, pair);
  // The kernel before this one (the keys', or a launch of the same call) lets it start only when
  // what came before that is complete: queries may be read at once.  Keys are read, and anything
  // is written, behind the wait (the copies' and the results' warps).
  if (w < kPSmWarps) {  // the first piece's rows
    Walk ahead = walk;
    Piece y;
    ahead.next(p, y);
    const PromptUnit& u = p.unit[y.unit];
    load_queries_begin(p, u.token, unit_row0(u) + cta_row0, unit_rows(u) - cta_row0, y.head, base + SM::kQ, 16 * w, 16 * w + 16, lane);
  }
  if (w == 0) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "r"(kTmemCols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_arrive();  // this CTA's barriers are there
  tc_fence_after();
  // All of tensor memory is the pair's, so its columns start at 0 in both.
  const bool whole = *tmem_slot == 0;
  if (!whole && tid == 0) record_error(p.err, PA_ERR_CUDA);
  if (w < kPSmWarps) load_queries_end(p, base + SM::kQ, 16 * w, 16 * w + 16, lane);
  cluster_wait();  // and the other's
  int issued = 0;
  uint32_t slots = 0, parities = 0;  // stages that this warp copied into, and their last use's parity
  Piece x;

  if (!whole) {
  } else if (w >= kCopyWarp) {
    // ---- copies: K(0), then K(j + 1) before V(j); a stage each 128 dims of K (64 keys: the CTA's) or
    // 64 keys of V (128 dims: the CTA's).  One warp copies K and one V, so that one's waits and set-up
    // overlap the other's copies (a copy of 16 KB holds its warp for 470 cycles; one warp for both takes 2600
    // cycles a tile, the copy engine alone 2040); both count all stages.  Each waits for its own stages alone,
    // which means the phase that it says: consecutive ones of a warp are at most three apart, so
    // when the earlier one's was free all that lie two uses back were.
    const bool is_k = w == kCopyWarp;
    bool live = true;
    auto stage = [&](bool mine, uint32_t bytes) -> int {  // the next stage, once it is free; -1: the other warp's, or the wait expired
      const int s = issued % kNStages, use = issued / kNStages;
      if (mine && live && use > 0 && !warp_wait(empty + 8 * s, (use - 1) & 1, p.err, abort)) live = false;
      if (!live) return -1;
      ++issued;
      if (!mine) return -1;
      slots |= 1u << s;
      parities = (parities & ~(1u << s)) | (uint32_t)(use & 1) << s;
      if (lane == 0) mbar_arrive_expect_tx(full + 8 * s, bytes);
      __syncwarp();
      return s;
    };
    // places v .. end - 1 of a plane
    auto copy = [&](const PromptUnit& u, const Span& s, int edge, const uint8_t* plane, int v, int end, int st) {
      for (int a = v; a < end;) {
        const Run r = run_of(u, s, edge, a, end);
        if (lane == 0)
          bulk_copy(base + SM::kRing + st * kStageBytes + ((a - v) >> 4) * kPlaneGroup, plane + (long long)r.group * kPlaneGroup,
                    ((r.stop - a) >> 4) * kPlaneGroup, full + 8 * st);
        a = r.stop;
      }
      __syncwarp();
    };
    auto keys = [&](const Piece& x, const Span& s, int j) {
      const PromptUnit& u = p.unit[x.unit];
      const uint8_t* k = p.k + ((long long)u.group0 * p.n_kv_heads + (long long)x.head * u.groups) * kGroupBytes;
      const int v = j * kKeys + 64 * (int)rank, end = max(v, min(v + 64, j * kKeys + whole16(tile_keys(s, j))));
      for (int h = 0; h < 2 && live; ++h) {
        const int st = stage(is_k, (uint32_t)(end - v) * 256);
        if (st >= 0) copy(u, s, -1, k + (long long)h * u.groups * kPlaneGroup, v, end, st);
      }
    };
    auto vals = [&](const Piece& x, const Span& s, int j) {
      const PromptUnit& u = p.unit[x.unit];
      const uint8_t* k = p.v + ((long long)u.group0 * p.n_kv_heads + (long long)x.head * u.groups) * kGroupBytes + (long long)rank * u.groups * kPlaneGroup;
      const int v = j * kKeys, n16 = whole16(tile_keys(s, j));
      for (int q = 0; q < n16 && live; q += 64) {
        const int m = min(64, n16 - q), st = stage(!is_k, (uint32_t)m * 256);
        if (st >= 0) copy(u, s, u.edge, k, v + q, v + q + m, st);
      }
    };
    bool more = walk.next(p, x);
    Span s = span_of(p.unit[x.unit], p.window, p.sinks);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (is_k && lane == 0) asm volatile("griddepcontrol.launch_dependents;");
    keys(x, s, x.j0);
    while (more && live) {
      for (int j = x.j0; j + 1 < x.j1 && live; ++j) {
        keys(x, s, j + 1);
        vals(x, s, j);
      }
      const Piece before = x;
      const Span was = s;
      more = walk.next(p, x);
      if (more && live) {
        s = span_of(p.unit[x.unit], p.window, p.sinks);
        keys(x, s, x.j0);
      }
      vals(before, was, before.j1 - 1);
    }
  } else if (w == kMmaWarp && rank != 0) {
    // ---- the second CTA's copies, told the first one
    int used = 0;
    bool live = true;
    auto pass = [&](int n) {
      for (int i = 0; i < n && live; ++i, ++used) {
        const int st = used % kNStages;
        live = warp_wait(full + 8 * st, (used / kNStages) & 1, p.err, abort);
        if (live && lane == 0) arrive_first(full + 8 * st, rank);
        __syncwarp();
      }
    };
    while (live && walk.next(p, x)) {
      const Span s = span_of(p.unit[x.unit], p.window, p.sinks);
      for (int t = x.j0; t < x.j1 && live; ++t) pass(2 + (whole16(tile_keys(s, t)) > 64 ? 2 : 1));
    }
  } else if (w == kMmaWarp) {
    // ---- MMA issue by the whole warp, an elected lane issuing.  After an expired wait no
    // further MMA is issued; what was ends before the pair does.
    const uint32_t leader = elect_one();
    bool dead = false;
    uint32_t stage = 0, phase = 0;  // the next stage, and its use's parity
    uint32_t scored = 0, piece = 0;  // pieces whose S, whose PV has begun
    auto wait = [&](uint32_t bar, uint32_t parity) {
      if (!dead) dead = !warp_wait(bar, parity, p.err, abort);
      return !dead;
    };
    auto next_stage = [&]() -> uint32_t {  // waits for it
      const uint32_t st = stage;
      wait(full + 8 * st, phase);
      tc_fence_after();
      if (++stage == kNStages) {
        stage = 0;
        phase ^= 1;
      }
      return st;
    };
    const uint32_t s_idesc = idesc_f16_f32(256, kKeys), pv_idesc = idesc_f16_f32(256, kD);
    // S of tile t of a piece, the range's j
    auto score = [&](const Piece& x, int t, int j) {
      if (t == x.j0) {
        if (!wait(q_full + 8 * (scored & 1), (scored >> 1) & 1)) return;
        ++scored;
      }
      const uint64_t qdesc = smem_desc(base + SM::kQ + ((scored - 1) & 1) * SM::kQBytes, 128, 4096);
      for (int h = 0; h < 2; ++h) {
        const uint32_t st = next_stage();
        if (dead) return;
        const uint64_t kdesc = smem_desc(base + SM::kRing + st * kStageBytes, 128, 2048);
        mma_scores(kPSCol + 128 * (j & 1), qdesc + 128 * h, kdesc, s_idesc, h, leader);
        commit_pair(empty + 8 * st);
      }
      commit_pair(s_full + 8 * (j & 1));
      if (t + 1 == x.j1) commit_pair(q_empty + 8 * ((scored - 1) & 1));
    };
    int j = 0;  // the range's tile
    bool more = walk.next(p, x);
    score(x, x.j0, 0);
    while (more && !dead) {
      const Piece now = x;
      const Span s = span_of(p.unit[now.unit], p.window, p.sinks);
      for (int t = now.j0; t < now.j1 && !dead; ++t, ++j) {
        if (t + 1 < now.j1) {
          score(now, t + 1, j + 1);
        } else {
          more = walk.next(p, x);
          if (more) score(x, x.j0, j + 1);
        }
        if (!wait(p_full + 8 * (j & 1), (j >> 1) & 1)) break;
        if (t == now.j0 && piece > 0 && !wait(o_free, (piece - 1) & 1)) break;
        tc_fence_after();
        const int n16 = whole16(tile_keys(s, t));
        for (int q = 0; q < n16 && !dead; q += 64) {
          const uint32_t st = next_stage();
          if (dead) break;
          const uint64_t vdesc = smem_desc(base + SM::kRing + st * kStageBytes, 2048, 128);
          const uint32_t a = kPSCol + 128 * (j & 1) + q / 2;
          mma_values(kPOCol, a, vdesc, pv_idesc, (uint32_t)((t - now.j0) | q), min(64, n16 - q) >> 4, leader);
          commit_pair(empty + 8 * st);
        }
        if (dead) break;
        commit_pair(pv_done + 8 * (j & 1));
      }
      ++piece;
    }
    // what was issued, and every commit, ends before the pair's memory is given back
    commit_pair(drain);
    mbar_wait(drain, 0, p.err, abort, /*honour_abort=*/false);
    __syncwarp();
  } else if (w >= kAuxWarp0) {
    // ---- query rows of a piece into Q, two pieces ahead of its results; a finished piece's O to its place
    const int quarter = w & 3;
    bool live = true;
    uint32_t loads = 0;  // pieces whose rows are in Q
    Walk ahead = walk;
    auto load = [&]() {  // the next piece's rows, if there is one
      Piece y;
      if (!live || !ahead.next(p, y)) return;
      if (loads > 1 && !(live = warp_wait(q_empty + 8 * (loads & 1), ((loads >> 1) - 1) & 1, p.err, abort))) return;
      const PromptUnit& u = p.unit[y.unit];
      const int rows = unit_rows(u) - cta_row0;  // of this CTA
      const uint32_t q = base + SM::kQ + (loads & 1) * SM::kQBytes;
      load_queries_begin(p, u.token, unit_row0(u) + cta_row0, rows, y.head, q, 32 * quarter, 32 * quarter + 32, lane);
      load_queries_end(p, q, 32 * quarter, 32 * quarter + 32, lane);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) arrive_first(q_full + 8 * (loads & 1), rank);
      __syncwarp();
      ++loads;
    };
    Piece first_piece;  // its rows are the softmax warps' to load, who have nothing else to do yet
    ahead.next(p, first_piece);
    loads = 1;
    load();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const float* sums = reinterpret_cast<const float*>(smem + SM::kSum);
    const float* refs = reinterpret_cast<const float*>(smem + SM::kRef);
    int tiles = 0;  // of the pieces so far
    for (uint32_t i = 0; live && walk.next(p, x); ++i) {
      tiles += x.j1 - x.j0;
      const uint32_t j = (uint32_t)tiles - 1;  // the piece's last tile: after its PV, its S is done too
      if (!(live = warp_wait(l_full + 8 * (i & 1), (i >> 1) & 1, p.err, abort) &&
                   warp_wait(pv_done + 8 * (j & 1), (j >> 1) & 1, p.err, abort)))
        break;
      tc_fence_after();
      const PromptUnit& u = p.unit[x.unit];
      const int row = 32 * quarter + lane, row0 = unit_row0(u) + cta_row0, rows = unit_rows(u) - cta_row0;
      const float l = sums[(i & 1) * 256 + row] + sums[(i & 1) * 256 + 128 + row], m = refs[(i & 1) * 128 + row];
      const uint32_t from = kPOCol + ((uint32_t)(32 * quarter) << 16);
      // by way of this warp's own query rows, whose last product is done and which load() below overwrites
      const uint32_t stage = base + SM::kQ + (i & 1) * SM::kQBytes + 32 * quarter * 512;
      auto done = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_first(o_free, rank);
        __syncwarp();
      };
      float f = 1.f;
      uint8_t* to = nullptr;
      int type = PA_DT_F32;
      if (x.first && x.last) {  // the whole segment: the result
        const bool other = __ldg(p.lens + u.seq) != u.len;
        if (other && row == 0) record_error(p.err, PA_ERR_BOUNDS);
        const float sum = other ? 0.f : l;
        const int rg = row0 + row, tok = rg / kGqa, h = x.head * kGqa + rg - tok * kGqa;
        f = sum != 0.f ? 1.f / sum : 0.f;
        type = p.out_type;
        if (row < rows) {
          if (p.lse) p.lse[(long long)(u.token + tok) * p.n_q_heads + h] = sum != 0.f ? (m + log2f(sum)) * pa_split::kLn2 : -INFINITY;
          to = p.out + ((u.token + tok) * p.out_stride + h * kD) * (type == PA_DT_F32 ? 4 : 2);
        }
      } else if (row < rows) {
        const long long slot = slot_of(x.first, x.last, pair, p.slot_rows) + cta_row0 + row;
        p.part_ml[slot] = make_float2(m, l);
        to = reinterpret_cast<uint8_t*>(p.part_o + slot * kD);
      }
      __syncwarp();
      write_rows(from, f, stage, lane, to, type, done);
      load();
    }
  } else {
    // ---- softmax: keys 64 half .. + 63 of a tile, row 32 quarter + lane
    const int half = w >> 2, quarter = w & 3, row = 32 * quarter + lane;
    const uint32_t lanes = (uint32_t)(32 * quarter) << 16;
    float* red = reinterpret_cast<float*>(smem + SM::kRed);
    float* sums = reinterpret_cast<float*>(smem + SM::kSum);
    float* refs = reinterpret_cast<float*>(smem + SM::kRef);
    const uint64_t scale2 = pack2(p.scale_log2, p.scale_log2);
    {
      fence_proxy_async_smem();
      __syncwarp();
      named_bar_sync(1 + quarter, 64);
      if (half == 0 && lane == 0) arrive_first(q_full, rank);
      __syncwarp();
    }
    if (p.wide) asm volatile("griddepcontrol.wait;" ::: "memory");  // which keys are wide
    // The two warps of a quarter share its rows, and meet in every tile (barrier 1 + quarter).  A
    // warp whose wait expired arrives nowhere any more and says so (the tile's `leave`) before
    // they meet first; after it both leave, until then both walk the same tiles, and so the
    // same barriers.
    const uint32_t meet = 1 + quarter;
    bool live = true, gone = false;
    uint32_t piece = 0;
    int j = 0;  // the CTA's tile
    while (!gone && walk.next(p, x)) {
      const PromptUnit& u = p.unit[x.unit];
      const Span s = span_of(u, p.window, p.sinks);
      const int last_pos = u.pos + (unit_row0(u) + unit_rows(u) - 1) / kGqa;
      const int last_lo = last_pos >= p.window ? last_pos - p.window + 1 : 0;
      const RowKeys mine = row_keys(u, s, cta_row0 + row, p.window);
      const long long reg = (long long)u.group0 * p.n_kv_heads + (long long)x.head * u.groups;
      float ref = 0.f;
      uint64_t l2 = 0;  // sums of weights over this thread's keys, in two
      // which keys of a tile are wide (all rows': the same), read a tile ahead
      uint16_t flags[4] = {};
      auto read_flags = [&](int t) {
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const int v = t * kKeys + 64 * half + 16 * g;
          flags[g] = p.wide && t < x.j1 && v < s.end ? __ldg(reinterpret_cast<const uint16_t*>(p.wide) + reg + group_of(u, s, v)) : 0;
        }
      };
      read_flags(x.j0);
      for (int t = x.j0; t < x.j1; ++t, ++j) {
        const int v0 = t * kKeys + 64 * half;
        const uint64_t wide = (uint64_t)(flags[0] | (uint32_t)flags[1] << 16) | (uint64_t)(flags[2] | (uint32_t)flags[3] << 16) << 32;
        if (p.wide) read_flags(t + 1);
        live = live && warp_wait(s_full + 8 * (j & 1), (j >> 1) & 1, p.err, abort);
        if (!live) leave[j & 1] = 1;
        tc_fence_after();
        const uint32_t s_at = kPSCol + 128 * (j & 1) + lanes;
        if (wide) {  // rare, and so in a loop of its own, in tensor memory
#pragma unroll 1
          for (int c = 0; c < 64; c += 8) {
            uint32_t y[8];
            tmem_ld8(s_at + 64 * half + c, y);
            tmem_ld_wait();
            loaded(y);
#pragma unroll
            for (int k = 0; k < 8; ++k) y[k] = __float_as_uint(__uint_as_float(y[k]) * ((wide >> c) >> k & 1 ? 256.f : 1.f));
            tmem_st8(s_at + 64 * half + c, y);
          }
          tmem_st_wait();
        }
        uint32_t a[2][32];
        tmem_ld32(s_at + 64 * half, a[0]);
        tmem_ld32(s_at + 64 * half + 32, a[1]);
        tmem_ld_wait();
        loaded(a[0]);
        loaded(a[1]);
        if (!sees_all(s, t * kKeys, u.pos, last_lo, p.sinks)) {  // what the row does not see becomes -inf
          const uint64_t seen = mine.bits(v0, p.sinks);
          const uint32_t word[2] = {(uint32_t)seen, (uint32_t)(seen >> 32)};
#pragma unroll
          for (int k = 0; k < 64; ++k)
            if (!(word[k >> 5] >> (k & 31) & 1)) a[k >> 5][k & 31] = 0xff800000u;
        }
        const uint64_t nref = pack2(-ref, -ref);
        float top = -INFINITY;
#pragma unroll
        for (int k = 0; k < 64; k += 2) {
          uint32_t* r = &a[k >> 5][k & 31];
          put2(r, fma2(get2(r), scale2, nref));
          top = fmaxf(top, fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1])));
        }
        const bool first_tile = t == x.j0;
        const bool raise = bar_or(meet, 64, first_tile || top > kLazyLog2);
        if (leave[j & 1]) {
          gone = true;
          break;
        }
        if (raise) {
          red[half * kCtaRows + row] = top;
          __syncwarp();
          named_bar_sync(meet, 64);
          const float m = fmaxf(red[row], red[kCtaRows + row]);
          // a row that sees no key yet keeps a reference of 0; it will see none later in the piece either
          const float d = first_tile ? (m == -INFINITY ? 0.f : m) : fmaxf(m, 0.f);
          ref += d;
          const uint64_t nd = pack2(-d, -d);
#pragma unroll
          for (int k = 0; k < 64; k += 2) {
            uint32_t* r = &a[k >> 5][k & 31];
            put2(r, add2(get2(r), nd));
          }
          if (first_tile) {
            l2 = 0;
          } else if (__any_sync(0xffffffffu, d != 0.f)) {  // O holds the tiles before: half of the dims
            const float f = ex2(-d);
            l2 = mul2(l2, pack2(f, f));
            if (!warp_wait(pv_done + 8 * ((j - 1) & 1), ((j - 1) >> 1) & 1, p.err, abort)) {
              live = false;
              leave[(j + 1) & 1] = 1;
            }
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < kD / 2; c += 8) {
              uint32_t o[8];
              tmem_ld8(kPOCol + 128 * half + c + lanes, o);
              tmem_ld_wait();
              loaded(o);
#pragma unroll
              for (int k = 0; k < 8; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
              tmem_st8(kPOCol + 128 * half + c + lanes, o);
            }
          }
        }
        uint32_t h[32];
#pragma unroll
        for (int k = 0; k < 32; ++k) {
          const uint32_t* r = &a[k >> 4][2 * (k & 15)];
          const float e0 = ex2(__uint_as_float(r[0])), e1 = ex2(__uint_as_float(r[1]));
          l2 = add2(l2, pack2(e0, e1));
          h[k] = pack_half2(e0, e1);
        }
        tmem_st32(s_at + 32 * half, h);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (live && lane == 0) arrive_first(p_full + 8 * (j & 1), rank);
        __syncwarp();
      }
      if (gone) break;
      const float2 l = unpack2(l2);
      sums[(piece & 1) * 256 + half * 128 + row] = l.x + l.y;
      if (half == 0) refs[(piece & 1) * 128 + row] = ref;
      __syncwarp();
      if (live && lane == 0) mbar_arrive(l_full + 8 * (piece & 1));
      __syncwarp();
      ++piece;
    }
  }
  tc_fence_before();
  __syncthreads();
  // after an expired wait, copies that nobody waited for must still land
  if (w >= kCopyWarp && *abort) {
    for (int i = 0; i < kNStages; ++i)
      if (slots >> i & 1) mbar_wait(full + 8 * i, parities >> i & 1, p.err, abort, false, kWaitTimeoutNs / 8);
  }
  __syncwarp();
  cluster_arrive();
  cluster_wait();  // no MMA, arrival or copy is on its way to either CTA any more
  if (w == 0) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(*tmem_slot), "r"(kTmemCols) : "memory");
  }
}

}  // namespace

namespace {

template <class P>
pa_status launch_one(void (*kernel)(P), const P& p, int grid, int cluster, int threads, int smem, cudaStream_t cs) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = cs;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, p) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace

pa_status launch_prepare(const PrepareParams& p, int sms, cudaStream_t cs) {
  const long long items = (long long)p.groups * 4 * p.n_kv_heads, ctas = (items + kPrepareWarps - 1) / kPrepareWarps;
  return launch_one(pa_prompt_prepare_kernel, p, (int)(ctas < 16ll * sms ? ctas : 16ll * sms), 1, 32 * kPrepareWarps, 0, cs);
}

pa_status launch_prompt(const PromptParams& p, cudaStream_t cs) {
  return launch_one(pa_prompt_kernel, p, 2 * p.n_ctas, 2, kPThreads, PSmem::kLaunch, cs);
}

pa_status prompt_ready() {
  return cudaFuncSetAttribute(pa_prompt_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, PSmem::kLaunch) == cudaSuccess ? PA_OK
                                                                                                                            : PA_ERR_CUDA;
}

}  // namespace pa_prefix
