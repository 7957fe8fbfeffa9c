// Decode with shared prefixes on the fifth-generation tensor core (sm_103a).
//
// The mathematics.  A group of sequences shares its first P keys; query row r
// (a token's query head) of any of its sequences attends to those P keys and
// to its own sequence's later ones.  The softmax splits: with m, l, O the
// maximum, the sum of weights and the weighted V of a part of the keys, the
// parts merge by log-sum-exp.  So a prefix is one dense contraction of all the
// group's query rows (6 per token and KV head) with its keys, read once, and
// each suffix a small one of its own.
//
//   segment  = (group, KV head, tile of 64 query rows) over the prefix's keys,
//              or (sequence, KV head, row tile) over the suffix's; cut into key
//              tiles of 128; all tiles of the batch are laid end to end by
//              their cost, every segment after a lead that stands for the cost
//              of a piece, and cut into one equal contiguous range per CTA (one
//              CTA per SM).  A range's share of a segment is a piece; every
//              piece leaves (m, l) and O in the workspace for the merge.
//   S^T      = K Q^T    tcgen05.mma M = 128 keys, N = query rows (16 to 64),
//   O^T     += V^T P^T  tcgen05.mma M = 128 dims (twice), N = query rows,
//              K = keys.
//
// Why transposed.  A decode has few query rows: as the MMA's M dimension (128)
// most of them would be padding, as its N dimension (a multiple of 16) none
// is.  K and V are then the A operands, and those may lie in tensor memory:
// a dequantising warp goes from raw quants in shared memory through registers
// into tensor memory, and the binary16 K and V never touch shared memory,
// whose bandwidth a kernel with both operands there runs out of first.  An MMA
// with A in tensor memory takes N / 2 cycles (measured: 24.6 with 48 columns, 32.4
// with 64; 44 to 48 with A in shared memory, whatever N), so 128 keys cost 32 of
// them, about 1000 cycles for 64 rows.
//
// Tensor memory (512 columns x 128 lanes): O^T dims 0-127 in columns 0-63 and
// dims 128-255 in 64-127 (lane = dim, column = query row), two buffers of S^T
// in 128-255 (lane = key), and four operand units of 64 columns.  A K unit is
// 128 keys x 128 dims (lane = key, a column = two dims), a V unit 64 keys x 256
// dims (lane = dim, a column = two keys, dims 128-255 in its upper 32 columns);
// each is worth eight MMAs and is refilled as soon as they have read it.
//
// Warps, hand-offs on mbarriers, every wait bounded:
//   0-7    K dequantisation: (half of the dims, lane quarter), thread = key; and
//          the query rows of every piece, eight by each warp;
//   8-15   V dequantisation: (half of the tile's keys, lane quarter), by
//          transposing ldmatrix;
//   16-23  softmax: 16 keys each, all query rows, in mma fragments; P^T goes to
//          shared memory by transposing stmatrix; they also rescale O^T (rarely:
//          the reference maximum is raised only past 2^8) and write the pieces,
//          each while the tile after it is multiplied;
//   24, 25 MMA issue, S^T and O^T; 26, 27 raw K and V copies (cp.async.bulk).
//
// What bounds it.  Neither the tensor core (11 % of a call of 8 x (32768 + 1024)
// keys in Q4_0, 22.9 us, by the counter; a third where tiles of 64 rows follow one
// another) nor the memory, but for binary16 (8 x 98304 keys: 70 us, 5.8 TB/s).  A
// tile of 64 rows takes about 1.6 us, and three chains are about equally long there:
// the softmax of a tile and the step to the next, the dequantisation of V plus half
// of its MMAs, and of K plus half of its.  Seven warps on a scheduler, each in code of
// its own, wait for instructions as much as for anything else: one softmax body for
// all widths instead of four and one copy function instead of two took 64 x (8192 +
// 300) keys from 61 to 49 us, the masks' own loop from 41 to 39.5; unrolling
// the dequantisation by four makes it 50, and operand units of half the size (more
// hand-offs) cost 8 per cent.  A call's first output starts some 8 us after its
// first instruction (table, keys, their conversion, two products, the merge), which
// is what short ones consist of.
//
// The key order inside a group of 16 is key16 below: it is the order in which
// a transposing ldmatrix delivers key pairs to the columns of a V unit, chosen so
// that both its rows and the K threads' row reads fall in different banks.
//
// Range.  A stored key may have values past binary16's 65504 (scale * quant goes to
// 8.3 * 10^6): the values of such a key are taken 2^-8 of what they are, its logits 2^8
// times (dequant_k).  That costs the ordinary case a vote on the scales, 0 to 1 per cent.
// A query value that rounds past 65504 makes its row NaN; a V value past it is infinite.
//
// Precision.  Q, K, V (scale * quant, rounded once) and P are binary16, products
// are accumulated in fp32, m, l and O are fp32, and l sums the weights before
// their rounding.  Rounding K costs a logit 2^-11 |q| |k| scale at most, as much as the
// rounding of Q that fp32 queries meet anyway; keeping K exact would take a second
// product and half again the dequantisation.  On N(0, 1) data the roundings of P, of V and
// of K move the output by 2.1, 1.6 to 2.1 and 1.7 to 2.2 x 10^-4 of its norm, a binary16
// output's own by 2.1.
#pragma once

#include "pa_decode_impl.cuh"
#include "pa_io.cuh"

namespace pa_prefix {

using namespace pa_dev;
using pa_layout::Fmt;
using pa_layout::kGroup;
using pa_split::kD;
using pa_split::kGqa;

constexpr int kKeys = 128;        // keys per tile
constexpr int kStageKeys = 64;    // keys per copy stage and per V unit
constexpr int kRows = 64;         // query rows per row tile
constexpr int kMaxSeqs = 256;     // sequences per launch
constexpr int kMaxGroups = 128;   // shared prefixes per launch (two sequences each at least)
constexpr int kKWarp0 = 0, kVWarp0 = 8, kSmWarp0 = 16, kSWarp = 24, kPvWarp = 25, kCopyKWarp = 26, kCopyVWarp = 27;
constexpr int kThreads = 28 * 32;
constexpr int kSmThreads = 256;
constexpr uint32_t kTmemCols = 512, kOCol = 0, kSCol = 128, kKCol = 256, kVCol = 384;
constexpr int kLead = 12, kTileCost = 9;
constexpr float kLazyLog2 = 8.f;  // logits may pass their reference by this

struct Params {
  static constexpr bool kWindow = false;
  const uint8_t* q;
  const uint8_t* k_pool;
  const uint8_t* v_pool;
  const int32_t* table;
  int32_t* err;
  float2* part_ml;  // (reference maximum in log2 units, sum of weights) per slot row
  float* part_o;    // [slot row][256]
  int q_type, n_qtok, n_kv_heads, n_q_heads, page_size, table_stride, n_blocks;
  int page_shift;  // log2 of page_size, or -1
  int n_seq, n_groups, n_ctas;
  int weigh;                  // 0: tiles take a place each
  int prefix_len, total_len;  // places of the prefixes, of all
  int total_tiles;
  int suffix_row_tiles, suffix_rows;  // row tiles of a suffix segment; rows of its slot
  int suffix_base;                    // first slot row of the suffixes
  float scale_log2;
  int32_t len[kMaxSeqs], start[kMaxSeqs];  // a suffix's keys are start .. len - 1
  int32_t seq_at[kMaxSeqs];                // places of the suffixes before a sequence's
  int32_t seq_tile[kMaxSeqs];              // tiles before a sequence's suffix
  int32_t group_first[kMaxGroups], group_seqs[kMaxGroups], group_keys[kMaxGroups];
  int32_t group_at[kMaxGroups], group_tile[kMaxGroups], group_seg[kMaxGroups];  // places, tiles, segments before a group
  using Live = int;  // live keys of a tile
};

// ------------------------------------------------------------------ the walk

__host__ __device__ constexpr int ceil_div(int a, int b) { return (a + b - 1) / b; }

// A segment of nt tiles takes lead + nt * cost places, a tile stands at the first
// of its own.  CTA i of G has the places i T / G .. (i + 1) T / G - 1 and the tiles
// that stand there: place x is CTA ((x + 1) G - 1) / T's.
struct Cost {
  int lead, tile;
};

// By the query rows of the unit: what tiles of up to 31, 63 and 64 rows and the
// pieces took, fitted over batches of short and long suffixes.  Equal tiles and no
// lead: 64 sequences of 128 + 4096 keys in Q4_0 155 us, 8 of 98304 + 16 in Q8_0 61 us;
// by cost 94.6 and 45.5.
__host__ __device__ constexpr Cost cost_of(int weigh, int rows) {
  return weigh ? Cost{kLead, kTileCost + (rows >= kRows ? 2 : rows / 32)} : Cost{0, 1};
}

struct Pos {
  int unit;        // group or sequence
  int head, rt, j;  // KV head, row tile, key tile
  int nt, nrt;     // key tiles of the segment, row tiles of the (unit, head)
  bool pre;
  int tile;        // number of the tile (set by locate)
};

__device__ __forceinline__ void pos_sizes(const Params& p, Pos& t) {
  if (t.pre) {
    t.nt = ceil_div(p.group_keys[t.unit], kKeys);
    t.nrt = ceil_div(kGqa * p.n_qtok * p.group_seqs[t.unit], kRows);
  } else {
    t.nt = ceil_div(p.len[t.unit] - p.start[t.unit], kKeys);
    t.nrt = p.suffix_row_tiles;
  }
}

__device__ __forceinline__ void advance(const Params& p, Pos& t) {
  if (++t.j < t.nt) return;
  t.j = 0;
  if (++t.rt < t.nrt) return;
  t.rt = 0;
  if (++t.head < p.n_kv_heads) return;
  t.head = 0;
  ++t.unit;
  if (t.pre && t.unit == p.n_groups) {
    t.pre = false;
    t.unit = 0;
  }
  if (!t.pre && t.unit >= p.n_seq) return;  // past the last tile
  pos_sizes(p, t);
}

// The first tile at place x or after it.
__device__ __forceinline__ Pos locate(const Params& p, int x) {
  Pos t;
  t.pre = x < p.prefix_len;
  const int32_t* cum = t.pre ? p.group_at : p.seq_at;
  if (!t.pre) x -= p.prefix_len;
  int lo = 0, hi = (t.pre ? p.n_groups : p.n_seq) - 1;  // the last unit whose first place is <= x
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (cum[mid] <= x) lo = mid; else hi = mid - 1;
  }
  t.unit = lo;
  x -= cum[lo];
  pos_sizes(p, t);
  const Cost c = cost_of(p.weigh, kGqa * p.n_qtok * (t.pre ? p.group_seqs[t.unit] : 1));
  const int len = c.lead + t.nt * c.tile;
  int seg = x / len;
  t.j = (max(x - seg * len - c.lead, 0) + c.tile - 1) / c.tile;
  t.tile = (t.pre ? p.group_tile : p.seq_tile)[t.unit] + seg * t.nt + t.j;
  t.head = seg / t.nrt;
  t.rt = seg - t.head * t.nrt;
  if (t.j == t.nt) {  // past the segment's last tile
    --t.j;
    advance(p, t);
  }
  return t;
}

__device__ __forceinline__ int pos_row0(const Params&, const Pos& t) { return t.rt * kRows; }
__device__ __forceinline__ int pos_seq(const Params& p, const Pos& t) { return t.pre ? p.group_first[t.unit] : t.unit; }
__device__ __forceinline__ int pos_token(const Params& p, const Pos& t) { return pos_seq(p, t) * p.n_qtok; }
__device__ __forceinline__ int pos_key0(const Params& p, const Pos& t) {
  return (t.pre ? 0 : p.start[t.unit]) + t.j * kKeys;
}
__device__ __forceinline__ int pos_end(const Params& p, const Pos& t) {
  return t.pre ? p.group_keys[t.unit] : p.len[t.unit];
}
// Query rows of the segment (the unit's rows of this head and row tile).
__device__ __forceinline__ int pos_rows(const Params& p, const Pos& t) {
  const int all = kGqa * p.n_qtok * (t.pre ? p.group_seqs[t.unit] : 1);
  return min(kRows, all - t.rt * kRows);
}
__device__ __forceinline__ int pos_slot_row(const Params& p, const Pos& t, int cta) {
  if (t.pre) return (cta + p.group_seg[t.unit] + t.head * t.nrt + t.rt) * kRows;
  return p.suffix_base + (cta + (t.unit * p.n_kv_heads + t.head) * t.nrt + t.rt) * p.suffix_rows;
}

// The row of a 16-key group at position p of the tile's key order.
__host__ __device__ constexpr int key16(int p) {
  const int t = p >> 2, e = p & 3;
  return e < 2 ? 2 * t + e : 8 + ((2 * t + (e & 1)) ^ 4);
}

// ------------------------------------------------------------------ shared memory

template <int KT, int VT, bool kWindow = false>
struct Smem {
  static constexpr int kKStage = 4 * pa_layout::group_bytes<KT>(), kVStage = 4 * pa_layout::group_bytes<VT>();
  static constexpr int kQBytes = kRows * kD * 2, kPBytes = kRows * kKeys * 2;
  static constexpr int kQ = 0, kP = kQBytes, kRing = kP + 2 * kPBytes;
  static constexpr int kLiveBytes = kWindow ? 16 * 16 : 64, kInvBytes = kWindow ? kRows * 4 : 0;
  // red, references, tiles, live keys, wide keys, reciprocal sums, barriers
  static constexpr int kTail = 8 * kRows * 4 + 2 * kRows * 4 + 17 * 32 + kLiveBytes + 64 + kInvBytes + 640;
  // K and V stages in rings of their own, both of an even number of stages: a
  // warp reads every second stage of its ring, and so sees every use of those it
  // reads (a parity wait must never be two phases ahead of its barrier).  Two
  // each, then two more to the ring with fewer, as long as they fit.
  static constexpr int kRoom = 232448 - 1024 - kRing - kTail;
  static constexpr int fit(bool v) {
    int nk = 2, nv = 2;
    for (int i = 0; i < 8; ++i) {
      const bool to_k = nk <= nv;
      if ((nk + 2 * to_k) * kKStage + (nv + 2 * !to_k) * kVStage > kRoom) {
        if ((nk + 2 * !to_k) * kKStage + (nv + 2 * to_k) * kVStage > kRoom) break;
        (to_k ? nv : nk) += 2;
      } else {
        (to_k ? nk : nv) += 2;
      }
    }
    return v ? nv : nk;
  }
  static constexpr int kKStages = fit(false), kVStages = fit(true);
  static_assert(2 * (kKStage + kVStage) <= kRoom, "a tile of stages does not fit");
  static constexpr int kVRing = kRing + kKStages * kKStage;
  static constexpr int kRed = kVRing + kVStages * kVStage;
  static constexpr int kRef = kRed + 8 * kRows * 4, kAlpha = kRef + kRows * 4;
  static constexpr int kTile = kAlpha + kRows * 4, kOpening = kTile + 16 * 32, kLeft = kOpening + 32,
                       kWide = kLeft + kLiveBytes, kInv = kWide + 16 * 4, kBar = kInv + kInvBytes;
  // K and V raw full / empty [stages], K and V unit full / empty [2], s full / empty [2], q full / empty [2],
  // p full, pv done, o free [2] each, drain [2], sink
  static constexpr int kNBar = 2 * (kKStages + kVStages) + 8 + 4 + 4 + 9;
  static constexpr int kMisc = kBar + 8 * kNBar;  // abort, tmem base, the softmax's leave, the first tile's place
  static constexpr int kTotal = kMisc + 16 + sizeof(Pos) + 12;
  static constexpr int kLaunch = kTotal + 1024;  // the base is aligned to 1024 inside
  static_assert(kTotal - kBar <= 640 && kLaunch <= 232448, "shared memory");
};

// Canonical K-major byte offset (core matrices of 8 rows x 16 bytes) of row r,
// 8-element slot s, of an operand with `slots` slots per row.
__device__ __forceinline__ uint32_t canon(int r, int s, int slots) {
  return (uint32_t)((((r >> 3) * slots + s) << 7) + ((r & 7) << 4));
}

// ------------------------------------------------------------------ tensor memory

__device__ __forceinline__ void tmem_ld16(uint32_t a, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(a));
}

__device__ __forceinline__ void tmem_ld8(uint32_t a, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(a));
}

__device__ __forceinline__ void tmem_st8(uint32_t a, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(a), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// 16 lanes x 16 columns in the mma fragment distribution: thread 4g + t gets
// (lane g, columns 2t, 2t + 1), (lane g + 8, the same), then columns 8 on.
__device__ __forceinline__ void tmem_ld_frag2(uint32_t a, uint32_t (&u)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7])
               : "r"(a));
}

// Registers of a tensor-memory load are read only after its wait: nothing that
// uses them moves above this.
template <int N>
__device__ __forceinline__ void loaded(uint32_t (&r)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 8)
    asm volatile("" : "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]), "+r"(r[i + 5]),
                      "+r"(r[i + 6]), "+r"(r[i + 7]));
}

// 16 lanes x 16 columns and 16 lanes x 8 columns, the same distribution, stored.
__device__ __forceinline__ void tmem_st_frag2(uint32_t a, const uint32_t (&u)[8]) {
  asm volatile("tcgen05.st.sync.aligned.16x256b.x2.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(a), "r"(u[0]), "r"(u[1]),
               "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7])
               : "memory");
}

__device__ __forceinline__ void tmem_st_frag1(uint32_t a, const uint32_t (&r)[4]) {
  asm volatile("tcgen05.st.sync.aligned.16x256b.x1.b32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(r[0]), "r"(r[1]), "r"(r[2]),
               "r"(r[3])
               : "memory");
}

// ------------------------------------------------------------------ dequantisation
//
// The loops are rolled (K two steps at a time): the roles' code runs side by side
// on every scheduler, and the instruction cache is the first thing that it runs out
// of.

constexpr uint32_t kM1152 = pa_split::kHalf2_m1152, kM1032 = pa_split::kHalf2_m1032, kR16 = pa_split::kHalf2_1_16,
                   kM72 = pa_split::kHalf2_m72, kMagic = pa_split::kMagic64, kR256 = 0x1c001c00u;  // 2^-8 twice

// The larger of two pairs of binary16 numbers, by magnitude.
__device__ __forceinline__ uint32_t larger2(uint32_t x, uint32_t y) {
  const __half2 m = __hmax2(__habs2(*reinterpret_cast<const __half2*>(&x)), __habs2(*reinterpret_cast<const __half2*>(&y)));
  return *reinterpret_cast<const uint32_t*>(&m);
}

// This thread's key, dims 128 kd .. + 127, from raw shared memory into a K
// unit's 64 columns at taddr, 32 dims (16 columns) at a time.  grp: the key's row
// group, r its row there.  Returns the warp's wide keys (lane = bit): those with a
// scale times which the largest quant (128, in Q4_0 8) is past binary16's range.
// Their values are made 2^-8 of what they are, both halves of the dims alike, and the
// softmax multiplies their logits by 2^8.
template <int T>
__device__ __forceinline__ uint32_t dequant_k(uint32_t grp, int r, int kd, uint32_t taddr) {
  const uint32_t row = grp + Fmt<T>::kScales + r * Fmt<T>::kRowQ;
  const int r7 = r & 7;
  uint2 sc = make_uint2(0u, 0u);
  uint32_t wide = 0;
  if constexpr (T != PA_F16) {
    const uint4 d = lds128(grp + 16 * r);  // the row's eight block scales
    sc = kd ? make_uint2(d.z, d.w) : make_uint2(d.x, d.y);
    // 2^9 (Q4_0: 2^13) is 0x6000 (0x7000): from there on the sum has bit 15
    const bool mine = (larger2(larger2(d.x, d.y), larger2(d.z, d.w)) + (T == PA_Q8_0 ? 0x20002000u : 0x10001000u)) & 0x80008000u;
    if (__any_sync(0xffffffffu, mine)) {
      wide = __ballot_sync(0xffffffffu, mine);
      if (mine) sc = make_uint2(hmul2(sc.x, kR256), hmul2(sc.y, kR256));
    }
  }
#pragma unroll 2
  for (int i = 0; i < 4; ++i) {
    const int b = 4 * kd + i;
    uint32_t out[16];
    if constexpr (T == PA_F16) {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const uint4 x = lds128(row + (((4 * b + c) ^ r7) << 4));
        out[4 * c] = x.x;
        out[4 * c + 1] = x.y;
        out[4 * c + 2] = x.z;
        out[4 * c + 3] = x.w;
      }
    } else {
      const uint32_t d2 = prmt((i & 2) ? sc.y : sc.x, 0u, (i & 1) ? 0x3232 : 0x1010);
      if constexpr (T == PA_Q8_0) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const uint4 x = lds128(row + (((2 * b + c) ^ r7) << 4));
          const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t u = w[k] ^ 0x80808080u;  // int8 -> 128 + q as an unsigned byte
            out[8 * c + 2 * k] = hmul2(hadd2(prmt(u, kMagic, 0x4140), kM1152), d2);
            out[8 * c + 2 * k + 1] = hmul2(hadd2(prmt(u, kMagic, 0x4342), kM1152), d2);
          }
        }
      } else {  // Q4_0: word k of the block holds dims 4k .. 4k+3 (low nibbles) and 16 + 4k .. (high)
        const uint4 x = lds128(row + ((b ^ r7) << 4));
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t u = w[k] >> 8;
          out[4 * k] = hmul2(hadd2(and_or(w[k], 0x000f000fu, 0x64006400u), kM1032), d2);
          out[4 * k + 1] = hmul2(hadd2(and_or(u, 0x000f000fu, 0x64006400u), kM1032), d2);
          out[4 * k + 2] = hmul2(hfma2(and_or(w[k], 0x00f000f0u, 0x64006400u), kR16, kM72), d2);
          out[4 * k + 3] = hmul2(hfma2(and_or(u, 0x00f000f0u, 0x64006400u), kR16, kM72), d2);
        }
      }
    }
    tmem_st16(taddr + 16 * i, out);
  }
  return wide;
}

// The four dims at load 0 and at load 1 of an 8-position slot of K's dim order,
// and their order: natural, or for Q4_0 the order of dequant_k's columns.
template <int T>
__device__ __forceinline__ int q_dim(int slot, int half) {
  if (T == PA_Q4_0) return (slot >> 2) * 32 + (slot & 3) * 4 + 16 * half;
  return 8 * slot + 4 * half;
}

// The dim of lane l (of 32) that dequant_v writes.
template <int T>
__host__ __device__ constexpr int v_dim(int l) {
  return T == PA_F16 ? l : 16 * (l >> 4) + 2 * (l & 7) + ((l >> 3) & 1);
}

// The live keys of a stage: its first n, or (of a window) those before a and from b to
// c - 1.
struct FirstKeys {
  int n;
  __device__ __forceinline__ bool all() const { return n >= kStageKeys; }
  __device__ __forceinline__ bool has(int k) const { return k < n; }
};
struct WindowKeys {
  int a, b, c;
  __host__ __device__ __forceinline__ bool all() const { return c >= kStageKeys && (b <= 0 || a >= b || a >= kStageKeys); }
  __host__ __device__ __forceinline__ bool has(int k) const { return k < c && (k < a || k >= b); }
};

// 64 keys x 32 dims twice (blocks b and b + 4) of a V stage into a V unit's 32
// lanes at taddr (lane field included): columns 0-31 and 32-63, eight for every
// 16 keys.  keys: the live keys of the stage; the others' values become zeros,
// whatever bytes lie there.
template <int T, class Keys>
__device__ __forceinline__ void dequant_v(uint32_t stage, int b, const Keys keys, uint32_t taddr, int lane) {
  constexpr int GB = pa_layout::group_bytes<T>(), RQ = Fmt<T>::kRowQ;
  // ldmatrix: matrices 0 and 2 hold rows 0..7 of a group, 1 and 3 rows 8 + (i ^ 4)
  const int mi = lane >> 3, i = lane & 7, r7 = (mi & 1) ? i ^ 4 : i, t = lane & 3;
  uint32_t row = stage + Fmt<T>::kScales + ((mi & 1) * 8 + r7) * RQ;
  // scales of the key pairs (2t, 2t + 1) and 8 + ((2t, 2t + 1) ^ 4): b + 4 is 128 bytes on
  uint32_t sa = stage + 64 * (b >> 1) + 8 * (b & 1) + 16 * t, sb = (sa ^ 32) + 4;
#pragma unroll 1
  for (int g = 0; g < 4; ++g) {
    uint32_t ma = 0xffffffffu, mb = 0xffffffffu;  // live keys of the pairs
    if (!keys.all()) {
      const int ka = 16 * g + 2 * t, kb = 16 * g + 8 + ((2 * t) ^ 4);
      ma = (keys.has(ka) ? 0xffffu : 0u) | (keys.has(ka + 1) ? 0xffff0000u : 0u);
      mb = (keys.has(kb) ? 0xffffu : 0u) | (keys.has(kb + 1) ? 0xffff0000u : 0u);
    }
    [[maybe_unused]] uint32_t xq[4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {  // block b, block b + 4
      [[maybe_unused]] uint32_t x[4];
      uint32_t lo[4], hi[4];  // lanes 0-15 and 16-31 of the quarter
      if constexpr (T == PA_F16) {
        ldsm_x4_trans(row + (((4 * b + 16 * h + (mi >> 1)) ^ r7) << 4), lo);
        ldsm_x4_trans(row + (((4 * b + 16 * h + 2 + (mi >> 1)) ^ r7) << 4), hi);
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          lo[m] &= (m & 1) ? mb : ma;
          hi[m] &= (m & 1) ? mb : ma;
        }
      } else {
        uint32_t da, db;
        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(da) : "r"(sa + 128 * h));
        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(db) : "r"(sb + 128 * h));
        da &= ma;
        db &= mb;
        if constexpr (T == PA_Q8_0) {
          ldsm_x4_trans(row + (((2 * b + 8 * h + (mi >> 1)) ^ r7) << 4), x);
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            const uint32_t u = x[m] ^ 0x80808080u, d2 = (m & 1) ? db : da;
            uint32_t* o = (m >> 1) ? hi : lo;
            // bytes 0, 2: dim 2g of the key pair; bytes 1, 3: dim 2g + 1
            o[m & 1] = hmul2(hadd2(prmt(u, kMagic, 0x4240), kM1152), d2);
            o[2 + (m & 1)] = hmul2(hadd2(prmt(u, kMagic, 0x4341), kM1152), d2);
          }
        } else {
          if (h == 0) ldsm_x4_trans(row + (((b + 4 * (mi >> 1)) ^ r7) << 4), xq);  // blocks b (0, 1) and b + 4 (2, 3)
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            const uint32_t u = xq[2 * h + m], v = u >> 8, d2 = m ? db : da;
            lo[m] = hmul2(hadd2(and_or(u, 0x000f000fu, 0x64006400u), kM1032), d2);
            lo[2 + m] = hmul2(hadd2(and_or(v, 0x000f000fu, 0x64006400u), kM1032), d2);
            hi[m] = hmul2(hfma2(and_or(u, 0x00f000f0u, 0x64006400u), kR16, kM72), d2);
            hi[2 + m] = hmul2(hfma2(and_or(v, 0x00f000f0u, 0x64006400u), kR16, kM72), d2);
          }
        }
      }
      tmem_st_frag1(taddr + 32 * h + 8 * g, lo);
      tmem_st_frag1(taddr + 32 * h + 8 * g + (16u << 16), hi);
    }
    row += GB;
    sa += GB;
    sb += GB;
  }
}

// ------------------------------------------------------------------ tiles

// What the other roles need to know of a tile; the K copy warp writes it,
// sixteen tiles deep (the roles are never that far apart: the copy stages and
// operand units between them hold fewer tiles).
struct alignas(16) Tile {
  uint32_t info;  // query rows of the segment | first tile of a piece << 8 | last << 9 | suffix << 10 | odd piece << 11 |
                  // 1 << 12 + q: wide keys in quarter q of the lanes (set by the K warps, before S^T)
  int open;       // keys of the tile that every row sees (<= 0: none; >= 128: no edge here); suffix row r sees
                  // (row0 + r) / 6 more
  int row0;       // first query row of the row tile
  int slot_row;   // first slot row of the piece
  int token;      // first token (row of heads) of the unit's queries
  int head;       // KV head
  int pad[2];
};
constexpr int kTiles = 16;

// Where a piece's rows lie among the 64 of Q and the 64 columns of O^T: pieces
// of up to 32 rows take the halves in turn, so that one is staged while the other
// is used, and written out while the next accumulates.  A piece waits for the one
// before the last, and for the last if either is wider.
__device__ __forceinline__ bool is_wide(uint32_t info) { return (info & 0xff) > 32; }
__device__ __forceinline__ uint32_t row0_of(uint32_t info) { return !is_wide(info) && ((info >> 11) & 1) ? 32u : 0u; }

// ------------------------------------------------------------------ query rows

// Eight query rows r8 .. r8 + 7 of a row tile by one warp as binary16 into the B
// operand at dst, slots in K's dim order, rows past the segment's as zeros.  Lane:
// row r8 + lane % 8, slots lane / 8 + 4 i.  begin starts asynchronous copies
// of 16-bit rows to their places (fp32 rows are converted at once), end waits for
// them and puts the pairs of a slot in order and bfloat16 into binary16.
template <int KT>
__device__ __forceinline__ uint4 q_slot(uint4 v) {  // Q4_0: the order of dequant_k's columns, 0, 2 | 1, 3
  if (KT != PA_Q4_0) return v;
  return make_uint4(prmt(v.x, v.y, 0x5410), prmt(v.x, v.y, 0x7632), prmt(v.z, v.w, 0x5410), prmt(v.z, v.w, 0x7632));
}

// Of a row of converted queries: top, the largest of this lane's values.  If one came out
// infinite the row gets a NaN (at its slot to): an infinite logit of either sign would
// pass for a key unseen or weigh alone.
__device__ __forceinline__ void q_range(uint32_t top, uint32_t to) {
  if ((top + 0x04000400u) & 0x80008000u)  // an exponent of all ones carries into bit 15
    asm volatile("st.shared.b16 [%0], %1;" ::"r"(to), "h"((unsigned short)0x7fff) : "memory");
}

// Where query head h of token t has its values, counted in values.
__device__ __forceinline__ long long query_at(const Params& p, int t, int h) { return ((long long)t * p.n_q_heads + h) * kD; }

template <int KT, class P>
__device__ __forceinline__ void stage_q_begin(const P& p, const Tile& t, uint32_t dst, int r8, int lane) {
  const int row = r8 + (lane & 7), rg = t.row0 + row, rows = t.info & 0xff;
  const uint32_t to = dst + canon(row, lane >> 3, kD / 8);
  if (row >= rows) {
#pragma unroll 1
    for (int i = 0; i < 8; ++i) sts128_zero(to + 512 * i);
    return;
  }
  const long long at = query_at(p, t.token + rg / kGqa, t.head * kGqa + rg % kGqa);
  if (p.q_type == PA_DT_F32) {
    const float* src = reinterpret_cast<const float*>(p.q) + at;
    uint32_t top = 0;
#pragma unroll 2
    for (int i = 0; i < 8; ++i) {
      const float4 x = *reinterpret_cast<const float4*>(src + q_dim<KT>((lane >> 3) + 4 * i, 0)),
                   y = *reinterpret_cast<const float4*>(src + q_dim<KT>((lane >> 3) + 4 * i, 1));
      const uint4 v = make_uint4(pack_half2(x.x, x.y), pack_half2(x.z, x.w), pack_half2(y.x, y.y), pack_half2(y.z, y.w));
      top = larger2(larger2(larger2(top, v.x), v.y), larger2(v.z, v.w));
      sts128(to + 512 * i, q_slot<KT>(v));
    }
    q_range(top, to);
  } else {
    const uint8_t* src = p.q + 2 * at;
#pragma unroll 2
    for (int i = 0; i < 8; ++i) {
      const int slot = (lane >> 3) + 4 * i;
      if (KT == PA_Q4_0) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
          asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(to + 512 * i + 8 * h),
                       "l"(src + 2 * q_dim<KT>(slot, h))
                       : "memory");
      } else {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + 512 * i), "l"(src + 16 * slot) : "memory");
      }
    }
  }
}

template <int KT, class P>
__device__ __forceinline__ void stage_q_end(const P& p, uint32_t dst, int r8, int lane) {
  asm volatile("cp.async.wait_all;" ::: "memory");
  const bool bf16 = p.q_type == PA_DT_BF16;
  if (p.q_type == PA_DT_F32 || (KT != PA_Q4_0 && !bf16)) return;
  const uint32_t to = dst + canon(r8 + (lane & 7), lane >> 3, kD / 8);
  uint32_t top = 0;
#pragma unroll 2
  for (int i = 0; i < 8; ++i) {
    uint4 v = lds128(to + 512 * i);
    if (bf16) {
      uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) u[k] = pack_half2(__uint_as_float(u[k] << 16), __uint_as_float(u[k] & 0xffff0000u));
      v = make_uint4(u[0], u[1], u[2], u[3]);
      top = larger2(larger2(larger2(top, v.x), v.y), larger2(v.z, v.w));
    }
    sts128(to + 512 * i, q_slot<KT>(v));
  }
  if (bf16) q_range(top, to);
}

// ------------------------------------------------------------------ the roles' common parts

// The pair of floats in two registers.
__device__ __forceinline__ uint64_t get2(const uint32_t* r) { return pack2(__uint_as_float(r[0]), __uint_as_float(r[1])); }
__device__ __forceinline__ void put2(uint32_t* r, uint64_t v) {
  const float2 f = unpack2(v);
  r[0] = __float_as_uint(f.x);
  r[1] = __float_as_uint(f.y);
}

__device__ __forceinline__ bool bar_or(uint32_t id, uint32_t count, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, "
      "q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)x), "r"(id), "r"(count)
      : "memory");
  return r != 0;
}

// Out-of-line part of warp_wait: false once the wait gave up (after
// kWaitTimeoutNs, which is recorded) or another role had to.
static __device__ __noinline__ bool warp_wait_slow(uint32_t bar, uint32_t parity, int32_t* err, volatile int* abort) {
  uint64_t t0 = 0;
  for (uint32_t i = 1;; ++i) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    if ((i & 63u) == 0) {  // the clock is slow to read: not before the wait is long
      if (i == 64) t0 = globaltimer();
      const bool late = globaltimer() - t0 > kWaitTimeoutNs;
      if (late) {
        record_error(err, PA_ERR_TIMEOUT);
        *abort = 1;
      }
      if (__any_sync(0xffffffffu, late || *abort != 0)) return false;
    }
  }
}

// A bounded wait of the whole warp, which branches as one (the vote keeps it
// free of the convergence barriers of a wait per lane).
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, int32_t* err, volatile int* abort) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  return warp_wait_slow(bar, parity, err, abort);
}

__device__ __forceinline__ FirstKeys live_keys(const Params&, int left, int from) { return FirstKeys{left - from}; }
__device__ __forceinline__ bool has_edge(const Params&, const Tile& t) { return t.open < kKeys; }

// The raw K or V row groups of the CTA's tiles into a ring of ns stages at ring,
// two stages per tile; returns the number of stages issued.  gb, rb: bytes of a
// group and of a row.  One function for both, with what differs as arguments: the
// roles' code competes for the instruction caches.
// Lane g (0..7) looks after row group g of the tile, all in one pass: its
// stage's wait, its copy; its table entry is read a tile ahead.  One warp in the
// company of twenty others executes an instruction every ten cycles or so, so
// what the tiles of a segment share is computed once per segment.
__device__ __forceinline__ int copy_role(const Params& p, Pos pos, int n, bool is_v, int gb, int rb, int ns, uint32_t ring,
                                         uint32_t full, uint32_t empty, Tile* tiles, int* lefts, volatile int* abort,
                                         int lane) {
  const uint8_t* pool = is_v ? p.v_pool : p.k_pool;
  const long long block_rows = (long long)p.n_kv_heads * p.page_size;
  const int half = (lane >> 2) & 1, lane_key = lane < 8 ? kGroup * lane : kKeys;  // lanes past 7 have no group
  const int page_shift = p.page_shift;
  // of the segment
  const int32_t* row = nullptr;
  int end = 0, key0 = 0, head_row = 0;
  uint32_t info = 0;
  int4 tile0 = make_int4(0, 0, 0, 0), tile1 = tile0;
  uint32_t odd = 1;
  int entry = -1, off = 0;
  int pair = 0;         // stages 2 pair, 2 pair + 1
  uint32_t parity = 1;  // of the wait for the stages' previous use; flips when the ring wraps
  bool last = true;
  for (int j = -1; j < n; ++j) {  // issues tile j, looks tile j + 1 up
    const int left = end - key0, tb = entry;
    const bool mine = lane_key < min(kKeys, left), ok = mine && (uint32_t)tb < (uint32_t)p.n_blocks;
    const uint8_t* src = pool + (tb * block_rows + (head_row + off)) * rb;
    if (j >= 0) {
      last = j + 1 == n || pos.j + 1 == pos.nt;
      if (lane == 0) {
        if (is_v) {
          lefts[j & (kTiles - 1)] = left;
        } else {
          int4* t = reinterpret_cast<int4*>(tiles + (j & (kTiles - 1)));
          t[0] = make_int4((int)(info | (last ? 1u << 9 : 0u)), tile0.y - key0, tile0.z, tile0.w);
          t[1] = tile1;
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
        row = p.table + (long long)pos_seq(p, pos) * p.table_stride;
        end = pos_end(p, pos);
        key0 = pos_key0(p, pos);
        head_row = pos.head * p.page_size;
        info = (uint32_t)pos_rows(p, pos) | (pos.pre ? 0u : 1u << 10) | 1u << 8 | odd << 11;
        // prefix: the live keys; suffix: the new tokens' keys open one by one
        tile0 = make_int4(0, pos.pre ? end : end - p.n_qtok + 1, pos.rt * kRows, pos_slot_row(p, pos, (int)blockIdx.x));
        tile1 = make_int4(pos_seq(p, pos) * p.n_qtok, pos.head, 0, 0);
      }
      const int k = key0 + lane_key;
      entry = -1;
      if (lane_key < kKeys && k < end) {
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

// Eight MMAs of an operand unit (columns a, a + 8, ...), issued by the lane
// whose leader is set: D[d] += A B for the descriptor steps b, b + 16, ... (kSplit
// false), or four into d and four into d + 64, for b .. b + 48 both times (true).
// acc 0: the first into each D overwrites it.  One statement, so that what
// they share is moved to uniform registers once: the issuing warp has the
// fewest issue slots to spare (12 instructions an MMA as separate statements, 6
// so).
template <bool kSplit>
__device__ __forceinline__ void mma8(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc, uint32_t leader) {
#define PA_MMA(D, AOFF, BOFF, P)                          \
  "add.u32 a1, %1, " #AOFF ";\n\tadd.u64 b1, %2, " #BOFF \
  ";\n\t@e tcgen05.mma.cta_group::1.kind::f16 [" D "], [a1], b1, %3, " P ";\n\t"
  if (kSplit)
    asm volatile("{\n\t.reg .pred p, e;\n\t.reg .b32 a1, d1;\n\t.reg .b64 b1;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.ne.u32 e, "
                 "%5, 0;\n\tadd.u32 d1, %0, 64;\n\t" PA_MMA("%0", 0, 0, "p") PA_MMA("%0", 8, 16, "1") PA_MMA("%0", 16, 32, "1")
                     PA_MMA("%0", 24, 48, "1") PA_MMA("d1", 32, 0, "p") PA_MMA("d1", 40, 16, "1") PA_MMA("d1", 48, 32, "1")
                         PA_MMA("d1", 56, 48, "1") "}" ::"r"(d),
                 "r"(a), "l"(b), "r"(idesc), "r"(acc), "r"(leader)
                 : "memory");
  else
    asm volatile("{\n\t.reg .pred p, e;\n\t.reg .b32 a1;\n\t.reg .b64 b1;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.ne.u32 e, %5, "
                 "0;\n\t" PA_MMA("%0", 0, 0, "p") PA_MMA("%0", 8, 16, "1") PA_MMA("%0", 16, 32, "1") PA_MMA("%0", 24, 48, "1")
                     PA_MMA("%0", 32, 64, "1") PA_MMA("%0", 40, 80, "1") PA_MMA("%0", 48, 96, "1") PA_MMA("%0", 56, 112, "1") "}" ::"r"(d),
                 "r"(a), "l"(b), "r"(idesc), "r"(acc), "r"(leader)
                 : "memory");
#undef PA_MMA
}

__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r;
}

// ------------------------------------------------------------------ the kernel

template <int KT, int VT, class P>
__global__ void __launch_bounds__(kThreads, 1) pa_prefix_kernel(const __grid_constant__ P p) {
  using SM = Smem<KT, VT, P::kWindow>;
  constexpr int NK = SM::kKStages, NV = SM::kVStages;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + ((1024 - (raw & 1023)) & 1023);
  const uint32_t base = smem_u32(smem);
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
  // Hand-offs (tile j, piece i of the CTA):
  //   kraw_*, vraw_* [(2 j + half) % stages]  copies <-> dequantisation (four warps read a stage)
  //   ku_*, vu_* [half]                 operand units: dequantisation (four warps) <-> MMA (commit)
  //   s_full / s_empty [j & 1]          S^T(j) in tensor memory / in the softmax registers
  //   p_full / pv_done [j & 1]          P^T(j) written / O^T holds tile j, P^T(j) is free
  //   q_full / q_empty [i & 1]          query rows of piece i staged / no longer needed
  //   o_free [i & 1]                    piece i's O^T has been read
  // A role whose wait expires stops: it arrives nowhere any more.
  const uint32_t kraw_full = base + SM::kBar, kraw_empty = kraw_full + 8 * NK, vraw_full = kraw_empty + 8 * NK,
                 vraw_empty = vraw_full + 8 * NV, ku_full = vraw_empty + 8 * NV, ku_empty = ku_full + 16,
                 vu_full = ku_empty + 16, vu_empty = vu_full + 16, s_full = vu_empty + 16, s_empty = s_full + 16,
                 q_full = s_empty + 16, q_empty = q_full + 16, p_full = q_empty + 16, pv_done = p_full + 16,
                 o_free = pv_done + 16, drain = o_free + 16, sink = drain + 16;
  volatile int* abort = reinterpret_cast<volatile int*>(smem + SM::kMisc);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + SM::kMisc + 4);
  volatile int* leave = reinterpret_cast<volatile int*>(smem + SM::kMisc + 8);  // of even, odd tiles
  Pos* start = reinterpret_cast<Pos*>(smem + SM::kMisc + 16);
  int* tiles_at = reinterpret_cast<int*>(smem + SM::kMisc + 16 + sizeof(Pos));  // the CTA's first tile, the next CTA's
  Tile* opening = reinterpret_cast<Tile*>(smem + SM::kOpening);                 // of the first tile, what its query rows need
  Tile* tiles = reinterpret_cast<Tile*>(smem + SM::kTile);
  auto* lefts = reinterpret_cast<typename P::Live*>(smem + SM::kLeft);
  // wide keys (dequant_k) of each quarter of the lanes, where the tile says so; four tiles
  // deep: K(j + 4) follows S^T(j + 3), and that the end of softmax(j + 1)
  uint32_t* wide_keys = reinterpret_cast<uint32_t*>(smem + SM::kWide);
  if (tid == 0) {
    *abort = leave[0] = leave[1] = 0;
    for (int i = 0; i < NK; ++i) {
      mbar_init(kraw_full + 8 * i, 1);
      mbar_init(kraw_empty + 8 * i, 4);
    }
    for (int i = 0; i < NV; ++i) {
      mbar_init(vraw_full + 8 * i, 1);
      mbar_init(vraw_empty + 8 * i, 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(ku_full + 8 * i, 4);
      mbar_init(ku_empty + 8 * i, 1);
      mbar_init(vu_full + 8 * i, 4);
      mbar_init(vu_empty + 8 * i, 1);
      mbar_init(s_full + 8 * i, 1);
      mbar_init(s_empty + 8 * i, 8);
      mbar_init(q_full + 8 * i, 8);
      mbar_init(q_empty + 8 * i, 1);
      mbar_init(p_full + 8 * i, 8);
      mbar_init(pv_done + 8 * i, 1);
      mbar_init(o_free + 8 * i, 8);
      mbar_init(drain + 8 * i, 1);
    }
    mbar_init(sink, 1);
    fence_mbar_init();
  }
  if constexpr (P::kWindow) {
    if (w == 1) {
      const Pos t = start_of(p, (int)blockIdx.x);
      if (lane == 0) {
        *start = t;
        *opening = Tile{(uint32_t)pos_rows(p, t) | 1u << 8, 0, pos_row0(p, t), 0, pos_token(p, t), t.head, {0, 0}};
        tiles_at[0] = t.tile;
        tiles_at[1] = p.start[blockIdx.x + 1].tile;
      }
    }
  } else if (w == 1 || w == 2) {
    const int x = (int)((long long)(blockIdx.x + w - 1) * p.total_len / p.n_ctas);
    if (x < p.total_len) {
      const Pos t = locate(p, x);
      if (lane == 0) {
        if (w == 1) {
          *start = t;
          *opening = Tile{(uint32_t)pos_rows(p, t) | 1u << 8, 0, pos_row0(p, t), 0, pos_token(p, t), t.head, {0, 0}};
        }
        tiles_at[w - 1] = t.tile;
      }
    } else if (lane == 0) {
      tiles_at[1] = p.total_tiles;
    }
  }
  if (w == 0) {
    tmem_alloc(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const int n = tiles_at[1] - tiles_at[0];  // at least 1
  // nothing that another kernel wrote is read before this
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (tid == 0) asm volatile("griddepcontrol.launch_dependents;");
  // All of tensor memory is this CTA's, so its columns start at 0; written as a
  // constant, the MMAs' addresses need no register that the compiler would have
  // to prove uniform.
  const bool whole = *tmem_slot == 0;
  if (!whole && tid == 0) record_error(p.err, PA_ERR_CUDA);
  // the copy warps': K's or V's
  const bool is_v = w == kCopyVWarp;
  const int ns = is_v ? NV : NK;
  const uint32_t raw_full = is_v ? vraw_full : kraw_full;
  int issued = 0;

  if (!whole) {
  } else if (w == kCopyKWarp || is_v) {
    issued = copy_role(p, *start, n, is_v, is_v ? SM::kVStage / 4 : SM::kKStage / 4, is_v ? Fmt<VT>::kRow : Fmt<KT>::kRow, ns,
                       base + (is_v ? SM::kVRing : SM::kRing), raw_full, is_v ? vraw_empty : kraw_empty, tiles, lefts, abort,
                       lane);
  } else if (w < kVWarp0) {
    // ---- K: thread = key (position 32 * quarter + lane), dims 128 kd .. + 127
    const int kd = w >> 2, quarter = w & 3, at = 32 * quarter + lane;
    const int r = key16(lane & 15);
    const uint32_t grp = base + SM::kRing + ((at >> 4) & 3) * pa_layout::group_bytes<KT>();
    const uint32_t t_lane = (uint32_t)(32 * quarter) << 16;
    // The query rows of a piece are staged here too, eight by each of the warps,
    // copied while the tile's K is converted.
    uint32_t piece = 0;
    bool wide = false;  // the piece before
    for (int j = 0; j < n; ++j) {
      const uint32_t stage = 2 * j + (quarter >> 1), slot = stage % NK;
      // the first piece's rows do not wait for its keys
      if (j > 0 && !warp_wait(kraw_full + 8 * slot, (stage / NK) & 1, p.err, abort)) break;
      const Tile& t = j > 0 ? tiles[j & (kTiles - 1)] : *opening;
      const uint32_t info = t.info, q_dst = base + SM::kQ + row0_of(info) * (kD * 2);
      const bool first_tile = (info >> 8) & 1, stage_q = first_tile && 8 * w < (int)(((info & 0xff) + 15) & ~15u);
      if (first_tile) {
        if (piece > 1 && !warp_wait(q_empty + 8 * (piece & 1), ((piece >> 1) - 1) & 1, p.err, abort)) break;
        if (piece > 0 && (wide || is_wide(info)) &&
            !warp_wait(q_empty + 8 * ((piece - 1) & 1), ((piece - 1) >> 1) & 1, p.err, abort))
          break;
        wide = is_wide(info);
      }
      if (stage_q) stage_q_begin<KT>(p, t, q_dst, 8 * w, lane);
      if (!(j > 0 ? warp_wait(ku_empty + 8 * kd, (j - 1) & 1, p.err, abort) : warp_wait(kraw_full + 8 * slot, 0, p.err, abort)))
        break;
      tc_fence_after();
      const uint32_t wide_lanes = dequant_k<KT>(grp + slot * SM::kKStage, r, kd, kKCol + 64 * kd + t_lane);
      if (KT != PA_F16 && wide_lanes != 0 && kd == 0 && lane == 0) {
        wide_keys[4 * (j & 3) + quarter] = wide_lanes;
        atomicOr(&tiles[j & (kTiles - 1)].info, 1u << (12 + quarter));
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(kraw_empty + 8 * slot);
      __syncwarp();
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(ku_full + 8 * kd);
      __syncwarp();
      if (first_tile) {
        if (stage_q) stage_q_end<KT>(p, q_dst, 8 * w, lane);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(q_full + 8 * (piece & 1));
        __syncwarp();
        ++piece;
      }
    }
  } else if (w < kSmWarp0) {
    // ---- V: keys 64 vh .. + 63 of the tile, block `quarter` of each half of the dims
    const int vh = (w - kVWarp0) >> 2, quarter = w & 3;
    const uint32_t t_lane = (uint32_t)(32 * quarter) << 16;
    for (int j = 0; j < n; ++j) {
      const uint32_t stage = 2 * j + vh, slot = stage % NV;
      if (!warp_wait(vraw_full + 8 * slot, (stage / NV) & 1, p.err, abort)) break;
      if (j > 0 && !warp_wait(vu_empty + 8 * vh, (j - 1) & 1, p.err, abort)) break;
      tc_fence_after();
      dequant_v<VT>(base + SM::kVRing + slot * SM::kVStage, quarter, live_keys(p, lefts[j & (kTiles - 1)], kStageKeys * vh),
                    kVCol + 64 * vh + t_lane, lane);
      __syncwarp();
      if (lane == 0) mbar_arrive(vraw_empty + 8 * slot);
      __syncwarp();
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(vu_full + 8 * vh);
    }
  } else if (w == kSWarp || w == kPvWarp) {
    // ---- MMA issue, S^T and O^T by a warp each: the whole warp runs its loop and
    // an elected lane issues, so that the operands stay in uniform registers: what
    // comes from shared memory goes through a warp reduction, and an expired wait
    // leaves the control flow as it is -- from then on all commits go to a barrier
    // that nobody waits on, and the MMAs are of 16 rows: the tile's record may not be
    // there, and a shape that there is none of would be a fault.  (The choice stands
    // before the reduction; behind it, or on the issuing lane, it costs 4 to 9 per cent.)
    const uint32_t leader = elect_one();
    bool dead = false;
    auto wait = [&](uint32_t bar, uint32_t parity) { dead |= !warp_wait(bar, parity, p.err, abort); };
    auto commit = [&](uint32_t bar) { tc_commit_warp(dead ? sink : bar); };
    auto info_of = [&](uint32_t j) { return __reduce_or_sync(0xffffffffu, dead ? 16u : tiles[j & (kTiles - 1)].info); };
    auto idesc_of = [](uint32_t info) { return idesc_f16_f32(128, 0) | (((info & 0xffu) + 15) >> 4 << 18); };
    uint32_t piece = 0;
    if (w == kSWarp) {
      const uint64_t qdesc = smem_desc(base + SM::kQ, 128, 4096);
      for (uint32_t j = 0; j < (uint32_t)n; ++j) {
        const uint32_t b = j & 1;
        wait(ku_full, b);
        const uint32_t info = info_of(j);
        if ((info >> 8) & 1) {
          wait(q_full + 8 * (piece & 1), (piece >> 1) & 1);
          ++piece;
        }
        if (j >= 2) wait(s_empty + 8 * b, ((j >> 1) - 1) & 1);
        tc_fence_after();
        const uint64_t qd = qdesc + row0_of(info) * (kD * 2 / 16);
        const uint32_t idesc = idesc_of(info), d = kSCol + 64 * b;
#pragma unroll 1
        for (uint32_t h = 0; h < 2; ++h) {
          if (h) wait(ku_full + 8, b);
          tc_fence_after();
          mma8<false>(d, kKCol + 64 * h, qd + 128 * h, idesc, h, leader);
          commit(ku_empty + 8 * h);
        }
        commit(s_full + 8 * b);
        if ((info >> 9) & 1) commit(q_empty + 8 * ((piece - 1) & 1));
      }
      // the last commits have arrived before the CTA's barriers go away
      for (int i = 0; i < 2; ++i) wait(ku_empty + 8 * i, (n - 1) & 1);
      for (uint32_t j = n < 2 ? 0 : n - 2; j < (uint32_t)n; ++j) wait(s_full + 8 * (j & 1), (j >> 1) & 1);
      for (uint32_t i = piece < 2 ? 0 : piece - 2; i < piece; ++i) wait(q_empty + 8 * (i & 1), (i >> 1) & 1);
    } else {
      const uint64_t pdesc = smem_desc(base + SM::kP, 128, 2048);
      uint32_t wide = 0;  // the piece before
      for (uint32_t j = 0; j < (uint32_t)n; ++j) {
        const uint32_t b = j & 1;
        wait(p_full + 8 * b, (j >> 1) & 1);
        const uint32_t info = info_of(j), first_tile = (info >> 8) & 1, idesc = idesc_of(info);
        if (first_tile) {
          if (piece > 1) wait(o_free + 8 * (piece & 1), ((piece >> 1) - 1) & 1);
          if (piece > 0 && (wide | (uint32_t)is_wide(info))) wait(o_free + 8 * ((piece - 1) & 1), ((piece - 1) >> 1) & 1);
          wide = is_wide(info);
          ++piece;
        }
#pragma unroll 1
        for (uint32_t h = 0; h < 2; ++h) {
          wait(vu_full + 8 * h, b);
          tc_fence_after();
          mma8<true>(kOCol + row0_of(info), kVCol + 64 * h, pdesc + (b * (SM::kPBytes >> 4) + 64 * h), idesc,
                     h | (first_tile ^ 1u), leader);
          commit(vu_empty + 8 * h);
        }
        commit(pv_done + 8 * b);
      }
      for (int i = 0; i < 2; ++i) wait(vu_empty + 8 * i, (n - 1) & 1);
      for (uint32_t j = n < 2 ? 0 : n - 2; j < (uint32_t)n; ++j) wait(pv_done + 8 * (j & 1), (j >> 1) & 1);
    }
    if (dead) {  // what was issued ends before shared and tensor memory are released
      const uint32_t bar = drain + 8 * (w - kSWarp);
      tc_commit_warp(bar);
      mbar_wait(bar, 0, p.err, abort, /*honour_abort=*/false);
    }
    __syncwarp();
  } else {
    // ---- softmax: keys 16 hh + 32 quarter .. + 15 of the tile, all query rows;
    // thread 4g + t holds keys g and g + 8 and columns 2t, 2t + 1 of every 8
    const int sw = w - kSmWarp0, hh = sw >> 2, quarter = w & 3, g = lane >> 2, t2 = 2 * (lane & 3), st = tid - 32 * kSmWarp0;
    float* red = reinterpret_cast<float*>(smem + SM::kRed);
    float* nref = reinterpret_cast<float*>(smem + SM::kRef);      // minus the reference maximum
    float* alpha = reinterpret_cast<float*>(smem + SM::kAlpha);
    const uint32_t s_addr = kSCol + ((uint32_t)(32 * quarter + 16 * hh) << 16);
    const uint32_t o_addr = kOCol + 64 * hh + ((uint32_t)(32 * quarter) << 16);
    const int tile_key = 16 * (2 * quarter + hh);
    const uint32_t p_addr = base + SM::kP + canon(8 * (lane >> 4) + (lane & 7), 4 * quarter + 2 * hh + ((lane >> 3) & 1), kKeys / 8);
    const uint64_t scale2 = pack2(p.scale_log2, p.scale_log2);
    uint64_t l[4][2] = {};  // sums of weights over this thread's keys: rows (16c + 8e + 2t, + 1)
    // A warp whose wait expired arrives nowhere any more and, before it would read another
    // tile's record, says so: it sets the tile's `leave` and comes to the barrier at which
    // the eight warps meet first in every tile, a vote.  After that all of them leave; until
    // then all walk the same records, and so the same barriers.
    bool live = true;
    // Logits of 16 rows in log2 units, less their references (none: zero ones).
    // Thread: [8 columns e, key g or g + 8, column 2t or 2t + 1] at 4e + 2k + i.
    auto logits = [&](uint32_t (&x)[8], const int c, const bool refs) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint64_t m = refs ? *reinterpret_cast<const uint64_t*>(nref + 16 * c + 8 * e + t2) : 0ull;
        put2(x + 4 * e, fma2(get2(x + 4 * e), scale2, m));
        put2(x + 4 * e + 2, fma2(get2(x + 4 * e + 2), scale2, m));
      }
    };
    // S^T is read twice in a first tile (maxima, then weights) and once in others:
    // kept in registers it made them spill.  The rows' sixteens are skipped, not
    // compiled for each number of them.
    auto tile = [&](const int j, const uint32_t info) -> bool {  // false: one of the warps has given up
      const int nc = ((info & 0xff) + 15) >> 4;  // query rows in sixteens
      const Tile& tl = tiles[j & (kTiles - 1)];
      const bool first_tile = (info >> 8) & 1;
      const uint32_t s_at = s_addr + 64 * (j & 1), p_to = p_addr + (j & 1) * SM::kPBytes;
      const bool has_wide = KT != PA_F16 && info >> (12 + quarter) & 1;
      if (has_edge(p, tl) || has_wide) {
        // The edge: what a row does not see becomes -inf in tensor memory, so that
        // the code of the other tiles has no mask in it.  Row r sees key k when r >= 6
        // (k - open + 1) (suffix) or k < open.  And the logits of wide keys.
        const uint32_t wide = has_wide ? wide_keys[4 * (j & 3) + quarter] >> (16 * hh) : 0u;
        const float fa = wide >> g & 1 ? 256.f : 1.f, fb = wide >> (g + 8) & 1 ? 256.f : 1.f;
        int la, lb;                   // the first row that sees the key, less this thread's column
        [[maybe_unused]] int ua, ub;  // of a window: the first one after those that see it
        if constexpr (P::kWindow) {
          const int2 a = rows_that_see(p, tl, tile_key + key16(g)), b = rows_that_see(p, tl, tile_key + key16(g + 8));
          la = a.x - t2;
          ua = a.y - t2;
          lb = b.x - t2;
          ub = b.y - t2;
        } else {
          const int ka = tile_key + key16(g) - tl.open, kb = tile_key + key16(g + 8) - tl.open;
          const bool causal = (info >> 10) & 1;
          la = causal ? kGqa * (ka + 1) - tl.row0 - t2 : ka < 0 ? -kRows : kRows;
          lb = causal ? kGqa * (kb + 1) - tl.row0 - t2 : kb < 0 ? -kRows : kRows;
        }
#pragma unroll 1
        for (int c = 0; c < nc; ++c) {
          uint32_t x[8];
          tmem_ld_frag2(s_at + 16 * c, x);
          tmem_ld_wait();
          loaded(x);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int r = 8 * (i >> 2) + (i & 1);
            bool hidden = r < ((i & 2) ? lb : la);
            if constexpr (P::kWindow) hidden |= r >= ((i & 2) ? ub : ua);
            x[i] = hidden ? 0xff800000u  // -inf
                          : __float_as_uint(__uint_as_float(x[i]) * ((i & 2) ? fb : fa));
          }
          tmem_st_frag2(s_at + 16 * c, x);
          la -= 16;
          lb -= 16;
          if constexpr (P::kWindow) {
            ua -= 16;
            ub -= 16;
          }
        }
        tmem_st_wait();
      }
      // The references are set at a piece's first tile and raised when a logit passes
      // them by 2^8; then the tile's weights are computed again.
      bool raise = first_tile;
      uint64_t ls[4][2];
      for (;;) {
        if (raise) {
          if (j > 0 && bar_or(1, kSmThreads, false)) return false;  // the others are done with the shared arrays
#pragma unroll 1
          for (int c = 0; c < nc; ++c) {
            uint32_t x[8];
            tmem_ld_frag2(s_at + 16 * c, x);
            tmem_ld_wait();
            loaded(x);
            logits(x, c, !first_tile);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float u = fmaxf(__uint_as_float(x[4 * e]), __uint_as_float(x[4 * e + 2])),
                    v = fmaxf(__uint_as_float(x[4 * e + 1]), __uint_as_float(x[4 * e + 3]));
#pragma unroll
              for (int o = 4; o < 32; o <<= 1) {
                u = fmaxf(u, __shfl_xor_sync(0xffffffffu, u, o));
                v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
              }
              if (g == 0) *reinterpret_cast<float2*>(red + sw * kRows + 16 * c + 8 * e + t2) = make_float2(u, v);
            }
          }
          __syncwarp();
          if (bar_or(1, kSmThreads, false)) return false;  // the first meeting of tile 0
          if (st < 16 * nc) {
            float v = red[st];
#pragma unroll
            for (int i = 1; i < 8; ++i) v = fmaxf(v, red[i * kRows + st]);
            // a row that sees no key yet keeps a reference of 0; it will see none later in the piece either
            const float d = first_tile ? (v == -INFINITY ? 0.f : v) : fmaxf(v, 0.f);
            nref[st] = first_tile ? -d : nref[st] - d;
            alpha[st] = ex2(-d);
          }
          __syncwarp();
          named_bar_sync(1, kSmThreads);
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              l[c][e] = first_tile ? 0ull : mul2(l[c][e], *reinterpret_cast<const uint64_t*>(alpha + 16 * c + 8 * e + t2));
          if (!first_tile) {  // O^T holds the tiles before: dims of this warp, every row
            live = live && warp_wait(pv_done + 8 * ((j - 1) & 1), ((j - 1) >> 1) & 1, p.err, abort);
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < 2 * nc; ++c) {
              uint32_t o[8];
              tmem_ld8(o_addr + row0_of(info) + 8 * c, o);
              tmem_ld_wait();
              loaded(o);
#pragma unroll
              for (int i = 0; i < 8; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha[8 * c + i]);
              tmem_st8(o_addr + row0_of(info) + 8 * c, o);
            }
            tmem_st_wait();
            tc_fence_before();
          }
        }
        float top = -INFINITY;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          ls[c][0] = ls[c][1] = 0ull;
          if (c >= nc) continue;
          uint32_t x[8];
          tmem_ld_frag2(s_at + 16 * c, x);
          tmem_ld_wait();
          loaded(x);
          logits(x, c, true);
#pragma unroll
          for (int i = 0; i < 8; i += 2) top = fmaxf(top, fmaxf(__uint_as_float(x[i]), __uint_as_float(x[i + 1])));
          uint32_t h[4];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float a0 = ex2(__uint_as_float(x[4 * e])), a1 = ex2(__uint_as_float(x[4 * e + 1])),
                        b0 = ex2(__uint_as_float(x[4 * e + 2])), b1 = ex2(__uint_as_float(x[4 * e + 3]));
            h[2 * e] = pack_half2(a0, a1);
            h[2 * e + 1] = pack_half2(b0, b1);
            ls[c][e] = add2(pack2(a0, a1), pack2(b0, b1));
          }
          if (c == 0 && j > 1 && live && !warp_wait(pv_done + 8 * (j & 1), ((j >> 1) - 1) & 1, p.err, abort)) {  // of P^T(j - 2)
            live = false;
            leave[j & 1] = 1;
            top = INFINITY;
          }
          stsm_x4_trans(p_to + c * (16 * kKeys * 2), h[0], h[1], h[2], h[3]);
        }
        if (raise) break;
        raise = bar_or(1, kSmThreads, top > kLazyLog2);
        if (!raise) break;
        if (leave[j & 1]) return false;
      }
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int e = 0; e < 2; ++e) l[c][e] = add2(l[c][e], ls[c][e]);
      tc_fence_before();
      fence_proxy_async_smem();
      __syncwarp();
      if (live && lane == 0) {
        mbar_arrive(p_full + 8 * (j & 1));
        mbar_arrive(s_empty + 8 * (j & 1));
      }
      __syncwarp();
      return true;
    };
    for (int j = 0; j <= n; ++j) {
      if (j < n) {
        live = live && warp_wait(s_full + 8 * (j & 1), (j >> 1) & 1, p.err, abort);
        if (!live) {
          leave[j & 1] = 1;
          bar_or(1, kSmThreads, true);
          break;
        }
        tc_fence_after();
        if (!tile(j, tiles[j & (kTiles - 1)].info)) break;
      }
      // ---- a piece's O^T, once the weights of the tile after it are on their way
      const Tile& t = tiles[(j - 1) & (kTiles - 1)];
      const uint32_t info = j > 0 ? t.info : 0u;
      if ((info >> 9) & 1) {
        const int rows = info & 0xff;
        const uint32_t from = o_addr + row0_of(info);
        live = live && warp_wait(pv_done + 8 * ((j - 1) & 1), ((j - 1) >> 1) & 1, p.err, abort);
        float* dst = p.part_o + (long long)t.slot_row * kD + 128 * hh + 32 * quarter + v_dim<VT>(lane);
        tc_fence_after();
#pragma unroll 1
        for (int r = 0; r < rows; r += 16) {
          uint32_t o[16];
          tmem_ld16(from + r, o);
          tmem_ld_wait();
          loaded(o);
          if constexpr (P::kWindow) {
            if (t.slot_row < 0) {  // the whole segment: the result
              write_out(p, t, r, rows, reinterpret_cast<const float*>(smem + SM::kInv), 128 * hh + 32 * quarter + v_dim<VT>(lane), o);
              continue;
            }
          }
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (r + i < rows) dst[(r + i) * kD] = __uint_as_float(o[i]);
        }
        tc_fence_before();
        __syncwarp();
        if (live && lane == 0) mbar_arrive(o_free + 8 * ((info >> 11) & 1));
        __syncwarp();
      }
      // ---- a piece's sums of weights, after its last tile
      if (j == n) break;
      const Tile& tl = tiles[j & (kTiles - 1)];
      if ((tl.info >> 9) & 1) {
        named_bar_sync(1, kSmThreads);
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            uint64_t v = l[c][e];
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) v = add2(v, __shfl_xor_sync(0xffffffffu, v, o));
            if (g == 0) *reinterpret_cast<uint64_t*>(red + sw * kRows + 16 * c + 8 * e + t2) = v;
          }
        __syncwarp();
        named_bar_sync(1, kSmThreads);
        if (st < (int)(tl.info & 0xff)) {
          float v = red[st];
#pragma unroll
          for (int i = 1; i < 8; ++i) v += red[i * kRows + st];
          bool result = false;
          if constexpr (P::kWindow) {
            result = tl.slot_row < 0;
            if (result) reinterpret_cast<float*>(smem + SM::kInv)[st] = finish_row(p, tl, st, -nref[st], v);
          }
          if (!result) p.part_ml[(long long)tl.slot_row + st] = make_float2(-nref[st], v);
        }
        if constexpr (P::kWindow) {
          __syncwarp();
          named_bar_sync(1, kSmThreads);
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  // after an expired wait, copies that nobody waited for must still land
  if ((w == kCopyKWarp || is_v) && *abort) {
    for (int i = max(0, issued - ns); i < issued; ++i)
      mbar_wait(raw_full + 8 * (i % ns), (uint32_t)((i / ns) & 1), p.err, abort, false, kWaitTimeoutNs / 8);
  }
  if (w == 0) {
    tc_fence_after();
    tmem_dealloc(*tmem_slot, kTmemCols);
  }
}

template <class P>
struct KernelOf {
  void (*fn)(P);
  int smem;
};
using KernelInfo = KernelOf<Params>;

#define PA_DECLARE_PREFIX(k, v) bool lookup_prefix_kernel_##k##_##v(KernelInfo* out);
PA_DECLARE_PREFIX(1, 1) PA_DECLARE_PREFIX(1, 2) PA_DECLARE_PREFIX(1, 8)
PA_DECLARE_PREFIX(2, 1) PA_DECLARE_PREFIX(2, 2) PA_DECLARE_PREFIX(2, 8)
PA_DECLARE_PREFIX(8, 1) PA_DECLARE_PREFIX(8, 2) PA_DECLARE_PREFIX(8, 8)
#undef PA_DECLARE_PREFIX

}  // namespace pa_prefix
