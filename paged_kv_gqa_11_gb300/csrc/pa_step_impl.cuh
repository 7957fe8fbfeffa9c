// Windowed attention of one new token per sequence, for batches that fill the device (sm_103a).
//
// The mathematics is that of pa_window_impl.cuh for the six query rows of one position and KV head:
// scores, softmax with a running reference, weighted sum of values, over the first keys and
// the window in the walk's order of row groups (16 keys).  The kernel of few tokens spends 1 to 2 us on a
// tile of 128 keys whatever the number of rows, its bulk copies of 2 to 4 KB (55 cycles each and 36 bytes per
// cycle) and the waits between its roles; a batch of single tokens is memory traffic, so here a warp is a
// pipeline of its own.  A segment (sequence, KV head) is a cluster of one to eight CTAs; a warp takes every
// fourth row group of its CTA's share, copies it by cp.async into its ring of three, two on their way while
// the third is multiplied by mma.sync:
//   S (16 keys x 8 rows) = K Q^T: per block of 32 dims two MMAs of exact quants, then the block's scale in
//                          fp32 on the four results: K is not rounded;
//   O (dims x 8 rows)   += V^T P^T: V by transposing ldmatrix, scaled in binary16; P^T by movmatrix, in two parts
//                          of binary16, so that only V is rounded (the second product is hidden: 29.1 and 29.2 us
//                          without and with it).
// The order of a contraction is free, so a thread's piece of K is whole words as they lie in the row,
// and Q's fragments take the same order.  Two of the eight rows are idle.  A warp's and then a
// cluster's states are joined in shared memory by log-sum-exp, in a fixed order: one launch, no workspace.
//
// What bounds it: a group is 850 instructions of dependent steps, 0.8 us for a warp that has its scheduler to
// itself; two CTAs on an SM hide each other's.  Eight warps to a CTA, one CTA on an SM, were slower
// (64 sequences, 1024 keys: 41.8 against 31.4 us).
//
// Both sides of step_cluster's rule (pa_window.cu), in us: this kernel / the kernel of few tokens, sequences x keys of 4
// heads, K and V Q8_0, eight caches in turn (at 256 and 1024 keys much of them stays in the L2):
//   where the rule takes this kernel   61 x 256 15.9 / 19.2, 76 x 256 16.6 / 17.0, 61 x 1024 31.0 / 42.4, 76 x 1024 34.6 /
//     42.4, 61 x 4096 90.6 / 110.3, 128 x 256 29.7 / 31.9, 128 x 1024 61.1 / 75.4, 128 x 4096 185 / 214; clusters of two 31 x 1024
//     22.4 / 26.9, 38 x 1024 23.0 / 24.1, 31 x 4096 52.5 / 62.8; of four 16 x 1024 17.2 / 18.0, 16 x 4096 32.2 / 37.6; of eight
//     8 x 4096 22.7 / 24.8; it loses at 38 x 256 (15.1 / 11.8: a segment to each SM suits the other) and 8 x 1024 (14.7 / 13.8);
//   where it takes the other   77 x 256 24.4 / 21.4, 77 x 1024 50.9 / 50.0, 77 x 4096 155 / 135, 40 x 4096 86.7 / 77.0, 9 x 1024
//     20.9 / 14.0, 19 x 1024 27.6 / 17.8; it loses between 48 and 60 sequences (60 x 256 15.8 / 19.2, 48 x 1024 30.2 / 35.5, 60 x 1024
//     30.9 / 41.9, 60 x 4096 89.9 / 108), at 30 (30 x 1024 22.4 / 26.2) and at 100 to 121 (121 x 1024 60.7 / 71.9): the
//     rule asks for four fifths of the device, and three would do at 1024 keys.
// Q4_0 keys gain little (64 x 1024 32.8 / 33.8) and F16 ones lose (57.7 / 51.6: one CTA on an SM), so only pairs with K Q8_0 and
// quantised V have the kernel.
#pragma once

#include "pa_io.cuh"
#include "pa_step.cuh"

namespace pa_prefix {

constexpr int kStepRows = kGqa;

template <int VT>
struct StepSmem {
  static constexpr int kK = pa_layout::group_bytes<PA_Q8_0>(), kV = pa_layout::group_bytes<VT>();
  static constexpr int kStage = kK + kV;
  static constexpr int kStages = 3;  // two groups on their way: with two CTAs on an SM, up to 139 KB
  static constexpr int kRing = kStepWarps * kStages * kStage;
  // the join: a warp's (or CTA's) state is rows x 256 of O, then (reference, sum) of the rows
  static constexpr int kState = kStepRows * kD * 4 + 8 * 8;
  static constexpr int kJoin = (kStepWarps + 1) * kState;
  static constexpr int kTotal = kRing > kJoin ? kRing : kJoin;
  static_assert(2 * (kTotal + 1024) <= 233472, "shared memory");
};

// The pair of binary16 numbers of bytes lo, lo + 1 (sel) of a word of int8 quants, exact.
__device__ __forceinline__ uint32_t step_q8(uint32_t u, uint32_t sel) { return hadd2(prmt(u, kMagic, sel), kM1152); }

// Query fragments: of the row g (its lane's), k-step i (16 of them) and this thread's t, the four
// dims of step_dim(i, t) as two pairs.
__device__ __forceinline__ int step_dim(int i, int t) { return 32 * (i >> 1) + 8 * t + 4 * (i & 1); }

__device__ __forceinline__ void step_queries(const StepParams& p, long long at, bool row, int t, uint32_t (&q)[32]) {
  bool wide = false;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int d = step_dim(i, t);
    uint32_t a = 0, b = 0;
    if (row) {
      if (p.q_type == PA_DT_F32) {
        const float4 x = __ldg(reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p.q) + at + d));
        a = pack_half2(x.x, x.y);
        b = pack_half2(x.z, x.w);
      } else {
        const uint2 x = __ldg(reinterpret_cast<const uint2*>(p.q + 2 * (at + d)));
        a = x.x;
        b = x.y;
        if (p.q_type == PA_DT_BF16) {
          a = pack_half2(__uint_as_float(x.x << 16), __uint_as_float(x.x & 0xffff0000u));
          b = pack_half2(__uint_as_float(x.y << 16), __uint_as_float(x.y & 0xffff0000u));
        }
      }
    }
    if (p.q_type != PA_DT_F16) wide |= ((larger2(a, b) + 0x04000400u) & 0x80008000u) != 0;
    q[2 * i] = a;
    q[2 * i + 1] = b;
  }
  if (wide) q[0] = 0x7fff7fffu;  // a value past binary16's range makes its row NaN
}

// S of a group: c0, c1: key g, rows 2t, 2t + 1; c2, c3: key g + 8.
__device__ __forceinline__ void step_scores(uint32_t grp, const uint32_t (&q)[32], int g, int t, float (&s)[4]) {
  s[0] = s[1] = s[2] = s[3] = 0.f;
  const uint32_t row = grp + Fmt<PA_Q8_0>::kScales + g * Fmt<PA_Q8_0>::kRowQ;  // row g + 8: eight rows on, the same swizzle
  constexpr uint32_t kDown = 8 * Fmt<PA_Q8_0>::kRowQ;
  const uint4 sg = lds128(grp + 16 * g), sh = lds128(grp + 16 * (g + 8));
  const uint32_t dg[4] = {sg.x, sg.y, sg.z, sg.w}, dh[4] = {sh.x, sh.y, sh.z, sh.w};
#pragma unroll
  for (int b = 0; b < 8; ++b) {
    float c[4] = {};
    const uint32_t at = row + ((((2 * b + (t >> 1)) ^ g) << 4) | (t & 1) << 3);
    const uint2 x = lds64(at), y = lds64(at + kDown);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint32_t u = (k ? x.y : x.x) ^ 0x80808080u, v = (k ? y.y : y.x) ^ 0x80808080u;
      const uint32_t a[4] = {step_q8(u, 0x4140), step_q8(v, 0x4140), step_q8(u, 0x4342), step_q8(v, 0x4342)};
      mma_16816(c, a, q[4 * b + 2 * k], q[4 * b + 2 * k + 1]);
    }
    const float fg = __half2float(__ushort_as_half((unsigned short)(b & 1 ? dg[b >> 1] >> 16 : dg[b >> 1] & 0xffffu)));
    const float fh = __half2float(__ushort_as_half((unsigned short)(b & 1 ? dh[b >> 1] >> 16 : dh[b >> 1] & 0xffffu)));
    s[0] = fmaf(fg, c[0], s[0]);
    s[1] = fmaf(fg, c[1], s[1]);
    s[2] = fmaf(fh, c[2], s[2]);
    s[3] = fmaf(fh, c[3], s[3]);
  }
}

// O += V^T P^T: tile i of O is dims 16 i + 2 g (c0, c1) and + 1 (c2, c3), rows
// 2t, 2t + 1.  la, lb: live keys among the pairs (2t, 2t + 1) and + 8, as masks.
template <int VT>
__device__ __forceinline__ void step_values(uint32_t grp, float (&o)[16][4], const uint32_t (&b)[4], uint32_t la, uint32_t lb, int lane) {
  const int mi = lane >> 3, r = (mi & 1) * 8 + (lane & 7), r7 = lane & 7, t = lane & 3;
  const uint32_t row = grp + Fmt<VT>::kScales + r * Fmt<VT>::kRowQ;
#pragma unroll
  for (int j = 0; j < 4; ++j) {  // blocks 2 j and 2 j + 1
    const uint4 d = lds128(grp + 64 * j + 16 * t);  // pairs (2t, 2t + 1), + 8 of block 2 j, then of 2 j + 1
    const uint32_t da[2] = {d.x & la, d.z & la}, db[2] = {d.y & lb, d.w & lb};
    if constexpr (VT == PA_Q8_0) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int blk = 2 * j + e;
        uint32_t x[4];
        ldsm_x4_trans(row + (((2 * blk + (mi >> 1)) ^ r7) << 4), x);
        uint32_t a[2][4];
#pragma unroll
        for (int k = 0; k < 2; ++k) {  // chunk 2 blk + k: bytes 0, 2 are dim 2 g of a key pair, 1, 3 dim 2 g + 1
          const uint32_t u = x[2 * k] ^ 0x80808080u, v = x[2 * k + 1] ^ 0x80808080u;
          a[k][0] = hmul2(step_q8(u, 0x4240), da[e]);
          a[k][1] = hmul2(step_q8(u, 0x4341), da[e]);
          a[k][2] = hmul2(step_q8(v, 0x4240), db[e]);
          a[k][3] = hmul2(step_q8(v, 0x4341), db[e]);
          mma_16816(o[2 * blk + k], a[k], b[0], b[1]);
        }
        mma_16816(o[2 * blk], a[0], b[2], b[3]);
        mma_16816(o[2 * blk + 1], a[1], b[2], b[3]);
      }
    } else {
      uint32_t x[4];
      ldsm_x4_trans(row + (((2 * j + (mi >> 1)) ^ r7) << 4), x);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint32_t u = x[2 * e], v = x[2 * e + 1], u8 = u >> 8, v8 = v >> 8;
        const uint32_t lo[4] = {hmul2(hadd2(and_or(u, 0x000f000fu, 0x64006400u), kM1032), da[e]),
                                hmul2(hadd2(and_or(u8, 0x000f000fu, 0x64006400u), kM1032), da[e]),
                                hmul2(hadd2(and_or(v, 0x000f000fu, 0x64006400u), kM1032), db[e]),
                                hmul2(hadd2(and_or(v8, 0x000f000fu, 0x64006400u), kM1032), db[e])};
        const uint32_t hi[4] = {hmul2(hfma2(and_or(u, 0x00f000f0u, 0x64006400u), kR16, kM72), da[e]),
                                hmul2(hfma2(and_or(u8, 0x00f000f0u, 0x64006400u), kR16, kM72), da[e]),
                                hmul2(hfma2(and_or(v, 0x00f000f0u, 0x64006400u), kR16, kM72), db[e]),
                                hmul2(hfma2(and_or(v8, 0x00f000f0u, 0x64006400u), kR16, kM72), db[e])};
        mma_16816(o[2 * (2 * j + e)], lo, b[0], b[1]);
        mma_16816(o[2 * (2 * j + e) + 1], hi, b[0], b[1]);
        mma_16816(o[2 * (2 * j + e)], lo, b[2], b[3]);
        mma_16816(o[2 * (2 * j + e) + 1], hi, b[2], b[3]);
      }
    }
  }
}

// A float of the same address in another CTA of the cluster.
__device__ __forceinline__ float4 ld_cluster4(uint32_t addr, uint32_t cta) {
  float4 v;
  asm volatile(
      "{\n\t.reg .b32 r;\n\tmapa.shared::cluster.u32 r, %4, %5;\n\tld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [r];\n\t}"
      : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
      : "r"(addr), "r"(cta)
      : "memory");
  return v;
}
__device__ __forceinline__ float2 ld_cluster2(uint32_t addr, uint32_t cta) {
  float2 v;
  asm volatile("{\n\t.reg .b32 r;\n\tmapa.shared::cluster.u32 r, %2, %3;\n\tld.shared::cluster.v2.f32 {%0, %1}, [r];\n\t}"
               : "=f"(v.x), "=f"(v.y)
               : "r"(addr), "r"(cta)
               : "memory");
  return v;
}

template <int VT>
__global__ void __launch_bounds__(kStepThreads, 2) pa_step_kernel(const __grid_constant__ StepParams p) {
  using SM = StepSmem<VT>;
  constexpr int NS = SM::kStages;
  extern __shared__ __align__(1024) uint8_t step_smem[];
  const uint32_t base = smem_u32(step_smem);
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int C = p.cluster, rank = (int)(blockIdx.x % C), seg = (int)(blockIdx.x / C);
  const int head = seg % p.n_kv_heads;
  const StepSeq& sq = p.seq[seg / p.n_kv_heads];
  const int pos = sq.len - 1;
  // the key order (pa_window_impl.cuh), in row groups, and this CTA's share of it
  const Unit u{0, 0, pos, sq.len, kStepRows, 0, 0};
  const Span sp = span_of(u, p.window, p.sinks);
  const int groups = ceil_div(sp.end, kGroup);
  const int g0 = (int)((long long)groups * rank / C), g1 = (int)((long long)groups * (rank + 1) / C);
  const int n = g1 - g0 > w ? (g1 - g0 - w + kStepWarps - 1) / kStepWarps : 0;  // groups of this warp: g0 + w + 4 i
  asm volatile("griddepcontrol.wait;" ::: "memory");  // nothing that another kernel wrote is read before this
  if (tid == 0) asm volatile("griddepcontrol.launch_dependents;");

  // ---- copies: lane i looks up the warp's groups i, i + 32, ...
  const int32_t* row = p.table + (long long)sq.seq * p.table_stride;
  auto place = [&](int i) -> long long {  // first row of the warp's group i in the pools; -1: outside
    if (i >= n) return -1;
    const int v = (g0 + w + kStepWarps * i) * kGroup, k = v < sp.s16 ? v : v + sp.shift;
    const int page = p.page_shift >= 0 ? k >> p.page_shift : k / p.page_size;
    const int entry = __ldg(row + page);
    if ((uint32_t)entry >= (uint32_t)p.n_blocks) {
      record_error(p.err, PA_ERR_BOUNDS);
      return -1;
    }
    return ((long long)entry * p.n_kv_heads + head) * p.page_size + (k - page * p.page_size);
  };
  long long places = place(lane);
  const uint32_t ring = base + w * NS * SM::kStage;
  auto copy = [&](int i) {  // group i into its stage; rows of an entry outside the pool read as zeros
    if (i < n) {
      if (i > 0 && (i & 31) == 0) places = place(i + lane);
      const long long at = __shfl_sync(0xffffffffu, places, i & 31);
      const uint32_t to = ring + (i % NS) * SM::kStage;
      const int size = at >= 0 ? 16 : 0;
      const uint8_t* k = p.k_pool + (at >= 0 ? at : 0) * Fmt<PA_Q8_0>::kRow;
      const uint8_t* v = p.v_pool + (at >= 0 ? at : 0) * Fmt<VT>::kRow;
#pragma unroll
      for (int c = 0; c < (SM::kK + 511) / 512; ++c) {
        const int off = 512 * c + 16 * lane;
        if (off < SM::kK)
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to + off), "l"(k + off), "r"(size) : "memory");
      }
#pragma unroll
      for (int c = 0; c < (SM::kV + 511) / 512; ++c) {
        const int off = 512 * c + 16 * lane;
        if (off < SM::kV)
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to + SM::kK + off), "l"(v + off), "r"(size) : "memory");
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < NS - 1; ++i) copy(i);

  uint32_t q[32];
  step_queries(p, sq.token * p.q_stride + (long long)(head * kGqa + g) * kD, g < kStepRows, t, q);
  float o[16][4] = {};
  float ref[2] = {0.f, 0.f}, l[2] = {0.f, 0.f};  // rows 2t, 2t + 1; l of this thread's keys
  bool live[2] = {false, false};                 // a reference has been set
  for (int i = 0; i < n; ++i) {
    asm volatile("cp.async.wait_group %0;" ::"n"(NS - 2) : "memory");
    __syncwarp();  // and the stage before has been read
    copy(i + NS - 1);
    const uint32_t grp = ring + (i % NS) * SM::kStage;
    float s[4];
    step_scores(grp, q, g, t, s);
#pragma unroll
    for (int k = 0; k < 4; ++k) s[k] = fmaf(s[k], p.scale_log2, -ref[k & 1]);
    // the ends of the runs: keys that the token does not see
    const int v0 = (g0 + w + kStepWarps * i) * kGroup;
    uint32_t la = ~0u, lb = ~0u;
    const int lo = sp.lo - sp.shift;
    if (v0 + kGroup > sp.end || (v0 < lo && v0 + kGroup > p.sinks)) {
      auto sees = [&](int k) { return v0 + k < sp.end && (v0 + k >= lo || v0 + k < p.sinks); };
      if (!sees(g)) s[0] = s[1] = -INFINITY;
      if (!sees(g + 8)) s[2] = s[3] = -INFINITY;
      la = (sees(2 * t) ? 0xffffu : 0u) | (sees(2 * t + 1) ? 0xffff0000u : 0u);
      lb = (sees(2 * t + 8) ? 0xffffu : 0u) | (sees(2 * t + 9) ? 0xffff0000u : 0u);
    }
    float top[2] = {fmaxf(s[0], s[2]), fmaxf(s[1], s[3])};
    if (__any_sync(0xffffffffu, fmaxf(top[0], top[1]) > kLazyLog2 || !(live[0] && live[1]))) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) top[k] = fmaxf(top[k], __shfl_xor_sync(0xffffffffu, top[k], x));
        // the first reference is the first maximum above -inf; it rises when its own row asks for it, so that a
        // row's result does not depend on its neighbours'
        const float d = top[k] > (live[k] ? kLazyLog2 : -INFINITY) ? top[k] : 0.f;
        const float f = live[k] ? ex2(-d) : 1.f;
        live[k] |= top[k] != -INFINITY;  // NaN too
        ref[k] += d;
        l[k] *= f;
        s[k] -= d;
        s[k + 2] -= d;
#pragma unroll
        for (int x = 0; x < 16; ++x) {
          o[x][k] *= f;
          o[x][k + 2] *= f;
        }
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) s[k] = ex2(s[k]);
    l[0] += s[0] + s[2];
    l[1] += s[1] + s[3];
    uint32_t b[4];  // P in two parts of binary16
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint32_t hi = pack_half2(s[2 * k], s[2 * k + 1]);
      const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&hi));
      b[k] = movmatrix_trans(hi);
      b[2 + k] = movmatrix_trans(pack_half2(s[2 * k] - x.x, s[2 * k + 1] - x.y));
    }
    step_values<VT>(grp + SM::kK, o, b, la, lb, lane);
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int x = 4; x < 32; x <<= 1) l[k] += __shfl_xor_sync(0xffffffffu, l[k], x);

  // ---- the join: the warps' states, then the CTAs'
  __syncthreads();  // the rings are done with
  const uint32_t mine = base + w * SM::kState, ml = SM::kState - 64;
  auto put = [&](int r, int dim, float x) { asm volatile("st.shared.f32 [%0], %1;" ::"r"(mine + (r * kD + dim) * 4), "f"(x) : "memory"); };
  if (t < 3) {
#pragma unroll
    for (int i = 0; i < 16; ++i)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        put(2 * t + k, 16 * i + 2 * g, o[i][k]);
        put(2 * t + k, 16 * i + 2 * g + 1, o[i][k + 2]);
      }
    if (g == 0)
      asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(mine + ml + 16 * t), "f"(ref[0]), "f"(l[0]), "f"(ref[1]), "f"(l[1]) : "memory");
  }
  __syncthreads();
  // Of `count` states (state j's word at addr is load4(j, addr)), four values of row r, and its (M, W).
  auto joined = [&](int r, int c4, int count, auto&& load4, auto&& load2, float2* mw) -> float4 {
    float M = -INFINITY, W = 0.f;
    float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int j = 0; j < count; ++j) {
      const float2 x = load2(j, ml + 8 * r);
      if (x.y == 0.f) continue;  // sees nothing there; not a sum that is NaN
      const float4 y = load4(j, (r * kD + 4 * c4) * 4);
      const float top = fmaxf(M, x.x), f = W != 0.f ? exp2f(M - top) : 0.f, h = exp2f(x.x - top);
      W = fmaf(h, x.y, W * f);
      O = make_float4(fmaf(h, y.x, O.x * f), fmaf(h, y.y, O.y * f), fmaf(h, y.z, O.z * f), fmaf(h, y.w, O.w * f));
      M = top;
    }
    *mw = make_float2(M, W);
    return O;
  };
  const bool other = __ldg(p.lens + sq.seq) != sq.len;
  if (other && tid == 0 && rank == 0) record_error(p.err, PA_ERR_BOUNDS);
  auto finish = [&](int r, int c4, float4 O, float2 mw) {
    if (other) mw.y = 0.f;
    const float f = mw.y != 0.f ? 1.f / mw.y : 0.f;
    O = mw.y != 0.f ? make_float4(O.x * f, O.y * f, O.z * f, O.w * f) : make_float4(0.f, 0.f, 0.f, 0.f);
    const int h = head * kGqa + r;
    const long long at = sq.token * p.out_stride + h * kD + 4 * c4;
    if (p.out_type == PA_DT_F32) {
      *reinterpret_cast<float4*>(p.out + 4 * at) = O;
    } else if (p.out_type == PA_DT_F16) {
      *reinterpret_cast<uint2*>(p.out + 2 * at) = make_uint2(pack_half2(O.x, O.y), pack_half2(O.z, O.w));
    } else {
      const __nv_bfloat162 a = __floats2bfloat162_rn(O.x, O.y), b = __floats2bfloat162_rn(O.z, O.w);
      *reinterpret_cast<uint2*>(p.out + 2 * at) = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
    }
    if (c4 == 0 && p.lse) p.lse[(long long)sq.token * p.n_q_heads + h] = mw.y != 0.f ? (mw.x + log2f(mw.y)) * pa_split::kLn2 : -INFINITY;
  };
  auto here4 = [&](int j, uint32_t a) { return lds128f(base + j * SM::kState + a); };
  auto here2 = [&](int j, uint32_t a) {
    const uint2 v = lds64(base + j * SM::kState + a);
    return make_float2(__uint_as_float(v.x), __uint_as_float(v.y));
  };
  const uint32_t all = base + kStepWarps * SM::kState;  // the CTA's state
  for (int i = tid; i < kStepRows * 64; i += kStepThreads) {
    const int r = i >> 6, c4 = i & 63;
    float2 mw;
    const float4 O = joined(r, c4, kStepWarps, here4, here2, &mw);
    if (C == 1) {
      finish(r, c4, O, mw);
    } else {
      asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(all + (r * kD + 4 * c4) * 4), "f"(O.x), "f"(O.y), "f"(O.z), "f"(O.w) : "memory");
      if (c4 == 0) asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(all + ml + 8 * r), "f"(mw.x), "f"(mw.y) : "memory");
    }
  }
  if (C > 1) {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    // every CTA joins its part of the values
    for (int i = kStepRows * 64 * rank / C + tid; i < kStepRows * 64 * (rank + 1) / C; i += kStepThreads) {
      const int r = i >> 6, c4 = i & 63;
      float2 mw;
      const float4 O = joined(r, c4, C, [&](int j, uint32_t a) { return ld_cluster4(all + a, (uint32_t)j); },
                              [&](int j, uint32_t a) { return ld_cluster2(all + a, (uint32_t)j); }, &mw);
      finish(r, c4, O, mw);
    }
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");  // until the others have read
  }
}

}  // namespace pa_prefix
