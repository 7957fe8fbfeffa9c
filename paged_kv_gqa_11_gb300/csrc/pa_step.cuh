// Windowed attention of one new token per sequence: parameters of its kernel (pa_step_impl.cuh)
// for the host side (pa_window.cu).
#pragma once

#include <cuda_runtime.h>

#include "pa_window_impl.cuh"

namespace pa_prefix {

constexpr int kMaxStepSeqs = 256;  // to a launch: its parameters stay below 4 KB

struct StepSeq {
  int32_t seq, token, len;  // row of the table, of the queries, length (the token is the last)
};

struct StepParams {
  const uint8_t* q;
  const uint8_t* k_pool;
  const uint8_t* v_pool;
  const int32_t* table;
  const int32_t* lens;  // device lengths, only compared
  int32_t* err;
  uint8_t* out;
  float* lse;
  long long q_stride, out_stride;  // values per token
  int q_type, out_type, n_kv_heads, n_q_heads, page_size, table_stride, n_blocks;
  int page_shift;  // log2 of page_size, or -1
  int cluster;     // CTAs of a segment
  int window, sinks;
  float scale_log2;
  StepSeq seq[kMaxStepSeqs];
};

constexpr int kStepWarps = 4, kStepThreads = 32 * kStepWarps;

using StepKernel = KernelOf<StepParams>;  // fn null: the pair has none

#define PA_DECLARE_STEP(k, v) bool lookup_step_kernel_##k##_##v(StepKernel* out);
PA_DECLARE_STEP(1, 1) PA_DECLARE_STEP(1, 2) PA_DECLARE_STEP(1, 8)
PA_DECLARE_STEP(2, 1) PA_DECLARE_STEP(2, 2) PA_DECLARE_STEP(2, 8)
PA_DECLARE_STEP(8, 1) PA_DECLARE_STEP(8, 2) PA_DECLARE_STEP(8, 8)
#undef PA_DECLARE_STEP

}  // namespace pa_prefix
