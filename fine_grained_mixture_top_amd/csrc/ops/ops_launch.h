// Launchers of the operators declared in include/moe_ops.h.  As in launch.h
// they only enqueue work on `st`; the ABI layer has validated every size.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../../include/moe_ops.h"

namespace moe {

// Plan sizes and device buffers as the kernels take them.
struct PlanArgs {
  int T, K, E, align;
  int cap;                   // rows of the row buffers
  const int32_t* offsets;    // null: no plan (dense)
  const int32_t* counts;
  const int32_t* row_token;
  const int32_t* slot_row;
};

// ---- permute_kernels.hip ----
size_t sort_ws_bytes(int64_t slots, int E);
hipError_t launch_sort(const PlanArgs& p, const int32_t* expert_idx, const moe_plan& out, void* ws, hipStream_t st);
hipError_t launch_permute(const PlanArgs& p, int dtype, int d, const void* x, void* xp, hipStream_t st);
hipError_t launch_permute_fp8(const PlanArgs& p, int dtype, int d, const void* x, uint8_t* q, float* s,
                              hipStream_t st);
// w null: weights of one
hipError_t launch_unpermute(const PlanArgs& p, int dtype, int d, const void* y, const float* w, void* o,
                            hipStream_t st);
hipError_t launch_unpermute_bwd(const PlanArgs& p, int dtype, int d, const void* d_o, const void* y, const float* w,
                                void* dy, float* dw, hipStream_t st);

// ---- fp8_kernels.hip ----
hipError_t launch_quant_rows_128(const PlanArgs& p, int dtype, int64_t R, int C, const void* src, uint8_t* q,
                                 float* s, hipStream_t st);
hipError_t launch_quant_weights_128(int dtype, int E, int K, int N, const void* w, uint8_t* q, uint8_t* qt, float* s,
                                    hipStream_t st);
hipError_t launch_quant_cols_128(const PlanArgs& p, int dtype, int C, bool gather, const void* src, uint8_t* q,
                                 float* s, hipStream_t st);
hipError_t launch_swiglu_fp8(const PlanArgs& p, int dtype, int64_t R, int n, const void* h, uint8_t* q, float* s,
                             void* a, hipStream_t st);
hipError_t launch_swiglu_bwd_rows(const PlanArgs& p, int dtype, int64_t R, int n, const void* da, const void* h,
                                  void* dh, hipStream_t st);

// ---- fp8_gemm.hip ----
struct Fp8MmArgs {
  const uint8_t* a;
  const float* sa;
  const uint8_t* b;
  const float* sb;
  void* c;
  int a_rows, rows, rows_used, E, K, N;
  int out;
  bool gather, sb_out_major;
};
hipError_t launch_fp8_mm(const PlanArgs& p, const Fp8MmArgs& g, hipStream_t st);
hipError_t launch_fp8_wgrad(const PlanArgs& p, int M, int N, int out, const uint8_t* a, const float* sa,
                            const uint8_t* b, const float* sb, void* dw, hipStream_t st);

}  // namespace moe
