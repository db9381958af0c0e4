// Launchers of the operators declared in include/moe_step_ops.h.  They only
// enqueue work on `st`; the ABI layer has validated every size.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <algorithm>

#include "../../../include/moe_step_ops.h"
#include "../device_common.h"
#include "ops_launch.h"

namespace moe {

// ---- balance_kernels.hip ----
struct BalanceArgs {
  int T, E, K, dtype;
  const void* z;
  const int32_t* idx;
  const uint8_t* valid;  // or null
  int32_t* counts;
  int32_t* tokens;
  float* load;
  float* lse;
  float* loss;
  void* ws;
};
size_t balance_ws_bytes(int T, int E, int K);
hipError_t launch_balance(const BalanceArgs& a, hipStream_t st);

struct BalanceBwdArgs {
  int T, E, K, dtype;
  const void* z;
  const int32_t* counts;
  const int32_t* tokens;
  const float* lse;
  const float* d_loss;
  const int32_t* idx;    // null: the losses' gradient alone
  const float* gate;
  const float* d_gate;
  void* dz;
};
hipError_t launch_balance_bwd(const BalanceBwdArgs& a, hipStream_t st);

// ---- ortho_kernels.hip ----
struct OrthoArgs {
  int E, M, N, dtype, steps;
  const float* coef;     // host, [steps][3]
  float eps, scale;
  const void* g;
  void* o;
  void* ws;
};
size_t ortho_ws_bytes(const OrthoArgs& a);
hipError_t launch_orthogonalize(const OrthoArgs& a, hipStream_t st);

// ---- mxfp4_kernels.hip ----
struct Mxfp4Args {
  const bf16_t* a;
  const uint8_t* q;
  const uint8_t* s;
  void* c;
  int a_rows, rows, rows_used, E, K, N;
  int out;
  bool gather;
};
// at most so many tiles of BM rows have a row
inline int64_t mxfp4_row_tiles(int64_t used, int E, int BM) {
  return std::min(used, (used + BM - 1) / BM + std::min<int64_t>(E, used));
}
// tiles of a launch, workgroups of 256 in whole eights (a grid has fewer than 2^32 threads)
constexpr int64_t MXFP4_MAX_TILES = (1 << 24) - 8;
hipError_t launch_mxfp4_weights(int dtype, int E, int K, int N, const void* w, uint8_t* q, uint8_t* s, hipStream_t st);
hipError_t launch_mxfp4_mm(const PlanArgs& p, const Mxfp4Args& m, hipStream_t st);

}  // namespace moe
