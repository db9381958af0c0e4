// C ABI of the operators in include/moe_step_ops.h: argument validation and
// launches.  Everything here runs on the host.
#include <stdint.h>

#include <algorithm>
#include <cmath>

#include "../../../include/moe_step_ops.h"
#include "step_launch.h"

namespace {

using namespace moe;

constexpr int64_t MAX_T = (1 << 24) - 1;
constexpr int64_t MAX_SLOTS = 1 << 30;
constexpr int MAX_K = 1024, MAX_E = 1024;

bool aligned(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

int check_dtype(int dtype) { return dtype == MOE_F32 || dtype == MOE_BF16 ? MOE_OK : MOE_EDTYPE; }

size_t elem_bytes(int dtype) { return dtype == MOE_F32 ? 4 : 2; }

// a workspace of `need` bytes
int check_ws(const void* ws, size_t ws_bytes, size_t need) {
  if (need == 0) return MOE_OK;
  if (!ws || !aligned(ws, 256)) return MOE_EINVAL;
  return ws_bytes < need ? MOE_EWORKSPACE : MOE_OK;
}

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

// Event pair around an operator's launches when the caller asked for timing.
template <typename F>
int timed(moe_profile* p, void* stream, int kernel, F launch) {
  hipStream_t st = (hipStream_t)stream;
  int slot = -1;
  if (p && p->count < p->capacity && p->start && p->stop) {
    slot = p->count++;
    if (p->kernel) p->kernel[slot] = kernel;
    (void)hipEventRecord((hipEvent_t)p->start[slot], st);
  }
  const hipError_t e = launch(st);
  if (slot >= 0) (void)hipEventRecord((hipEvent_t)p->stop[slot], st);
  return e == hipSuccess ? MOE_OK : MOE_EHIP;
}

int check_balance(const moe_balance_desc* d) {
  if (!d || d->flags || d->reserved) return MOE_EINVAL;
  if (d->T < 0 || d->K < 1 || d->E < 1) return MOE_EINVAL;
  const int s = check_dtype(d->dtype);
  if (s != MOE_OK) return s;
  if (d->T > MAX_T || d->K > MAX_K || d->E > MAX_E || (int64_t)d->T * d->K > MAX_SLOTS) return MOE_ESHAPE;
  return MOE_OK;
}

constexpr int MAX_DIM = 1 << 20;

int check_mxfp4(int E, int K, int N) {
  if (E < 1 || K < 1 || N < 1) return MOE_EINVAL;
  return E <= MAX_E && K % 32 == 0 && N % 16 == 0 && K <= MAX_DIM && N <= MAX_DIM ? MOE_OK : MOE_ESHAPE;
}

constexpr int MAX_STEPS = 64, MAX_SIDE = 16384;
constexpr int64_t MAX_MATRIX = (int64_t)1 << 29;  // a two-part matrix's byte offsets stay below 2^31

int check_ortho(const moe_ortho_desc* d) {
  if (!d || d->flags || d->reserved) return MOE_EINVAL;
  if (d->E < 1 || d->M < 1 || d->N < 1 || d->steps < 1 || !d->coef) return MOE_EINVAL;
  const int s = check_dtype(d->dtype);
  if (s != MOE_OK) return s;
  if (d->E > MAX_E || d->steps > MAX_STEPS || std::min(d->M, d->N) > MAX_SIDE) return MOE_ESHAPE;
  if (((int64_t)d->M + 63) / 64 * 64 * (((int64_t)d->N + 63) / 64 * 64) >= MAX_MATRIX) return MOE_ESHAPE;
  if (!std::isfinite(d->eps) || d->eps < 0.f || !std::isfinite(d->scale)) return MOE_EINVAL;
  for (int i = 0; i < 3 * d->steps; ++i)
    if (!std::isfinite(d->coef[i])) return MOE_EINVAL;
  return MOE_OK;
}

OrthoArgs ortho_args(const moe_ortho_desc* d, const void* g, void* o, void* ws) {
  return OrthoArgs{d->E, d->M, d->N, d->dtype, d->steps, d->coef, d->eps, d->scale, g, o, ws};
}

}  // namespace

extern "C" {

size_t moe_balance_workspace_bytes(const moe_balance_desc* desc) {
  return check_balance(desc) == MOE_OK ? up256(balance_ws_bytes(desc->T, desc->E, desc->K)) : 0;
}

int moe_balance(const moe_balance_desc* desc, const void* logits, const int32_t* expert_idx, const uint8_t* valid,
                int32_t* counts, int32_t* tokens, float* load, float* lse, float* loss, void* ws, size_t ws_bytes,
                void* stream) {
  int s = check_balance(desc);
  if (s != MOE_OK) return s;
  if (!counts || !tokens || !load || !loss) return MOE_EINVAL;
  if (!aligned(counts, 4) || !aligned(tokens, 4) || !aligned(load, 4) || !aligned(loss, 4)) return MOE_EINVAL;
  if (desc->T > 0 && (!logits || !expert_idx || !lse)) return MOE_EINVAL;
  if (!aligned(logits, elem_bytes(desc->dtype)) || !aligned(expert_idx, 4) || !aligned(lse, 4)) return MOE_EINVAL;
  s = check_ws(ws, ws_bytes, moe_balance_workspace_bytes(desc));
  if (s != MOE_OK) return s;
  const BalanceArgs a{desc->T, desc->E, desc->K, desc->dtype, logits, expert_idx, valid, counts, tokens, load, lse,
                      loss, ws};
  return timed(desc->profile, stream, MOE_STEP_K_BALANCE, [&](hipStream_t st) { return launch_balance(a, st); });
}

int moe_balance_bwd(const moe_balance_desc* desc, const void* logits, const int32_t* counts, const int32_t* tokens,
                    const float* lse, const float* d_loss, const int32_t* expert_idx, const float* gate,
                    const float* d_gate, void* dz, void* stream) {
  const int s = check_balance(desc);
  if (s != MOE_OK) return s;
  if ((expert_idx || gate || d_gate) && !(expert_idx && gate && d_gate)) return MOE_EINVAL;
  if (desc->T == 0) return MOE_OK;
  if (!logits || !counts || !tokens || !lse || !d_loss || !dz) return MOE_EINVAL;
  const size_t e = elem_bytes(desc->dtype);
  if (!aligned(logits, e) || !aligned(dz, e) || !aligned(counts, 4) || !aligned(tokens, 4) || !aligned(lse, 4) ||
      !aligned(d_loss, 4) || !aligned(expert_idx, 4) || !aligned(gate, 4) || !aligned(d_gate, 4))
    return MOE_EINVAL;
  const BalanceBwdArgs a{desc->T, desc->E, desc->K, desc->dtype, logits, counts, tokens, lse, d_loss,
                         expert_idx, gate, d_gate, dz};
  return timed(desc->profile, stream, MOE_STEP_K_BALANCE_BWD,
               [&](hipStream_t st) { return launch_balance_bwd(a, st); });
}

size_t moe_orthogonalize_workspace_bytes(const moe_ortho_desc* desc) {
  return check_ortho(desc) == MOE_OK ? up256(ortho_ws_bytes(ortho_args(desc, nullptr, nullptr, nullptr))) : 0;
}

int moe_orthogonalize(const moe_ortho_desc* desc, const void* g, void* o, void* ws, size_t ws_bytes, void* stream) {
  int s = check_ortho(desc);
  if (s != MOE_OK) return s;
  const size_t e = elem_bytes(desc->dtype);
  if (!g || !o || !aligned(g, e) || !aligned(o, e)) return MOE_EINVAL;
  const OrthoArgs a = ortho_args(desc, g, o, ws);
  s = check_ws(ws, ws_bytes, up256(ortho_ws_bytes(a)));
  if (s != MOE_OK) return s;
  return timed(desc->profile, stream, MOE_STEP_K_ORTHOGONALIZE,
               [&](hipStream_t st) { return launch_orthogonalize(a, st); });
}

int moe_mxfp4_quant_weights(int dtype, int E, int K, int N, const void* w, void* q, void* s, moe_profile* profile,
                            void* stream) {
  int e = check_dtype(dtype);
  if (e == MOE_OK) e = check_mxfp4(E, K, N);
  if (e != MOE_OK) return e;
  if ((int64_t)K * N > ((int64_t)1 << 37) / E) return MOE_ESHAPE;
  if (!w || !q || !s || !aligned(w, 16) || !aligned(q, 16)) return MOE_EINVAL;
  return timed(profile, stream, MOE_STEP_K_MXFP4_WEIGHTS, [&](hipStream_t st) {
    return launch_mxfp4_weights(dtype, E, K, N, w, (uint8_t*)q, (uint8_t*)s, st);
  });
}

int moe_mxfp4_mm(const moe_mm_desc* desc, const void* a, const void* q, const void* s, const moe_plan* plan, void* c,
                 void* stream) {
  if (!desc || desc->reserved || (desc->flags & ~MOE_MM_GATHER)) return MOE_EINVAL;
  const bool gather = (desc->flags & MOE_MM_GATHER) != 0;
  if (desc->a_rows < 0 || desc->rows < 0 || desc->rows_used < 0 || desc->rows_used > desc->rows) return MOE_EINVAL;
  int e = check_dtype(desc->out);
  if (e == MOE_OK) e = check_mxfp4(desc->E, desc->K, desc->N);
  if (e != MOE_OK) return e;
  if (!plan && (desc->E != 1 || gather)) return MOE_EINVAL;
  if (!gather && desc->a_rows != desc->rows) return MOE_EINVAL;
  if ((int64_t)desc->N * desc->K >= INT32_MAX) return MOE_ESHAPE;
  if (gather && (int64_t)desc->a_rows * desc->K >= ((int64_t)1 << 30)) return MOE_ESHAPE;
  if (desc->rows == 0) return MOE_OK;
  const int64_t used = desc->rows_used > 0 ? desc->rows_used : desc->rows;
  if (mxfp4_row_tiles(used, desc->E, 128) * (((int64_t)desc->N + 255) / 256) >= MXFP4_MAX_TILES) return MOE_ESHAPE;
  if (desc->a_rows == 0) return MOE_EINVAL;  // rows of no token
  if (plan && (!plan->offsets || !plan->counts || (gather && !plan->row_token))) return MOE_EINVAL;
  if (!a || !q || !s || !c || !aligned(a, 16) || !aligned(q, 16) || !aligned(c, 16)) return MOE_EINVAL;
  PlanArgs p{};
  if (plan) {
    p.offsets = plan->offsets;
    p.counts = plan->counts;
    p.row_token = plan->row_token;
  }
  const Mxfp4Args g{(const bf16_t*)a, (const uint8_t*)q, (const uint8_t*)s, c, desc->a_rows, desc->rows,
                    (int)used, desc->E, desc->K, desc->N, desc->out, gather};
  return timed(desc->profile, stream, MOE_STEP_K_MXFP4_MM, [&](hipStream_t st) { return launch_mxfp4_mm(p, g, st); });
}

}  // extern "C"
