// C ABI of the single operators (declared in include/moe_ops.h): argument
// validation and launches.  Everything here runs on the host.
#include <stdint.h>

#include <algorithm>

#include "../../../include/moe_ops.h"
#include "ops_launch.h"

namespace {

using namespace moe;

constexpr int64_t MAX_T = (1 << 24) - 1;   // a grid of 256 threads per token stays below 2^32
constexpr int64_t MAX_SLOTS = 1 << 30;
constexpr int MAX_K = 1024, MAX_E = 1024, MAX_ALIGN = 256;
constexpr int MAX_DIM = 1 << 20;
constexpr int64_t MAX_ELEMS = (int64_t)1 << 37;  // quantizers: values of a call

bool aligned(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

int check_plan_desc(const moe_plan_desc* d) {
  if (!d || d->flags || d->reserved) return MOE_EINVAL;
  if (d->T < 0 || d->K < 1 || d->E < 1 || d->align < 1) return MOE_EINVAL;
  if (d->T > MAX_T || d->K > MAX_K || d->E > MAX_E || d->align > MAX_ALIGN) return MOE_ESHAPE;
  if ((int64_t)d->T * d->K > MAX_SLOTS) return MOE_ESHAPE;
  return MOE_OK;
}

int64_t plan_rows(const moe_plan_desc* d) {
  const int64_t slots = (int64_t)d->T * d->K;
  return slots + std::min<int64_t>(d->E, slots) * (d->align - 1);
}

PlanArgs plan_args(const moe_plan_desc* d, const moe_plan* p) {
  return PlanArgs{d->T, d->K, d->E, d->align, (int)plan_rows(d), p->offsets, p->counts, p->row_token, p->slot_row};
}

// no rows at all: every buffer but offsets and counts may be null
bool plan_ok(const moe_plan_desc* d, const moe_plan* p) {
  if (!p || !p->offsets || !p->counts) return false;
  return d->T == 0 || (p->row_token && p->slot_row);
}

int check_dtype(int dtype) { return dtype == MOE_F32 || dtype == MOE_BF16 ? MOE_OK : MOE_EDTYPE; }

int check_width(int d) {
  if (d < 1) return MOE_EINVAL;
  return d % 16 == 0 && d <= MAX_DIM ? MOE_OK : MOE_ESHAPE;
}

// descriptor, plan, element type and row width of the row-moving calls
int check_rows(const moe_plan_desc* d, const moe_plan* p, int dtype, int width) {
  int s = check_plan_desc(d);
  if (s == MOE_OK && !plan_ok(d, p)) s = MOE_EINVAL;
  if (s == MOE_OK) s = check_dtype(dtype);
  if (s == MOE_OK) s = check_width(width);
  return s;
}

// an optional plan beside R rows: both of desc and plan, or neither
int check_optional_plan(const moe_plan_desc* d, const moe_plan* p, int64_t R, PlanArgs* out) {
  *out = PlanArgs{};
  if (R < 0) return MOE_EINVAL;
  if (!d && !p) return MOE_OK;
  int s = check_plan_desc(d);
  if (s != MOE_OK) return s;
  if (!plan_ok(d, p) || R != plan_rows(d)) return MOE_EINVAL;
  *out = plan_args(d, p);
  return MOE_OK;
}

// Event pair around an operator's launches when the caller asked for timing.
struct Timed {
  moe_profile* p;
  hipStream_t st;
  int slot;
  Timed(moe_profile* prof, hipStream_t s, int kernel) : p(prof), st(s), slot(-1) {
    if (p && p->count < p->capacity && p->start && p->stop) {
      slot = p->count++;
      if (p->kernel) p->kernel[slot] = kernel;
      (void)hipEventRecord((hipEvent_t)p->start[slot], st);
    }
  }
  ~Timed() {
    if (slot >= 0) (void)hipEventRecord((hipEvent_t)p->stop[slot], st);
  }
};

template <typename F>
int timed(moe_profile* p, void* stream, int kernel, F launch) {
  Timed t(p, (hipStream_t)stream, kernel);
  return launch((hipStream_t)stream) == hipSuccess ? MOE_OK : MOE_EHIP;
}

}  // namespace

extern "C" {

size_t moe_plan_rows(const moe_plan_desc* desc) {
  return check_plan_desc(desc) == MOE_OK ? (size_t)plan_rows(desc) : 0;
}

size_t moe_sort_workspace_bytes(const moe_plan_desc* desc) {
  if (check_plan_desc(desc) != MOE_OK) return 0;
  return (sort_ws_bytes((int64_t)desc->T * desc->K, desc->E) + 255) / 256 * 256;
}

int moe_sort(const moe_plan_desc* desc, const int32_t* expert_idx, const moe_plan* plan, void* ws, size_t ws_bytes,
             void* stream) {
  int s = check_plan_desc(desc);
  if (s != MOE_OK) return s;
  if (!plan_ok(desc, plan) || (desc->T > 0 && !expert_idx)) return MOE_EINVAL;
  const size_t need = moe_sort_workspace_bytes(desc);
  if (need > 0) {
    if (!ws || !aligned(ws, 256)) return MOE_EINVAL;
    if (ws_bytes < need) return MOE_EWORKSPACE;
  }
  return timed(desc->profile, stream, MOE_OPS_K_SORT,
               [&](hipStream_t st) { return launch_sort(plan_args(desc, plan), expert_idx, *plan, ws, st); });
}

int moe_permute(const moe_plan_desc* desc, const moe_plan* plan, int dtype, int d, const void* x, void* xp,
                void* stream) {
  int s = check_rows(desc, plan, dtype, d);
  if (s != MOE_OK) return s;
  if (desc->T == 0) return MOE_OK;
  if (!x || !xp || !aligned(x, 16) || !aligned(xp, 16)) return MOE_EINVAL;
  return timed(desc->profile, stream, MOE_OPS_K_PERMUTE,
               [&](hipStream_t st) { return launch_permute(plan_args(desc, plan), dtype, d, x, xp, st); });
}

int moe_permute_fp8(const moe_plan_desc* desc, const moe_plan* plan, int dtype, int d, const void* x, void* q,
                    float* s, void* stream) {
  int e = check_rows(desc, plan, dtype, d);
  if (e != MOE_OK) return e;
  if (desc->T == 0) return MOE_OK;
  if (!x || !q || !s || !aligned(x, 16) || !aligned(q, 16) || !aligned(s, 4)) return MOE_EINVAL;
  return timed(desc->profile, stream, MOE_OPS_K_PERMUTE_FP8, [&](hipStream_t st) {
    return launch_permute_fp8(plan_args(desc, plan), dtype, d, x, (uint8_t*)q, s, st);
  });
}

int moe_permute_bwd(const moe_plan_desc* desc, const moe_plan* plan, int dtype, int d, const void* dxp, void* dx,
                    void* stream) {
  int s = check_rows(desc, plan, dtype, d);
  if (s != MOE_OK) return s;
  if (desc->T == 0) return MOE_OK;
  if (!dxp || !dx || !aligned(dxp, 16) || !aligned(dx, 16)) return MOE_EINVAL;
  return timed(desc->profile, stream, MOE_OPS_K_UNPERMUTE,
               [&](hipStream_t st) { return launch_unpermute(plan_args(desc, plan), dtype, d, dxp, nullptr, dx, st); });
}

int moe_unpermute(const moe_plan_desc* desc, const moe_plan* plan, int dtype, int d, const void* y, const float* w,
                  void* o, void* stream) {
  int s = check_rows(desc, plan, dtype, d);
  if (s != MOE_OK) return s;
  if (desc->T == 0) return MOE_OK;
  if (!y || !w || !o || !aligned(y, 16) || !aligned(w, 4) || !aligned(o, 16)) return MOE_EINVAL;
  return timed(desc->profile, stream, MOE_OPS_K_UNPERMUTE,
               [&](hipStream_t st) { return launch_unpermute(plan_args(desc, plan), dtype, d, y, w, o, st); });
}

int moe_unpermute_bwd(const moe_plan_desc* desc, const moe_plan* plan, int dtype, int d, const void* d_o,
                      const void* y, const float* w, void* dy, float* dw, void* stream) {
  int s = check_rows(desc, plan, dtype, d);
  if (s != MOE_OK) return s;
  if (!dy && !dw) return MOE_EINVAL;
  if (desc->T == 0) return MOE_OK;
  if (!d_o || (dw && !y) || (dy && !w)) return MOE_EINVAL;
  if (!aligned(d_o, 16) || !aligned(y, 16) || !aligned(w, 4) || !aligned(dy, 16) || !aligned(dw, 4)) return MOE_EINVAL;
  return timed(desc->profile, stream, MOE_OPS_K_UNPERMUTE_BWD, [&](hipStream_t st) {
    return launch_unpermute_bwd(plan_args(desc, plan), dtype, d, d_o, y, w, dy, dw, st);
  });
}

int moe_fp8_quant_rows(const moe_plan_desc* desc, const moe_plan* plan, int dtype, int64_t R, int C, const void* src,
                       void* q, float* s, moe_profile* profile, void* stream) {
  PlanArgs p;
  int e = check_optional_plan(desc, plan, R, &p);
  if (e == MOE_OK) e = check_dtype(dtype);
  if (e == MOE_OK) e = check_width(C);
  if (e != MOE_OK) return e;
  if (R > MAX_ELEMS / C) return MOE_ESHAPE;
  if (R == 0) return MOE_OK;
  if (!src || !q || !s || !aligned(src, 16) || !aligned(q, 16) || !aligned(s, 4)) return MOE_EINVAL;
  return timed(profile, stream, MOE_OPS_K_QUANT_ROWS,
               [&](hipStream_t st) { return launch_quant_rows_128(p, dtype, R, C, src, (uint8_t*)q, s, st); });
}

int moe_fp8_quant_weights(int dtype, int E, int K, int N, const void* w, void* q, void* qt, float* s,
                          moe_profile* profile, void* stream) {
  if (E < 1) return MOE_EINVAL;
  int e = check_dtype(dtype);
  if (e == MOE_OK) e = check_width(K);
  if (e == MOE_OK) e = check_width(N);
  if (e != MOE_OK) return e;
  if (E > MAX_E || (int64_t)K * N > MAX_ELEMS / E) return MOE_ESHAPE;
  if (!w || !s || (!q && !qt) || !aligned(w, 16) || !aligned(q, 16) || !aligned(qt, 16) || !aligned(s, 4))
    return MOE_EINVAL;
  return timed(profile, stream, MOE_OPS_K_QUANT_WEIGHTS, [&](hipStream_t st) {
    return launch_quant_weights_128(dtype, E, K, N, w, (uint8_t*)q, (uint8_t*)qt, s, st);
  });
}

int moe_fp8_quant_cols(const moe_plan_desc* desc, const moe_plan* plan, int dtype, int C, int gather, const void* src,
                       void* q, float* s, void* stream) {
  int e = check_rows(desc, plan, dtype, C);
  if (e != MOE_OK) return e;
  if (desc->align % 128 != 0 || plan_rows(desc) > MAX_ELEMS / C) return MOE_ESHAPE;
  if (desc->T == 0) return MOE_OK;
  if (!src || !q || !s || !aligned(src, 16) || !aligned(q, 16) || !aligned(s, 4)) return MOE_EINVAL;
  return timed(desc->profile, stream, MOE_OPS_K_QUANT_COLS, [&](hipStream_t st) {
    return launch_quant_cols_128(plan_args(desc, plan), dtype, C, gather != 0, src, (uint8_t*)q, s, st);
  });
}

int moe_fp8_mm(const moe_mm_desc* desc, const void* a, const float* sa, const void* b, const float* sb,
               const moe_plan* plan, void* c, void* stream) {
  if (!desc || desc->reserved || (desc->flags & ~(MOE_MM_GATHER | MOE_MM_SB_OUT_MAJOR))) return MOE_EINVAL;
  const bool gather = (desc->flags & MOE_MM_GATHER) != 0;
  if (desc->a_rows < 0 || desc->rows < 0 || desc->E < 1) return MOE_EINVAL;
  if (desc->rows_used < 0 || desc->rows_used > desc->rows) return MOE_EINVAL;
  int e = check_dtype(desc->out);
  if (e == MOE_OK) e = check_width(desc->K);
  if (e == MOE_OK) e = check_width(desc->N);
  if (e != MOE_OK) return e;
  if (!plan && (desc->E != 1 || gather)) return MOE_EINVAL;
  if (!gather && desc->a_rows != desc->rows) return MOE_EINVAL;
  if (desc->E > MAX_E) return MOE_ESHAPE;
  if ((int64_t)desc->N * desc->K >= INT32_MAX) return MOE_ESHAPE;
  // the scales' byte offsets are at most four to a code's 128 (and to a row of K < 128)
  const int64_t line = std::max<int64_t>(desc->K, 4 * ((desc->K + 127) / 128));
  if (gather && (int64_t)desc->a_rows * line >= INT32_MAX) return MOE_ESHAPE;
  if (desc->rows == 0) return MOE_OK;
  if (desc->a_rows == 0) return MOE_EINVAL;  // rows of no token
  if (plan && (!plan->offsets || !plan->counts || (gather && !plan->row_token))) return MOE_EINVAL;
  if (!a || !sa || !b || !sb || !c) return MOE_EINVAL;
  if (!aligned(a, 16) || !aligned(b, 16) || !aligned(c, 16) || !aligned(sa, 4) || !aligned(sb, 4)) return MOE_EINVAL;
  const int used = desc->rows_used > 0 ? desc->rows_used : desc->rows;
  PlanArgs p{};
  if (plan) {
    p.offsets = plan->offsets;
    p.counts = plan->counts;
    p.row_token = plan->row_token;
  }
  const Fp8MmArgs g{(const uint8_t*)a, sa, (const uint8_t*)b, sb, c, desc->a_rows, desc->rows, used, desc->E, desc->K,
                    desc->N, desc->out, gather, (desc->flags & MOE_MM_SB_OUT_MAJOR) != 0};
  return timed(desc->profile, stream, MOE_OPS_K_FP8_MM, [&](hipStream_t st) { return launch_fp8_mm(p, g, st); });
}

int moe_fp8_wgrad(const moe_plan_desc* desc, const moe_plan* plan, int M, int N, int out, const void* a,
                  const float* sa, const void* b, const float* sb, void* dw, void* stream) {
  int e = check_rows(desc, plan, out, M);
  if (e == MOE_OK) e = check_width(N);
  if (e != MOE_OK) return e;
  if (desc->align % 128 != 0) return MOE_ESHAPE;
  if (!dw || !aligned(dw, 16)) return MOE_EINVAL;
  if (desc->T > 0 && (!a || !sa || !b || !sb)) return MOE_EINVAL;
  if (!aligned(a, 16) || !aligned(b, 16) || !aligned(sa, 4) || !aligned(sb, 4)) return MOE_EINVAL;
  return timed(desc->profile, stream, MOE_OPS_K_FP8_WGRAD, [&](hipStream_t st) {
    return launch_fp8_wgrad(plan_args(desc, plan), M, N, out, (const uint8_t*)a, sa, (const uint8_t*)b, sb, dw, st);
  });
}

int moe_swiglu_fp8(const moe_plan_desc* desc, const moe_plan* plan, int dtype, int64_t R, int n, const void* h,
                   void* q, float* s, void* a, moe_profile* profile, void* stream) {
  PlanArgs p;
  int e = check_optional_plan(desc, plan, R, &p);
  if (e == MOE_OK) e = check_dtype(dtype);
  if (e == MOE_OK) e = check_width(n);
  if (e != MOE_OK) return e;
  if (R > MAX_ELEMS / n) return MOE_ESHAPE;
  if (R == 0) return MOE_OK;
  if (!h || !q || !s || !aligned(h, 16) || !aligned(q, 16) || !aligned(s, 4) || !aligned(a, 16)) return MOE_EINVAL;
  return timed(profile, stream, MOE_OPS_K_SWIGLU_FP8,
               [&](hipStream_t st) { return launch_swiglu_fp8(p, dtype, R, n, h, (uint8_t*)q, s, a, st); });
}

int moe_swiglu_bwd(const moe_plan_desc* desc, const moe_plan* plan, int dtype, int64_t R, int n, const void* da,
                   const void* h, void* dh, moe_profile* profile, void* stream) {
  PlanArgs p;
  int e = check_optional_plan(desc, plan, R, &p);
  if (e == MOE_OK) e = check_dtype(dtype);
  if (e == MOE_OK) e = check_width(n);
  if (e != MOE_OK) return e;
  if (R > MAX_ELEMS / n) return MOE_ESHAPE;
  if (R == 0) return MOE_OK;
  if (!da || !h || !dh || !aligned(da, 16) || !aligned(h, 16) || !aligned(dh, 16)) return MOE_EINVAL;
  return timed(profile, stream, MOE_OPS_K_SWIGLU_BWD,
               [&](hipStream_t st) { return launch_swiglu_bwd_rows(p, dtype, R, n, da, h, dh, st); });
}

}  // extern "C"
