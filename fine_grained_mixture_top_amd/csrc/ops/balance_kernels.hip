// The router's balance and z losses and the gradient of its logits
// (include/moe_step_ops.h: moe_balance, moe_balance_bwd).
//
// A row of E logits lies across L lanes (a power of two), V neighbouring
// columns per lane and vector, R vectors: column (r L + lane % L) V + v.  A
// wave holds 64 / L rows at once, so a lane sees the same columns in every row
// and sums their probabilities in registers.  Every workgroup leaves one line of
// sums (probabilities, counts, lse^2, tokens), a second launch adds the lines up
// in fixed order: no floating-point atomics.  Calls of few logits are one
// workgroup and one launch.
#include <algorithm>
#include <type_traits>

#include "../device_common.h"
#include "step_launch.h"

namespace moe {

namespace {

constexpr float NEG_INF = -__builtin_inff();
constexpr int MAX_E = 1024;
constexpr int FWD_BLOCKS = 512;

template <typename T, int V> struct Vec;
template <> struct Vec<float, 1> { typedef float type; };
template <> struct Vec<float, 4> { typedef float4 type; };
template <> struct Vec<bf16_t, 1> { typedef bf16_t type; };
template <> struct Vec<bf16_t, 4> { typedef uint2 type; };
template <> struct Vec<bf16_t, 8> { typedef uint4 type; };

template <typename T, int V>
__device__ __forceinline__ void load_vec(const T* p, float (&v)[V]) {
  typedef typename Vec<T, V>::type W;
  const W w = *reinterpret_cast<const W*>(p);
  T e[V];
  __builtin_memcpy(e, &w, sizeof(w));
#pragma unroll
  for (int i = 0; i < V; ++i) v[i] = Elem<T>::to_f(e[i]);
}
template <typename T, int V>
__device__ __forceinline__ void store_vec(T* p, const float (&v)[V]) {
  typedef typename Vec<T, V>::type W;
  T e[V];
#pragma unroll
  for (int i = 0; i < V; ++i) e[i] = Elem<T>::from_f(v[i]);
  W w;
  __builtin_memcpy(&w, e, sizeof(w));
  *reinterpret_cast<W*>(p) = w;
}

// The other value of a pair of lanes 2^K apart (K < 4), in lanes that are alike within 2^K:
// moves between lanes of the vector unit.
template <int K> __device__ __forceinline__ float partner(float v) {
  const int i = __float_as_int(v);
  if constexpr (K == 0) return __int_as_float(__builtin_amdgcn_mov_dpp(i, 0xB1, 15, 15, true));   // quad_perm 1 0 3 2
  if constexpr (K == 1) return __int_as_float(__builtin_amdgcn_mov_dpp(i, 0x4E, 15, 15, true));   // quad_perm 2 3 0 1
  if constexpr (K == 2) return __int_as_float(__builtin_amdgcn_mov_dpp(i, 0x141, 15, 15, true));  // mirror in 8 lanes
  return __int_as_float(__builtin_amdgcn_mov_dpp(i, 0x140, 15, 15, true));                        // mirror in 16
}
// f over the 2^log_l lanes that hold a row, U rows side by side
template <int K = 0, int U, typename F>
__device__ __forceinline__ void over_row(float (&v)[U], int log_l, F f) {
  if (log_l > K) {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      if constexpr (K < 4) {
        v[i] = f(v[i], partner<K>(v[i]));
      } else {  // rows of 16 (halves) of one copy change places with those of another: both have a pair's two values
        const int x = __float_as_int(v[i]);
        const auto two = K == 4 ? __builtin_amdgcn_permlane16_swap(x, x, false, false)
                                : __builtin_amdgcn_permlane32_swap(x, x, false, false);
        v[i] = f(__int_as_float((int)two[0]), __int_as_float((int)two[1]));
      }
    }
    if constexpr (K < 5) over_row<K + 1>(v, log_l, f);
  }
}
template <int U> __device__ __forceinline__ void row_sum(float (&v)[U], int log_l) {
  over_row(v, log_l, [](float a, float b) { return a + b; });
}
// (a NaN has to come through: fmaxf drops it, so it counts as +inf, whose exponentials are
// NaN as well)
__device__ __forceinline__ float max_nan(float m, float v) { return v != v ? __builtin_inff() : fmaxf(m, v); }
template <int U> __device__ __forceinline__ void row_max(float (&v)[U], int log_l) {
  over_row(v, log_l, [](float a, float b) { return fmaxf(a, b); });
}

// lines of the workspace: E sums of probabilities, E counts, lse^2, tokens
__host__ __device__ inline int line_words(int E) { return 2 * E + 2; }
// (behind them the final launch's sums of counts * load, one a workgroup, and an arrival count)
constexpr int FINAL_COLS = 16;
constexpr int TAIL_WORDS = MAX_E / FINAL_COLS + 1;

struct Fwd {
  BalanceArgs a;
  int logL;
  uint32_t* line;   // [gridDim.x][line_words]
  uint32_t* tail;   // [TAIL_WORDS]
};

// One unit: 64 / L rows, one per group of L lanes.
template <typename T, int V, int R>
struct Unit {
  float z[R][V];
  int t;
  bool there, valid;
  __device__ __forceinline__ void load(const Fwd& f, int64_t unit, int lane) {
    const int L = 1 << f.logL, j = lane & (L - 1);
    const int64_t row = unit * (64 >> f.logL) + (lane >> f.logL);
    there = row < f.a.T;
    t = (int)(there ? row : f.a.T - 1);  // (rows past the end repeat the last one, and count for nothing)
    const T* p = (const T*)f.a.z + (int64_t)t * f.a.E;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int c = ((r << f.logL) + j) * V;
      if (c < f.a.E) {
        load_vec<T, V>(p + c, z[r]);
      } else {
#pragma unroll
        for (int v = 0; v < V; ++v) z[r][v] = NEG_INF;
      }
    }
    valid = there && (!f.a.valid || f.a.valid[t]);
  }
};

// A whole workgroup of W waves; ONE: the only one, which also writes the results.
// 32768 x 128 in fp32 8.2 us, 2.1 TB/s: as long again as the bytes take for the launch,
// the first loads and the sums at the end.
template <typename T, int V, int R, int W, bool ONE>
__global__ void __launch_bounds__(64 * W)
k_balance(Fwd f) {
  // rows in flight per lane: what 32 registers of logits allow
  constexpr int U = R * V <= 8 ? 4 : R * V <= 16 ? 2 : 1;
  __shared__ int hist[MAX_E];
  __shared__ float sums[W][MAX_E];
  __shared__ float zs[W];
  __shared__ int ns[W];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const BalanceArgs& a = f.a;
  const int L = 1 << f.logL, rows = 64 >> f.logL;
  float acc[R][V];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int v = 0; v < V; ++v) acc[r][v] = 0.f;
  float zsum = 0.f;
  int n = 0;
  const int64_t units = ((int64_t)a.T + rows - 1) / rows;
  const int64_t step = (int64_t)gridDim.x * W;
  Unit<T, V, R> x[U];
  int choice[U];
  int64_t u0 = (int64_t)blockIdx.x * W + w;
  auto load = [&] {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      x[i].load(f, min(u0 + i * step, units - 1), lane);
      if (u0 + i * step >= units) x[i].there = x[i].valid = false;
      const int k = lane & (L - 1);
      choice[i] = k < a.K ? a.idx[(int64_t)x[i].t * a.K + k] : -1;
    }
  };
  if (u0 < units) load();
  for (int e = tid; e < a.E; e += 64 * W) hist[e] = 0;
  lds_sync();  // (the loads stay under way)
  while (u0 < units) {
    float m[U], s[U], p[U][R][V];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      m[i] = NEG_INF;
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int v = 0; v < V; ++v) m[i] = max_nan(m[i], x[i].z[r][v]);
    }
    row_max(m, f.logL);
#pragma unroll
    for (int i = 0; i < U; ++i) {
      s[i] = 0.f;
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int v = 0; v < V; ++v) {
          p[i][r][v] = __expf(x[i].z[r][v] - m[i]);
          s[i] += p[i][r][v];
        }
    }
    row_sum(s, f.logL);
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const bool counting = x[i].valid && m[i] > NEG_INF;
      const float inv = 1.f / s[i];
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int v = 0; v < V; ++v) acc[r][v] = counting ? fmaf(p[i][r][v], inv, acc[r][v]) : acc[r][v];
      const float lse = counting ? m[i] + __logf(s[i]) : NEG_INF;
      const int j = lane & (L - 1);
      if (x[i].there && j == 0) a.lse[x[i].t] = lse;
      if (counting) {
        if (j == 0) {
          zsum = fmaf(lse, lse, zsum);
          ++n;
        }
        if ((unsigned)choice[i] < (unsigned)a.E) atomicAdd(&hist[choice[i]], 1);
        for (int k = j + L; k < a.K; k += L) {
          const int e = a.idx[(int64_t)x[i].t * a.K + k];
          if ((unsigned)e < (unsigned)a.E) atomicAdd(&hist[e], 1);
        }
      }
    }
    u0 += U * step;
    if (u0 < units) load();
  }

  // groups of the wave, then waves, in order
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int v = 0; v < V; ++v) {
      for (int s = L; s < 64; s <<= 1) acc[r][v] += __shfl_xor(acc[r][v], s, 64);
      const int c = ((r << f.logL) + (lane & (L - 1))) * V + v;
      if (lane < L && c < a.E) sums[w][c] = acc[r][v];
    }
  for (int s = 1; s < 64; s <<= 1) {
    zsum += __shfl_xor(zsum, s, 64);
    n += __shfl_xor(n, s, 64);
  }
  if (lane == 0) {
    zs[w] = zsum;
    ns[w] = n;
  }
  __syncthreads();
  zsum = 0.f;
  n = 0;
  for (int x = 0; x < W; ++x) {
    zsum += zs[x];
    n += ns[x];
  }
  if constexpr (ONE) {
    const float per = n > 0 ? 1.f / (float)n : 0.f;
    __shared__ float dots[W];
    float dot = 0.f;
    for (int e = tid; e < a.E; e += 64 * W) {
      float p = 0.f;
      for (int x = 0; x < W; ++x) p += sums[x][e];
      a.load[e] = p * per;
      a.counts[e] = hist[e];
      dot = fmaf((float)hist[e], p * per, dot);
    }
    dot = wave_sum(dot);
    if (lane == 0) dots[w] = dot;
    __syncthreads();
    if (tid == 0) {
      dot = 0.f;
      for (int x = 0; x < W; ++x) dot += dots[x];
      a.tokens[0] = n;
      a.loss[0] = dot * per * ((float)a.E / (float)a.K);
      a.loss[1] = zsum * per;
    }
  } else {
    uint32_t* line = f.line + (int64_t)blockIdx.x * line_words(a.E);
    for (int e = tid; e < a.E; e += 64 * W) {
      float p = 0.f;
      for (int x = 0; x < W; ++x) p += sums[x][e];
      line[e] = __float_as_uint(p);
      line[a.E + e] = (uint32_t)hist[e];
    }
    if (tid == 0) {
      line[2 * a.E] = __float_as_uint(zsum);
      line[2 * a.E + 1] = (uint32_t)n;
      if (blockIdx.x == 0) f.tail[TAIL_WORDS - 1] = 0;  // arrivals of the final launch
    }
  }
}

// The lines' sums: 16 columns per workgroup, 64 threads each, so that a thread's loads
// are in flight together (64 columns with 16 threads each took 6.7 us at E = 128, this 4.8);
// the workgroup that arrives last adds up the balance loss.
__global__ void __launch_bounds__(1024)
k_balance_final(Fwd f, int lines) {
  __shared__ float sp[16][FINAL_COLS];
  __shared__ int sc[16][FINAL_COLS];
  __shared__ float szw[16];
  __shared__ int snw[16];
  const BalanceArgs& a = f.a;
  const int tid = threadIdx.x, c = tid & 15, s = tid >> 4, w = tid >> 6, lane = tid & 63;
  const int e = blockIdx.x * FINAL_COLS + c, words = line_words(a.E);
  float p = 0.f, z = 0.f;
  int cnt = 0, n = 0;
  if (e < a.E) {
    const uint32_t* from = f.line + e;
    float pv[FWD_BLOCKS / 64];
    int cv[FWD_BLOCKS / 64];
#pragma unroll
    for (int i = 0; i < FWD_BLOCKS / 64; ++i) {
      const int g = min(s + 64 * i, lines - 1);
      pv[i] = __uint_as_float(from[(int64_t)g * words]);
      cv[i] = (int)from[(int64_t)g * words + a.E];
    }
#pragma unroll
    for (int i = 0; i < FWD_BLOCKS / 64; ++i) {
      p += s + 64 * i < lines ? pv[i] : 0.f;
      cnt += s + 64 * i < lines ? cv[i] : 0;
    }
  }
  if (tid < lines) {  // (at most 512 lines)
    z = __uint_as_float(f.line[(int64_t)tid * words + 2 * a.E]);
    n = (int)f.line[(int64_t)tid * words + 2 * a.E + 1];
  }
  for (int x = 16; x < 64; x <<= 1) {
    p += __shfl_xor(p, x, 64);
    cnt += __shfl_xor(cnt, x, 64);
  }
  for (int x = 1; x < 64; x <<= 1) {
    z += __shfl_xor(z, x, 64);
    n += __shfl_xor(n, x, 64);
  }
  if (lane < FINAL_COLS) {
    sp[w][c] = p;
    sc[w][c] = cnt;
  }
  if (lane == 0) {
    szw[w] = z;
    snw[w] = n;
  }
  __syncthreads();
  if (tid >= 16) return;
  p = z = 0.f;
  cnt = n = 0;
  for (int x = 0; x < 16; ++x) {
    p += sp[x][c];
    cnt += sc[x][c];
    z += szw[x];
    n += snw[x];
  }
  const float per = n > 0 ? 1.f / (float)n : 0.f;
  float dot = 0.f;
  if (e < a.E) {
    a.load[e] = p * per;
    a.counts[e] = cnt;
    dot = (float)cnt * (p * per);
  }
  dot = sum16(dot);
  if (c > 0) return;
  if (gridDim.x > 1) {
    __hip_atomic_store(&f.tail[blockIdx.x], __float_as_uint(dot), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (__hip_atomic_fetch_add(&f.tail[TAIL_WORDS - 1], 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) != gridDim.x - 1)
      return;
    dot = 0.f;
#pragma unroll 8
    for (unsigned x = 0; x < gridDim.x; ++x)
      dot += __uint_as_float(__hip_atomic_load(&f.tail[x], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
  }
  a.tokens[0] = n;
  a.loss[0] = dot * per * ((float)a.E / (float)a.K);
  a.loss[1] = z * per;
}

struct Bwd {
  BalanceBwdArgs a;
  int logL;
};

// One pass: p from the log-sum-exp that the forward call left, so a row needs one sum between
// lanes.  16384 x 256 in fp32 with the gates' share 11.3 us, 3.0 TB/s: the exponentials
// and the gates' words through LDS beside the bytes; 4099 x 60 in bf16 alone 3.6 us, a launch.
template <typename T, int V, int R, bool GATES>
__global__ void __launch_bounds__(256)
k_balance_bwd(Bwd f) {
  constexpr int U = R * V <= 8 ? 2 : 1;
  const BalanceBwdArgs& a = f.a;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int L = 1 << f.logL, rows = 64 >> f.logL, j = lane & (L - 1);
  __shared__ __attribute__((aligned(16))) int cols[GATES ? 4 * 64 * V * R : 1];
  volatile int* const own = cols + (GATES ? w * 64 * V * R : 0);  // this wave's rows, as bits
  const int64_t units = ((int64_t)a.T + rows - 1) / rows;
  const int64_t step = (int64_t)gridDim.x * 4;
  float z[U][R][V], lse[U], gt[U], dg[U];
  int t[U], id[U];
  bool there[U];
  int64_t u0 = (int64_t)blockIdx.x * 4 + w;
  auto load = [&] {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int64_t row = min(u0 + i * step, units - 1) * rows + (lane >> f.logL);
      there[i] = row < a.T && u0 + i * step < units;
      t[i] = (int)min(row, (int64_t)a.T - 1);
      const T* p = (const T*)a.z + (int64_t)t[i] * a.E;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int c = ((r << f.logL) + j) * V;
        if (c < a.E) {
          load_vec<T, V>(p + c, z[i][r]);
        } else {
#pragma unroll
          for (int v = 0; v < V; ++v) z[i][r][v] = NEG_INF;
        }
      }
      lse[i] = a.lse[t[i]];
      if constexpr (GATES) {
        const int64_t at = (int64_t)t[i] * a.K + min(j, a.K - 1);
        id[i] = a.idx[at];
        gt[i] = a.gate[at];
        dg[i] = a.d_gate[at];
      }
    }
  };
  if (u0 < units) load();
  if constexpr (GATES)
    for (int i = lane; i < 64 * V * R; i += 64) own[i] = 0;
  const int n = a.tokens[0];
  const float per = n > 0 ? 1.f / (float)n : 0.f;
  const float gb = a.d_loss[0] * (per * per * ((float)a.E / (float)a.K)), gz = a.d_loss[1] * 2.f * per;
  float cf[R][V];  // what the balance loss gains by a probability
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = ((r << f.logL) + j) * V + v;
      cf[r][v] = c < a.E ? gb * (float)a.counts[c] : 0.f;
    }
  while (u0 < units) {
    if constexpr (GATES) {
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (j >= a.K || (unsigned)id[i] >= (unsigned)a.E) {
          id[i] = -1;
          gt[i] = dg[i] = 0.f;
        }
    }
    bool counting[U], coarse[U], any = false;
    float p[U][R][V], s[U], inner[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      counting[i] = lse[i] != NEG_INF;
      // A large lse is too coarse a number for that (a row masked by its type's lowest
      // value throughout has lse = -3.4e38 and equal p): those rows normalise again.
      coarse[i] = counting[i] && fabsf(lse[i]) > 32.f;
      any |= coarse[i];
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int v = 0; v < V; ++v) p[i][r][v] = counting[i] ? __expf(z[i][r][v] - lse[i]) : 0.f;
    }
    const bool some = __any(any);
    if (some) {
      float m[U], sum[U];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        m[i] = NEG_INF;
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int v = 0; v < V; ++v) m[i] = max_nan(m[i], z[i][r][v]);
      }
      row_max(m, f.logL);
#pragma unroll
      for (int i = 0; i < U; ++i) {
        sum[i] = 0.f;
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int v = 0; v < V; ++v) sum[i] += __expf(z[i][r][v] - m[i]);
      }
      row_sum(sum, f.logL);
#pragma unroll
      for (int i = 0; i < U; ++i)
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int v = 0; v < V; ++v) p[i][r][v] = coarse[i] ? __expf(z[i][r][v] - m[i]) / sum[i] : p[i][r][v];
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      s[i] = 0.f;
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int v = 0; v < V; ++v) s[i] = fmaf(p[i][r][v], cf[r][v], s[i]);
    }
    row_sum(s, f.logL);
    if constexpr (GATES) {
#pragma unroll
      for (int i = 0; i < U; ++i) {
        // the choices lie across the row's lanes, L at a time
        inner[i] = gt[i] * dg[i];
        for (int k = j + L; k < a.K; k += L) {
          const int64_t at = (int64_t)t[i] * a.K + k;
          if ((unsigned)a.idx[at] < (unsigned)a.E) inner[i] = fmaf(a.gate[at], a.d_gate[at], inner[i]);
        }
      }
      row_sum(inner, f.logL);
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      // (with few tokens, gz lse may pass fp32's range where p gz lse does not: logits at their type's ends)
      const float far = gz * lse[i], add = counting[i] ? far - s[i] : 0.f;
      const bool huge = coarse[i] && fabsf(far) == __builtin_inff();
      if (some && __any(huge)) {
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int v = 0; v < V; ++v)
            p[i][r][v] = huge ? fmaf(p[i][r][v], cf[r][v] - s[i], p[i][r][v] * lse[i] * gz) : p[i][r][v] * (cf[r][v] + add);
      } else {
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int v = 0; v < V; ++v) p[i][r][v] *= cf[r][v] + add;
      }
      if constexpr (GATES) {
        // A row's choices are few and lie in one lane each: they go to their columns through
        // the row's words in LDS, zeros but for this.  (Every lane comparing its columns
        // with every choice took 190 instructions a row in place of 80.)
        // (volatile: other lanes of the wave read what one wrote, in order)
        volatile int* const row = own + (lane >> f.logL << f.logL) * (V * R);
        bool one = a.K <= L;
        if (one) {  // an expert chosen twice?  (whose sum's order a write would not keep)
          if (id[i] >= 0) row[id[i]] = j;
          one = !__any(id[i] >= 0 && row[max(id[i], 0)] != j);
        }
        if (one) {
          if (id[i] >= 0) row[id[i]] = __float_as_int(gt[i] * (dg[i] - inner[i]));
#pragma unroll
          for (int r = 0; r < R; ++r) {
            const volatile int* from = row + ((r << f.logL) + j) * V;
#pragma unroll
            for (int v = 0; v < V; ++v) p[i][r][v] += __int_as_float(from[v]);
          }
          if (id[i] >= 0) row[id[i]] = 0;
        } else {
          if (a.K <= L && id[i] >= 0) row[id[i]] = 0;
          for (int k = 0; k < a.K; ++k) {
            const int64_t at = (int64_t)t[i] * a.K + k;
            const int e = a.idx[at];
            const float val = (unsigned)e < (unsigned)a.E ? a.gate[at] * (a.d_gate[at] - inner[i]) : 0.f;
            const int to = (unsigned)e < (unsigned)a.E ? e - j * V : -1;  // its place among this lane's columns
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
              for (int v = 0; v < V; ++v) p[i][r][v] += to == (r << f.logL) * V + v ? val : 0.f;
          }
        }
      }
      if (there[i]) {
        T* o = (T*)a.dz + (int64_t)t[i] * a.E;
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const int c = ((r << f.logL) + j) * V;
          if (c < a.E) store_vec<T, V>(o + c, p[i][r]);
        }
      }
    }
    u0 += U * step;
    if (u0 < units) load();
  }
}

int log2_up(int n) {
  int l = 0;
  while ((1 << l) < n) ++l;
  return l;
}

// Columns per vector: 16 bytes, or 8, where the rows' stride and address keep them aligned.
int vec_width(int E, int dtype, const void* p, const void* q) {
  const uintptr_t at = (uintptr_t)p | (uintptr_t)q;
  if (dtype == MOE_F32) return E % 4 == 0 && at % 16 == 0 ? 4 : 1;
  return E % 8 == 0 && at % 16 == 0 ? 8 : E % 4 == 0 && at % 8 == 0 ? 4 : 1;
}

// f(type, V, R): the instance for a row of E columns; log2 of its lanes
template <typename T, int V, typename F>
hipError_t by_vectors(int E, F f) {
  const int nv = (E + V - 1) / V, log_l = std::min(log2_up(nv), 6), r = (nv + (1 << log_l) - 1) >> log_l;
  if (r <= 1) return f(std::integral_constant<int, V>(), std::integral_constant<int, 1>(), T(), log_l);
  if (r <= 2) return f(std::integral_constant<int, V>(), std::integral_constant<int, 2>(), T(), log_l);
  if constexpr (V < 8)
    if (r <= 4) return f(std::integral_constant<int, V>(), std::integral_constant<int, 4>(), T(), log_l);
  if constexpr (V == 1) {
    if (r <= 8) return f(std::integral_constant<int, V>(), std::integral_constant<int, 8>(), T(), log_l);
    return f(std::integral_constant<int, V>(), std::integral_constant<int, 16>(), T(), log_l);
  }
  return hipErrorInvalidValue;
}
template <typename F>
hipError_t by_shape(int E, int dtype, int V, F f) {
  if (dtype == MOE_F32) return V == 4 ? by_vectors<float, 4>(E, f) : by_vectors<float, 1>(E, f);
  return V == 8 ? by_vectors<bf16_t, 8>(E, f) : V == 4 ? by_vectors<bf16_t, 4>(E, f) : by_vectors<bf16_t, 1>(E, f);
}

// Few logits: one workgroup, one launch.  us a call, one workgroup / two launches: 512 x 32
// 7.3 / 9.3, 512 x 48 11.4 / 9.7, 2048 x 16 11.1 / 9.1, 1024 x 64 19.5 / 10.1.  Few choices too, as
// its lanes count them: 512 x 32 with K = 128 21.7 / 11.4, 16384 x 1 with K = 1024 14003 / 447.
bool one_block(int T, int E, int K) { return (int64_t)T * std::max(E, K) <= 16384; }

}  // namespace

size_t balance_ws_bytes(int T, int E, int K) {
  if (one_block(T, E, K)) return 0;
  return 4 * ((size_t)FWD_BLOCKS * line_words(E) + TAIL_WORDS);
}

hipError_t launch_balance(const BalanceArgs& a, hipStream_t st) {
  Fwd f{};
  f.a = a;
  f.line = (uint32_t*)a.ws;
  f.tail = f.line + (size_t)FWD_BLOCKS * line_words(a.E);
  return by_shape(a.E, a.dtype, vec_width(a.E, a.dtype, a.z, nullptr), [&](auto v, auto r, auto t, int log_l) {
    constexpr int V = decltype(v)::value, R = decltype(r)::value;
    typedef decltype(t) T;
    f.logL = log_l;
    if (one_block(a.T, a.E, a.K)) {
      hipLaunchKernelGGL((k_balance<T, V, R, 8, true>), dim3(1), dim3(512), 0, st, f);
      return hipGetLastError();
    }
    const int64_t units = ((int64_t)a.T + (64 >> log_l) - 1) / (64 >> log_l);
    const int grid = (int)std::min<int64_t>(FWD_BLOCKS, (units + 7) / 8);
    hipLaunchKernelGGL((k_balance<T, V, R, 8, false>), dim3(grid), dim3(512), 0, st, f);
    hipLaunchKernelGGL(k_balance_final, dim3((a.E + FINAL_COLS - 1) / FINAL_COLS), dim3(1024), 0, st, f, grid);
    return hipGetLastError();
  });
}

hipError_t launch_balance_bwd(const BalanceBwdArgs& a, hipStream_t st) {
  Bwd f{};
  f.a = a;
  return by_shape(a.E, a.dtype, vec_width(a.E, a.dtype, a.z, a.dz), [&](auto v, auto r, auto t, int log_l) {
    constexpr int V = decltype(v)::value, R = decltype(r)::value;
    typedef decltype(t) T;
    f.logL = log_l;
    const int64_t units = ((int64_t)a.T + (64 >> log_l) - 1) / (64 >> log_l);
    const unsigned grid = (unsigned)std::min<int64_t>(2048, (units + 3) / 4);
    if (a.idx) hipLaunchKernelGGL((k_balance_bwd<T, V, R, true>), dim3(grid), dim3(256), 0, st, f);
    else hipLaunchKernelGGL((k_balance_bwd<T, V, R, false>), dim3(grid), dim3(256), 0, st, f);
    return hipGetLastError();
  });
}

}  // namespace moe
