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

// over the L lanes that hold a row
__device__ __forceinline__ float row_sum(float v, int L) {
  for (int s = 1; s < L; s <<= 1) v += __shfl_xor(v, s, 64);
  return v;
}
__device__ __forceinline__ float row_max(float v, int L) {
  // a NaN has to come through: fmaxf drops it, so it is turned into +inf, whose
  // exponentials are NaN as well
  v = v != v ? __builtin_inff() : v;
  for (int s = 1; s < L; s <<= 1) v = fmaxf(v, __shfl_xor(v, s, 64));
  return v;
}

// lines of the workspace: E sums of probabilities, E counts, lse^2, tokens
__host__ __device__ inline int line_words(int E) { return 2 * E + 2; }
// (behind them the final launch's sums: 16 of counts * load, and an arrival count)
constexpr int TAIL_WORDS = 17;

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
  for (int e = tid; e < a.E; e += 64 * W) hist[e] = 0;
  __syncthreads();

  float acc[R][V];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int v = 0; v < V; ++v) acc[r][v] = 0.f;
  float zsum = 0.f;
  int n = 0;
  const int64_t units = ((int64_t)a.T + rows - 1) / rows;
  const int64_t step = (int64_t)gridDim.x * W;
  for (int64_t u0 = (int64_t)blockIdx.x * W + w; u0 < units; u0 += U * step) {
    Unit<T, V, R> x[U];
    int choice[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      x[i].load(f, min(u0 + i * step, units - 1), lane);
      if (u0 + i * step >= units) x[i].there = x[i].valid = false;
      const int k = lane & (L - 1);
      choice[i] = k < a.K ? a.idx[(int64_t)x[i].t * a.K + k] : -1;
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      float m = NEG_INF;
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int v = 0; v < V; ++v) m = (x[i].z[r][v] != x[i].z[r][v]) ? __builtin_inff() : fmaxf(m, x[i].z[r][v]);
      m = row_max(m, L);
      const bool counting = x[i].valid && m > NEG_INF;
      float s = 0.f, p[R][V];
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int v = 0; v < V; ++v) {
          p[r][v] = __expf(x[i].z[r][v] - m);
          s += p[r][v];
        }
      s = row_sum(s, L);
      const float inv = 1.f / s;
      if (counting) {
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int v = 0; v < V; ++v) acc[r][v] = fmaf(p[r][v], inv, acc[r][v]);
      }
      const float lse = counting ? m + __logf(s) : NEG_INF;
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

// The lines' sums: 64 columns per workgroup, 16 threads each; the workgroup that
// arrives last adds up the balance loss.
__global__ void __launch_bounds__(1024)
k_balance_final(Fwd f, int lines) {
  __shared__ float sp[16][64];
  __shared__ int sc[16][64];
  __shared__ float szw[16];
  __shared__ int snw[16];
  __shared__ bool last;
  const BalanceArgs& a = f.a;
  const int tid = threadIdx.x, c = tid & 63, s = tid >> 6;
  const int e = blockIdx.x * 64 + c, words = line_words(a.E);
  float p = 0.f, z = 0.f;
  int cnt = 0, n = 0;
  if (e < a.E) {
#pragma unroll 8
    for (int g = s; g < lines; g += 16) {
      p += __uint_as_float(f.line[(int64_t)g * words + e]);
      cnt += (int)f.line[(int64_t)g * words + a.E + e];
    }
  }
  if (tid < lines) {  // (at most 512 lines)
    z = __uint_as_float(f.line[(int64_t)tid * words + 2 * a.E]);
    n = (int)f.line[(int64_t)tid * words + 2 * a.E + 1];
  }
  sp[s][c] = p;
  sc[s][c] = cnt;
  for (int x = 1; x < 64; x <<= 1) {
    z += __shfl_xor(z, x, 64);
    n += __shfl_xor(n, x, 64);
  }
  if (c == 0) {
    szw[s] = z;
    snw[s] = n;
  }
  __syncthreads();
  if (s > 0) return;
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
  dot = wave_sum(dot);
  const float scale = per * ((float)a.E / (float)a.K);
  if (c == 0) {
    last = true;
    if (gridDim.x > 1) {
      __hip_atomic_store(&f.tail[blockIdx.x], __float_as_uint(dot), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      last = __hip_atomic_fetch_add(&f.tail[TAIL_WORDS - 1], 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) ==
             gridDim.x - 1;
      if (last) {
        dot = 0.f;
        for (unsigned x = 0; x < gridDim.x; ++x)
          dot += __uint_as_float(__hip_atomic_load(&f.tail[x], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
      }
    }
    if (last) {
      a.tokens[0] = n;
      a.loss[0] = dot * scale;
      a.loss[1] = z * per;
    }
  }
}

struct Bwd {
  BalanceBwdArgs a;
  int logL;
};

template <typename T, int V, int R, bool GATES>
__global__ void __launch_bounds__(256)
k_balance_bwd(Bwd f) {
  constexpr int U = R * V <= 8 ? 2 : 1;
  const BalanceBwdArgs& a = f.a;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int L = 1 << f.logL, rows = 64 >> f.logL, j = lane & (L - 1), base = lane & ~(L - 1);
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
  const int64_t units = ((int64_t)a.T + rows - 1) / rows;
  const int64_t step = (int64_t)gridDim.x * 4;
  for (int64_t u0 = (int64_t)blockIdx.x * 4 + w; u0 < units; u0 += U * step) {
    float z[U][R][V], lse[U];
    int t[U], id[U];
    float gt[U], dg[U];
    bool there[U];
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
        if (j >= a.K || (unsigned)id[i] >= (unsigned)a.E) {
          id[i] = -1;
          gt[i] = dg[i] = 0.f;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const bool counting = lse[i] != NEG_INF;
      float p[R][V], s = 0.f;
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int v = 0; v < V; ++v) p[r][v] = counting ? __expf(z[i][r][v] - lse[i]) : 0.f;
      // A large lse is too coarse a number for that (a row masked by its type's lowest
      // value throughout has lse = -3.4e38 and equal p): those rows normalise again.
      const bool coarse = counting && fabsf(lse[i]) > 32.f;
      if (__any(coarse)) {
        float m = NEG_INF, q[R][V], sum = 0.f;
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int v = 0; v < V; ++v) m = fmaxf(m, z[i][r][v]);
        m = row_max(m, L);
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int v = 0; v < V; ++v) {
            q[r][v] = __expf(z[i][r][v] - m);
            sum += q[r][v];
          }
        sum = row_sum(sum, L);
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int v = 0; v < V; ++v) p[r][v] = coarse ? q[r][v] / sum : p[r][v];
      }
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int v = 0; v < V; ++v) s = fmaf(p[r][v], cf[r][v], s);
      s = row_sum(s, L);
      const float add = counting ? gz * lse[i] - s : 0.f;
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int v = 0; v < V; ++v) p[r][v] *= cf[r][v] + add;
      if constexpr (GATES) {
        // the choices lie across the row's lanes, L at a time
        float inner = gt[i] * dg[i];
        for (int k = j + L; k < a.K; k += L) {
          const int64_t at = (int64_t)t[i] * a.K + k;
          if ((unsigned)a.idx[at] < (unsigned)a.E) inner = fmaf(a.gate[at], a.d_gate[at], inner);
        }
        inner = row_sum(inner, L);
        for (int k0 = 0; k0 < a.K; k0 += L) {
          int e = id[i];
          float g = gt[i], d = dg[i];
          if (k0 > 0) {
            const int64_t at = (int64_t)t[i] * a.K + k0 + j;
            e = k0 + j < a.K ? a.idx[at] : -1;
            g = d = 0.f;
            if ((unsigned)e < (unsigned)a.E) {
              g = a.gate[at];
              d = a.d_gate[at];
            }
          }
          const float val = g * (d - inner);
          const int most = min(L, a.K - k0);
          for (int k = 0; k < most; ++k) {
            const int ek = __shfl(e, base + k, 64);
            const float vk = __shfl(val, base + k, 64);
            const int at = ek - j * V;  // its place among this lane's columns
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
              for (int v = 0; v < V; ++v)
                if (at == (r << f.logL) * V + v) p[r][v] += vk;
          }
        }
      }
      if (there[i]) {
        T* o = (T*)a.dz + (int64_t)t[i] * a.E;
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const int c = ((r << f.logL) + j) * V;
          if (c < a.E) store_vec<T, V>(o + c, p[r]);
        }
      }
    }
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

// Few logits: one workgroup, one launch.
bool one_block(int T, int E) { return (int64_t)T * E <= 16384; }

}  // namespace

size_t balance_ws_bytes(int T, int E) {
  if (one_block(T, E)) return 0;
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
    if (one_block(a.T, a.E)) {
      hipLaunchKernelGGL((k_balance<T, V, R, 8, true>), dim3(1), dim3(512), 0, st, f);
      return hipGetLastError();
    }
    const int64_t units = ((int64_t)a.T + (64 >> log_l) - 1) / (64 >> log_l);
    const int grid = (int)std::min<int64_t>(FWD_BLOCKS, (units + 3) / 4);
    hipLaunchKernelGGL((k_balance<T, V, R, 4, false>), dim3(grid), dim3(256), 0, st, f);
    hipLaunchKernelGGL(k_balance_final, dim3((a.E + 63) / 64), dim3(1024), 0, st, f, grid);
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
