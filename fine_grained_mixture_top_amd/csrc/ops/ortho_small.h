// Orthogonalised updates whose smaller side m is at most 128: the m x m matrices of a
// step fit a CU's LDS, so a workgroup goes through whole steps without a launch
// between two products (ortho_kernels.hip has the formulas, ortho_gemm.h the numbers).
//
// The larger side is cut into chunks of 128.  A matrix in LDS is MP or 128 rows
// of K numbers (MP = 64 or 128, padded with zeros): two parts, K / 32 planes of lines of 128
// bytes (32 numbers' hi, then their lo); one part, K / 64 planes of 64 numbers.
// Eight waves, two along the rows of a product and four along its columns.
#pragma once

#include <type_traits>

#include "ortho_gemm.h"

namespace moe {
namespace ortho {

constexpr int CHUNK = 128;
constexpr int SMALL_THREADS = 512;

// line address of row r, plane c of a matrix of ROWS rows, and the slot of 16 bytes in it
template <int ROWS> __device__ __forceinline__ int line_at(int c, int r) { return (c * ROWS + r) * 128; }

// Where the lanes of a wave find a piece of 16 x 16 at row R, column K (multiples of
// 16, the same in all lanes) of a two-part matrix of ROWS rows: lane p + 16 h has four numbers
// of row p from column 4 h on; turned (see turn4), of row 4 h + p % 4 from column
// p / 4 * 4 on.  Slots of 16 bytes are xored with row % 8, the lo lies in the slot 4 further on:
// all that depends on the lane is one offset, xored with 32 (odd half of a plane) and 64.
template <int ROWS>
struct Place {
  uint32_t d, t;
  __device__ __forceinline__ explicit Place(int lane) {
    const int p = lane & 15, h = lane >> 4, tr = 4 * h + (p & 3);
    d = p * 128 + (((h >> 1) ^ (p & 7)) * 16) + (h & 1) * 8;
    t = tr * 128 + (((p >> 3) ^ (tr & 7)) * 16) + ((p >> 2) & 1) * 8;
  }
  static __device__ __forceinline__ uint32_t piece(int R, int K) { return ((K >> 5) * ROWS + R) * 128; }
  __device__ __forceinline__ uint32_t direct(int R, int K) const { return piece(R, K) + (d ^ (K & 16) * 2); }
  __device__ __forceinline__ uint32_t turned(int R, int K) const { return piece(R, K) + (t ^ (K & 16) * 2); }
};

__device__ __forceinline__ void split4(const f32x4_v v, f16x4_v& hi, f16x4_v& lo) {
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    _Float16 vh, vl;
    split(v[x], vh, vl);
    hi[x] = vh;
    lo[x] = vl;
  }
}
__device__ __forceinline__ void put(char* m, uint32_t at, const f16x4_v hi, const f16x4_v lo) {
  *reinterpret_cast<f16x4_v*>(m + at) = hi;
  *reinterpret_cast<f16x4_v*>(m + (at ^ 64)) = lo;
}
__device__ __forceinline__ f32x4_v get(const char* m, uint32_t at) {
  const f16x4_v hi = *reinterpret_cast<const f16x4_v*>(m + at), lo = *reinterpret_cast<const f16x4_v*>(m + (at ^ 64));
  f32x4_v v;
#pragma unroll
  for (int x = 0; x < 4; ++x) v[x] = (float)hi[x] + (float)lo[x];
  return v;
}

// A piece on or below the diagonal of a symmetric matrix, and its mirror.  (Products of
// matrices that commute are symmetric up to their rounding, and what is not would grow
// with the steps: 63 x 65, five steps, error 3.7e-2 with both halves as computed.)
template <int ROWS>
__device__ __forceinline__ void put_mirrored(char* m, int R, int K, const f32x4_v v, const Place<ROWS>& at, int lane) {
  f16x4_v hi, lo;
  split4(v, hi, lo);
  if (R == K) {  // (every number is written once: no order between the lanes' writes matters)
    put(m, at.direct(R, K), lower_mirrored(hi, lane), lower_mirrored(lo, lane));
    return;
  }
  put(m, at.direct(R, K), hi, lo);
  put(m, at.turned(K, R), turn4(hi, lane), turn4(lo, lane));
}

// acc = A B^T for the rows ra0 .. and rb0 .. of two matrices in LDS, over PLANES times 32
// of the reduction.  ROWS_FIRST: a lane holds, of row p of A, four neighbouring rows of B;
// else of row p of B four of A.
template <int FM, int FN, int RA, int RB, int PLANES, int PA, int PB, bool FINE, bool ROWS_FIRST>
__device__ __forceinline__ void product(f32x4_v (&acc)[FM][FN], const char* a, int ra0, const char* b, int rb0, int lane) {
  const int p = lane & 15, h = lane >> 4;
#pragma unroll
  for (int j = 0; j < FM; ++j)
#pragma unroll
    for (int i = 0; i < FN; ++i) acc[j][i] = f32x4_v{0.f, 0.f, 0.f, 0.f};
  auto mul = [](const f16x8_v x, const f16x8_v y, const f32x4_v c) {  // x rows of A, y rows of B
    return ROWS_FIRST ? __builtin_amdgcn_mfma_f32_16x16x32_f16(y, x, c, 0, 0, 0)
                      : __builtin_amdgcn_mfma_f32_16x16x32_f16(x, y, c, 0, 0, 0);
  };
  // (what depends on the lane: one offset, and it xored with 64)
  const uint32_t at = p * 128 + ((h ^ (p & 7)) * 16);
  a += ra0 * 128;
  b += rb0 * 128;
#pragma unroll
  for (int c = 0; c < PLANES; ++c) {
    f16x8_v fa[FM][PA], fb[FN][PB];
#pragma unroll
    for (int j = 0; j < FM; ++j)
#pragma unroll
      for (int x = 0; x < PA; ++x)
        fa[j][x] = *reinterpret_cast<const f16x8_v*>(a + (at ^ ((PA == 2 ? x : c & 1) * 64)) + line_at<RA>(PA == 2 ? c : c >> 1, 16 * j));
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
      for (int x = 0; x < PB; ++x)
        fb[i][x] = *reinterpret_cast<const f16x8_v*>(b + (at ^ ((PB == 2 ? x : c & 1) * 64)) + line_at<RB>(PB == 2 ? c : c >> 1, 16 * i));
#pragma unroll
    for (int j = 0; j < FM; ++j)
#pragma unroll
      for (int i = 0; i < FN; ++i) {
        if constexpr (FINE) {
          f32x4_v d = mul(fa[j][0], fb[i][1], f32x4_v{0.f, 0.f, 0.f, 0.f});
          d = mul(fa[j][1], fb[i][0], d);
          acc[j][i] = mul(fa[j][0], fb[i][0], acc[j][i]);
          acc[j][i] += d;
        } else {
          acc[j][i] = mul(fa[j][0], fb[i][0], acc[j][i]);
          if constexpr (PB == 2) acc[j][i] = mul(fa[j][0], fb[i][1], acc[j][i]);
          if constexpr (PA == 2) acc[j][i] = mul(fa[j][1], fb[i][0], acc[j][i]);
        }
      }
  }
}

// A chunk of the update on its way into LDS: gr x gc numbers (row stride ld) of GR x GC,
// zeros past them, 8 of a row per thread and task.  First all loads, then, times 2^ex, as a
// matrix in P parts; TURN: its columns become the rows.  A wave takes whole rows, or to
// turn them over 16 of them and 32 columns: 64 bytes of each (of whole rows, lanes would write
// to the same banks 16 times over; the product of 128 x 1000 with Q 10.8 -> 8.0 us).
template <typename T, int GR, int GC, bool TURN>
struct Chunk {
  static constexpr int V = 8, TASKS = GR * GC / V / SMALL_THREADS;
  float v[TASKS][V];
  static __device__ __forceinline__ void at(int t, int tid, int& r, int& c) {
    const int id = t * SMALL_THREADS + tid;
    if constexpr (TURN) {
      const int tile = id >> 6, lane = id & 63;
      r = tile / (GC / 32) * 16 + (lane & 15);
      c = tile % (GC / 32) * 32 + (lane >> 4) * 8;
    } else {
      r = id / (GC / V);
      c = id % (GC / V) * V;
    }
  }
  __device__ __forceinline__ void fetch(const T* g, int64_t ld, int gr, int gc, bool vec, int tid) {
#pragma unroll
    for (int t = 0; t < TASKS; ++t) {
      int r, c;
      at(t, tid, r, c);
      const T* p = g + r * ld + c;
      if (r < gr && c + V <= gc && vec) {
        T x[V];
        const uint4* u = reinterpret_cast<const uint4*>(p);
        uint4 w[sizeof(T) * V / 16];
#pragma unroll
        for (int y = 0; y < (int)(sizeof(T) * V / 16); ++y) w[y] = u[y];
        __builtin_memcpy(x, w, sizeof(x));
#pragma unroll
        for (int y = 0; y < V; ++y) v[t][y] = Elem<T>::to_f(x[y]);
      } else {
#pragma unroll
        for (int y = 0; y < V; ++y) v[t][y] = r < gr && c + y < gc ? Elem<T>::to_f(p[y]) : 0.f;
      }
    }
  }
  template <int P>
  __device__ __forceinline__ void place(char* m, int ex, int tid) const {
    constexpr int ROWS = TURN ? GC : GR;
#pragma unroll
    for (int t = 0; t < TASKS; ++t) {
      int r, c;
      at(t, tid, r, c);
      f16x8_v hi, lo;
#pragma unroll
      for (int y = 0; y < V; ++y) {
        _Float16 vh, vl;
        split(ldexpf(v[t][y], ex), vh, vl);
        hi[y] = vh;
        lo[y] = vl;
      }
      if constexpr (TURN) {
        // number k = r of the rows c .. c + 7
#pragma unroll
        for (int y = 0; y < V; ++y) {
          const int row = c + y, plane = P == 2 ? r >> 5 : r >> 6, slot = P == 2 ? (r & 31) >> 3 : (r & 63) >> 3;
          char* line = m + line_at<ROWS>(plane, row) + (r & 7) * 2;
          *reinterpret_cast<_Float16*>(line + ((slot ^ (row & 7)) * 16)) = hi[y];
          if constexpr (P == 2) *reinterpret_cast<_Float16*>(line + (((slot + 4) ^ (row & 7)) * 16)) = lo[y];
        }
      } else {
        const int plane = P == 2 ? c >> 5 : c >> 6, slot = P == 2 ? (c & 31) >> 3 : (c & 63) >> 3;
        char* line = m + line_at<ROWS>(plane, r);
        *reinterpret_cast<f16x8_v*>(line + ((slot ^ (r & 7)) * 16)) = hi;
        if constexpr (P == 2) *reinterpret_cast<f16x8_v*>(line + (((slot + 4) ^ (r & 7)) * 16)) = lo;
      }
    }
  }
};

// A call's sizes, for matrices e = blockIdx.y
struct Small {
  const void* g;         // the updates
  void* o;
  int M, N, m, k;        // m <= k, k = N or (tall) M
  int chunks, per;       // chunks of k; chunks of a slice
  int slices;            // of the sums
  bool vec;              // rows of g and o lie at multiples of 16 bytes
  const double* sums;    // partial sums of squares
  int parts;
  float eps;
  float* part;           // [matrices][slices][MP * MP], sums of X X^T as the threads hold them
  char* gram;            // [matrices] A, as it lies in LDS
  char* x;               // fp32 updates: X between two steps, two parts [matrices][chunks * 128][MP]
  char* q;               // bf16 updates: Q [matrices], as it lies in LDS
  float* back;           // see Convert
  float* on;
};

template <int MP> struct SmallCfg {
  static constexpr int FM = MP / 32, FN = MP / 64;   // pieces of a wave, of an MP x MP matrix
  static constexpr int XN = CHUNK / 64;              // of an MP x 128 one along its columns
  static constexpr int SQUARE = MP * MP * 4;         // bytes, two parts
  static constexpr int WIDE = MP * CHUNK * 4;
};

// a chunk of an update whose rows (TALL: columns) are X's, MP of them at most, as X, m
// rows of 128, or TRANSPOSED
template <typename T, int MP, bool TALL, bool TRANSPOSED>
struct UpdateChunk : Chunk<T, TALL ? CHUNK : MP, TALL ? MP : CHUNK, TALL != TRANSPOSED> {
  __device__ __forceinline__ void load(const Small& a, int e, int chunk, int tid) {
    const int k0 = chunk * CHUNK, left = min(CHUNK, a.k - k0);
    const T* g = (const T*)a.g + (int64_t)e * a.M * a.N;
    if constexpr (TALL) this->fetch(g + (int64_t)k0 * a.N, a.N, left, a.m, a.vec, tid);
    else this->fetch(g + k0, a.N, a.m, left, a.vec, tid);
  }
};

template <int MP>
__device__ __forceinline__ void put_square(char* to, const f32x4_v (&v)[SmallCfg<MP>::FM][SmallCfg<MP>::FN], int w, int lane) {
  using C = SmallCfg<MP>;
  const Place<MP> at(lane);
#pragma unroll
  for (int j = 0; j < C::FM; ++j)
#pragma unroll
    for (int i = 0; i < C::FN; ++i) {
      f16x4_v hi, lo;
      split4(v[j][i], hi, lo);
      put(to, at.direct((w >> 2) * (MP / 2) + 16 * j, (w & 3) * (MP / 4) + 16 * i), hi, lo);
    }
}

// v = diag I + beta a + alpha v, for the rows and columns below m
template <int MP>
__device__ __forceinline__ void polynomial(f32x4_v (&v)[SmallCfg<MP>::FM][SmallCfg<MP>::FN],
                                           const f32x4_v (&a)[SmallCfg<MP>::FM][SmallCfg<MP>::FN], float diag, float beta,
                                           float alpha, int m, int w, int lane) {
  using C = SmallCfg<MP>;
  const int r0 = (w >> 2) * (MP / 2) + (lane & 15), c0 = (w & 3) * (MP / 4) + 4 * (lane >> 4);
#pragma unroll
  for (int j = 0; j < C::FM; ++j)
#pragma unroll
    for (int i = 0; i < C::FN; ++i)
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int r = r0 + 16 * j, c = c0 + 16 * i + x;
        v[j][i][x] = fmaf(beta, a[j][i][x], alpha * v[j][i][x]) + (r == c && r < m ? diag : 0.f);
      }
}

// A wave's piece j, i lies above the diagonal: its mirror stands for it.
template <int MP>
__device__ __forceinline__ bool above(int j, int i, int w) {
  return (w >> 2) * (MP / 2) + 16 * j < (w & 3) * (MP / 4) + 16 * i;
}

// The lower half of a slice's sum, as the threads hold it
template <int MP>
__device__ __forceinline__ void write_part(float* part, int slices, int e, int slice,
                                           const f32x4_v (&v)[SmallCfg<MP>::FM][SmallCfg<MP>::FN], int w, int tid) {
  using C = SmallCfg<MP>;
  f32x4_v* p = reinterpret_cast<f32x4_v*>(part + ((int64_t)e * slices + slice) * (MP * MP)) + tid;
#pragma unroll
  for (int j = 0; j < C::FM; ++j)
#pragma unroll
    for (int i = 0; i < C::FN; ++i)
      if (!above<MP>(j, i, w)) p[(j * C::FN + i) * SMALL_THREADS] = v[j][i];
}
// A call's arguments where they lie: an index that the compiler does not know would
// have it copy them to every thread's own memory.
template <typename A>
__device__ __forceinline__ const __attribute__((address_space(4))) A* arguments() {
  return (const __attribute__((address_space(4))) A*)__builtin_amdgcn_kernarg_segment_ptr();
}

// A matrix's norm, from its partial sums (a wave, a lane each)
__device__ __forceinline__ double norm_of(const double* sums, int parts, int e) {
  static_assert(NORM_PARTS == 64, "a lane each");
  const int lane = threadIdx.x & 63;
  double s = lane < parts ? sums[(int64_t)e * NORM_PARTS + lane] : 0.0;
  for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o, 64);
  return sqrt(s);
}
// the power of two of a matrix's stored numbers, and X_0 over them (a matrix of zeros,
// as an expert without rows has it, stays one)
__device__ __forceinline__ int power_of(double norm) {
  return norm > 0.0 && norm < __builtin_inf() ? X_EXP - ilogb(norm) : 0;
}
__device__ __forceinline__ double first_of(double norm, double eps) {
  if (!(norm < __builtin_inf())) return __builtin_nan("");
  return norm == 0.0 ? 0.0 : scalbn(1.0 / (norm + eps), -power_of(norm));
}

// The factors that go with the groups of steps.  A matrix whose norm is far below eps
// starts far below 1 and grows with the steps; so that its parts keep their bits, the X
// between two groups carries a power of two of its own, from a bound of its norm that
// is followed through the steps:
//     back[i]    X of group i over its stored numbers (but for the exponent that all have)
//     on[i]      what the stored numbers of group i + 1 are of Q times those of group i
struct Factors {
  const double* sums;
  int parts;
  float eps;
  float* back;    // [groups][matrices]
  float* on;
  int groups;
  uint8_t steps[MAX_STEPS];  // of each group
  float coef[3 * MAX_STEPS];
};
// (one wave)
__device__ __forceinline__ void factors(const __attribute__((address_space(4))) Factors& a, double norm, int e, int nb) {
  const double first = first_of(norm, a.eps);
  const bool fine = norm < __builtin_inf();
  const float nan = __builtin_nanf("");
  const int lane = threadIdx.x & 63;
  if (lane == 0) a.back[e] = (float)first;
  if (lane == 0 && a.groups == 1) a.on[e] = (float)power_of(norm);  // (no next group: the update's exponent)
  float most = norm == 0.0 ? 0.f : (float)(norm / (norm + (double)a.eps));  // of |X|
  int t = 0, c = 0;
  for (int i = 0; i + 1 < a.groups; ++i) {
    for (int s = 0; s < a.steps[i]; ++s, c += 3) {
      const float v = most * (float)(lane + 1) * 0.015625f, l = v * v;
      float m = fabsf(v * fmaf(l, fmaf(l, a.coef[c + 2], a.coef[c + 1]), a.coef[c]));
      for (int o = 32; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor(m, o, 64));
      most = m;
    }
    const int next = most > 0.f && most < __builtin_inff() ? max(-60, min(120, -ilogbf(most))) : 0;
    const double f = i == 0 ? first : scalbn(1.0, -t);
    if (lane == 0) {
      a.on[i * nb + e] = fine ? (float)scalbn(f, next) : nan;
      a.back[(i + 1) * nb + e] = fine ? (float)scalbn(1.0, -next) : nan;
    }
    t = next;
  }
}

// ---- X X^T of the update, slice by slice (1536 x 128 in fp32 8.2 us: loads, then a
// product per chunk) ----
template <typename T, int P, int MP, bool TALL>
__global__ void __launch_bounds__(SMALL_THREADS, 2)
k_small_gram(Small a) {
  using C = SmallCfg<MP>;
  extern __shared__ __attribute__((aligned(1024))) char smem[];
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int e = blockIdx.y, slice = blockIdx.x;
  UpdateChunk<T, MP, TALL, false> update;
  update.load(a, e, slice * a.per, tid);
  const int ex = power_of(norm_of(a.sums, a.parts, e));
  f32x4_v tot[C::FM][C::FN], acc[C::FM][C::FN];
#pragma unroll
  for (int j = 0; j < C::FM; ++j)
#pragma unroll
    for (int i = 0; i < C::FN; ++i) tot[j][i] = f32x4_v{0.f, 0.f, 0.f, 0.f};
  const int last = min(a.chunks, (slice + 1) * a.per);
  for (int c = slice * a.per; c < last; ++c) {
    if (c > slice * a.per) {
      update.load(a, e, c, tid);
      __syncthreads();
    }
    update.template place<P>(smem, ex, tid);
    __syncthreads();
    product<C::FM, C::FN, MP, MP, CHUNK / 32, P, P, P == 2, true>(acc, smem, (w >> 2) * (MP / 2), smem, (w & 3) * (MP / 4), lane);
#pragma unroll
    for (int j = 0; j < C::FM; ++j)
#pragma unroll
      for (int i = 0; i < C::FN; ++i) tot[j][i] += acc[j][i];
  }
  write_part<MP>(a.part, a.slices, e, slice, tot, w, tid);
}

// ---- A from the slices' sums: a thread per float4, the slices in order.  (By the
// workgroups that use it, 12 slices took 6.5 us and their parts 3.2.)  The first time
// the last workgroup of a matrix makes its factors. ----
struct ReduceArgs {
  Small a;
  float gram;      // A over the sums (times back^2)
  int first;
  Factors f;
};
template <int MP>
__global__ void __launch_bounds__(256)
k_small_reduce(ReduceArgs) {
  using C = SmallCfg<MP>;
  const auto* g = arguments<ReduceArgs>();
  const int e = blockIdx.y, nb = gridDim.y, tid = threadIdx.x;
  constexpr int BLOCKS = MP * MP / 4 / 256;
  if (blockIdx.x == BLOCKS) {
    if (tid < 64) factors(g->f, norm_of(g->a.sums, g->a.parts, e), e, nb);
    return;
  }
  const int id = blockIdx.x * 256 + tid, lane = id & 63, w = id / 64 % 8, piece = id / SMALL_THREADS;
  const int j = piece / C::FN, i = piece % C::FN;
  if (above<MP>(j, i, w)) return;
  const int slices = g->a.slices;
  const f32x4_v* p = reinterpret_cast<const f32x4_v*>(g->a.part + (int64_t)e * slices * (MP * MP)) + id;
  f32x4_v v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 16
  for (int s = 0; s < slices; ++s) v += p[(int64_t)s * (MP * MP / 4)];
  const float f = g->first ? (float)first_of(norm_of(g->a.sums, g->a.parts, e), g->a.eps) : g->a.back[e];
  v *= g->gram * f * f;
  const int R = (w >> 2) * (MP / 2) + 16 * j, K = (w & 3) * (MP / 4) + 16 * i;
  char* to = g->a.gram + (int64_t)e * C::SQUARE;
  put_mirrored<MP>(to, R, K, v, Place<MP>(lane), lane);
}

// a matrix as it lies in LDS, from memory
template <int BYTES>
__device__ __forceinline__ void copy_in(char* to, const char* from, int tid) {
  constexpr int N = BYTES / 16 / SMALL_THREADS;
  uint4 v[N];
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = reinterpret_cast<const uint4*>(from)[i * SMALL_THREADS + tid];
#pragma unroll
  for (int i = 0; i < N; ++i) reinterpret_cast<uint4*>(to)[i * SMALL_THREADS + tid] = v[i];
}
// ... and as the waves hold its pieces
template <int MP>
__device__ __forceinline__ void get_square(f32x4_v (&v)[SmallCfg<MP>::FM][SmallCfg<MP>::FN], const char* m, int w, int lane) {
  using C = SmallCfg<MP>;
  const Place<MP> at(lane);
#pragma unroll
  for (int j = 0; j < C::FM; ++j)
#pragma unroll
    for (int i = 0; i < C::FN; ++i) v[j][i] = get(m, at.direct((w >> 2) * (MP / 2) + 16 * j, (w & 3) * (MP / 4) + 16 * i));
}

// A call's X = Q X, times alpha, at its place in o
template <typename O, int MP, bool TALL, bool ROWS_FIRST>
__device__ __forceinline__ void write_out(const Small& a, int e, int chunk,
                                          const f32x4_v (&y)[SmallCfg<MP>::FM][SmallCfg<MP>::XN], float alpha, int w, int lane) {
  using C = SmallCfg<MP>;
  static_assert(ROWS_FIRST != TALL, "four neighbours along o's rows");
  const int p = lane & 15, h = lane >> 4, k0 = chunk * CHUNK, left = min(CHUNK, a.k - k0);
  O* o = (O*)a.o + (int64_t)e * a.M * a.N + (TALL ? (int64_t)k0 * a.N : k0);
#pragma unroll
  for (int j = 0; j < C::FM; ++j)
#pragma unroll
    for (int i = 0; i < C::XN; ++i) {
      const int mr = (w >> 2) * (MP / 2) + 16 * j, kr = (w & 3) * 32 + 16 * i;
      const int r = TALL ? kr + p : mr + p, c = TALL ? mr + 4 * h : kr + 4 * h;
      const int rows = TALL ? left : a.m, cols = TALL ? a.m : left;
      if (r >= rows) continue;
      O* to = o + (int64_t)r * a.N + c;
      const f32x4_v v = y[j][i] * alpha;
      if (a.vec && c + 4 <= cols) {
        if constexpr (sizeof(O) == 2) *reinterpret_cast<uint2*>(to) = make_uint2(f2bf2(v[0], v[1]), f2bf2(v[2], v[3]));
        else *reinterpret_cast<float4*>(to) = make_float4(v[0], v[1], v[2], v[3]);
      } else {
#pragma unroll
        for (int x = 0; x < 4; ++x)
          if (c + x < cols) to[x] = Elem<O>::from_f(v[x]);
      }
    }
}

// ---- a step of fp32 updates: A from the slices' sums, P, and per chunk X = P X and the
// next sums (1536 x 128 12.8 us: three products one after the other, 4.5 us of matrix
// instructions, with their LDS writes and barriers between them) ----
struct StepArgs {
  Small a;
  float diag, beta, alpha;  // P = diag I + beta A + alpha A^2
  float x;                  // X over P X (times on[0], or at the end back[0])
};
template <int MP, bool TALL, bool FIRST, bool LAST>
__global__ void __launch_bounds__(SMALL_THREADS, 2)
k_small_step(StepArgs s) {
  using C = SmallCfg<MP>;
  extern __shared__ __attribute__((aligned(1024))) char smem[];
  char *const b0 = smem, *const b1 = smem + C::WIDE;  // (an MP x 128 matrix is the larger one)
  const Small& a = s.a;
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int e = blockIdx.y, slice = blockIdx.x;
  const int wr = (w >> 2) * (MP / 2), wc = (w & 3) * (MP / 4);
  f32x4_v A[C::FM][C::FN], P[C::FM][C::FN];
  copy_in<C::SQUARE>(b0, a.gram + (int64_t)e * C::SQUARE, tid);
  __syncthreads();
  get_square<MP>(A, b0, w, lane);
  product<C::FM, C::FN, MP, MP, MP / 32, 2, 2, true, true>(P, b0, wr, b0, wc, lane);
  polynomial<MP>(P, A, s.diag, s.beta, s.alpha, a.m, w, lane);
  put_square<MP>(b1, P, w, lane);

  int ex = 0;
  if constexpr (FIRST) ex = power_of(norm_of(a.sums, a.parts, e));
  const float ax = s.x * (LAST ? a.back[e] : a.on[e]);
  f32x4_v tot[C::FM][C::FN];
#pragma unroll
  for (int j = 0; j < C::FM; ++j)
#pragma unroll
    for (int i = 0; i < C::FN; ++i) tot[j][i] = f32x4_v{0.f, 0.f, 0.f, 0.f};
  const int end = min(a.chunks, (slice + 1) * a.per);
  for (int c = slice * a.per; c < end; ++c) {
    __syncthreads();  // everybody is done with b0
    char* image = a.x + ((int64_t)e * a.chunks + c) * C::WIDE;
    if constexpr (FIRST) {
      UpdateChunk<float, MP, TALL, true> update;
      update.load(a, e, c, tid);
      update.template place<2>(b0, ex, tid);
    } else {
      copy_in<C::WIDE>(b0, image, tid);
    }
    __syncthreads();
    f32x4_v y[C::FM][C::XN];
    product<C::FM, C::XN, MP, CHUNK, MP / 32, 2, 2, true, LAST && !TALL>(y, b1, wr, b0, (w & 3) * 32, lane);
    if constexpr (LAST) {
      write_out<float, MP, TALL, !TALL>(a, e, c, y, ax, w, lane);
    } else {
      __syncthreads();
      // X^T as it will be read next, and X over the old one; a lane holds, of row k = p,
      // four neighbouring m
      const Place<CHUNK> xt(lane);
      const Place<MP> x(lane);
#pragma unroll
      for (int j = 0; j < C::FM; ++j)
#pragma unroll
        for (int i = 0; i < C::XN; ++i) {
          const int k = (w & 3) * 32 + 16 * i, m = wr + 16 * j;
          f16x4_v hi, lo;
          split4(y[j][i] * ax, hi, lo);
          put(image, xt.direct(k, m), hi, lo);
          put(b0, x.turned(m, k), turn4(hi, lane), turn4(lo, lane));
        }
      __syncthreads();
      f32x4_v acc[C::FM][C::FN];
      product<C::FM, C::FN, MP, MP, CHUNK / 32, 2, 2, true, true>(acc, b0, wr, b0, wc, lane);
#pragma unroll
      for (int j = 0; j < C::FM; ++j)
#pragma unroll
        for (int i = 0; i < C::FN; ++i) tot[j][i] += acc[j][i];
    }
  }
  if constexpr (!LAST) write_part<MP>(a.part, a.slices, e, slice, tot, w, tid);
}

// ---- bf16 updates: all steps on the m x m matrices, a workgroup per update (five steps
// 16.5 us up to 64 rows, 56 up to 128: a chain of 14 products on one CU) ----
struct Recurrence {
  float diag, beta, alpha;  // P = diag I + beta A + alpha A^2
  float t, next, q;         // of T = P A, A = T P, Q = P Q
};
struct StepsArgs {
  Small a;
  int steps;
  Recurrence s[MAX_STEPS];
};
template <int MP>
__global__ void __launch_bounds__(SMALL_THREADS, 2)
k_small_steps(StepsArgs) {
  using C = SmallCfg<MP>;
  extern __shared__ __attribute__((aligned(1024))) char smem[];
  char *const b0 = smem, *const b1 = smem + C::SQUARE;
  const auto* g = arguments<StepsArgs>();
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), e = blockIdx.x;
  const int wr = (w >> 2) * (MP / 2), wc = (w & 3) * (MP / 4), m = g->a.m;
  f32x4_v A[C::FM][C::FN], P[C::FM][C::FN], Q[C::FM][C::FN];
  auto scaled = [&](f32x4_v (&v)[C::FM][C::FN], float by) {
#pragma unroll
    for (int j = 0; j < C::FM; ++j)
#pragma unroll
      for (int i = 0; i < C::FN; ++i) v[j][i] *= by;
  };
  auto times = [&](f32x4_v (&v)[C::FM][C::FN], const char* x, const char* y) {
    product<C::FM, C::FN, MP, MP, MP / 32, 2, 2, false, true>(v, x, wr, y, wc, lane);
  };
  const Place<MP> at(lane);
  auto put_lower = [&](char* to, const f32x4_v (&v)[C::FM][C::FN], float scale) {
#pragma unroll
    for (int j = 0; j < C::FM; ++j)
#pragma unroll
      for (int i = 0; i < C::FN; ++i)
        if (!above<MP>(j, i, w)) put_mirrored<MP>(to, wr + 16 * j, wc + 16 * i, v[j][i] * scale, at, lane);
  };
  copy_in<C::SQUARE>(b0, g->a.gram + (int64_t)e * C::SQUARE, tid);
  __syncthreads();
  get_square<MP>(A, b0, w, lane);
  const int steps = g->steps;
  for (int s = 0; s < steps; ++s) {
    const float diag = g->s[s].diag, beta = g->s[s].beta, alpha = g->s[s].alpha;
    if (s > 0) {
      __syncthreads();  // the buffers are free
      put_lower(b0, A, 1.f);
      __syncthreads();
    }
    times(P, b0, b0);
    polynomial<MP>(P, A, diag, beta, alpha, m, w, lane);
    put_lower(b1, P, 1.f);
    __syncthreads();
    if (s + 1 < steps) {
      times(A, b1, b0);  // T = P A
      __syncthreads();
      put_lower(b0, A, g->s[s].t);
      __syncthreads();
      times(A, b0, b1);  // the next A = T P
      scaled(A, g->s[s].next);
    }
    if (s == 0) {
#pragma unroll
      for (int j = 0; j < C::FM; ++j)
#pragma unroll
        for (int i = 0; i < C::FN; ++i) Q[j][i] = P[j][i];
    } else {
      __syncthreads();
      put_lower(b0, Q, 1.f);
      __syncthreads();
      times(Q, b1, b0);
      scaled(Q, g->s[s].q);
    }
  }
  put_lower(g->a.q + (int64_t)e * C::SQUARE, Q, 1.f);
}

// ---- o = Q X ----
struct ApplyArgs {
  Small a;
  float x;
};
template <int MP, bool TALL>
__global__ void __launch_bounds__(SMALL_THREADS, 2)
k_small_apply(ApplyArgs s) {
  using C = SmallCfg<MP>;
  extern __shared__ __attribute__((aligned(1024))) char smem[];
  char *const b0 = smem, *const b1 = smem + MP * CHUNK * 2;  // X^T in one part, Q
  const Small& a = s.a;
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int e = blockIdx.y;
  const int begin = blockIdx.x * a.per, end = min(a.chunks, begin + a.per);
  UpdateChunk<bf16_t, MP, TALL, true> update;
  update.load(a, e, begin, tid);
  const int ex = (int)a.on[e];
  const float ax = s.x * a.back[e];
  copy_in<C::SQUARE>(b1, a.q + (int64_t)e * C::SQUARE, tid);
  for (int c = begin; c < end; ++c) {
    if (c > begin) {
      update.load(a, e, c, tid);
      __syncthreads();
    }
    update.template place<1>(b0, ex, tid);
    __syncthreads();
    f32x4_v y[C::FM][C::XN];
    product<C::FM, C::XN, MP, CHUNK, MP / 32, 2, 1, false, !TALL>(y, b1, (w >> 2) * (MP / 2), b0, (w & 3) * 32, lane);
    write_out<bf16_t, MP, TALL, !TALL>(a, e, c, y, ax, w, lane);
  }
}

}  // namespace ortho
}  // namespace moe
