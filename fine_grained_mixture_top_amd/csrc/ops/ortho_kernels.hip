// An update orthogonalised by Newton-Schulz products (include/moe_step_ops.h:
// moe_orthogonalize).
//
// X is the update, m x k with m <= k (transposed where it is tall), over its
// Frobenius norm; a step is X <- (a I + b A + c A^2) X with A = X X^T.  A, its
// polynomials P = a I + b A + c A^2 and their products commute and are symmetric, so
// steps can run on them alone:
//     A_1 = P A P,   Q = P_n ... P_1,   X_n = Q X_0
// which needs one product with the m x k matrix for a group of steps, and half the
// tiles of every product but that one.
//   Rounding.  A singular value s enters A as s^2 beside the largest one's 1, so what A lost
// (2^-23 of an element in its two parts, and its sums' roundings) stands beside s^2, grows by
// a^2 with every step that A goes through, and each P loses |b| / a of it: see group_steps.
// Error of bf16 results before their rounding, which is 1.7e-3 of their norm, five steps with
// a = 3.4445 in one group, spectra gaussian / 1/i / one direction beside 3e-4:
//     160 x 160     2e-5 / 1e-4 / 3.4e-4      129 x 50000   1e-6 / 8e-5 / 5.0e-4
//     256 x 1536    2e-6 / 1.4e-4 / 3.0e-4    16 x 1000     3e-6 / 2e-6 / 7.0e-4
//     2048 x 2048   1e-5 / 1.7e-4 / 2.1e-4    8 x 8000      1e-6 / 1e-6 / 9.1e-4
// fp32 results with one step a group 1e-6 / 3e-6 / 2.6e-5 at most (products in fp32 throughout: 3e-6 /
// 4e-6 / 4e-5).  So fp32 results take one step a group, and bf16 results as many as add less than
// their rounding.
#include <algorithm>
#include <cmath>

#include "launch_util.h"
#include "ortho_gemm.h"
#include "ortho_small.h"
#include "step_launch.h"

namespace moe {

namespace {

using namespace ortho;

// ---- sum of squares, in 64 bits: no scaling is needed for any finite input.  One reading:
// 64 x 2048 x 2048 in bf16 127 us, 4.2 TB/s ----
template <typename T, int V>
__global__ void __launch_bounds__(256)
k_ortho_norm(const T* g, int64_t elems, int parts, double* sums) {
  const int e = blockIdx.y;
  const T* p = g + (int64_t)e * elems;
  double s = 0.0;
  const int64_t vecs = elems / V, step = (int64_t)parts * 256;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < vecs; i += step) {
    T v[V];
    if constexpr (V > 1) {
      const uint4 u = reinterpret_cast<const uint4*>(p)[i];
      __builtin_memcpy(v, &u, 16);
    } else {
      v[0] = p[i];
    }
#pragma unroll
    for (int x = 0; x < V; ++x) {
      const double d = (double)Elem<T>::to_f(v[x]);
      s = fma(d, d, s);
    }
  }
  for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o, 64);
  __shared__ double ws[4];
  if ((threadIdx.x & 63) == 0) ws[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) sums[(int64_t)e * NORM_PARTS + blockIdx.x] = (ws[0] + ws[1]) + (ws[2] + ws[3]);
}

// The update as fp16 parts in both layouts, times a power of two that brings its norm
// to 2^13 .. 2^14.  Bytes bound it: 64 x 2048 x 2048 in bf16 519 us, 3.1 TB/s read and
// written (pieces of 128 bytes a row).
struct Convert {
  const void* g;
  int M, N;
  const double* sums;
  int parts;      // partial sums of a matrix
  double eps;
  char* same;     // rows of g
  char* trans;    // columns of g
  int64_t ssame, strans;
  float* back;    // [groups][gridDim.y]
};

// (a launch of its own, for more than one group)
__global__ void __launch_bounds__(64)
k_ortho_factors(Factors) {
  const auto* a = arguments<Factors>();
  factors(*a, norm_of(a->sums, a->parts, blockIdx.x), blockIdx.x, gridDim.x);
}

template <typename T, int P>
__global__ void __launch_bounds__(256)
k_ortho_convert(Convert a) {
  __shared__ float tile[64][65];
  // (both sides may have more tiles than a grid's second axis)
  const int wide = (a.N + 63) / 64, e = blockIdx.y, tid = threadIdx.x;
  const int r0 = (int)(blockIdx.x / (unsigned)wide) * 64, c0 = (int)(blockIdx.x % (unsigned)wide) * 64;
  const double norm = norm_of(a.sums, a.parts, e);
  const int ex = power_of(norm);
  if (blockIdx.x == 0 && tid == 0) a.back[e] = (float)first_of(norm, a.eps);
  const T* g = (const T*)a.g + (int64_t)e * a.M * a.N;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int r = i * 4 + (tid >> 6), c = tid & 63;
    tile[r][c] = r0 + r < a.M && c0 + c < a.N
                     ? ldexpf(Elem<T>::to_f(g[(int64_t)(r0 + r) * a.N + c0 + c]), ex) : 0.f;
  }
  __syncthreads();
  const int line = tid >> 3, x0 = (tid & 7) * 8;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const int r = half * 32 + line;
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      if (side == 0 ? r0 + r >= a.M : c0 + r >= a.N) continue;
      f16x8_v hi, lo;
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        _Float16 vh, vl;
        split(side == 0 ? tile[r][x0 + x] : tile[x0 + x][r], vh, vl);
        hi[x] = vh;
        lo[x] = vl;
      }
      const int row = side == 0 ? r0 + r : c0 + r, col = (side == 0 ? c0 : r0) + x0;
      char* to = side == 0 ? a.same + e * a.ssame + row * pitch(a.N, P) : a.trans + e * a.strans + row * pitch(a.M, P);
      if constexpr (P == 1) {
        *reinterpret_cast<f16x8_v*>(to + col * 2) = hi;
      } else {
        *reinterpret_cast<f16x8_v*>(to + at2(col)) = hi;
        *reinterpret_cast<f16x8_v*>(to + at2(col) + 64) = lo;
      }
    }
  }
}

// ---- launches ----
template <int BM, int BN, int WM, int WN, int BUFS, int PA, int PB, bool FINE, Epi EPI, typename O>
hipError_t launch_gemm(const Args& a, int64_t tiles, hipStream_t st) {
  using C = Cfg<BM, BN, WM, WN, BUFS, PA, PB>;
  auto* k = k_ortho_gemm<BM, BN, WM, WN, BUFS, PA, PB, FINE, EPI, O>;
  static std::atomic<uint64_t> done{0};
  const hipError_t e = allow_lds(k, C::SMEM, device(), done);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(k, dim3((unsigned)((tiles + 7) / 8 * 8)), dim3(C::NTH), C::SMEM, st, a);
  return hipGetLastError();
}

// Tiles.  Few of them: a stage takes as long as its loads, so tiles of 64 x 64 with three
// stages ahead; while 128 x 128 fill no CU twice, one of those with three stages ahead for
// each; else two of them with one stage ahead; many: 256 x 256, which load least.  128 x 128
// have eight waves (four instead, two stage buffers: 24 x 720 x 1040 849 us in place of 809, in
// fp32 1076 in place of 1035).  A whole call, us, with one kind throughout, and by this rule:
//                            64 x 64   128, 3 ahead   128, 1 ahead   256    rule
//   bf16   1 x 512 x 512         158            258            255   648    158
//          2 x 1024 x 1024       309            412            414  1088    295
//          4 x 1024 x 1024       509            487            461  1096    458
//          64 x 256 x 1536       330            321            308   555    307
//          128 x 256 x 1536      596            625            533   702    534
//          24 x 720 x 1040      1021            919            777  1146    773
//          32 x 1024 x 1024     3148           2764           2477  2715   2479
//          64 x 2048 x 2048                   35009          30439 28395  28336
//          342 x 300 x 4000                    4056           3544  4661   4532
//   fp32   1 x 512 x 512         159            252            251          159
//          4 x 1024 x 1024       503            435            430          435
//          1 x 2048 x 2048       877            733            741          733
//          64 x 256 x 1536       841            759            815          724
//          24 x 720 x 1040      1370           1161           1014         1020
//          64 x 2048 x 2048                   35412          30616        30702
// (The rule counts tiles, not what of them lies outside: 300 rows fill 256 x 256 worst.  FINE's
// sums of two kinds do not fit the registers with 256 x 256.)
constexpr int LONG = 6;  // sides from which on bf16 X X^T is summed in pieces throughout
template <int PA, int PB, bool FINE, Epi EPI, typename O>
hipError_t gemm_by_size(const Args& a, hipStream_t st) {
  auto tiles = [&](int B) {
    const int64_t mt = div_up(a.ra, B), nt = div_up(a.rb, B);
    return a.batch * a.jobs * (EPI == SYM ? mt * (mt + 1) / 2 : mt * nt);
  };
  const int64_t t64 = tiles(64);
  if constexpr (!FINE) {
    // (not for X X^T whose sums are long: see lost)
    const bool pieces = PA == 1 && PB == 1 && (int64_t)a.stages * 64 > LONG * (int64_t)a.ra;
    const int64_t t256 = tiles(256);
    if (t256 >= 1024 && !pieces) return launch_gemm<256, 256, 2, 4, 2, PA, PB, FINE, EPI, O>(a, t256, st);
  }
  const int64_t t128 = tiles(128), cus = cu_count(device());
  if (t64 <= 2 * cus) return launch_gemm<64, 64, 2, 2, 4, PA, PB, FINE, EPI, O>(a, t64, st);
  if (t128 <= cus) return launch_gemm<128, 128, 4, 2, 4, PA, PB, FINE, EPI, O>(a, t128, st);
  return launch_gemm<128, 128, 4, 2, 2, PA, PB, FINE, EPI, O>(a, t128, st);
}

// (fp32 updates are two parts throughout, and FINE)
template <int PA, int PB, Epi EPI, typename O = bf16_t>
hipError_t gemm(const Args& a, bool fine, hipStream_t st) {
  if constexpr (PA == 2 && PB == 2) {
    if (fine) return gemm_by_size<PA, PB, true, EPI, float>(a, st);
  }
  return gemm_by_size<PA, PB, false, EPI, O>(a, st);
}

// What the singular values and with them the matrices of a step can be: samples of
// the spectrum followed through the steps.
struct Spectrum {
  static constexpr int N = 97;
  double s[N], l[N], q[N];
  Spectrum() {
    for (int i = 0; i < N; ++i) s[i] = (double)i / (N - 1);  // norms of X_0 are at most 1
  }
  void begin() {
    for (int i = 0; i < N; ++i) {
      l[i] = s[i] * s[i];
      q[i] = 1.0;
    }
  }
  // largest |P|, |P A|, |P A P|, |Q| of a step
  void step(const float* c, double* p, double* t, double* a, double* qm) {
    *p = *t = *a = *qm = 0.0;
    for (int i = 0; i < N; ++i) {
      const double v = c[0] + l[i] * (c[1] + l[i] * c[2]);
      *p = std::max(*p, std::fabs(v));
      *t = std::max(*t, std::fabs(v * l[i]));
      l[i] *= v * v;
      q[i] *= v;
      *a = std::max(*a, std::fabs(l[i]));
      *qm = std::max(*qm, std::fabs(q[i]));
    }
  }
  void end() {
    for (int i = 0; i < N; ++i) s[i] = std::fabs(s[i] * q[i]);
  }
};

// The exponent that brings numbers up to `most` below 2^13, four times below what
// fp16 holds (the samples' gaps, and rounding).
int exponent_for(double most) {
  if (!(most > 0.0) || !std::isfinite(most)) return 0;
  return std::max(-30, std::min(30, 13 - std::ilogb(most) - 1));
}

struct Sizes {
  int m, k, parts, nb;           // parts of the update; matrices at a time
  int64_t sx, sxt, sm;           // bytes of X, its transpose (two parts), an m x m matrix
  int groups, mats;              // m x m matrices
  int64_t x0, xt0, x1, xt1, mat, f, sums, total;
};

// What A = X X^T loses beside a small direction's share, in root mean square over m directions: an
// element is off by 2^-25 sqrt(4 + sums) of itself, 2^-24 in its two parts and half a step for each
// rounding of its sum (`sums`: their mean square, n roundings of a sum that grows evenly being n / 3);
// elements of one large direction over all rows are about 1 / m.
double lost(int m, double sums) { return std::ldexp(std::sqrt((4.0 + sums) * (m - 1)) / m, -25); }
// ... products of any size: one sum over k, rounded once for eight products, or pieces of 512
double lost(const OrthoArgs& a) {
  const int m = std::min(a.M, a.N), k = std::max(a.M, a.N);
  const double pieces = std::ceil(k / 512.0);
  return lost(m, k <= (int64_t)LONG * m ? k / 24.0 : (64.0 / pieces + pieces) / 3.0);
}

// How many steps from step s on form a group: those whose P lose at most 1.5e-3 of the result
// together, when a direction far above the others hides these from A.  X X^T of
// long sides is summed in pieces for that: 129 x 50000 in one sum loses 3.4e-3, or takes 4 + 1
// steps and 788 us; in pieces 5.0e-4, 337 us.)
int group_steps(const OrthoArgs& a, int s, double lost) {
  if (a.dtype == MOE_F32) return 1;
  double grown = 0.0, power = 1.0;  // of A's error; of a small direction
  int n = 0;
  while (s + n < a.steps) {
    const float* c = a.coef + 3 * (s + n);
    const double up = std::max(1.0, std::fabs((double)c[0]));
    // (without a b, P loses by c once A has grown)
    grown += std::max(std::fabs((double)c[1]), std::fabs((double)c[2])) / up * power * power;
    power *= up;
    // (and Q, which holds a small direction's growth beside the large ones' near 1, keeps its bits)
    if (n > 0 && (lost * grown > 1.5e-3 || power > 512.0)) break;
    ++n;
  }
  return n;
}

Sizes sizes(const OrthoArgs& a) {
  Sizes z{};
  z.m = std::min(a.M, a.N);
  z.k = std::max(a.M, a.N);
  z.parts = a.dtype == MOE_F32 ? 2 : 1;
  // Matrices at a time: enough for nine rounds of 256 x 256 tiles over 256 CUs (whatever the long
  // side: X X^T has no more tiles for it)
  const int64_t mt = div_up(z.m, 256), tiles = mt * (mt + 1) / 2;
  const int64_t most = std::min<int64_t>(a.E, div_up(2304, tiles));
  z.nb = (int)div_up(a.E, div_up(a.E, most));
  for (int s = 0; s < a.steps; s += group_steps(a, s, lost(a))) ++z.groups;
  z.sx = z.m * pitch(z.k, 2);
  z.sxt = z.k * pitch(z.m, 2);
  z.sm = z.m * pitch(z.m, 2);
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t here = at;
    at += (bytes + 255) / 256 * 256;
    return here;
  };
  z.x0 = take(z.nb * z.sx * z.parts / 2);
  z.xt0 = take(z.nb * z.sxt * z.parts / 2);
  if (z.groups > 1) {
    // X in two parts for the groups after the first, which one-part input leaves no place for
    const int n = z.parts == 1 && z.groups > 2 ? 2 : 1;
    z.x1 = take(z.nb * z.sx * n);
    z.xt1 = take(z.nb * z.sxt * n);
  }
  // A and P; with more steps in a group T = P A and Q, the old one and the next
  z.mats = z.groups == a.steps ? 2 : 5;
  z.mat = take(z.mats * z.nb * z.sm);
  z.f = take(4 * z.nb * 2 * z.groups);
  z.sums = take(8 * (int64_t)z.nb * NORM_PARTS);
  z.total = at;
  return z;
}

Factors factors_of(const OrthoArgs& a, int groups, int nb, const double* sums, int parts, float* back) {
  Factors f{};
  f.sums = sums; f.parts = parts; f.eps = a.eps;
  f.back = back; f.on = back + groups * nb; f.groups = groups;
  for (int s = 0, i = 0; s < a.steps; s += f.steps[i], ++i) f.steps[i] = (uint8_t)(groups == 1 ? a.steps : group_steps(a, s, lost(a)));
  std::copy(a.coef, a.coef + 3 * a.steps, f.coef);
  return f;
}

// the sums of squares of nb updates; returns their number of parts
template <typename T>
int launch_norm(const T* g, int64_t elems, int nb, double* sums, hipStream_t st) {
  constexpr int V = 16 / sizeof(T);
  const bool vec = elems % V == 0 && ((uintptr_t)g & 15) == 0;
  const int parts = (int)std::min<int64_t>(NORM_PARTS, div_up(elems, 256 * 16));
  if (vec) hipLaunchKernelGGL((k_ortho_norm<T, V>), dim3(parts, nb), dim3(256), 0, st, g, elems, parts, sums);
  else hipLaunchKernelGGL((k_ortho_norm<T, 1>), dim3(parts, nb), dim3(256), 0, st, g, elems, parts, sums);
  return parts;
}

template <typename T>
hipError_t prepare(const OrthoArgs& a, const Sizes& z, int e0, int nb, hipStream_t st) {
  char* ws = (char*)a.ws;
  const int64_t elems = (int64_t)a.M * a.N;
  const T* g = (const T*)a.g + e0 * elems;
  double* sums = (double*)(ws + z.sums);
  const int parts = launch_norm(g, elems, nb, sums, st);
  const bool tall = a.M > a.N;
  constexpr int P = sizeof(T) == 4 ? 2 : 1;
  Convert c{};
  c.g = g; c.M = a.M; c.N = a.N; c.sums = sums; c.parts = parts; c.eps = a.eps;
  char *x = ws + z.x0, *xt = ws + z.xt0;
  const int64_t sx = z.sx * P / 2, sxt = z.sxt * P / 2;
  c.same = tall ? xt : x;
  c.trans = tall ? x : xt;
  c.ssame = tall ? sxt : sx;
  c.strans = tall ? sx : sxt;
  c.back = (float*)(ws + z.f);
  if (z.groups > 1) {
    const Factors f = factors_of(a, z.groups, nb, sums, parts, c.back);
    hipLaunchKernelGGL(k_ortho_factors, dim3(nb), dim3(64), 0, st, f);
  }
  hipLaunchKernelGGL((k_ortho_convert<T, P>), dim3((a.N + 63) / 64 * ((a.M + 63) / 64), nb), dim3(256), 0, st, c);
  return hipGetLastError();
}

// ---- the smaller side at most 128 (ortho_small.h) ----
struct SmallSizes {
  int mp, chunks, nb, slices, per, groups;
  int64_t part, gram, x, q, f, sums, total;
};
SmallSizes small_sizes(const OrthoArgs& a) {
  SmallSizes z{};
  const bool two = a.dtype == MOE_F32;
  z.mp = std::min(a.M, a.N) <= 64 ? 64 : 128;
  z.chunks = (int)div_up(std::max(a.M, a.N), CHUNK);
  z.groups = two ? a.steps : 1;
  const int64_t square = (int64_t)z.mp * z.mp * 4, wide = (int64_t)z.mp * CHUNK * 4 * z.chunks;
  // matrices at a time: X of fp32 updates within 1 GB (or one of them)
  z.nb = two ? (int)std::max<int64_t>(1, std::min<int64_t>(a.E, ((int64_t)1 << 30) / wide)) : a.E;
  z.nb = (int)div_up(a.E, div_up(a.E, z.nb));
  // slices: two workgroups for every CU, and few enough for one workgroup to add up
  z.slices = (int)std::min<int64_t>(std::min(z.chunks, 16), div_up(512, z.nb));
  z.per = (int)div_up(z.chunks, z.slices);
  z.slices = (int)div_up(z.chunks, z.per);
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t here = at;
    at += (bytes + 255) / 256 * 256;
    return here;
  };
  z.part = take(square * z.slices * z.nb);
  z.gram = take(square * z.nb);
  if (two) z.x = take(wide * z.nb);
  else z.q = take(square * z.nb);
  z.f = take(4 * (int64_t)z.nb * 2 * z.groups);
  z.sums = take(8 * (int64_t)z.nb * NORM_PARTS);
  z.total = at;
  return z;
}

// (bf16: all steps in one group.  Sums over a chunk's 16 roundings, over a slice's chunks, over slices)
bool is_small(const OrthoArgs& a) {
  const int m = std::min(a.M, a.N);
  if (m > 128 || a.dtype == MOE_F32) return m <= 128;
  const SmallSizes z = small_sizes(a);
  const double sums = (16.0 / z.chunks + (double)z.per / z.slices + z.slices) / 3.0;
  return group_steps(a, 0, lost(m, sums)) == a.steps;
}

template <typename K, typename A>
hipError_t small_launch(K* k, dim3 grid, int lds, const A& args, std::atomic<uint64_t>& done, hipStream_t st) {
  const hipError_t e = allow_lds(k, lds, device(), done);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(k, grid, dim3(SMALL_THREADS), lds, st, args);
  return hipGetLastError();
}

template <typename T, int MP, bool TALL>
hipError_t small_gram(const Small& s, int nb, hipStream_t st) {
  constexpr int P = sizeof(T) == 4 ? 2 : 1;
  static std::atomic<uint64_t> done{0};
  return small_launch(k_small_gram<T, P, MP, TALL>, dim3(s.slices, nb), MP * CHUNK * 2 * P, s, done, st);
}
template <int MP>
hipError_t small_reduce(const ReduceArgs& r, int nb, hipStream_t st) {
  hipLaunchKernelGGL(k_small_reduce<MP>, dim3(MP * MP / 4 / 256 + r.first, nb), dim3(256), 0, st, r);
  return hipGetLastError();
}
template <int MP, bool TALL, bool FIRST, bool LAST>
hipError_t small_step(const StepArgs& s, int nb, hipStream_t st) {
  static std::atomic<uint64_t> done{0};
  return small_launch(k_small_step<MP, TALL, FIRST, LAST>, dim3(s.a.slices, nb), SmallCfg<MP>::WIDE + SmallCfg<MP>::SQUARE, s,
                      done, st);
}

template <int MP, bool TALL>
hipError_t launch_small_as(const OrthoArgs& a, hipStream_t st) {
  const SmallSizes z = small_sizes(a);
  char* ws = (char*)a.ws;
  const bool two = a.dtype == MOE_F32;
  auto pow2 = [](int n) { return (float)std::ldexp(1.0, n); };
  for (int e0 = 0; e0 < a.E; e0 += z.nb) {
    const int nb = std::min(z.nb, a.E - e0);
    Small s{};
    const int64_t elems = (int64_t)a.M * a.N;
    s.g = two ? (const void*)((const float*)a.g + e0 * elems) : (const void*)((const bf16_t*)a.g + e0 * elems);
    s.o = two ? (void*)((float*)a.o + e0 * elems) : (void*)((bf16_t*)a.o + e0 * elems);
    s.M = a.M; s.N = a.N; s.m = std::min(a.M, a.N); s.k = std::max(a.M, a.N);
    s.chunks = z.chunks; s.per = z.per; s.slices = z.slices;
    s.vec = a.N % (two ? 4 : 8) == 0 && (((uintptr_t)a.g | (uintptr_t)a.o) & 15) == 0;
    s.eps = a.eps;
    double* sums = (double*)(ws + z.sums);
    s.sums = sums;
    s.parts = two ? launch_norm((const float*)s.g, elems, nb, sums, st) : launch_norm((const bf16_t*)s.g, elems, nb, sums, st);
    s.part = (float*)(ws + z.part);
    s.gram = ws + z.gram;
    s.x = ws + z.x;
    s.q = ws + z.q;
    s.back = (float*)(ws + z.f);
    s.on = s.back + z.groups * nb;
    hipError_t err = two ? small_gram<float, MP, TALL>(s, nb, st) : small_gram<bf16_t, MP, TALL>(s, nb, st);
    if (err != hipSuccess) return err;
    Spectrum spec;
    spec.begin();
    int ea = exponent_for(1.0);
    ReduceArgs r{s, pow2(ea), 1, factors_of(a, z.groups, nb, sums, s.parts, s.back)};
    err = small_reduce<MP>(r, nb, st);
    if (err != hipSuccess) return err;
    r.first = 0;
    if (!two) {
      StepsArgs q{};
      q.a = s;
      q.steps = a.steps;
      int eq = 0;
      for (int i = 0; i < a.steps; ++i) {
        const float* c = a.coef + 3 * i;
        double pm, tm, am, qm;
        spec.step(c, &pm, &tm, &am, &qm);
        const int ep = exponent_for(pm), et = exponent_for(tm), en = exponent_for(am), eqn = i == 0 ? ep : exponent_for(qm);
        q.s[i] = Recurrence{c[0] * pow2(ep), c[1] * pow2(ep - ea), c[2] * pow2(ep - 2 * ea), pow2(et - ep - ea),
                            pow2(en - et - ep), pow2(eqn - ep - eq)};
        ea = en;
        eq = eqn;
      }
      static std::atomic<uint64_t> done{0}, done_apply{0};
      err = small_launch(k_small_steps<MP>, dim3(nb), 2 * SmallCfg<MP>::SQUARE, q, done, st);
      if (err != hipSuccess) return err;
      ApplyArgs p{s, a.scale * pow2(-eq)};
      // (a Q is read by every workgroup: chunks enough for two of them on a CU)
      p.a.per = (int)std::max<int64_t>(1, (int64_t)z.chunks * nb / 1024);
      err = small_launch(k_small_apply<MP, TALL>, dim3((unsigned)div_up(z.chunks, p.a.per), nb),
                         MP * CHUNK * 2 + SmallCfg<MP>::SQUARE, p, done_apply, st);
      if (err != hipSuccess) return err;
      continue;
    }
    int x_exp = 0;
    for (int i = 0; i < a.steps; ++i) {
      const float* c = a.coef + 3 * i;
      double pm, tm, am, qm;
      spec.step(c, &pm, &tm, &am, &qm);
      spec.end();
      const int ep = exponent_for(pm);
      const bool last = i + 1 == a.steps;
      const int nx = X_EXP - 1;
      StepArgs q{s, c[0] * pow2(ep), c[1] * pow2(ep - ea), c[2] * pow2(ep - 2 * ea),
                 last ? a.scale * pow2(-ep - x_exp) : pow2(nx - ep - x_exp)};
      err = i == 0 ? (last ? small_step<MP, TALL, true, true>(q, nb, st) : small_step<MP, TALL, true, false>(q, nb, st))
                   : (last ? small_step<MP, TALL, false, true>(q, nb, st) : small_step<MP, TALL, false, false>(q, nb, st));
      if (err != hipSuccess) return err;
      if (last) break;
      x_exp = nx;
      s.back += nb;
      s.on += nb;
      spec.begin();
      ea = exponent_for(*std::max_element(spec.l, spec.l + Spectrum::N));
      r.a = s;
      r.gram = pow2(ea - 2 * x_exp);
      err = small_reduce<MP>(r, nb, st);
      if (err != hipSuccess) return err;
    }
  }
  return hipSuccess;
}

hipError_t launch_small(const OrthoArgs& a, hipStream_t st) {
  const bool tall = a.M > a.N;
  if (std::min(a.M, a.N) <= 64) return tall ? launch_small_as<64, true>(a, st) : launch_small_as<64, false>(a, st);
  return tall ? launch_small_as<128, true>(a, st) : launch_small_as<128, false>(a, st);
}

}  // namespace

size_t ortho_ws_bytes(const OrthoArgs& a) { return (size_t)(is_small(a) ? small_sizes(a).total : sizes(a).total); }

hipError_t launch_orthogonalize(const OrthoArgs& a, hipStream_t st) {
  if (is_small(a)) return launch_small(a, st);
  const Sizes z = sizes(a);
  const bool tall = a.M > a.N, fine = a.dtype == MOE_F32;
  char* ws = (char*)a.ws;
  for (int e0 = 0; e0 < a.E; e0 += z.nb) {
    const int nb = std::min(z.nb, a.E - e0);
    hipError_t err = a.dtype == MOE_F32 ? prepare<float>(a, z, e0, nb, st) : prepare<bf16_t>(a, z, e0, nb, st);
    if (err != hipSuccess) return err;
    Spectrum spec;
    char *x = ws + z.x0, *xt = ws + z.xt0;
    int parts = z.parts, x_exp = 0;
    const float *back = (const float*)(ws + z.f), *on = back + z.groups * nb;
    char* mats[5] = {};
    for (int i = 0; i < z.mats; ++i) mats[i] = ws + z.mat + i * nb * z.sm;
    auto two = [](int n) { return (float)std::ldexp(1.0, n); };

    bool second = false;  // which of the later groups' buffers is free
    for (int s = 0; s < a.steps;) {
      const int n = group_steps(a, s, lost(a));
      spec.begin();
      // (T and the spare ones for more than one step)
      char *A = mats[0], *P = mats[1], *T = mats[2], *Q = nullptr, *spare[2] = {mats[3], mats[4]};
      double lmax = 0.0;
      for (int i = 0; i < Spectrum::N; ++i) lmax = std::max(lmax, spec.l[i]);
      int ea = exponent_for(lmax), eq = 0;

      Args g{};
      g.batch = nb;
      g.jobs = 1;
      g.ra = g.rb = z.m;
      g.pc = (int)pitch(z.m, 2);
      g.sc = z.sm;
      // A = X X^T
      g.job[0] = Job{x, x, A, nullptr, two(ea - 2 * x_exp), 0.f, 0.f};
      g.alpha_e = back;
      g.square = true;
      g.sa = g.sb = z.sx * parts / 2;
      g.pa = g.pb = (int)pitch(z.k, parts);
      g.stages = (int)((z.k + 63) / 64) * (parts == 1 ? 1 : 2);
      err = parts == 1 ? gemm<1, 1, SYM>(g, fine, st) : gemm<2, 2, SYM>(g, fine, st);
      if (err != hipSuccess) return err;
      g.alpha_e = nullptr;
      g.sa = g.sb = z.sm;
      g.pa = g.pb = g.pc;
      g.stages = (int)((z.m + 63) / 64) * 2;
      for (int i = 0; i < n; ++i) {
        const float* c = a.coef + 3 * (s + i);
        double pm, tm, am, qm;
        spec.step(c, &pm, &tm, &am, &qm);
        const int ep = exponent_for(pm), et = exponent_for(tm), en = exponent_for(am), eqn = exponent_for(qm);
        const bool last = i + 1 == n;
        // P = a I + b A + c A^2
        g.jobs = 1;
        g.job[0] = Job{A, A, P, A, c[2] * two(ep - 2 * ea), c[1] * two(ep - ea), c[0] * two(ep)};
        err = gemm<2, 2, SYM>(g, fine, st);
        if (err != hipSuccess) return err;
        // T = P A and the next Q = P Q
        g.jobs = 0;
        char* qn = nullptr;
        if (!last) g.job[g.jobs++] = Job{P, A, T, nullptr, two(et - ep - ea), 0.f, 0.f};
        if (Q) {
          qn = spare[0];
          g.job[g.jobs++] = Job{P, Q, qn, nullptr, two(eqn - ep - eq), 0.f, 0.f};
        }
        if (g.jobs > 0) {
          err = gemm<2, 2, SYM>(g, fine, st);
          if (err != hipSuccess) return err;
        }
        if (!last) {  // the next A = T P
          g.jobs = 1;
          g.job[0] = Job{T, P, A, nullptr, two(en - et - ep), 0.f, 0.f};
          err = gemm<2, 2, SYM>(g, fine, st);
          if (err != hipSuccess) return err;
          ea = en;
        }
        if (Q) {
          spare[0] = Q;  // free again
          Q = qn;
          eq = eqn;
        } else {
          Q = P;
          eq = ep;
          P = spare[1];
        }
      }
      s += n;
      spec.end();
      // X = Q X, as rows of X or, for a tall update's result, of its transpose
      const bool final = s == a.steps;
      const bool swap = final && tall;
      Args r{};
      r.batch = nb;
      r.jobs = 1;
      r.stages = (int)((z.m + 63) / 64) * 2;
      r.alpha_e = final ? back : on;
      r.square = false;
      const int nx_exp = X_EXP - 1;  // (a norm below 2, with its own power of two)
      const float alpha = final ? a.scale * two(-eq - x_exp) : two(nx_exp - eq - x_exp);
      const int px = (int)pitch(z.m, parts);
      const int64_t sxt = z.sxt * parts / 2;
      if (swap) {
        r.job[0] = Job{xt, Q, nullptr, nullptr, alpha, 0.f, 0.f};
        r.ra = z.k; r.rb = z.m; r.sa = sxt; r.sb = z.sm; r.pa = px; r.pb = g.pc;
      } else {
        r.job[0] = Job{Q, xt, nullptr, nullptr, alpha, 0.f, 0.f};
        r.ra = z.m; r.rb = z.k; r.sa = z.sm; r.sb = sxt; r.pa = g.pc; r.pb = px;
      }
      if (final) {
        r.so = (int64_t)a.M * a.N;
        r.o = fine ? (void*)((float*)a.o + e0 * r.so) : (void*)((bf16_t*)a.o + e0 * r.so);
        err = parts == 2 ? gemm<2, 2, OUT>(r, fine, st) : swap ? gemm<1, 2, OUT>(r, fine, st) : gemm<2, 1, OUT>(r, fine, st);
        if (err != hipSuccess) return err;
      } else {
        const int64_t half = z.parts == 1 && second ? 1 : 0;
        char* nx = z.parts == 1 || !second ? ws + z.x1 + half * nb * z.sx : ws + z.x0;
        char* nxt = z.parts == 1 || !second ? ws + z.xt1 + half * nb * z.sxt : ws + z.xt0;
        second = !second;
        r.job[0].c = nx;
        r.sc = z.sx;
        r.pc = (int)pitch(z.k, 2);
        r.ct = nxt;
        r.sct = z.sxt;
        r.pct = (int)pitch(z.m, 2);
        err = parts == 2 ? gemm<2, 2, SPLIT>(r, fine, st) : gemm<2, 1, SPLIT>(r, fine, st);
        if (err != hipSuccess) return err;
        x = nx;
        xt = nxt;
        parts = 2;
        x_exp = nx_exp;
        back += nb;
        on += nb;
      }
    }
  }
  return hipSuccess;
}

}  // namespace moe
