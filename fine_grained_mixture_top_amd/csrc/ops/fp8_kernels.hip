// Quantizers to E4M3 with a scale per block of 128, and the SwiGLU kernels
// between the experts' two products (include/moe_ops.h).  All of them are
// bound by memory: every value is read once and its code written once.  On one
// MI355X (device copy of 1 GiB: 5.2 TB/s), bf16:
//   rows      131072 x 2048                  134 us  6.0 TB/s
//   weights   64 x 2048 x 1024, both layouts 102 us  5.3 TB/s
//   columns   131072 x 2048                  153 us  5.3 TB/s
//   SwiGLU    262144 x 256                    62 us  5.4 TB/s
//   its gradient  131072 x 1024              230 us  5.8 TB/s
#include <algorithm>

#include "fp8_block.h"
#include "ops_launch.h"

namespace moe {

namespace {

// A plan's rows as a kernel over row numbers sees them: every row without one.
struct RowFilter {
  const int32_t* offsets;    // null: every row
  const int32_t* row_token;
  int E;
  __device__ __forceinline__ bool operator()(int64_t r) const {
    return !offsets || (r < offsets[E] && row_token[r] >= 0);
  }
};

constexpr int64_t MAX_GRID = 1 << 22;  // workgroups; the kernels stride over what is left

unsigned grid_for(int64_t threads) { return (unsigned)std::min<int64_t>((threads + 255) / 256, MAX_GRID); }

// rows [R][C] -> codes and scales, eight lanes per block of 128
template <typename T>
__global__ void __launch_bounds__(256)
k_quant_rows_128(const T* __restrict__ src, int64_t R, int C, RowFilter rows, bool stream,
                 uint8_t* __restrict__ q, float* __restrict__ s) {
  const int nb = (C + 127) / 128;
  const int64_t blocks = R * nb;
  for (int64_t b = ((int64_t)blockIdx.x * 256 + threadIdx.x) >> 3; b < blocks; b += (int64_t)gridDim.x * 32) {
    const int64_t r = b >> 32 ? b / nb : (int64_t)((uint32_t)b / (uint32_t)nb);
    const int cb = (int)(b - r * nb), col = cb * 128 + (threadIdx.x & 7) * 16;
    const bool on = rows(r);
    float v[16];
    if (on && col < C) {
      load16(src + r * C + col, v);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = 0.f;
    }
    float sc;
    const uint4 code = quant_block8(v, sc);
    if (!on) continue;
    if (col < C) store_as(reinterpret_cast<uint4*>(q + r * C + col), code, stream);
    if ((threadIdx.x & 7) == 0) s[b] = sc;
  }
}

// logistic sigmoid to 5 * 2^-24 of itself whatever g is (correct rounding: 1): the
// exponential's argument in two parts, the reciprocal with a Newton step; 0 below 2^-126.
// (device_common.h's sigmoidf_ is off by |g| steps, and a value near the border
// of two codes then falls on the other side more often than it needs to.)
__device__ __forceinline__ float sigmoid_(float g) {
  constexpr float L = 1.44269502f, L_LO = 1.92596299e-8f;  // log2(e) = L + L_LO
  const float hi = -g * L;
  const float lo = fmaf(-g, L, -hi) - g * L_LO;
  const float p = __builtin_amdgcn_exp2f(hi);
  const float e = fabsf(hi) < 126.f ? fmaf(p, lo * 0.693147181f, p) : p;
  const float d = fminf(1.f + e, 0x1p127f);  // (finite: the Newton step of an infinite d would be NaN)
  const float r = __builtin_amdgcn_rcpf(d);
  return fmaf(r, fmaf(-d, r, 1.f), r);
}

// A = silu(G) U of rows h [R][2n], quantized; A itself too when `a` is set
template <typename T>
__global__ void __launch_bounds__(256)
k_swiglu_fp8(const T* __restrict__ h, int64_t R, int n, RowFilter rows, bool stream, uint8_t* __restrict__ q,
             float* __restrict__ s, T* __restrict__ a) {
  const int nb = (n + 127) / 128;
  const int64_t blocks = R * nb;
  for (int64_t b = ((int64_t)blockIdx.x * 256 + threadIdx.x) >> 3; b < blocks; b += (int64_t)gridDim.x * 32) {
    const int64_t r = b >> 32 ? b / nb : (int64_t)((uint32_t)b / (uint32_t)nb);
    const int cb = (int)(b - r * nb), col = cb * 128 + (threadIdx.x & 7) * 16;
    const bool on = rows(r);
    float v[16];
    if (on && col < n) {
      float g[16], u[16];
      load16(h + r * 2 * n + col, g);
      load16(h + r * 2 * n + n + col, u);
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = g[i] * sigmoid_(g[i]) * u[i];
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = 0.f;
    }
    float sc;
    const uint4 code = quant_block8(v, sc);
    if (!on) continue;
    if (col < n) {
      store_as(reinterpret_cast<uint4*>(q + r * n + col), code, stream);
      if (a) store16(a + r * n + col, v);
    }
    if ((threadIdx.x & 7) == 0) s[b] = sc;
  }
}

// dh = (da U s (1 + G (1 - s)), da silu(G)), s = sigmoid(G); 16 bytes of each
// matrix per thread, so that every store instruction writes whole lines (32
// bytes in two stores, past the caches: 3.2 instead of 5.4 TB/s)
template <typename T>
__global__ void __launch_bounds__(256)
k_swiglu_bwd_rows(const T* __restrict__ da, const T* __restrict__ h, int64_t R, int n, RowFilter rows, bool stream,
                  T* __restrict__ dh) {
  constexpr int V = 16 / (int)sizeof(T);
  const int per = n / V;
  const int64_t total = R * per;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t r = total >> 32 ? i / per : (int64_t)((uint32_t)i / (uint32_t)per);
    const int col = (int)(i - r * per) * V;
    if (!rows(r)) continue;
    float d[V], g[V], u[V];
    unpack16<T>(*reinterpret_cast<const uint4*>(da + r * n + col), d);
    unpack16<T>(*reinterpret_cast<const uint4*>(h + r * 2 * n + col), g);
    unpack16<T>(*reinterpret_cast<const uint4*>(h + r * 2 * n + n + col), u);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const float sg = sigmoid_(g[j]), dj = d[j];
      d[j] = dj * u[j] * sg * (1.f + g[j] * (1.f - sg));
      u[j] = dj * g[j] * sg;
    }
    store_as(reinterpret_cast<uint4*>(dh + r * 2 * n + col), pack16<T>(d), stream);
    store_as(reinterpret_cast<uint4*>(dh + r * 2 * n + n + col), pack16<T>(u), stream);
  }
}

// ---- 128 x 128 tiles ----
// 256 threads; thread t holds the 8 x 8 values at rows 8 (t / 16), columns
// 8 (t % 16), so that both a row's codes and a column's are eight bytes of it.

// The 8 x 8 values as loaded, their largest magnitudes and their codes.
// fp32: magnitudes as the value's bits, a word per column.
template <typename T> struct Tile8;
template <> struct Tile8<float> {
  float v[8][8];
  typedef uint32_t Mag[8];  // per column
  __device__ __forceinline__ void load(int i, const float* p) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    v[i][0] = a.x; v[i][1] = a.y; v[i][2] = a.z; v[i][3] = a.w;
    v[i][4] = b.x; v[i][5] = b.y; v[i][6] = b.z; v[i][7] = b.w;
  }
  __device__ __forceinline__ void zero(int i) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
  }
  __device__ __forceinline__ void column_mags(Mag& m) const {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      m[j] = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) m[j] = max(m[j], mag_bits(v[i][j]));
    }
  }
  static __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return max(a, b); }
  static __device__ __forceinline__ uint32_t bits(const Mag& m, int j) { return m[j]; }
  __device__ __forceinline__ float value(int i, int j) const { return v[i][j]; }
};
// bf16: two columns in a word, which an integer maximum of 16-bit halves
// orders just as well
template <> struct Tile8<bf16_t> {
  uint4 w[8];
  typedef uint32_t Mag[4];
  typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
  __device__ __forceinline__ void load(int i, const bf16_t* p) { w[i] = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void zero(int i) { w[i] = make_uint4(0, 0, 0, 0); }
  static __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) {
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a), __builtin_bit_cast(u16x2, b)));
  }
  __device__ __forceinline__ uint32_t word(int i, int c) const {
    return c == 0 ? w[i].x : c == 1 ? w[i].y : c == 2 ? w[i].z : w[i].w;
  }
  __device__ __forceinline__ void column_mags(Mag& m) const {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      m[c] = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) m[c] = larger(m[c], word(i, c) & 0x7fff7fffu);
    }
  }
  static __device__ __forceinline__ uint32_t bits(const Mag& m, int j) {
    return j & 1 ? m[j >> 1] & 0xffff0000u : m[j >> 1] << 16;
  }
  __device__ __forceinline__ float value(int i, int j) const {
    return __uint_as_float(j & 1 ? word(i, j >> 1) & 0xffff0000u : word(i, j >> 1) << 16);
  }
};

// 4 x 4 bytes transposed: word i's byte j -> word j's byte i
__device__ __forceinline__ void transpose4(uint32_t (&w)[4]) {
  const uint32_t a = __builtin_amdgcn_perm(w[1], w[0], 0x05010400), b = __builtin_amdgcn_perm(w[1], w[0], 0x07030602);
  const uint32_t c = __builtin_amdgcn_perm(w[3], w[2], 0x05010400), d = __builtin_amdgcn_perm(w[3], w[2], 0x07030602);
  w[0] = __builtin_amdgcn_perm(c, a, 0x05040100);
  w[1] = __builtin_amdgcn_perm(c, a, 0x07060302);
  w[2] = __builtin_amdgcn_perm(d, b, 0x05040100);
  w[3] = __builtin_amdgcn_perm(d, b, 0x07060302);
}

// codes c [8 rows][2 words] as eight bytes of each column: t [8 columns][2 words]
__device__ __forceinline__ void transpose8(const uint32_t (&c)[8][2], uint32_t (&t)[8][2]) {
#pragma unroll
  for (int r = 0; r < 2; ++r)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t w[4] = {c[4 * r][h], c[4 * r + 1][h], c[4 * r + 2][h], c[4 * r + 3][h]};
      transpose4(w);
#pragma unroll
      for (int j = 0; j < 4; ++j) t[4 * h + j][r] = w[j];
    }
}

constexpr int TP = 128 + 16;  // LDS pitch of a transposed tile's row (bytes)

// weights [K][N] of expert blockIdx.z, tile (blockIdx.y, blockIdx.x)
template <typename T>
__global__ void __launch_bounds__(256)
k_quant_weights_128(const T* __restrict__ w, int K, int N, bool stream, uint8_t* __restrict__ q,
                    uint8_t* __restrict__ qt, float* __restrict__ s) {
  __shared__ uint32_t wmax[4];
  __shared__ __attribute__((aligned(16))) uint8_t tile[128 * TP];
  const int tid = threadIdx.x;
  const int k0 = blockIdx.y * 128, n0 = blockIdx.x * 128;
  const int rk = (tid >> 4) * 8, cn = (tid & 15) * 8;
  const size_t base = (size_t)blockIdx.z * K * N;
  Tile8<T> v;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int k = k0 + rk + i, n = n0 + cn;
    if (k < K && n < N) v.load(i, w + base + (size_t)k * N + n);
    else v.zero(i);
  }
  uint32_t m = 0;
  {
    typename Tile8<T>::Mag cm;
    v.column_mags(cm);
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, Tile8<T>::bits(cm, j));
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, o, 64));
  if ((tid & 63) == 0) wmax[tid >> 6] = m;
  __syncthreads();
  m = max(max(wmax[0], wmax[1]), max(wmax[2], wmax[3]));
  const float sc = block_scale(m), inv = __fdiv_rn(1.f, sc);
  if (tid == 0) s[((size_t)blockIdx.z * gridDim.y + blockIdx.y) * gridDim.x + blockIdx.x] = sc;
  uint32_t c[8][2];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    c[i][0] = e4m3x4(v.value(i, 0) * inv, v.value(i, 1) * inv, v.value(i, 2) * inv, v.value(i, 3) * inv);
    c[i][1] = e4m3x4(v.value(i, 4) * inv, v.value(i, 5) * inv, v.value(i, 6) * inv, v.value(i, 7) * inv);
  }
  if (q) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int k = k0 + rk + i, n = n0 + cn;
      if (k < K && n < N)
        store_as(reinterpret_cast<uint2*>(q + base + (size_t)k * N + n), make_uint2(c[i][0], c[i][1]), stream);
    }
  }
  if (qt) {
    uint32_t ct[8][2];
    transpose8(c, ct);
#pragma unroll
    for (int j = 0; j < 8; ++j) *reinterpret_cast<uint2*>(tile + (cn + j) * TP + rk) = make_uint2(ct[j][0], ct[j][1]);
    __syncthreads();
    // 16 bytes per thread: eight threads per column's 128 rows
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int n = i * 32 + (tid >> 3), k = (tid & 7) * 16;
      if (n0 + n < N && k0 + k < K)
        store_as(reinterpret_cast<uint4*>(qt + base + (size_t)(n0 + n) * K + k0 + k),
                 *reinterpret_cast<const uint4*>(tile + n * TP + k), stream);
    }
  }
}

// columns of the segments: one workgroup per block of 128 rows and 128 columns.
// Gathered rows go column block by column block, each on one XCD, whose L2 then
// holds much of the column block of all tokens for its K readings (131072 tokens,
// K = 2, C = 2048 323 -> 288 us; 32768, 8, 1536 196 -> 189; 16384, 4, 2048 79 -> 78, with
// nothing in the caches before); the plan's own rows go as they lie.
template <typename T>
__global__ void __launch_bounds__(256)
k_quant_cols_128(const T* __restrict__ src, int C, int Tn, bool gather, PlanArgs p, bool stream,
                 uint8_t* __restrict__ q, float* __restrict__ s) {
  typedef Tile8<T> V;
  constexpr int MW = sizeof(typename V::Mag) / 4;
  __shared__ typename V::Mag cmax[4][16];
  __shared__ __attribute__((aligned(16))) uint8_t tile[128 * TP];
  const int tid = threadIdx.x;
  const int ct = (C + 127) / 128;
  const int nb = p.cap / 128;
  const int v = gather ? xcd_virtual_id(blockIdx.x, gridDim.x) : (int)blockIdx.x;
  const int64_t blk = gather ? v % nb : v / ct;
  const int r0 = (int)(blk * 128), c0 = (gather ? v / nb : v % ct) * 128;
  if (c0 >= C || r0 >= p.offsets[p.E]) return;
  const int rk = (tid >> 4) * 8, cn = (tid & 15) * 8;
  int tok[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) tok[i] = p.row_token[r0 + rk + i];
  V t8;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if ((unsigned)tok[i] < (unsigned)Tn && c0 + cn < C)
      t8.load(i, src + (size_t)(gather ? tok[i] : r0 + rk + i) * C + c0 + cn);
    else
      t8.zero(i);
  }
  // the columns' magnitudes: over this thread's rows, the wave's, the block's
  typename V::Mag m;
  t8.column_mags(m);
#pragma unroll
  for (int j = 0; j < MW; ++j) {
    m[j] = V::larger(m[j], (uint32_t)__shfl_xor((int)m[j], 16, 64));
    m[j] = V::larger(m[j], (uint32_t)__shfl_xor((int)m[j], 32, 64));
  }
  if ((tid & 63) < 16)
#pragma unroll
    for (int j = 0; j < MW; ++j) cmax[tid >> 6][tid & 15][j] = m[j];
  __syncthreads();
#pragma unroll
  for (int j = 0; j < MW; ++j)
    m[j] = V::larger(V::larger(cmax[0][tid & 15][j], cmax[1][tid & 15][j]),
                     V::larger(cmax[2][tid & 15][j], cmax[3][tid & 15][j]));
  float inv[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float sc = block_scale(V::bits(m, j));
    inv[j] = __fdiv_rn(1.f, sc);
    if (tid < 16 && c0 + cn + j < C) s[blk * C + c0 + cn + j] = sc;
  }
  uint32_t c[8][2], t[8][2];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    c[i][0] = e4m3x4(t8.value(i, 0) * inv[0], t8.value(i, 1) * inv[1], t8.value(i, 2) * inv[2], t8.value(i, 3) * inv[3]);
    c[i][1] = e4m3x4(t8.value(i, 4) * inv[4], t8.value(i, 5) * inv[5], t8.value(i, 6) * inv[6], t8.value(i, 7) * inv[7]);
  }
  transpose8(c, t);
#pragma unroll
  for (int j = 0; j < 8; ++j) *reinterpret_cast<uint2*>(tile + (cn + j) * TP + rk) = make_uint2(t[j][0], t[j][1]);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int n = i * 32 + (tid >> 3), k = (tid & 7) * 16;
    if (c0 + n < C)
      store_as(reinterpret_cast<uint4*>(q + (blk * C + c0 + n) * 128 + k),
               *reinterpret_cast<const uint4*>(tile + n * TP + k), stream);
  }
}

int64_t bytes_of(int dtype) { return dtype == MOE_BF16 ? 2 : 4; }

RowFilter filter_of(const PlanArgs& p) { return RowFilter{p.offsets, p.row_token, p.E}; }

}  // namespace

hipError_t launch_quant_rows_128(const PlanArgs& p, int dtype, int64_t R, int C, const void* src, uint8_t* q,
                                 float* s, hipStream_t st) {
  const dim3 grid(grid_for(R * ((C + 127) / 128) * 8));
  const bool stream = streams(R * C * (bytes_of(dtype) + 1));
  if (dtype == MOE_BF16)
    hipLaunchKernelGGL(k_quant_rows_128<bf16_t>, grid, dim3(256), 0, st, (const bf16_t*)src, R, C, filter_of(p), stream,
                       q, s);
  else
    hipLaunchKernelGGL(k_quant_rows_128<float>, grid, dim3(256), 0, st, (const float*)src, R, C, filter_of(p), stream,
                       q, s);
  return hipGetLastError();
}

hipError_t launch_swiglu_fp8(const PlanArgs& p, int dtype, int64_t R, int n, const void* h, uint8_t* q, float* s,
                             void* a, hipStream_t st) {
  const dim3 grid(grid_for(R * ((n + 127) / 128) * 8));
  const bool stream = streams(R * n * ((a ? 3 : 2) * bytes_of(dtype) + 1));
  if (dtype == MOE_BF16)
    hipLaunchKernelGGL(k_swiglu_fp8<bf16_t>, grid, dim3(256), 0, st, (const bf16_t*)h, R, n, filter_of(p), stream, q, s,
                       (bf16_t*)a);
  else
    hipLaunchKernelGGL(k_swiglu_fp8<float>, grid, dim3(256), 0, st, (const float*)h, R, n, filter_of(p), stream, q, s,
                       (float*)a);
  return hipGetLastError();
}

hipError_t launch_swiglu_bwd_rows(const PlanArgs& p, int dtype, int64_t R, int n, const void* da, const void* h,
                                  void* dh, hipStream_t st) {
  const dim3 grid(grid_for(R * (n / (16 / bytes_of(dtype)))));
  const bool stream = streams(R * n * 5 * bytes_of(dtype));
  if (dtype == MOE_BF16)
    hipLaunchKernelGGL(k_swiglu_bwd_rows<bf16_t>, grid, dim3(256), 0, st, (const bf16_t*)da, (const bf16_t*)h, R, n,
                       filter_of(p), stream, (bf16_t*)dh);
  else
    hipLaunchKernelGGL(k_swiglu_bwd_rows<float>, grid, dim3(256), 0, st, (const float*)da, (const float*)h, R, n,
                       filter_of(p), stream, (float*)dh);
  return hipGetLastError();
}

hipError_t launch_quant_weights_128(int dtype, int E, int K, int N, const void* w, uint8_t* q, uint8_t* qt, float* s,
                                    hipStream_t st) {
  const dim3 grid((N + 127) / 128, (K + 127) / 128, E);
  const bool stream = streams((int64_t)E * K * N * (bytes_of(dtype) + (q ? 1 : 0) + (qt ? 1 : 0)));
  if (dtype == MOE_BF16)
    hipLaunchKernelGGL(k_quant_weights_128<bf16_t>, grid, dim3(256), 0, st, (const bf16_t*)w, K, N, stream, q,
                       qt, s);
  else
    hipLaunchKernelGGL(k_quant_weights_128<float>, grid, dim3(256), 0, st, (const float*)w, K, N, stream, q,
                       qt, s);
  return hipGetLastError();
}

hipError_t launch_quant_cols_128(const PlanArgs& p, int dtype, int C, bool gather, const void* src, uint8_t* q,
                                 float* s, hipStream_t st) {
  dim3 grid((unsigned)((int64_t)(p.cap / 128) * ((C + 127) / 128)));
  if (grid.x == 0) return hipSuccess;
  if (gather) grid.x = (grid.x + 7) / 8 * 8;  // whole turns over the XCDs
  const bool stream = streams((int64_t)p.cap * C * (bytes_of(dtype) + 1));
  if (dtype == MOE_BF16)
    hipLaunchKernelGGL(k_quant_cols_128<bf16_t>, grid, dim3(256), 0, st, (const bf16_t*)src, C, p.T, gather,
                       p, stream, q, s);
  else
    hipLaunchKernelGGL(k_quant_cols_128<float>, grid, dim3(256), 0, st, (const float*)src, C, p.T, gather, p,
                       stream, q, s);
  return hipGetLastError();
}

}  // namespace moe
