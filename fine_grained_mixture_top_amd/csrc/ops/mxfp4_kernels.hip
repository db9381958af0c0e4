// Weights in OCP MXFP4 and the launches of their products (mxfp4_gemm.h).
#include <algorithm>

#include "launch_util.h"
#include "mxfp4_gemm.h"

namespace moe {

namespace {

// ---------------------------------------------------------------------------
// w [E,K,N] -> codes [E,N,K/2], scale codes [E,N,K/32].  A workgroup turns 128 x 64
// of a matrix over in LDS; a thread quantizes one block of 32 along K, the
// instruction for two values rounds to nearest, ties to even, and cuts off at 6.  Bytes bound
// it: 64 x 2048 x 2048 in bf16 162 us, 4.2 TB/s, in fp32 243 us, 5.0.
// ---------------------------------------------------------------------------
template <typename T>
__global__ void __launch_bounds__(256)
k_mxfp4_weights(const T* w, uint8_t* q, uint8_t* s, int K, int N) {
  __shared__ float tile[128][65];
  const int e = blockIdx.z, k0 = blockIdx.y * 128, n0 = blockIdx.x * 64, tid = threadIdx.x;
  constexpr int V = 16 / sizeof(T);
  const T* p = w + ((int64_t)e * K + k0) * N + n0;
  for (int i = tid; i < 128 * 64 / V; i += 256) {
    const int k = i / (64 / V), n = i % (64 / V) * V;
    float v[V];
    if (k0 + k < K && n0 + n < N) {  // (N a multiple of 16: whole vectors)
      const uint4 u = *reinterpret_cast<const uint4*>(p + (int64_t)k * N + n);
      T x[V];
      __builtin_memcpy(x, &u, 16);
#pragma unroll
      for (int y = 0; y < V; ++y) v[y] = Elem<T>::to_f(x[y]);
    } else {
#pragma unroll
      for (int y = 0; y < V; ++y) v[y] = 0.f;
    }
#pragma unroll
    for (int y = 0; y < V; ++y) tile[k][n + y] = v[y];
  }
  __syncthreads();
  // four blocks of a column lie in neighbouring threads: 64 bytes of codes
  const int n = tid >> 2, b = tid & 3;
  if (n0 + n >= N || k0 + 32 * b >= K) return;
  uint32_t amax = 0;
#pragma unroll
  for (int i = 0; i < 32; ++i) amax = max(amax, __float_as_uint(tile[32 * b + i][n]) & 0x7fffffffu);
  // floor(log2(amax)) - 2, 2 being the exponent of 6; an infinity or a NaN: 255
  const int exponent = (int)(amax >> 23);
  const uint32_t code = exponent == 255 ? 255u : (uint32_t)max(exponent - 2, 0);
  const float scale = __uint_as_float(code << 23);
  uint32_t words[4];
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    uint32_t u = 0;
    const float* v = &tile[32 * b + 8 * x][n];
    u = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(u, v[0], v[65], scale, 0);
    u = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(u, v[2 * 65], v[3 * 65], scale, 1);
    u = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(u, v[4 * 65], v[5 * 65], scale, 2);
    u = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(u, v[6 * 65], v[7 * 65], scale, 3);
    words[x] = code == 255u ? 0u : u;
  }
  const int64_t at = ((int64_t)e * N + n0 + n) * (K / 32) + k0 / 32 + b;
  *reinterpret_cast<uint4*>(q + 16 * at) = make_uint4(words[0], words[1], words[2], words[3]);
  s[at] = (uint8_t)code;
}

int64_t row_tiles(const f4::Args& a, int64_t used, int BM) { return mxfp4_row_tiles(used, a.E, BM); }

template <int FN>
hipError_t launch_thin(int out, const f4::Args& a, int64_t used, hipStream_t st) {
  const dim3 grid((unsigned)(row_tiles(a, used, 16) * div_up(a.N, 16 * FN)));
  if (out == MOE_BF16) hipLaunchKernelGGL((f4::k_mxfp4_thin<FN, bf16_t>), grid, dim3(256), 0, st, a);
  else hipLaunchKernelGGL((f4::k_mxfp4_thin<FN, float>), grid, dim3(256), 0, st, a);
  return hipGetLastError();
}

template <int BM, int BN, int WM, int WN, typename O>
hipError_t launch_tile(const f4::Args& a, int64_t used, hipStream_t st) {
  using C = f4::Cfg<BM, BN, WM, WN>;
  auto* k = f4::k_mxfp4_tile<BM, BN, WM, WN, O>;
  static std::atomic<uint64_t> done{0};
  const hipError_t e = allow_lds(k, C::SMEM, device(), done);
  if (e != hipSuccess) return e;
  const int64_t tiles = row_tiles(a, used, BM) * div_up(a.N, BN);
  hipLaunchKernelGGL(k, dim3((unsigned)((tiles + 7) / 8 * 8)), dim3(C::NTH), C::SMEM, st, a);
  return hipGetLastError();
}

template <int BM, int BN, int WM, int WN>
hipError_t launch_tile(int out, const f4::Args& a, int64_t used, hipStream_t st) {
  return out == MOE_BF16 ? launch_tile<BM, BN, WM, WN, bf16_t>(a, used, st) : launch_tile<BM, BN, WM, WN, float>(a, used, st);
}

}  // namespace

hipError_t launch_mxfp4_weights(int dtype, int E, int K, int N, const void* w, uint8_t* q, uint8_t* s, hipStream_t st) {
  const dim3 grid((N + 63) / 64, (K + 127) / 128, E);
  if (dtype == MOE_F32) hipLaunchKernelGGL(k_mxfp4_weights<float>, grid, dim3(256), 0, st, (const float*)w, q, s, K, N);
  else hipLaunchKernelGGL(k_mxfp4_weights<bf16_t>, grid, dim3(256), 0, st, (const bf16_t*)w, q, s, K, N);
  return hipGetLastError();
}

hipError_t launch_mxfp4_mm(const PlanArgs& p, const Mxfp4Args& m, hipStream_t st) {
  f4::Args a{};
  a.a = m.a; a.q = m.q; a.s = m.s; a.c = m.c;
  a.offsets = p.offsets; a.counts = p.counts;
  a.row_token = m.gather ? p.row_token : nullptr;
  a.a_rows = m.a_rows; a.rows = m.rows; a.E = m.E; a.K = m.K; a.N = m.N;
  const int64_t used = m.rows_used;
  // Thin tiles read an expert's weights once per 16 rows; the others' time is at least
  // their stages', one after the other, however few they are.  So thin up to 16 rows per expert, and
  // while there is little to compute.  Measured, thin and tiles of 64 (us):
  //   64 experts of 2048 x 2048, 16 rows each 42 and 47, 24 54 and 49
  //   128 experts of 1536 x 512, 16 rows each 21 and 28, 32 32 and 29
  //   8 experts of 736 x 1040, 400 rows (416000) 8.4 and 12.8, 1600 (1664000) 24 and 14
  //   one of 2048 x 2048, 256 rows (524288) 10 and 25, 1024 (2097152) 28.5 and 25
  // The average and the rows times N decide as well where a few experts hold all rows, and whatever K:
  //   128 experts of 1536 x 512, 2048 rows in 8 of them 17 and 27, in one 17 and 27
  //   64 of 2048 x 2048, 1024 in 8 31 and 45, in one 30 and 43
  //   256 of 7168 x 4096, 4096 in all 1071 and 1338, in 8 614 and 1065, in one 611 and 1051
  //   one of K x 2048, 512 rows (1048576), K = 512 11 and 10, 2048 18 and 26, 7168 44 and 81
  // (a grid has fewer than 2^24 workgroups of 256)
  const int64_t thin = row_tiles(a, used, 16) * div_up(a.N, 64);
  if ((used <= 16 * (int64_t)a.E || used * a.N <= (1 << 20)) && thin < MXFP4_MAX_TILES) {
    // under half a workgroup of 64 columns per CU: workgroups of 16 (one row, 7168 x 4096
    // 8.6 us in place of 13.7; 64 of 2048 x 2048, where it is the other way, 8.0 and 7.9)
    if (thin < cu_count(device()) / 2) return launch_thin<1>(m.out, a, used, st);
    return launch_thin<4>(m.out, a, used, st);
  }
  // Tiles of 64 or 128 rows (us): 64 experts of 2048 x 2048, 128 rows each 92 and 100, 512 269
  // and 254, 2048 1084 and 893; 128 experts of 1536 x 512, 256 rows each 63 and 67, 1024 208 and
  // 193.  Up to four tiles of 128 per CU too: one of 2048 x 2048, 1024 rows 25 and 37, 8192 76
  // and 88, 16384 132 and 135.
  if ((used <= 256 * (int64_t)a.E || row_tiles(a, used, 128) * div_up(a.N, 256) <= 4 * cu_count(device())) &&
      row_tiles(a, used, 64) * div_up(a.N, 256) < MXFP4_MAX_TILES)
    return launch_tile<64, 256, 1, 4>(m.out, a, used, st);
  return launch_tile<128, 256, 1, 4>(m.out, a, used, st);
}

}  // namespace moe
