// Launches of the E4M3 products (fp8_gemm.h).
#include <algorithm>
#include <atomic>

#include "fp8_gemm.h"

namespace moe {

namespace {

// the current device, or -1
int device() {
  int dev = -1;
  return hipGetDevice(&dev) == hipSuccess ? dev : -1;
}

int cu_count(int dev) {
  int cus = 0;
  if (dev < 0 || hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || cus <= 0)
    return 256;
  return cus;
}

// Dynamic LDS beyond the default, allowed once per kernel (its `done`) and device.
template <typename K>
hipError_t allow_lds(K* kernel, int bytes, int dev, std::atomic<uint64_t>& done) {
  const uint64_t bit = dev >= 0 && dev < 64 ? 1ull << dev : 0;
  if (bit && (done.load(std::memory_order_relaxed) & bit)) return hipSuccess;
  const hipError_t e =
      hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == hipSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

template <int BM, int BN, int WM, int WN, bool WG, typename O>
hipError_t launch_tiles(const f8::Args& a, int64_t tiles, hipStream_t st) {
  using C = f8::Cfg<BM, BN, WM, WN, WG>;
  auto* k = f8::k_fp8_gemm<BM, BN, WM, WN, WG, O>;
  static std::atomic<uint64_t> done{0};
  const int dev = device();
  const hipError_t e = allow_lds(k, C::SMEM, dev, done);
  if (e != hipSuccess) return e;
  const int64_t most = (int64_t)cu_count(dev) * (C::SMEM > 72 * 1024 ? 1 : 2);
  unsigned grid = (unsigned)std::min<int64_t>(std::max<int64_t>(tiles, 1), most);
  if (grid > 8) grid = (grid + 7) / 8 * 8;  // whole turns over the XCDs
  hipLaunchKernelGGL(k, dim3(grid), dim3(C::NTH), C::SMEM, st, a);
  return hipGetLastError();
}

int64_t div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Row tiles at most: every segment with rows may end inside one.
int64_t row_tiles(const f8::Args& a, int64_t used, int BM) { return div_up(used, BM) + std::min<int64_t>(a.E, used); }

template <int RT, int FN, int UNR>
hipError_t launch_thin(int out, const f8::Args& a, int64_t used, hipStream_t st) {
  const int64_t tiles = row_tiles(a, used, 16 * RT) * div_up(a.N, 16 * FN);
  if (out == MOE_BF16)
    hipLaunchKernelGGL((f8::k_fp8_thin<RT, FN, UNR, bf16_t>), dim3((unsigned)tiles), dim3(256), 0, st, a);
  else
    hipLaunchKernelGGL((f8::k_fp8_thin<RT, FN, UNR, float>), dim3((unsigned)tiles), dim3(256), 0, st, a);
  return hipGetLastError();
}

}  // namespace

// Which kernel, by the rows per expert (avg; the host knows no segment's own).
// Times in us at E = 64, K = N = 2048 and at E = 128, K = 1536, N = 512:
//   avg                          4          8          12         16         24         32
//   bf16, 16 rows, 64 columns    45 / -     47 / 20.5  50 / -     63 / 28    82 / -     - / 41
//         32 rows, 64 columns    48 / -     50 / 23.8  51 / -     54 / 25    60 / -     - / 34
//         64 x 128 tiles                                                                - / 28
//         128 x 128 tiles        52 / -     50 / 29.6  53 / -     53 / 30    54 / -     - / 31
//   fp32, 16 rows, 64 columns    45 / -     48 / 20.7  52 / -     65 / 28    85 / -     - / 42
//         32 rows, 64 columns    50 / -     50 / 23.8  53 / -     56 / 25    63 / -     - / 34
//   avg                          64         128        256        512
//   bf16, 64 x 128 tiles         71 / -     112 / -    - / 67     295 / -
//         128 x 128 tiles        64 / -     100 / -    - / 61     225 / -
//         256 x 256 tiles        69 / -     81 / -     - / 62     193 / -
//   fp32, 32 rows, 64 columns    (avg 48: 106, avg 64: 127)
//         64 x 128 tiles         90 / -     145 / -    - / 96     396 / -
//         128 x 256 tiles        85 / -     152 / -    - / 93     331 / -
// Below one row per expert 32 columns give twice the workgroups (E = 256,
// K = 2048, N = 512, 128 rows: 22.9 against 24.3; 8 rows: 6.5 against 9.4).
// Large tiles need enough of them: 3003 rows, E = 24, K = 720, N = 1040 take
// 21 (fp32) and 16.4 (bf16) with 64 x 128 tiles, 25 with 128 x 256, 17.5 with
// 128 x 128.
hipError_t launch_fp8_mm(const PlanArgs& p, const Fp8MmArgs& m, hipStream_t st) {
  f8::Args a{};
  a.a = m.a; a.sa = m.sa; a.b = m.b; a.sb = m.sb; a.c = m.c;
  a.offsets = p.offsets; a.counts = p.counts;
  a.row_token = m.gather ? p.row_token : nullptr;
  a.a_rows = m.a_rows; a.rows = m.rows; a.E = m.E;
  a.K = m.K; a.N = m.N;
  a.kb = (m.K + 127) / 128;
  const int nbn = (m.N + 127) / 128;
  a.sb_k = m.sb_out_major ? 1 : nbn;
  a.sb_n = m.sb_out_major ? a.kb : 1;
  const int64_t used = m.rows_used, E = m.E;
  const bool wide = m.out == MOE_F32;
  // (their grids, one workgroup per tile, stay below 2^32 threads)
  const bool thin = row_tiles(a, used, 16) * div_up(a.N, 32) < (1 << 24);
  if (thin && used < E) return launch_thin<1, 2, 1>(m.out, a, used, st);
  if (thin && used <= 12 * E) return launch_thin<1, 4, 1>(m.out, a, used, st);
  if (thin && used <= (wide ? 40 : 18) * E) return launch_thin<2, 4, 1>(m.out, a, used, st);
  // tiles of a size, about
  auto full = [&](int BM, int BN) { return (used / BM + 1) * div_up(m.N, BN); };
  auto bound = [&](int BM, int BN) { return row_tiles(a, used, BM) * div_up(m.N, BN); };
  const int cus = cu_count(device());
  if (wide) {
    if (m.N > 128 && full(128, 256) >= cus) return launch_tiles<128, 256, 2, 4, false, float>(a, bound(128, 256), st);
    return launch_tiles<64, 128, 1, 4, false, float>(a, bound(64, 128), st);
  }
  if (used >= 96 * E && m.N > 128 && full(256, 256) >= cus)
    return launch_tiles<256, 256, 2, 4, false, bf16_t>(a, bound(256, 256), st);
  if (used < 48 * E || full(128, 128) < cus)
    return launch_tiles<64, 128, 1, 4, false, bf16_t>(a, bound(64, 128), st);
  return launch_tiles<128, 128, 2, 2, false, bf16_t>(a, bound(128, 128), st);
}

// Weight gradients.  192 x 256 tiles (256 x 256 do not fit the registers: two
// scales per value) read less than 128 x 128 ones, where they waste little at
// the edges and there is one for every CU: 65536 rows, E = 64, 2048 x 1024
// 251 against 272 us, 262144 rows, E = 128, 1536 x 512 307 against 332; 3000
// rows, E = 16, 1040 x 720 19.4 against 16.2.
hipError_t launch_fp8_wgrad(const PlanArgs& p, int M, int N, int out, const uint8_t* qa, const float* sa,
                            const uint8_t* qb, const float* sb, void* dw, hipStream_t st) {
  f8::Args a{};
  a.a = qa; a.sa = sa; a.b = qb; a.sb = sb; a.c = dw;
  a.offsets = p.offsets; a.counts = p.counts;
  a.rows = p.cap; a.E = p.E;
  a.M = M; a.N = N;
  auto tiles = [&](int BM, int BN) { return a.E * div_up(M, BM) * div_up(N, BN); };
  if (out == MOE_F32) return launch_tiles<128, 64, 2, 2, true, float>(a, tiles(128, 64), st);
  const int64_t covered = div_up(M, 192) * 192 * div_up(N, 256) * 256;
  if (100 * covered <= 105 * (int64_t)M * N && tiles(192, 256) >= cu_count(device()))
    return launch_tiles<192, 256, 2, 4, true, bf16_t>(a, tiles(192, 256), st);
  return launch_tiles<128, 128, 2, 2, true, bf16_t>(a, tiles(128, 128), st);
}

}  // namespace moe
