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

// tiles of a row product, at most (every segment may end inside one)
int64_t row_tiles(const f8::Args& a, int BM, int BN) {
  return (div_up(a.rows, BM) + std::min(a.E, a.rows)) * div_up(a.N, BN);
}
int64_t wgrad_tiles(const f8::Args& a, int BM, int BN) { return a.E * div_up(a.M, BM) * div_up(a.N, BN); }

}  // namespace

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
  if (m.out == MOE_F32) return launch_tiles<128, 64, 2, 2, false, float>(a, row_tiles(a, 128, 64), st);
  static const char* v = getenv("F8V");
  if (v && v[0] == '1') return launch_tiles<128, 128, 2, 2, false, bf16_t>(a, row_tiles(a, 128, 128), st);
  if (v && v[0] == '2') return launch_tiles<256, 128, 4, 2, false, bf16_t>(a, row_tiles(a, 256, 128), st);
  return launch_tiles<256, 256, 2, 4, false, bf16_t>(a, row_tiles(a, 256, 256), st);
}

hipError_t launch_fp8_wgrad(const PlanArgs& p, int M, int N, int out, const uint8_t* qa, const float* sa,
                            const uint8_t* qb, const float* sb, void* dw, hipStream_t st) {
  f8::Args a{};
  a.a = qa; a.sa = sa; a.b = qb; a.sb = sb; a.c = dw;
  a.offsets = p.offsets; a.counts = p.counts;
  a.rows = p.cap; a.E = p.E;
  a.M = M; a.N = N;
  if (out == MOE_F32) return launch_tiles<128, 64, 2, 2, true, float>(a, wgrad_tiles(a, 128, 64), st);
  static const char* v = getenv("F8V");
  if (v && v[0] == '1') return launch_tiles<128, 128, 2, 2, true, bf16_t>(a, wgrad_tiles(a, 128, 128), st);
  if (v && v[0] == '2') return launch_tiles<256, 128, 4, 2, true, bf16_t>(a, wgrad_tiles(a, 256, 128), st);
  if (v && v[0] == '3') return launch_tiles<128, 256, 2, 4, true, bf16_t>(a, wgrad_tiles(a, 128, 256), st);
  return launch_tiles<256, 256, 2, 4, true, bf16_t>(a, wgrad_tiles(a, 256, 256), st);
}

}  // namespace moe
