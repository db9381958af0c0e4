// Launches of the E4M3 products (fp8_gemm.h).
#include <algorithm>

#include "fp8_gemm.h"
#include "launch_util.h"

namespace moe {

namespace {

template <int BM, int BN, int WM, int WN, bool WG, typename O, int LATE = 0>
hipError_t launch_tiles(const f8::Args& a, int64_t tiles, hipStream_t st) {
  using C = f8::Cfg<BM, BN, WM, WN, WG>;
  auto* k = f8::k_fp8_gemm<BM, BN, WM, WN, WG, O, LATE>;
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

// Row tiles at most: every segment with rows may end inside one.
int64_t row_tiles(const f8::Args& a, int64_t used, int BM) { return div_up(used, BM) + std::min<int64_t>(a.E, used); }

template <int RT, int FN>
hipError_t launch_thin(int out, const f8::Args& a, int64_t used, hipStream_t st) {
  const int64_t tiles = row_tiles(a, used, 16 * RT) * div_up(a.N, 16 * FN);
  if (out == MOE_BF16)
    hipLaunchKernelGGL((f8::k_fp8_thin<RT, FN, bf16_t>), dim3((unsigned)tiles), dim3(256), 0, st, a);
  else
    hipLaunchKernelGGL((f8::k_fp8_thin<RT, FN, float>), dim3((unsigned)tiles), dim3(256), 0, st, a);
  return hipGetLastError();
}

}  // namespace

// Which kernel for a row product.  The host knows the rows and the experts, not
// each expert's rows.
//
// Thin tiles or 64 x 128 ones: thin tiles have the CUs busy where there are few
// of the others, and lose with more rows per expert (their codes go through the
// bf16 matrix cores, and every 16 or 32 rows read the weights again) and with
// more tiles than the card holds at once.  us, thin / 64 x 128, at E x K x N:
//   rows per expert              2            8            16           24           32
//   bf16, 16 x 4096 x 1024       15.0 / 26.5  16.5 / 26.8  18.8 / 27.2  19.9 / 27.6  31.9 / 28.0
//         60 x 2048 x 1408       28.4 / 37.3  33.5 / 38.1  41.2 / 38.5  44.0 / 38.8
//         64 x 2048 x 2048       38.1 / 41.5  45.3 / 44.2  56.6 / 43.4  62.0 / 44.4
//         256 x 1024 x 2048      94.6 / 85.1  124 / 105    161 / 108    178 / 114
//   fp32, 16 x 4096 x 1024       15.0 / 33.6  16.5 / 33.7  18.9 / 34.1  19.7 / 34.3  31.7 / 34.8
//         60 x 2048 x 1408       28.4 / 46.6  33.9 / 46.6  41.3 / 47.1  43.9 / 47.9  56.0 / 49.1
//         256 x 1024 x 2048      94.8 / 95.6  123 / 113    160 / 117    178 / 125
// Thin tiles of 16 rows and 32, 16 and 64, 32 rows and 64 columns:
//   rows per expert              1                    4                    12
//   16 x 4096 x 1024             10.7 / 14.7 / 15.8   16.7 / 16.7 / 18.0   22.3 / 25.1 / 18.4
//   24 x 720 x 1040              5.9 / 6.1 / 6.6      6.9 / 7.6 / 8.3      7.6 / 7.7 / 8.6
//   128 x 1536 x 512             14.7 / 17.0 / 20.1   21.7 / 20.7 / 24.6
//   256 x 2048 x 512             33.3 / 30.7 / 34.2   50.8 / 45.8 / 51.2
// Returns 0 for none.
int thin_tiles(const f8::Args& a, int64_t used, bool wide, int64_t cus) {
  // (their grids, one workgroup per tile, stay below 2^32 threads)
  if (row_tiles(a, used, 16) * div_up(a.N, 32) >= (1 << 24)) return 0;
  const int64_t E = a.E, touched = std::min(E, used);
  const int64_t t = touched * div_up(a.N, 128), t64 = touched * div_up(a.N, 64);
  const int64_t most = t < cus ? (wide ? 40 : 24) : t < 4 * cus ? (wide ? 12 : 8) : t < 8 * cus ? (wide ? 8 : 3) : (wide ? 2 : 0);
  if (used > most * E) return 0;
  if ((t64 < 2 * cus && used <= 8 * E) || (t64 < 8 * cus && used <= E)) return 1;
  return used <= 10 * E ? 2 : 3;
}

// The tile that ends first: rounds of tiles over the CUs, times what a stage
// takes with its CU to itself (one) or beside another workgroup's (two), times the
// stages of the reduction and those that a tile's start and end are worth (ends).
// Fitted (us) to ten shapes from 16 x 4096 x 1024 to 256 x 512 x 128 with 16 to
// 256 rows per expert:
//          bf16    64 x 128    128 x 128    256 x 256    fp32    64 x 128    128 x 256
//   one            0.8         1.1          1.9                  0.7         1.6
//   two            1.1         1.45         -                    1.4         -
//   ends           0           1            1                    0           2
// Half of an expert's last tile is taken to be empty (a lone expert's rows are
// known).  The choice is 0.7% (bf16) and 0.4% (fp32) behind the best one, in the
// mean.  At 32 x 2048 x 1536 with 64 rows per expert 64 x 128, 128 x 128 and
// 256 x 256 take 35, 28 and 33 us, at 128 x 1536 x 512 with 128 rows 39, 39.5 and
// 31, at 64 x 2048 x 2048 with 512 rows 295, 225 and 193, at 1 x 2048 x 2048 with
// 2048 rows 20.5, 26 and 35; in fp32 64 x 128 and 128 x 256 take 19.7 and 22.7 us
// at 24 x 720 x 1040 with 125 rows, 209 and 196 at 64 x 2048 x 2048 with 256.
double tiles_time(const f8::Args& a, int64_t used, int64_t cus, int BM, int BN, double one, double two, int ends) {
  const double touched = (double)std::min<int64_t>(a.E, used);
  const double row_tiles =
      a.E == 1 ? (double)div_up(used, BM) : std::max(touched, (double)used / BM + 0.5 * touched);
  const double n = row_tiles * (double)div_up(a.N, BN);
  const double stages = a.kb + ends;
  if (two == 0.0) return std::ceil(n / (double)cus) * one * stages;
  const double rounds = std::floor(n / (2.0 * (double)cus)), rest = n - rounds * 2.0 * (double)cus;
  return (rounds * two + (rest == 0.0 ? 0.0 : rest <= (double)cus ? one : two)) * stages;
}

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
  const int64_t used = m.rows_used;
  const bool wide = m.out == MOE_F32;
  const int64_t cus = cu_count(device());
  switch (thin_tiles(a, used, wide, cus)) {
    case 1: return launch_thin<1, 2>(m.out, a, used, st);
    case 2: return launch_thin<1, 4>(m.out, a, used, st);
    case 3: return launch_thin<2, 4>(m.out, a, used, st);
  }
  auto bound = [&](int BM, int BN) { return row_tiles(a, used, BM) * div_up(m.N, BN); };
  auto time = [&](int BM, int BN, double one, double two, int ends) {
    return tiles_time(a, used, cus, BM, BN, one, two, ends);
  };
  if (wide) {
    if (time(128, 256, 1.6, 0.0, 2) < time(64, 128, 0.7, 1.4, 0))
      return launch_tiles<128, 256, 2, 4, false, float>(a, bound(128, 256), st);
    return launch_tiles<64, 128, 1, 4, false, float>(a, bound(64, 128), st);
  }
  const double t64 = time(64, 128, 0.8, 1.1, 0), t128 = time(128, 128, 1.1, 1.45, 1), t256 = time(256, 256, 1.9, 0.0, 1);
  if (t256 < std::min(t64, t128)) {
    // Gathered rows come later; spread over three more pieces their loads keep the
    // matrix cores waiting less (262144 rows, E = 64, 2048 x 2048 1.19 -> 1.16 ms);
    // rows as they lie lose by it (4096^3 66.7 -> 68.1 us, 8192^3 no change), and so do
    // smaller tiles (1 to 10%).
    if (m.gather) return launch_tiles<256, 256, 2, 4, false, bf16_t, 3>(a, bound(256, 256), st);
    return launch_tiles<256, 256, 2, 4, false, bf16_t>(a, bound(256, 256), st);
  }
  if (t128 < t64) return launch_tiles<128, 128, 2, 2, false, bf16_t>(a, bound(128, 128), st);
  return launch_tiles<64, 128, 1, 4, false, bf16_t>(a, bound(64, 128), st);
}

// Weight gradients.  192 x 256 tiles (256 x 256 do not fit the registers: two
// scales per value) read less than 128 x 128 ones, where they waste little at
// the edges and there is one for every CU; 64 x 128 ones keep more CUs busy.  us,
// 192 x 256 / 128 x 128 / 64 x 128, at rows, E, M x N:
//   65536, 64, 2048 x 1024     205 / 233 / 294     3000, 16, 1040 x 720     18.2 / 15.0 / 17.1
//   262144, 128, 1536 x 512    265 / 299 / 376     8192, 8, 1024 x 1024     23.0 / 20.0 / 22.2
//   65536, 32, 1408 x 2048     243 / 276 / 351     4096, 32, 768 x 768      19.5 / 19.6 / 19.2
//   2048, 64, 2048 x 1024      69 / 86 / 91        65536, 8, 512 x 512      99 / 67 / 51
// fp32 results take 128 x 64 tiles whatever the sizes; no choice is made.  us, 128 x 64 /
// 128 x 128:
//   65536, 64, 2048 x 1024     500 / 450           3000, 16, 1040 x 720     24.7 / 22.7
//   262144, 128, 1536 x 512    660 / 545           65536, 8, 512 x 512      76 / 103
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
  const int64_t cus = cu_count(device());
  if (100 * covered <= 110 * (int64_t)M * N && tiles(192, 256) >= cus)
    return launch_tiles<192, 256, 2, 4, true, bf16_t>(a, tiles(192, 256), st);
  if (2 * tiles(128, 128) <= cus) return launch_tiles<64, 128, 1, 4, true, bf16_t>(a, tiles(64, 128), st);
  return launch_tiles<128, 128, 2, 2, true, bf16_t>(a, tiles(128, 128), st);
}

}  // namespace moe
