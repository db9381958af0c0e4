// Products of E4M3 operands with an fp32 scale per block of 128 along the
// reduction (include/moe_ops.h: moe_fp8_mm, moe_fp8_wgrad).
//
// One stage of the reduction is one block of 128, so a stage's product of a
// wave's 16 x 16 piece is one v_mfma_f32_16x16x128_f8f6f4 that starts from
// zero, and its four results per lane join the fp32 sums by one fma each,
// times the block's scale.  (The matrix core's own block scales are powers of
// two; these are not.)  That makes four vector instructions for every matrix
// instruction of eight times their length, which the second wave of the SIMD
// fills.
//
// Precision.  The 8-bit matrix cores add eight neighbouring products at a
// time, cut off 13 bits below the largest one's leading power of two (measured:
// beside 256 * 256 a product of 2^3 counts, one of 2^2 does not, and eight
// codes further on everything counts down to 2^-7); those sums then add up in
// fp32.  Seven products may lose less than 2^-13 of the largest each: less than
// 7 * 2^-13 of sum |a b|, and on normally distributed values 1.35e-5 of the result in
// the mean square (fp32 products: 3e-7), where a bf16 result's rounding is 1.7e-3.  An fp32
// result is for callers who need more, so there the codes turn into bf16, exactly,
// and run on the bf16 matrix cores, at half their rate or less.
//
//  * Both operands are lines of 128 codes: a row's block (moe_fp8_mm: rows of
//    a, gathered or not, and rows of b) or a column's block of 128 rows
//    (moe_fp8_wgrad).  A stage goes straight into LDS, 16 bytes per lane.  Two
//    stage buffers: a stage's fragments are all in registers before its last
//    two row pieces are multiplied, so the barrier of a stage stands there, the
//    stage after next starts loading into the same buffer, and the next
//    stage's fragments are read beside those pieces' matrix instructions.
//  * The N-side operand is the MFMA's first: lane l then holds, for the row
//    l % 16 of a piece, four columns.
//  * Persistent workgroups walk the tiles expert by expert, neighbouring tiles
//    on one XCD; loading runs two stages ahead across the tiles' borders.
//
// What it reaches (one MI355X; a library product with one scale for everything:
// 2910 TFLOP/s at 8192^3): 262144 gathered rows, E = 64, K = N = 2048, bf16 result
// 1.16 to 1.19 ms, 1850 to 1900 TFLOP/s; dense 8192^3 551 us, 1990, 32768 x 2048 x 2048 128 us, 2140.
// What bounds it: of a 256 x 256 stage's 4100 cycles a SIMD's matrix instructions
// take 2048, its two waves' other vector instructions 1400 (the sums 1024 of them;
// 24 fewer of the others were 4%), the CU's LDS reads 930 (no bank conflicts); the
// waves wait for data or the barrier 34% of the time, and the card lowers its clock
// to 1.7..2.0 GHz.  (Larger pieces of a wave, one wave per SIMD, do not fit the
// registers: the vector units reach the fp32 sums only in the first half of them.)
// Without its loads, stores and sums the same loop runs at 2800 to 3100 TFLOP/s; of
// 1.24 ms the loads accounted for 0.25, the stores for 0.23, the sums for 0.12.
// Tried and slower: loads spread over the whole stage (1.40 ms), 128 x 128 tiles
// (1.57), 256 x 128 (1.69), a tile's stores beside the next tile's first stage
// (1.26), stores of whole lines after exchanging halves between lanes (1.23), stores
// past the caches (no change), staggered starts (no change), three stage buffers
// for the 64 x 128 tiles (no change: a lone workgroup's stage is bound by its
// instructions, not by the loads' latency).
// Touching the lines of the stage after next into L2: 1.20 when this took 1.21, but 2
// to 7% slower on dense products.
#pragma once

#include <type_traits>

#include "../device_common.h"
#include "ops_launch.h"

namespace moe {
namespace f8 {

typedef int i32x4_v __attribute__((ext_vector_type(4)));
typedef int i32x8_v __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) void lds_void_t;
typedef const __attribute__((address_space(3))) char* lds_ptr_t;
template <typename T> __device__ __forceinline__ T lds_ld(lds_ptr_t p) {
  return *reinterpret_cast<const __attribute__((address_space(3))) T*>(p);
}

constexpr int MAX_E = 1024;
constexpr uint32_t OOB = 0x80000000u;  // past every record count

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes, 0x00020000);
}
__device__ __forceinline__ void load16_lds(__amdgpu_buffer_rsrc_t r, char* lds, uint32_t voff, uint32_t soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void_t*)lds, 16, voff, soff, 0, 0);
}
__device__ __forceinline__ void load4_lds(__amdgpu_buffer_rsrc_t r, char* lds, uint32_t voff, uint32_t soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void_t*)lds, 4, voff, soff, 0, 0);
}
// all but the newest N vector memory operations of this wave are complete
// (loads and stores complete in the order they were issued)
template <int N>
__device__ __forceinline__ void wait_vm() {
  static_assert(N < 64, "vmcnt has six bits");
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x0F70 | (N & 15) | ((N >> 4) << 14));  // lgkmcnt, expcnt at their maximum
  asm volatile("" ::: "memory");
}

// 16 x 16 x 128 product of E4M3 operands from zero (no block scales: both
// scale operands zero selects the unscaled instruction)
__device__ __forceinline__ f32x4_v mfma128(i32x8_v a, i32x8_v b) {
  const f32x4_v z = {0.f, 0.f, 0.f, 0.f};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, z, 0, 0, 0, 0, 0, 0);
}

// One of a block's two scales, s = power(s) rest(s), the power of two kept within
// 2^-100..2^100.  The sums' factor, the product of both scales, need not be a normal number
// where they and the result are (rows of 1e-30 beside weights of 1e-9).  Codes that turn
// into bf16 take the one scale's power with them, which costs nothing there; a block's sums
// of them stay between 2^-118 and 2^125, and the rest times the other scale is below the
// normal numbers only where the result is, and finite for products below 2^228.  (In the
// 8-bit matrix instruction a power of two costs 15 to 25% of the call.)
__device__ __forceinline__ int exponent(float s) {
  return min(max((int)(__float_as_uint(s) >> 23) & 255, 127 - 100), 127 + 100);
}
__device__ __forceinline__ float power(float s) { return __uint_as_float((uint32_t)exponent(s) << 23); }
__device__ __forceinline__ float rest(float s) { return __builtin_amdgcn_ldexpf(s, 127 - exponent(s)); }

// A lane's 32 of the 128 codes of a line, as read, and as the matrix cores take
// them (as bf16: times a power of two).  Both operands place equal k in equal lanes
// and bytes, so any split of the 128 does.
template <bool EXACT> struct Frag;
template <> struct Frag<false> {
  i32x8_v v;
  __device__ __forceinline__ Frag() {}
  __device__ __forceinline__ explicit Frag(const i32x8_v r) : v(r) {}
};
template <> struct Frag<true> {
  bf16x8_v v[4];
  __device__ __forceinline__ Frag() {}
  __device__ __forceinline__ explicit Frag(const i32x8_v r, float power = 1.f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const bf16x2_v a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(r[i], power, false);
      const bf16x2_v b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(r[i], power, true);
      v[i >> 1][4 * (i & 1)] = a[0];
      v[i >> 1][4 * (i & 1) + 1] = a[1];
      v[i >> 1][4 * (i & 1) + 2] = b[0];
      v[i >> 1][4 * (i & 1) + 3] = b[1];
    }
  }
};

// 16 x 16 product over a block, from zero
__device__ __forceinline__ f32x4_v dot(const Frag<false>& a, const Frag<false>& b) { return mfma128(a.v, b.v); }
__device__ __forceinline__ f32x4_v dot(const Frag<true>& a, const Frag<true>& b) {
  f32x4_v d = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 4; ++i) d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v[i], b.v[i], d, 0, 0, 0);
  return d;
}

__device__ __forceinline__ i32x8_v join(const i32x4_v lo, const i32x4_v hi) {
  return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}
__device__ __forceinline__ i32x8_v join(const uint4 lo, const uint4 hi) {
  return i32x8_v{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
}

// Chunk c of line r of an operand's stage sits in slot c ^ key(r); the lines
// that eight neighbouring lanes read at once have eight different keys.
__device__ __forceinline__ int key_a(int r) { return r & 7; }
// N side: a lane's results are to be neighbouring columns, 16 bytes of them at
// once, so with 2-byte results the position p of piece i takes the column
// 32 (i / 2) + 8 (p / 4) + 4 (i % 2) + p % 4 of the wave's 64.
// (its lines 4 (i % 2) apart share the low bits, hence another key)
template <bool WIDE> __device__ __forceinline__ int key_b(int r) { return WIDE ? r & 7 : (r & 3) | ((r >> 1) & 4); }
template <bool WIDE> __device__ __forceinline__ int column(int i, int p) {
  return WIDE ? 16 * i + p : 32 * (i >> 1) + 8 * (p >> 2) + 4 * (i & 1) + (p & 3);
}

struct Args {
  const uint8_t* a;
  const float* sa;
  const uint8_t* b;
  const float* sb;
  void* c;
  const int32_t* offsets;    // null: one segment of `rows` rows
  const int32_t* counts;
  const int32_t* row_token;  // gathered rows of a, or null
  int a_rows, rows, E;
  int M, K, N;               // M: wgrad only
  int kb;                    // blocks of the reduction (row product)
  int sb_k, sb_n;            // strides of sb in (reduction block, column block)
};

// n rows from row o on, as far as they lie in the buffers (rows past them are never touched)
__device__ __forceinline__ int rows_in(const Args& g, int o, int n) {
  return o < 0 || o >= g.rows ? 0 : max(0, min(n, g.rows - o));
}

// BM x BN tiles, WM x WN waves.  WG: weight gradient (tiles of dw over the
// segment's blocks), else rows of c.
template <int BM, int BN, int WM, int WN, bool WG>
struct Cfg {
  static constexpr int W = WM * WN, NTH = 64 * W;
  static constexpr int TM = BM / WM, TN = BN / WN;          // a wave's share
  static constexpr int FM = TM / 16, FN = TN / 16;
  static constexpr int IA = BM / 8 / W, IB = BN / 8 / W;    // 1 KB loads per wave and stage
  static constexpr int SA_OFF = (BM + BN) * 128;
  static constexpr int SB_OFF = SA_OFF + BM * 4;
  static constexpr int SBN = WG ? BN : 64;                  // scale words of b per stage
  static constexpr int STAGE = SB_OFF + SBN * 4;
  static constexpr int SMEM = 2 * STAGE;
  static_assert(BM % (8 * W) == 0 && BN % (8 * W) == 0 && TM % 32 == 0 && TN % 32 == 0, "tile split");
  static_assert(WG || 128 % TN == 0, "a wave's columns lie in one block of 128");
  static_assert(WG ? BM / 64 + BN / 64 <= W : BM / 64 + 1 <= W, "one scale load per wave");
  static_assert(STAGE % 256 == 0, "alignment");
};

// One tile: expert, first row in its segment (weight gradient: first column of
// a), first column, stages; first row and rows of the segment from there on
// (weight gradient: of the segment).
struct Tile {
  int e, m0, n0, nk, row0, rows;
};

// LATE: that many of a stage's parts of loads go beside the next stage's first pieces.
template <int BM, int BN, int WM, int WN, bool WG, typename O, int LATE = 0>
__global__ void __launch_bounds__(64 * WM * WN, 2)
k_fp8_gemm(Args g) {
  using C = Cfg<BM, BN, WM, WN, WG>;
  constexpr bool EX = sizeof(O) == 4;  // fp32 results on the bf16 matrix cores
  constexpr int FM = C::FM, FN = C::FN;
  extern __shared__ __attribute__((aligned(1024))) char smem[];
  __shared__ int seg0[MAX_E];         // first row of each segment
  __shared__ int segn[MAX_E];         // its rows
  __shared__ int tprefix[MAX_E + 1];  // row tiles before it
  __shared__ int tok[2][WG ? 1 : BM];
  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = w / WN, wn = w % WN;
  const int NT = (g.N + BN - 1) / BN;

  // segments and the prefix of their row tiles (a weight gradient has the same
  // number of tiles for every expert)
  const int MT = WG ? (g.M + BM - 1) / BM : 0;
  {
    __shared__ int wsum[C::W];
    int carry = 0;
    for (int e0 = 0; e0 < g.E; e0 += C::NTH) {
      const int e = e0 + tid;
      int o = 0, n = 0;
      if (e < g.E) {
        o = g.offsets ? g.offsets[e] : 0;
        n = rows_in(g, o, g.offsets ? g.counts[e] : g.rows);
        seg0[e] = o;
        segn[e] = n;
      }
      const int tiles = WG ? MT : (n + BM - 1) / BM;
      int incl = e < g.E ? tiles : 0;
      for (int s = 1; s < 64; s <<= 1) {
        const int y = __shfl_up(incl, s, 64);
        if (lane >= s) incl += y;
      }
      if (lane == 63) wsum[w] = incl;
      __syncthreads();
      int base = carry, tot = 0;
      for (int x = 0; x < C::W; ++x) {
        if (x < w) base += wsum[x];
        tot += wsum[x];
      }
      if (e < g.E) tprefix[e] = base + incl - tiles;
      carry += tot;
      __syncthreads();
    }
    if (tid == 0) tprefix[g.E] = carry;
    __syncthreads();
  }
  // (a result that fits the memory has far fewer than 2^31 tiles)
  const int total = __builtin_amdgcn_readfirstlane(tprefix[g.E]) * NT;
  const int G = gridDim.x;
  const int t0 = xcd_virtual_id(blockIdx.x, G);
  if (t0 >= total) return;

  // tile t, at or behind expert e
  auto uniform = [](int v) { return __builtin_amdgcn_readfirstlane(v); };
  auto uniform_ptr = [&](const char* p) {
    const uint64_t v = reinterpret_cast<uint64_t>(p);
    return reinterpret_cast<const char*>((uint64_t)(uint32_t)uniform((int)(v >> 32)) << 32 | (uint32_t)uniform((int)v));
  };
  auto tile_at = [&](int t, int e) {
    Tile q;
    const int mg = (int)((unsigned)t / (unsigned)NT);
    q.n0 = (t - mg * NT) * BN;
    // 64 experts at a time (one by one, at LDS latency each, a first tile behind
    // 255 experts took 22 us)
    for (int n = 64; n == 64; e += n) {
      const int i = e + 1 + lane;
      n = __popcll(__ballot(i <= g.E && tprefix[min(i, g.E)] <= mg));
    }
    q.e = e;
    q.m0 = (mg - uniform(tprefix[e])) * BM;
    q.row0 = uniform(seg0[e]) + (WG ? 0 : q.m0);
    q.rows = uniform(segn[e]) - (WG ? 0 : q.m0);
    // (a segment never reaches past the last whole block of the buffers)
    q.nk = WG ? max(0, min((q.rows + 127) >> 7, (g.rows >> 7) - (q.row0 >> 7))) : g.kb;
    return q;
  };

  // ---- loading: a cursor over the stages of this workgroup's tiles ----
  const int sub = lane >> 3;  // line of a 1 KB load
  const uint32_t cha = (uint32_t)((lane & 7) ^ key_a(sub)) * 16u;
  auto chb = [&](int i) { return (uint32_t)((lane & 7) ^ key_b<EX>((C::IB * w + i) * 8 + sub)) * 16u; };
  uint32_t oa[C::IA], ob[C::IB], os;  // lane offsets of the cursor's tile
  const char *pa, *pb, *psa, *psb;
  uint32_t na, nb, nsa, nsb;          // record counts
  int lt = t0;                        // the cursor's tile, -1 behind the last one
  int lk = 0;                         // and stage
  Tile lq = tile_at(t0, 0);
  // gathered rows: the tokens of the cursor's next tile go into LDS one tile
  // ahead, into one buffer while other waves may still read the other
  int tp = 0;
  auto fetch_tokens = [&](const Tile& q) {
    if (!WG && g.row_token && w < BM / 64)
      load4_lds(rsrc(g.row_token + q.row0, (uint32_t)min(q.rows, BM) * 4u), reinterpret_cast<char*>(tok[tp] + 64 * w),
                (uint32_t)(64 * w + lane) * 4u, 0);
  };
  auto setup = [&](const Tile& q, const int* tok) {
    if constexpr (WG) {
      const int64_t blk = q.row0 >> 7;
      pa = (const char*)g.a + blk * g.M * 128;
      pb = (const char*)g.b + blk * g.N * 128;
      psa = (const char*)(g.sa + blk * g.M);
      psb = (const char*)(g.sb + blk * g.N);
      na = (uint32_t)g.M * 128u;
      nb = (uint32_t)g.N * 128u;
      nsa = (uint32_t)g.M * 4u;
      nsb = (uint32_t)g.N * 4u;
#pragma unroll
      for (int i = 0; i < C::IA; ++i) oa[i] = (uint32_t)(q.m0 + (C::IA * w + i) * 8 + sub) * 128u + cha;
#pragma unroll
      for (int i = 0; i < C::IB; ++i) ob[i] = (uint32_t)(q.n0 + (C::IB * w + i) * 8 + sub) * 128u + chb(i);
      os = w < BM / 64 ? (uint32_t)(q.m0 + 64 * w + lane) * 4u : (uint32_t)(q.n0 + 64 * (w - BM / 64) + lane) * 4u;
    } else {
      const bool gather = g.row_token != nullptr;
      // line of a for row i of the tile, relative to pa; OOB for none
      auto arow = [&](int i) -> uint32_t {
        if (i >= q.rows) return OOB;
        if (!gather) return (uint32_t)i;
        return (unsigned)tok[i] < (unsigned)g.a_rows ? (uint32_t)tok[i] : OOB;
      };
      const int64_t abase = gather ? 0 : q.row0;
      const uint32_t alines = gather ? (uint32_t)g.a_rows : (uint32_t)min(q.rows, BM);
      pa = (const char*)g.a + abase * g.K;
      na = alines * (uint32_t)g.K;
      psa = (const char*)(g.sa + abase * g.kb);
      nsa = alines * (uint32_t)g.kb * 4u;
      pb = (const char*)g.b + (int64_t)q.e * g.N * g.K;
      nb = (uint32_t)g.N * (uint32_t)g.K;
      const int nbn = (g.N + 127) >> 7;
      psb = (const char*)(g.sb + (int64_t)q.e * g.kb * nbn);
      nsb = (uint32_t)(g.kb * nbn) * 4u;
#pragma unroll
      for (int i = 0; i < C::IA; ++i) {
        const uint32_t r = arow((C::IA * w + i) * 8 + sub);
        oa[i] = r == OOB ? OOB : r * (uint32_t)g.K + cha;
      }
#pragma unroll
      for (int i = 0; i < C::IB; ++i) {
        const int n = q.n0 + (C::IB * w + i) * 8 + sub;
        ob[i] = n < g.N ? (uint32_t)n * (uint32_t)g.K + chb(i) : OOB;
      }
      if (w < BM / 64) {
        const uint32_t r = arow(64 * w + lane);
        os = r == OOB ? OOB : r * (uint32_t)g.kb * 4u;
      } else {
        const int nblk = (q.n0 >> 7) + lane;
        os = lane < (BN + 127) / 128 && nblk < nbn ? (uint32_t)(nblk * g.sb_n) * 4u : OOB;
      }
    }
  };
  // A stage's loads.  begin starts the cursor's stage in buffer `par`: on entry lq
  // is the cursor's tile (lk == 0: not set up yet) or, for lk > 0, the next one.
  // The loads then come in PARTS, since every wave's load instructions in one
  // burst would keep the matrix cores waiting for their issue; the last part
  // moves the cursor on.
  //   EARLY: the columns' codes of a stage are all in registers when it starts, so
  // after a second barrier there, begin loads the stage after next's into their
  // place, and only the rows' codes wait for the stage's end.  It pays for the
  // weight gradient (65536 rows, E = 64, 2048 x 1024, with both quantizers 360 -> 335
  // us), not for the row product (262144 rows 1.22 -> 1.21 ms, dense 8192^3 590 ->
  // 600 us).
  constexpr bool EARLY = WG;  // (never with gathered rows: begin's tokens would have to be waited for too)
  constexpr int PARTS = FN + LATE;
  static_assert(LATE == 0 || (!EARLY && LATE <= FM - 2), "the parts have pieces to go beside");
  int lnk = 0;
  auto load_cols = [&](int i, int par, uint32_t k0) {
    const __amdgpu_buffer_rsrc_t rb = rsrc(uniform_ptr(pb), (uint32_t)uniform((int)nb));
    load16_lds(rb, smem + par * C::STAGE + BM * 128 + (C::IB * w + i) * 1024, ob[i], k0);
  };
  auto begin = [&](int par) -> bool {
    if (lt < 0) return false;
    if (lk == 0) {
      // the next tile with stages (a weight gradient may have none)
      while (WG && lq.nk == 0) {
        lt += G;
        if (lt >= total) {
          lt = -1;
          return false;
        }
        lq = tile_at(lt, lq.e);
      }
      setup(lq, tok[tp]);
      tp ^= 1;
      lnk = lq.nk;
      if (lt + G < total) {
        lq = tile_at(lt + G, lq.e);
        fetch_tokens(lq);
      }
    }
    if constexpr (EARLY) {
#pragma unroll
      for (int i = 0; i < C::IB; ++i) load_cols(i, par, 0u);
    }
    return true;
  };
  auto load_part = [&](int part, int par) {
    if (lt < 0) return;
    char* st = smem + par * C::STAGE;
    // (a descriptor shared by the parts would travel through vector registers)
    const __amdgpu_buffer_rsrc_t ra = rsrc(uniform_ptr(pa), (uint32_t)uniform((int)na));
    const uint32_t k0 = WG ? 0u : (uint32_t)lk * 128u;
    // a shorter last block, the tile's last: its missing codes are zeros on both sides
    if (!WG && part == 0 && k0 + 128u > (uint32_t)g.K) {
      asm volatile("");  // a branch, not selects in every stage
#pragma unroll
      for (int i = 0; i < C::IA; ++i) oa[i] = cha < (uint32_t)g.K - k0 ? oa[i] : OOB;
#pragma unroll
      for (int i = 0; i < C::IB; ++i) ob[i] = chb(i) < (uint32_t)g.K - k0 ? ob[i] : OOB;
    }
    constexpr int L = C::IA + (EARLY ? 0 : C::IB);
#pragma unroll
    for (int i = 0; i < C::IA; ++i)
      if (part == i * PARTS / L)
        load16_lds(ra, st + (C::IA * w + i) * 1024, oa[i], k0);
    if constexpr (!EARLY) {
#pragma unroll
      for (int i = 0; i < C::IB; ++i)
        if (part == (C::IA + i) * PARTS / L) load_cols(i, par, k0);
    }
    if (part != PARTS - 1) return;
    auto rsa = [&] { return rsrc(uniform_ptr(psa), (uint32_t)uniform((int)nsa)); };
    auto rsb = [&] { return rsrc(uniform_ptr(psb), (uint32_t)uniform((int)nsb)); };
    if constexpr (WG) {
      if (w < BM / 64) load4_lds(rsa(), st + C::SA_OFF + w * 256, os, 0);
      else if (w < BM / 64 + BN / 64) load4_lds(rsb(), st + C::SB_OFF + (w - BM / 64) * 256, os, 0);
      pa += na; pb += nb; psa += nsa; psb += nsb;  // the next block's
    } else {
      if (w < BM / 64) load4_lds(rsa(), st + C::SA_OFF + w * 256, os, (uint32_t)lk * 4u);
      else if (w == BM / 64) load4_lds(rsb(), st + C::SB_OFF, os, (uint32_t)(lk * g.sb_k) * 4u);
    }
    if (++lk == lnk) {
      lk = 0;
      lt = lt + G < total ? lt + G : -1;
    }
    lt = uniform(lt);
    lk = uniform(lk);
  };
  auto load_stage = [&](int par) {
    begin(par);
#pragma unroll
    for (int part = 0; part < PARTS; ++part) load_part(part, par);
  };

  // ---- computing: row pieces j of a stage in turn.  The sums of a piece run
  // beside the matrix instructions of the next one.  The last two pieces go
  // column by column, so that a column's codes of the next stage can be read as
  // soon as its last two instructions are out. ----
  const int la = wm * C::TM + (lane & 15);                 // line of a's piece 0
  const int lb = wn * C::TN + column<EX>(0, lane & 15);    // of b's piece 0
  // the two chunks of a line and the scales in stage buffer 0 (as LDS pointers: from
  // offsets the base would be added in every stage)
  auto slot = [&](int c, int key) { return (c ^ key) * 16; };
  const int h = lane >> 4, ka = key_a(lane & 15), kbl = key_b<EX>(column<EX>(0, lane & 15));
  const lds_ptr_t stage = (lds_ptr_t)smem;
  lds_ptr_t al = stage + la * 128 + slot(h, ka), ah = stage + la * 128 + slot(h + 4, ka);
  lds_ptr_t bl = stage + (BM + lb) * 128 + slot(h, kbl), bh = stage + (BM + lb) * 128 + slot(h + 4, kbl);
  lds_ptr_t sal = stage + C::SA_OFF + la * 4;
  lds_ptr_t sbl = stage + C::SB_OFF + (WG ? wn * C::TN + column<EX>(0, 4 * h) : (wn * C::TN) >> 7) * 4;
  int step = C::STAGE;  // to the other buffer
  auto other_buffer = [&] {
    al += step; ah += step; bl += step; bh += step; sal += step; sbl += step;
    step = -step;
  };
  i32x8_v nr[FN];   // codes of the next stage's columns
  auto read_cols = [&](int i) {
    nr[i] = join(lds_ld<i32x4_v>(bl + column<EX>(i, 0) * 128), lds_ld<i32x4_v>(bh + column<EX>(i, 0) * 128));
  };
  auto read_row = [&](int j, i32x8_v& m, float& sc) {
    m = join(lds_ld<i32x4_v>(al + j * 2048), lds_ld<i32x4_v>(ah + j * 2048));
    sc = lds_ld<float>(sal + j * 64);
  };

  const bool gathered = !WG && g.row_token != nullptr;
  fetch_tokens(lq);
  if (gathered) {
    wait_vm<0>();
    lds_sync();
  }
  load_stage(0);
  if (gathered && lk == 0) {  // the second stage is the next tile's: its tokens
    wait_vm<0>();
    lds_sync();
  }
  load_stage(1);
  wait_vm<0>();
  lds_sync();
  i32x8_v mr;        // codes and scale of the next row piece
  float sm, sbn = 0.f;
  f32x4_v sn[WG ? FN : 1];
#pragma unroll
  for (int i = 0; i < FN; ++i) read_cols(i);
  read_row(0, mr, sm);
  if constexpr (!WG) sbn = lds_ld<float>(sbl);

  // A whole tile's stores are issued unconditionally, so their number is known
  // and the wait for the next stage's loads, which are older, can leave them be.
  constexpr int STORES = FM * FN / (EX ? 1 : 2);
  // Of the two waves of a SIMD one goes first, so that they do not both wait for
  // issue and then both for data (262144 rows, K = N = 2048, E = 64 1.20 -> 1.17 ms;
  // weight gradients the same either way).
  if constexpr (C::W == 8 && !WG) {
    if (w >= 4) __builtin_amdgcn_s_setprio(1);
  }
  bool stores = false;
  bool late = false;  // the last begun stage's LATE parts are still to come
  int par = 0;
  Tile q = tile_at(t0, 0);
  for (int t = t0; t < total; t += G) {
    if (t != t0) q = tile_at(t, q.e);
    f32x4_v acc[FN][FM], d[FN];
    float sp = 0.f;  // scale of the piece whose sums are due
#pragma unroll
    for (int i = 0; i < FN; ++i) {
#pragma unroll
      for (int j = 0; j < FM; ++j) acc[i][j] = f32x4_v{0.f, 0.f, 0.f, 0.f};
      d[i] = f32x4_v{0.f, 0.f, 0.f, 0.f};
      if constexpr (WG) sn[i] = f32x4_v{0.f, 0.f, 0.f, 0.f};
    }
    auto add = [&](const f32x4_v& v, float sc, int i, int j) {  // piece (i, j) joins the sums
#pragma unroll
      for (int x = 0; x < 4; ++x) acc[i][j][x] = fmaf(v[x], WG ? sc * sn[i][x] : sc, acc[i][j][x]);
      // stays here: the compiler would gather the sums behind the branch of
      // the next loads, and their summands with them
      asm volatile("" : "+v"(acc[i][j]));
    };
#pragma unroll 1
    for (int k = 0; k < q.nk; ++k) {
      Frag<EX> nf[FN];
#pragma unroll
      for (int i = 0; i < FN; ++i) {
        if constexpr (EX && !WG) nf[i] = Frag<EX>(nr[i], power(sbn));
        else nf[i] = Frag<EX>(nr[i]);
      }
      const float sbk = WG ? 1.f : EX ? rest(sbn) : sbn;
      // a row piece as the matrix cores take it, and its sums' factor (weight gradient: of two)
      auto row_frag = [&](const i32x8_v& r, float sc) {
        if constexpr (EX && WG) return Frag<EX>(r, power(sc));
        else return Frag<EX>(r);
      };
      auto row_scale = [&](float sc) { return !WG ? sc * sbk : EX ? rest(sc) : sc; };
      i32x8_v mx;
      float sx = 0.f;
      bool sent = false;  // begin's loads are under way
#pragma unroll
      for (int j = 0; j < FM - 2; ++j) {
        const Frag<EX> mf = row_frag(mr, sm);
        const float sj = row_scale(sm);
        if (EARLY && j == 1) {
          lds_sync();  // every wave has read its columns of this stage
          sent = begin(par);
        }
        if (j < LATE && late) load_part(FN + j, par ^ 1);
        read_row(j + 1, mr, sm);
        if (j == FM - 3) read_row(FM - 1, mx, sx);
#pragma unroll
        for (int i = 0; i < FN; ++i) {
          add(d[i], sp, i, (j + FM - 1) % FM);
          d[i] = dot(nf[i], mf);
          __builtin_amdgcn_sched_barrier(0);
          if constexpr (WG) {
            if (j == 0) sn[i] = lds_ld<f32x4_v>(sbl + column<EX>(i, 0) * 4);
          }
        }
        sp = sj;
      }
      const Frag<EX> m0 = row_frag(mr, sm), m1 = row_frag(mx, sx);
      const float s0 = row_scale(sm), s1 = row_scale(sx);
      // This stage is read; the next one is there once everybody's loads are: all
      // but begin's and the stores, which are newer.
      if (sent) {
        if (stores) wait_vm<STORES + C::IB>();
        else wait_vm<C::IB>();
      } else if (stores) {
        wait_vm<STORES>();
      } else {
        wait_vm<0>();
      }
      stores = false;
      lds_sync();
      other_buffer();
      read_row(0, mr, sm);
      if constexpr (!WG) sbn = lds_ld<float>(sbl);
      if constexpr (!EARLY) late = begin(par);
      f32x4_v last;
#pragma unroll
      for (int i = 0; i < FN; ++i) {
        load_part(i, par);
        add(d[i], sp, i, FM - 3);
        const f32x4_v v = dot(nf[i], m0);
        __builtin_amdgcn_sched_barrier(0);
        if (i > 0) add(last, s0, i - 1, FM - 2);
        last = v;
        d[i] = dot(nf[i], m1);
        __builtin_amdgcn_sched_barrier(0);
        read_cols(i);
      }
      add(last, s0, FN - 1, FM - 2);
      sp = s1;
      par ^= 1;
    }
    if (LATE > 0 && late) {  // before the stores, which the next wait leaves be
#pragma unroll
      for (int n = 0; n < LATE; ++n) load_part(FN + n, par ^ 1);
      late = false;
    }
#pragma unroll
    for (int i = 0; i < FN; ++i) add(d[i], sp, i, FM - 1);

    // results: lane l holds the row l % 16 of a piece
    const int left = WG ? g.M - q.m0 : q.rows;
    const int64_t crow0 = WG ? (int64_t)q.e * g.M + q.m0 : (int64_t)q.row0;
    const int c0 = q.n0 + wn * C::TN + column<EX>(0, 4 * (lane >> 4));
    O* const out = reinterpret_cast<O*>(g.c) + (crow0 + la) * g.N + c0;
    auto store = [&](auto whole) {
#pragma unroll
      for (int j = 0; j < FM; ++j) {
        O* row = out + (int64_t)(16 * j) * g.N;
        if (!whole && la + 16 * j >= left) continue;
#pragma unroll
        for (int i = 0; i < FN; i += EX ? 1 : 2) {
          const int n = column<EX>(i, 0);
          if (!whole && c0 + n >= g.N) continue;
          const f32x4_v u = acc[i][j];
          if constexpr (EX) {
            *reinterpret_cast<float4*>(row + n) = make_float4(u[0], u[1], u[2], u[3]);
          } else {
            const f32x4_v v = acc[i + 1][j];
            *reinterpret_cast<uint4*>(row + n) =
                make_uint4(f2bf2(u[0], u[1]), f2bf2(u[2], u[3]), f2bf2(v[0], v[1]), f2bf2(v[2], v[3]));
          }
        }
      }
    };
    stores = left >= BM && q.n0 + BN <= g.N;
    if (stores) store(std::true_type());
    else store(std::false_type());
  }
}

// Row product for segments of few rows (decode): the weights' bytes are all the
// work, and every touched expert's are read once, straight into registers.  A
// workgroup takes 16 RT rows of a segment and 16 FN columns; its four waves split
// the reduction's blocks (wave w: blocks w, w + 4, ...) and add up their sums in wave
// order.  The matrix work is small, so it runs on the bf16 matrix cores whatever the
// result's type.  Bound by the weights' bytes: 8 rows of 8 experts of K = 7168, N = 4096
// 38.9 us (6.0 TB/s), 512 rows over 64 experts of K = N = 2048 43.7 us (6.1 TB/s), 128 rows
// over 101 of 256 experts of K = 2048, N = 512 23 us (4.7 TB/s: about 4 us are launch
// and look-up).
template <int RT, int FN, typename O>
__global__ void __launch_bounds__(256)
k_fp8_thin(Args g) {
  constexpr int BN = 16 * FN, BM = 16 * RT;
  __shared__ float part[3][RT][FN][64][4];
  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int NT = (g.N + BN - 1) / BN;
  const int mg = (int)(blockIdx.x / (unsigned)NT), n0 = (int)(blockIdx.x % (unsigned)NT) * BN;

  // The row tile's segment: lanes scan `per` experts each, four at a time
  // (loads of four in flight; up to 256 experts they stay in registers).
  const int per = (g.E + 63) >> 6;
  int first[4], rws[4];
  int mine = 0;
  for (int x0 = 0; x0 < per; x0 += 4) {
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int e = lane * per + x0 + x;
      const bool is = x0 + x < per && e < g.E;
      first[x] = is && g.offsets ? g.offsets[e] : 0;
      rws[x] = is ? (g.offsets ? g.counts[e] : g.rows) : 0;
    }
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      rws[x] = rows_in(g, first[x], rws[x]);
      mine += (rws[x] + BM - 1) / BM;
    }
  }
  int incl = mine;
  for (int s = 1; s < 64; s <<= 1) {
    const int y = __shfl_up(incl, s, 64);
    if (lane >= s) incl += y;
  }
  const uint64_t past = __ballot(incl > mg);
  if (past == 0) return;  // no such tile
  const int src = __builtin_amdgcn_readfirstlane(__builtin_ctzll(past));
  int left = mg - (__builtin_amdgcn_readlane(incl, src) - __builtin_amdgcn_readlane(mine, src));
  int e = src * per, n = 0, row0 = 0;
  if (per <= 4) {
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int nx = __builtin_amdgcn_readlane(rws[x], src), tiles = (nx + BM - 1) / BM;
      if (left >= 0 && left < tiles) {
        e = src * per + x;
        n = nx;
        row0 = __builtin_amdgcn_readlane(first[x], src) + left * BM;
        n -= left * BM;
        left = -1;
      }
      if (left >= 0) left -= tiles;
    }
  } else {
    for (;; ++e) {
      row0 = __builtin_amdgcn_readfirstlane(g.offsets[e]);
      n = rows_in(g, row0, __builtin_amdgcn_readfirstlane(g.counts[e]));
      const int tiles = (n + BM - 1) / BM;
      if (left < tiles) break;
      left -= tiles;
    }
    row0 += left * BM;
    n -= left * BM;
  }
  e = __builtin_amdgcn_readfirstlane(e);
  row0 = __builtin_amdgcn_readfirstlane(row0);
  const int rows = min(__builtin_amdgcn_readfirstlane(n), BM);

  const int p = lane & 15, h = lane >> 4;
  // rows and columns past the end repeat the last one (their results are dropped)
  const uint8_t* pa[RT];
  const float* psa[RT];
  bool real[RT];
  int64_t row[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    row[r] = row0 + min(16 * r + p, rows - 1);
    if (g.row_token) row[r] = g.row_token[row[r]];
  }
  const uint8_t* pb[FN];
#pragma unroll
  for (int i = 0; i < FN; ++i) pb[i] = g.b + ((int64_t)e * g.N + min(n0 + 16 * i + p, g.N - 1)) * g.K + 16 * h;
  const float* psb = g.sb + (int64_t)e * g.kb * ((g.N + 127) >> 7) + (int64_t)(n0 >> 7) * g.sb_n;

  // Block k's loads: none under a condition; past the reduction they read its
  // first codes, and both sides' become zeros later.
  uint4 ra[RT][2], rb[FN][2];
  float sa[RT], sb;
  auto from = [&](int k, int c) {  // this lane's chunk: 16 h further on
    const int at = k * 128 + 64 * c;
    return at + 16 * h < g.K ? at : -16 * h;
  };
  auto load_b = [&](int k) {
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int i = 0; i < FN; ++i) rb[i][c] = *reinterpret_cast<const uint4*>(pb[i] + from(k, c));
    sb = psb[(int64_t)min(k, g.kb - 1) * g.sb_k];
  };
  auto load_a = [&](int k) {
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int r = 0; r < RT; ++r) ra[r][c] = *reinterpret_cast<const uint4*>(pa[r] + from(k, c));
#pragma unroll
    for (int r = 0; r < RT; ++r) sa[r] = psa[r][min(k, g.kb - 1)];
  };
  load_b(w);  // (on the way while the tokens arrive)
  __builtin_amdgcn_sched_barrier(0);
  bool ghosts = false;
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    // a token that does not exist counts as zeros: in place of its codes, which are
    // then row 0's and may be NaN, and of their scales
    real[r] = (uint64_t)row[r] < (uint64_t)g.a_rows;
    ghosts |= __any(!real[r]);
    if (!real[r]) row[r] = 0;
    pa[r] = g.a + row[r] * g.K + 16 * h;
    psa[r] = g.sa + row[r] * g.kb;
  }
  load_a(w);

  f32x4_v acc[RT][FN];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int i = 0; i < FN; ++i) acc[r][i] = f32x4_v{0.f, 0.f, 0.f, 0.f};
  for (int k = w; k < g.kb; k += 4) {
    if (k > w) {
      load_b(k);
      load_a(k);
    }
    __builtin_amdgcn_sched_barrier(0);
    if ((k + 1) * 128 > g.K || ghosts) {
      const uint4 z = make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const bool past = k * 128 + 64 * c + 16 * h >= g.K;
#pragma unroll
        for (int i = 0; i < FN; ++i)
          if (past) rb[i][c] = z;
#pragma unroll
        for (int r = 0; r < RT; ++r)
          if (past || !real[r]) ra[r][c] = z;
      }
    }
    Frag<true> mf[RT];
    float sc[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      mf[r] = Frag<true>(join(ra[r][0], ra[r][1]));
      sc[r] = real[r] ? sa[r] * rest(sb) : 0.f;
    }
#pragma unroll
    for (int i = 0; i < FN; ++i) {
      const Frag<true> nf(join(rb[i][0], rb[i][1]), power(sb));
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        const f32x4_v d = dot(nf, mf[r]);
#pragma unroll
        for (int x = 0; x < 4; ++x) acc[r][i][x] = fmaf(d[x], sc[r], acc[r][i][x]);
      }
    }
  }
  if (w > 0)
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int i = 0; i < FN; ++i) *reinterpret_cast<f32x4_v*>(part[w - 1][r][i][lane]) = acc[r][i];
  __syncthreads();
  if (w > 0) return;
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    const int m = 16 * r + p;
    if (m >= rows) continue;
    O* out = reinterpret_cast<O*>(g.c) + ((int64_t)row0 + m) * g.N;
#pragma unroll
    for (int i = 0; i < FN; ++i) {
      f32x4_v v = acc[r][i];
#pragma unroll
      for (int x = 0; x < 3; ++x) v += *reinterpret_cast<const f32x4_v*>(part[x][r][i][lane]);
      const int c = n0 + 16 * i + 4 * h;
      if (c >= g.N) continue;
      if constexpr (sizeof(O) == 2) *reinterpret_cast<uint2*>(out + c) = make_uint2(f2bf2(v[0], v[1]), f2bf2(v[2], v[3]));
      else *reinterpret_cast<float4*>(out + c) = make_float4(v[0], v[1], v[2], v[3]);
    }
  }
}

}  // namespace f8
}  // namespace moe
