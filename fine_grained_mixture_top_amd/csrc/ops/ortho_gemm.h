// Products of the matrices that orthogonalise an update (include/moe_step_ops.h:
// moe_orthogonalize).
//
// Numbers.  The matrices of the iteration are fp32 numbers times a power of two,
// held as the sum of two fp16 numbers (22 bits: the second holds what the first's
// rounding left), and a product of two of them is three fp16 products summed in
// fp32, hi hi + hi lo + lo hi; the fourth is below 2^-22 of the product.  The fp16
// matrix cores do that at a third of 2.5 PFLOP/s where the fp32 ones reach 0.16.
// bf16 input needs one fp16 number per value (its 8 bits fit, scaled by a power of
// two), so products with it take one or two.
//
// Layout.  Both operands of C = A B^T are rows with the reduction contiguous,
// padded with zeros to a multiple of 64: one part, the fp16 numbers themselves; two
// parts, lines of 128 bytes with 32 numbers' hi and then their lo.
#pragma once

#include "lds_stage.h"

namespace moe {
namespace ortho {

constexpr int NORM_PARTS = 64;    // partial sums of a matrix's norm at most
constexpr int X_EXP = 13;         // X's norm in fp16 parts lies in [2^13, 2^14)
constexpr int MAX_STEPS = 64;

typedef _Float16 f16x8_v __attribute__((ext_vector_type(8)));
typedef _Float16 f16x4_v __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_v __attribute__((ext_vector_type(2)));

// x as hi + lo.  (x has to be the one rounded fp32 number for both: the compiler would
// round a product straight to fp16 for the hi that is stored and take the lo from another)
__device__ __forceinline__ void split(float x, _Float16& hi, _Float16& lo) {
  asm("" : "+v"(x));
  hi = (_Float16)x;
  lo = (_Float16)(x - (float)hi);
}

// Four neighbouring lanes hold four numbers each, a 4 x 4 block of 16-bit values by rows;
// by columns afterwards.
__device__ __forceinline__ f16x4_v turn4(const f16x4_v v, int lane) {
  const u32x2_v d = __builtin_bit_cast(u32x2_v, v);
  auto swap1 = [](uint32_t x) { return (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0xB1, 15, 15, true); };  // lane ^ 1
  auto swap2 = [](uint32_t x) { return (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x4E, 15, 15, true); };  // lane ^ 2
  const uint32_t o0 = swap1(d[0]), o1 = swap1(d[1]);
  // columns 0 and 2 of two rows in even lanes, 1 and 3 in odd ones
  const uint32_t pick = lane & 1 ? 0x03020706u : 0x05040100u;
  const uint32_t e0 = __builtin_amdgcn_perm(o0, d[0], pick), e1 = __builtin_amdgcn_perm(o1, d[1], pick);
  const bool high = lane & 2;
  const uint32_t got = swap2(high ? e0 : e1);
  return __builtin_bit_cast(f16x4_v, high ? u32x2_v{got, e1} : u32x2_v{e0, got});
}

// A 16 x 16 piece on the diagonal of a symmetric matrix: lane p + 16 h has four numbers of row p
// from column 4 h on, and gets those above the diagonal from the lanes that hold their mirror.
__device__ __forceinline__ f16x4_v lower_mirrored(const f16x4_v v, int lane) {
  const int p = lane & 15, h = lane >> 4;
  const u32x2_v t = __builtin_bit_cast(u32x2_v, turn4(v, lane));  // row 4 h + p % 4 from column p / 4 * 4 on
  const int from = ((p >> 2) * 16 + 4 * h + (p & 3)) * 4;
  const u32x2_v row = {(uint32_t)__builtin_amdgcn_ds_bpermute(from, (int)t[0]),
                       (uint32_t)__builtin_amdgcn_ds_bpermute(from, (int)t[1])};
  const f16x4_v m = __builtin_bit_cast(f16x4_v, row);
  f16x4_v o;
#pragma unroll
  for (int x = 0; x < 4; ++x) o[x] = 4 * h + x > p ? m[x] : v[x];
  return o;
}

// bytes of a row of n numbers in `parts` parts
__host__ __device__ inline int64_t pitch(int64_t n, int parts) { return (n + 63) / 64 * 128 * parts; }
// byte of number i of a row of two parts (its lo is 64 bytes further on)
__device__ __forceinline__ int64_t at2(int i) { return (int64_t)(i >> 5) * 128 + (i & 31) * 2; }

// One product per matrix of the batch.  c = alpha * acc, and where d is given
// + beta * d + diag * I; alpha times alpha_e[matrix] (power_e: its square) when given.
struct Job {
  const char* a;
  const char* b;
  char* c;
  const char* d;
  float alpha, beta, diag;
};

struct Args {
  Job job[2];
  int jobs, batch;
  const float* alpha_e;
  bool square;              // alpha_e squared
  int ra, rb;               // rows of a and b (of c, and its columns)
  int stages;
  int64_t sa, sb, sc;       // bytes from one matrix to the next
  int pa, pb, pc;           // bytes of a row (pc: of c, in two parts)
  // results of the last product
  void* o;
  int64_t so;               // elements from one matrix to the next
  // products between groups of steps: c in two parts, and its transpose
  char* ct;
  int64_t sct;
  int pct;
};

enum Epi { SYM, SPLIT, OUT };

template <int BM, int BN, int WM, int WN, int BUFS, int PA, int PB>
struct Cfg {
  static constexpr int W = WM * WN, NTH = 64 * W;
  static constexpr int TM = BM / WM, TN = BN / WN, FM = TM / 16, FN = TN / 16;
  // one part on both sides: 64 numbers of the reduction per stage, else 32
  static constexpr bool WIDE = PA == 1 && PB == 1;
  static constexpr int LA = WIDE || PA == 2 ? 128 : 64, LB = WIDE || PB == 2 ? 128 : 64;  // bytes of a line per stage
  static constexpr int IA = BM * LA / 1024 / W, IB = BN * LB / 1024 / W;                  // 1 KB loads per wave
  static constexpr int STAGE = BM * LA + BN * LB;
  // X X^T of one part is summed in pieces of 512, so that a long sum is rounded once for each of
  // those and not for every eight products: 129 x 50000, 317 -> 337 us, error 3.4e-3 -> 5.0e-4; 256 x 1536
  // the same time, 4.8e-4 -> 3.0e-4 (but for 256 x 256 tiles, whose registers are full)
  static constexpr bool PIECES = WIDE && FM * FN <= 16;
  static constexpr int PIECE = 8;
  static constexpr int HALF = TM * TN * 2;  // bytes of half of a wave's results
  static constexpr int SMEM = BUFS * STAGE > W * HALF ? BUFS * STAGE : W * HALF;
  static_assert(SMEM <= 160 * 1024 && (BUFS - 2) * (IA + IB) < 64, "LDS, and outstanding loads");
  static_assert(BM * LA % (1024 * W) == 0 && BN * LB % (1024 * W) == 0, "loads per wave");
};

// The 16-byte chunk c of line r of a stage lies in slot c ^ key(r), so that eight
// lanes that read a chunk of eight neighbouring lines hit eight different ones.
template <int LINE> __device__ __forceinline__ int key(int r) { return LINE == 128 ? r & 7 : (r >> 1) & 3; }

// waits until at most the newest min(N, n) stages of L loads each are outstanding
template <int N, int L>
__device__ __forceinline__ void wait_stages(int n) {
  if constexpr (N > 0) {
    if (n < N) {
      wait_stages<N - 1, L>(n);
      return;
    }
  }
  wait_vm<N * L>();
}

// A tile's stages go through BUFS buffers, loaded straight into LDS; matrix instructions
// bound large calls (64 symmetric products of 2048 x 2048 in two parts 1542 us, 1200
// TFLOP/s, where the card's power holds the clock down), loads and results small ones
// (128 of 256 x 256 21 us, of which the instructions are 5).
//   FINE: the two products with a lo, which are small, have sums of their own, added once at
// the end; a matrix instruction rounds its sum four times (eight products at a time), so
// four roundings of a large sum take the place of twelve per 32 of the reduction.  Error of
// five fp32 steps of 720 x 1040 against 64 bits, without and with it: 3.5e-6 and 2.1e-6 (fp32
// products 2.4e-6).  (The sums of every stage added
// to the large ones instead: 2.3e-6, and vector instructions between the matrix ones, 1137 us in
// place of 1069 for 24 of 720 x 1040.)
template <int BM, int BN, int WM, int WN, int BUFS, int PA, int PB, bool FINE, Epi EPI, typename O>
__global__ void __launch_bounds__(64 * WM * WN, 2)
k_ortho_gemm(Args g) {
  using C = Cfg<BM, BN, WM, WN, BUFS, PA, PB>;
  constexpr int FM = C::FM, FN = C::FN;
  static_assert(!FINE || (PA == 2 && PB == 2 && FM * FN <= 16), "products with a lo on both sides, registers");
  extern __shared__ __attribute__((aligned(1024))) char smem[];
  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = w / WN, wn = w % WN;

  // ---- the tile: matrix by matrix, a matrix's tiles on one XCD ----
  const int MT = (g.ra + BM - 1) / BM, NT = (g.rb + BN - 1) / BN;
  const int per = EPI == SYM ? MT * (MT + 1) / 2 : MT * NT;
  int id = xcd_virtual_id(blockIdx.x, gridDim.x);
  if (id >= per * g.jobs * g.batch) return;
  const int e = id / (per * g.jobs);
  id -= e * per * g.jobs;
  const int jb = id / per;
  id -= jb * per;
  const Job& job = g.job[jb];
  int ti, tj;
  if constexpr (EPI == SYM) {  // the lower triangle, row by row
    ti = (int)((sqrtf(8.f * (float)id + 1.f) - 1.f) * 0.5f);
    while (ti * (ti + 1) / 2 > id) --ti;
    while ((ti + 1) * (ti + 2) / 2 <= id) ++ti;
    tj = id - ti * (ti + 1) / 2;
  } else {
    ti = id / NT;
    tj = id - ti * NT;
  }
  const int m0 = ti * BM, n0 = tj * BN;

  // A symmetric product's tile on the diagonal, and a wave whose pieces all lie above it: it only
  // loads (128 x 256 x 1536 619 -> 576 us; in tiles of 64 loads bound, 1 x 512 x 512 157.6 and 161.6).
  const bool diagonal = EPI == SYM && ti == tj, above = BM > 64 && diagonal && wn * C::TN >= (wm + 1) * C::TM;

  // ---- loads ----
  const __amdgpu_buffer_rsrc_t ra = rsrc(job.a + e * g.sa, (uint32_t)(g.ra * (int64_t)g.pa));
  const __amdgpu_buffer_rsrc_t rb = rsrc(job.b + e * g.sb, (uint32_t)(g.rb * (int64_t)g.pb));
  auto offset = [&](auto line, int i, int first, int rows, int pitch) -> uint32_t {
    constexpr int LINE = decltype(line)::value, SLOTS = LINE / 16;
    const int r = i * (1024 / LINE) + lane / SLOTS;  // line of the stage
    const int c = (lane & (SLOTS - 1)) ^ key<LINE>(r);
    return first + r < rows ? (uint32_t)(first + r) * (uint32_t)pitch + c * 16u : OOB;
  };
  uint32_t oa[C::IA], ob[C::IB];
#pragma unroll
  for (int i = 0; i < C::IA; ++i) oa[i] = offset(std::integral_constant<int, C::LA>(), C::IA * w + i, m0, g.ra, g.pa);
#pragma unroll
  for (int i = 0; i < C::IB; ++i) ob[i] = offset(std::integral_constant<int, C::LB>(), C::IB * w + i, n0, g.rb, g.pb);
  auto load = [&](int s, int buf) {
    char* st = smem + buf * C::STAGE;
#pragma unroll
    for (int i = 0; i < C::IA; ++i) load16_lds(ra, st + (C::IA * w + i) * 1024, oa[i], (uint32_t)(s * C::LA));
#pragma unroll
    for (int i = 0; i < C::IB; ++i) load16_lds(rb, st + BM * C::LA + (C::IB * w + i) * 1024, ob[i], (uint32_t)(s * C::LB));
  };

  // ---- products ----
  f32x4_v acc[FM][FN];
#pragma unroll
  for (int j = 0; j < FM; ++j)
#pragma unroll
    for (int i = 0; i < FN; ++i) acc[j][i] = f32x4_v{0.f, 0.f, 0.f, 0.f};
  constexpr bool LOW = FINE || C::PIECES;  // the small products' sums, or those of the pieces before
  f32x4_v low[LOW ? FM : 1][LOW ? FN : 1];
  if constexpr (LOW)
#pragma unroll
    for (int j = 0; j < FM; ++j)
#pragma unroll
      for (int i = 0; i < FN; ++i) low[j][i] = f32x4_v{0.f, 0.f, 0.f, 0.f};
  const int p = lane & 15, h = lane >> 4;
  constexpr int NA = C::LA / 64, NB = C::LB / 64;  // fragments of a line
  const lds_ptr_t la = (lds_ptr_t)smem + (wm * C::TM + p) * C::LA;
  const lds_ptr_t lb = (lds_ptr_t)smem + BM * C::LA + (wn * C::TN + p) * C::LB;
  int slot_a[NA], slot_b[NB];
#pragma unroll
  for (int x = 0; x < NA; ++x) slot_a[x] = ((h + 4 * x) ^ key<C::LA>(p)) * 16;
#pragma unroll
  for (int x = 0; x < NB; ++x) slot_b[x] = ((h + 4 * x) ^ key<C::LB>(p)) * 16;

  constexpr int L = C::IA + C::IB, AHEAD = BUFS - 1;
#pragma unroll
  for (int s = 0; s < AHEAD; ++s)
    if (s < g.stages) load(s, s);
  int buf = 0;
  for (int s = 0; s < g.stages; ++s) {
    // this stage is there when all but the loads of the stages behind it are
    wait_stages<AHEAD - 1, L>(g.stages - 1 - s);
    lds_sync();  // ... everybody's, and everybody is done with the buffer before it
    if (s + AHEAD < g.stages) load(s + AHEAD, buf == 0 ? BUFS - 1 : buf - 1);
    const int at = buf * C::STAGE;
    buf = buf + 1 == BUFS ? 0 : buf + 1;
    if (above) continue;
    f16x8_v fb[FN][NB], fa[2][NA];
#pragma unroll
    for (int x = 0; x < NA; ++x) fa[0][x] = lds_ld<f16x8_v>(la + at + slot_a[x]);
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
      for (int x = 0; x < NB; ++x) fb[i][x] = lds_ld<f16x8_v>(lb + at + 16 * i * C::LB + slot_b[x]);
#pragma unroll
    for (int j = 0; j < FM; ++j) {
      if (j + 1 < FM)
#pragma unroll
        for (int x = 0; x < NA; ++x) fa[(j + 1) & 1][x] = lds_ld<f16x8_v>(la + at + 16 * (j + 1) * C::LA + slot_a[x]);
      auto mul = [&](int xa, int xb) {
#pragma unroll
        for (int i = 0; i < FN; ++i)
          acc[j][i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(fb[i][xb], fa[j & 1][xa], acc[j][i], 0, 0, 0);
      };
      mul(0, 0);
      if constexpr (FINE) {
#pragma unroll
        for (int i = 0; i < FN; ++i)
          low[j][i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(fb[i][1], fa[j & 1][0], low[j][i], 0, 0, 0);
#pragma unroll
        for (int i = 0; i < FN; ++i)
          low[j][i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(fb[i][0], fa[j & 1][1], low[j][i], 0, 0, 0);
      } else if constexpr (C::WIDE) {
        mul(1, 1);  // the next 32 of the reduction
      } else {
        if constexpr (PB == 2) mul(0, 1);
        if constexpr (PA == 2) mul(1, 0);
      }
    }
    if constexpr (C::PIECES)
      if (s % C::PIECE == C::PIECE - 1)
#pragma unroll
        for (int j = 0; j < FM; ++j)
#pragma unroll
          for (int i = 0; i < FN; ++i) {
            low[j][i] += acc[j][i];
            acc[j][i] = f32x4_v{0.f, 0.f, 0.f, 0.f};
          }
  }

  if constexpr (LOW)
#pragma unroll
    for (int j = 0; j < FM; ++j)
#pragma unroll
      for (int i = 0; i < FN; ++i) acc[j][i] += low[j][i];

  // ---- results: a lane holds, of row p of a piece, the columns 4 h .. 4 h + 3 ----
  float alpha = job.alpha;
  if (g.alpha_e) alpha *= g.square ? g.alpha_e[e] * g.alpha_e[e] : g.alpha_e[e];
  const int r1 = m0 + wm * C::TM, c1 = n0 + wn * C::TN;
  char* const mine = smem + w * C::HALF;
  if constexpr (EPI == OUT) {
    O* const out = reinterpret_cast<O*>(g.o) + e * g.so;
    constexpr int PER = 16 / sizeof(O);  // numbers of 16 bytes
    if (g.rb % PER == 0 && (reinterpret_cast<uintptr_t>(out) & 15) == 0) {
      // half of a wave's rows at a time through LDS, for lanes in a row to write whole lines
      constexpr int L = C::TN * sizeof(O), KEYS = L / 16 < 8 ? L / 16 - 1 : 7;
      lds_sync();  // (all products' operands are read)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
#pragma unroll
        for (int jj = 0; jj < FM / 2; ++jj)
#pragma unroll
          for (int i = 0; i < FN; ++i) {
            const int l = 16 * jj + p, s = (16 * i + 4 * h) * (int)sizeof(O) / 16;
            char* at = mine + l * L + (s ^ (l & KEYS)) * 16;
            const f32x4_v v = acc[half * (FM / 2) + jj][i] * alpha;
            if constexpr (sizeof(O) == 2)
              *reinterpret_cast<u32x2_v*>(at + (h & 1) * 8) = u32x2_v{f2bf2(v[0], v[1]), f2bf2(v[2], v[3])};
            else
              *reinterpret_cast<f32x4_v*>(at) = v;
          }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
        for (int k = 0; k < C::TM / 2 * L / 1024; ++k) {
          const int l = (64 * k + lane) / (L / 16), s = (64 * k + lane) % (L / 16);
          const u32x4_lv v = *reinterpret_cast<const u32x4_lv*>(mine + l * L + (s ^ (l & KEYS)) * 16);
          const int r = r1 + half * (C::TM / 2) + l, c = c1 + s * PER;
          if (r < g.ra && c < g.rb) *reinterpret_cast<u32x4_lv*>(out + (int64_t)r * g.rb + c) = v;
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      }
      return;
    }
#pragma unroll
    for (int j = 0; j < FM; ++j) {
      const int r = r1 + 16 * j + p;
      if (r >= g.ra) continue;
      O* row = out + (int64_t)r * g.rb;
#pragma unroll
      for (int i = 0; i < FN; ++i) {
        const int c = c1 + 16 * i + 4 * h;
        const f32x4_v v = acc[j][i] * alpha;
#pragma unroll
        for (int x = 0; x < 4; ++x)
          if (c + x < g.rb) row[c + x] = Elem<O>::from_f(v[x]);
      }
    }
  } else {
    // c [ra][columns up to the padding] and its transpose: a symmetric product's other half,
    // or the next group's other layout.  Of a symmetric product's tile on the diagonal the
    // pieces on and below it and the mirror of those below: a product of matrices that commute is
    // symmetric up to its rounding only, and what is not symmetric would grow with the steps
    // (bf16 updates of 256 x 1536 with one large direction, both halves as computed: error
    // 6.4e-3 of the result's norm in place of 3.0e-4).  Half of a wave's
    // tile at a time goes through LDS, where lines have their final layout (slots of 16
    // bytes xored with line % 8), for lanes in a row to write whole lines: 8 bytes of
    // sixteen lines at a time, as the products leave them, one costs the L1 as much as a
    // line (64 matrices of 2048 x 2048, bf16, 31.1 ms in place of 29.1; 128 of 256 x 1536 0.65 in place of 0.59).
    constexpr int HALF = C::HALF, LD = C::TN * 4, LT = C::TM * 4;  // bytes, of lines
    static_assert(FM % 2 == 0 && FN % 2 == 0, "halves of the pieces");
    const int cols = (g.rb + 63) & ~63, rows = (g.ra + 63) & ~63;
    char* const out = job.c + e * g.sc;
    char* const outt = EPI == SYM ? out : g.ct + e * g.sct;
    const int pt = EPI == SYM ? g.pc : g.pct;
    const char* const d = job.d ? job.d + e * g.sc : nullptr;
    auto put = [&](int at, const f16x4_v hi, const f16x4_v lo) {
      *reinterpret_cast<f16x4_v*>(mine + at) = hi;
      *reinterpret_cast<f16x4_v*>(mine + (at ^ 64)) = lo;
    };
    lds_sync();  // (all products' operands are read)
    if (above) return;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int rh = r1 + half * (C::TM / 2);
      // the lines' 16 bytes number k of this lane
      auto line = [&](int k) { return (64 * k + lane) / (LD / 16); };
      auto slot = [&](int k) { return (64 * k + lane) % (LD / 16); };
      auto at = [&](int k) { return line(k) * LD + (slot(k) ^ (line(k) & 7)) * 16; };
      auto where = [&](int k) { return (int64_t)(rh + line(k)) * g.pc + c1 * 4 + slot(k) * 16; };
      if (EPI == SYM && d) {
#pragma unroll
        for (int k = 0; k < HALF / 1024; ++k)
          if (rh + line(k) < g.ra && c1 < cols)
            *reinterpret_cast<f16x8_v*>(mine + at(k)) = *reinterpret_cast<const f16x8_v*>(d + where(k));
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      }
#pragma unroll
      for (int jj = 0; jj < FM / 2; ++jj) {
        const int j = half * (FM / 2) + jj, r = r1 + 16 * j + p;
#pragma unroll
        for (int i = 0; i < FN; ++i) {
          const int c = c1 + 16 * i + 4 * h, l = 16 * jj + p;
          const int to = l * LD + (i >> 1) * 128 + ((((i & 1) * 2 + (h >> 1)) ^ (l & 7)) * 16) + (h & 1) * 8;
          f32x4_v v = acc[j][i] * alpha;
          if (EPI == SYM && d) {
            f32x4_v u = {0.f, 0.f, 0.f, 0.f};
            if (r < g.ra && c1 < cols) {
              const f16x4_v dh = *reinterpret_cast<const f16x4_v*>(mine + to), dl = *reinterpret_cast<const f16x4_v*>(mine + (to ^ 64));
#pragma unroll
              for (int x = 0; x < 4; ++x) u[x] = (float)dh[x] + (float)dl[x];
            }
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              v[x] = fmaf(job.beta, u[x], v[x]);
              if (r == c + x && r < g.ra) v[x] += job.diag;
            }
          }
          f16x8_v parts;
          f16x4_v hi, lo;
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            _Float16 vh, vl;
            split(v[x], vh, vl);
            parts[x] = hi[x] = vh;
            parts[4 + x] = lo[x] = vl;
          }
          if (diagonal && r1 + 16 * j == c1 + 16 * i) {
            hi = lower_mirrored(hi, lane);
            lo = lower_mirrored(lo, lane);
          }
          put(to, hi, lo);
          acc[j][i] = __builtin_bit_cast(f32x4_v, parts);
        }
      }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
      for (int k = 0; k < HALF / 1024; ++k) {
        const f16x8_v v = *reinterpret_cast<const f16x8_v*>(mine + at(k));
        const int r = rh + line(k), c = c1 + (slot(k) >> 3) * 32 + (slot(k) & 3) * 8;
        if (r < g.ra && c1 < cols && !(diagonal && (c >> 4) > (r >> 4))) *reinterpret_cast<f16x8_v*>(out + where(k)) = v;
      }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int ch = c1 + half * (C::TN / 2);
#pragma unroll
      for (int ii = 0; ii < FN / 2; ++ii)
#pragma unroll
        for (int j = 0; j < FM; ++j) {
          const f16x8_v parts = __builtin_bit_cast(f16x8_v, acc[j][half * (FN / 2) + ii]);
          const f16x4_v hi = turn4(f16x4_v{parts[0], parts[1], parts[2], parts[3]}, lane);
          const f16x4_v lo = turn4(f16x4_v{parts[4], parts[5], parts[6], parts[7]}, lane);
          const int l = 16 * ii + 4 * h + (p & 3);
          put(l * LT + (j >> 1) * 128 + ((((j & 1) * 2 + (p >> 3)) ^ (l & 7)) * 16) + ((p >> 2) & 1) * 8, hi, lo);
        }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
      for (int k = 0; k < HALF / 1024; ++k) {
        const int l = (64 * k + lane) / (LT / 16), s = (64 * k + lane) % (LT / 16);
        const f16x8_v v = *reinterpret_cast<const f16x8_v*>(mine + l * LT + (s ^ (l & 7)) * 16);
        const int r = ch + l, c = r1 + (s >> 3) * 32 + (s & 3) * 8;
        if (r < g.rb && r1 + (s >> 3) * 32 < rows && !(diagonal && (r >> 4) >= (c >> 4)))
          *reinterpret_cast<f16x8_v*>(outt + (int64_t)(ch + l) * pt + r1 * 4 + s * 16) = v;
      }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }
  }
}

}  // namespace ortho
}  // namespace moe
