// Products of bf16 rows with MXFP4 weights (include/moe_step_ops.h: moe_mxfp4_mm).
//
// A code (E2M1) times its block's scale (2^(code - 127)) is a bf16 number exactly, and
// one instruction turns two codes into two of them, so the weights stay 4-bit up to
// the registers and the products run on the bf16 matrix cores: every product exact, sums
// in fp32.  Any split of the reduction over lanes does as long as both operands agree.
#pragma once

#include <type_traits>

#include "lds_stage.h"
#include "segments.h"
#include "step_launch.h"

namespace moe {
namespace f4 {

struct Args {
  const bf16_t* a;
  const uint8_t* q;
  const uint8_t* s;
  void* c;
  const int32_t* offsets;    // null: one segment of `rows` rows
  const int32_t* counts;
  const int32_t* row_token;  // gathered rows of a, or null
  int a_rows, rows, E, K, N;
};

// 8 codes (a word, the first in its lowest bits) as bf16 values, times 2^(scale - 127);
// 255 is NaN
__device__ __forceinline__ bf16x8_v values(uint32_t w, uint32_t scale) {
  const float f = __uint_as_float(scale << 23);
  const bf16x2_v v0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, f, 0);
  const bf16x2_v v1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, f, 1);
  const bf16x2_v v2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, f, 2);
  const bf16x2_v v3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, f, 3);
  return bf16x8_v{v0[0], v0[1], v1[0], v1[1], v2[0], v2[1], v3[0], v3[1]};
}

// the value of lane p (of 0..15) in the lanes p, 16 + p, 32 + p and 48 + p
__device__ __forceinline__ uint32_t from_first_row(uint32_t v) {
  const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  const auto b = __builtin_amdgcn_permlane32_swap(a[0], a[0], false, false);
  return b[0];
}

// ---------------------------------------------------------------------------
// Few rows per expert (decode): the weights' bytes are the work, every touched expert's
// are read once, straight into registers, the next chunk's during this one's products.  A
// workgroup takes 16 rows of a segment and 16 FN columns; its four waves split the
// reduction (chunks of 256: wave w takes w, w + 4, ...) and add up their sums in wave
// order.  A lane's 16 bytes of codes are one block of 32 and have one scale.
//   Next to those bytes the L1 bounds it: one access per cycle, 16 bytes where
// neighbouring lanes read different lines.  So the rows go through LDS, 512
// contiguous bytes of each per chunk, and scales are read as 8 bytes per column by the
// lanes 0..15, who tell the others (both straight into the lanes that use them: 16 rows
// for each of 64 experts of 2048 x 2048 47 us in place of 40).
// ---------------------------------------------------------------------------
template <int FN, typename O>
__global__ void __launch_bounds__(256)
k_mxfp4_thin(Args g) {
  constexpr int W = 4, BN = 16 * FN, BM = 16, ROW = 512, ROWS = BM * ROW;
  __shared__ __attribute__((aligned(1024))) char rows_lds[W][ROWS];
  __shared__ float part[W - 1][FN][64][4];
  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int NT = (g.N + BN - 1) / BN;
  const int mg = (int)(blockIdx.x / (unsigned)NT), n0 = (int)(blockIdx.x % (unsigned)NT) * BN;
  int e, row0, rows;
  if (!segment_tile<BM>(g.offsets, g.counts, g.E, g.rows, mg, lane, e, row0, rows)) return;  // no such tile

  const int p = lane & 15, h = lane >> 4;
  const int kb = g.K / 32, chunks = (kb + 7) / 8;
  int token = p;
  if (g.row_token) token = g.row_token[row0 + min(p, rows - 1)];
  // columns past the end repeat the last one (their results are dropped)
  const uint8_t *pq[FN], *ps[FN];
#pragma unroll
  for (int i = 0; i < FN; ++i) {
    const int64_t n = (int64_t)e * g.N + min(n0 + 16 * i + p, g.N - 1);
    pq[i] = g.q + n * (g.K / 2);
    ps[i] = g.s + n * kb;
  }
  struct Codes {
    uint4 q[2][FN];
    uint2 s[FN];
  };
  Codes cur, ahead;
  auto block = [&](int k, int c) { return 8 * k + 4 * c + h; };
  // chunk k; past the reduction the first block's codes again, where the rows are zeros
  auto load_q = [&](int k, Codes& d) {
    if (lane < 16) {
#pragma unroll
      for (int i = 0; i < FN; ++i) {
        if (8 * k + 8 <= kb) {
          __builtin_memcpy(&d.s[i], ps[i] + 8 * k, 8);
        } else {
          uint32_t v[2] = {0, 0};
#pragma unroll
          for (int y = 0; y < 8; ++y)
            if (8 * k + y < kb) v[y >> 2] |= (uint32_t)ps[i][8 * k + y] << (8 * (y & 3));
          d.s[i] = make_uint2(v[0], v[1]);
        }
      }
    }
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int b = block(k, c) < kb ? block(k, c) : 0;
#pragma unroll
      for (int i = 0; i < FN; ++i) d.q[c][i] = *reinterpret_cast<const uint4*>(pq[i] + 16 * (int64_t)b);
    }
  };
  load_q(w < chunks ? w : 0, cur);  // (on the way while the tokens arrive)
  __builtin_amdgcn_sched_barrier(0);
  // Rows: lane l loads 16 bytes (unit l mod 32, xored with the row for the banks) of the
  // rows l / 32, 2 + l / 32, ...; rows past the end and tokens that do not exist are zeros.
  const int known = g.row_token ? g.a_rows : rows;
  const __amdgpu_buffer_rsrc_t ra =
      rsrc(g.row_token ? g.a : g.a + (int64_t)row0 * g.K, (uint32_t)known * (uint32_t)g.K * 2u);
  uint32_t oa[ROWS / 1024];
#pragma unroll
  for (int i = 0; i < ROWS / 1024; ++i) {
    const int r = 2 * i + (lane >> 5);
    const uint32_t at = (uint32_t)__shfl(token, r, 64);
    oa[i] = r < rows && at < (uint32_t)known ? at * (uint32_t)g.K * 2u + (((uint32_t)lane & 31u) ^ (r & 7)) * 16u : OOB;
  }
  auto load_a = [&](int k) {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // (what lay there has been read)
#pragma unroll
    for (int i = 0; i < ROWS / 1024; ++i) {
      const int unit = (lane & 31) ^ ((2 * i + (lane >> 5)) & 7);
      load16_lds(ra, rows_lds[w] + 1024 * i, 32 * k + unit < 4 * kb ? oa[i] : OOB, (uint32_t)k * ROW);
    }
    asm volatile("" ::: "memory");
  };
  const char* const mine = rows_lds[w] + p * ROW;

  f32x4_v acc[FN];
#pragma unroll
  for (int i = 0; i < FN; ++i) acc[i] = f32x4_v{0.f, 0.f, 0.f, 0.f};
  for (int k = w; k < chunks; k += W) {
    load_a(k);
    if (k + W < chunks) {
      load_q(k + W, ahead);
      wait_vm<3 * FN>();  // all but those
    } else {
      wait_vm<0>();
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const bool there = block(k, c) < kb;
      bf16x8_v a[4];
#pragma unroll
      for (int x = 0; x < 4; ++x)
        a[x] = *reinterpret_cast<const bf16x8_v*>(mine + ((16 * c + 4 * h + x) ^ (p & 7)) * 16);
#pragma unroll
      for (int i = 0; i < FN; ++i) {
        const uint32_t four = from_first_row(c ? cur.s[i].y : cur.s[i].x);
        const uint32_t sc = there ? (four >> (8 * h)) & 255u : 127u;  // (zeros times a NaN would not be zeros)
        const uint32_t words[4] = {cur.q[c][i].x, cur.q[c][i].y, cur.q[c][i].z, cur.q[c][i].w};
#pragma unroll
        for (int x = 0; x < 4; ++x)
          acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(values(words[x], sc), a[x], acc[i], 0, 0, 0);
      }
    }
    cur = ahead;
  }
  if (w > 0)
#pragma unroll
    for (int i = 0; i < FN; ++i) *reinterpret_cast<f32x4_v*>(part[w - 1][i][lane]) = acc[i];
  __syncthreads();
  if (w > 0 || p >= rows) return;
  O* out = reinterpret_cast<O*>(g.c) + ((int64_t)row0 + p) * g.N;
#pragma unroll
  for (int i = 0; i < FN; ++i) {
    f32x4_v v = acc[i];
#pragma unroll
    for (int x = 0; x < W - 1; ++x) v += *reinterpret_cast<const f32x4_v*>(part[x][i][lane]);
    const int c = n0 + 16 * i + 4 * h;
    if (c >= g.N) continue;
    if constexpr (sizeof(O) == 2) *reinterpret_cast<uint2*>(out + c) = make_uint2(f2bf2(v[0], v[1]), f2bf2(v[2], v[3]));
    else *reinterpret_cast<float4*>(out + c) = make_float4(v[0], v[1], v[2], v[3]);
  }
}

// ---------------------------------------------------------------------------
// Many rows per expert: tiles of BM x BN, WM x WN waves.  A stage is 64 of the
// reduction: 128 bytes of every row and 32 of every column's codes go straight into
// LDS, three stages in turn.  Scales: 16 bytes of every column, eight stages' worth, go
// there through registers, a thread per column (byte by byte into the lanes that use
// them they were more than half of the loads, 1580 us in place of 1170 with 131072 rows,
// 64 experts of 2048 x 2048; 880 us today, 1250 TFLOP/s, where the clock gives way before
// the matrix cores are full).
// ---------------------------------------------------------------------------
template <int BM, int BN, int WM, int WN>
struct Cfg {
  static constexpr int W = WM * WN, NTH = 64 * W;
  static constexpr int TM = BM / WM, TN = BN / WN, FM = TM / 16, FN = TN / 16;
  static constexpr int IA = BM / 8 / W, IB = BN / 32 / W;  // 1 KB loads per wave and stage
  static constexpr int STAGE = BM * 128 + BN * 32;
  static constexpr int BUFS = 3, SMEM = BUFS * STAGE + BN * 16;
  static_assert(BM % (8 * W) == 0 && BN % (32 * W) == 0 && BN == NTH, "loads per wave, scales per thread");
};

template <int BM, int BN, int WM, int WN, typename O>
__global__ void __launch_bounds__(64 * WM * WN, 2)
k_mxfp4_tile(Args g) {
  using C = Cfg<BM, BN, WM, WN>;
  constexpr int FM = C::FM, FN = C::FN;
  extern __shared__ __attribute__((aligned(1024))) char smem[];
  typedef uint32_t u32x2_q __attribute__((ext_vector_type(2)));
  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = w / WN, wn = w % WN;
  const int NT = (g.N + BN - 1) / BN;
  const int id = xcd_virtual_id(blockIdx.x, gridDim.x);
  const int mg = id / NT, n0 = (id - mg * NT) * BN;
  int e, row0, rows;
  if (!segment_tile<BM>(g.offsets, g.counts, g.E, g.rows, mg, lane, e, row0, rows)) return;  // no such tile

  // ---- loads ----
  const int kb = g.K / 32, stages = (kb + 1) / 2;
  const bool gather = g.row_token != nullptr;
  const int sub = lane >> 3, ca = ((lane & 7) ^ sub) * 8;  // line of a 1 KB load, first of its 8 values
  uint32_t oa[C::IA], oq[C::IB];
#pragma unroll
  for (int i = 0; i < C::IA; ++i) {
    const int r = (C::IA * w + i) * 8 + sub;
    uint32_t line = OOB;
    if (r < rows) {
      const uint32_t t = gather ? (uint32_t)g.row_token[row0 + r] : (uint32_t)r;
      if (!gather || t < (uint32_t)g.a_rows) line = t * (uint32_t)g.K * 2u + ca * 2u;
    }
    oa[i] = line;
  }
  // (a column's two halves of 16 bytes change places every four columns, so that a
  // wave's reads, half of every one, meet all banks)
  const int cq = (lane & 1) ^ ((lane >> 3) & 1);
#pragma unroll
  for (int i = 0; i < C::IB; ++i) {
    const int n = n0 + (C::IB * w + i) * 32 + (lane >> 1);
    oq[i] = n < g.N ? (uint32_t)n * (uint32_t)(g.K / 2) + cq * 16u : OOB;
  }
  const bf16_t* a0 = gather ? g.a : g.a + (int64_t)row0 * g.K;
  const __amdgpu_buffer_rsrc_t ra = rsrc(a0, (uint32_t)(gather ? g.a_rows : rows) * (uint32_t)g.K * 2u);
  const __amdgpu_buffer_rsrc_t rq = rsrc(g.q + (int64_t)e * g.N * (g.K / 2), (uint32_t)g.N * (uint32_t)(g.K / 2));
  auto load = [&](int s, int buf) {
    char* st = smem + buf * C::STAGE;
    // (a last stage of 32: the missing values are zeros, whatever codes lie there)
    const bool half = 2 * s + 1 >= kb;
#pragma unroll
    for (int i = 0; i < C::IA; ++i)
      load16_lds(ra, st + (C::IA * w + i) * 1024, half && ca >= 32 ? OOB : oa[i], (uint32_t)s * 128u);
#pragma unroll
    for (int i = 0; i < C::IB; ++i)
      load16_lds(rq, st + BM * 128 + (C::IB * w + i) * 1024, half && cq ? OOB : oq[i], (uint32_t)s * 32u);
  };
  // this thread's column's scales of the stages 8 b .. 8 b + 7; zeros past the reduction
  const uint8_t* const ps = g.s + ((int64_t)e * g.N + min(n0 + tid, g.N - 1)) * kb;
  u32x4_lv sc;
  auto load_scales = [&](int b) {
    if (16 * b + 16 <= kb) {
      __builtin_memcpy(&sc, ps + 16 * b, 16);
    } else {
      uint32_t v[4] = {0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (16 * b + i < kb) v[i >> 2] |= (uint32_t)ps[16 * b + i] << (8 * (i & 3));
      sc = u32x4_lv{v[0], v[1], v[2], v[3]};
    }
  };
  char* const scales = smem + C::BUFS * C::STAGE;

  // ---- products ----
  f32x4_v acc[FN][FM];
#pragma unroll
  for (int i = 0; i < FN; ++i)
#pragma unroll
    for (int j = 0; j < FM; ++j) acc[i][j] = f32x4_v{0.f, 0.f, 0.f, 0.f};
  // a lane's 16 of a stage's 64: 16 h .. 16 h + 15
  const int p = lane & 15, h = lane >> 4;
  const lds_ptr_t la = (lds_ptr_t)smem + (wm * C::TM + p) * 128;
  const lds_ptr_t lq = (lds_ptr_t)smem + BM * 128 + (wn * C::TN + p) * 32 + (((h >> 1) ^ ((p >> 2) & 1)) * 16) + (h & 1) * 8;
  const lds_ptr_t ls = (lds_ptr_t)scales + (wn * C::TN + p) * 16;
  const int slot0 = ((2 * h) ^ (p & 7)) * 16, slot1 = ((2 * h + 1) ^ (p & 7)) * 16;

  load_scales(0);
  load(0, 0);
  if (stages > 1) load(1, 1);
  int buf = 0;
  uint32_t s4[FN];  // two stages' scales of a column
  for (int s = 0; s < stages; ++s) {
    // this stage is there once all but the next stage's loads are (scales are older)
    if (s + 1 < stages) wait_vm<C::IA + C::IB>();
    else wait_vm<0>();
    lds_sync();
    if ((s & 7) == 0) {
      *reinterpret_cast<u32x4_lv*>(scales + tid * 16) = sc;
      lds_sync();
    }
    if ((s & 7) == 5 && 2 * (s + 3) < kb) load_scales((s + 3) >> 3);
    if (s + 2 < stages) load(s + 2, buf == 0 ? 2 : buf - 1);
    const int at = buf * C::STAGE;
    bf16x8_v fa[FM][2];
#pragma unroll
    for (int j = 0; j < FM; ++j) {
      fa[j][0] = lds_ld<bf16x8_v>(la + at + j * 2048 + slot0);
      fa[j][1] = lds_ld<bf16x8_v>(la + at + j * 2048 + slot1);
    }
    if ((s & 1) == 0) {
#pragma unroll
      for (int i = 0; i < FN; ++i) s4[i] = lds_ld<uint32_t>(ls + i * 256 + (s & 7) * 2);
    }
    const int byte = 16 * (s & 1) + 8 * (h >> 1);
#pragma unroll
    for (int i = 0; i < FN; ++i) {
      const u32x2_q c = lds_ld<u32x2_q>(lq + at + i * 512);
      const uint32_t scale = (s4[i] >> byte) & 255u;
      const bf16x8_v b0 = values(c[0], scale), b1 = values(c[1], scale);
#pragma unroll
      for (int j = 0; j < FM; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b0, fa[j][0], acc[i][j], 0, 0, 0);
#pragma unroll
      for (int j = 0; j < FM; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b1, fa[j][1], acc[i][j], 0, 0, 0);
    }
    buf = buf == 2 ? 0 : buf + 1;
  }

  // Results: a lane holds, of row p of a piece, the columns 4 h .. 4 h + 3.  Half of a
  // wave's rows at a time go through LDS (slots of 16 bytes xored with row % 8), for lanes
  // in a row to write whole lines.
  constexpr int LINE = C::TN * sizeof(O), SLOTS = LINE / 16;
  static_assert(C::W * (C::TM / 2) * LINE <= C::SMEM && SLOTS >= 8 && FM % 2 == 0, "halves of all waves' rows");
  char* const mine = smem + w * (C::TM / 2) * LINE;
  const int c0 = n0 + wn * C::TN;
  lds_sync();  // (all products' operands are read)
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    O* const out = reinterpret_cast<O*>(g.c) + ((int64_t)row0 + wm * C::TM + half * (C::TM / 2)) * g.N + c0;
    const int left = rows - wm * C::TM - half * (C::TM / 2);
#pragma unroll
    for (int j = 0; j < FM / 2; ++j)
#pragma unroll
      for (int i = 0; i < FN; ++i) {
        const int l = 16 * j + p, s = (16 * i + 4 * h) * (int)sizeof(O) / 16;
        char* at = mine + l * LINE + (s ^ (l & 7)) * 16;
        const f32x4_v v = acc[i][half * (FM / 2) + j];
        if constexpr (sizeof(O) == 2) *reinterpret_cast<u32x2_q*>(at + (h & 1) * 8) = u32x2_q{f2bf2(v[0], v[1]), f2bf2(v[2], v[3])};
        else *reinterpret_cast<f32x4_v*>(at) = v;
      }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
    for (int k = 0; k < C::TM / 2 * LINE / 1024; ++k) {
      const int l = (64 * k + lane) / SLOTS, s = (64 * k + lane) % SLOTS, c = s * (16 / (int)sizeof(O));
      const u32x4_lv v = *reinterpret_cast<const u32x4_lv*>(mine + l * LINE + (s ^ (l & 7)) * 16);
      if (l >= left || c0 + c >= g.N) continue;
      *reinterpret_cast<u32x4_lv*>(out + (int64_t)l * g.N + c) = v;
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  }
}

}  // namespace f4
}  // namespace moe
