// Tokens sorted by expert and back (moe_sort, moe_permute, moe_unpermute and
// their gradients).
//
// Sort: a stable counting sort of the T*K expert choices.  A choice's row is
//   offsets[e] + (choices of e in earlier chunks) + (earlier in its chunk),
// and each of the three terms is an integer count, so the result does not
// depend on the order in which workgroups run.
//
// Moving rows: bandwidth is all there is (device copy of 1 GiB: 5.2 TB/s).  The
// permutation walks tokens, not rows: a token's row is read once and written to
// its K places, where a walk over rows would read it K times.  The way back
// walks tokens too, with the K rows' loads in flight together.  At T = 16384,
// K = 8, d = 2048, bf16: permute 106 us (5.7 TB/s), to 8 bits 54 us (6.3),
// weighted sum 115 us (5.3), its two gradients 212 us (5.4).  Few tokens are
// bound by launch and latency: a token's row is split over waves then (T = 1,
// d = 7168: 2.5 us; weighted sum of T = 8: 2.85 us).
#include <algorithm>

#include "../device_common.h"
#include "fp8_block.h"
#include "ops_launch.h"

namespace moe {

namespace {

constexpr int SORT_NT = 1024;      // threads of a sort workgroup = slots per step
constexpr int SORT_WAVES = SORT_NT / 64;
constexpr int SORT_MAX_CHUNKS = 256;
constexpr int SORT_MAX_E = 1024;

// Rank of every lane among the lanes of its wave with the same key (ascending
// lane), and how many those are.  keys < 2^bits.
__device__ __forceinline__ void wave_rank(int key, int bits, int lane, int& rank, int& count) {
  uint64_t same = ~0ull;
  for (int b = 0; b < bits; ++b) {
    const bool one = (key >> b) & 1;
    const uint64_t m = __ballot(one);
    same &= one ? m : ~m;
  }
  rank = __popcll(same & ((1ull << lane) - 1));
  count = __popcll(same);
}

// Choices per expert and chunk of `chunk` slots: cnt [chunks][E].  Two launches
// (this and k_sort_place) take 12.4 us for 262144 choices of 128 experts, 7 for
// 16396; both are chains of latencies, not bandwidth.  Counting all choices
// again in every workgroup instead of this launch takes 14.5 us for 16396.
__global__ void __launch_bounds__(SORT_NT)
k_sort_count(const int32_t* __restrict__ idx, int slots, int E, int chunk, int32_t* __restrict__ cnt) {
  __shared__ int h[SORT_MAX_E];
  for (int e = threadIdx.x; e < E; e += SORT_NT) h[e] = 0;
  __syncthreads();
  const int s0 = blockIdx.x * chunk, s1 = min(slots - s0, chunk) + s0;
  for (int s = s0 + (int)threadIdx.x; s < s1; s += SORT_NT) {
    const int e = idx[s];
    if ((unsigned)e < (unsigned)E) atomicAdd(&h[e], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += SORT_NT) cnt[(size_t)blockIdx.x * E + e] = h[e];
}

// Exclusive scan over the workgroup's threads; wsum: one word per wave
__device__ __forceinline__ int block_scan(int v, int lane, int wave, int* wsum) {
  int incl = v;
  for (int o = 1; o < 64; o <<= 1) {
    const int y = __shfl_up(incl, o, 64);
    if (lane >= o) incl += y;
  }
  if (lane == 63) wsum[wave] = incl;
  __syncthreads();
  int before = incl - v;
#pragma unroll
  for (int w = 0; w < SORT_WAVES; ++w) before += w < wave ? wsum[w] : 0;
  return before;
}

// The choices of the waves before wave `wave` (of WAVES) for expert e
__device__ __forceinline__ int waves_before(const int (*wcount)[SORT_MAX_E], int e, int wave) {
  int n = 0;
#pragma unroll
  for (int w = 0; w < SORT_WAVES; ++w) n += w < wave ? wcount[w][e] : 0;
  return n;
}

// Up to 1024 choices (one per thread) and experts: one workgroup, each choice
// read once.  Launched with at least E threads.  2.8 us for 8 choices of 256
// experts, a launch and four barriers.
__global__ void __launch_bounds__(SORT_NT)
k_sort_small(const int32_t* __restrict__ idx, int slots, int K, int E, int align, int32_t* __restrict__ offsets,
             int32_t* __restrict__ counts, int32_t* __restrict__ row_token, int32_t* __restrict__ slot_row) {
  __shared__ int wcount[SORT_WAVES][SORT_MAX_E];
  __shared__ int seg[SORT_MAX_E];
  __shared__ int wsum[SORT_WAVES];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int waves = (slots + 63) >> 6;  // with choices
  const int id = tid < slots ? idx[tid] : -1;
  for (int w = 0; w < waves; ++w)
    if (tid < E) wcount[w][tid] = 0;
  if (tid < SORT_WAVES) wsum[tid] = 0;
  const bool kept = (unsigned)id < (unsigned)E;
  int rank, same;
  wave_rank(kept ? id : E, 32 - __clz(E), lane, rank, same);
  __syncthreads();
  if (kept && rank == 0) wcount[wave][id] = same;
  __syncthreads();
  int n = 0;
  if (tid < E)
    for (int w = 0; w < waves; ++w) n += wcount[w][tid];
  const int padded = (n + align - 1) / align * align;
  const int first = block_scan(padded, lane, wave, wsum);
  if (tid < E) {
    seg[tid] = first;
    offsets[tid] = first;
    counts[tid] = n;
    if (tid == E - 1) offsets[E] = first + padded;
    for (int r = first + n; r < first + padded; ++r) row_token[r] = -1;
  }
  __syncthreads();
  int row = -1;
  if (kept) {
    row = seg[id] + rank + waves_before(wcount, id, wave);
    row_token[row] = tid / K;
  }
  if (tid < slots) slot_row[tid] = row;
}

// Rows of one chunk's choices, cnt [chunks][E] from k_sort_count.
__global__ void __launch_bounds__(SORT_NT)
k_sort_place(const int32_t* __restrict__ idx, int slots, int K, int E, int align, int chunk,
             const int32_t* __restrict__ cnt, int32_t* __restrict__ offsets, int32_t* __restrict__ counts,
             int32_t* __restrict__ row_token, int32_t* __restrict__ slot_row) {
  __shared__ int total[SORT_MAX_E];                 // choices of each expert
  __shared__ int seg[SORT_MAX_E];                   // its segment's first row
  __shared__ int before[SORT_MAX_E];                // choices in earlier chunks, then the next free row
  __shared__ int wcount[SORT_WAVES][SORT_MAX_E];    // this step's choices per wave and expert
  __shared__ int wsum[SORT_WAVES];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int chunks = gridDim.x, me = blockIdx.x;
  const int s0 = me * chunk, s1 = min(slots - s0, chunk) + s0;
  int next = s0 + tid < s1 ? idx[s0 + tid] : -1;  // (on the way beside the counts)

  if (tid < E) {
    total[tid] = before[tid] = 0;
    for (int w = 0; w < SORT_WAVES; ++w) wcount[w][tid] = 0;
  }
  __syncthreads();
  {
    // thread groups of E take the chunks in turn; integer sums
    const int groups = max(1, SORT_NT / E);
    const int g = tid / E, e = tid % E;
    if (g < groups) {
      int t = 0, b = 0;
#pragma unroll 16
      for (int c = g; c < chunks; c += groups) {
        const int v = cnt[(size_t)c * E + e];
        t += v;
        if (c < me) b += v;
      }
      atomicAdd(&total[e], t);
      atomicAdd(&before[e], b);
    }
  }
  __syncthreads();

  // exclusive scan of the padded lengths (thread e = expert e)
  const int n = tid < E ? total[tid] : 0;
  const int padded = (n + align - 1) / align * align;
  const int first = block_scan(padded, lane, wave, wsum);
  if (tid < E) {
    seg[tid] = first;
    before[tid] += first;
    if (me == 0) {
      offsets[tid] = first;
      counts[tid] = n;
      if (tid == E - 1) offsets[E] = first + padded;
    }
  }
  const int bits = 32 - __clz(E);  // E itself marks a dropped choice

  for (int base = s0;; base += SORT_NT) {
    const int s = base + tid;
    const int id = next;
    next = s + SORT_NT < s1 ? idx[s + SORT_NT] : -1;
    const bool kept = (unsigned)id < (unsigned)E;
    const int e = kept ? id : E;
    int rank, same;
    wave_rank(e, bits, lane, rank, same);
    if (kept && rank == 0) wcount[wave][e] = same;
    __syncthreads();  // (also: seg and before are complete)
    int row = -1;
    if (kept) {
      row = before[e] + rank + waves_before(wcount, e, wave);
      row_token[row] = s / K;
    }
    if (s < s1) slot_row[s] = row;
    if (base + SORT_NT >= s1) break;
    __syncthreads();
    if (tid < E) {
      before[tid] += waves_before(wcount, tid, SORT_WAVES);
      for (int w = 0; w < SORT_WAVES; ++w) wcount[w][tid] = 0;
    }
    __syncthreads();
  }

  // the rows that fill up the segments, dealt to the workgroups by expert
  if (align > 1)
    for (int e = me; e < E; e += chunks) {
      const int end = total[e] + seg[e];
      const int fill = (total[e] + align - 1) / align * align - total[e];
      if (tid < fill) row_token[end + tid] = -1;
    }
}

int sort_chunk(int64_t slots) {
  const int64_t per = (slots + SORT_MAX_CHUNKS - 1) / SORT_MAX_CHUNKS;
  return (int)((std::max<int64_t>(per, 1) + SORT_NT - 1) / SORT_NT * SORT_NT);
}

// Up to this many slots one workgroup sorts them, a choice per thread.
constexpr int SORT_ONE = SORT_NT;

// xp[slot_row[t,k]] = x[t], 16-byte pieces; `splits` waves share a token's row
__global__ void __launch_bounds__(256)
k_permute(const uint4* __restrict__ x, const int32_t* __restrict__ slot_row, int T, int K, int cap, int pieces,
          int splits, bool stream, uint4* __restrict__ xp) {
  const int lane = threadIdx.x & 63;
  const int64_t w = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int t = (int)(w / splits);
  if (t >= T) return;
  const int32_t* rows = slot_row + (size_t)t * K;
  for (int c = (int)(w % splits) * 64 + lane; c < pieces; c += splits * 64) {
    const uint4 v = x[(size_t)t * pieces + c];
    for (int k = 0; k < K; ++k) {
      const int r = rows[k];
      if ((unsigned)r < (unsigned)cap) store_as(xp + (size_t)r * pieces + c, v, stream);
    }
  }
}

// The same with the row quantized on the way: eight lanes per block of 128.
template <typename T>
__global__ void __launch_bounds__(256)
k_permute_fp8(const T* __restrict__ x, const int32_t* __restrict__ slot_row, int Tn, int K, int cap, int d,
              int splits, bool stream, uint8_t* __restrict__ q, float* __restrict__ s) {
  const int lane = threadIdx.x & 63;
  const int64_t w = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int t = (int)(w / splits);
  if (t >= Tn) return;
  const int32_t* rows = slot_row + (size_t)t * K;
  const int nb = (d + 127) / 128;
  for (int b0 = (int)(w % splits) * 8; b0 < nb; b0 += splits * 8) {
    const int b = b0 + (lane >> 3), col = b * 128 + (lane & 7) * 16;
    float v[16];
    if (col < d) {
      load16(x + (size_t)t * d + col, v);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = 0.f;
    }
    float sc;
    const uint4 code = quant_block8(v, sc);
    for (int k = 0; k < K; ++k) {
      const int r = rows[k];
      if ((unsigned)r >= (unsigned)cap) continue;
      if (col < d) store_as(reinterpret_cast<uint4*>(q + (size_t)r * d + col), code, stream);
      if ((lane & 7) == 0 && b < nb) s[(size_t)r * nb + b] = sc;
    }
  }
}

template <typename T> constexpr int VEC = 16 / (int)sizeof(T);

constexpr int ROWS_UNR = 8;  // rows of a token in flight

// o[t] = sum over k of w[t,k] y[slot_row[t,k]] in ascending k (w null: ones)
template <typename T>
__global__ void __launch_bounds__(256)
k_unpermute(const uint4* __restrict__ y, const float* __restrict__ wt, const int32_t* __restrict__ slot_row, int Tn,
            int K, int cap, int pieces, int splits, uint4* __restrict__ o) {
  constexpr int V = VEC<T>;
  const int lane = threadIdx.x & 63;
  const int64_t w = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int t = (int)(w / splits);
  if (t >= Tn) return;
  const int32_t* rows = slot_row + (size_t)t * K;
  // (every lane stays to the end, since its choices are read by the others)
  for (int c0 = (int)(w % splits) * 64; c0 < pieces; c0 += splits * 64) {
    const int c = min(c0 + lane, pieces - 1);
    float acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.f;
    for (int k0 = 0; k0 < K; k0 += ROWS_UNR) {
      // (lane j reads choice j: from uniform addresses the choices come one by one,
      // 8 tokens of 8 choices 3.1 us instead of 2.85)
      const int kj = min(k0 + (lane & (ROWS_UNR - 1)), K - 1);
      const int row = rows[kj];
      const float weight = wt ? wt[(size_t)t * K + kj] : 1.f;
      uint4 raw[ROWS_UNR];
      float g[ROWS_UNR];
      bool ok[ROWS_UNR];
#pragma unroll
      for (int j = 0; j < ROWS_UNR; ++j) {
        const int r = k0 + j < K ? __builtin_amdgcn_readlane(row, j) : -1;
        ok[j] = (unsigned)r < (unsigned)cap;
        g[j] = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(weight), j));
        raw[j] = ok[j] ? load_stream(y + (size_t)r * pieces + c) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int j = 0; j < ROWS_UNR; ++j) {
        if (!ok[j]) continue;
        float v[V];
        unpack16<T>(raw[j], v);
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = fmaf(g[j], v[i], acc[i]);
      }
    }
    if (c0 + lane < pieces) o[(size_t)t * pieces + c] = pack16<T>(acc);
  }
}

// dy[r] = w[t,k] d_o[t] and dw[t,k] = <d_o[t], y[r]>, r = slot_row[t,k]: one
// workgroup of NT threads per token; the dot products end in a fixed order over
// lanes and waves
template <typename T, int NT>
__global__ void __launch_bounds__(NT)
k_unpermute_bwd(const uint4* __restrict__ d_o, const uint4* __restrict__ y, const float* __restrict__ wt,
                const int32_t* __restrict__ slot_row, int K, int cap, int pieces, bool stream,
                uint4* __restrict__ dy, float* __restrict__ dw) {
  constexpr int V = VEC<T>;
  constexpr int KG = ROWS_UNR;
  __shared__ float part[NT / 64][KG];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int t = blockIdx.x;
  const int32_t* rows = slot_row + (size_t)t * K;
  for (int k0 = 0; k0 < K; k0 += KG) {
    const int kj = min(k0 + (lane & (KG - 1)), K - 1);  // (lane j reads choice j, as above)
    const int row = rows[kj];
    const float weight = dy ? wt[(size_t)t * K + kj] : 0.f;
    int r[KG];
    float g[KG], dot[KG];
#pragma unroll
    for (int j = 0; j < KG; ++j) {
      r[j] = k0 + j < K ? __builtin_amdgcn_readlane(row, j) : -1;
      if ((unsigned)r[j] >= (unsigned)cap) r[j] = -1;
      g[j] = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(weight), j));
      dot[j] = 0.f;
    }
    for (int c = tid; c < pieces; c += NT) {
      float a[V];
      unpack16<T>(d_o[(size_t)t * pieces + c], a);
      if (dw) {
        uint4 raw[KG];
#pragma unroll
        for (int j = 0; j < KG; ++j)
          raw[j] = r[j] >= 0 ? load_stream(y + (size_t)r[j] * pieces + c) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int j = 0; j < KG; ++j) {
          if (r[j] < 0) continue;
          float v[V];
          unpack16<T>(raw[j], v);
#pragma unroll
          for (int i = 0; i < V; ++i) dot[j] = fmaf(a[i], v[i], dot[j]);
        }
      }
      if (dy) {
#pragma unroll
        for (int j = 0; j < KG; ++j) {
          if (r[j] < 0) continue;
          float v[V];
#pragma unroll
          for (int i = 0; i < V; ++i) v[i] = g[j] * a[i];
          store_as(dy + (size_t)r[j] * pieces + c, pack16<T>(v), stream);
        }
      }
    }
    if (dw) {
#pragma unroll
      for (int j = 0; j < KG; ++j) {
        const float s = wave_sum(dot[j]);
        if (lane == 0) part[wave][j] = s;
      }
      __syncthreads();
      if (tid < KG && k0 + tid < K) {
        float s = 0.f;
#pragma unroll
        for (int x = 0; x < NT / 64; x += 4)
          s += (part[x][tid] + part[x + 1][tid]) + (part[x + 2][tid] + part[x + 3][tid]);
        dw[(size_t)t * K + k0 + tid] = s;
      }
      __syncthreads();
    }
  }
}

// Tokens for which long rows get 1024 threads each instead of 256, 256 / 1024 in us:
// 8 tokens of K = 8, d = 7168 9.7 / 6.8; 256 of d = 4096 10.1 / 8.7; 512 15.8 / 18.6.
constexpr int BWD_FEW = 256;

// Waves per token: rows of one token are split until there are 4096 waves, four
// for each SIMD of the card, and no finer than one pass of 64 lanes.
int row_splits(int T, int passes) {
  const int want = (4096 + T - 1) / std::max(T, 1);
  return std::max(1, std::min(want, passes));
}

// T rows of so many bytes on one side and T*K on the other
bool streamed(const PlanArgs& p, int64_t one, int64_t many) { return streams((int64_t)p.T * (one + p.K * many)); }

unsigned wave_blocks(int T, int splits) { return (unsigned)(((int64_t)T * splits + 3) / 4); }

}  // namespace

size_t sort_ws_bytes(int64_t slots, int E) {
  if (slots <= SORT_ONE) return 0;
  const int chunk = sort_chunk(slots);
  return (size_t)((slots + chunk - 1) / chunk) * E * sizeof(int32_t);
}

hipError_t launch_sort(const PlanArgs& p, const int32_t* expert_idx, const moe_plan& out, void* ws, hipStream_t st) {
  const int slots = p.T * p.K;
  if (slots <= SORT_ONE) {
    const int nt = (std::max(std::max(slots, p.E), 64) + 63) / 64 * 64;
    hipLaunchKernelGGL(k_sort_small, dim3(1), dim3(nt), 0, st, expert_idx, slots, p.K, p.E, p.align, out.offsets,
                       out.counts, out.row_token, out.slot_row);
    return hipGetLastError();
  }
  const int chunk = sort_chunk(slots);
  const unsigned chunks = (unsigned)(((int64_t)slots + chunk - 1) / chunk);
  hipLaunchKernelGGL(k_sort_count, dim3(chunks), dim3(SORT_NT), 0, st, expert_idx, slots, p.E, chunk, (int32_t*)ws);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(k_sort_place, dim3(chunks), dim3(SORT_NT), 0, st, expert_idx, slots, p.K, p.E, p.align, chunk,
                     (const int32_t*)ws, out.offsets, out.counts, out.row_token, out.slot_row);
  return hipGetLastError();
}

hipError_t launch_permute(const PlanArgs& p, int dtype, int d, const void* x, void* xp, hipStream_t st) {
  const int pieces = (int)((int64_t)d * (dtype == MOE_BF16 ? 2 : 4) / 16);
  const int splits = row_splits(p.T, (pieces + 63) / 64);
  hipLaunchKernelGGL(k_permute, dim3(wave_blocks(p.T, splits)), dim3(256), 0, st, (const uint4*)x, p.slot_row, p.T,
                     p.K, p.cap, pieces, splits, streamed(p, (int64_t)pieces * 16, (int64_t)pieces * 16), (uint4*)xp);
  return hipGetLastError();
}

hipError_t launch_permute_fp8(const PlanArgs& p, int dtype, int d, const void* x, uint8_t* q, float* s,
                              hipStream_t st) {
  const int splits = row_splits(p.T, (d + 1023) / 1024);
  const dim3 grid(wave_blocks(p.T, splits));
  const bool stream = streamed(p, (int64_t)d * (dtype == MOE_BF16 ? 2 : 4), d);
  if (dtype == MOE_BF16)
    hipLaunchKernelGGL(k_permute_fp8<bf16_t>, grid, dim3(256), 0, st, (const bf16_t*)x, p.slot_row, p.T, p.K, p.cap,
                       d, splits, stream, q, s);
  else
    hipLaunchKernelGGL(k_permute_fp8<float>, grid, dim3(256), 0, st, (const float*)x, p.slot_row, p.T, p.K, p.cap, d,
                       splits, stream, q, s);
  return hipGetLastError();
}

hipError_t launch_unpermute(const PlanArgs& p, int dtype, int d, const void* y, const float* w, void* o,
                            hipStream_t st) {
  const int pieces = (int)((int64_t)d * (dtype == MOE_BF16 ? 2 : 4) / 16);
  const int splits = row_splits(p.T, (pieces + 63) / 64);
  const dim3 grid(wave_blocks(p.T, splits));
  if (dtype == MOE_BF16)
    hipLaunchKernelGGL(k_unpermute<bf16_t>, grid, dim3(256), 0, st, (const uint4*)y, w, p.slot_row, p.T, p.K, p.cap,
                       pieces, splits, (uint4*)o);
  else
    hipLaunchKernelGGL(k_unpermute<float>, grid, dim3(256), 0, st, (const uint4*)y, w, p.slot_row, p.T, p.K, p.cap,
                       pieces, splits, (uint4*)o);
  return hipGetLastError();
}

hipError_t launch_unpermute_bwd(const PlanArgs& p, int dtype, int d, const void* d_o, const void* y, const float* w,
                                void* dy, float* dw, hipStream_t st) {
  const int pieces = (int)((int64_t)d * (dtype == MOE_BF16 ? 2 : 4) / 16);
  const bool stream = streamed(p, (int64_t)pieces * 16, (int64_t)pieces * 16 * ((dy ? 1 : 0) + (dw ? 1 : 0)));
  auto launch = [&](auto* k, int threads) {
    hipLaunchKernelGGL(k, dim3(p.T), dim3(threads), 0, st, (const uint4*)d_o, (const uint4*)y, w, p.slot_row, p.K,
                       p.cap, pieces, stream, (uint4*)dy, dw);
    return hipGetLastError();
  };
  if (p.T <= BWD_FEW && pieces > 256)
    return dtype == MOE_BF16 ? launch(k_unpermute_bwd<bf16_t, 1024>, 1024) : launch(k_unpermute_bwd<float, 1024>, 1024);
  return dtype == MOE_BF16 ? launch(k_unpermute_bwd<bf16_t, 256>, 256) : launch(k_unpermute_bwd<float, 256>, 256);
}

}  // namespace moe
