// E4M3 blocks with one fp32 scale per 128 values: scale and conversion shared
// by every kernel that writes them.
#pragma once

#include "../device_common.h"

namespace moe {

constexpr float FP8_MAX = 448.f;
constexpr uint32_t INF_BITS = 0x7f800000u;
constexpr uint32_t TINY_BITS = 0x00800000u;  // 2^-126

// |x| as an unsigned word: orders as the magnitudes do, with infinities and
// NaNs above every finite value, so an integer maximum carries them along.
__device__ __forceinline__ uint32_t mag_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// scale of a block whose largest magnitude has the bits `amax`: amax / 448, at
// least 2^-126 (so that its reciprocal is finite); NaN where amax is not finite
__device__ __forceinline__ float block_scale(uint32_t amax) {
  if (amax >= INF_BITS) return __uint_as_float(0x7fc00000u);
  return fmaxf(__fdiv_rn(__uint_as_float(amax), FP8_MAX), __uint_as_float(TINY_BITS));
}

// E4M3 codes of four scaled values (value i in byte i), nearest, ties to even.
// A value times its block's rounded reciprocal is at most 448 (1 + 2^-22), which
// rounds to 448, so no clamp is needed.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
  return (uint32_t)w;
}

// 16-byte accesses that a cache does not keep.  The result of a call that moves
// more than the memory-side cache holds is not there any more when its reader
// comes, and written past the caches it takes less.  With inputs that are not
// in the caches either: combination gradient, 1.1 GB, 220 -> 201 us; weights,
// 0.54 GB, 106 -> 102; permutation, 0.9 GB, 189 -> 185; SwiGLU, 0.34 GB, 64 -> 62.
// Below that size a result stays where it is read next.
typedef uint32_t u32x4_m __attribute__((ext_vector_type(4)));
__device__ __forceinline__ void store_stream(uint4* p, uint4 v) {
  __builtin_nontemporal_store(u32x4_m{v.x, v.y, v.z, v.w}, reinterpret_cast<u32x4_m*>(p));
}
__device__ __forceinline__ uint4 load_stream(const uint4* p) {
  const u32x4_m v = __builtin_nontemporal_load(reinterpret_cast<const u32x4_m*>(p));
  return make_uint4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void store_as(uint4* p, uint4 v, bool stream) {
  if (stream) store_stream(p, v);
  else *p = v;
}
__device__ __forceinline__ void store_as(uint2* p, uint2 v, bool stream) {
  typedef uint32_t u32x2_m __attribute__((ext_vector_type(2)));
  if (stream) __builtin_nontemporal_store(u32x2_m{v.x, v.y}, reinterpret_cast<u32x2_m*>(p));
  else *p = v;
}
// whether a call that reads and writes so many bytes streams its result
inline bool streams(int64_t bytes) { return bytes >= ((int64_t)256 << 20); }

// 16 consecutive values of a row as fp32
template <typename T>
__device__ __forceinline__ void load16(const T* p, float (&v)[16]) {
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint4 u = reinterpret_cast<const uint4*>(p)[h];
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[8 * h + 2 * i] = __uint_as_float(w[i] << 16);
        v[8 * h + 2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      }
    }
  } else {
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      const float4 u = reinterpret_cast<const float4*>(p)[h];
      v[4 * h] = u.x; v[4 * h + 1] = u.y; v[4 * h + 2] = u.z; v[4 * h + 3] = u.w;
    }
  }
}

// (two or four stores with gaps between the lanes: through the caches, which
// put the lines together)
template <typename T>
__device__ __forceinline__ void store16(T* p, const float (&v)[16]) {
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      reinterpret_cast<uint4*>(p)[h] = make_uint4(f2bf2(v[8 * h], v[8 * h + 1]), f2bf2(v[8 * h + 2], v[8 * h + 3]),
                                                  f2bf2(v[8 * h + 4], v[8 * h + 5]), f2bf2(v[8 * h + 6], v[8 * h + 7]));
  } else {
#pragma unroll
    for (int h = 0; h < 4; ++h)
      reinterpret_cast<float4*>(p)[h] = make_float4(v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]);
  }
}

// 16 bytes as fp32 values and back
template <typename T>
__device__ __forceinline__ void unpack16(const uint4 u, float (&v)[16 / sizeof(T)]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(w[i]);
  }
}

template <typename T>
__device__ __forceinline__ uint4 pack16(const float (&v)[16 / sizeof(T)]) {
  if constexpr (sizeof(T) == 2)
    return make_uint4(f2bf2(v[0], v[1]), f2bf2(v[2], v[3]), f2bf2(v[4], v[5]), f2bf2(v[6], v[7]));
  else
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
}

// Eight lanes hold a block of 128 values, 16 each (zeros past the row's end):
// the block's scale, and this lane's 16 codes.  Every lane of the eight runs it.
__device__ __forceinline__ uint4 quant_block8(const float (&v)[16], float& scale) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) m = max(m, mag_bits(v[i]));
  m = max(m, (uint32_t)__shfl_xor((int)m, 1, 64));
  m = max(m, (uint32_t)__shfl_xor((int)m, 2, 64));
  m = max(m, (uint32_t)__shfl_xor((int)m, 4, 64));
  scale = block_scale(m);
  const float inv = __fdiv_rn(1.f, scale);
  return make_uint4(e4m3x4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv),
                    e4m3x4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv),
                    e4m3x4(v[8] * inv, v[9] * inv, v[10] * inv, v[11] * inv),
                    e4m3x4(v[12] * inv, v[13] * inv, v[14] * inv, v[15] * inv));
}

}  // namespace moe
