// Device helpers of the kernels around the experts' products (routing, combine, the
// norms of the residual stream, the 8-bit activation checkpoint): reductions inside a
// wavefront by data-parallel moves (no LDS), and bf16 / e4m3 conversion of the eight
// values a lane holds.
#pragma once
#include "fp8bs_device.hpp"

namespace fp8bs {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// v of another lane of the same 16-lane row: quad_perm [1,0,3,2] and [2,3,0,1]
// (lane ^ 1, lane ^ 2), row_half_mirror (7 - lane in each eight) and row_mirror
// (15 - lane).  After the steps in this order every lane of the row holds the
// reduction of all sixteen.
template <int CTRL>
__device__ __forceinline__ float dpp_f(float v) {
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), CTRL, 0xf, 0xf, true));
}
constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kHalfMirror = 0x141, kMirror = 0x140;

__device__ __forceinline__ float row16_sum(float v) {
  v += dpp_f<kXor1>(v);
  v += dpp_f<kXor2>(v);
  v += dpp_f<kHalfMirror>(v);
  v += dpp_f<kMirror>(v);
  return v;
}
__device__ __forceinline__ float row16_max(float v) {
  v = __builtin_fmaxf(v, dpp_f<kXor1>(v));
  v = __builtin_fmaxf(v, dpp_f<kXor2>(v));
  v = __builtin_fmaxf(v, dpp_f<kHalfMirror>(v));
  v = __builtin_fmaxf(v, dpp_f<kMirror>(v));
  return v;
}
__device__ __forceinline__ float read_lane(float v, int lane) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane));
}
// Sum / max over the 64 lanes, the same value in every lane.  All lanes must be active.
__device__ __forceinline__ float wave_sum(float v) {
  v = row16_sum(v);
  return (read_lane(v, 0) + read_lane(v, 16)) + (read_lane(v, 32) + read_lane(v, 48));
}
__device__ __forceinline__ float wave_max(float v) {
  v = row16_max(v);
  return __builtin_fmaxf(__builtin_fmaxf(read_lane(v, 0), read_lane(v, 16)),
                         __builtin_fmaxf(read_lane(v, 32), read_lane(v, 48)));
}

// Sum over a workgroup of `waves` wavefronts (at most 16), the same value in every
// thread.  `part` is sixteen floats of LDS; a caller that reduces again uses another
// `part` in between (the barrier of that one separates the two uses of this one).
__device__ __forceinline__ float block_sum(float v, float* part, int waves) {
  v = wave_sum(v);
  if (waves == 1) return v;
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = 0.0f;
  for (int w = 0; w < waves; ++w) s += part[w];
  return s;
}

// Two fp32 values as packed bf16, round to nearest even (infinities and NaN kept).
__device__ __forceinline__ uint32_t bf16x2_rne(float a, float b) {
  const f32x2 v = {a, b};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}
__device__ __forceinline__ void unpack_bf16x8(u32x4 v, float* f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16_lo(v[i]);
    f[2 * i + 1] = bf16_hi(v[i]);
  }
}
__device__ __forceinline__ u32x4 pack_bf16x8(const float* f) {
  u32x4 v;
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = bf16x2_rne(f[2 * i], f[2 * i + 1]);
  return v;
}

// Eight codes e4m3 -> fp32.
__device__ __forceinline__ void unpack_e4m3x8(u32x2 v, float* f) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)v[i], false);
    const f32x2 hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)v[i], true);
    f[4 * i] = lo[0];
    f[4 * i + 1] = lo[1];
    f[4 * i + 2] = hi[0];
    f[4 * i + 3] = hi[1];
  }
}

// UE8M0 exponent of the 128 values that the sixteen lanes of a row hold, eight each.
__device__ __forceinline__ int group_exponent(const float* f) {
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = __builtin_fmaxf(amax, __builtin_fabsf(f[i]));
  return ue8m0_exponent(row16_max(amax));
}
// Codes of eight values at scale 2^e, as one 64-bit word.
__device__ __forceinline__ uint64_t codes_at(const float* f, int e) {
  const float s = exp2i(-e);  // exact: -e in [-120, 42]
  float g[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) g[i] = f[i] * s;
  const uint2 o = e4m3x8(g);
  return ((uint64_t)o.y << 32) | o.x;
}
// The packed scale word of the four groups of a wavefront (512 columns) from each
// group's exponent byte (0 for a group past the row's end).
__device__ __forceinline__ uint32_t scale_word(uint32_t byte) {
  return (uint32_t)__builtin_amdgcn_readlane((int)byte, 0) | ((uint32_t)__builtin_amdgcn_readlane((int)byte, 16) << 8) |
         ((uint32_t)__builtin_amdgcn_readlane((int)byte, 32) << 16) |
         ((uint32_t)__builtin_amdgcn_readlane((int)byte, 48) << 24);
}

}  // namespace fp8bs
