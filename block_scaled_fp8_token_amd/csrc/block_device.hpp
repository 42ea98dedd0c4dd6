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

// Sixteen bytes that are read once, and values that this kernel does not read again: past
// what the caches keep (what it measured stands at the kernels).
__device__ __forceinline__ u32x4 load_stream(const void* p) {
  return __builtin_nontemporal_load(static_cast<const u32x4*>(p));
}
template <typename V>
__device__ __forceinline__ void store_stream(void* p, V v) {
  __builtin_nontemporal_store(v, static_cast<V*>(p));
}

// A run of memory that the whole wavefront shares, read and written at 32-bit offsets
// without a branch: a lane whose offset is past `bytes` gets zeros, and its store is
// dropped.  (Branch-free, so that the compiler counts the memory instructions in flight
// exactly and waits for no more of them than it has to.)
__device__ __forceinline__ __amdgpu_buffer_rsrc_t shared_run(const void* base, uint32_t bytes) {
  const uint64_t a = reinterpret_cast<uint64_t>(base);
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)a);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(a >> 32));
  void* ptr = reinterpret_cast<void*>(((uint64_t)hi << 32) | lo);
  return __builtin_amdgcn_make_buffer_rsrc(ptr, (short)0, __builtin_amdgcn_readfirstlane((int)bytes), 0x00020000);
}
constexpr int kStream = 2;  // cache policy of a buffer instruction: streaming
__device__ __forceinline__ u32x4 run_load16(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, (int)off, 0, kStream));
}
__device__ __forceinline__ u32x2 run_load8(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(r, (int)off, 0, kStream));
}
__device__ __forceinline__ void run_store(__amdgpu_buffer_rsrc_t r, uint32_t off, u32x4 v) {
  __builtin_amdgcn_raw_buffer_store_b128(v, r, (int)off, 0, kStream);
}
__device__ __forceinline__ void run_store(__amdgpu_buffer_rsrc_t r, uint32_t off, u32x2 v) {
  __builtin_amdgcn_raw_buffer_store_b64(v, r, (int)off, 0, kStream);
}
__device__ __forceinline__ void run_store(__amdgpu_buffer_rsrc_t r, uint32_t off, uint32_t v) {
  __builtin_amdgcn_raw_buffer_store_b32(v, r, (int)off, 0, 0);
}

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
// The same of values that are not negative, whose bits order as they do: one instruction a
// step (a float maximum of moved bits costs three).
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_u(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, false);
}
__device__ __forceinline__ uint32_t max_u(uint32_t a, uint32_t b) { return a > b ? a : b; }
__device__ __forceinline__ uint32_t row16_max_bits(float v) {
  uint32_t u = __float_as_uint(v);
  u = max_u(u, dpp_u<kXor1>(u));
  u = max_u(u, dpp_u<kXor2>(u));
  u = max_u(u, dpp_u<kHalfMirror>(u));
  return max_u(u, dpp_u<kMirror>(u));
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

// UE8M0 byte of a group whose largest magnitude has these bits: e + 127 for the smallest e
// with 448 * 2^e >= max(amax, 1e-10).  448 is 1.75 * 2^8, so the exponent goes up by one
// where the mantissa is past 0x600000: that much below the carry into it.  Small groups
// end at 85, the floor's byte.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax_bits) {
  return max_u((amax_bits + 0x1FFFFFu) >> 23, 85 + 8) - 8;
}
// Largest magnitude of eight values (a NaN among them does not count).
__device__ __forceinline__ float amax8(const float* f) {
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = __builtin_fmaxf(amax, __builtin_fabsf(f[i]));
  return amax;
}
// UE8M0 byte of the 128 values that the sixteen lanes of a row hold, eight each.
__device__ __forceinline__ uint32_t group_byte(const float* f) { return scale_byte(row16_max_bits(amax8(f))); }
// Codes of eight values at the scale of a UE8M0 byte.  The hardware conversion divides by
// the scale before it rounds, so finite values (at most 448 scales by the choice of the
// byte) get the codes that multiplying, clamping and converting gives them, without those
// 16 instructions; a value that is not finite becomes the NaN code.
__device__ __forceinline__ u32x2 codes_at(const float* f, uint32_t byte) {
  typedef short s16x2 __attribute__((ext_vector_type(2)));
  const float scale = __uint_as_float(byte << 23);
  u32x2 o;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    s16x2 v = {0, 0};
    v = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(v, f[4 * i], f[4 * i + 1], scale, false);
    v = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(v, f[4 * i + 2], f[4 * i + 3], scale, true);
    o[i] = __builtin_bit_cast(uint32_t, v);
  }
  return o;
}
// The packed scale word of the four groups of a wavefront (512 columns) from each
// group's exponent byte (0 for a group past the row's end).
__device__ __forceinline__ uint32_t scale_word(uint32_t byte) {
  return (uint32_t)__builtin_amdgcn_readlane((int)byte, 0) | ((uint32_t)__builtin_amdgcn_readlane((int)byte, 16) << 8) |
         ((uint32_t)__builtin_amdgcn_readlane((int)byte, 32) << 16) |
         ((uint32_t)__builtin_amdgcn_readlane((int)byte, 48) << 24);
}

}  // namespace fp8bs
