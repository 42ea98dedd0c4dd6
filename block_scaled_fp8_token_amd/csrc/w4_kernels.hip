// Products of a few rows with weights of 4 bits under group scales, and what makes those
// weights: the quantization in row order and the layout that the products read.
//
// The layout.  Codes lie in tiles of 16 rows by 128 columns, 1 KB each, that a wavefront
// loads with one 16-byte instruction: lane 16 c + r holds row r,
//   e2m1      columns 32 c .. 32 c + 31 in order (one scale, and the operand of the scaled
//             matrix instruction as it is)
//   integers  in word i the columns 32 i + 8 c + 0, 2, 4, 6, 1, 3, 5, 7 (so the same word of
//             every lane lies in one group, and one shift and mask give two neighbours)
// Scales lie in units of 512 columns: e2m1 [tile][unit][lane][4 blocks], integers
// [tile][unit][16 rows][groups of the unit], as a lane reads them in one piece.
#include "block_device.hpp"
#include "decode_launch.hpp"

namespace fp8bs {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
constexpr uint32_t kOut = 0x80000000u;  // an offset past every run: the load gives zeros

// ------------------------------------------------------------------ product

// out[t][n] = sum over k of x[t][k] w[n][k] for 16 rows n of w and up to 16 CB tokens t.
// GP is the number of groups in 128 columns (of integers; 0: e2m1), Z whether they have zero
// points.  The tokens are the first operand of v_mfma_f32_16x16x32_bf16 and the weights the
// second, so the result's lane 16 c + r holds tokens 4 c + i of row r, and a group's scale is
// one number a lane.
//
// e2m1 codes become bf16 with their scale by one conversion for two (exact: a power of two).
// Integer codes c become 16 + c by putting them into the mantissa of a bf16, a shift and a
// mask for two; with S = sum of x over the group (a product with ones, in the same lanes),
//   sum x s (c - z) = s (sum x (16 + c) - (16 + z) S).
// 16 is the smallest offset that takes all sixteen codes; the subtraction costs the fp32 sum
// at most (16 + 15 + 16 + 15) / 1 of its relative error in the largest term, far under the
// bf16 rounding of the result.
template <int GP, bool Z, int CB>
__global__ __launch_bounds__(256) void w4_gemv_kernel(const W4Problem p) {
  constexpr bool E2M1 = GP == 0;
  constexpr int NS = E2M1 ? 1 : 2 * GP, NZ = Z ? GP : 1;  // words of scales and zero points a lane and unit
  __shared__ __attribute__((aligned(16))) float part[4][CB][64][4];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane >> 4, r = lane & 15;
  const int64_t tile = blockIdx.x, t0 = (int64_t)blockIdx.y * 64;
  const int T = (int)(p.T - t0 < 16 * CB ? p.T - t0 : 16 * CB);
  const int KB = (int)(p.K / 128), units = (KB + 3) / 4;
  const auto rw = shared_run(p.codes + tile * KB * 1024, KB * 1024u);
  const auto rx = shared_run(p.x + t0 * p.ldx, (uint32_t)(((T - 1) * p.ldx + p.K) * 2));
  const auto rs = shared_run(static_cast<const uint8_t*>(p.scales) + tile * units * (E2M1 ? 256 : 128 * GP),
                             units * (E2M1 ? 256u : 128u * GP));
  const auto rz = shared_run(Z ? p.zeros + tile * units * (64 * GP) : p.codes, Z ? units * 64u * GP : 0u);
  uint32_t x_at[CB];
#pragma unroll
  for (int b = 0; b < CB; ++b)
    x_at[b] = 16 * b + r < T ? (uint32_t)((16 * b + r) * p.ldx * 2) + (E2M1 ? 64 * c : 16 * c) : kOut;

  const int u0 = units * wave / 4, u1 = units * (wave + 1) / 4;
  u32x4 w[4];
  uint32_t s[NS], z[NZ], s_next[NS], z_next[NZ];
  v4f acc[CB];
#pragma unroll
  for (int b = 0; b < CB; ++b) acc[b] = v4f{0, 0, 0, 0};
  auto load_w = [&](int j, int i) { w[i] = run_load16(rw, j < KB ? (uint32_t)(j * 1024 + 16 * lane) : kOut); };
  auto load_s = [&](int u) {
    const uint32_t past = u < units ? 0 : kOut;
    if constexpr (E2M1) {
      s_next[0] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(rs, (int)((uint32_t)(u * 256 + 4 * lane) | past), 0, 0);
    } else {
      const uint32_t o = (uint32_t)((u * 16 + r) * 8 * GP) | past;
#pragma unroll
      for (int i = 0; i < NS; i += 2) {
        const u32x2 v = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(rs, (int)(o + 4 * i), 0, 0));
        s_next[i] = v[0];
        s_next[i + 1] = v[1];
      }
      if constexpr (Z) {
#pragma unroll
        for (int i = 0; i < NZ; ++i)
          z_next[i] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(rz, (int)((uint32_t)((u * 16 + r) * 4 * GP + 4 * i) | past), 0, 0);
      }
    }
  };
  if (u0 < u1) {
    load_s(u0);
#pragma unroll
    for (int i = 0; i < 4; ++i) load_w(4 * u0 + i, i);
  }
  for (int u = u0; u < u1; ++u) {
#pragma unroll
    for (int i = 0; i < NS; ++i) s[i] = s_next[i];
#pragma unroll
    for (int i = 0; i < NZ; ++i) z[i] = Z ? z_next[i] : 0;
    load_s(u + 1 < u1 ? u + 1 : units);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int j = 4 * u + i;
      bf16x8 x[CB][4];
#pragma unroll
      for (int b = 0; b < CB; ++b)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          x[b][k] = __builtin_bit_cast(
              bf16x8, __builtin_amdgcn_raw_buffer_load_b128(
                          rx, (int)(j < KB ? x_at[b] + (uint32_t)(256 * j + (E2M1 ? 16 : 64) * k) : kOut), 0, 0));
      bf16x8 v[4];
      if constexpr (E2M1) {
        const uint32_t byte = (s[0] >> (8 * i)) & 0xFF;
        const float scale = __uint_as_float(byte ? byte << 23 : 0x400000u);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const bf16x2 v0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[i][k], scale, 0);
          const bf16x2 v1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[i][k], scale, 1);
          const bf16x2 v2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[i][k], scale, 2);
          const bf16x2 v3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[i][k], scale, 3);
          v[k] = bf16x8{v0[0], v0[1], v1[0], v1[1], v2[0], v2[1], v3[0], v3[1]};
        }
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t d = w[i][k];
          const u32x4 o = {((d << 3) & 0x00780078u) | 0x41804180u, ((d >> 1) & 0x00780078u) | 0x41804180u,
                           ((d >> 5) & 0x00780078u) | 0x41804180u, ((d >> 9) & 0x00780078u) | 0x41804180u};
          v[k] = __builtin_bit_cast(bf16x8, o);
        }
      }
      load_w(j + 4 < 4 * u1 ? j + 4 : KB, i);
      if constexpr (E2M1) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int b = 0; b < CB; ++b) acc[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[b][k], v[k], acc[b], 0, 0, 0);
      } else {
        const __bf16 one = (__bf16)1.0f;
        const bf16x8 ones = {one, one, one, one, one, one, one, one};
#pragma unroll
        for (int gr = 0; gr < GP; ++gr) {
          const int at = i * GP + gr;
          const float scale = at & 1 ? bf16_hi(s[at / 2]) : bf16_lo(s[at / 2]);
          const float off = Z ? 16.0f + (float)((z[at / 4] >> (8 * (at % 4))) & 0xFF) : 24.0f;
#pragma unroll
          for (int b = 0; b < CB; ++b) {
            v4f d = {0, 0, 0, 0}, sx = {0, 0, 0, 0};
#pragma unroll
            for (int k = gr * (4 / GP); k < (gr + 1) * (4 / GP); ++k) {
              d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[b][k], v[k], d, 0, 0, 0);
              sx = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[b][k], ones, sx, 0, 0, 0);
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) acc[b][q] = __builtin_fmaf(scale, __builtin_fmaf(-off, sx[q], d[q]), acc[b][q]);
          }
        }
      }
    }
  }
#pragma unroll
  for (int b = 0; b < CB; ++b) *reinterpret_cast<v4f*>(part[wave][b][lane]) = acc[b];
  __syncthreads();
  for (int i = threadIdx.x; i < CB * 256; i += 256) {
    const int n = i & 15, t = i >> 4;  // of lane 16 (t % 16 / 4) + n, register t % 4
    if (t < T && tile * 16 + n < p.N) {
      const int l = 16 * ((t & 15) >> 2) + n, b = t >> 4, q = t & 3;
      const float v = (part[0][b][l][q] + part[1][b][l][q]) + (part[2][b][l][q] + part[3][b][l][q]);
      p.out[(t0 + t) * p.ld_out + tile * 16 + n] = (uint16_t)(bf16x2_rne(v, v) & 0xFFFF);
    }
  }
}

// ------------------------------------------------------------------ weights

// A lane takes eight columns, GROUP / 8 neighbours a group.  rows * K values in all.
template <bool E2M1, bool Z>
__global__ __launch_bounds__(256) void w4_quant_kernel(const uint16_t* __restrict__ w, int64_t pieces, int group,
                                                       uint8_t* __restrict__ codes, void* __restrict__ scales,
                                                       uint8_t* __restrict__ zeros) {
  const int64_t stride = (int64_t)gridDim.x * 256;
  const int lanes = group / 8;
  // a group's lanes take part in its reduction together: the number of pieces is a multiple of them
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < pieces; i += stride) {
    float f[8];
    unpack_bf16x8(load_stream(w + 8 * i), f);
    float lo = 0.0f, hi = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      lo = __builtin_fminf(lo, f[k]);
      hi = __builtin_fmaxf(hi, f[k]);
    }
    for (int d = 1; d < lanes; d *= 2) {
      lo = __builtin_fminf(lo, __shfl_xor(lo, d));
      hi = __builtin_fmaxf(hi, __shfl_xor(hi, d));
    }
    const float most = __builtin_fmaxf(-lo, hi);
    uint32_t word = 0;
    if constexpr (E2M1) {
      // smallest 2^e with 6 * 2^e >= most: 6 is 1.5 * 2^2
      const uint32_t up = (__float_as_uint(most) + 0x3FFFFFu) >> 23;
      const uint32_t byte = up < 3 ? 1 : up - 2;
      const float scale = __uint_as_float(byte << 23);
      word = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(word, f[0], f[1], scale, 0);
      word = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(word, f[2], f[3], scale, 1);
      word = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(word, f[4], f[5], scale, 2);
      word = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(word, f[6], f[7], scale, 3);
      if (i % lanes == 0) static_cast<uint8_t*>(scales)[i / lanes] = (uint8_t)byte;
    } else {
      const uint32_t bits = bf16x2_rne(Z ? (hi - lo) / 15.0f : most / 7.0f, 0.0f) & 0xFFFF;
      const float scale = bf16_lo(bits);
      float zero = 8.0f;
      if constexpr (Z) zero = scale > 0.0f ? __builtin_fminf(__builtin_rintf(-lo / scale), 15.0f) : 0.0f;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float v = scale > 0.0f ? __builtin_rintf(f[k] / scale) + zero : zero;
        word |= (uint32_t)__builtin_fminf(__builtin_fmaxf(v, 0.0f), 15.0f) << (4 * k);
      }
      if (i % lanes == 0) {
        static_cast<uint16_t*>(scales)[i / lanes] = (uint16_t)bits;
        if constexpr (Z) zeros[i / lanes] = (uint8_t)zero;
      }
    }
    reinterpret_cast<uint32_t*>(codes)[i] = word;
  }
}

// One thread a word of the tiles: [E][tiles][KB][64 lanes][4 words] from [E][N][K / 2].
template <bool E2M1>
__global__ __launch_bounds__(256) void w4_codes_kernel(const uint8_t* __restrict__ codes, int64_t words, int64_t N,
                                                       int64_t K, uint32_t* __restrict__ out) {
  const int64_t tiles = (N + 15) / 16, KB = K / 128;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < words; i += (int64_t)gridDim.x * 256) {
    const int k = (int)(i & 3), lane = (int)(i >> 2) & 63, c = lane >> 4;
    const int64_t block = i >> 8, kb = block % KB, tile = block / KB % tiles, e = block / KB / tiles;
    const int64_t n = tile * 16 + (lane & 15);
    uint32_t d = 0;
    if (n < N) {
      const int64_t col = 128 * kb + (E2M1 ? 32 * c + 8 * k : 32 * k + 8 * c);
      d = *reinterpret_cast<const uint32_t*>(codes + ((e * N + n) * K + col) / 2);
      if constexpr (!E2M1) {  // columns 0..7 to the nibbles 0, 4, 1, 5, 2, 6, 3, 7
        uint32_t even = 0, odd = 0;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          even |= (d >> (8 * q) & 15) << (4 * q);
          odd |= (d >> (8 * q + 4) & 15) << (4 * q);
        }
        d = even | odd << 16;
      }
    }
    out[i] = d;
  }
}

// One thread a scale (or zero point) of the units.
template <typename V, bool E2M1>
__global__ __launch_bounds__(256) void w4_scales_kernel(const V* __restrict__ scales, int64_t count, int64_t N,
                                                        int64_t groups, int per, V* __restrict__ out) {
  const int64_t tiles = (N + 15) / 16, units = (groups + per - 1) / per;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < count; i += (int64_t)gridDim.x * 256) {
    const int64_t unit = i / (16 * per), u = unit % units, tile = unit / units % tiles, e = unit / units / tiles;
    const int in = (int)(i - unit * 16 * per);
    // e2m1: byte b of lane 16 c + r is group 4 b + c of row r
    const int r = E2M1 ? (in >> 2) & 15 : in / per;
    const int64_t g = u * per + (E2M1 ? 4 * (in & 3) + (in >> 6) : in % per), n = tile * 16 + r;
    out[i] = n < N && g < groups ? scales[(e * N + n) * groups + g] : (V)0;
  }
}

template <int GP, bool Z>
hipError_t launch_gemv(const W4Problem& p, hipStream_t stream) {
  const dim3 grid((unsigned)((p.N + 15) / 16), (unsigned)((p.T + 63) / 64));
  const int64_t most = p.T < 64 ? p.T : 64;
  switch ((most + 15) / 16) {
    case 1: w4_gemv_kernel<GP, Z, 1><<<grid, 256, 0, stream>>>(p); break;
    case 2: w4_gemv_kernel<GP, Z, 2><<<grid, 256, 0, stream>>>(p); break;
    case 3: w4_gemv_kernel<GP, Z, 3><<<grid, 256, 0, stream>>>(p); break;
    default: w4_gemv_kernel<GP, Z, 4><<<grid, 256, 0, stream>>>(p); break;
  }
  return hipGetLastError();
}

unsigned blocks_of(int64_t threads) {
  const int64_t n = (threads + 255) / 256;
  return (unsigned)(n < 8192 ? n : 8192);
}

}  // namespace

hipError_t launch_w4_gemv(const W4Problem& p, hipStream_t stream) {
  if (p.e2m1) return launch_gemv<0, false>(p, stream);
  switch (128 / p.group) {
    case 1: return p.zeros ? launch_gemv<1, true>(p, stream) : launch_gemv<1, false>(p, stream);
    case 2: return p.zeros ? launch_gemv<2, true>(p, stream) : launch_gemv<2, false>(p, stream);
    default: return p.zeros ? launch_gemv<4, true>(p, stream) : launch_gemv<4, false>(p, stream);
  }
}

hipError_t launch_w4_quant(const uint16_t* w, int64_t rows, int64_t K, bool e2m1, int group, uint8_t* codes,
                           void* scales, uint8_t* zeros, hipStream_t stream) {
  const int64_t pieces = rows * K / 8;
  const unsigned grid = blocks_of(pieces);
  if (e2m1) w4_quant_kernel<true, false><<<grid, 256, 0, stream>>>(w, pieces, group, codes, scales, zeros);
  else if (zeros) w4_quant_kernel<false, true><<<grid, 256, 0, stream>>>(w, pieces, group, codes, scales, zeros);
  else w4_quant_kernel<false, false><<<grid, 256, 0, stream>>>(w, pieces, group, codes, scales, zeros);
  return hipGetLastError();
}

hipError_t launch_w4_preshuffle(const uint8_t* codes, const void* scales, const uint8_t* zeros, int64_t E, int64_t N,
                                int64_t K, bool e2m1, int group, uint8_t* codes_out, void* scales_out,
                                uint8_t* zeros_out, hipStream_t stream) {
  const int64_t tiles = E * ((N + 15) / 16), words = tiles * (K / 128) * 256;
  uint32_t* out = reinterpret_cast<uint32_t*>(codes_out);
  if (e2m1) w4_codes_kernel<true><<<blocks_of(words), 256, 0, stream>>>(codes, words, N, K, out);
  else w4_codes_kernel<false><<<blocks_of(words), 256, 0, stream>>>(codes, words, N, K, out);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  const int64_t groups = K / group;
  const int per = 512 / group;
  const int64_t count = tiles * ((groups + per - 1) / per) * 16 * per;
  const unsigned grid = blocks_of(count);
  if (e2m1)
    w4_scales_kernel<uint8_t, true><<<grid, 256, 0, stream>>>(static_cast<const uint8_t*>(scales), count, N, groups, per,
                                                              static_cast<uint8_t*>(scales_out));
  else
    w4_scales_kernel<uint16_t, false><<<grid, 256, 0, stream>>>(static_cast<const uint16_t*>(scales), count, N, groups,
                                                                per, static_cast<uint16_t*>(scales_out));
  err = hipGetLastError();
  if (err != hipSuccess || !zeros) return err;
  w4_scales_kernel<uint8_t, false><<<grid, 256, 0, stream>>>(zeros, count, N, groups, per, zeros_out);
  return hipGetLastError();
}

}  // namespace fp8bs
