// Products of a few rows with weights of 4 bits under group scales, and what makes those
// weights: the quantization in row order and the layout that the products read.
//
// The layout.  Codes lie in tiles of 16 rows by 128 columns, 1 KB each, that a wavefront
// loads with one 16-byte instruction: lane 16 c + r holds row r,
//   e2m1      columns 32 c .. 32 c + 31 in order (one scale; a word is the eight columns of
//             one operand once they are bf16)
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

// A K-block of one tile as a lane holds it.  GP: groups in its 128 columns of integers (0: e2m1).
template <int GP, bool Z>
struct Block {
  static constexpr bool E2M1 = GP == 0;
  u32x4 w;
  uint32_t s[GP == 4 ? 2 : 1], z;

  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t rw, __amdgpu_buffer_rsrc_t rs, __amdgpu_buffer_rsrc_t rz, int q,
                                       int j, uint32_t past, int KB, uint32_t s_tile, uint32_t z_tile, int lane) {
    load_codes(rw, q, j, past, KB, lane);
    load_scales(rs, rz, q, j, past, s_tile, z_tile, lane);
  }
  __device__ __forceinline__ void load_codes(__amdgpu_buffer_rsrc_t rw, int q, int j, uint32_t past, int KB, int lane) {
    w = run_load16(rw, (uint32_t)((q * KB + j) * 1024 + 16 * lane) | past);
  }
  __device__ __forceinline__ void load_scales(__amdgpu_buffer_rsrc_t rs, __amdgpu_buffer_rsrc_t rz, int q, int j,
                                              uint32_t past, uint32_t s_tile, uint32_t z_tile, int lane) {
    const uint32_t u = (uint32_t)j >> 2, k = (uint32_t)j & 3, r = lane & 15;
    if constexpr (E2M1) {
      s[0] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b8(rs, (int)((q * s_tile + u * 256 + 4 * lane + k) | past), 0, 0);
    } else {
      const uint32_t o = (q * s_tile + (u * 16 + r) * 8 * GP + k * 2 * GP) | past;
      if constexpr (GP == 1) s[0] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b16(rs, (int)o, 0, 0);
      if constexpr (GP == 2) s[0] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(rs, (int)o, 0, 0);
      if constexpr (GP == 4) {
        const u32x2 v = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(rs, (int)o, 0, 0));
        s[0] = v[0];
        s[1] = v[1];
      }
      if constexpr (Z) {
        const uint32_t oz = (q * z_tile + (u * 16 + r) * 4 * GP + k * GP) | past;
        if constexpr (GP == 1) z = (uint32_t)__builtin_amdgcn_raw_buffer_load_b8(rz, (int)oz, 0, 0);
        if constexpr (GP == 2) z = (uint32_t)__builtin_amdgcn_raw_buffer_load_b16(rz, (int)oz, 0, 0);
        if constexpr (GP == 4) z = (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(rz, (int)oz, 0, 0);
      }
    }
  }
  // The codes as bf16: e2m1 with their scale, integers as 16 + c.
  __device__ __forceinline__ void decode(bf16x8 (&v)[4]) const {
    if constexpr (E2M1) {
      const uint32_t byte = s[0] & 0xFF;
      const float scale = __uint_as_float(byte ? byte << 23 : 0x400000u);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const bf16x2 v0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[k], scale, 0);
        const bf16x2 v1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[k], scale, 1);
        const bf16x2 v2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[k], scale, 2);
        const bf16x2 v3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[k], scale, 3);
        v[k] = bf16x8{v0[0], v0[1], v1[0], v1[1], v2[0], v2[1], v3[0], v3[1]};
      }
    } else {
      // mantissa bits of a code, and 16 in bf16, twice; in registers, so that both take one instruction
      uint32_t mask = 0x00780078u, base = 0x41804180u;
      asm("" : "+s"(mask), "+v"(base));
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t d = w[k];
        const u32x4 o = {((d << 3) & mask) | base, ((d >> 1) & mask) | base, ((d >> 5) & mask) | base,
                         ((d >> 9) & mask) | base};
        v[k] = __builtin_bit_cast(bf16x8, o);
      }
    }
  }
  __device__ __forceinline__ float scale(int g) const { return g & 1 ? bf16_hi(s[g / 2]) : bf16_lo(s[g / 2]); }
  __device__ __forceinline__ float zero(int g) const { return (float)((z >> (8 * g)) & 0xFF); }
};

// The scales (and zero points) of a unit of four K-blocks of one tile, as they lie side by side: one or two loads where each
// K-block's own took four to eight.
template <int GP, bool Z>
struct UnitScales {
  static constexpr int NS = GP == 0 ? 1 : 2 * GP, NZ = Z ? GP : 1;
  uint32_t s[NS], z[NZ];

  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t rs, __amdgpu_buffer_rsrc_t rz, uint32_t s_at, uint32_t z_at,
                                       int u, uint32_t past, int lane) {
    const uint32_t at = (s_at + (GP == 0 ? u * 256 + 4 * lane : (u * 16 + (lane & 15)) * 8 * GP)) | past;
    words<NS>(s, rs, at);
    if constexpr (Z) words<NZ>(z, rz, (z_at + (u * 16 + (lane & 15)) * 4 * GP) | past);
  }
  template <int N>
  static __device__ __forceinline__ void words(uint32_t (&to)[N], __amdgpu_buffer_rsrc_t r, uint32_t at) {
    if constexpr (N == 1) {
      to[0] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(r, (int)at, 0, 0);
    } else if constexpr (N == 2) {
      const u32x2 v = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(r, (int)at, 0, 0));
      to[0] = v[0];
      to[1] = v[1];
    } else {
#pragma unroll
      for (int i = 0; i < N; i += 4) {
        const u32x4 v = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, (int)(at + 4 * i), 0, 0));
#pragma unroll
        for (int k = 0; k < 4; ++k) to[i + k] = v[k];
      }
    }
  }
  // Those of K-block I.
  template <int I>
  __device__ __forceinline__ void give(Block<GP, Z>& b) const {
    if constexpr (GP == 0) b.s[0] = s[0] >> (8 * I);
    if constexpr (GP == 1) b.s[0] = s[I / 2] >> (16 * (I & 1));
    if constexpr (GP == 2) b.s[0] = s[I];
    if constexpr (GP == 4) {
      b.s[0] = s[2 * I];
      b.s[1] = s[2 * I + 1];
    }
    if constexpr (Z) b.z = GP == 4 ? z[I % NZ] : GP == 2 ? z[I / 2 % NZ] >> (16 * (I & 1)) : z[0] >> (8 * I);
  }
};

__device__ __forceinline__ bf16x8 eight_of(float v) {
  const __bf16 b = (__bf16)v;
  return bf16x8{b, b, b, b, b, b, b, b};
}

// acc[q] += x (16 tokens) times a K-block of RT tiles.  x: the lane's four operands.
template <int GP, bool Z, int RT>
__device__ __forceinline__ void multiply(v4f (&acc)[RT], const bf16x8 (&x)[4], const Block<GP, Z> (&w)[RT],
                                         const bf16x8 (&v)[RT][4]) {
  if constexpr (GP == 0) {
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int q = 0; q < RT; ++q) acc[q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[k], v[q][k], acc[q], 0, 0, 0);
  } else {
    constexpr int N = GP == 0 ? 4 : 4 / GP;  // operands a group
    // what the codes' values have too much: with zero points 16, without them 24
    const bf16x8 much = eight_of(Z ? -16.0f : -24.0f), ones = eight_of(1.0f);
#pragma unroll
    for (int g = 0; g < GP; ++g) {
      v4f o = {0, 0, 0, 0}, sx = {0, 0, 0, 0};
#pragma unroll
      for (int k = g * N; k < (g + 1) * N; ++k) {  // the same for every tile
        o = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[k], much, o, 0, 0, 0);
        if constexpr (Z) sx = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[k], ones, sx, 0, 0, 0);
      }
#pragma unroll
      for (int q = 0; q < RT; ++q) {
        v4f d = o;
#pragma unroll
        for (int k = g * N; k < (g + 1) * N; ++k) d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[k], v[q][k], d, 0, 0, 0);
        const float s = w[q].scale(g);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          acc[q][i] = __builtin_fmaf(s, Z ? __builtin_fmaf(-w[q].zero(g), sx[i], d[i]) : d[i], acc[q][i]);
      }
    }
  }
  // the sums are brought up to here before anything after it: left to itself the compiler puts them off and
  // keeps what they are of in registers
#pragma unroll
  for (int q = 0; q < RT; ++q) asm volatile("" : "+v"(acc[q]));
}

// ------------------------------------------------------------------ product

// out[t][n] = sum over k of x[t][k] w[n][k] for 16 rows n of w and up to 16 CB tokens t.
// GP is the number of groups in 128 columns (of integers; 0: e2m1), Z whether they have zero
// points.  The tokens are the first operand of v_mfma_f32_16x16x32_bf16 and the weights the
// second, so the result's lane 16 c + r holds tokens 4 c + i of row r, and a group's scale is
// one number a lane.
//
// e2m1 codes become bf16 with their scale by one conversion for two (exact: a power of two).
// Integer codes c become 16 + c by putting them into the mantissa of a bf16, a shift and a
// mask for two, and a second product takes 16 + z times the sum of x off again:
//   sum x s (c - z) = s (sum x (16 + c) - sum x (16 + z)).
// 16 is the smallest offset that takes all sixteen codes: the fp32 sum's error grows by the ratio
// of 16 + c to |c - z|, far under the bf16 rounding of the result.
template <int GP, bool Z, int SL, int CB, int RT, int NW>
__global__ __launch_bounds__(NW * 64, 2) void w4_gemv_kernel(const W4Problem p) {
  constexpr bool E2M1 = GP == 0;
  constexpr int D = CB == 1 ? 4 : 2;  // K-blocks ahead, as registers allow (more spills: 20 tokens 30 us against 17)
  constexpr bool UNITS = CB <= 2;     // scales a unit at a time; with more tokens its registers are wanted elsewhere
  constexpr int TS = 16 / SL;         // tokens a slot
  __shared__ __attribute__((aligned(16))) float part[NW][CB * RT][64][4];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane >> 4, r = lane & 15;
  const int64_t tile = (int64_t)blockIdx.x * RT, t0 = (int64_t)blockIdx.y * 64;
  const int tiles = (int)((p.N + 15) / 16 - tile < RT ? (p.N + 15) / 16 - tile : RT);
  const int T = (int)(p.T - t0 < TS * CB ? p.T - t0 : TS * CB);
  const int KB = (int)(p.K / 128), units = (KB + 3) / 4;
  const uint32_t s_tile = units * (E2M1 ? 256u : 128u * GP), z_tile = units * 64u * GP;
  const auto rw = shared_run(p.codes + tile * KB * 1024, tiles * KB * 1024u);
  const auto rx = shared_run(p.x + t0 * p.ldx, (uint32_t)(((T - 1) * p.ldx + p.K) * 2));
  const auto rs = shared_run(static_cast<const uint8_t*>(p.scales) + tile * s_tile, tiles * s_tile);
  const auto rz = shared_run(Z ? p.zeros + tile * z_tile : p.codes, Z ? tiles * z_tile : 0u);
  uint32_t x_at[CB];
#pragma unroll
  for (int b = 0; b < CB; ++b)
    x_at[b] = 16 * b + r % TS < T ? (uint32_t)((16 * b + r % TS) * p.ldx * 2) + (E2M1 ? 64 * c : 16 * c) + 256 * (r / TS)
                                 : kOut;

  // this wavefront's K-blocks: whole units of four where there are enough of them
  int j0 = KB * wave / NW, j1 = KB * (wave + 1) / NW;
  if (units >= NW) {
    j0 = 4 * (units * wave / NW);
    j1 = 4 * (units * (wave + 1) / NW);
    j1 = j1 < KB ? j1 : KB;
  }
  const int first = j0 & ~3;
  Block<GP, Z> w[D][RT];
  UnitScales<GP, Z> scales[RT], scales_ahead[RT];
  bf16x8 x[D / SL][CB][4], x_ahead[CB][4];
  v4f acc[CB][SL][RT];
#pragma unroll
  for (int b = 0; b < CB; ++b)
#pragma unroll
    for (int i = 0; i < SL * RT; ++i) acc[b][i / RT][i % RT] = v4f{0, 0, 0, 0};
  auto load_w = [&](int j, int i) {
    const uint32_t past = j >= j0 && j < j1 ? 0 : kOut;
#pragma unroll
    for (int q = 0; q < RT; ++q) {
      w[i][q].load_codes(rw, q, j, past, KB, lane);
      if constexpr (!UNITS) w[i][q].load_scales(rs, rz, q, j, past, s_tile, z_tile, lane);
    }
  };
  auto load_s = [&](int j) {
#pragma unroll
    for (int q = 0; UNITS && q < RT; ++q) scales_ahead[q].load(rs, rz, q * s_tile, q * z_tile, j >> 2, j < j1 ? 0 : kOut, lane);
  };
  // tokens of the SL K-blocks from j; a slot past the range has zeros (what lies there is the next token's, and a value
  // of it that is not finite would not vanish against weights of zero)
  auto load_x = [&](int j, bf16x8(&to)[CB][4]) {
    const uint32_t past = j + r / TS >= j0 && j + r / TS < j1 ? 0 : kOut;
#pragma unroll
    for (int b = 0; b < CB; ++b)
#pragma unroll
      for (int k = 0; k < 4; ++k)
        to[b][k] = __builtin_bit_cast(bf16x8, __builtin_amdgcn_raw_buffer_load_b128(
                                                    rx, (int)((x_at[b] + (uint32_t)(256 * j + (E2M1 ? 16 : 64) * k)) | past), 0, 0));
  };
#pragma unroll
  for (int i = 0; i < D; ++i) {
    load_w(first + i, i);
    if (i % SL == 0) load_x(first + i, x[i / SL]);
    if (i == 0) load_s(first);
    __builtin_amdgcn_sched_barrier(0);  // in the loop's order, or its waits are for all of them
  }
  auto step = [&](int j, auto i_tag) {
    constexpr int I = decltype(i_tag)::value, IX = I % D / SL, S = I % SL;
    if constexpr (SL == D && S == 0) load_x(j + D, x_ahead);
    if constexpr (I == 0) load_s(j + 4);
    bf16x8 v[RT][4];
#pragma unroll
    for (int q = 0; q < RT; ++q) {
      if constexpr (UNITS) scales[q].template give<I>(w[I % D][q]);
      w[I % D][q].decode(v[q]);
    }
#pragma unroll
    for (int b = 0; b < CB; ++b) multiply<GP, Z, RT>(acc[b][S], x[IX][b], w[I % D], v);
    load_w(j + D, I % D);
    if constexpr (SL < D && S == SL - 1) load_x(j - S + D, x[IX]);
    __builtin_amdgcn_sched_barrier(0);  // the loads stay here: D K-blocks ahead of their products
  };
  for (int j = first; j < j1; j += 4) {
    // K-blocks outside the range have weights and tokens of zeros
#pragma unroll
    for (int q = 0; UNITS && q < RT; ++q) scales[q] = scales_ahead[q];
    step(j, std::integral_constant<int, 0>{});
    step(j + 1, std::integral_constant<int, 1>{});
    step(j + 2, std::integral_constant<int, 2>{});
    step(j + 3, std::integral_constant<int, 3>{});
    if constexpr (SL == D) {
#pragma unroll
      for (int k = 0; k < 4; ++k) x[0][0][k] = x_ahead[0][k];
    }
  }
  // of the rows 4 c + i, slot s has its own: those of c / (4 / SL) == s
#pragma unroll
  for (int b = 0; b < CB; ++b)
#pragma unroll
    for (int q = 0; q < RT; ++q) {
      v4f v = acc[b][0][q];
#pragma unroll
      for (int i = 1; i < SL; ++i)
        if (c / (4 / SL) == i) v = acc[b][i][q];
      *reinterpret_cast<v4f*>(part[wave][b * RT + q][lane]) = v;
    }
  __syncthreads();
  for (int i = threadIdx.x; i < CB * RT * 16 * TS; i += NW * 64) {
    // row n of tile q and token t: register t % 4 of lanes 16 c + n, c = t % 16 / 4 and the same of the other slots
    const int n = i % (16 * RT), q = n >> 4, t = i / (16 * RT);
    if (t < T && tile * 16 + n < p.N) {
      const int l = 16 * ((t & 15) >> 2) + (n & 15), at = (t >> 4) * RT + q;
      float v = 0.0f;
#pragma unroll
      for (int k = 0; k < NW; ++k)
#pragma unroll
        for (int s2 = 0; s2 < SL; ++s2) v += part[k][at][l + 64 / SL * s2][t & 3];
      p.out[(t0 + t) * p.ld_out + tile * 16 + n] = (uint16_t)(bf16x2_rne(v, v) & 0xFFFF);
    }
  }
}

// The same for up to 16 CB tokens that four wavefronts of different rows share through LDS, 64 RT rows a
// workgroup: the tokens are read from the L2 once for all of them, KC K-blocks at a time, each chunk while
// the one before it is worked on.  KS such groups of four divide K.  (16 x 18432 x 7168 in e2m1: 18.7 us; w4_gemv_kernel,
// whose wavefronts each read all tokens: 30.  64 tokens, integers: with KS = 2 45 us, with 1 54.)
template <int GP, bool Z, int CB, int RT, int KS>
__global__ __launch_bounds__(256 * KS, 2) void w4_batch_kernel(const W4Problem p) {
  constexpr bool E2M1 = GP == 0;
  constexpr int KC = CB <= 2 ? 4 : 2;  // K-blocks a chunk of tokens
  constexpr int PIECES = CB * KC;      // pieces of eight values that a thread brings
  constexpr int XB = KC * 16 * CB * 256;
  extern __shared__ __attribute__((aligned(16))) uint8_t x_lds[]; // [part][2][block][token][16 pieces, piece k at k ^ token % 16]
  const int tid = threadIdx.x & 255, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), part = __builtin_amdgcn_readfirstlane(threadIdx.x >> 8);
  uint8_t* const xl = x_lds + part * (2 * XB);
  const int c = lane >> 4, r = lane & 15;
  const int all_tiles = (int)((p.N + 15) / 16);
  const int tile = ((int)blockIdx.x * 4 + wave) * RT;
  const int64_t t0 = (int64_t)blockIdx.y * 64;
  const int T = (int)(p.T - t0 < 16 * CB ? p.T - t0 : 16 * CB);
  const int tiles = all_tiles - tile < 0 ? 0 : all_tiles - tile < RT ? all_tiles - tile : RT;
  const int KB = (int)(p.K / 128), units = (KB + 3) / 4;
  const int j0 = KB * part / KS, j1 = KB * (part + 1) / KS;  // this part's K-blocks
  const uint32_t s_tile = units * (E2M1 ? 256u : 128u * GP), z_tile = units * 64u * GP;
  const auto rw = shared_run(p.codes + (int64_t)tile * KB * 1024, tiles * KB * 1024u);
  const auto rx = shared_run(p.x + t0 * p.ldx, (uint32_t)(((T - 1) * p.ldx + p.K) * 2));
  const auto rs = shared_run(static_cast<const uint8_t*>(p.scales) + tile * (int64_t)s_tile, tiles * s_tile);
  const auto rz = shared_run(Z ? p.zeros + tile * (int64_t)z_tile : p.codes, Z ? tiles * z_tile : 0u);
  Block<GP, Z> w[KC][RT];
  u32x4 xn[PIECES];
  v4f acc[CB][RT];
#pragma unroll
  for (int b = 0; b < CB; ++b)
#pragma unroll
    for (int q = 0; q < RT; ++q) acc[b][q] = v4f{0, 0, 0, 0};
  auto load_w = [&](int j, int i) {
#pragma unroll
    for (int q = 0; q < RT; ++q) w[i][q].load(rw, rs, rz, q, j, j < j1 ? 0 : kOut, KB, s_tile, z_tile, lane);
  };
  // pieces of a chunk: thread -> (token, K-block, piece), the pieces of a token's chunk side by side
  auto load_x = [&](int j) {
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      const int at = i * 256 + tid, t = at / (16 * KC), k = at % (16 * KC);
      const uint32_t o = t < T && j + k / 16 < j1 ? (uint32_t)(t * p.ldx * 2 + j * 256 + k * 16) : kOut;
      xn[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rx, (int)o, 0, 0));
    }
  };
  auto store_x = [&](int buf) {
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      const int at = i * 256 + tid, t = at / (16 * KC), k = at % (16 * KC), kb = k / 16, piece = k & 15;
      *reinterpret_cast<u32x4*>(&xl[buf * XB + ((kb * 16 * CB + t) * 16 + (piece ^ (t & 15))) * 16]) = xn[i];
    }
  };
  load_x(j0);
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int i = 0; i < KC; ++i) {
    load_w(j0 + i, i);
    __builtin_amdgcn_sched_barrier(0);
  }
  store_x(0);
  __syncthreads();
  auto chunk = [&](int j, int buf) {
    load_x(j + KC);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < KC; ++i) {
      bf16x8 v[RT][4];
#pragma unroll
      for (int q = 0; q < RT; ++q) w[i][q].decode(v[q]);
#pragma unroll
      for (int b = 0; b < CB; ++b) {
        bf16x8 x[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          x[k] = *reinterpret_cast<const bf16x8*>(
              &xl[buf * XB + ((i * 16 * CB + 16 * b + r) * 16 + ((E2M1 ? 4 * c + k : 4 * k + c) ^ r)) * 16]);
        multiply<GP, Z, RT>(acc[b], x, w[i], v);
        __builtin_amdgcn_sched_barrier(0);
      }
      load_w(j + KC + i, i);
      __builtin_amdgcn_sched_barrier(0);
    }
    store_x(buf ^ 1);
    __syncthreads();
  };
  // (every part takes as many turns, a shorter one's last over zeros)
  const int turns = ((KB + KS - 1) / KS + KC - 1) / KC;
  for (int i = 0; i < turns; ++i) chunk(j0 + KC * i, i & 1);
  if constexpr (KS > 1) {
    // the parts' sums, in order (the tokens are no longer read)
    v4f* const sums = reinterpret_cast<v4f*>(x_lds);
    if (part > 0) {
#pragma unroll
      for (int i = 0; i < CB * RT; ++i) sums[((part - 1) * 4 + wave) * (64 * CB * RT) + 64 * i + lane] = acc[i / RT][i % RT];
    }
    __syncthreads();
    if (part > 0) return;
#pragma unroll
    for (int s = 0; s < KS - 1; ++s)
#pragma unroll
      for (int i = 0; i < CB * RT; ++i) acc[i / RT][i % RT] += sums[(s * 4 + wave) * (64 * CB * RT) + 64 * i + lane];
  }
#pragma unroll
  for (int b = 0; b < CB; ++b)
#pragma unroll
    for (int q = 0; q < RT; ++q)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = 16 * b + 4 * c + i;
        const int64_t n = (int64_t)(tile + q) * 16 + r;
        if (t < T && n < p.N) p.out[(t0 + t) * p.ld_out + n] = (uint16_t)(bf16x2_rne(acc[b][q][i], 0.0f) & 0xFFFF);
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
      // (hi - lo) / 15 by halves, which changes no bit but lets no difference of two finite values pass fp32's range
      const uint32_t bits = bf16x2_rne(Z ? (0.5f * hi - 0.5f * lo) / 7.5f : most / 7.0f, 0.0f) & 0xFFFF;
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

template <int GP, bool Z, int RT>
hipError_t launch_rows(const W4Problem& p, int most, dim3 grid, hipStream_t stream) {
  constexpr int NW = 4;
  if (most <= 4) w4_gemv_kernel<GP, Z, 4, 1, RT, NW><<<grid, NW * 64, 0, stream>>>(p);
  else if (most <= 8) w4_gemv_kernel<GP, Z, 2, 1, RT, NW><<<grid, NW * 64, 0, stream>>>(p);
  else if (most <= 16) w4_gemv_kernel<GP, Z, 1, 1, RT, NW><<<grid, NW * 64, 0, stream>>>(p);
  else if (most <= 32) w4_gemv_kernel<GP, Z, 1, 2, RT, NW><<<grid, NW * 64, 0, stream>>>(p);
  else if (most <= 48) w4_gemv_kernel<GP, Z, 1, 3, RT, NW><<<grid, NW * 64, 0, stream>>>(p);
  else w4_gemv_kernel<GP, Z, 1, 4, RT, NW><<<grid, NW * 64, 0, stream>>>(p);
  return hipGetLastError();
}

template <int GP, bool Z, int RT>
hipError_t launch_batch(const W4Problem& p, int most, unsigned chunks, hipStream_t stream) {
  constexpr int KS = 2;
  const dim3 grid((unsigned)(((p.N + 15) / 16 + 4 * RT - 1) / (4 * RT)), chunks);
  const int blocks = (most + 15) / 16;
  const int lds = KS * 2 * (blocks <= 2 ? 4 : 2) * 16 * blocks * 256;  // two chunks of tokens a part
  switch (blocks) {
    case 1: w4_batch_kernel<GP, Z, 1, RT, KS><<<grid, 256 * KS, lds, stream>>>(p); break;
    case 2: w4_batch_kernel<GP, Z, 2, RT, KS><<<grid, 256 * KS, lds, stream>>>(p); break;
    case 3: w4_batch_kernel<GP, Z, 3, RT, KS><<<grid, 256 * KS, lds, stream>>>(p); break;
    default: w4_batch_kernel<GP, Z, 4, RT, KS><<<grid, 256 * KS, lds, stream>>>(p); break;
  }
  return hipGetLastError();
}

// Which kernel.  Up to one tile a compute unit (256, or with few tokens, which cost little to read twice, 320), each is a
// workgroup's, so that all of them work; with more, a wavefront takes two and reads its tokens once for both.  From 5 tokens
// on, more than 512 tiles fill the chip with wavefronts that share the tokens through LDS, four tiles a workgroup, and from
// 1024 on eight.  Both sides, in us with K = 7168 where it is not named:
//   one tile a workgroup, two (1 token, int4 of 128)       257 tiles 6.1, 7.0   320: 6.7, 6.9   448: 7.0, 7.2 (of K = 18432
//                                                          12.9, 12.6)
//   (5 tokens, int4 of 32 with zero points; int4 of 128)   257 tiles 8.7, 9.5; 8.0, 7.7         320: 9.9, 9.7; 9.0, 7.7
//   (8 tokens, the same)                                   257 tiles 10.5, 9.8; 9.7, 8.4        320: 11.7, 10.0; 10.8, 8.5
//   (9 tokens, int4 of 128)                                200 tiles 7.7, 8.8   257: 11.3, 8.9
//   (64 tokens, int4 of 128 with zero points)              448 tiles, K = 2048: 19.7, 12.8
//   two tiles a workgroup, four through LDS (int4 of 128; e2m1)
//                    5 tokens   512 tiles 8.2, 13.2; 8.1, 11.3     576: 11.7, 13.0; 12.1, 11.3    960: 12.6, 14.0; 13.0, 12.5
//                   16 tokens   512 tiles 11.5, 13.5; 12.2, 12.0   576: 18.7, 13.7; 20.4, 12.2    960: 19.5, 14.3; 21.2, 13.4
//                   64 tokens   512 tiles 30.9, 32.4; 32.2, 27.0   576: 57.4, 32.6; 61.3, 27.2    960: 58.2, 34.4; 62.9, 29.1
//   four tiles through LDS, eight (16 tokens)              1024 tiles, int4 of 128: 14.6, 19.0    1152, e2m1: 22.6, 18.7
// So the ends are not the best for all: 320 costs up to 3 us with 5 to 8 tokens, except with zero points of small groups
// near 257 tiles; sharing the tokens of 5 costs 1.4 with integers, and 64 of e2m1 would gain by it from fewer tiles on (448
// of K = 18432: 75.8, 61.7); at 1024 tiles, which are one workgroup of four tiles for each compute unit, eight tiles cost 4 to 11.
template <int GP, bool Z>
hipError_t launch_gemv(const W4Problem& p, hipStream_t stream) {
  const int64_t tiles = (p.N + 15) / 16;
  const int most = (int)(p.T < 64 ? p.T : 64);
  const unsigned chunks = (unsigned)((p.T + 63) / 64);
  if (most > 4 && tiles >= 1024) return launch_batch<GP, Z, 2>(p, most, chunks, stream);
  if (most > 4 && tiles > 512) return launch_batch<GP, Z, 1>(p, most, chunks, stream);
  return tiles <= (most <= 8 ? 320 : 256) ? launch_rows<GP, Z, 1>(p, most, dim3((unsigned)tiles, chunks), stream)
                      : launch_rows<GP, Z, 2>(p, most, dim3((unsigned)((tiles + 1) / 2), chunks), stream);
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
