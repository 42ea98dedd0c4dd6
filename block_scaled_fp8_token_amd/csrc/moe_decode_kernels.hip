// A mixture-of-experts layer for a few tokens, from the router's choice to the layer's
// output, in two launches:
//
//   moe_gate_up_kernel   y[t, j] = quantized(silu(x[t] W13g[e]^T) * (x[t] W13u[e]^T)),  e = ids[t, j]
//   moe_down_kernel      out[t]  = base[t] + sum_j weights[t, j] * (y[t, j] W2[e]^T)
//
// Every weight of an expert that some token has chosen is read once and used for all its
// tokens; with at most 64 tokens that reading is what the layer costs, so both kernels
// are built to keep it going: a wavefront owns 16 rows of a weight matrix, each lane loads
// its operand bytes of the scaled matrix instruction straight into registers four K-blocks
// ahead (streaming loads), and the few activation bytes come from the L2.
//
// Operands: v_mfma_f32_16x16x32_bf16 with the weights as the first operand (16 rows) and up
// to 16 tokens as the second; codes of 8 and 4 bits become bf16 with their power-of-two scale by
// one conversion for two, without rounding.  (The matrix instruction on e4m3 operands adds its
// products to about 2^-18 of their magnitudes; a gated activation next to the middle between
// two codes would go to the other one in some 4 of 10^4 places, against 1 in 10^6 here.  The
// conversions take a third of the vector units' time at the rate that the weights arrive.)
// Lane l = 16 c + r holds of a 128-wide K-block of row (or token) r: of e4m3 the columns
// 16 c .. 16 c + 15 and 64 + 16 c .. + 15, of e2m1 the columns 32 c .. 32 c + 31, eight of
// them a product; the result holds rows 4 c + i, i < 4, of token r.
#include "block_device.hpp"
#include "decode_launch.hpp"

namespace fp8bs {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
constexpr uint32_t kOut = 0x80000000u;  // an offset past every run: the load gives zeros

struct MoeArgs {
  MoeDecodeProblem m;
  uint8_t* y;       // e4m3 [T * topk][H]
  uint32_t* y_sf;   // [T * topk][ceil(H / 512)], the bytes of four groups to a word
};

__device__ __forceinline__ u32x4 cached16(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, (int)off, 0, 0));
}
__device__ __forceinline__ uint32_t cached4(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  return (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(r, (int)off, 0, 0);
}

// Four K-blocks (512 columns) of 16 rows of a weight matrix, as a lane holds them.
template <Weights F>
struct Unit {
  static constexpr int L = F == Weights::kW4 ? 1 : 2;
  u32x4 w[4][L];
  uint32_t s[F == Weights::kW4 ? 1 : 4];
  uint32_t s_ahead;  // 4-bit weights: the next unit's word of scales

  __device__ __forceinline__ void begin() {
    if constexpr (F == Weights::kW4) s[0] = s_ahead;
  }
};

// Sixteen rows of one expert's matrix [N][K], from row n0 (a multiple of 16).
template <Weights F>
struct Rows {
  __amdgpu_buffer_rsrc_t w, s;
  uint32_t at;
  int KB;

  __device__ __forceinline__ Rows(const uint8_t* weights, const void* scales, int64_t e, int N, int K, int n0, int lane)
      : KB(K / 128) {
    const int r = lane & 15, c = lane >> 4;
    const int64_t matrix = (int64_t)N * K;
    if constexpr (F == Weights::kW4) {
      const int units = (KB + 3) / 4;
      w = shared_run(weights + (e * matrix + (int64_t)n0 * K) / 2, (uint32_t)(8 * K));
      s = shared_run(static_cast<const uint8_t*>(scales) + ((e * N + n0) / 16) * (int64_t)units * 256, units * 256u);
      at = 16 * lane;
    } else {
      if constexpr (F == Weights::kShuffled) {
        // 4 KB of a K-block of 32 rows: pieces q = 0..3 of 1 KB, 16 bytes of (half, row) each; column
        // 64 (q / 2) + 32 half + 16 (q % 2)
        w = shared_run(weights + e * matrix + (int64_t)(n0 & ~31) * K, (uint32_t)(32 * K));
        at = (c & 1) * 1024 + (c >> 1) * 512 + 16 * ((n0 & 16) + r);
      } else {
        w = shared_run(weights + e * matrix + (int64_t)n0 * K, (uint32_t)(16 * K));
        at = r * K + 16 * c;
      }
      s = shared_run(static_cast<const float*>(scales) + (e * (N / 128) + n0 / 128) * KB, KB * 4u);
    }
  }
  // K-block j = 4 u + i
  __device__ __forceinline__ void load(Unit<F>& v, int j, int i) const {
    const uint32_t past = j < KB ? 0 : kOut;
    if constexpr (F == Weights::kW4) {
      v.w[i][0] = run_load16(w, (at + j * 1024) | past);
      if (i == 0) v.s_ahead = cached4(s, (uint32_t)(j * 64 + at / 4) | past);
    } else {
      const uint32_t o = at + j * (F == Weights::kShuffled ? 4096 : 128);
      v.w[i][0] = run_load16(w, o | past);
      v.w[i][1] = run_load16(w, (o + (F == Weights::kShuffled ? 2048 : 64)) | past);
      v.s[i] = cached4(s, (uint32_t)(j * 4) | past);
    }
  }
};

// Eight e4m3 codes as bf16 at a power-of-two scale.
__device__ __forceinline__ bf16x8 from_e4m3(uint32_t lo, uint32_t hi, float scale) {
  const bf16x2 v0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false);
  const bf16x2 v1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true);
  const bf16x2 v2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false);
  const bf16x2 v3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true);
  return bf16x8{v0[0], v0[1], v1[0], v1[1], v2[0], v2[1], v3[0], v3[1]};
}
// The scale of byte i of a word of UE8M0 bytes.
__device__ __forceinline__ float scale_of(uint32_t word, int i) { return __uint_as_float((word >> (8 * i) & 0xFF) << 23); }

// Columns 8 m .. 8 m + 7 (as the lane holds them) of K-block I of a unit.
template <Weights F, int I>
__device__ __forceinline__ bf16x8 rows_of(const Unit<F>& v, int m) {
  if constexpr (F == Weights::kW4) {
    const float scale = scale_of(v.s[0], I);
    const uint32_t w = v.w[I][0][m];
    const bf16x2 v0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0);
    const bf16x2 v1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1);
    const bf16x2 v2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2);
    const bf16x2 v3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3);
    return bf16x8{v0[0], v0[1], v1[0], v1[1], v2[0], v2[1], v3[0], v3[1]};
  } else {
    // block scales are powers of two, of which the exponent field counts
    const u32x4 w = v.w[I][m >> 1];
    return from_e4m3(w[2 * (m & 1)], w[2 * (m & 1) + 1], __uint_as_float(v.s[I] & 0x7F800000u));
  }
}
__device__ __forceinline__ bf16x8 tokens_of(const u32x4 (&x)[2], int m, float scale) {
  const u32x4 w = x[m >> 1];
  return from_e4m3(w[2 * (m & 1)], w[2 * (m & 1) + 1], scale);
}
// Where a lane's second 16 bytes of a K-block of a token lie behind the first, and the first
// ones of c: the weights' columns.
template <Weights F>
constexpr int kFirst = F == Weights::kW4 ? 32 : 16;
template <Weights F>
constexpr int kSecond = F == Weights::kW4 ? 16 : 64;

// The bytes of a scale word that belong to K-blocks past the end are cleared.
__device__ __forceinline__ uint32_t valid_bytes(uint32_t word, int blocks_left) {
  return blocks_left >= 4 ? word : blocks_left <= 0 ? 0 : word & ((1u << (8 * blocks_left)) - 1);
}

// The experts that some token has chosen, as bits; ids [T][topk] to LDS.  Every thread calls it.
__device__ __forceinline__ void chosen(const MoeDecodeProblem& m, int* ids, uint32_t* bits) {
  const int pairs = m.T * m.topk;
  if (threadIdx.x < 32) bits[threadIdx.x] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < pairs; i += blockDim.x) {
    const int e = m.ids[i];
    ids[i] = e;
    if (e >= 0 && e < m.E) atomicOr(&bits[e >> 5], 1u << (e & 31));
  }
  __syncthreads();
}

// ------------------------------------------------------------------ gate_up

template <Weights F>
__global__ __launch_bounds__(512) void moe_gate_up_kernel(const MoeArgs p) {
  __shared__ int ids[kMoeDecodeMaxT * kMoeDecodeMaxTopk];
  __shared__ uint32_t bits[32];
  __shared__ int token[64], pair[64];
  __shared__ float most[8][64];
  const MoeDecodeProblem& m = p.m;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int HB = m.H / 128;
  int a = blockIdx.x / HB;
  const int g = blockIdx.x - a * HB;
  chosen(m, ids, bits);
  int e = -1;
  for (int i = 0; i < (m.E + 31) / 32; ++i) {  // the a-th bit that is set
    uint32_t b = bits[i];
    const int n = __builtin_popcount(b);
    if (a < n) {
      for (; a > 0; --a) b &= b - 1;
      e = 32 * i + __builtin_ctz(b);
      break;
    }
    a -= n;
  }
  e = __builtin_amdgcn_readfirstlane(e);
  if (e < 0) return;
  // its tokens, in order (a token that names it twice has one column)
  if (wave == 0) {
    int mine = -1;
    if (lane < m.T)
      for (int j = m.topk - 1; j >= 0; --j)
        if (ids[lane * m.topk + j] == e) mine = lane * m.topk + j;
    const uint64_t have = __ballot(mine >= 0);
    const int at = __builtin_popcountll(have & ((1ull << lane) - 1));
    token[lane] = pair[lane] = -1;
    if (mine >= 0) {
      token[at] = lane;
      pair[at] = mine;
    }
  }
  __syncthreads();
  const int KB = m.K / 128, units = (KB + 3) / 4;
  const int c = lane >> 4, r = lane & 15;
  const Rows<F> gate(m.w13, m.s13, e, 2 * m.H, m.K, 128 * g + 16 * wave, lane);
  const Rows<F> up(m.w13, m.s13, e, 2 * m.H, m.K, m.H + 128 * g + 16 * wave, lane);
  const auto rq = shared_run(m.q, (uint32_t)((m.T - 1) * m.ldq + m.K));
  const auto rs = shared_run(m.sf, (uint32_t)(((units - 1) * m.ld_sf + m.T) * 4));

  auto body = [&](auto cb_tag) {
    constexpr int CB = decltype(cb_tag)::value;
    uint32_t q_at[CB], s_at[CB];
#pragma unroll
    for (int b = 0; b < CB; ++b) {
      const int t = token[16 * b + r];
      q_at[b] = t < 0 ? kOut : (uint32_t)(t * m.ldq + kFirst<F> * c);
      s_at[b] = t < 0 ? kOut : (uint32_t)(t * 4);
    }
    Unit<F> wg, wu;
    u32x4 x[4][CB][2];
    uint32_t xs[CB], xs_next[CB];
    v4f ag[CB], au[CB];
    auto load_x = [&](int j, int i) {
      const uint32_t past = j < KB ? 0 : kOut;
#pragma unroll
      for (int b = 0; b < CB; ++b) {
        x[i][b][0] = cached16(rq, (q_at[b] + 128 * j) | past);
        x[i][b][1] = cached16(rq, (q_at[b] + 128 * j + kSecond<F>) | past);
      }
    };
    auto load_xs = [&](int u) {
#pragma unroll
      for (int b = 0; b < CB; ++b)
        xs_next[b] = cached4(rs, u < units && s_at[b] != kOut ? s_at[b] + (uint32_t)(u * m.ld_sf * 4) : kOut);
    };
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      gate.load(wg, i, i);
      up.load(wu, i, i);
      load_x(i, i);
    }
    load_xs(0);
#pragma unroll
    for (int b = 0; b < CB; ++b) ag[b] = au[b] = v4f{0, 0, 0, 0};
    for (int u = 0; u < units; ++u) {
#pragma unroll
      for (int b = 0; b < CB; ++b) xs[b] = valid_bytes(xs_next[b], KB - 4 * u);
      load_xs(u + 1);
      wg.begin();
      wu.begin();
      auto step = [&](auto i_tag) {
        constexpr int I = decltype(i_tag)::value;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const bf16x8 vg = rows_of<F, I>(wg, k), vu = rows_of<F, I>(wu, k);
#pragma unroll
          for (int b = 0; b < CB; ++b) {
            const bf16x8 vx = tokens_of(x[I][b], k, scale_of(xs[b], I));
            ag[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vg, vx, ag[b], 0, 0, 0);
            au[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vu, vx, au[b], 0, 0, 0);
          }
        }
        const int j = 4 * u + 4 + I;
        gate.load(wg, j, I);
        up.load(wu, j, I);
        load_x(j, I);
      };
      step(std::integral_constant<int, 0>{});
      step(std::integral_constant<int, 1>{});
      step(std::integral_constant<int, 2>{});
      step(std::integral_constant<int, 3>{});
    }
    // silu(gate) * up in fp32, and the largest magnitude of each token's 128 columns
    float y[CB][4];
#pragma unroll
    for (int b = 0; b < CB; ++b) {
#pragma unroll
      for (int i = 0; i < 4; ++i) y[b][i] = ag[b][i] / (1.0f + expf(-ag[b][i])) * au[b][i];
      float v = __builtin_fmaxf(__builtin_fmaxf(__builtin_fabsf(y[b][0]), __builtin_fabsf(y[b][1])),
                                __builtin_fmaxf(__builtin_fabsf(y[b][2]), __builtin_fabsf(y[b][3])));
      v = __builtin_fmaxf(v, __shfl_xor(v, 16));
      v = __builtin_fmaxf(v, __shfl_xor(v, 32));
      if (c == 0) most[wave][16 * b + r] = v;
    }
    __syncthreads();
#pragma unroll
    for (int b = 0; b < CB; ++b) {
      float v = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) v = __builtin_fmaxf(v, most[i][16 * b + r]);
      const uint32_t byte = scale_byte(__float_as_uint(v));
      const int at = pair[16 * b + r];
      if (at >= 0) {
        typedef short s16x2 __attribute__((ext_vector_type(2)));
        const float scale = __uint_as_float(byte << 23);
        s16x2 o = {0, 0};
        o = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(o, y[b][0], y[b][1], scale, false);
        o = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(o, y[b][2], y[b][3], scale, true);
        *reinterpret_cast<uint32_t*>(p.y + (int64_t)at * m.H + 128 * g + 16 * wave + 4 * c) =
            __builtin_bit_cast(uint32_t, o);
        if (c == 0 && wave == 0) reinterpret_cast<uint8_t*>(p.y_sf)[(int64_t)at * 4 * ((HB + 3) / 4) + g] = (uint8_t)byte;
      }
    }
  };
  const int blocks = __builtin_amdgcn_readfirstlane(token[48] >= 0 ? 4 : token[32] >= 0 ? 3 : token[16] >= 0 ? 2 : 1);
  switch (blocks) {
    case 1: body(std::integral_constant<int, 1>{}); break;
    case 2: body(std::integral_constant<int, 2>{}); break;
    case 3: body(std::integral_constant<int, 3>{}); break;
    default: body(std::integral_constant<int, 4>{}); break;
  }
}

// ------------------------------------------------------------------ down and combine

template <Weights F, int CB>
__global__ __launch_bounds__(512) void moe_down_kernel(const MoeArgs p) {
  __shared__ int ids[kMoeDecodeMaxT * kMoeDecodeMaxTopk];
  __shared__ uint32_t bits[32];
  __shared__ uint16_t list[kMoeDecodeMaxE];
  __shared__ __attribute__((aligned(16))) float part[8][CB][64][4];
  const MoeDecodeProblem& m = p.m;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane >> 4, r = lane & 15;
  const int n0 = 16 * blockIdx.x;
  const int KB = m.H / 128, units = (KB + 3) / 4;
  chosen(m, ids, bits);
  for (int i = threadIdx.x; i < m.E; i += blockDim.x) {
    if (bits[i >> 5] >> (i & 31) & 1) {
      int rank = __builtin_popcount(bits[i >> 5] & ((1u << (i & 31)) - 1));
      for (int k = 0; k < i >> 5; ++k) rank += __builtin_popcount(bits[k]);
      list[rank] = (uint16_t)i;
    }
  }
  int active = 0;
  for (int k = 0; k < (m.E + 31) / 32; ++k) active += __builtin_popcount(bits[k]);
  active = __builtin_amdgcn_readfirstlane(active);
  __syncthreads();

  // this wavefront's units of the active experts' rows, in the experts' order
  const int total = active * units, u0 = total * wave / 8, u1 = total * (wave + 1) / 8;
  v4f sum[CB], acc[CB];
#pragma unroll
  for (int b = 0; b < CB; ++b) sum[b] = acc[b] = v4f{0, 0, 0, 0};
  const auto ry = shared_run(p.y, (uint32_t)(m.T * m.topk * m.H));
  const auto rs = shared_run(p.y_sf, (uint32_t)(m.T * m.topk * units * 4));
  if (u0 < u1) {
    // loads run one unit ahead of the products, and so does the expert that they are of
    int k_ahead = u0 / units, ua = u0 - k_ahead * units;
    int e_ahead = 0;
    uint32_t row[CB];  // the pair's row of y, per token
    auto find = [&]() {
      e_ahead = __builtin_amdgcn_readfirstlane(list[k_ahead]);
#pragma unroll
      for (int b = 0; b < CB; ++b) {
        const int t = 16 * b + r;
        row[b] = kOut;
        if (t < m.T)
          for (int j = m.topk - 1; j >= 0; --j)
            if (ids[t * m.topk + j] == e_ahead) row[b] = t * m.topk + j;
      }
    };
    Unit<F> w;
    u32x4 x[4][CB][2];
    uint32_t xs[CB], xs_next[CB];
    auto load_x = [&](int j, int i) {
#pragma unroll
      for (int b = 0; b < CB; ++b) {
        const uint32_t o = row[b] == kOut || j >= KB ? kOut : row[b] * m.H + 128 * j + kFirst<F> * c;
        x[i][b][0] = cached16(ry, o);
        x[i][b][1] = cached16(ry, o + kSecond<F>);
      }
    };
    auto load_xs = [&]() {
#pragma unroll
      for (int b = 0; b < CB; ++b)
        xs_next[b] = cached4(rs, row[b] == kOut ? kOut : (row[b] * units + ua) * 4);
    };
    find();
    {
      const Rows<F> rows(m.w2, m.s2, e_ahead, m.K, m.H, n0, lane);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        rows.load(w, 4 * ua + i, i);
        load_x(4 * ua + i, i);
      }
      load_xs();
    }
    for (int u = u0; u < u1; ++u) {
      const int now = ua;
      const int e = e_ahead;
#pragma unroll
      for (int b = 0; b < CB; ++b) xs[b] = valid_bytes(xs_next[b], KB - 4 * now);
      bool last = false;
      if (++ua == units) {
        ua = 0;
        ++k_ahead;
        last = true;
        if (u + 1 < u1) find();
      }
      last |= u + 1 == u1;
      const bool more = u + 1 < u1;
      const Rows<F> rows(m.w2, m.s2, e_ahead, m.K, m.H, n0, lane);
      if (more) load_xs();
      w.begin();
      auto step = [&](auto i_tag) {
        constexpr int I = decltype(i_tag)::value;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const bf16x8 v = rows_of<F, I>(w, k);
#pragma unroll
          for (int b = 0; b < CB; ++b)
            acc[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, tokens_of(x[I][b], k, scale_of(xs[b], I)), acc[b], 0, 0, 0);
        }
        if (more) {
          rows.load(w, 4 * ua + I, I);
          load_x(4 * ua + I, I);
        }
      };
      step(std::integral_constant<int, 0>{});
      step(std::integral_constant<int, 1>{});
      step(std::integral_constant<int, 2>{});
      step(std::integral_constant<int, 3>{});
      if (last) {
        // the expert's part of its tokens; the others' columns may hold what a weight that is not
        // finite makes of zeros, and are left out
#pragma unroll
        for (int b = 0; b < CB; ++b) {
          const int t = 16 * b + r;
          float weight = 0.0f;
          bool has = false;
          if (t < m.T)
            for (int j = 0; j < m.topk; ++j)
              if (ids[t * m.topk + j] == e) {
                weight += m.weights[t * m.topk + j];
                has = true;
              }
#pragma unroll
          for (int i = 0; i < 4; ++i) sum[b][i] = has ? __builtin_fmaf(weight, acc[b][i], sum[b][i]) : sum[b][i];
          acc[b] = v4f{0, 0, 0, 0};
        }
      }
    }
  }
#pragma unroll
  for (int b = 0; b < CB; ++b) *reinterpret_cast<v4f*>(part[wave][b][lane]) = sum[b];
  __syncthreads();
  // thread -> token and four columns (as the lanes hold them)
  for (int i = threadIdx.x; i < CB * 64; i += 512) {
    const int l = i & 63, t = 16 * (i >> 6) + (l & 15), n = n0 + 4 * (l >> 4);
    if (t >= m.T) continue;
    v4f v = {0, 0, 0, 0};
    if (m.base) {
      const u32x2 b = *reinterpret_cast<const u32x2*>(m.base + t * m.ld_base + n);
      v = v4f{bf16_lo(b[0]), bf16_hi(b[0]), bf16_lo(b[1]), bf16_hi(b[1])};
    }
    for (int k = 0; k < 8; ++k) v += *reinterpret_cast<const v4f*>(part[k][i >> 6][l]);
    *reinterpret_cast<u32x2*>(m.out + t * m.ld_out + n) = u32x2{bf16x2_rne(v[0], v[1]), bf16x2_rne(v[2], v[3])};
  }
}

template <Weights F>
hipError_t launch(const MoeArgs& a, hipStream_t stream) {
  const MoeDecodeProblem& m = a.m;
  const int pairs = m.T * m.topk, experts = m.E < pairs ? m.E : pairs;
  moe_gate_up_kernel<F><<<experts * (m.H / 128), 512, 0, stream>>>(a);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  const int grid = m.K / 16;
  switch ((m.T + 15) / 16) {
    case 1: moe_down_kernel<F, 1><<<grid, 512, 0, stream>>>(a); break;
    case 2: moe_down_kernel<F, 2><<<grid, 512, 0, stream>>>(a); break;
    case 3: moe_down_kernel<F, 3><<<grid, 512, 0, stream>>>(a); break;
    default: moe_down_kernel<F, 4><<<grid, 512, 0, stream>>>(a); break;
  }
  return hipGetLastError();
}

}  // namespace

size_t moe_decode_scratch_bytes(int64_t T, int64_t topk, int64_t H) {
  return (size_t)(T * topk) * (size_t)(H + 4 * ((H + 511) / 512));
}

hipError_t launch_moe_decode(const MoeDecodeProblem& p, Weights kind, void* scratch, hipStream_t stream) {
  MoeArgs a;
  a.m = p;
  a.y = static_cast<uint8_t*>(scratch);
  a.y_sf = reinterpret_cast<uint32_t*>(a.y + (int64_t)p.T * p.topk * p.H);
  switch (kind) {
    case Weights::kPlain: return launch<Weights::kPlain>(a, stream);
    case Weights::kShuffled: return launch<Weights::kShuffled>(a, stream);
    default: return launch<Weights::kW4>(a, stream);
  }
}

}  // namespace fp8bs
