// A mixture-of-experts layer for a few tokens, from the router's choice to the layer's
// output, in two launches:
//
//   moe_gate_up_kernel   y[t, j] = quantized(silu(x[t] W13g[e]^T) * (x[t] W13u[e]^T)),  e = ids[t, j]
//   moe_down_kernel      out[t]  = base[t] + sum_j weights[t, j] * (y[t, j] W2[e]^T)
//
// Every weight of an expert that some token has chosen is read once and used for all its
// tokens; with at most 64 tokens that reading is what the layer costs, so both kernels
// are built to keep it going: a wavefront owns 16 or 32 rows of a weight matrix, each lane
// loads its operand's bytes straight into registers four K-blocks ahead (streaming loads,
// but cached ones of plain rows), and the few bytes of the tokens come from LDS or the L2.
//
// Operands: v_mfma_f32_16x16x32_bf16 with the weights as the first operand (16 rows) and up
// to 16 tokens as the second; codes of 8 and 4 bits become bf16 with their power-of-two scale by
// one conversion for two, without rounding.  (The matrix instruction on e4m3 operands adds its
// products to about 2^-18 of their magnitudes, and a gated activation next to the middle between
// two codes went to the other one in 2 of 16384 places of a test, one of them 3% of its token.
// The conversions run at the full vector rate.)
// Lane l = 16 c + r holds of a 128-wide K-block of row (or token) r: of e4m3 the columns
// 16 c .. 16 c + 15 and 64 + 16 c .. + 15, of e2m1 the columns 32 c .. 32 c + 31, eight of
// them a product; the result holds rows 4 c + i, i < 4, of token r.
#include <type_traits>

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
  float* y32;       // or y in fp32 [T * topk][H], where few experts are chosen
};

// Bytes of a row of y quantized in LDS: whole units of 512, and 16 more that keep the rows of a product's tokens apart in
// the banks.
__host__ __device__ constexpr int row_bytes(int H) { return (H + 511) / 512 * 512 + 16; }

// In how many parts the first kernel takes K.  Where few experts are chosen, workgroups of 128 columns would not be one a
// compute unit; they take 64 or 32 then, if y is small enough for every workgroup of the second kernel to quantize all of it.
int parts_of(const MoeDecodeProblem& m) {
  const int pairs = m.T * m.topk, experts = m.E < pairs ? m.E : pairs;
  if (pairs > 64 || m.T > 16 || experts * (m.H / 128) >= 256 || pairs * row_bytes(m.H) > 36864) return 1;
  return experts * (m.H / 64) >= 192 ? 2 : 4;
}

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
  using Scales = std::conditional_t<F == Weights::kW4, uint32_t, u32x4>;
  Scales s, s_ahead;  // of this unit and the next

  // Scales of the unit from K-block j, of KB in all (those past the end are zeros).
  __device__ __forceinline__ void begin(int j, int KB) {
    s = s_ahead;
    if constexpr (F != Weights::kW4) {
#pragma unroll
      for (int i = 1; i < 4; ++i) s[i] = j + i < KB ? s[i] : 0;
    }
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
  // K-block j = 4 u + i (nothing from `end` on)
  __device__ __forceinline__ void load(Unit<F>& v, int j, int i, int end) const {
    const uint32_t past = j < end ? 0 : kOut;
    if constexpr (F == Weights::kW4) {
      v.w[i][0] = run_load16(w, (at + j * 1024) | past);
      if (i == 0) v.s_ahead = cached4(s, (uint32_t)(j * 64 + at / 4) | past);
    } else {
      const uint32_t o = at + j * (F == Weights::kShuffled ? 4096 : 128);
      // Plain rows come half a cache line an instruction, so the line has to stay for the other half: streaming loads took
      // 183 us of a gate_up product of 16 tokens, these 152.
      v.w[i][0] = F == Weights::kPlain ? cached16(w, o | past) : run_load16(w, o | past);
      v.w[i][1] = F == Weights::kPlain ? cached16(w, (o + 64) | past) : run_load16(w, (o + 2048) | past);
      if (i == 0) v.s_ahead = cached16(s, (uint32_t)(j * 4) | past);
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
    const float scale = scale_of(v.s, I);
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

// The sums are brought up to here before anything after it: left to itself the compiler puts them off and keeps what
// they are of in registers.
template <int N>
__device__ __forceinline__ void pin(v4f (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+v"(v[i]));
}

// The bytes of a scale word that belong to K-blocks past the end are cleared.
__device__ __forceinline__ uint32_t valid_bytes(uint32_t word, int blocks_left) {
  return blocks_left >= 4 ? word : blocks_left <= 0 ? 0 : word & ((1u << (8 * blocks_left)) - 1);
}

// ------------------------------------------------------------------ routing

// The tokens of one expert as columns of the products, an entry each, in the tokens' order.
struct Columns {
  int token[64], pair[64];
  float weight[64];
};

// What a workgroup knows of the routing.  Up to 64 pairs (SMALL) lie one a lane and each wavefront finds its way among them
// by itself; more go to LDS, ids and weights [choice][token], with the list of the experts that some token has
// chosen.  Experts come in the order of the first pair that names them (SMALL) or in their own.
template <bool SMALL>
struct Routing {
  // SMALL: this lane's pair
  int id = -1;
  float weight = 0.0f;   // of the token's pairs of this expert together
  bool column = false;   // the first of them
  uint64_t firsts = 0;   // lanes whose expert no earlier pair has
  // else
  const int* ids = nullptr;
  const float* weights = nullptr;
  const uint16_t* list = nullptr;
  int T = 0, topk = 0, active = 0;

  static constexpr int words(int topk) { return SMALL ? 0 : 2 * 64 * topk + kMoeDecodeMaxE / 2 + 32; }

  // Every thread of the workgroup; lds: words(topk) words (none if SMALL).
  __device__ __forceinline__ void open(const MoeDecodeProblem& m, int lane, uint32_t* lds, bool with_weights) {
    T = m.T;
    topk = m.topk;
    const int pairs = m.T * m.topk;
    if constexpr (SMALL) {
      const bool has = lane < pairs;
      int e = has ? m.ids[lane] : -1;
      const float w = has && with_weights ? m.weights[lane] : 0.0f;
      id = e >= 0 && e < m.E ? e : -1;
      const int t = lane / topk;
      bool first = true;
      column = id >= 0;
      for (int p = 0; p < pairs; ++p) {
        const int other = __builtin_amdgcn_readlane(id, p);
        const bool same = other == id, mine = same && p / topk == t;
        if (mine) weight += read_lane(w, p);
        first &= !(same && p < lane);
        column &= !(mine && p < lane);
      }
      firsts = __ballot(id >= 0 && first);
      active = __builtin_popcountll(firsts);
    } else {
      int* to_ids = reinterpret_cast<int*>(lds);
      float* to_weights = reinterpret_cast<float*>(lds + 64 * topk);
      uint16_t* to_list = reinterpret_cast<uint16_t*>(lds + 128 * topk);
      uint32_t* bits = lds + 128 * topk + kMoeDecodeMaxE / 2;
      if (threadIdx.x < 32) bits[threadIdx.x] = 0;
      __syncthreads();
      for (int i = threadIdx.x; i < pairs; i += blockDim.x) {
        const int at = i % topk * 64 + i / topk, e = m.ids[i];
        to_ids[at] = e;
        if (with_weights) to_weights[at] = m.weights[i];
        if (e >= 0 && e < m.E) atomicOr(&bits[e >> 5], 1u << (e & 31));
      }
      __syncthreads();
      const int n = (m.E + 31) / 32;
      for (int i = threadIdx.x; i < m.E; i += blockDim.x) {
        if (bits[i >> 5] >> (i & 31) & 1) {
          int rank = __builtin_popcount(bits[i >> 5] & ((1u << (i & 31)) - 1));
          for (int k = 0; k < (i >> 5); ++k) rank += __builtin_popcount(bits[k]);
          to_list[rank] = (uint16_t)i;
        }
      }
      for (int k = 0; k < n; ++k) active += __builtin_popcount(bits[k]);
      active = __builtin_amdgcn_readfirstlane(active);
      __syncthreads();
      ids = to_ids;
      weights = to_weights;
      list = to_list;
    }
  }
  // The a-th of the active experts.
  __device__ __forceinline__ int expert(int a, int lane) const {
    if constexpr (SMALL) {
      const int rank = __builtin_popcountll(firsts & ((1ull << lane) - 1));
      return __builtin_amdgcn_readlane(id, (int)__builtin_ctzll(__ballot((firsts >> lane & 1) && rank == a)));
    } else {
      return __builtin_amdgcn_readfirstlane(list[a]);
    }
  }
  // Its columns, written by the calling wavefront; how many.
  __device__ __forceinline__ int columns(int e, int lane, Columns& to) const {
    int pair = -1, t = lane;
    float w = 0.0f;
    if constexpr (SMALL) {
      if (column && id == e) pair = lane;
      t = lane / topk;
      w = weight;
    } else {
      if (lane < T) {
#pragma unroll 8
        for (int j = topk - 1; j >= 0; --j) {
          if (ids[j * 64 + lane] == e) {
            pair = lane * topk + j;
            w += weights[j * 64 + lane];
          }
        }
      }
    }
    const uint64_t have = __ballot(pair >= 0);
    to.token[lane] = to.pair[lane] = -1;
    const int at = __builtin_popcountll(have & ((1ull << lane) - 1));
    if (pair >= 0) {
      to.token[at] = t;
      to.pair[at] = pair;
      to.weight[at] = w;
    }
    __builtin_amdgcn_wave_barrier();
    return __builtin_popcountll(have);
  }
};

// ------------------------------------------------------------------ gate_up

// One workgroup per chosen expert and 128 / KW columns of y.  Eight wavefronts own 16 rows of gate and 16 of up each, over a
// KW-th of K, and share the tokens of it through LDS, where they lie as bf16, a unit of four K-blocks ahead (each wavefront
// reading them from the L2 by itself: 163 us for 64 tokens; so 145).  With KW = 1 y goes out quantized.  The others are for
// few experts, where workgroups of 128 columns would leave compute units without work (1 token of 8 experts of 7168 x 2048:
// 46.3 us, with KW = 2 38.8; of 2 experts 38.4, 23.7 and with KW = 4 18.0); y stays in fp32 for moe_down_kernel to quantize, since no workgroup has a whole group.
template <Weights F, bool SMALL, int KW>
__global__ __launch_bounds__(512) void moe_gate_up_kernel(const MoeArgs p) {
  constexpr int RW = 8 / KW;
  extern __shared__ __attribute__((aligned(16))) uint32_t lds[];
  __shared__ Columns cols;
  __shared__ __attribute__((aligned(16))) float rest[KW == 1 ? 1 : KW - 1][RW][2][64][4];  // the other parts of K
  __shared__ float most[8][64];
  const MoeDecodeProblem& m = p.m;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int HB = m.H / (16 * RW), a = blockIdx.x / HB, g = blockIdx.x - a * HB;
  const int h0 = 16 * (RW * g + wave % RW), part = wave / RW;  // this wavefront's columns of y, and its part of K
  Routing<SMALL> routing;
  routing.open(m, lane, lds, false);
  if (a >= routing.active) return;
  const int e = routing.expert(a, lane);
  if (wave == 0) routing.columns(e, lane, cols);
  __syncthreads();
  const int KB = m.K / 128, units = (KB + 3) / 4;
  const int u0 = units * part / KW, u1 = units * (part + 1) / KW;
  const int c = lane >> 4, r = lane & 15;
  const Rows<F> gate(m.w13, m.s13, e, 2 * m.H, m.K, h0, lane);
  const Rows<F> up(m.w13, m.s13, e, 2 * m.H, m.K, m.H + h0, lane);
  const auto rq = shared_run(m.q, (uint32_t)((m.T - 1) * m.ldq + m.K));
  const auto rs = shared_run(m.sf, (uint32_t)(((units - 1) * m.ld_sf + m.T) * 4));

  auto body = [&](auto cb_tag) {
    constexpr int CB = decltype(cb_tag)::value;
    constexpr int GT = 512 / KW;           // threads that bring the tokens of one part of K
    constexpr int P = CB * 512 / GT;       // pieces of 16 codes that a thread brings
    constexpr bool DOUBLE = CB <= 2;       // two units of tokens in LDS
    constexpr int XB = 4 * 16 * CB * 256;  // bytes of one: [block][token][16 chunks of 8 columns, chunk k at k ^ token % 16]
    uint8_t* const xl = reinterpret_cast<uint8_t*>(lds + Routing<SMALL>::words(m.topk)) + part * (2 * XB);
    const int at0 = threadIdx.x % GT;
    uint32_t q_at[P], s_at[P];
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int t = cols.token[(i * GT + at0) >> 5];
      q_at[i] = t < 0 ? kOut : (uint32_t)(t * m.ldq + 16 * (at0 & 31));
      s_at[i] = t < 0 ? kOut : (uint32_t)(t * 4);
    }
    Unit<F> wg, wu;
    u32x4 xq[P];
    uint32_t xs[P];
    v4f ag[CB], au[CB];
    const int end = 4 * u1 < KB ? 4 * u1 : KB;
    auto load_w = [&](int j, int i) {
      gate.load(wg, j, i, end);
      up.load(wu, j, i, end);
    };
    auto load_x = [&](int u) {
#pragma unroll
      for (int i = 0; i < P; ++i) {
        const bool out = q_at[i] == kOut || 4 * u + ((at0 & 31) >> 3) >= end;
        xq[i] = cached16(rq, out ? kOut : q_at[i] + 512 * u);
        xs[i] = cached4(rs, out ? kOut : s_at[i] + (uint32_t)(u * m.ld_sf * 4));
      }
    };
    // as bf16 with their scale (exact), eight columns a chunk
    auto store_x = [&](int buf) {
#pragma unroll
      for (int i = 0; i < P; ++i) {
        const int t = (i * GT + at0) >> 5, piece = at0 & 31, block = piece >> 3, chunk = 2 * (piece & 7);
        const float scale = scale_of(xs[i], block);
        uint8_t* row = xl + (DOUBLE ? buf * XB : 0) + (block * 16 * CB + t) * 256;
        *reinterpret_cast<bf16x8*>(row + ((chunk ^ (t & 15)) << 4)) = from_e4m3(xq[i][0], xq[i][1], scale);
        *reinterpret_cast<bf16x8*>(row + (((chunk + 1) ^ (t & 15)) << 4)) = from_e4m3(xq[i][2], xq[i][3], scale);
      }
    };
    load_x(u0);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      load_w(4 * u0 + i, i);
      __builtin_amdgcn_sched_barrier(0);  // in the loop's order, or its waits are for all of them
    }
    store_x(0);
    __syncthreads();
#pragma unroll
    for (int b = 0; b < CB; ++b) ag[b] = au[b] = v4f{0, 0, 0, 0};
    // (all parts take as many turns, the shorter ones' last over zeros)
    const int turns = (units + KW - 1) / KW;
    for (int n = 0; n < turns; ++n) {
      const int u = u0 + n;
      load_x(u + 1);
      __builtin_amdgcn_sched_barrier(0);
      wg.begin(4 * u, KB);
      wu.begin(4 * u, KB);
      auto step = [&](auto i_tag) {
        constexpr int I = decltype(i_tag)::value;
        const uint8_t* from = xl + (DOUBLE ? (n & 1) * XB : 0) + I * 16 * CB * 256;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const bf16x8 vg = rows_of<F, I>(wg, k), vu = rows_of<F, I>(wu, k);
          const int chunk = F == Weights::kW4 ? 4 * c + k : 8 * (k >> 1) + 2 * c + (k & 1);
#pragma unroll
          for (int b = 0; b < CB; ++b) {
            const bf16x8 vx = *reinterpret_cast<const bf16x8*>(from + ((16 * b + r) * 16 + (chunk ^ r)) * 16);
            ag[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vg, vx, ag[b], 0, 0, 0);
            au[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vu, vx, au[b], 0, 0, 0);
          }
        }
        pin(ag);
        pin(au);
        load_w(4 * u + 4 + I, I);
        __builtin_amdgcn_sched_barrier(0);  // the loads stay here: four K-blocks ahead of their products
      };
      step(std::integral_constant<int, 0>{});
      step(std::integral_constant<int, 1>{});
      step(std::integral_constant<int, 2>{});
      step(std::integral_constant<int, 3>{});
      if constexpr (!DOUBLE) __syncthreads();
      store_x((n + 1) & 1);
      __syncthreads();
    }
    if constexpr (KW > 1) {
      static_assert(CB == 1);
      if (part > 0) {
        *reinterpret_cast<v4f*>(rest[part - 1][wave % RW][0][lane]) = ag[0];
        *reinterpret_cast<v4f*>(rest[part - 1][wave % RW][1][lane]) = au[0];
      }
      __syncthreads();
      if (part > 0) return;
#pragma unroll
      for (int i = 0; i < KW - 1; ++i) {
        ag[0] += *reinterpret_cast<const v4f*>(rest[i][wave][0][lane]);
        au[0] += *reinterpret_cast<const v4f*>(rest[i][wave][1][lane]);
      }
    }
    // silu(gate) * up in fp32
    v4f y[CB];
#pragma unroll
    for (int b = 0; b < CB; ++b)
#pragma unroll
      for (int i = 0; i < 4; ++i) y[b][i] = ag[b][i] / (1.0f + expf(-ag[b][i])) * au[b][i];
    if constexpr (KW > 1) {
#pragma unroll
      for (int b = 0; b < CB; ++b) {
        const int at = cols.pair[16 * b + r];
        if (at >= 0) *reinterpret_cast<v4f*>(p.y32 + (int64_t)at * m.H + h0 + 4 * c) = y[b];
      }
    } else {
      // the largest magnitude of each token's 128 columns
#pragma unroll
      for (int b = 0; b < CB; ++b) {
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
        const int at = cols.pair[16 * b + r];
        if (at >= 0) {
          typedef short s16x2 __attribute__((ext_vector_type(2)));
          const float scale = __uint_as_float(byte << 23);
          s16x2 o = {0, 0};
          o = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(o, y[b][0], y[b][1], scale, false);
          o = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(o, y[b][2], y[b][3], scale, true);
          *reinterpret_cast<uint32_t*>(p.y + (int64_t)at * m.H + h0 + 4 * c) = __builtin_bit_cast(uint32_t, o);
          if (c == 0 && wave == 0)
            reinterpret_cast<uint8_t*>(p.y_sf)[(int64_t)at * 4 * ((m.H + 511) / 512) + g] = (uint8_t)byte;
        }
      }
    }
  };
  const int blocks = __builtin_amdgcn_readfirstlane(cols.token[48] >= 0   ? 4
                                                    : cols.token[32] >= 0 ? 3
                                                    : cols.token[16] >= 0 ? 2
                                                                          : 1);
  if constexpr (KW > 1) {  // for at most 16 tokens
    body(std::integral_constant<int, 1>{});
  } else {
    switch (blocks) {
      case 1: body(std::integral_constant<int, 1>{}); break;
      case 2: body(std::integral_constant<int, 2>{}); break;
      case 3: body(std::integral_constant<int, 3>{}); break;
      default: body(std::integral_constant<int, 4>{}); break;
    }
  }
}

// ------------------------------------------------------------------ down and combine

// One workgroup per 16 RT output columns, over all chosen experts: its wavefronts share the list of (expert, four K-blocks)
// in equal runs.  An expert's products have its own tokens as columns, packed together; at the end of a run of one expert
// they are weighted and added to the wavefront's sums of the tokens in LDS, which are joined in order.  MAXC: 16-column
// blocks that an expert can have.  Y32: y comes in fp32, and the workgroup quantizes it into LDS while its first weights
// are on the way.
template <Weights F, bool SMALL, bool Y32, int MAXC, int NW, int RT>
__global__ __launch_bounds__(NW * 64) void moe_down_kernel(const MoeArgs p) {
  extern __shared__ __attribute__((aligned(16))) uint32_t lds[];  // sums [NW][16 MAXC tokens][16 RT], then the routing's
  __shared__ Columns cols[NW];
  const MoeDecodeProblem& m = p.m;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane >> 4, r = lane & 15;
  const int n0 = 16 * RT * blockIdx.x;
  const int KB = m.H / 128, units = (KB + 3) / 4;
  v4f* const sums = reinterpret_cast<v4f*>(lds) + wave * (64 * MAXC * RT);  // [token][4 RT of 4 columns]
#pragma unroll
  for (int i = 0; i < MAXC * RT; ++i) sums[64 * i + lane] = v4f{0, 0, 0, 0};
  Routing<SMALL> routing;
  routing.open(m, lane, lds + NW * 256 * MAXC * RT, true);

  const int total = routing.active * units, i0 = total * wave / NW, i1 = total * (wave + 1) / NW;
  const int rows_y = m.T * m.topk;
  const auto ry = shared_run(p.y, Y32 ? 0u : (uint32_t)(rows_y * m.H));
  const auto rs = shared_run(p.y_sf, Y32 ? 0u : (uint32_t)(rows_y * units * 4));
  uint8_t* const yl = reinterpret_cast<uint8_t*>(lds + NW * 256 * MAXC * RT);  // Y32: codes [pair][row_bytes], then bytes
  uint8_t* const yl_sf = yl + rows_y * row_bytes(m.H);
  int k = i0 / units, ua = i0 - k * units;  // the expert, and its unit whose weights are loaded
  int e = 0, left = i1 - i0;
  Unit<F> w[RT];
  auto load_w = [&](int of, int j, int i) {
#pragma unroll
    for (int q = 0; q < RT; ++q) Rows<F>(m.w2, m.s2, of, m.K, m.H, n0 + 16 * q, lane).load(w[q], j, i, KB);
  };
  if (left > 0) {
    e = routing.expert(k, lane);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      load_w(e, 4 * ua + i, i);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  if constexpr (Y32) {
    // a wavefront takes 512 columns of a pair, a lane eight
    for (int i = wave; i < rows_y * units; i += NW) {
      const int pair = i / units, u = i - pair * units, col = 512 * u + 8 * lane;
      u32x4 v[2] = {u32x4{0, 0, 0, 0}, u32x4{0, 0, 0, 0}};
      if (col < m.H) {
        v[0] = *reinterpret_cast<const u32x4*>(p.y32 + (int64_t)pair * m.H + col);
        v[1] = *reinterpret_cast<const u32x4*>(p.y32 + (int64_t)pair * m.H + col + 4);
      }
      float f[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) f[q] = __uint_as_float(v[q / 4][q % 4]);
      const uint32_t byte = group_byte(f);
      *reinterpret_cast<u32x2*>(yl + pair * row_bytes(m.H) + col) = codes_at(f, byte);
      if (lane % 16 == 0) yl_sf[i * 4 + lane / 16] = (uint8_t)byte;
    }
    __syncthreads();
  }
  if (left > 0) {
    while (left > 0) {
      // this wavefront's run of expert e: units ua .. ub - 1; then the next one's first unit
      const int ub = ua + left < units ? ua + left : units;
      left -= ub - ua;
      const int next = left > 0 ? routing.expert(k + 1, lane) : e;
      const int n = routing.columns(e, lane, cols[wave]);
      auto run = [&](auto cb_tag) {
        constexpr int CB = decltype(cb_tag)::value;
        constexpr int XD = CB <= 2 ? 4 : 1;  // K-blocks of y ahead, as registers allow
        uint32_t at[CB], s_at[CB];
#pragma unroll
        for (int b = 0; b < CB; ++b) {
          const int pair = cols[wave].pair[16 * b + r];
          // (of LDS a column without a token reads the first pair's row; nothing uses its sums)
          if constexpr (Y32) {
            at[b] = (pair < 0 ? 0 : pair * row_bytes(m.H)) + kFirst<F> * c;
            s_at[b] = pair < 0 ? 0 : pair * units * 4;
          } else {
            at[b] = pair < 0 ? kOut : (uint32_t)(pair * m.H + kFirst<F> * c);
            s_at[b] = pair < 0 ? kOut : (uint32_t)(pair * units * 4);
          }
        }
        u32x4 x[XD][CB][2];
        uint32_t xs[CB], xs_next[CB];
        v4f acc[RT][CB];
        auto load_x = [&](int j, int i) {
          [[maybe_unused]] const uint32_t past = j < 4 * ub && j < KB ? 0 : kOut;
#pragma unroll
          for (int b = 0; b < CB; ++b) {
            if constexpr (Y32) {
              const uint8_t* from = yl + at[b] + 128 * (j < 4 * ub ? j : 0);  // K-blocks past H have zeros
              x[i][b][0] = *reinterpret_cast<const u32x4*>(from);
              x[i][b][1] = *reinterpret_cast<const u32x4*>(from + kSecond<F>);
            } else {
              x[i][b][0] = cached16(ry, (at[b] + 128 * j) | past);
              x[i][b][1] = cached16(ry, (at[b] + 128 * j + kSecond<F>) | past);
            }
          }
        };
        auto load_xs = [&](int u) {
#pragma unroll
          for (int b = 0; b < CB; ++b) {
            if constexpr (Y32) xs_next[b] = *reinterpret_cast<const uint32_t*>(yl_sf + s_at[b] + 4 * (u < ub ? u : 0));
            else xs_next[b] = cached4(rs, u < ub && s_at[b] != kOut ? s_at[b] + 4 * u : kOut);
          }
        };
        load_xs(ua);
#pragma unroll
        for (int i = 0; i < XD; ++i) {
          load_x(4 * ua + i, i);
          __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int i = 0; i < RT * CB; ++i) acc[i / CB][i % CB] = v4f{0, 0, 0, 0};
        for (int u = ua; u < ub; ++u) {
#pragma unroll
          for (int b = 0; b < CB; ++b) xs[b] = valid_bytes(xs_next[b], KB - 4 * u);
#pragma unroll
          for (int q = 0; q < RT; ++q) w[q].begin(4 * u, KB);
          // ahead: this expert's next unit, the next expert's first, or nothing (no branch, so that the waits are for as few
          // loads as have to be)
          const bool on = u + 1 < ub;
          const int e_ahead = on ? e : next, j_ahead = on ? 4 * u + 4 : left > 0 ? 0 : KB;
          auto step = [&](auto i_tag) {
            constexpr int I = decltype(i_tag)::value;
#pragma unroll
            for (int k4 = 0; k4 < 4; ++k4) {
              bf16x8 v[RT];
#pragma unroll
              for (int q = 0; q < RT; ++q) v[q] = rows_of<F, I>(w[q], k4);
#pragma unroll
              for (int b = 0; b < CB; ++b) {
                const bf16x8 vx = tokens_of(x[I % XD][b], k4, scale_of(xs[b], I));
#pragma unroll
                for (int q = 0; q < RT; ++q) acc[q][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v[q], vx, acc[q][b], 0, 0, 0);
              }
            }
#pragma unroll
            for (int q = 0; q < RT; ++q) pin(acc[q]);
            load_w(e_ahead, j_ahead + I, I);
            load_x(4 * u + XD + I, I % XD);
            if constexpr (I == 0) load_xs(u + 1);
            __builtin_amdgcn_sched_barrier(0);
          };
          step(std::integral_constant<int, 0>{});
          step(std::integral_constant<int, 1>{});
          step(std::integral_constant<int, 2>{});
          step(std::integral_constant<int, 3>{});
        }
#pragma unroll
        for (int b = 0; b < CB; ++b) {
          const int t = cols[wave].token[16 * b + r];
          if (t >= 0) {
            const float weight = cols[wave].weight[16 * b + r];
#pragma unroll
            for (int q = 0; q < RT; ++q) {
              v4f v = sums[4 * (RT * t + q) + c];
#pragma unroll
              for (int i = 0; i < 4; ++i) v[i] = __builtin_fmaf(weight, acc[q][b][i], v[i]);
              sums[4 * (RT * t + q) + c] = v;
            }
          }
        }
        __builtin_amdgcn_wave_barrier();
      };
      if constexpr (MAXC == 1) {
        run(std::integral_constant<int, 1>{});
      } else if constexpr (MAXC == 2) {
        if (n <= 16) run(std::integral_constant<int, 1>{});
        else run(std::integral_constant<int, 2>{});
      } else {
        if (n <= 16) run(std::integral_constant<int, 1>{});
        else if (n <= 32) run(std::integral_constant<int, 2>{});
        else run(std::integral_constant<int, 4>{});
      }
      ++k;
      ua = 0;
      e = next;
    }
  }
  __syncthreads();
  // thread -> token and four columns
  for (int i = threadIdx.x; i < 4 * RT * m.T; i += NW * 64) {
    const int t = i / (4 * RT), n = n0 + 4 * (i % (4 * RT));
    v4f v = {0, 0, 0, 0};
    if (m.base) {
      const u32x2 b = *reinterpret_cast<const u32x2*>(m.base + t * m.ld_base + n);
      v = v4f{bf16_lo(b[0]), bf16_hi(b[0]), bf16_lo(b[1]), bf16_hi(b[1])};
    }
#pragma unroll
    for (int q = 0; q < NW; ++q) v += reinterpret_cast<const v4f*>(lds)[q * (64 * MAXC * RT) + i];
    *reinterpret_cast<u32x2*>(m.out + t * m.ld_out + n) = u32x2{bf16x2_rne(v[0], v[1]), bf16x2_rne(v[2], v[3])};
  }
}

template <Weights F, bool SMALL, bool Y32, int RT>
hipError_t launch_down(const MoeArgs& a, hipStream_t stream) {
  const MoeDecodeProblem& m = a.m;
  constexpr int NW = 8;
  const int grid = m.K / (16 * RT), routing = 4 * Routing<SMALL>::words(m.topk), sums = NW * 1024 * RT;
  if constexpr (Y32) {
    const int y = m.T * m.topk * (row_bytes(m.H) + (m.H + 511) / 512 * 4);
    moe_down_kernel<F, SMALL, Y32, 1, NW, RT><<<grid, 512, sums + routing + y, stream>>>(a);
  } else {
    if (m.T <= 16) moe_down_kernel<F, SMALL, Y32, 1, NW, RT><<<grid, 512, sums + routing, stream>>>(a);
    else if (m.T <= 32) moe_down_kernel<F, SMALL, Y32, 2, NW, RT><<<grid, 512, 2 * sums + routing, stream>>>(a);
    else moe_down_kernel<F, SMALL, Y32, 4, NW, RT><<<grid, 512, 4 * sums + routing, stream>>>(a);
  }
  return hipGetLastError();
}

template <Weights F>
hipError_t launch(const MoeArgs& a, hipStream_t stream) {
  const MoeDecodeProblem& m = a.m;
  const int pairs = m.T * m.topk, experts = m.E < pairs ? m.E : pairs, KW = parts_of(m);
  const bool small = pairs <= 64;
  // two units of tokens for up to two blocks of 16, or one for up to four
  const int routing = 4 * Routing<false>::words(m.topk), tokens = m.T <= 16 ? 32768 : 65536;
  if (KW == 4) moe_gate_up_kernel<F, true, 4><<<experts * (m.H / 32), 512, 4 * 32768, stream>>>(a);
  else if (KW == 2) moe_gate_up_kernel<F, true, 2><<<experts * (m.H / 64), 512, 2 * 32768, stream>>>(a);
  else if (small) moe_gate_up_kernel<F, true, 1><<<experts * (m.H / 128), 512, tokens, stream>>>(a);
  else moe_gate_up_kernel<F, false, 1><<<experts * (m.H / 128), 512, routing + tokens, stream>>>(a);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  if (KW > 1) return launch_down<F, true, true, 1>(a, stream);
  // 32 output columns a workgroup, for the tokens that both halves then share (16 tokens of 32 experts: 83.5 us with 16
  // columns, 71.4), unless 16 still leave compute units without one
  if (m.K / 16 <= 256) return small ? launch_down<F, true, false, 1>(a, stream) : launch_down<F, false, false, 1>(a, stream);
  return small ? launch_down<F, true, false, 2>(a, stream) : launch_down<F, false, false, 2>(a, stream);
}

}  // namespace

size_t moe_decode_scratch_bytes(int64_t T, int64_t topk, int64_t H) {
  const int64_t pairs = T * topk, quantized = pairs * (H + 4 * ((H + 511) / 512));
  return (size_t)(pairs <= 64 && 4 * pairs * H > quantized ? 4 * pairs * H : quantized);  // up to 64 pairs may be in fp32
}

hipError_t launch_moe_decode(const MoeDecodeProblem& p, Weights kind, void* scratch, hipStream_t stream) {
  MoeArgs a;
  a.m = p;
  a.y = static_cast<uint8_t*>(scratch);
  a.y_sf = reinterpret_cast<uint32_t*>(a.y + (int64_t)p.T * p.topk * p.H);
  a.y32 = static_cast<float*>(scratch);
  switch (kind) {
    case Weights::kPlain: return launch<Weights::kPlain>(a, stream);
    case Weights::kShuffled: return launch<Weights::kShuffled>(a, stream);
    default: return launch<Weights::kW4>(a, stream);
  }
}

}  // namespace fp8bs
