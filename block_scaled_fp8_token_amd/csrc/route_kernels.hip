// Routing of tokens to experts, and its backward pass.
//
// For the logits l of one token over E experts: scores s = sigmoid(l) or softmax(l);
// the experts are ranked by s + bias where there is a bias (which balances their load
// and stays out of the weights) and by l otherwise; with groups of E / G consecutive
// experts only the topk_groups groups of the best group score take part; the topk
// highest ranks are chosen, ties to the lowest index, and weighted by
// scale * s, or scale * s / (sum of the chosen s).
//
// Two kernels.  route_row_kernel, for up to eight of up to 512 experts: sixteen lanes route
// one token, each lane sorts the ranks it holds, and four merges leave the token's eight
// best in every lane.  route_kernel, for everything else: one wavefront routes one token
// and takes one maximum per choice.
//
// Bound by vector instructions (about 1350 in a wavefront for four tokens; the memory would
// take 2 us below) and, for few tokens, by the length of their chain.  Measured in a graph,
// bf16 logits, 16384 tokens, 256 experts: 8 chosen in 4 of 8 groups by biased sigmoid scores
// 11.3 us, 8 by softmax 7.1 us; 9 chosen, which the second kernel takes, 18 us, in groups 38 us
// (8 in groups 36).  512 experts: 8 chosen 15.9 and 10.0 us, 9 chosen 27 us, 10 chosen 32 us.
// One token of 256: 5.6 and 3.6 us.  Backward, softmax not renormalised: 11.1 us, 14.9 us with
// a memory instruction for every 64 logits and a comparison of every choice with every expert;
// with inputs past the caches 13.0 us, and 10.5 us for the forms whose gradients stay at the
// chosen experts.
#include <type_traits>

#include "block_device.hpp"
#include "block_launch.hpp"

namespace fp8bs {

namespace {

constexpr float kNone = -__builtin_inff();  // rank of an expert that cannot be chosen
constexpr float kMost = 3.402823466e38f;    // the largest finite fp32

template <bool F32>
__device__ __forceinline__ float load_logit(const void* p, int64_t i) {
  if constexpr (F32) return static_cast<const float*>(p)[i];
  return __uint_as_float((uint32_t) static_cast<const uint16_t*>(p)[i] << 16);
}

__device__ __forceinline__ float sigmoid(float l) { return 1.0f / (1.0f + expf(-l)); }

// The same bits of every logit above -87 (lower ones score as -87: no two scores under 2e-38
// rank apart), in seven instructions less: one Newton step on a reciprocal of 1 ulp with two
// fused multiply-adds rounds 1 / d correctly (Markstein, 1990) for d in [1, 2^126), which a
// comparison with the division over all of those d confirmed.
__device__ __forceinline__ float rank_sigmoid(float l) {
  const float d = 1.0f + expf(-__builtin_fmaxf(l, -87.0f));
  const float r = __builtin_amdgcn_rcpf(d);
  return __builtin_fmaf(__builtin_fmaf(-d, r, 1.0f), r, r);
}

// A logit as the operator takes it: NaN and -infinity mean an expert that is not
// available; +infinity is the largest finite value, so that differences stay numbers.
__device__ __forceinline__ float clean_logit(float l) {
  return l > kNone ? __builtin_fminf(l, kMost) : kNone;
}

// (a, b) = the two largest of (a, b) and (c, d), a >= b.
__device__ __forceinline__ void merge_two(float& a, float& b, float c, float d) {
  const float lo = __builtin_fminf(a, c);
  a = __builtin_fmaxf(a, c);
  b = __builtin_fmaxf(lo, __builtin_fmaxf(b, d));
}
template <int CTRL>
__device__ __forceinline__ void merge_two_dpp(float& a, float& b) {
  merge_two(a, b, dpp_f<CTRL>(a), dpp_f<CTRL>(b));
}

// Score of one group from its two best values: the best, or the sum of both (one that
// does not exist adds nothing).
__device__ __forceinline__ float group_score(float a, float b, int group_top) {
  return group_top == 2 && b > kNone ? a + b : a;
}

// ---- sixteen lanes per token ----
//
// A rank and its expert are one fp64 number: the fp32 rank is exact in its upper bits and
// the low ten bits of its mantissa hold the expert so that of equal ranks the lower expert
// is the larger number.  All numbers differ, a comparison of two is one instruction each for
// the larger and the smaller, and ties need no case of their own.
constexpr int kList = 8;             // ranks a lane keeps, sorted
constexpr int kNoneHi = 0xC8078000;  // upper half of about -1e39: below every fp32

// Experts of a token over the sixteen lanes of a row: a group (all experts where there are
// no groups) has `lanes` of them, each takes `per_lane` consecutive experts of its group.
struct RowLayout {
  int lanes, per_lane;
  int groups, size;
  bool wide, wide_bias;  // a lane's logits, its biases, are whole aligned 16-byte words
};

__device__ __forceinline__ double rank_of(float rank, int expert) {
  // + 0: -0 ranks as 0; an infinite rank ranks as the largest number
  const uint64_t u = __builtin_bit_cast(uint64_t, (double)__builtin_fminf(rank + 0.0f, kMost));
  const int hi = (int)(u >> 32);
  const uint32_t code = (uint32_t)((expert ^ 1023) ^ ((hi >> 31) & 1023));
  const uint32_t top = (uint32_t)(rank > kNone ? hi : kNoneHi);
  return __builtin_bit_cast(double, ((uint64_t)top << 32) | (uint32_t)u | code);
}
__device__ __forceinline__ double without_rank(double r) {
  return __builtin_bit_cast(double, ((uint64_t)(uint32_t)kNoneHi << 32) | (uint32_t)__builtin_bit_cast(uint64_t, r));
}
// The expert of a rank, or -1.
__device__ __forceinline__ int expert_of(double r) {
  const uint64_t u = __builtin_bit_cast(uint64_t, r);
  const int hi = (int)(u >> 32);
  return hi == kNoneHi ? -1 : (int)(((uint32_t)u & 1023) ^ 1023 ^ ((hi >> 31) & 1023));
}
template <int CTRL>
__device__ __forceinline__ double dpp_d(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)u, CTRL, 0xf, 0xf, true);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_mov_dpp((int)(u >> 32), CTRL, 0xf, 0xf, true);
  return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

__device__ __forceinline__ void order(double& a, double& b) {  // a >= b
  const double lo = __builtin_fmin(a, b);
  a = __builtin_fmax(a, b);
  b = lo;
}
// Descending order of eight: Batcher's odd-even merge sort, 19 comparators.
__device__ __forceinline__ void sort8(double* v) {
  order(v[0], v[1]); order(v[2], v[3]); order(v[4], v[5]); order(v[6], v[7]);
  order(v[0], v[2]); order(v[1], v[3]); order(v[4], v[6]); order(v[5], v[7]);
  order(v[1], v[2]); order(v[5], v[6]);
  order(v[0], v[4]); order(v[1], v[5]); order(v[2], v[6]); order(v[3], v[7]);
  order(v[2], v[4]); order(v[3], v[5]);
  order(v[1], v[2]); order(v[3], v[4]); order(v[5], v[6]);
}
// The eight largest of two descending lists, descending: the larger of opposite ends are
// they, first falling, then rising, which three rounds of comparators straighten.
__device__ __forceinline__ void merge8(double* v, const double* w) {
#pragma unroll
  for (int i = 0; i < kList; ++i) v[i] = __builtin_fmax(v[i], w[kList - 1 - i]);
#pragma unroll
  for (int d = 4; d > 0; d >>= 1)
#pragma unroll
    for (int i = 0; i < kList; ++i)
      if (!(i & d)) order(v[i], v[i + d]);
}
template <int CTRL>
__device__ __forceinline__ void merge_lanes(double* v) {
  double w[kList];
#pragma unroll
  for (int i = 0; i < kList; ++i) w[i] = dpp_d<CTRL>(v[i]);
  merge8(v, w);
}
// Groups (one number per lane, the same in all lanes of a group) ahead of the lane's own.
template <int R>
__device__ __forceinline__ int groups_ahead(double mine, int lanes) {
  constexpr int kRowRor = 0x120;
  int n = 0;
  if (R % lanes == 0) n = dpp_d<kRowRor + R>(mine) > mine ? 1 : 0;  // uniform condition
  if constexpr (R < 15) n += groups_ahead<R + 1>(mine, lanes);
  return n;
}

// V values of a lane from expert `first` of a row on, `n` of them there (kNone past them).
template <int V, bool F32>
__device__ __forceinline__ void load_lane(const void* values, int64_t row, int first, int n, bool wide, float* l) {
#pragma unroll
  for (int i = 0; i < V; ++i) l[i] = kNone;
  if (wide) {  // uniform
    constexpr int M = F32 ? 4 : 8;
#pragma unroll
    for (int i = 0; i < V; i += M)
      if (i < n) {
        const u32x4 v = *reinterpret_cast<const u32x4*>(static_cast<const char*>(values) +
                                                        (row + first + i) * (F32 ? 4 : 2));
        if constexpr (F32) {
#pragma unroll
          for (int k = 0; k < 4; ++k) l[i + k] = __uint_as_float(v[k]);
        } else {
          unpack_bf16x8(v, l + i);
        }
      }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < n) l[i] = load_logit<F32>(values, row + first + i);
  }
}

template <int V, bool F32, bool SOFTMAX>
__global__ __launch_bounds__(64) void route_row_kernel(const void* __restrict__ logits, int64_t ld, int64_t T,
                                                       RowLayout at, const float* __restrict__ bias, int topk_groups,
                                                       int group_top, int topk, int renormalize, float scale,
                                                       int32_t* __restrict__ ids, float* __restrict__ weights) {
  const int sub = threadIdx.x & 15;
  const int64_t token = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 4);
  const int64_t t = token < T ? token : T - 1;  // rows past the end work on the last one and store nothing
  const int group = sub / at.lanes, part = sub - group * at.lanes;
  const int first = group * at.size + part * at.per_lane;
  int n = at.size - part * at.per_lane;  // experts of this lane
  n = group < at.groups ? (n < at.per_lane ? n : at.per_lane) : 0;
  float l[V];
  load_lane<V, F32>(logits, t * ld, first, n, at.wide, l);
#pragma unroll
  for (int i = 0; i < V; ++i) l[i] = clean_logit(l[i]);
  const bool two = at.groups > 1 && group_top == 2;
  float top = 0.0f, sum = 1.0f;
  if constexpr (SOFTMAX) {
    if (bias != nullptr || two || !renormalize) {  // the weights of a renormalised choice need no other
      top = kNone;
#pragma unroll
      for (int i = 0; i < V; ++i) top = __builtin_fmaxf(top, l[i]);
      top = row16_max(top);
      if (!(top > kNone)) top = 0.0f;  // no expert at all
      sum = 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) sum += expf(l[i] - top);
      sum = row16_sum(sum);
    }
  }
  float key[V];
#pragma unroll
  for (int i = 0; i < V; ++i) key[i] = l[i];
  if (bias != nullptr) {
    float b[V];
    load_lane<V, true>(bias, 0, first, n, at.wide_bias, b);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float s = SOFTMAX ? expf(l[i] - top) / sum : rank_sigmoid(l[i]);
      const float c = s + (l[i] > kNone ? b[i] : kNone);
      key[i] = c > kNone ? c : kNone;
    }
  }
  bool kept = true;
  if (at.groups > 1) {
    float a = kNone, b = kNone;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float v = key[i];
      // without a bias the ranks are logits: a sum of two wants their scores (the softmax's
      // common denominator changes no order)
      if (two && bias == nullptr && v > kNone) v = SOFTMAX ? expf(v - top) : rank_sigmoid(v);
      b = __builtin_amdgcn_fmed3f(a, b, v);  // a >= b: the second largest of the three
      a = __builtin_fmaxf(a, v);
    }
    if (at.lanes > 1) merge_two_dpp<kXor1>(a, b);
    if (at.lanes > 2) merge_two_dpp<kXor2>(a, b);
    if (at.lanes > 4) merge_two_dpp<kHalfMirror>(a, b);
    const double mine = rank_of(group_score(a, b, group_top), group);
    kept = groups_ahead<1>(mine, at.lanes) < topk_groups;
  }
  double v[V];
#pragma unroll
  for (int i = 0; i < V; ++i) v[i] = rank_of(key[i], first + i);
  sort8(v);
#pragma unroll
  for (int i = kList; i < V; i += kList) {
    sort8(v + i);
    merge8(v, v + i);
  }
  if (at.groups > 1) {
#pragma unroll
    for (int i = 0; i < kList; ++i) v[i] = kept ? v[i] : without_rank(v[i]);
  }
  merge_lanes<kXor1>(v);
  merge_lanes<kXor2>(v);
  merge_lanes<kHalfMirror>(v);
  merge_lanes<kMirror>(v);
  double mine = v[0];  // of choice `sub`
#pragma unroll
  for (int i = 1; i < kList; ++i) mine = sub == i ? v[i] : mine;
  const int32_t id = sub < topk ? expert_of(mine) : -1;
  const bool chosen = id >= 0;
  const float cl = chosen ? clean_logit(load_logit<F32>(logits, t * ld + id)) : kNone;
  float s;
  if constexpr (SOFTMAX) {
    if (renormalize) top = row16_max(cl);
    s = chosen ? expf(cl - top) : 0.0f;
    if (!renormalize) s = chosen ? s / sum : 0.0f;
  } else {
    s = chosen ? sigmoid(cl) : 0.0f;
  }
  if (renormalize) {
    const float z = row16_sum(s);
    s = z > 0.0f ? s / z : 0.0f;
  }
  if (sub < topk && token < T) {
    ids[t * topk + sub] = id;
    weights[t * topk + sub] = s * scale;
  }
}

// ---- one wavefront per token: expert i * 64 + lane sits in register i of its lane ----
template <int VPL, bool F32, bool SOFTMAX>
__global__ __launch_bounds__(256) void route_kernel(const void* __restrict__ logits, int64_t ld, int64_t T, int E,
                                                    const float* __restrict__ bias, int groups, int group_size,
                                                    int topk_groups, int group_top, int topk, int renormalize,
                                                    float scale, int32_t* __restrict__ ids,
                                                    float* __restrict__ weights) {
  const int lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (t >= T) return;
  float l[VPL], key[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = i * 64 + lane;
    l[i] = e < E ? clean_logit(load_logit<F32>(logits, t * ld + e)) : kNone;
  }
  // softmax: the largest logit and the sum of exponentials
  float top = 0.0f, sum = 1.0f;
  if constexpr (SOFTMAX) {
    top = kNone;
#pragma unroll
    for (int i = 0; i < VPL; ++i) top = __builtin_fmaxf(top, l[i]);
    top = wave_max(top);
    if (!(top > kNone)) top = 0.0f;  // no expert at all
    sum = 0.0f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) sum += expf(l[i] - top);
    sum = wave_sum(sum);
  }
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = i * 64 + lane;
    key[i] = l[i];
    if (bias != nullptr && e < E && l[i] > kNone) {
      const float s = SOFTMAX ? expf(l[i] - top) / sum : rank_sigmoid(l[i]);
      const float c = s + bias[e];
      key[i] = c > kNone ? c : kNone;
    }
  }
  if (groups > 1) {
    float mine = kNone;  // lane g: the score of group g
    int of[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) of[i] = (i * 64 + lane) / group_size;
    for (int g = 0; g < groups; ++g) {
      float a = kNone, b = kNone;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        float v = of[i] == g ? key[i] : kNone;
        // without a bias the ranks are logits: a sum of two wants their scores (the
        // softmax's common denominator changes no order)
        if (group_top == 2 && bias == nullptr && v > kNone) v = SOFTMAX ? expf(v - top) : rank_sigmoid(v);
        merge_two(a, b, v, kNone);
      }
      merge_two_dpp<kXor1>(a, b);
      merge_two_dpp<kXor2>(a, b);
      merge_two_dpp<kHalfMirror>(a, b);
      merge_two_dpp<kMirror>(a, b);
      float x = read_lane(a, 0), y = read_lane(b, 0);
      merge_two(x, y, read_lane(a, 16), read_lane(b, 16));
      merge_two(x, y, read_lane(a, 32), read_lane(b, 32));
      merge_two(x, y, read_lane(a, 48), read_lane(b, 48));
      if (lane == g) mine = group_score(x, y, group_top);
    }
    int ahead = 0;
    for (int g = 0; g < groups; ++g) {
      const float s = read_lane(mine, g);
      ahead += (s > mine || (s == mine && g < lane)) ? 1 : 0;
    }
    const uint64_t kept = __ballot(lane < groups && ahead < topk_groups);
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (!((kept >> (of[i] & 63)) & 1)) key[i] = kNone;
  }
  // topk rounds: the best rank of the wavefront, the lowest expert that has it
  int32_t my_id = -1;
  float my_l = kNone;
  for (int j = 0; j < topk; ++j) {
    float best = key[0], best_l = l[0];
    int at = 0;
#pragma unroll
    for (int i = 1; i < VPL; ++i) {
      const bool more = key[i] > best;
      best = more ? key[i] : best;
      best_l = more ? l[i] : best_l;
      at = more ? i : at;
    }
    const float m = wave_max(best);
    if (!(m > kNone)) break;  // uniform
    uint64_t has = __ballot(best == m);
    int lowest = at * 64 + lane, from = __builtin_ctzll(has);
    int e = __builtin_amdgcn_readlane(lowest, from);
    has &= has - 1;
    while (has) {  // more than one lane holds the best rank (rare; uniform)
      const int other = __builtin_ctzll(has);
      const int oe = __builtin_amdgcn_readlane(lowest, other);
      if (oe < e) {
        e = oe;
        from = other;
      }
      has &= has - 1;
    }
    const float el = read_lane(best_l, from);
    if (lane == j) {
      my_id = e;
      my_l = el;
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (lowest == e && i == at) key[i] = kNone;
  }
  // weights: the softmax over the chosen logits needs no other sum, and cannot underflow
  const bool chosen = my_id >= 0;
  float s;
  if constexpr (SOFTMAX) {
    if (renormalize) top = wave_max(my_l);
    s = chosen ? expf(my_l - top) : 0.0f;
    if (!renormalize && chosen) s = s / sum;
  } else {
    s = chosen ? sigmoid(my_l) : 0.0f;
  }
  if (renormalize) {
    const float z = wave_sum(s);
    s = z > 0.0f ? s / z : 0.0f;
  }
  if (lane < topk) {
    ids[t * topk + lane] = my_id;
    weights[t * topk + lane] = s * scale;
  }
}

// The VPL logits of a lane, kept or written as one piece where they are (WIDE: experts
// lane * VPL .. of a row, aligned to all of them or to 16 bytes), else one by one (experts
// lane, lane + 64, ..).
template <int VPL, bool F32, bool WIDE>
struct LaneRow {
  static constexpr int kBytes = VPL * (F32 ? 4 : 2);
  typedef std::conditional_t<F32, float, uint16_t> T;
  struct alignas(kBytes < 16 ? kBytes : 16) Piece {
    T v[VPL];
  };
  static __device__ __forceinline__ int expert(int lane, int i) { return WIDE ? lane * VPL + i : i * 64 + lane; }
  static __device__ __forceinline__ void load(const void* row, int lane, int E, float* l) {
    const T* from = static_cast<const T*>(row);
    Piece p = {};
    if constexpr (WIDE) {
      if (lane * VPL < E) p = *reinterpret_cast<const Piece*>(from + lane * VPL);
    } else {
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (expert(lane, i) < E) p.v[i] = from[expert(lane, i)];
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      float v;
      if constexpr (F32) v = p.v[i];
      else v = __uint_as_float((uint32_t)p.v[i] << 16);
      l[i] = expert(lane, i) < E ? clean_logit(v) : kNone;
    }
  }
  static __device__ __forceinline__ void store(void* row, int lane, int E, const float* d) {
    T* to = static_cast<T*>(row);
    Piece p;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      if constexpr (F32) p.v[i] = d[i];
      else p.v[i] = (uint16_t)bf16x2_rne(d[i], 0.0f);
    }
    if constexpr (WIDE) {
      if (lane * VPL < E) *reinterpret_cast<Piece*>(to + lane * VPL) = p;
    } else {
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (expert(lane, i) < E) to[expert(lane, i)] = p.v[i];
    }
  }
};

// With r_j = s_j / sum of the chosen s and D = sum_j dw_j r_j, the gradient is
//   renormalised: c r_j (dw_j - D) at the chosen experts, for sigmoid scores times
//   1 - s_j = sigmoid(-l_j) (the softmax's own sum cancels: it divides every s alike);
//   else: sigmoid c dw_j s_j (1 - s_j) at the chosen experts, softmax
//   p_e (c dw_e - c sum_j dw_j p_j) at every expert (dw_e = 0 where not chosen).
// Every row is written whole, zeros included.  The value of choice j is written into the
// register and lane of its expert, both of which the whole wavefront knows.
template <int VPL, bool F32, bool SOFTMAX, bool WIDE>
__global__ __launch_bounds__(256) void route_backward_kernel(const void* __restrict__ logits, int64_t ld, int64_t T,
                                                             int E, const int32_t* __restrict__ ids,
                                                             const float* __restrict__ d_weights, int topk,
                                                             int renormalize, float scale, void* __restrict__ d_logits,
                                                             int64_t ld_d) {
  using Row = LaneRow<VPL, F32, WIDE>;
  constexpr int kBytes = F32 ? 4 : 2;
  const int lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (t >= T) return;
  const bool dense = SOFTMAX && !renormalize;
  float l[VPL];
  if (dense) Row::load(static_cast<const char*>(logits) + t * ld * kBytes, lane, E, l);
  // the chosen experts: lane j holds choice j
  int32_t id = -1;
  float dw = 0.0f, cl = kNone;
  if (lane < topk) {
    const int32_t e = ids[t * topk + lane];
    if (e >= 0 && e < E) {
      cl = clean_logit(load_logit<F32>(logits, t * ld + e));
      if (cl > kNone) {
        id = e;
        dw = d_weights[t * topk + lane] * scale;
      }
    }
  }
  const bool chosen = id >= 0;
  float g = 0.0f;      // of choice `lane`
  float inner = 0.0f;  // dense: sum_j dw_j p_j
  if (dense) {
    float top = kNone;
#pragma unroll
    for (int i = 0; i < VPL; ++i) top = __builtin_fmaxf(top, l[i]);
    top = wave_max(top);
    if (!(top > kNone)) top = 0.0f;
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      l[i] = expf(l[i] - top);
      sum += l[i];
    }
    sum = wave_sum(sum);
    const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;  // no expert at all: every share is 0
#pragma unroll
    for (int i = 0; i < VPL; ++i) l[i] *= inv;
    g = dw;
    inner = wave_sum(chosen ? dw * (expf(cl - top) * inv) : 0.0f);
  } else {
    float s;
    if constexpr (SOFTMAX) {
      const float m = wave_max(cl);
      s = chosen ? expf(cl - m) : 0.0f;
    } else {
      s = chosen ? sigmoid(cl) : 0.0f;
    }
    if (renormalize) {
      const float z = wave_sum(s);
      const float r = z > 0.0f ? s / z : 0.0f;
      g = r * (dw - wave_sum(chosen ? dw * r : 0.0f));
    } else {
      g = dw * s;
    }
    if constexpr (!SOFTMAX) g = chosen ? g * sigmoid(-cl) : 0.0f;
  }
  float d[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) d[i] = 0.0f;
  for (int j = 0; j < topk; ++j) {
    const int e = __builtin_amdgcn_readlane(id, j);
    if (e < 0) continue;  // uniform, as all of this
    const float gj = read_lane(g, j);
    const int at = WIDE ? e % VPL : e >> 6, owner = WIDE ? e / VPL : e & 63;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (at == i) d[i] = lane == owner ? gj : d[i];
  }
  if (dense) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) d[i] = l[i] * (d[i] - inner);
  }
  Row::store(static_cast<char*>(d_logits) + t * ld_d * kBytes, lane, E, d);
}

template <int V>
using Int = std::integral_constant<int, V>;
template <bool V>
using Bool = std::integral_constant<bool, V>;

// fn(Bool<F32>, Bool<SOFTMAX>)
template <typename Fn>
hipError_t by_types(const RouteProblem& p, Fn fn) {
  if (p.f32) return p.softmax ? fn(Bool<true>{}, Bool<true>{}) : fn(Bool<true>{}, Bool<false>{});
  return p.softmax ? fn(Bool<false>{}, Bool<true>{}) : fn(Bool<false>{}, Bool<false>{});
}
// fn(Int<VPL>, Bool<F32>, Bool<SOFTMAX>) for the registers per lane that E needs.
template <typename Fn>
hipError_t by_shape(const RouteProblem& p, Fn fn) {
  auto types = [&](auto vpl) { return by_types(p, [&](auto f32, auto softmax) { return fn(vpl, f32, softmax); }); };
  if (p.E <= 64) return types(Int<1>{});
  if (p.E <= 128) return types(Int<2>{});
  if (p.E <= 256) return types(Int<4>{});
  if (p.E <= 512) return types(Int<8>{});
  return types(Int<16>{});
}

}  // namespace

hipError_t launch_route(const RouteProblem& p, const float* bias, int groups, int topk_groups, int group_top,
                        int32_t* ids, float* weights, hipStream_t stream) {
  // sixteen lanes per token: a group's lanes (a power of two) by groups, up to 32 experts each
  if (p.topk <= kList && groups <= 16) {
    RowLayout at;
    at.lanes = 16;
    while (16 / at.lanes < groups) at.lanes /= 2;
    at.groups = groups;
    at.size = p.E / groups;
    at.per_lane = (at.size + at.lanes - 1) / at.lanes;
    const int bytes = p.f32 ? 4 : 2;
    at.wide = at.size % at.lanes == 0 && at.per_lane * bytes % 16 == 0 && p.ld * bytes % 16 == 0 &&
              reinterpret_cast<uintptr_t>(p.logits) % 16 == 0;
    at.wide_bias = at.size % at.lanes == 0 && at.per_lane % 4 == 0 && reinterpret_cast<uintptr_t>(bias) % 16 == 0;
    auto by_lane = [&](auto v) {
      return by_types(p, [&](auto f32, auto softmax) {
        hipLaunchKernelGGL((route_row_kernel<v.value, f32.value, softmax.value>), dim3((unsigned)((p.T + 3) / 4)),
                           dim3(64), 0, stream, p.logits, p.ld, p.T, at, bias, topk_groups, group_top, p.topk,
                           (int)p.renormalize, p.scale, ids, weights);
        return hipGetLastError();
      });
    };
    if (at.per_lane <= kList) return by_lane(Int<kList>{});
    if (at.per_lane <= 2 * kList) return by_lane(Int<2 * kList>{});
    if (at.per_lane <= 4 * kList) return by_lane(Int<4 * kList>{});
  }
  return by_shape(p, [&](auto vpl, auto f32, auto softmax) {
    hipLaunchKernelGGL((route_kernel<vpl.value, f32.value, softmax.value>), dim3((unsigned)((p.T + 3) / 4)), dim3(256),
                       0, stream, p.logits, p.ld, p.T, p.E, bias, groups, p.E / groups, topk_groups, group_top, p.topk,
                       (int)p.renormalize, p.scale, ids, weights);
    return hipGetLastError();
  });
}

hipError_t launch_route_backward(const RouteProblem& p, const int32_t* ids, const float* d_weights, void* d_logits,
                                 int64_t ld_d, hipStream_t stream) {
  return by_shape(p, [&](auto vpl, auto f32, auto softmax) {
    const uintptr_t piece = vpl.value * (p.f32 ? 4 : 2), align = piece < 16 ? piece : 16;
    const int64_t row = p.f32 ? 4 : 2;
    const bool wide = p.E % vpl.value == 0 && p.ld * row % align == 0 && ld_d * row % align == 0 &&
                      reinterpret_cast<uintptr_t>(p.logits) % align == 0 &&
                      reinterpret_cast<uintptr_t>(d_logits) % align == 0;
    auto launch = [&](auto w) {
      hipLaunchKernelGGL((route_backward_kernel<vpl.value, f32.value, softmax.value, w.value>),
                         dim3((unsigned)((p.T + 3) / 4)), dim3(256), 0, stream, p.logits, p.ld, p.T, p.E, ids,
                         d_weights, p.topk, (int)p.renormalize, p.scale, d_logits, ld_d);
      return hipGetLastError();
    };
    return wide ? launch(Bool<true>{}) : launch(Bool<false>{});
  });
}

}  // namespace fp8bs
