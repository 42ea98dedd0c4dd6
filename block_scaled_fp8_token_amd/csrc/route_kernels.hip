// Routing of tokens to experts, and its backward pass.
//
// For the logits l of one token over E experts: scores s = sigmoid(l) or softmax(l);
// the experts are ranked by s + bias where there is a bias (which balances their load
// and stays out of the weights) and by l otherwise; with groups of E / G consecutive
// experts only the topk_groups groups of the best group score take part; the topk
// highest ranks are chosen, ties to the lowest index, and weighted by
// scale * s, or scale * s / (sum of the chosen s).
//
// One wavefront routes one token: expert i * 64 + lane sits in register i of its lane,
// so the loads are coalesced at any row stride and the selection needs no LDS.
#include <type_traits>

#include "block_device.hpp"
#include "block_launch.hpp"

namespace fp8bs {

namespace {

constexpr float kNone = -__builtin_inff();  // rank of an expert that cannot be chosen

template <bool F32>
__device__ __forceinline__ float load_logit(const void* p, int64_t i) {
  if constexpr (F32) return static_cast<const float*>(p)[i];
  return __uint_as_float((uint32_t) static_cast<const uint16_t*>(p)[i] << 16);
}

__device__ __forceinline__ float sigmoid(float l) { return 1.0f / (1.0f + expf(-l)); }

// A logit as the operator takes it: NaN and -infinity mean an expert that is not
// available; +infinity is the largest finite value, so that differences stay numbers.
__device__ __forceinline__ float clean_logit(float l) {
  return l > kNone ? __builtin_fminf(l, 3.402823466e38f) : kNone;
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
      const float s = SOFTMAX ? expf(l[i] - top) / sum : sigmoid(l[i]);
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
        if (group_top == 2 && bias == nullptr && v > kNone) v = SOFTMAX ? expf(v - top) : sigmoid(v);
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

// With r_j = s_j / sum of the chosen s and D = sum_j dw_j r_j, the gradient is
//   renormalised: c r_j (dw_j - D) at the chosen experts, for sigmoid scores times
//   1 - s_j = sigmoid(-l_j) (the softmax's own sum cancels: it divides every s alike);
//   else: sigmoid c dw_j s_j (1 - s_j) at the chosen experts, softmax
//   p_e (c dw_e - c sum_j dw_j p_j) at every expert (dw_e = 0 where not chosen).
// Every row is written whole, zeros included.
template <int VPL, bool F32, bool SOFTMAX>
__global__ __launch_bounds__(256) void route_backward_kernel(const void* __restrict__ logits, int64_t ld, int64_t T,
                                                             int E, const int32_t* __restrict__ ids,
                                                             const float* __restrict__ d_weights, int topk,
                                                             int renormalize, float scale, void* __restrict__ d_logits,
                                                             int64_t ld_d) {
  const int lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (t >= T) return;
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
  const bool dense = SOFTMAX && !renormalize;
  float l[VPL], top = 0.0f, sum = 1.0f;
  if (dense) {
    top = kNone;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = i * 64 + lane;
      l[i] = e < E ? clean_logit(load_logit<F32>(logits, t * ld + e)) : kNone;
      top = __builtin_fmaxf(top, l[i]);
    }
    top = wave_max(top);
    if (!(top > kNone)) top = 0.0f;
    sum = 0.0f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      l[i] = expf(l[i] - top);
      sum += l[i];
    }
    sum = wave_sum(sum);
    if (!(sum > 0.0f)) sum = 1.0f;  // no expert at all: every share is 0
  }
  float g = 0.0f;      // of choice `lane`
  float inner = 0.0f;  // dense: sum_j dw_j p_j
  if (dense) {
    g = dw;
    inner = wave_sum(chosen ? dw * (expf(cl - top) / sum) : 0.0f);
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
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = i * 64 + lane;
    float d = 0.0f;
    for (int j = 0; j < topk; ++j) {
      const int32_t ej = __builtin_amdgcn_readlane(id, j);
      const float gj = read_lane(g, j);
      if (ej == e) d += gj;
    }
    if (dense) d = (l[i] / sum) * (d - inner);
    if (e < E) {
      if constexpr (F32)
        static_cast<float*>(d_logits)[t * ld_d + e] = d;
      else
        static_cast<uint16_t*>(d_logits)[t * ld_d + e] = (uint16_t)bf16x2_rne(d, 0.0f);
    }
  }
}

template <int V>
using Int = std::integral_constant<int, V>;
template <bool V>
using Bool = std::integral_constant<bool, V>;

// fn(Int<VPL>, Bool<F32>, Bool<SOFTMAX>) for the registers per lane that E needs.
template <typename Fn>
hipError_t by_shape(const RouteProblem& p, Fn fn) {
  auto types = [&](auto vpl) {
    if (p.f32) return p.softmax ? fn(vpl, Bool<true>{}, Bool<true>{}) : fn(vpl, Bool<true>{}, Bool<false>{});
    return p.softmax ? fn(vpl, Bool<false>{}, Bool<true>{}) : fn(vpl, Bool<false>{}, Bool<false>{});
  };
  if (p.E <= 64) return types(Int<1>{});
  if (p.E <= 128) return types(Int<2>{});
  if (p.E <= 256) return types(Int<4>{});
  if (p.E <= 512) return types(Int<8>{});
  return types(Int<16>{});
}

}  // namespace

hipError_t launch_route(const RouteProblem& p, const float* bias, int groups, int topk_groups, int group_top,
                        int32_t* ids, float* weights, hipStream_t stream) {
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
    hipLaunchKernelGGL((route_backward_kernel<vpl.value, f32.value, softmax.value>), dim3((unsigned)((p.T + 3) / 4)),
                       dim3(256), 0, stream, p.logits, p.ld, p.T, p.E, ids, d_weights, p.topk, (int)p.renormalize,
                       p.scale, d_logits, ld_d);
    return hipGetLastError();
  });
}

}  // namespace fp8bs
