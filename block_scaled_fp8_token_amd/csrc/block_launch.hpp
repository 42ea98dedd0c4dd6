// Internal launchers of the kernels around the experts' products: routing, combine, the
// norms of the residual stream and the 8-bit activation checkpoint.  The C-ABI layer
// validates every argument before calling these; the launchers only pick grid shapes
// and launch on the caller's stream.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fp8bs {

// Routing.  Expert ids, choice counts and groups are bounded by the limits below.
constexpr int64_t kRouteMaxE = 1024;
constexpr int kRouteMaxTopk = 64;
struct RouteProblem {
  const void* logits;  // [T][ld], fp32 or bf16
  bool f32;
  int64_t ld, T;
  int E, topk;
  bool softmax, renormalize;
  float scale;
};
hipError_t launch_route(const RouteProblem& p, const float* bias, int groups, int topk_groups, int group_top,
                        int32_t* ids, float* weights, hipStream_t stream);
hipError_t launch_route_backward(const RouteProblem& p, const int32_t* ids, const float* d_weights, void* d_logits,
                                 int64_t ld_d, hipStream_t stream);

// Combine: the experts' rows y [E][M_max][N] of token t's pairs, weighted and summed.
struct CombineProblem {
  const int32_t* ids;    // [T][topk]
  const int32_t* slots;  // [T][topk]
  const float* weights;  // [T][topk], or nullptr for ones
  int64_t T, E, M_max, N;
  int topk;
};
hipError_t launch_combine(const CombineProblem& p, const uint16_t* y, const uint16_t* base, int64_t ld_base,
                          uint16_t* out, int64_t ld_out, hipStream_t stream);
hipError_t launch_combine_backward(const CombineProblem& p, const uint16_t* d_out, int64_t ld_d, const uint16_t* y,
                                   uint16_t* d_y, uint8_t* q, uint32_t* sf, float* d_weights, hipStream_t stream);

// Norms of the residual stream.  Null pointers switch the optional parts off.
constexpr int64_t kNormMaxN = 16384;
struct NormProblem {
  bool f32;  // residual stream (x, h, d_h, d_x) in fp32 rather than bf16
  int64_t T, N;
  const uint16_t* y;
  int64_t ldy;
  const uint16_t* w_post;
  const uint16_t* gate;
  int64_t ld_gate;  // 0: one row for every token
  const uint16_t* w_pre;
  float residual_scale, eps, offset;
};
hipError_t launch_norm(const NormProblem& p, const void* x, int64_t ldx, void* h, int64_t ldh, uint16_t* z,
                       int64_t ldz, uint8_t* q, int64_t ldq, uint32_t* sf, int64_t ld_sf, hipStream_t stream);
struct NormGradients {
  const uint16_t* d_z;
  int64_t ld_dz;
  const void* d_h;  // or nullptr
  int64_t ld_dh;
  const void* h;
  int64_t ldh;
  void* d_x;
  int64_t ld_dx;
  uint16_t* d_y;
  int64_t ld_dy;
  float* d_w_pre;
  float* d_w_post;
  void* d_gate;  // fp32 [N] if ld_gate == 0, else bf16 [T][ld_dgate]
  int64_t ld_dgate;
};
// partials: norm_backward_scratch_bytes() of device memory (none: not read).
hipError_t launch_norm_backward(const NormProblem& p, const NormGradients& g, float* partials, hipStream_t stream);
size_t norm_backward_scratch_bytes(const NormProblem& p);

// 8-bit activation checkpoint of the gated activation, over a masked expert batch.
constexpr int64_t kCheckpointMaxE = 1024;
hipError_t launch_silu_checkpoint(const uint16_t* x, const int32_t* masked_m, int64_t E, int64_t M_max, int64_t H,
                                  uint8_t* q, uint32_t* sf, uint8_t* cq, uint32_t* csf, hipStream_t stream);
hipError_t launch_silu_backward(const uint16_t* d_y, const int32_t* masked_m, int64_t E, int64_t M_max, int64_t H,
                                const uint8_t* cq, const uint32_t* csf, uint16_t* d_x, uint8_t* q, uint32_t* sf,
                                hipStream_t stream);

}  // namespace fp8bs
