// Combine of the experts' rows, and its backward pass.
//
// Pair (t, j) of token t is row slots[t][j] of expert ids[t][j] in the masked layout
// y [E][M_max][N]; a pair without a row (slot < 0, or past the layout) is left out.
//   out[t] = base[t] + sum_j w[t][j] y[e][s],  in fp32, j ascending, one rounding
//   d_y[e][s] = w[t][j] d_out[t],   d_w[t][j] = <d_out[t], y[e][s]>
// Every row of the layout belongs to one pair at most, so nothing is accumulated in
// memory and the results do not depend on any order.  All of it is bound by memory:
// the rows of the pairs are read (and in the backward pass written) once.
#include "block_device.hpp"
#include "block_launch.hpp"

namespace fp8bs {

namespace {

constexpr int kBatch = 8;  // pairs whose loads are in flight together

// Row of pair (t, j) in the layout, or -1.
__device__ __forceinline__ int64_t pair_row(const int32_t* __restrict__ ids, const int32_t* __restrict__ slots,
                                            int64_t p, int64_t E, int64_t M_max) {
  const int32_t e = ids[p], s = slots[p];
  return (e >= 0 && e < E && s >= 0 && s < M_max) ? (int64_t)e * M_max + s : -1;
}

// One workgroup per token and 2048 columns: each thread owns eight columns of the
// output and issues the loads of up to eight pairs before it uses the first.
__global__ __launch_bounds__(256) void combine_kernel(const int32_t* __restrict__ ids,
                                                      const int32_t* __restrict__ slots,
                                                      const float* __restrict__ weights, int topk, int64_t E,
                                                      int64_t M_max, int64_t N, const uint16_t* __restrict__ y,
                                                      const uint16_t* __restrict__ base, int64_t ld_base,
                                                      uint16_t* __restrict__ out, int64_t ld_out, int64_t tiles) {
  const int64_t t = (int64_t)blockIdx.x / tiles;
  const int64_t col = ((int64_t)blockIdx.x - t * tiles) * 2048 + threadIdx.x * 8;
  if (col >= N) return;
  float acc[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = 0.0f;
  if (base != nullptr) unpack_bf16x8(*reinterpret_cast<const u32x4*>(base + t * ld_base + col), acc);
  for (int j0 = 0; j0 < topk; j0 += kBatch) {
    u32x4 v[kBatch];
    float w[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      v[j] = u32x4{0u, 0u, 0u, 0u};
      w[j] = 0.0f;
      if (j0 + j < topk) {  // uniform, as everything that depends on the pair alone
        const int64_t p = t * topk + j0 + j, row = pair_row(ids, slots, p, E, M_max);
        if (row >= 0) {
          w[j] = weights != nullptr ? weights[p] : 1.0f;
          v[j] = *reinterpret_cast<const u32x4*>(y + row * N + col);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      float f[8];
      unpack_bf16x8(v[j], f);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] = __builtin_fmaf(w[j], f[i], acc[i]);
    }
  }
  *reinterpret_cast<u32x4*>(out + t * ld_out + col) = pack_bf16x8(acc);
}

// One workgroup per token: d_out's row is read once and kept while the pairs are
// walked; each pair's row of y is read for its weight's gradient and its row of d_y (or
// of the codes) written.  Threads beyond N / 8 take part in the reductions only.
template <bool QUANT>
__global__ __launch_bounds__(256) void combine_backward_kernel(
    const int32_t* __restrict__ ids, const int32_t* __restrict__ slots, const float* __restrict__ weights, int topk,
    int64_t E, int64_t M_max, int64_t N, const uint16_t* __restrict__ d_out, int64_t ld_d,
    const uint16_t* __restrict__ y, uint16_t* __restrict__ d_y, uint8_t* __restrict__ q, uint32_t* __restrict__ sf,
    int64_t W, float* __restrict__ d_weights) {
  __shared__ float part[2][16];
  const int64_t t = blockIdx.x;
  const int lane = threadIdx.x & 63;
  int turn = 0;  // of the two halves of `part`: consecutive sums use different ones
  for (int j = 0; j < topk; ++j) {
    const int64_t p = t * topk + j, row = pair_row(ids, slots, p, E, M_max);
    if (row < 0) {  // uniform
      if (d_weights != nullptr && threadIdx.x == 0) d_weights[p] = 0.0f;
      continue;
    }
    const float w = weights != nullptr ? weights[p] : 1.0f;
    const int64_t e = row / M_max, s = row - e * M_max;
    float dot = 0.0f;
    for (int64_t c0 = 0; c0 < N; c0 += 2048) {
      const int64_t col = c0 + threadIdx.x * 8;
      const bool valid = col < N;
      float f[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
      if (valid) {
        unpack_bf16x8(*reinterpret_cast<const u32x4*>(d_out + t * ld_d + col), f);
        if (d_weights != nullptr) {
          float v[8];
          unpack_bf16x8(*reinterpret_cast<const u32x4*>(y + row * N + col), v);
#pragma unroll
          for (int i = 0; i < 8; ++i) dot = __builtin_fmaf(f[i], v[i], dot);
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] *= w;
      if constexpr (QUANT) {
        const int ex = group_exponent(f);
        const uint32_t word = scale_word(valid ? (uint32_t)(ex + 127) : 0u);
        if (valid) *reinterpret_cast<uint64_t*>(q + row * N + col) = codes_at(f, ex);
        if (lane == 0 && valid) sf[(e * W + col / 512) * M_max + s] = word;
      } else {
        if (valid) *reinterpret_cast<u32x4*>(d_y + row * N + col) = pack_bf16x8(f);
      }
    }
    if (d_weights != nullptr) {
      turn ^= 1;
      dot = block_sum(dot, part[turn], 4);
      if (threadIdx.x == 0) d_weights[p] = dot;
    }
  }
}

}  // namespace

hipError_t launch_combine(const CombineProblem& p, const uint16_t* y, const uint16_t* base, int64_t ld_base,
                          uint16_t* out, int64_t ld_out, hipStream_t stream) {
  const int64_t tiles = (p.N + 2047) / 2048;
  hipLaunchKernelGGL(combine_kernel, dim3((unsigned)(p.T * tiles)), dim3(256), 0, stream, p.ids, p.slots, p.weights,
                     p.topk, p.E, p.M_max, p.N, y, base, ld_base, out, ld_out, tiles);
  return hipGetLastError();
}

hipError_t launch_combine_backward(const CombineProblem& p, const uint16_t* d_out, int64_t ld_d, const uint16_t* y,
                                   uint16_t* d_y, uint8_t* q, uint32_t* sf, float* d_weights, hipStream_t stream) {
  const int64_t W = (p.N / 128 + 3) / 4;
  if (q != nullptr)
    hipLaunchKernelGGL(combine_backward_kernel<true>, dim3((unsigned)p.T), dim3(256), 0, stream, p.ids, p.slots,
                       p.weights, p.topk, p.E, p.M_max, p.N, d_out, ld_d, y, d_y, q, sf, W, d_weights);
  else
    hipLaunchKernelGGL(combine_backward_kernel<false>, dim3((unsigned)p.T), dim3(256), 0, stream, p.ids, p.slots,
                       p.weights, p.topk, p.E, p.M_max, p.N, d_out, ld_d, y, d_y, q, sf, W, d_weights);
  return hipGetLastError();
}

}  // namespace fp8bs
