// Combine of the experts' rows, and its backward pass.
//
// Pair (t, j) of token t is row slots[t][j] of expert ids[t][j] in the masked layout
// y [E][M_max][N]; a pair without a row (slot < 0, or past the layout) is left out.
//   out[t] = base[t] + sum_j w[t][j] y[e][s],  in fp32, j ascending, one rounding
//   d_y[e][s] = w[t][j] d_out[t],   d_w[t][j] = <d_out[t], y[e][s]>
// Every row of the layout belongs to one pair at most, so nothing is accumulated in
// memory and the results do not depend on any order.  All of it is bound by memory:
// the rows of the pairs are read (and in the backward pass written) once, as streams.
//
// Measured, 8 pairs of 7168 columns a token: 4096 tokens forward with a base 93.7 us, 581
// MB, 6.2 TB/s (114 us without the streaming policy on the rows and the result); 2048
// tokens backward with codes and weights' gradients 75.5 us, 378 MB, 5.0 TB/s (85 us without
// it; 94 us with one pair at a time and a barrier for each), to bf16 95.5 us, 492 MB, 5.15 TB/s.
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

// One workgroup per token and tile of columns (equal tiles of at most 2048): each thread
// owns eight columns of the output and issues the loads of up to eight pairs before it uses
// the first.
__global__ __launch_bounds__(256) void combine_kernel(const int32_t* __restrict__ ids,
                                                      const int32_t* __restrict__ slots,
                                                      const float* __restrict__ weights, int topk, int64_t E,
                                                      int64_t M_max, int64_t N, const uint16_t* __restrict__ y,
                                                      const uint16_t* __restrict__ base, int64_t ld_base,
                                                      uint16_t* __restrict__ out, int64_t ld_out, unsigned tiles) {
  const int64_t t = blockIdx.x / tiles;
  const uint32_t col = (blockIdx.x % tiles * blockDim.x + threadIdx.x) * 8;
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
          v[j] = load_stream(y + row * N + col);
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
  store_stream(out + t * ld_out + col, pack_bf16x8(acc));
}

// One workgroup per token (and batch of pairs): each thread reads eight columns of d_out
// once, issues the loads of the same columns of up to eight pairs' rows of y, and writes
// those pairs' rows of d_y (or their codes).  The weights' gradients stay in registers
// until the row ends, so a batch costs one barrier.  A row of 7168 in two passes of 448
// threads takes 74 us for 2048 tokens of 8 pairs, as it does in four of 256 or seven of 128;
// in one of 896 it takes 84.
//
// Codes (e4m3, since the masked GEMM that takes the gradient on reads nothing wider): the group's largest |w d| is |w| times its largest |d| (rounding is monotonic), so
// the reduction over the group is made once for all pairs.
template <bool QUANT>
__global__ __launch_bounds__(512) void combine_backward_kernel(
    const int32_t* __restrict__ ids, const int32_t* __restrict__ slots, const float* __restrict__ weights, int topk,
    int64_t E, int64_t M_max, int64_t N, const uint16_t* __restrict__ d_out, int64_t ld_d,
    const uint16_t* __restrict__ y, uint16_t* __restrict__ d_y, uint8_t* __restrict__ q, uint32_t* __restrict__ sf,
    int64_t W, float* __restrict__ d_weights) {
  __shared__ float part[8][kBatch];
  const int64_t t = blockIdx.x;
  const int lane = threadIdx.x & 63;
  const int j0 = blockIdx.y * kBatch;
  int64_t row[kBatch];
  float w[kBatch], dot[kBatch];
#pragma unroll
  for (int j = 0; j < kBatch; ++j) {
    row[j] = -1;
    w[j] = dot[j] = 0.0f;
    if (j0 + j < topk) {  // uniform, as everything that depends on the pair alone
      const int64_t p = t * topk + j0 + j;
      row[j] = pair_row(ids, slots, p, E, M_max);
      w[j] = weights != nullptr ? weights[p] : 1.0f;
    }
  }
  for (uint32_t c0 = 0; c0 < N; c0 += blockDim.x * 8) {
    const uint32_t col = c0 + threadIdx.x * 8;
    const bool valid = col < N;
    u32x4 dv = {0u, 0u, 0u, 0u}, yv[kBatch];
    if (valid) dv = *reinterpret_cast<const u32x4*>(d_out + t * ld_d + col);
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      yv[j] = u32x4{0u, 0u, 0u, 0u};
      if (d_weights != nullptr && row[j] >= 0 && valid) yv[j] = load_stream(y + row[j] * N + col);
    }
    float d[8], amax = 0.0f;
    unpack_bf16x8(dv, d);
    if constexpr (QUANT) amax = __uint_as_float(row16_max_bits(amax8(d)));
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      if (row[j] < 0) continue;
      float f[8];
      unpack_bf16x8(yv[j], f);
#pragma unroll
      for (int i = 0; i < 8; ++i) dot[j] = __builtin_fmaf(d[i], f[i], dot[j]);
      if constexpr (QUANT) {
        const uint32_t byte = scale_byte(__float_as_uint(__builtin_fabsf(w[j]) * amax));
        const uint32_t word = scale_word(valid ? byte : 0u);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = d[i] * w[j];
        if (valid) store_stream(q + row[j] * N + col, codes_at(f, byte));
        if (lane == 0 && valid) {
          const int64_t e_of = ids[t * topk + j0 + j];
          sf[(e_of * W + col / 512) * M_max + (row[j] - e_of * M_max)] = word;
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = d[i] * w[j];
        if (valid) store_stream(d_y + row[j] * N + col, pack_bf16x8(f));
      }
    }
  }
  if (d_weights == nullptr) return;
#pragma unroll
  for (int j = 0; j < kBatch; ++j) {
    const float s = wave_sum(dot[j]);
    if (lane == 0) part[threadIdx.x >> 6][j] = s;
  }
  __syncthreads();
  if (threadIdx.x < kBatch && j0 + (int)threadIdx.x < topk) {
    float s = 0.0f;
    for (unsigned k = 0; k < blockDim.x >> 6; ++k) s += part[k][threadIdx.x];
    d_weights[t * topk + j0 + threadIdx.x] = s;
  }
}

// Threads that take a row of N in `parts` equal parts, eight columns each.
unsigned threads_of(int64_t N, int64_t parts) { return (unsigned)((N / 8 + 64 * parts - 1) / (64 * parts) * 64); }

}  // namespace

hipError_t launch_combine(const CombineProblem& p, const uint16_t* y, const uint16_t* base, int64_t ld_base,
                          uint16_t* out, int64_t ld_out, hipStream_t stream) {
  const unsigned tiles = (unsigned)((p.N / 8 + 255) / 256);
  // 2^24 workgroups of 256 are 2^32 threads, one more than a launch takes: tokens past 2^23
  // workgroups go to launches of their own
  const int64_t most = (1 << 23) / tiles;
  for (int64_t t0 = 0; t0 < p.T; t0 += most) {
    const int64_t T = p.T - t0 < most ? p.T - t0 : most, pair = t0 * p.topk;
    hipLaunchKernelGGL(combine_kernel, dim3((unsigned)(T * tiles)), dim3(threads_of(p.N, tiles)), 0, stream,
                       p.ids + pair, p.slots + pair, p.weights != nullptr ? p.weights + pair : nullptr, p.topk, p.E,
                       p.M_max, p.N, y, base != nullptr ? base + t0 * ld_base : nullptr, ld_base, out + t0 * ld_out,
                       ld_out, tiles);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_combine_backward(const CombineProblem& p, const uint16_t* d_out, int64_t ld_d, const uint16_t* y,
                                   uint16_t* d_y, uint8_t* q, uint32_t* sf, float* d_weights, hipStream_t stream) {
  const int64_t W = (p.N / 128 + 3) / 4;
  const unsigned threads = threads_of(p.N, (p.N / 8 + 511) / 512);
  const dim3 grid((unsigned)p.T, (unsigned)((p.topk + kBatch - 1) / kBatch));
  if (q != nullptr)
    hipLaunchKernelGGL(combine_backward_kernel<true>, grid, dim3(threads), 0, stream, p.ids, p.slots, p.weights,
                       p.topk, p.E, p.M_max, p.N, d_out, ld_d, y, d_y, q, sf, W, d_weights);
  else
    hipLaunchKernelGGL(combine_backward_kernel<false>, grid, dim3(threads), 0, stream, p.ids, p.slots, p.weights,
                       p.topk, p.E, p.M_max, p.N, d_out, ld_d, y, d_y, q, sf, W, d_weights);
  return hipGetLastError();
}

}  // namespace fp8bs
