// Norms before and after a block, fused with the block's gate and the scale of the
// residual stream, and their backward pass.  For every token
//   b = y / sqrt(mean(y^2) + eps) * (w_post + offset)      (b = y without w_post)
//   h = residual_scale * x + gate * b                       the residual stream
//   z = h / sqrt(mean(h^2) + eps) * (w_pre + offset)        input of the next block
// in fp32, each output rounded once: h in the stream's type, z in bf16 and / or as e4m3
// with 1x128 UE8M0 scales (z comes from the unrounded h).
//
// A workgroup takes whole rows, its threads eight columns per chunk, and keeps a row in
// registers from the first reduction to the last store, so each input is read once and
// each output written once: bound by memory.
#include "block_device.hpp"
#include "block_launch.hpp"

namespace fp8bs {

namespace {

// Eight values of the residual stream (bf16 or fp32).
template <bool F32>
__device__ __forceinline__ void load8(const void* p, int64_t i, float* f) {
  if constexpr (F32) {
    const float* q = static_cast<const float*>(p) + i;
    const float4 a = *reinterpret_cast<const float4*>(q), b = *reinterpret_cast<const float4*>(q + 4);
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  } else {
    unpack_bf16x8(*reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(p) + i), f);
  }
}
template <bool F32>
__device__ __forceinline__ void store8(void* p, int64_t i, const float* f) {
  if constexpr (F32) {
    float* q = static_cast<float*>(p) + i;
    *reinterpret_cast<float4*>(q) = make_float4(f[0], f[1], f[2], f[3]);
    *reinterpret_cast<float4*>(q + 4) = make_float4(f[4], f[5], f[6], f[7]);
  } else {
    *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(p) + i) = pack_bf16x8(f);
  }
}
__device__ __forceinline__ void load_bf16x8(const uint16_t* p, float* f) {
  unpack_bf16x8(*reinterpret_cast<const u32x4*>(p), f);
}

template <bool F32, int CH>
__global__ __launch_bounds__(1024) void norm_kernel(NormProblem p, const void* __restrict__ x, int64_t ldx,
                                                    void* __restrict__ h, int64_t ldh, uint16_t* __restrict__ z,
                                                    int64_t ldz, uint8_t* __restrict__ q, int64_t ldq,
                                                    uint32_t* __restrict__ sf, int64_t ld_sf) {
  __shared__ float part[2][16];
  const int waves = blockDim.x >> 6;
  const int lane = threadIdx.x & 63;
  const float inv_n = 1.0f / (float)p.N;
  int turn = 0;  // of the halves of `part`: consecutive sums use different ones
  for (int64_t r = blockIdx.x; r < p.T; r += gridDim.x) {
    float v[CH][8];
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) v[c][i] = 0.0f;
    if (p.y != nullptr) {
      float ss = 0.0f;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int64_t col = (int64_t)(c * blockDim.x + threadIdx.x) * 8;
        if (col < p.N) load_bf16x8(p.y + r * p.ldy + col, v[c]);
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = __builtin_fmaf(v[c][i], v[c][i], ss);
      }
      float inv = 1.0f;
      if (p.w_post != nullptr) inv = rsqrtf(block_sum(ss, part[turn ^= 1], waves) * inv_n + p.eps);
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int64_t col = (int64_t)(c * blockDim.x + threadIdx.x) * 8;
        if (col < p.N) {
          float w[8];
          if (p.w_post != nullptr) {
            load_bf16x8(p.w_post + col, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[c][i] *= inv * (w[i] + p.offset);
          }
          if (p.gate != nullptr) {
            load_bf16x8(p.gate + r * p.ld_gate + col, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[c][i] *= w[i];
          }
        }
      }
    }
    float ss = 0.0f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int64_t col = (int64_t)(c * blockDim.x + threadIdx.x) * 8;
      if (col < p.N) {
        float a[8];
        load8<F32>(x, r * ldx + col, a);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          v[c][i] = __builtin_fmaf(p.residual_scale, a[i], v[c][i]);
          ss = __builtin_fmaf(v[c][i], v[c][i], ss);
        }
        if (h != nullptr) store8<F32>(h, r * ldh + col, v[c]);
      }
    }
    const float inv = rsqrtf(block_sum(ss, part[turn ^= 1], waves) * inv_n + p.eps);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int64_t col = (int64_t)(c * blockDim.x + threadIdx.x) * 8;
      const bool valid = col < p.N;
      if (valid) {
        float w[8];
        load_bf16x8(p.w_pre + col, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[c][i] *= inv * (w[i] + p.offset);
        if (z != nullptr) *reinterpret_cast<u32x4*>(z + r * ldz + col) = pack_bf16x8(v[c]);
      }
      if (q != nullptr) {
        const int e = group_exponent(v[c]);
        const uint32_t word = scale_word(valid ? (uint32_t)(e + 127) : 0u);
        if (valid) *reinterpret_cast<uint64_t*>(q + r * ldq + col) = codes_at(v[c], e);
        if (lane == 0 && valid) sf[(col / 512) * ld_sf + r] = word;
      }
    }
  }
}

// Sums of (a, b) over the workgroup.
__device__ __forceinline__ void block_sum2(float& a, float& b, float2* part, int waves) {
  a = wave_sum(a);
  b = wave_sum(b);
  if (waves == 1) return;
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = make_float2(a, b);
  __syncthreads();
  a = b = 0.0f;
  for (int w = 0; w < waves; ++w) {
    a += part[w].x;
    b += part[w].y;
  }
}

// Backward pass.  With hh = h * rh, rh = 1 / sqrt(mean(h^2) + eps), u = d_z (w_pre + offset):
//   dh = d_h + rh (u - hh mean(u hh)),  d_x = residual_scale dh,  d_w_pre = sum_t d_z hh
// and, with yh = y * ry, db = dh * gate, v = db (w_post + offset):
//   d_gate = dh b,  d_w_post = sum_t db yh,  d_y = ry (v - yh mean(v yh))   (db without w_post)
// Each workgroup walks rows blockIdx.x, + gridDim.x, ... and keeps the sums over its
// rows of the gradients of the weights (and of a gate shared by all tokens) in
// registers; they go to partials [sums][gridDim.x][N], which norm_sums_kernel adds up
// in a fixed order.
template <bool F32, int CH>
__global__ __launch_bounds__(1024) void norm_backward_kernel(NormProblem p, NormGradients g,
                                                             float* __restrict__ partials) {
  __shared__ float2 part[2][16];
  const int waves = blockDim.x >> 6;
  const float inv_n = 1.0f / (float)p.N;
  const bool shared_gate = p.gate != nullptr && p.ld_gate == 0;
  float s_pre[CH][8], s_post[CH][8], s_gate[CH][8];
#pragma unroll
  for (int c = 0; c < CH; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i) s_pre[c][i] = s_post[c][i] = s_gate[c][i] = 0.0f;
  int turn = 0;  // of the halves of `part`: consecutive sums use different ones
  for (int64_t r = blockIdx.x; r < p.T; r += gridDim.x) {
    float h[CH][8], u[CH][8];
    float ss = 0.0f, dot = 0.0f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int64_t col = (int64_t)(c * blockDim.x + threadIdx.x) * 8;
#pragma unroll
      for (int i = 0; i < 8; ++i) h[c][i] = u[c][i] = 0.0f;
      if (col < p.N) {
        float w[8];
        load8<F32>(g.h, r * g.ldh + col, h[c]);
        load_bf16x8(g.d_z + r * g.ld_dz + col, u[c]);
        load_bf16x8(p.w_pre + col, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          ss = __builtin_fmaf(h[c][i], h[c][i], ss);
          dot = __builtin_fmaf(u[c][i] * (w[i] + p.offset), h[c][i], dot);
        }
      }
    }
    block_sum2(ss, dot, part[turn ^= 1], waves);
    const float rh = rsqrtf(ss * inv_n + p.eps);
    const float mean = dot * rh * inv_n;  // of u hh
    float y[CH][8];
    float ss_y = 0.0f, dot_y = 0.0f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int64_t col = (int64_t)(c * blockDim.x + threadIdx.x) * 8;
#pragma unroll
      for (int i = 0; i < 8; ++i) y[c][i] = 0.0f;
      if (col < p.N) {
        float w[8], dh[8];
        load_bf16x8(p.w_pre + col, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) dh[i] = 0.0f;
        if (g.d_h != nullptr) load8<F32>(g.d_h, r * g.ld_dh + col, dh);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float hh = h[c][i] * rh;
          s_pre[c][i] = __builtin_fmaf(u[c][i], hh, s_pre[c][i]);
          u[c][i] = dh[i] + rh * (u[c][i] * (w[i] + p.offset) - hh * mean);  // dh
          dh[i] = p.residual_scale * u[c][i];
        }
        store8<F32>(g.d_x, r * g.ld_dx + col, dh);
        if (p.y != nullptr) {
          load_bf16x8(p.y + r * p.ldy + col, y[c]);
          float gt[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) w[i] = gt[i] = 1.0f;
          if (p.gate != nullptr) load_bf16x8(p.gate + r * p.ld_gate + col, gt);
          if (p.w_post != nullptr) {
            load_bf16x8(p.w_post + col, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float v = u[c][i] * gt[i] * (w[i] + p.offset);
              ss_y = __builtin_fmaf(y[c][i], y[c][i], ss_y);
              dot_y = __builtin_fmaf(v, y[c][i], dot_y);
            }
          }
        }
      }
    }
    if (p.y == nullptr) continue;
    float ry = 1.0f, mean_y = 0.0f;
    if (p.w_post != nullptr) {
      block_sum2(ss_y, dot_y, part[turn ^= 1], waves);
      ry = rsqrtf(ss_y * inv_n + p.eps);
      mean_y = dot_y * ry * inv_n;
    }
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int64_t col = (int64_t)(c * blockDim.x + threadIdx.x) * 8;
      if (col < p.N) {
        float w[8], gt[8], dy[8], dg[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = gt[i] = 1.0f;
        if (p.gate != nullptr) load_bf16x8(p.gate + r * p.ld_gate + col, gt);
        if (p.w_post != nullptr) {
          load_bf16x8(p.w_post + col, w);
#pragma unroll
          for (int i = 0; i < 8; ++i) w[i] += p.offset;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float yh = y[c][i] * ry, db = u[c][i] * gt[i];
          dg[i] = u[c][i] * yh * w[i];
          s_gate[c][i] += dg[i];
          if (p.w_post != nullptr) {
            s_post[c][i] = __builtin_fmaf(db, yh, s_post[c][i]);
            dy[i] = ry * (db * w[i] - yh * mean_y);
          } else {
            dy[i] = db;
          }
        }
        store8<false>(g.d_y, r * g.ld_dy + col, dy);
        if (p.gate != nullptr && !shared_gate) store8<false>(g.d_gate, r * g.ld_dgate + col, dg);
      }
    }
  }
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int64_t col = (int64_t)(c * blockDim.x + threadIdx.x) * 8;
    if (col < p.N) {
      float* to = partials + (int64_t)blockIdx.x * p.N;
      const int64_t next = (int64_t)gridDim.x * p.N;
      store8<true>(to, col, s_pre[c]);
      if (p.w_post != nullptr) {
        to += next;
        store8<true>(to, col, s_post[c]);
      }
      if (shared_gate) store8<true>(to + next, col, s_gate[c]);
    }
  }
}

// Sums of the partials: 64 columns per workgroup, its four wavefronts a quarter of the
// rows each, joined in a fixed order.
__global__ __launch_bounds__(256) void norm_sums_kernel(const float* __restrict__ partials, int rows, int64_t N,
                                                        float* __restrict__ a, float* __restrict__ b,
                                                        float* __restrict__ c) {
  __shared__ float part[4][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t col = (int64_t)blockIdx.x * 64 + lane;
  const float* from = partials + (int64_t)blockIdx.y * rows * N;
  float s = 0.0f;
  if (col < N)
    for (int r = wave; r < rows; r += 4) s += from[(int64_t)r * N + col];
  part[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && col < N) {
    float* to = blockIdx.y == 0 ? a : (blockIdx.y == 1 ? b : c);
    to[col] = (part[0][lane] + part[1][lane]) + (part[2][lane] + part[3][lane]);
  }
}

int backward_blocks(const NormProblem& p) { return (int)(p.T < 256 ? p.T : 256); }
int sums_of(const NormProblem& p) {
  return 1 + (p.w_post != nullptr ? 1 : 0) + (p.gate != nullptr && p.ld_gate == 0 ? 1 : 0);
}

// Threads of a workgroup whose threads hold ch chunks each.
unsigned threads_for(int64_t N, int ch) { return (unsigned)(64 * ((N / 8 + 64 * ch - 1) / (64 * ch))); }

template <bool F32>
hipError_t norm_as(const NormProblem& p, const void* x, int64_t ldx, void* h, int64_t ldh, uint16_t* z, int64_t ldz,
                   uint8_t* q, int64_t ldq, uint32_t* sf, int64_t ld_sf, hipStream_t stream) {
  const unsigned blocks = (unsigned)(p.T < 65536 ? p.T : 65536);
  if (p.N <= 8192)
    hipLaunchKernelGGL((norm_kernel<F32, 1>), dim3(blocks), dim3(threads_for(p.N, 1)), 0, stream, p, x, ldx, h, ldh, z,
                       ldz, q, ldq, sf, ld_sf);
  else
    hipLaunchKernelGGL((norm_kernel<F32, 2>), dim3(blocks), dim3(threads_for(p.N, 2)), 0, stream, p, x, ldx, h, ldh, z,
                       ldz, q, ldq, sf, ld_sf);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_norm(const NormProblem& p, const void* x, int64_t ldx, void* h, int64_t ldh, uint16_t* z,
                       int64_t ldz, uint8_t* q, int64_t ldq, uint32_t* sf, int64_t ld_sf, hipStream_t stream) {
  return p.f32 ? norm_as<true>(p, x, ldx, h, ldh, z, ldz, q, ldq, sf, ld_sf, stream)
               : norm_as<false>(p, x, ldx, h, ldh, z, ldz, q, ldq, sf, ld_sf, stream);
}

size_t norm_backward_scratch_bytes(const NormProblem& p, const NormGradients&) {
  return (size_t)sums_of(p) * backward_blocks(p) * p.N * sizeof(float);
}

hipError_t launch_norm_backward(const NormProblem& p, const NormGradients& g, float* partials, hipStream_t stream) {
  const int blocks = backward_blocks(p);
  const dim3 grid((unsigned)blocks);
  if (p.N <= 8192) {
    if (p.f32)
      hipLaunchKernelGGL((norm_backward_kernel<true, 1>), grid, dim3(threads_for(p.N, 1)), 0, stream, p, g, partials);
    else
      hipLaunchKernelGGL((norm_backward_kernel<false, 1>), grid, dim3(threads_for(p.N, 1)), 0, stream, p, g, partials);
  } else {
    if (p.f32)
      hipLaunchKernelGGL((norm_backward_kernel<true, 2>), grid, dim3(threads_for(p.N, 2)), 0, stream, p, g, partials);
    else
      hipLaunchKernelGGL((norm_backward_kernel<false, 2>), grid, dim3(threads_for(p.N, 2)), 0, stream, p, g, partials);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  float* sums[3] = {g.d_w_pre, nullptr, nullptr};
  int n = 1;
  if (p.w_post != nullptr) sums[n++] = g.d_w_post;
  if (p.gate != nullptr && p.ld_gate == 0) sums[n++] = static_cast<float*>(g.d_gate);
  hipLaunchKernelGGL(norm_sums_kernel, dim3((unsigned)((p.N + 63) / 64), (unsigned)n), dim3(256), 0, stream, partials,
                     blocks, p.N, sums[0], sums[1], sums[2]);
  return hipGetLastError();
}

}  // namespace fp8bs
