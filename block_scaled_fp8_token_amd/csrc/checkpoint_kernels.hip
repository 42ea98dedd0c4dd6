// 8-bit activation checkpoint of the gated activation, over a masked expert batch.
//
// Forward: for every valid row, y = silu(gate) * up quantized for the next product
// (value for value what silu_mul_quant_group_pack writes) and, from the same read, gate
// and up themselves as e4m3 with 1x128 UE8M0 scales: half the bytes of the bf16
// activations to keep until the backward pass.
// Backward, from the checkpoint: with s = sigmoid(gate),
//   d_gate = d_y up s (1 + gate (1 - s)),   d_up = d_y gate s
// in bf16, or quantized for the product that takes the gradient on.
//
// Streams bound by memory.  One wavefront takes one (row, 512 columns of H) unit: eight
// columns of gate and of up per lane, sixteen lanes per quantization group, no LDS for
// the data.  Each wavefront walks one contiguous run of the valid units, so padded rows
// cost nothing and a run's expert is looked up once.
#include "block_device.hpp"
#include "block_launch.hpp"

namespace fp8bs {

namespace {

// The run of valid (row, word) units of one wavefront.
struct Units {
  int64_t u, end;   // unit and end of the run
  int64_t r;        // row in its expert
  int e, w;         // expert, word of the row
  int count;        // valid rows of e
};

// Sums of the clamped counts of the experts up to each (LDS, E + 1 entries), by a
// workgroup of 256 threads; then the run of wavefront `wave` of `waves`.
__device__ __forceinline__ Units find_units(const int32_t* __restrict__ masked_m, int E, int64_t M_max, int W,
                                            int* upto, int64_t wave, int64_t waves) {
  __shared__ int chunk[4];
  const int tid = threadIdx.x, lane = tid & 63;
  int base = 0;
  for (int e0 = 0; e0 < E; e0 += 256) {
    int c = 0;
    if (e0 + tid < E) {
      const int64_t m = masked_m[e0 + tid];
      c = (int)(m < 0 ? 0 : (m > M_max ? M_max : m));
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(c, d);
      if (lane >= d) c += o;
    }
    if (lane == 63) chunk[tid >> 6] = c;
    __syncthreads();
    for (int k = 0; k < (tid >> 6); ++k) c += chunk[k];
    if (e0 + tid < E) upto[e0 + tid + 1] = base + c;
    base += chunk[0] + chunk[1] + chunk[2] + chunk[3];
    __syncthreads();
  }
  if (tid == 0) upto[0] = 0;
  __syncthreads();
  Units s;
  const int64_t total = (int64_t)base * W;
  const int64_t per = (total + waves - 1) / waves;
  s.u = wave * per;
  s.end = s.u + per < total ? s.u + per : total;
  if (s.u >= s.end) return s;
  const int row = (int)(s.u / W);  // among all valid rows
  s.w = (int)(s.u - (int64_t)row * W);
  int lo = 0, hi = E;  // upto[lo] <= row < upto[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (upto[mid] <= row) lo = mid; else hi = mid;
  }
  s.e = lo;
  s.r = row - upto[lo];
  s.count = upto[lo + 1] - upto[lo];
  return s;
}

__device__ __forceinline__ void next_unit(Units& s, const int* upto, int W) {
  ++s.u;
  if (++s.w < W) return;
  s.w = 0;
  if (++s.r < s.count || s.u >= s.end) return;
  s.r = 0;
  do {
    ++s.e;
    s.count = upto[s.e + 1] - upto[s.e];
  } while (s.count == 0);  // units are left, so an expert with rows follows
}

__global__ __launch_bounds__(256) void silu_checkpoint_kernel(const uint16_t* __restrict__ x,
                                                              const int32_t* __restrict__ masked_m, int E,
                                                              int64_t M_max, int64_t H, int W,
                                                              uint8_t* __restrict__ q, uint32_t* __restrict__ sf,
                                                              uint8_t* __restrict__ cq, uint32_t* __restrict__ csf) {
  __shared__ int upto[kCheckpointMaxE + 1];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  for (Units s = find_units(masked_m, E, M_max, W, upto, (int64_t)blockIdx.x * 4 + wave, (int64_t)gridDim.x * 4);
       s.u < s.end; next_unit(s, upto, W)) {
    const int64_t row = s.e * M_max + s.r;
    const int64_t col = (int64_t)s.w * 512 + lane * 8;
    const bool valid = col < H;
    float g[8], up[8], y[8];
    u32x4 gv = {0u, 0u, 0u, 0u}, uv = {0u, 0u, 0u, 0u};
    if (valid) {
      gv = *reinterpret_cast<const u32x4*>(x + row * 2 * H + col);
      uv = *reinterpret_cast<const u32x4*>(x + row * 2 * H + H + col);
    }
    unpack_bf16x8(gv, g);
    unpack_bf16x8(uv, up);
    // reciprocal of 1 ulp, as the forward without a checkpoint has it
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = g[i] * __builtin_amdgcn_rcpf(1.0f + expf(-g[i])) * up[i];
    const int ey = group_exponent(y), eg = group_exponent(g), eu = group_exponent(up);
    if (valid) {
      *reinterpret_cast<uint64_t*>(q + row * H + col) = codes_at(y, ey);
      *reinterpret_cast<uint64_t*>(cq + row * 2 * H + col) = codes_at(g, eg);
      *reinterpret_cast<uint64_t*>(cq + row * 2 * H + H + col) = codes_at(up, eu);
    }
    const uint32_t wy = scale_word(valid ? (uint32_t)(ey + 127) : 0u);
    const uint32_t wg = scale_word(valid ? (uint32_t)(eg + 127) : 0u);
    const uint32_t wu = scale_word(valid ? (uint32_t)(eu + 127) : 0u);
    if (lane == 0) {
      sf[((int64_t)s.e * W + s.w) * M_max + s.r] = wy;
      csf[((int64_t)s.e * 2 * W + s.w) * M_max + s.r] = wg;
      csf[((int64_t)s.e * 2 * W + W + s.w) * M_max + s.r] = wu;
    }
  }
}

template <bool QUANT>
__global__ __launch_bounds__(256) void silu_backward_kernel(const uint16_t* __restrict__ d_y,
                                                            const int32_t* __restrict__ masked_m, int E,
                                                            int64_t M_max, int64_t H, int W,
                                                            const uint8_t* __restrict__ cq,
                                                            const uint32_t* __restrict__ csf,
                                                            uint16_t* __restrict__ d_x, uint8_t* __restrict__ q,
                                                            uint32_t* __restrict__ sf) {
  __shared__ int upto[kCheckpointMaxE + 1];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  for (Units s = find_units(masked_m, E, M_max, W, upto, (int64_t)blockIdx.x * 4 + wave, (int64_t)gridDim.x * 4);
       s.u < s.end; next_unit(s, upto, W)) {
    const int64_t row = s.e * M_max + s.r;
    const int64_t col = (int64_t)s.w * 512 + lane * 8;
    const bool valid = col < H;
    u32x4 dv = {0u, 0u, 0u, 0u};
    u32x2 gv = {0u, 0u}, uv = {0u, 0u};
    if (valid) {
      dv = *reinterpret_cast<const u32x4*>(d_y + row * H + col);
      gv = *reinterpret_cast<const u32x2*>(cq + row * 2 * H + col);
      uv = *reinterpret_cast<const u32x2*>(cq + row * 2 * H + H + col);
    }
    const uint32_t wg = csf[((int64_t)s.e * 2 * W + s.w) * M_max + s.r];
    const uint32_t wu = csf[((int64_t)s.e * 2 * W + W + s.w) * M_max + s.r];
    const int sh = 8 * (lane >> 4);
    const float sg = __uint_as_float(((wg >> sh) & 0xFFu) << 23), su = __uint_as_float(((wu >> sh) & 0xFFu) << 23);
    float d[8], g[8], up[8], dg[8], du[8];
    unpack_bf16x8(dv, d);
    unpack_e4m3x8(gv, g);
    unpack_e4m3x8(uv, up);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float gate = g[i] * sg, u = up[i] * su;
      const float e = expf(-gate);
      const float sig = __builtin_amdgcn_rcpf(1.0f + e);
      // 1 - s = e s, without the cancellation; at gates so low that e overflows s is 0
      // and both gradients are 0
      const float rest = e < 3e38f ? e * sig : 1.0f;
      dg[i] = d[i] * u * sig * __builtin_fmaf(gate, rest, 1.0f);
      du[i] = d[i] * gate * sig;
    }
    if constexpr (QUANT) {
      const int eg = group_exponent(dg), eu = group_exponent(du);
      if (valid) {
        *reinterpret_cast<uint64_t*>(q + row * 2 * H + col) = codes_at(dg, eg);
        *reinterpret_cast<uint64_t*>(q + row * 2 * H + H + col) = codes_at(du, eu);
        // scale bytes of the row's 2H / 128 groups: the up half starts inside a word where
        // H is no multiple of 512, so each group's byte is stored by itself
        if ((lane & 15) == 0) {
          uint8_t* to = reinterpret_cast<uint8_t*>(sf);
          const int64_t W2 = (2 * H / 128 + 3) / 4;
          const int64_t gg = col / 128, gu = (H + col) / 128;
          to[(((int64_t)s.e * W2 + gg / 4) * M_max + s.r) * 4 + gg % 4] = (uint8_t)(eg + 127);
          to[(((int64_t)s.e * W2 + gu / 4) * M_max + s.r) * 4 + gu % 4] = (uint8_t)(eu + 127);
          // the last word's bytes past the row's groups are zero
          if (gu == 2 * H / 128 - 1)
            for (int64_t k = gu + 1; k < 4 * W2; ++k) to[(((int64_t)s.e * W2 + k / 4) * M_max + s.r) * 4 + k % 4] = 0;
        }
      }
    } else if (valid) {
      *reinterpret_cast<u32x4*>(d_x + row * 2 * H + col) = pack_bf16x8(dg);
      *reinterpret_cast<u32x4*>(d_x + row * 2 * H + H + col) = pack_bf16x8(du);
    }
  }
}

unsigned unit_blocks(int64_t E, int64_t M_max, int64_t W) {
  const int64_t most = (E * M_max * W + 3) / 4;
  return (unsigned)(most < 2048 ? most : 2048);
}

}  // namespace

hipError_t launch_silu_checkpoint(const uint16_t* x, const int32_t* masked_m, int64_t E, int64_t M_max, int64_t H,
                                  uint8_t* q, uint32_t* sf, uint8_t* cq, uint32_t* csf, hipStream_t stream) {
  const int64_t W = (H / 128 + 3) / 4;
  hipLaunchKernelGGL(silu_checkpoint_kernel, dim3(unit_blocks(E, M_max, W)), dim3(256), 0, stream, x, masked_m, (int)E,
                     M_max, H, (int)W, q, sf, cq, csf);
  return hipGetLastError();
}

hipError_t launch_silu_backward(const uint16_t* d_y, const int32_t* masked_m, int64_t E, int64_t M_max, int64_t H,
                                const uint8_t* cq, const uint32_t* csf, uint16_t* d_x, uint8_t* q, uint32_t* sf,
                                hipStream_t stream) {
  const int64_t W = (H / 128 + 3) / 4;
  const dim3 grid(unit_blocks(E, M_max, W));
  if (q != nullptr)
    hipLaunchKernelGGL(silu_backward_kernel<true>, grid, dim3(256), 0, stream, d_y, masked_m, (int)E, M_max, H, (int)W,
                       cq, csf, d_x, q, sf);
  else
    hipLaunchKernelGGL(silu_backward_kernel<false>, grid, dim3(256), 0, stream, d_y, masked_m, (int)E, M_max, H, (int)W,
                       cq, csf, d_x, q, sf);
  return hipGetLastError();
}

}  // namespace fp8bs
