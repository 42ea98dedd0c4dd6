// 8-bit activation checkpoint of the gated activation, over a masked expert batch.
//
// Forward: for every valid row, y = silu(gate) * up quantized for the next product
// (value for value what silu_mul_quant_group_pack writes) and, from the same read, gate
// and up themselves as e4m3 with 1x128 UE8M0 scales: half the bytes of the bf16
// activations to keep until the backward pass.
// Backward, from the checkpoint: with s = sigmoid(gate),
//   d_gate = d_y up s (1 + gate (1 - s)),   d_up = d_y gate s
// in fp32, rounded once: to bf16, or to e4m3 for the masked GEMM that takes the gradient on.
// The checkpoint's own rounding (at most 2^-4 of a value) is what half the memory costs.
//
// Streams bound by memory.  One wavefront takes one (row, 512 columns of H) unit: eight
// columns of gate and of up per lane, sixteen lanes per quantization group, no LDS for
// the data.  A grid sized to the chip strides over the units of the valid rows, so padded
// rows cost nothing, and each wavefront has the loads of its next unit in flight while it
// works on one.
//
// Measured, 32768 valid rows of H = 2048 in 32 experts: forward 92.5 us, 471 MB, 5.1 TB/s (it
// issues about 250 vector instructions a unit, three quarters of the time that memory
// takes); backward to bf16 99 us, 538 MB, 5.4 TB/s, to codes 81 us, 405 MB, 5.0 TB/s.  A copy of
// 400 MB reaches 5.4 TB/s.
// Before: waiting for each unit's own loads 108 and 116 us, and a contiguous run of units
// for each wavefront 118 us forward.
#include "block_device.hpp"
#include "block_launch.hpp"

namespace fp8bs {

namespace {

// Sums of the clamped counts of the experts before each (LDS, E + 1 entries; the entries up
// to the next multiple of 64 are past every row) by a workgroup of 256 threads; returns the
// number of valid rows.
__device__ __forceinline__ int sum_counts(const int32_t* __restrict__ masked_m, int E, int64_t M_max, int* before) {
  __shared__ int chunk[4];
  const int tid = threadIdx.x, lane = tid & 63;
  int base = 0;
  if (tid == 0) before[0] = 0;
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
    if (e0 + tid < (E + 63) / 64 * 64) before[e0 + tid + 1] = e0 + tid < E ? base + c : INT32_MAX;
    base += chunk[0] + chunk[1] + chunk[2] + chunk[3];
    __syncthreads();
  }
  return base;
}

// The (row, word) units of one wavefront: every `stride`-th unit of the valid rows from `u`
// on, so that the wavefronts of the chip read neighbouring memory.
struct Units {
  int row, w;  // row among the valid rows, word of the row: the unit
  int rows;    // valid rows
  int row_step, w_step;
  int W;
  const int* before;
  int e, r;  // expert of the row, row in the expert

  // The first expert whose rows reach past the row, 64 at a time.
  __device__ __forceinline__ void find() {
    const int lane = threadIdx.x & 63;
    for (e = 0;; e += 64) {
      const uint64_t past = __ballot(before[e + lane + 1] > row);
      if (past != 0) {
        e += __builtin_ctzll(past);
        break;
      }
    }
    r = row - __builtin_amdgcn_readfirstlane(before[e]);
  }
  __device__ __forceinline__ bool next() {
    row += row_step;
    w += w_step;
    if (w >= W) {
      w -= W;
      ++row;
    }
    if (row >= rows) return false;  // e and r stay those of the last unit
    find();
    return true;
  }
};

// The wavefront's first unit, if it has one.
__device__ __forceinline__ bool first_unit(Units& s, const int32_t* __restrict__ masked_m, int E, int64_t M_max, int W,
                                           int* before) {
  s.rows = __builtin_amdgcn_readfirstlane(sum_counts(masked_m, E, M_max, before));
  const int first = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), stride = gridDim.x * 4;
  s.row = first / W;
  s.w = first - s.row * W;
  s.row_step = stride / W;
  s.w_step = stride - s.row_step * W;
  s.W = W;
  s.before = before;
  if (s.row >= s.rows) return false;
  s.find();
  return true;
}

__global__ __launch_bounds__(256) void silu_checkpoint_kernel(const uint16_t* __restrict__ x,
                                                              const int32_t* __restrict__ masked_m, int E,
                                                              int64_t M_max, int64_t H, int W,
                                                              uint8_t* __restrict__ q, uint32_t* __restrict__ sf,
                                                              uint8_t* __restrict__ cq, uint32_t* __restrict__ csf) {
  __shared__ int before[kCheckpointMaxE + 1];
  const int lane = threadIdx.x & 63;
  Units s;
  if (!first_unit(s, masked_m, E, M_max, W, before)) return;
  // one unit: issue the loads of the next one into (gn, un), then work on (gv, uv).  The
  // loop alternates two register sets: a copy would wait for the loads in flight.
  auto load = [&](bool more, u32x4& gn, u32x4& un) {
    const uint16_t* from = x + ((int64_t)s.e * M_max + s.r) * 2 * H;
    const uint32_t bytes = more ? (uint32_t)(2 * H) : 0u, off = (s.w * 512 + lane * 8) * 2;
    gn = run_load16(shared_run(from, bytes), off);
    un = run_load16(shared_run(from + H, bytes), off);
  };
  auto unit = [&](const u32x4& gv, const u32x4& uv, u32x4& gn, u32x4& un) -> bool {
    const int64_t row = (int64_t)s.e * M_max + s.r, word = ((int64_t)s.e * W + s.w) * M_max + s.r;
    const int64_t words = ((int64_t)s.e * 2 * W + s.w) * M_max + s.r;
    const uint32_t col = s.w * 512 + lane * 8;
    const bool valid = col < H;
    const bool more = s.next();
    load(more, gn, un);
    __builtin_amdgcn_sched_barrier(0);  // the next unit's loads go out before this one is worked on
    float g[8], up[8], y[8];
    unpack_bf16x8(gv, g);
    unpack_bf16x8(uv, up);
    // reciprocal of 1 ulp, as the forward without a checkpoint has it
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = g[i] * __builtin_amdgcn_rcpf(1.0f + expf(-g[i])) * up[i];
    const uint32_t by = group_byte(y), bg = group_byte(g), bu = group_byte(up);
    const uint32_t bytes = (uint32_t)H;
    run_store(shared_run(q + row * H, bytes), col, codes_at(y, by));
    run_store(shared_run(cq + row * 2 * H, bytes), col, codes_at(g, bg));
    run_store(shared_run(cq + row * 2 * H + H, bytes), col, codes_at(up, bu));
    // one word each, by lane 0
    run_store(shared_run(sf + word, 4), lane * 4, scale_word(valid ? by : 0u));
    run_store(shared_run(csf + words, 4), lane * 4, scale_word(valid ? bg : 0u));
    run_store(shared_run(csf + words + W * M_max, 4), lane * 4, scale_word(valid ? bu : 0u));
    return more;
  };
  u32x4 g0, u0, g1, u1;
  load(true, g0, u0);
  while (unit(g0, u0, g1, u1) && unit(g1, u1, g0, u0)) {
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
  __shared__ int before[kCheckpointMaxE + 1];
  const int lane = threadIdx.x & 63;
  Units s;
  if (!first_unit(s, masked_m, E, M_max, W, before)) return;
  const int64_t W2 = (2 * H / 128 + 3) / 4;
  struct Loaded {
    u32x4 d;
    u32x2 g, u;
    uint32_t wg, wu;  // scale words
  };
  auto load = [&](bool more, Loaded& n) {
    const int64_t row = (int64_t)s.e * M_max + s.r;
    const uint32_t bytes = more ? (uint32_t)H : 0u, col = s.w * 512 + lane * 8;
    n.d = run_load16(shared_run(d_y + row * H, 2 * bytes), col * 2);
    n.g = run_load8(shared_run(cq + row * 2 * H, bytes), col);
    n.u = run_load8(shared_run(cq + row * 2 * H + H, bytes), col);
    const uint32_t* words = csf + ((int64_t)s.e * 2 * W + s.w) * M_max + s.r;
    n.wg = words[0];
    n.wu = words[W * M_max];
  };
  // one unit, with the next one's loads in flight, as in the forward pass
  auto unit = [&](const Loaded& v, Loaded& n) -> bool {
    const int64_t e = s.e, r = s.r, row = e * M_max + r;
    const uint32_t col = s.w * 512 + lane * 8;
    const bool more = s.next();
    load(more, n);
    __builtin_amdgcn_sched_barrier(0);
    const int sh = 8 * (lane >> 4);
    const float sg = __uint_as_float(((v.wg >> sh) & 0xFFu) << 23);
    const float su = __uint_as_float(((v.wu >> sh) & 0xFFu) << 23);
    float d[8], g[8], up[8], dg[8], du[8];
    unpack_bf16x8(v.d, d);
    unpack_e4m3x8(v.g, g);
    unpack_e4m3x8(v.u, up);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float gate = g[i] * sg, u = up[i] * su;
      // s and 1 - s from e^-|g| <= 1: 1 / (1 + e^-|g|) and e^-|g| times that, without the
      // cancellation, and small only where they are (the reciprocal of 1 + e^88 would be 0)
      const float ex = expf(-__builtin_fabsf(gate));
      const float r = __builtin_amdgcn_rcpf(1.0f + ex), re = r * ex;
      const float sig = gate < 0.0f ? re : r, rest = gate < 0.0f ? r : re;
      dg[i] = d[i] * u * sig * __builtin_fmaf(gate, rest, 1.0f);
      du[i] = d[i] * gate * sig;
    }
    if constexpr (QUANT) {
      const uint32_t bg = group_byte(dg), bu = group_byte(du);
      run_store(shared_run(q + row * 2 * H, (uint32_t)H), col, codes_at(dg, bg));
      run_store(shared_run(q + row * 2 * H + H, (uint32_t)H), col, codes_at(du, bu));
      // scale bytes of the row's 2H / 128 groups: the up half starts inside a word where H is
      // no multiple of 512, so each group's byte is stored by itself
      if (col < H && (lane & 15) == 0) {
        uint8_t* to = reinterpret_cast<uint8_t*>(sf);
        const int64_t gg = col / 128, gu = (H + col) / 128;
        to[((e * W2 + gg / 4) * M_max + r) * 4 + gg % 4] = (uint8_t)bg;
        to[((e * W2 + gu / 4) * M_max + r) * 4 + gu % 4] = (uint8_t)bu;
        // the last word's bytes past the row's groups are zero
        if (gu == 2 * H / 128 - 1)
          for (int64_t k = gu + 1; k < 4 * W2; ++k) to[((e * W2 + k / 4) * M_max + r) * 4 + k % 4] = 0;
      }
    } else {
      run_store(shared_run(d_x + row * 2 * H, (uint32_t)(2 * H)), col * 2, pack_bf16x8(dg));
      run_store(shared_run(d_x + row * 2 * H + H, (uint32_t)(2 * H)), col * 2, pack_bf16x8(du));
    }
    return more;
  };
  Loaded a, b;
  load(true, a);
  while (unit(a, b) && unit(b, a)) {
  }
}

// Seven workgroups on each of the 256 compute units, what the registers of the quantizing
// backward pass leave room for (forward, 32768 rows of H = 2048: 92.5 us; 94 with eight, 96
// with four; the backward pass is within 1% between four and eight).
unsigned unit_blocks(int64_t E, int64_t M_max, int64_t W) {
  const int64_t most = (E * M_max * W + 3) / 4;
  return (unsigned)(most < 7 * 256 ? most : 7 * 256);
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
