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
// each output written once: bound by memory.  A grid that fits the chip strides over the
// rows; weights stay in registers, and the next row's loads are in flight while a row is
// worked on.
//
// Measured: forward, 8192 x 7168 from bf16 with both norms and a shared gate to a bf16
// stream and codes, 73 us, 411 MB, 5.6 TB/s (a copy of 400 MB reaches 5.4): 115 us with a
// workgroup per row and x loaded after the first reduction, 83 us with the next row's loads
// ahead, 76 us with those loads and the stores free of branches, 73 us with the weights
// unpacked once.  Backward, 4097 x 7168 with an fp32 stream, 104 us, 528 MB and 22 MB of
// partial sums, 5.3 TB/s, and 5.3 us for the sums over the workgroups (154 us in all without the
// loads ahead, 139 where all three sums stayed in registers and spilled).
#include <type_traits>

#include "block_device.hpp"
#include "block_launch.hpp"

namespace fp8bs {

namespace {

// A row of the residual stream (bf16 or fp32).  Rows are addressed by a pointer that is
// the same for the whole workgroup (scalar registers) and a 32-bit column per thread.
template <bool F32>
using Stream = std::conditional_t<F32, float, uint16_t>;

// Eight of its values, as loaded.
template <bool F32>
struct Raw {
  u32x4 v[F32 ? 2 : 1];
};
// A row of a tensor as memory that the workgroup shares (no bytes: one that is not there,
// which reads as zeros and is not written).
template <typename T>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t row_run(const T* p, int64_t ld, int64_t r, int64_t N, bool there) {
  return shared_run(p + r * ld, there && p != nullptr ? (uint32_t)(N * sizeof(T)) : 0u);
}
template <bool F32>
__device__ __forceinline__ Raw<F32> load_raw(__amdgpu_buffer_rsrc_t row, uint32_t col) {
  Raw<F32> r;
#pragma unroll
  for (int k = 0; k < (F32 ? 2 : 1); ++k) r.v[k] = run_load16(row, col * (F32 ? 4 : 2) + 16 * k);
  return r;
}
template <bool F32>
__device__ __forceinline__ void unpack_raw(const Raw<F32>& r, float* f) {
  if constexpr (F32) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(r.v[i / 4][i % 4]);
  } else {
    unpack_bf16x8(r.v[0], f);
  }
}
template <bool F32>
__device__ __forceinline__ void store8(__amdgpu_buffer_rsrc_t row, uint32_t col, const float* f) {
  if constexpr (F32) {
    u32x4 a, b;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      a[i] = __float_as_uint(f[i]);
      b[i] = __float_as_uint(f[4 + i]);
    }
    run_store(row, col * 4, a);
    run_store(row, col * 4 + 16, b);
  } else {
    run_store(row, col * 2, pack_bf16x8(f));
  }
}
// Eight of a vector that every row uses.
__device__ __forceinline__ u32x4 load_weights(const uint16_t* w, uint32_t col) {
  return *reinterpret_cast<const u32x4*>(w + col);
}

// Keeps the compiler from knowing a register's contents, so that a row stays packed between
// the phases that unpack it instead of being kept unpacked in twice as many registers.
__device__ __forceinline__ void keep_packed(u32x4& v) { asm volatile("" : "+v"(v)); }

// One row as loaded, the chunks of one thread.  FULL: a gate of its own for every token.
template <bool F32, bool FULL, int CH>
struct NormRow {
  Raw<F32> x[CH];
  u32x4 y[CH], gate[FULL ? CH : 1];
};

// 1 / sqrt(mean + eps) of a sum of squares over n (1 / n as a sum of two fp32).  One Newton
// step on the 1 ulp of rsqrtf, as an error here is one of the whole row and moves its codes; a
// mean of 0 or past fp32 keeps rsqrtf's answer.
__device__ __forceinline__ float inverse_rms(float sum, float inv_n, float inv_n_lo, float eps) {
  const float m = __builtin_fmaf(sum, inv_n, sum * inv_n_lo) + eps, r = rsqrtf(m);
  const float e = __builtin_fmaf(-(m * r), r, 1.0f);
  return __builtin_fabsf(e) < 1.0f ? __builtin_fmaf(0.5f * r, e, r) : r;
}

// Sum over a workgroup of at most sixteen wavefronts, the same value in every thread: each
// lane takes one wavefront's sum and the sixteen lanes of a row add theirs.  `part` is
// sixteen floats of LDS, zero past the wavefronts that there are; a caller that sums again
// uses another `part` in between (that one's barrier separates two uses of this one).
__device__ __forceinline__ float block_sum(float v, float* part, int waves) {
  v = wave_sum(v);
  if (waves == 1) return v;
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  return row16_sum(part[threadIdx.x & 15]);
}

template <bool F32, bool FULL, bool QUANT, int CH>
__global__ __launch_bounds__(1024) void norm_kernel(
    NormProblem p, const Stream<F32>* __restrict__ x, int64_t ldx, Stream<F32>* __restrict__ h, int64_t ldh,
    uint16_t* __restrict__ z, int64_t ldz, uint8_t* __restrict__ q, int64_t ldq, uint32_t* __restrict__ sf,
    int64_t ld_sf) {
  __shared__ float part[2][16];
  const int waves = blockDim.x >> 6;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const float inv_n = 1.0f / (float)p.N, inv_n_lo = __builtin_fmaf(-inv_n, (float)p.N, 1.0f) * inv_n;
  if (threadIdx.x < 32) part[threadIdx.x >> 4][threadIdx.x & 15] = 0.0f;
  __syncthreads();
  int turn = 0;  // of the halves of `part`: consecutive sums use different ones
  // weights of the columns, in fp32: the branch's (w_post + offset, times a shared gate), z's
  float w_branch[CH][8], w_z[CH][8];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const uint32_t col = (c * blockDim.x + threadIdx.x) * 8;
    float g[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w_branch[c][i] = g[i] = w_z[c][i] = 1.0f;
    if (col < p.N) {
      unpack_bf16x8(load_weights(p.w_pre, col), w_z[c]);
      if (p.w_post != nullptr) unpack_bf16x8(load_weights(p.w_post, col), w_branch[c]);
      if (!FULL && p.gate != nullptr) unpack_bf16x8(load_weights(p.gate, col), g);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (p.w_post != nullptr) w_branch[c][i] += p.offset;
      w_branch[c][i] *= g[i];
      w_z[c][i] += p.offset;
    }
  }
  using Row = NormRow<F32, FULL, CH>;
  auto load = [&](int64_t r, bool there, Row& row) {
    const auto ys = row_run(p.y, p.ldy, r, p.N, there), xs = row_run(x, ldx, r, p.N, there);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const uint32_t col = (c * blockDim.x + threadIdx.x) * 8;
      row.y[c] = run_load16(ys, col * 2);
      row.x[c] = load_raw<F32>(xs, col);
      if constexpr (FULL) row.gate[c] = run_load16(row_run(p.gate, p.ld_gate, r, p.N, there), col * 2);
    }
  };
  // one row: issue the loads of the workgroup's next one, then work on this one.  The loop
  // alternates two register sets: a copy would wait for the loads in flight.
  int64_t r = blockIdx.x;  // grid <= T: every workgroup has a row
  auto work = [&](Row& cur, Row& next) -> bool {
    const int64_t now = r;
    r += gridDim.x;
    const bool more = r < p.T;
    load(r, more, next);
    __builtin_amdgcn_sched_barrier(0);  // those loads go out before this row is worked on
    float v[CH][8];
    float ss = 0.0f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      unpack_bf16x8(cur.y[c], v[c]);
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = __builtin_fmaf(v[c][i], v[c][i], ss);
    }
    float inv = 1.0f;
    if (p.w_post != nullptr) inv = inverse_rms(block_sum(ss, part[turn ^= 1], waves), inv_n, inv_n_lo, p.eps);
    const auto hs = row_run(h, ldh, now, p.N, true);
    ss = 0.0f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const uint32_t col = (c * blockDim.x + threadIdx.x) * 8;
      float x8[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[c][i] *= inv * w_branch[c][i];
      if constexpr (FULL) {
        float g[8];
        unpack_bf16x8(cur.gate[c], g);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[c][i] *= g[i];
      }
      unpack_raw<F32>(cur.x[c], x8);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[c][i] = __builtin_fmaf(p.residual_scale, x8[i], v[c][i]);
        ss = __builtin_fmaf(v[c][i], v[c][i], ss);
      }
      store8<F32>(hs, col, v[c]);
    }
    inv = inverse_rms(block_sum(ss, part[turn ^= 1], waves), inv_n, inv_n_lo, p.eps);
    const auto zs = row_run(z, ldz, now, p.N, true);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const uint32_t col = (c * blockDim.x + threadIdx.x) * 8;
#pragma unroll
      for (int i = 0; i < 8; ++i) v[c][i] *= inv * w_z[c][i];
      store8<false>(zs, col, v[c]);
      if constexpr (QUANT) {
        const uint32_t byte = group_byte(v[c]);
        run_store(row_run(q, ldq, now, p.N, true), col, codes_at(v[c], byte));
        // the word of the wavefront's 512 columns, by lane 0 (which a word past the row has not)
        const uint32_t word = c * waves + wave;
        run_store(shared_run(sf + word * ld_sf + now, word * 512 < p.N ? 4u : 0u), lane * 4,
                  scale_word(col < p.N ? byte : 0u));
      }
    }
    return more;
  };
  Row a, b;
  load(r, true, a);
  while (work(a, b) && work(b, a)) {
  }
}

// Sums of (a, b) over the workgroup, as block_sum.
__device__ __forceinline__ void block_sum2(float& a, float& b, float2* part, int waves) {
  a = wave_sum(a);
  b = wave_sum(b);
  if (waves == 1) return;
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = make_float2(a, b);
  __syncthreads();
  const float2 v = part[threadIdx.x & 15];
  a = row16_sum(v.x);
  b = row16_sum(v.y);
}

// Backward pass.  With hh = h * rh, rh = 1 / sqrt(mean(h^2) + eps), u = d_z (w_pre + offset):
//   dh = d_h + rh (u - hh mean(u hh)),  d_x = residual_scale dh,  d_w_pre = sum_t d_z hh
// and, with yh = y * ry, db = dh * gate, v = db (w_post + offset):
//   d_gate = dh b,  d_w_post = sum_t db yh,  d_y = ry (v - yh mean(v yh))   (db without w_post)
// Each workgroup walks rows blockIdx.x, + gridDim.x, ... and keeps the sums over its
// rows: those of the weights' gradients in LDS, that of a gate shared by all tokens in
// registers.  They go to partials [sums][gridDim.x][N], which norm_sums_kernel adds up
// in a fixed order.
template <bool F32, bool FULL>
struct GradRow {
  Raw<F32> h, d_h;
  u32x4 d_z, y, gate;
};
template <bool F32, bool FULL>
__device__ __forceinline__ void load_row(const NormProblem& p, const NormGradients& g, int64_t r, uint32_t col,
                                         bool there, GradRow<F32, FULL>& row) {
  const auto* h = static_cast<const Stream<F32>*>(g.h);
  const auto* d_h = static_cast<const Stream<F32>*>(g.d_h);
  row.h = load_raw<F32>(row_run(h, g.ldh, r, p.N, there), col);
  row.d_z = run_load16(row_run(g.d_z, g.ld_dz, r, p.N, there), col * 2);
  row.d_h = load_raw<F32>(row_run(d_h, g.ld_dh, r, p.N, there), col);
  row.y = run_load16(row_run(p.y, p.ldy, r, p.N, there), col * 2);
  if constexpr (FULL) row.gate = run_load16(row_run(p.gate, p.ld_gate, r, p.N, there), col * 2);
}

// Where the sums over the tokens go: rows of N of each of the three, one per workgroup.
struct NormSums {
  float *pre, *post, *gate;
};

// Registers: a row stays in them from its loads to its last store.  With one chunk per
// thread (AHEAD) so do the weights, and the next row is loaded while this one is worked on;
// with two there is room for neither, and an fp32 stream's rows do not fit whole: 16 registers
// of a thread (2 with a gate for every token) go through scratch memory.  2048 x 16384 with a shared
// gate: 110 us from bf16, 163 from fp32, 3.7 TB/s.
template <bool F32, bool FULL, int CH>
__global__ __launch_bounds__(1024) void norm_backward_kernel(NormProblem p, NormGradients g, NormSums sums) {
  constexpr bool AHEAD = CH == 1;
  __shared__ float2 part[2][16];
  const int waves = blockDim.x >> 6;
  const float inv_n = 1.0f / (float)p.N, inv_n_lo = __builtin_fmaf(-inv_n, (float)p.N, 1.0f) * inv_n;
  const u32x4 none = {0u, 0u, 0u, 0u};
  // sums of d_w_pre and d_w_post: four floats of a thread per entry, [2][CH][2][blockDim]
  extern __shared__ u32x4 lds_sums[];
  float s_gate[CH][8];
  if (threadIdx.x < 32) part[threadIdx.x >> 4][threadIdx.x & 15] = make_float2(0.0f, 0.0f);
  __syncthreads();
  float kept[3][8] = {};  // AHEAD: w_pre + offset, w_post + offset, a gate shared by the tokens
#pragma unroll
  for (int c = 0; c < CH; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i) s_gate[c][i] = 0.0f;
#pragma unroll
  for (int k = 0; k < 4 * CH; ++k) lds_sums[k * blockDim.x + threadIdx.x] = none;
  auto sum_at = [&](int which, int c, int half) -> u32x4& {
    return lds_sums[((which * CH + c) * 2 + half) * blockDim.x + threadIdx.x];
  };
  // adds eight terms to a sum in LDS; a thread touches its own entries only
  auto add_sum = [&](int which, int c, const float* t) {
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      u32x4 v = sum_at(which, c, half);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) + t[4 * half + i]);
      sum_at(which, c, half) = v;
    }
  };
  if constexpr (AHEAD) {
    const uint32_t col = threadIdx.x * 8;
    if (col < p.N) {
      unpack_bf16x8(load_weights(p.w_pre, col), kept[0]);
      if (p.w_post != nullptr) unpack_bf16x8(load_weights(p.w_post, col), kept[1]);
      if (!FULL && p.gate != nullptr) unpack_bf16x8(load_weights(p.gate, col), kept[2]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      kept[0][i] += p.offset;
      kept[1][i] += p.offset;
    }
  }
  // eight of w_pre + offset (which = 0), w_post + offset (1) or a shared gate (2)
  auto weights = [&](int which, int c, float* w) {
    if constexpr (AHEAD) {
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = kept[which][i];
    } else {
      const uint32_t col = (c * blockDim.x + threadIdx.x) * 8;
      const uint16_t* from = which == 0 ? p.w_pre : (which == 1 ? p.w_post : p.gate);
      unpack_bf16x8(col < p.N ? load_weights(from, col) : none, w);
      if (which < 2)
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] += p.offset;
    }
  };
  struct Row {
    GradRow<F32, FULL> c[CH];
  };
  auto load = [&](int64_t r, bool there, Row& row) {
#pragma unroll
    for (int c = 0; c < CH; ++c) load_row(p, g, r, (c * blockDim.x + threadIdx.x) * 8, there, row.c[c]);
  };
  // chunk c of the row, at the start of each phase: packed again, not unpacked values of the
  // phase before
  auto chunk_of = [&](int c, Row& row) -> GradRow<F32, FULL>& {
    GradRow<F32, FULL>& cur = row.c[c];
    for (u32x4& v : cur.h.v) keep_packed(v);
    keep_packed(cur.d_z);
    keep_packed(cur.y);
    return cur;
  };
  auto gates = [&](int c, const GradRow<F32, FULL>& cur, float* w) {
    if constexpr (FULL) unpack_bf16x8(cur.gate, w);
    else weights(2, c, w);
  };
  int turn = 0;  // of the halves of `part`: consecutive sums use different ones
  int64_t r = blockIdx.x;  // grid <= T: every workgroup has a row
  // one row; AHEAD: issue the loads of the workgroup's next one first.  The loop alternates
  // two register sets: a copy would wait for the loads in flight.
  auto work = [&](Row& row, Row& next) -> bool {
    const int64_t now = r;
    r += gridDim.x;
    const bool more = r < p.T;
    if constexpr (AHEAD) load(r, more, next);
    else load(now, true, row);
    __builtin_amdgcn_sched_barrier(0);  // those loads go out before this row is worked on
    float ss = 0.0f, dot = 0.0f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      GradRow<F32, FULL>& cur = chunk_of(c, row);
      float h[8], u[8], w[8];
      unpack_raw<F32>(cur.h, h);
      unpack_bf16x8(cur.d_z, u);
      weights(0, c, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        ss = __builtin_fmaf(h[i], h[i], ss);
        dot = __builtin_fmaf(u[i] * w[i], h[i], dot);
      }
    }
    block_sum2(ss, dot, part[turn ^= 1], waves);
    const float rh = inverse_rms(ss, inv_n, inv_n_lo, p.eps);
    const float mean = dot * rh * inv_n;  // of u hh
    float d[CH][8];                       // dh
    float ss_y = 0.0f, dot_y = 0.0f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const uint32_t col = (c * blockDim.x + threadIdx.x) * 8;
      GradRow<F32, FULL>& cur = chunk_of(c, row);
      float h[8], u[8], w[8], dx[8], t[8];
      unpack_raw<F32>(cur.h, h);
      unpack_bf16x8(cur.d_z, u);
      weights(0, c, w);
      unpack_raw<F32>(cur.d_h, d[c]);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float hh = h[i] * rh;
        t[i] = u[i] * hh;
        d[c][i] += rh * (u[i] * w[i] - hh * mean);
        dx[i] = p.residual_scale * d[c][i];
      }
      add_sum(0, c, t);
      store8<F32>(row_run(static_cast<Stream<F32>*>(g.d_x), g.ld_dx, now, p.N, true), col, dx);
      if (p.w_post != nullptr) {
        weights(1, c, w);
        unpack_bf16x8(cur.y, h);
#pragma unroll
        for (int i = 0; i < 8; ++i) u[i] = d[c][i] * w[i];
        if (p.gate != nullptr) {
          gates(c, cur, w);
#pragma unroll
          for (int i = 0; i < 8; ++i) u[i] *= w[i];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          ss_y = __builtin_fmaf(h[i], h[i], ss_y);
          dot_y = __builtin_fmaf(u[i], h[i], dot_y);
        }
      }
    }
    if (p.y == nullptr) return more;
    float ry = 1.0f, mean_y = 0.0f;
    if (p.w_post != nullptr) {
      block_sum2(ss_y, dot_y, part[turn ^= 1], waves);
      ry = inverse_rms(ss_y, inv_n, inv_n_lo, p.eps);
      mean_y = dot_y * ry * inv_n;
    }
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const uint32_t col = (c * blockDim.x + threadIdx.x) * 8;
      GradRow<F32, FULL>& cur = chunk_of(c, row);
      float y[8], w[8], gt[8], dy[8], dg[8], t[8];
      unpack_bf16x8(cur.y, y);
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = gt[i] = 1.0f;
      if (p.gate != nullptr) gates(c, cur, gt);
      if (p.w_post != nullptr) {
        weights(1, c, w);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float yh = y[i] * ry, db = d[c][i] * gt[i];
        dg[i] = d[c][i] * yh * w[i];
        if constexpr (!FULL) s_gate[c][i] += dg[i];
        if (p.w_post != nullptr) {
          t[i] = db * yh;
          dy[i] = ry * (db * w[i] - yh * mean_y);
        } else {
          dy[i] = db;
        }
      }
      if (p.w_post != nullptr) add_sum(1, c, t);
      store8<false>(row_run(g.d_y, g.ld_dy, now, p.N, true), col, dy);
      if constexpr (FULL) store8<false>(row_run(static_cast<uint16_t*>(g.d_gate), g.ld_dgate, now, p.N, true), col, dg);
    }
    return more;
  };
  Row a, b;
  if constexpr (AHEAD) load(r, true, a);
  while (work(a, b) && work(b, a)) {
  }
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const uint32_t col = (c * blockDim.x + threadIdx.x) * 8;
    if (col < p.N) {
      const int64_t row = (int64_t)blockIdx.x * p.N;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        *reinterpret_cast<u32x4*>(sums.pre + row + col + 4 * half) = sum_at(0, c, half);
        if (sums.post != nullptr) *reinterpret_cast<u32x4*>(sums.post + row + col + 4 * half) = sum_at(1, c, half);
        if (!FULL && sums.gate != nullptr)
          *reinterpret_cast<float4*>(sums.gate + row + col + 4 * half) =
              make_float4(s_gate[c][4 * half], s_gate[c][4 * half + 1], s_gate[c][4 * half + 2], s_gate[c][4 * half + 3]);
      }
    }
  }
}

// Sums of the partials of every workgroup, in a fixed order: 64 columns per workgroup of
// sixteen wavefronts, each of which adds every sixteenth row with eight loads in flight.
__global__ __launch_bounds__(1024) void norm_sums_kernel(const float* __restrict__ partials, int rows, int64_t N,
                                                         float* __restrict__ a, float* __restrict__ b,
                                                         float* __restrict__ c) {
  __shared__ float part[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t col = (int64_t)blockIdx.x * 64 + lane;
  const float* from = partials + (int64_t)blockIdx.y * rows * N + col;
  float s = 0.0f;
  if (col < N)
    for (int r0 = wave; r0 < rows; r0 += 128) {
      float v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = r0 + 16 * k < rows ? from[(int64_t)(r0 + 16 * k) * N] : 0.0f;
#pragma unroll
      for (int k = 0; k < 8; ++k) s += v[k];
    }
  part[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && col < N) {
    s = 0.0f;
#pragma unroll
    for (int k = 0; k < 16; ++k) s += part[k][lane];
    float* to = blockIdx.y == 0 ? a : (blockIdx.y == 1 ? b : c);
    to[col] = s;
  }
}

constexpr int kCUs = 256;

// Threads of a workgroup whose threads hold ch chunks each.
unsigned threads_for(int64_t N, int ch) { return (unsigned)(64 * ((N / 8 + 64 * ch - 1) / (64 * ch))); }

// Chunks per thread: rows of up to 1024 threads' one chunk, else two.
int chunks_for(int64_t N) { return N <= 8192 ? 1 : 2; }

// Workgroups of the backward pass: what a compute unit's registers hold (sixteen
// wavefronts), but at least eight rows for each past one workgroup a compute unit, as each
// writes a row of partial sums (4096 x 2048: 31.5 us with 512 workgroups, 36 with 1024 or
// 256; 65536 x 512: 103 us with 4096, 176 with 512).
int backward_blocks(const NormProblem& p) {
  const int64_t fit = (int64_t)kCUs * (1024 / threads_for(p.N, chunks_for(p.N)));
  const int64_t few = p.T < kCUs ? p.T : kCUs, eight = p.T / 8;
  const int64_t want = eight > few ? eight : few;
  return (int)(want < fit ? want : fit);
}

template <bool V>
using Bool = std::integral_constant<bool, V>;
template <int V>
using Int = std::integral_constant<int, V>;

// fn(Bool<F32>, Bool<FULL>, Int<CH>) for the types and the size of a problem.
template <typename Fn>
hipError_t by_shape(const NormProblem& p, Fn fn) {
  auto chunks = [&](auto f32, auto full) {
    return chunks_for(p.N) == 1 ? fn(f32, full, Int<1>{}) : fn(f32, full, Int<2>{});
  };
  if (p.f32) return p.ld_gate != 0 ? chunks(Bool<true>{}, Bool<true>{}) : chunks(Bool<true>{}, Bool<false>{});
  return p.ld_gate != 0 ? chunks(Bool<false>{}, Bool<true>{}) : chunks(Bool<false>{}, Bool<false>{});
}

}  // namespace

hipError_t launch_norm(const NormProblem& p, const void* x, int64_t ldx, void* h, int64_t ldh, uint16_t* z,
                       int64_t ldz, uint8_t* q, int64_t ldq, uint32_t* sf, int64_t ld_sf, hipStream_t stream) {
  return by_shape(p, [&](auto f32, auto full, auto ch) {
    using S = Stream<f32.value>;
    auto launch = [&](auto quant) {
      const unsigned threads = threads_for(p.N, ch.value);
      // sixteen wavefronts on each compute unit (8192 x 7168: 79 us with one workgroup of
      // fourteen there, 82 with two, 121 with a workgroup for every row, before the last steps;
      // 85 where each had a contiguous run of the rows).  Rounded down: rows of 4104 to 7680
      // columns have one workgroup of nine to fifteen (8192 x 5120 to codes: 56.7 us, 5.2 TB/s)
      const int64_t fit = (int64_t)kCUs * (1024 / threads);
      hipLaunchKernelGGL((norm_kernel<f32.value, full.value, quant.value, ch.value>),
                         dim3((unsigned)(p.T < fit ? p.T : fit)), dim3(threads), 0, stream, p,
                         static_cast<const S*>(x), ldx, static_cast<S*>(h), ldh, z, ldz, q, ldq, sf, ld_sf);
      return hipGetLastError();
    };
    return q != nullptr ? launch(Bool<true>{}) : launch(Bool<false>{});
  });
}

size_t norm_backward_scratch_bytes(const NormProblem& p) {
  const int blocks = backward_blocks(p);
  return blocks > 1 ? 3 * (size_t)blocks * p.N * sizeof(float) : 0;
}

hipError_t launch_norm_backward(const NormProblem& p, const NormGradients& g, float* partials, hipStream_t stream) {
  const int blocks = backward_blocks(p);
  float* const d_gate = p.gate != nullptr && p.ld_gate == 0 ? static_cast<float*>(g.d_gate) : nullptr;
  // the sums that are wanted, in order; one workgroup has no partial sums to be joined
  float* to[3] = {g.d_w_pre, nullptr, nullptr};
  int n = 1;
  if (g.d_w_post != nullptr) to[n++] = g.d_w_post;
  if (d_gate != nullptr) to[n++] = d_gate;
  NormSums sums = {g.d_w_pre, g.d_w_post, d_gate};
  if (blocks > 1) {
    const int64_t one = (int64_t)blocks * p.N;
    sums.pre = partials;
    sums.post = g.d_w_post != nullptr ? partials + one : nullptr;
    sums.gate = d_gate != nullptr ? partials + (n - 1) * one : nullptr;
  }
  hipError_t e = by_shape(p, [&](auto f32, auto full, auto ch) {
    hipLaunchKernelGGL((norm_backward_kernel<f32.value, full.value, ch.value>), dim3((unsigned)blocks),
                       dim3(threads_for(p.N, ch.value)), 4 * ch.value * 16 * threads_for(p.N, ch.value), stream, p, g,
                       sums);
    return hipGetLastError();
  });
  if (e != hipSuccess || blocks == 1) return e;
  hipLaunchKernelGGL(norm_sums_kernel, dim3((unsigned)((p.N + 63) / 64), (unsigned)n), dim3(1024), 0, stream, partials,
                     blocks, p.N, to[0], to[1], to[2]);
  return hipGetLastError();
}

}  // namespace fp8bs
