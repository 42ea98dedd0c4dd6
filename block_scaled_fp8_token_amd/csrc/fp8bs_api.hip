// C-ABI layer of the block-scaled FP8 library: argument validation, status codes,
// the per-(device, stream) split-K workspace, and dispatch to the gfx950 kernels.
// The operations and their preconditions are stated in include/fp8bs.h.
#include <hip/hip_runtime.h>

#include <climits>
#include <cstdint>
#include <cstring>
#include <map>
#include <mutex>
#include <utility>
#include <vector>

#include "../../include/fp8bs.h"
#include "block_launch.hpp"
#include "fp8bs_launch.hpp"

namespace {

thread_local int g_last_hip_error = 0;

int fail_hip(hipError_t e) {
  g_last_hip_error = (int)e;
  return FP8BS_ERR_LAUNCH;
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// gfx950 check, cached per device.
int check_device() {
  static std::mutex mu;
  static std::map<int, bool> ok;
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return fail_hip(e);
  std::lock_guard<std::mutex> lk(mu);
  auto it = ok.find(dev);
  if (it == ok.end()) {
    hipDeviceProp_t prop;
    e = hipGetDeviceProperties(&prop, dev);
    if (e != hipSuccess) return fail_hip(e);
    const bool is950 = std::strncmp(prop.gcnArchName, "gfx950", 6) == 0;
    it = ok.emplace(dev, is950).first;
  }
  return it->second ? FP8BS_OK : FP8BS_ERR_DEVICE;
}

// Fill kernel: clears the arrival counters at the front of a fresh workspace on the
// caller's stream (stream-ordered, and a kernel rather than a memset node when the
// call is being captured into a HIP graph).
__global__ __launch_bounds__(256) void zero_words_kernel(uint32_t* __restrict__ p, int64_t n) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) p[i] = 0u;
}

hipError_t zero_words(void* p, size_t bytes, hipStream_t stream) {
  const int64_t n = (int64_t)(bytes / 4);
  if (n == 0) return hipSuccess;
  hipLaunchKernelGGL(zero_words_kernel, dim3(64), dim3(256), 0, stream, static_cast<uint32_t*>(p), n);
  return hipGetLastError();
}

// Split-K workspace: one buffer per (device, stream), grown on demand.  It holds
// the per-tile arrival counters of the fused split-K reduction (zeroed once, on the
// caller's stream, when the buffer is allocated; every call leaves them at zero)
// and the fp32 partials
// of the call in flight on that stream, which every split overwrites before they
// are read.  A buffer that is outgrown is kept, never freed: a HIP graph captured
// earlier on the stream still launches kernels that use it.
// A call holds the buffer's mutex until its last launch that uses it: of two host threads
// that call on one stream, neither puts a launch between two launches of the other's call.
struct Workspace {
  std::mutex mu;
  void* ptr = nullptr;
  size_t bytes = 0;
  std::vector<void*> retired;
};

int get_workspace(size_t need, hipStream_t stream, void** out, std::unique_lock<std::mutex>* held) {
  static std::mutex mu;
  static std::map<std::pair<int, uintptr_t>, Workspace> pool;  // entries stay where they are
  *out = nullptr;
  if (need == 0) return FP8BS_OK;
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return fail_hip(e);
  std::unique_lock<std::mutex> lk(mu);
  Workspace& w = pool[std::make_pair(dev, reinterpret_cast<uintptr_t>(stream))];
  lk.unlock();  // a call on another stream does not wait for this one's launches
  *held = std::unique_lock<std::mutex>(w.mu);
  if (w.bytes >= need) {
    *out = w.ptr;
    return FP8BS_OK;
  }
  hipStreamCaptureStatus cap = hipStreamCaptureStatusNone;
  e = hipStreamIsCapturing(stream, &cap);
  if (e != hipSuccess) return fail_hip(e);
  if (cap != hipStreamCaptureStatusNone) return FP8BS_ERR_ALLOC;
  // at least double on growth, so that the retired buffers add up to less than the
  // live one
  size_t sz = need < (size_t(1) << 20) ? (size_t(1) << 20) : need;
  if (sz < 2 * w.bytes) sz = 2 * w.bytes;
  sz = (sz + (size_t(1) << 20) - 1) & ~((size_t(1) << 20) - 1);
  void* p = nullptr;
  e = hipMalloc(&p, sz);
  if (e != hipSuccess) {
    g_last_hip_error = (int)e;
    return FP8BS_ERR_ALLOC;
  }
  e = zero_words(p, fp8bs::gemm_workspace_zeroed_prefix(), stream);
  if (e != hipSuccess) {
    (void)hipFree(p);
    return fail_hip(e);
  }
  if (w.ptr) w.retired.push_back(w.ptr);  // earlier work or captured graphs may still use it
  w.ptr = p;
  w.bytes = sz;
  *out = p;
  return FP8BS_OK;
}

// Scratch of the entry point that allocates nothing: one file-scope device array
// (each GPU the library runs on holds its own copy until the process ends).  Host
// code never uses the array's name as an address: its device address comes from
// hipGetSymbolAddress, once per device, with that device current.  The arrival
// counters at its front are cleared by a fill kernel on the first call's stream;
// every call leaves them at zero.  All calls on one GPU share it, each holding the mutex until
// its last launch, as with a workspace.
constexpr size_t kStaticScratchBytes = size_t(8) << 20;
static __device__ __align__(256) unsigned char scratch[kStaticScratchBytes];

int static_scratch(hipStream_t stream, void** out, std::unique_lock<std::mutex>* held) {
  static std::mutex mu;
  static std::map<int, void*> ptrs;
  *out = nullptr;
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return fail_hip(e);
  *held = std::unique_lock<std::mutex>(mu);
  auto it = ptrs.find(dev);
  if (it == ptrs.end()) {
    void* ptr = nullptr;
    e = hipGetSymbolAddress(&ptr, HIP_SYMBOL(scratch));
    if (e != hipSuccess || ptr == nullptr) return fail_hip(e != hipSuccess ? e : hipErrorInvalidSymbol);
    e = zero_words(ptr, fp8bs::gemm_workspace_zeroed_prefix(), stream);
    if (e != hipSuccess) return fail_hip(e);
    it = ptrs.emplace(dev, ptr).first;
  }
  *out = it->second;
  return FP8BS_OK;
}

int run_gemm(const fp8bs::GemmProblem& prob, const fp8bs::GemmConfig& cfg, hipStream_t stream) {
  if (cfg.kernel < 0) return FP8BS_ERR_SHAPE;  // no table entry takes this problem
  void* ws = nullptr;
  std::unique_lock<std::mutex> held;
  const size_t need = fp8bs::gemm_workspace_bytes(prob, cfg);
  int st = get_workspace(need, stream, &ws, &held);
  if (st != FP8BS_OK) return st;
  hipError_t e = fp8bs::launch_gemm(prob, cfg, ws, stream);
  return e == hipSuccess ? FP8BS_OK : fail_hip(e);
}

int check_dense(const void* a, const uint32_t* sfa, int64_t ld_sfa, const void* b, const float* sfb,
                const void* c, int64_t ldc, int64_t M, int64_t N, int64_t K) {
  if (M < 0 || N < 0 || K < 0) return FP8BS_ERR_SHAPE;
  if (K < 128 || K % 128 != 0 || N % 64 != 0) return FP8BS_ERR_SHAPE;
  if (M == 0 || N == 0) return 1;  // no-op
  if (!a || !sfa || !b || !sfb || !c) return FP8BS_ERR_NULL;
  if (ld_sfa < M || ldc < N) return FP8BS_ERR_SHAPE;
  if (!aligned(a, 16) || !aligned(b, 16) || !aligned(c, 16) || ldc % 8 != 0) return FP8BS_ERR_ALIGN;
  if (!aligned(sfa, 4) || !aligned(sfb, 4)) return FP8BS_ERR_ALIGN;
  return FP8BS_OK;
}

int check_masked(const void* a, const uint32_t* sfa, const void* b, const float* sfb, const void* c,
                 const int32_t* masked_m, int64_t E, int64_t M_max, int64_t N, int64_t K) {
  if (E < 0 || M_max < 0 || N < 0 || K < 0) return FP8BS_ERR_SHAPE;
  if (K < 128 || K % 128 != 0 || N % 64 != 0) return FP8BS_ERR_SHAPE;
  if (E == 0 || M_max == 0 || N == 0) return 1;  // no-op
  if (!a || !sfa || !b || !sfb || !c || !masked_m) return FP8BS_ERR_NULL;
  if (!aligned(a, 16) || !aligned(b, 16) || !aligned(c, 16)) return FP8BS_ERR_ALIGN;
  if (!aligned(sfa, 4) || !aligned(sfb, 4) || !aligned(masked_m, 4)) return FP8BS_ERR_ALIGN;
  return FP8BS_OK;
}

fp8bs::GemmProblem dense_problem(const void* a, const uint32_t* sfa, int64_t ld_sfa, const void* b,
                                 const float* sfb, void* c, int64_t ldc, int64_t M, int64_t N, int64_t K) {
  fp8bs::GemmProblem p;
  p.a = static_cast<const uint8_t*>(a);
  p.sfa = sfa;
  p.b = static_cast<const uint8_t*>(b);
  p.sfb = sfb;
  p.c = static_cast<uint16_t*>(c);
  p.masked_m = nullptr;
  p.E = 1;
  p.M = M;
  p.N = N;
  p.K = K;
  p.ld_sfa = ld_sfa;
  p.ldc = ldc;
  return p;
}

fp8bs::GemmProblem masked_problem(const void* a, const uint32_t* sfa, const void* b, const float* sfb,
                                  void* c, const int32_t* masked_m, int64_t E, int64_t M_max, int64_t N,
                                  int64_t K) {
  fp8bs::GemmProblem p;
  p.a = static_cast<const uint8_t*>(a);
  p.sfa = sfa;
  p.b = static_cast<const uint8_t*>(b);
  p.sfb = sfb;
  p.c = static_cast<uint16_t*>(c);
  p.masked_m = masked_m;
  p.E = E;
  p.M = M_max;
  p.N = N;
  p.K = K;
  p.ld_sfa = M_max;
  p.ldc = N;
  return p;
}

int check_contiguous(const void* a, const uint32_t* sfa, int64_t ld_sfa, const void* b, const float* sfb,
                     const void* c, int64_t ldc, const int32_t* m_indices, int64_t E, int64_t M, int64_t N,
                     int64_t K) {
  if (E < 0) return FP8BS_ERR_SHAPE;
  const int st = check_dense(a, sfa, ld_sfa, b, sfb, c, ldc, M, N, K);
  if (st != FP8BS_OK) return st;
  if (E == 0) return 1;  // no expert: every row is padding
  if (!m_indices) return FP8BS_ERR_NULL;
  if (!aligned(m_indices, 4)) return FP8BS_ERR_ALIGN;
  return FP8BS_OK;
}

fp8bs::GemmProblem contiguous_problem(const void* a, const uint32_t* sfa, int64_t ld_sfa, const void* b,
                                      const float* sfb, void* c, int64_t ldc, const int32_t* m_indices,
                                      int64_t E, int64_t M, int64_t N, int64_t K) {
  fp8bs::GemmProblem p = dense_problem(a, sfa, ld_sfa, b, sfb, c, ldc, M, N, K);
  p.m_indices = m_indices;
  p.groups = E;
  return p;
}

// A problem of the given layout (0 dense, 1 masked, 2 contiguous) for host-side
// configuration queries only: its pointers are placeholders that are never read.
// (3: dense with float scales, 4: dense with pre-shuffled weights, 5: masked with
// pre-shuffled weights, 6: dense with float scales and pre-shuffled weights)
fp8bs::GemmProblem host_problem(int layout, int64_t M, int64_t N, int64_t K) {
  static const int32_t placeholder = 0;
  if (layout == 1 || layout == 5) {
    fp8bs::GemmProblem p = masked_problem(nullptr, nullptr, nullptr, nullptr, nullptr, &placeholder, 1, M, N, K);
    p.b_shuffled = layout == 5;
    return p;
  }
  if (layout == 2)
    return contiguous_problem(nullptr, nullptr, M, nullptr, nullptr, nullptr, N, &placeholder, 1, M, N, K);
  fp8bs::GemmProblem p = dense_problem(nullptr, nullptr, M, nullptr, nullptr, nullptr, N, M, N, K);
  p.float_scales = layout == 3 || layout == 6;
  p.b_shuffled = layout == 4 || layout == 6;
  return p;
}

// Pointers and row strides of the operators around the experts' products.  A row of
// bf16 or fp32 values is read and written 16 bytes at a time.
bool aligned_or_null(const void* p, uintptr_t a) { return p == nullptr || aligned(p, a); }
bool bad_rows(const void* p, int64_t ld, int64_t N) { return p != nullptr && ld < N; }
bool misaligned_rows(const void* p, int64_t ld) { return p != nullptr && (!aligned(p, 16) || ld % 8 != 0); }

// Tokens of one call: with it every grid is under 2^32 threads (the combine's, which has a
// workgroup for each 2048 columns of a token, as launches of at most 2^23 workgroups).
constexpr int64_t kMostRows = 1 << 22;

int check_route(int64_t ld, int64_t T, int64_t E, int32_t logits_f32, int32_t scoring, int32_t topk) {
  if (T < 0 || E < 1 || E > fp8bs::kRouteMaxE || ld < E || T > kMostRows) return FP8BS_ERR_SHAPE;
  if (topk < 1 || topk > fp8bs::kRouteMaxTopk || topk > E) return FP8BS_ERR_SHAPE;
  if ((logits_f32 != 0 && logits_f32 != 1) || (scoring != FP8BS_SIGMOID && scoring != FP8BS_SOFTMAX))
    return FP8BS_ERR_SHAPE;
  return FP8BS_OK;
}

fp8bs::RouteProblem route_problem(const void* logits, int32_t logits_f32, int64_t ld, int64_t T, int64_t E,
                                  int32_t scoring, int32_t topk, int32_t renormalize, float scale) {
  fp8bs::RouteProblem p;
  p.logits = logits;
  p.f32 = logits_f32 != 0;
  p.ld = ld;
  p.T = T;
  p.E = (int)E;
  p.topk = topk;
  p.softmax = scoring == FP8BS_SOFTMAX;
  p.renormalize = renormalize != 0;
  p.scale = scale;
  return p;
}

// Sizes of the combine and its backward pass; 1: nothing to do.
int check_combine(int64_t T, int32_t topk, int64_t E, int64_t M_max, int64_t N) {
  if (T < 0 || E < 0 || M_max < 0 || N < 0 || N % 8 != 0 || topk < 1 || topk > 64) return FP8BS_ERR_SHAPE;
  if (T > kMostRows || E > INT32_MAX || M_max > INT32_MAX || N > (1 << 20) || T * ((N + 2047) / 2048) > 4 * kMostRows)
    return FP8BS_ERR_SHAPE;
  return T == 0 || N == 0 ? 1 : FP8BS_OK;
}

// Arguments that the norm and its backward pass share.
int check_norm(int32_t residual_f32, const void* y, int64_t ldy, const void* w_post, const void* gate, int64_t ld_gate,
               const void* w_pre, int64_t T, int64_t N) {
  if (T < 0 || N < 0 || N % 8 != 0 || N > fp8bs::kNormMaxN || (residual_f32 != 0 && residual_f32 != 1))
    return FP8BS_ERR_SHAPE;
  if (N == 0) return 1;
  if (!w_pre || ((w_post || gate) && !y)) return FP8BS_ERR_NULL;
  if (bad_rows(y, ldy, N) || (gate && ld_gate != 0 && ld_gate < N)) return FP8BS_ERR_SHAPE;
  if (misaligned_rows(y, ldy) || misaligned_rows(gate, ld_gate) || !aligned(w_pre, 16) || !aligned_or_null(w_post, 16))
    return FP8BS_ERR_ALIGN;
  return FP8BS_OK;
}

fp8bs::NormProblem norm_problem(int32_t residual_f32, const void* y, int64_t ldy, const void* w_post, const void* gate,
                                int64_t ld_gate, const void* w_pre, float residual_scale, float eps, float offset,
                                int64_t T, int64_t N) {
  fp8bs::NormProblem p;
  if (gate == nullptr) ld_gate = 0;  // ld_gate != 0 means a gate row per token
  p.f32 = residual_f32 != 0;
  p.T = T;
  p.N = N;
  p.y = static_cast<const uint16_t*>(y);
  p.ldy = ldy;
  p.w_post = static_cast<const uint16_t*>(w_post);
  p.gate = static_cast<const uint16_t*>(gate);
  p.ld_gate = ld_gate;
  p.w_pre = static_cast<const uint16_t*>(w_pre);
  p.residual_scale = residual_scale;
  p.eps = eps;
  p.offset = offset;
  return p;
}

// The norm's backward pass with its partial sums in `scratch` (given), or else in the stream's
// workspace.
int run_norm_backward(bool given, void* scratch, int64_t scratch_bytes, const void* d_z, int64_t ld_dz, const void* d_h,
                      int64_t ld_dh, const void* h, int64_t ldh, int32_t residual_f32, const void* y, int64_t ldy,
                      const void* w_post, const void* gate, int64_t ld_gate, const void* w_pre, float residual_scale,
                      float eps, float weight_offset, int64_t T, int64_t N, void* d_x, int64_t ld_dx, void* d_y,
                      int64_t ld_dy, float* d_w_pre, float* d_w_post, void* d_gate, int64_t ld_dgate, void* stream) {
  if (T < 0 || N < 0 || N % 8 != 0 || N > fp8bs::kNormMaxN) return FP8BS_ERR_SHAPE;
  if (T == 0) {
    if (N == 0) return FP8BS_OK;
    if (!d_w_pre) return FP8BS_ERR_NULL;
    int st = check_device();
    if (st != FP8BS_OK) return st;
    float* sums[3] = {d_w_pre, d_w_post, ld_gate == 0 ? static_cast<float*>(d_gate) : nullptr};
    for (float* s : sums) {
      if (s == nullptr) continue;
      if (!aligned(s, 16)) return FP8BS_ERR_ALIGN;
      hipError_t e = zero_words(s, (size_t)N * sizeof(float), static_cast<hipStream_t>(stream));
      if (e != hipSuccess) return fail_hip(e);
    }
    return FP8BS_OK;
  }
  int st = check_norm(residual_f32, y, ldy, w_post, gate, ld_gate, w_pre, T, N);
  if (st != FP8BS_OK) return st > 0 ? FP8BS_OK : st;
  if (!d_z || !h || !d_x || !d_w_pre || !y != !d_y || !w_post != !d_w_post || !gate != !d_gate) return FP8BS_ERR_NULL;
  if (ld_dz < N || bad_rows(d_h, ld_dh, N) || ldh < N || ld_dx < N || bad_rows(d_y, ld_dy, N) ||
      (gate && ld_gate != 0 && ld_dgate < N))
    return FP8BS_ERR_SHAPE;
  if (misaligned_rows(d_z, ld_dz) || misaligned_rows(d_h, ld_dh) || misaligned_rows(h, ldh) ||
      misaligned_rows(d_x, ld_dx) || misaligned_rows(d_y, ld_dy) || !aligned(d_w_pre, 16) ||
      !aligned_or_null(d_w_post, 16) || !aligned_or_null(d_gate, 16) || (gate && ld_gate != 0 && ld_dgate % 8 != 0))
    return FP8BS_ERR_ALIGN;
  const fp8bs::NormProblem p = norm_problem(residual_f32, y, ldy, w_post, gate, ld_gate, w_pre, residual_scale, eps,
                                            weight_offset, T, N);
  const size_t sums = fp8bs::norm_backward_scratch_bytes(p);
  if (given && sums > 0) {
    if (!scratch) return FP8BS_ERR_NULL;
    if (!aligned(scratch, 16)) return FP8BS_ERR_ALIGN;
    if (scratch_bytes < (int64_t)sums) return FP8BS_ERR_SCRATCH;
  }
  st = check_device();
  if (st != FP8BS_OK) return st;
  const fp8bs::NormGradients g = {static_cast<const uint16_t*>(d_z), ld_dz, d_h, ld_dh, h, ldh, d_x, ld_dx,
                                  static_cast<uint16_t*>(d_y), ld_dy, d_w_pre, d_w_post, d_gate, ld_dgate};
  std::unique_lock<std::mutex> held;
  if (!given && sums > 0) {  // past the split-K arrival counters
    const size_t off = fp8bs::gemm_workspace_zeroed_prefix();
    void* ws = nullptr;
    st = get_workspace(off + sums, static_cast<hipStream_t>(stream), &ws, &held);
    if (st != FP8BS_OK) return st;
    scratch = static_cast<char*>(ws) + off;
  }
  hipError_t e = fp8bs::launch_norm_backward(p, g, static_cast<float*>(scratch), static_cast<hipStream_t>(stream));
  return e == hipSuccess ? FP8BS_OK : fail_hip(e);
}

int check_checkpoint(int64_t E, int64_t M_max, int64_t H) {
  if (E < 0 || E > fp8bs::kCheckpointMaxE || M_max < 0 || H < 0 || H % 128 != 0) return FP8BS_ERR_SHAPE;
  if (M_max > INT32_MAX || E * M_max > INT32_MAX || H > (1 << 28)) return FP8BS_ERR_SHAPE;
  return E == 0 || M_max == 0 || H == 0 ? 1 : FP8BS_OK;
}

}  // namespace

extern "C" {

int fp8_quant_group_pack(const void* x, int64_t ldx, int64_t M, int64_t K, void* q, int64_t ldq,
                         uint32_t* sf, int64_t ld_sf, void* stream) {
  if (M < 0 || K < 0 || K % 128 != 0) return FP8BS_ERR_SHAPE;
  if (M == 0 || K == 0) return FP8BS_OK;
  if (!x || !q || !sf) return FP8BS_ERR_NULL;
  if (ldx < K || ldq < K || ld_sf < M) return FP8BS_ERR_SHAPE;
  if (!aligned(x, 16) || !aligned(q, 16) || ldx % 8 != 0 || ldq % 16 != 0 || !aligned(sf, 4))
    return FP8BS_ERR_ALIGN;
  int st = check_device();
  if (st != FP8BS_OK) return st;
  hipError_t e = fp8bs::launch_quant_group_pack(static_cast<const uint16_t*>(x), ldx, M, K,
                                                static_cast<uint8_t*>(q), ldq, sf, ld_sf,
                                                static_cast<hipStream_t>(stream));
  return e == hipSuccess ? FP8BS_OK : fail_hip(e);
}

int silu_mul_quant_group_pack(const void* x, const int32_t* masked_m, int64_t E, int64_t M_max, int64_t H,
                              void* q, uint32_t* sf, void* stream) {
  if (E < 0 || M_max < 0 || H < 0 || H % 128 != 0) return FP8BS_ERR_SHAPE;
  if (E == 0 || M_max == 0 || H == 0) return FP8BS_OK;
  if (!x || !masked_m || !q || !sf) return FP8BS_ERR_NULL;
  if (!aligned(x, 16) || !aligned(q, 16) || !aligned(sf, 4) || !aligned(masked_m, 4)) return FP8BS_ERR_ALIGN;
  int st = check_device();
  if (st != FP8BS_OK) return st;
  hipError_t e = fp8bs::launch_silu_mul_quant(static_cast<const uint16_t*>(x), masked_m, E, M_max, H,
                                              static_cast<uint8_t*>(q), sf, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? FP8BS_OK : fail_hip(e);
}

int fp8_quant_group_float(const void* x, int64_t ldx, int64_t M, int64_t K, void* q, int64_t ldq, float* sf,
                          int64_t ld_sf, void* stream) {
  if (M < 0 || K < 0 || K % 128 != 0) return FP8BS_ERR_SHAPE;
  if (M == 0 || K == 0) return FP8BS_OK;
  if (!x || !q || !sf) return FP8BS_ERR_NULL;
  if (ldx < K || ldq < K || ld_sf < M) return FP8BS_ERR_SHAPE;
  if (!aligned(x, 16) || !aligned(q, 16) || ldx % 8 != 0 || ldq % 16 != 0 || !aligned(sf, 4))
    return FP8BS_ERR_ALIGN;
  int st = check_device();
  if (st != FP8BS_OK) return st;
  hipError_t e = fp8bs::launch_quant_group_float(static_cast<const uint16_t*>(x), ldx, M, K,
                                                 static_cast<uint8_t*>(q), ldq, sf, ld_sf,
                                                 static_cast<hipStream_t>(stream));
  return e == hipSuccess ? FP8BS_OK : fail_hip(e);
}

int fp8_block_quant_128x128_float(const void* w, int64_t N, int64_t K, void* q, float* sfb, void* stream) {
  if (N < 0 || K < 0 || K % 128 != 0) return FP8BS_ERR_SHAPE;
  if (N == 0 || K == 0) return FP8BS_OK;
  if (!w || !q || !sfb) return FP8BS_ERR_NULL;
  if (!aligned(w, 16) || !aligned(q, 16) || !aligned(sfb, 4)) return FP8BS_ERR_ALIGN;
  int st = check_device();
  if (st != FP8BS_OK) return st;
  hipError_t e = fp8bs::launch_block_quant_float(static_cast<const uint16_t*>(w), N, K,
                                                 static_cast<uint8_t*>(q), sfb, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? FP8BS_OK : fail_hip(e);
}

int fp8_quant_group_pack_to_experts(const void* x, int64_t ldx, int64_t T, int64_t K, const int32_t* topk_ids,
                                    int32_t topk, int64_t E, int64_t M_max, void* q, uint32_t* sf,
                                    int32_t* masked_m, int32_t* slot_of, void* stream) {
  if (T < 0 || K < 0 || K % 128 != 0 || E < 0 || M_max < 0) return FP8BS_ERR_SHAPE;
  if (topk < 1 || topk > 64 || E > fp8bs::kQuantToExpertsMaxExperts || T * (int64_t)topk > INT32_MAX)
    return FP8BS_ERR_SHAPE;
  if (E == 0) return FP8BS_OK;
  if (!masked_m || (T > 0 && (!x || !topk_ids || !slot_of)) || (M_max > 0 && K > 0 && (!q || !sf)))
    return FP8BS_ERR_NULL;
  if (T > 0 && ldx < K) return FP8BS_ERR_SHAPE;
  if ((x && !aligned(x, 16)) || (q && !aligned(q, 16)) || ldx % 8 != 0 || (sf && !aligned(sf, 4)) ||
      !aligned(masked_m, 4) || (topk_ids && !aligned(topk_ids, 4)) || (slot_of && !aligned(slot_of, 4)))
    return FP8BS_ERR_ALIGN;
  int st = check_device();
  if (st != FP8BS_OK) return st;
  // pair ranks and per-chunk counts live in the stream's workspace past the counters
  const size_t off = fp8bs::gemm_workspace_zeroed_prefix();
  void* ws = nullptr;
  std::unique_lock<std::mutex> held;
  st = get_workspace(off + fp8bs::quant_to_experts_scratch_bytes(T, topk, E), static_cast<hipStream_t>(stream),
                     &ws, &held);
  if (st != FP8BS_OK) return st;
  hipError_t e = fp8bs::launch_quant_to_experts(static_cast<const uint16_t*>(x), ldx, T, K, topk_ids, topk, E,
                                                M_max, static_cast<uint8_t*>(q), sf, masked_m, slot_of,
                                                reinterpret_cast<int32_t*>(static_cast<char*>(ws) + off),
                                                static_cast<hipStream_t>(stream));
  return e == hipSuccess ? FP8BS_OK : fail_hip(e);
}

int fp8_block_quant_128x128(const void* w, int64_t N, int64_t K, void* q, float* sfb, void* stream) {
  if (N < 0 || K < 0 || K % 128 != 0) return FP8BS_ERR_SHAPE;
  if (N == 0 || K == 0) return FP8BS_OK;
  if (!w || !q || !sfb) return FP8BS_ERR_NULL;
  if (!aligned(w, 16) || !aligned(q, 16) || !aligned(sfb, 4)) return FP8BS_ERR_ALIGN;
  int st = check_device();
  if (st != FP8BS_OK) return st;
  hipError_t e = fp8bs::launch_block_quant(static_cast<const uint16_t*>(w), N, K, static_cast<uint8_t*>(q),
                                           sfb, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? FP8BS_OK : fail_hip(e);
}

int fp8_block_gemm_nt(const void* a, const uint32_t* sfa, int64_t ld_sfa, const void* b, const float* sfb,
                      void* c, int64_t ldc, int64_t M, int64_t N, int64_t K, void* stream) {
  int st = check_dense(a, sfa, ld_sfa, b, sfb, c, ldc, M, N, K);
  if (st != FP8BS_OK) return st > 0 ? FP8BS_OK : st;
  st = check_device();
  if (st != FP8BS_OK) return st;
  const fp8bs::GemmProblem p = dense_problem(a, sfa, ld_sfa, b, sfb, c, ldc, M, N, K);
  return run_gemm(p, fp8bs::choose_gemm_config(p), static_cast<hipStream_t>(stream));
}

int fp8_block_gemm_nt_cfg(const void* a, const uint32_t* sfa, int64_t ld_sfa, const void* b, const float* sfb,
                          void* c, int64_t ldc, int64_t M, int64_t N, int64_t K, int32_t kernel, int32_t splits,
                          void* stream) {
  int st = check_dense(a, sfa, ld_sfa, b, sfb, c, ldc, M, N, K);
  if (st != FP8BS_OK) return st > 0 ? FP8BS_OK : st;
  st = check_device();
  if (st != FP8BS_OK) return st;
  const fp8bs::GemmProblem p = dense_problem(a, sfa, ld_sfa, b, sfb, c, ldc, M, N, K);
  fp8bs::GemmConfig cfg;
  if (!fp8bs::gemm_config_by_index(kernel, p, splits < 1 ? 1 : splits, &cfg)) return FP8BS_ERR_SHAPE;
  return run_gemm(p, cfg, static_cast<hipStream_t>(stream));
}

int fp8_weight_preshuffle(const void* w, int64_t rows, int64_t K, void* out, void* stream) {
  if (rows < 0 || K < 0 || rows % 32 != 0 || K % 128 != 0) return FP8BS_ERR_SHAPE;
  if (rows == 0 || K == 0) return FP8BS_OK;
  if (!w || !out) return FP8BS_ERR_NULL;
  if (!aligned(w, 16) || !aligned(out, 16)) return FP8BS_ERR_ALIGN;
  int st = check_device();
  if (st != FP8BS_OK) return st;
  hipError_t e = fp8bs::launch_weight_preshuffle(static_cast<const uint8_t*>(w), rows, K, static_cast<uint8_t*>(out),
                                                 static_cast<hipStream_t>(stream));
  return e == hipSuccess ? FP8BS_OK : fail_hip(e);
}

int fp8_block_gemm_nt_preshuffled(const void* a, const uint32_t* sfa, int64_t ld_sfa, const void* b,
                                  const float* sfb, void* c, int64_t ldc, int64_t M, int64_t N, int64_t K,
                                  void* stream) {
  int st = check_dense(a, sfa, ld_sfa, b, sfb, c, ldc, M, N, K);
  if (st != FP8BS_OK) return st > 0 ? FP8BS_OK : st;
  st = check_device();
  if (st != FP8BS_OK) return st;
  fp8bs::GemmProblem p = dense_problem(a, sfa, ld_sfa, b, sfb, c, ldc, M, N, K);
  p.b_shuffled = true;
  const fp8bs::GemmConfig cfg = fp8bs::choose_gemm_config(p);
  if (cfg.kernel < 0) return FP8BS_ERR_SHAPE;
  return run_gemm(p, cfg, static_cast<hipStream_t>(stream));
}

int fp8_block_gemm_nt_preshuffled_noalloc(const void* a, const uint32_t* sfa, int64_t ld_sfa, const void* b,
                                          const float* sfb, void* c, int64_t ldc, int64_t M, int64_t N, int64_t K,
                                          void* stream) {
  int st = check_dense(a, sfa, ld_sfa, b, sfb, c, ldc, M, N, K);
  if (st != FP8BS_OK) return st > 0 ? FP8BS_OK : st;
  st = check_device();
  if (st != FP8BS_OK) return st;
  fp8bs::GemmProblem p = dense_problem(a, sfa, ld_sfa, b, sfb, c, ldc, M, N, K);
  p.b_shuffled = true;
  const fp8bs::GemmConfig cfg = fp8bs::choose_gemm_config(p);
  if (cfg.kernel < 0) return FP8BS_ERR_SHAPE;
  const size_t need = fp8bs::gemm_workspace_bytes(p, cfg);
  if (need > kStaticScratchBytes) return FP8BS_ERR_SCRATCH;
  void* ws = nullptr;
  std::unique_lock<std::mutex> held;
  if (need > 0) {
    st = static_scratch(static_cast<hipStream_t>(stream), &ws, &held);
    if (st != FP8BS_OK) return st;
  }
  hipError_t e = fp8bs::launch_gemm(p, cfg, ws, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? FP8BS_OK : fail_hip(e);
}

int fp8_block_gemm_nt_preshuffled_cfg(const void* a, const uint32_t* sfa, int64_t ld_sfa, const void* b,
                                      const float* sfb, void* c, int64_t ldc, int64_t M, int64_t N, int64_t K,
                                      int32_t kernel, int32_t splits, void* stream) {
  int st = check_dense(a, sfa, ld_sfa, b, sfb, c, ldc, M, N, K);
  if (st != FP8BS_OK) return st > 0 ? FP8BS_OK : st;
  st = check_device();
  if (st != FP8BS_OK) return st;
  fp8bs::GemmProblem p = dense_problem(a, sfa, ld_sfa, b, sfb, c, ldc, M, N, K);
  p.b_shuffled = true;
  fp8bs::GemmConfig cfg;
  if (!fp8bs::gemm_config_by_index(kernel, p, splits < 1 ? 1 : splits, &cfg)) return FP8BS_ERR_SHAPE;
  return run_gemm(p, cfg, static_cast<hipStream_t>(stream));
}

int fp8_block_gemm_grouped_masked_preshuffled(const void* a, const uint32_t* sfa, const void* b, const float* sfb,
                                              void* c, const int32_t* masked_m, int64_t E, int64_t M_max, int64_t N,
                                              int64_t K, void* stream) {
  int st = check_masked(a, sfa, b, sfb, c, masked_m, E, M_max, N, K);
  if (st != FP8BS_OK) return st > 0 ? FP8BS_OK : st;
  st = check_device();
  if (st != FP8BS_OK) return st;
  fp8bs::GemmProblem p = masked_problem(a, sfa, b, sfb, c, masked_m, E, M_max, N, K);
  p.b_shuffled = true;
  const fp8bs::GemmConfig cfg = fp8bs::choose_gemm_config(p);
  if (cfg.kernel < 0) return FP8BS_ERR_SHAPE;
  return run_gemm(p, cfg, static_cast<hipStream_t>(stream));
}

int fp8_block_gemm_grouped_masked_preshuffled_cfg(const void* a, const uint32_t* sfa, const void* b,
                                                  const float* sfb, void* c, const int32_t* masked_m, int64_t E,
                                                  int64_t M_max, int64_t N, int64_t K, int32_t kernel,
                                                  void* stream) {
  int st = check_masked(a, sfa, b, sfb, c, masked_m, E, M_max, N, K);
  if (st != FP8BS_OK) return st > 0 ? FP8BS_OK : st;
  st = check_device();
  if (st != FP8BS_OK) return st;
  fp8bs::GemmProblem p = masked_problem(a, sfa, b, sfb, c, masked_m, E, M_max, N, K);
  p.b_shuffled = true;
  fp8bs::GemmConfig cfg;
  if (!fp8bs::gemm_config_by_index(kernel, p, 1, &cfg)) return FP8BS_ERR_SHAPE;
  return run_gemm(p, cfg, static_cast<hipStream_t>(stream));
}

int fp8_block_gemm_grouped_masked(const void* a, const uint32_t* sfa, const void* b, const float* sfb, void* c,
                                  const int32_t* masked_m, int64_t E, int64_t M_max, int64_t N, int64_t K,
                                  void* stream) {
  int st = check_masked(a, sfa, b, sfb, c, masked_m, E, M_max, N, K);
  if (st != FP8BS_OK) return st > 0 ? FP8BS_OK : st;
  st = check_device();
  if (st != FP8BS_OK) return st;
  const fp8bs::GemmProblem p = masked_problem(a, sfa, b, sfb, c, masked_m, E, M_max, N, K);
  return run_gemm(p, fp8bs::choose_gemm_config(p), static_cast<hipStream_t>(stream));
}

int fp8_block_gemm_grouped_masked_cfg(const void* a, const uint32_t* sfa, const void* b, const float* sfb,
                                      void* c, const int32_t* masked_m, int64_t E, int64_t M_max, int64_t N,
                                      int64_t K, int32_t kernel, void* stream) {
  int st = check_masked(a, sfa, b, sfb, c, masked_m, E, M_max, N, K);
  if (st != FP8BS_OK) return st > 0 ? FP8BS_OK : st;
  st = check_device();
  if (st != FP8BS_OK) return st;
  const fp8bs::GemmProblem p = masked_problem(a, sfa, b, sfb, c, masked_m, E, M_max, N, K);
  fp8bs::GemmConfig cfg;
  if (!fp8bs::gemm_config_by_index(kernel, p, 1, &cfg)) return FP8BS_ERR_SHAPE;
  return run_gemm(p, cfg, static_cast<hipStream_t>(stream));
}

int fp8_block_gemm_grouped_contiguous(const void* a, const uint32_t* sfa, int64_t ld_sfa, const void* b,
                                      const float* sfb, void* c, int64_t ldc, const int32_t* m_indices, int64_t E,
                                      int64_t M, int64_t N, int64_t K, void* stream) {
  int st = check_contiguous(a, sfa, ld_sfa, b, sfb, c, ldc, m_indices, E, M, N, K);
  if (st != FP8BS_OK) return st > 0 ? FP8BS_OK : st;
  st = check_device();
  if (st != FP8BS_OK) return st;
  const fp8bs::GemmProblem p = contiguous_problem(a, sfa, ld_sfa, b, sfb, c, ldc, m_indices, E, M, N, K);
  return run_gemm(p, fp8bs::choose_gemm_config(p), static_cast<hipStream_t>(stream));
}

int fp8_block_gemm_grouped_contiguous_cfg(const void* a, const uint32_t* sfa, int64_t ld_sfa, const void* b,
                                          const float* sfb, void* c, int64_t ldc, const int32_t* m_indices,
                                          int64_t E, int64_t M, int64_t N, int64_t K, int32_t kernel,
                                          void* stream) {
  int st = check_contiguous(a, sfa, ld_sfa, b, sfb, c, ldc, m_indices, E, M, N, K);
  if (st != FP8BS_OK) return st > 0 ? FP8BS_OK : st;
  st = check_device();
  if (st != FP8BS_OK) return st;
  const fp8bs::GemmProblem p = contiguous_problem(a, sfa, ld_sfa, b, sfb, c, ldc, m_indices, E, M, N, K);
  fp8bs::GemmConfig cfg;
  if (!fp8bs::gemm_config_by_index(kernel, p, 1, &cfg)) return FP8BS_ERR_SHAPE;
  return run_gemm(p, cfg, static_cast<hipStream_t>(stream));
}

int fp8_block_gemm_nt_float_scales(const void* a, const float* sfa, int64_t ld_sfa, const void* b, const float* sfb,
                                   void* c, int64_t ldc, int64_t M, int64_t N, int64_t K, void* stream) {
  int st = check_dense(a, reinterpret_cast<const uint32_t*>(sfa), ld_sfa, b, sfb, c, ldc, M, N, K);
  if (st != FP8BS_OK) return st > 0 ? FP8BS_OK : st;
  st = check_device();
  if (st != FP8BS_OK) return st;
  fp8bs::GemmProblem p = dense_problem(a, reinterpret_cast<const uint32_t*>(sfa), ld_sfa, b, sfb, c, ldc, M, N, K);
  p.float_scales = true;
  return run_gemm(p, fp8bs::choose_gemm_config(p), static_cast<hipStream_t>(stream));
}

int fp8_block_gemm_nt_float_scales_cfg(const void* a, const float* sfa, int64_t ld_sfa, const void* b,
                                       const float* sfb, void* c, int64_t ldc, int64_t M, int64_t N, int64_t K,
                                       int32_t kernel, int32_t splits, void* stream) {
  int st = check_dense(a, reinterpret_cast<const uint32_t*>(sfa), ld_sfa, b, sfb, c, ldc, M, N, K);
  if (st != FP8BS_OK) return st > 0 ? FP8BS_OK : st;
  st = check_device();
  if (st != FP8BS_OK) return st;
  fp8bs::GemmProblem p = dense_problem(a, reinterpret_cast<const uint32_t*>(sfa), ld_sfa, b, sfb, c, ldc, M, N, K);
  p.float_scales = true;
  fp8bs::GemmConfig cfg;
  if (!fp8bs::gemm_config_by_index(kernel, p, splits < 1 ? 1 : splits, &cfg)) return FP8BS_ERR_SHAPE;
  return run_gemm(p, cfg, static_cast<hipStream_t>(stream));
}

int fp8_block_gemm_nt_float_scales_preshuffled(const void* a, const float* sfa, int64_t ld_sfa, const void* b,
                                                const float* sfb, void* c, int64_t ldc, int64_t M, int64_t N,
                                                int64_t K, void* stream) {
  int st = check_dense(a, reinterpret_cast<const uint32_t*>(sfa), ld_sfa, b, sfb, c, ldc, M, N, K);
  if (st != FP8BS_OK) return st > 0 ? FP8BS_OK : st;
  st = check_device();
  if (st != FP8BS_OK) return st;
  fp8bs::GemmProblem p = dense_problem(a, reinterpret_cast<const uint32_t*>(sfa), ld_sfa, b, sfb, c, ldc, M, N, K);
  p.float_scales = true;
  p.b_shuffled = true;
  const fp8bs::GemmConfig cfg = fp8bs::choose_gemm_config(p);
  if (cfg.kernel < 0) return FP8BS_ERR_SHAPE;
  return run_gemm(p, cfg, static_cast<hipStream_t>(stream));
}

int fp8_block_gemm_nt_float_scales_preshuffled_cfg(const void* a, const float* sfa, int64_t ld_sfa, const void* b,
                                                    const float* sfb, void* c, int64_t ldc, int64_t M, int64_t N,
                                                    int64_t K, int32_t kernel, int32_t splits, void* stream) {
  int st = check_dense(a, reinterpret_cast<const uint32_t*>(sfa), ld_sfa, b, sfb, c, ldc, M, N, K);
  if (st != FP8BS_OK) return st > 0 ? FP8BS_OK : st;
  st = check_device();
  if (st != FP8BS_OK) return st;
  fp8bs::GemmProblem p = dense_problem(a, reinterpret_cast<const uint32_t*>(sfa), ld_sfa, b, sfb, c, ldc, M, N, K);
  p.float_scales = true;
  p.b_shuffled = true;
  fp8bs::GemmConfig cfg;
  if (!fp8bs::gemm_config_by_index(kernel, p, splits < 1 ? 1 : splits, &cfg)) return FP8BS_ERR_SHAPE;
  return run_gemm(p, cfg, static_cast<hipStream_t>(stream));
}

int moe_route_topk(const void* logits, int32_t logits_f32, int64_t ld, int64_t T, int64_t E, const float* bias,
                   int32_t scoring, int32_t groups, int32_t topk_groups, int32_t group_top, int32_t topk,
                   int32_t renormalize, float scale, int32_t* topk_ids, float* weights, void* stream) {
  int st = check_route(ld, T, E, logits_f32, scoring, topk);
  if (st != FP8BS_OK) return st;
  if (groups < 1 || groups > 64 || E % groups != 0 || topk_groups < 1 || topk_groups > groups) return FP8BS_ERR_SHAPE;
  if (topk > topk_groups * (E / groups) || group_top < 1 || group_top > 2 || group_top > E / groups)
    return FP8BS_ERR_SHAPE;
  if (T == 0) return FP8BS_OK;
  if (!logits || !topk_ids || !weights) return FP8BS_ERR_NULL;
  if (!aligned(logits, logits_f32 ? 4 : 2) || !aligned_or_null(bias, 4) || !aligned(topk_ids, 4) ||
      !aligned(weights, 4))
    return FP8BS_ERR_ALIGN;
  st = check_device();
  if (st != FP8BS_OK) return st;
  const fp8bs::RouteProblem p = route_problem(logits, logits_f32, ld, T, E, scoring, topk, renormalize, scale);
  hipError_t e = fp8bs::launch_route(p, bias, groups, topk_groups, group_top, topk_ids, weights,
                                     static_cast<hipStream_t>(stream));
  return e == hipSuccess ? FP8BS_OK : fail_hip(e);
}

int moe_route_topk_backward(const void* logits, int32_t logits_f32, int64_t ld, int64_t T, int64_t E,
                            const int32_t* topk_ids, const float* d_weights, int32_t scoring, int32_t topk,
                            int32_t renormalize, float scale, void* d_logits, int64_t ld_d, void* stream) {
  int st = check_route(ld, T, E, logits_f32, scoring, topk);
  if (st != FP8BS_OK) return st;
  if (ld_d < E) return FP8BS_ERR_SHAPE;
  if (T == 0) return FP8BS_OK;
  if (!logits || !topk_ids || !d_weights || !d_logits) return FP8BS_ERR_NULL;
  if (!aligned(logits, logits_f32 ? 4 : 2) || !aligned(d_logits, logits_f32 ? 4 : 2) || !aligned(topk_ids, 4) ||
      !aligned(d_weights, 4))
    return FP8BS_ERR_ALIGN;
  st = check_device();
  if (st != FP8BS_OK) return st;
  const fp8bs::RouteProblem p = route_problem(logits, logits_f32, ld, T, E, scoring, topk, renormalize, scale);
  hipError_t e =
      fp8bs::launch_route_backward(p, topk_ids, d_weights, d_logits, ld_d, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? FP8BS_OK : fail_hip(e);
}

int moe_combine(const void* y, const int32_t* topk_ids, const int32_t* slot_of, const float* weights, const void* base,
                int64_t ld_base, int64_t T, int32_t topk, int64_t E, int64_t M_max, int64_t N, void* out,
                int64_t ld_out, void* stream) {
  int st = check_combine(T, topk, E, M_max, N);
  if (st != FP8BS_OK) return st > 0 ? FP8BS_OK : st;
  if (!topk_ids || !slot_of || !out || (!y && E > 0 && M_max > 0)) return FP8BS_ERR_NULL;
  if (bad_rows(base, ld_base, N) || ld_out < N) return FP8BS_ERR_SHAPE;
  if (!aligned_or_null(y, 16) || misaligned_rows(base, ld_base) || misaligned_rows(out, ld_out) ||
      !aligned(topk_ids, 4) || !aligned(slot_of, 4) || !aligned_or_null(weights, 4))
    return FP8BS_ERR_ALIGN;
  st = check_device();
  if (st != FP8BS_OK) return st;
  const fp8bs::CombineProblem p = {topk_ids, slot_of, weights, T, E, M_max, N, topk};
  hipError_t e = fp8bs::launch_combine(p, static_cast<const uint16_t*>(y), static_cast<const uint16_t*>(base), ld_base,
                                       static_cast<uint16_t*>(out), ld_out, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? FP8BS_OK : fail_hip(e);
}

int moe_combine_backward(const void* d_out, int64_t ld_d, const void* y, const int32_t* topk_ids,
                         const int32_t* slot_of, const float* weights, int64_t T, int32_t topk, int64_t E,
                         int64_t M_max, int64_t N, void* d_y, void* q, uint32_t* sf, float* d_weights, void* stream) {
  int st = check_combine(T, topk, E, M_max, N);
  if (st < 0) return st;
  if (st > 0) {
    if (T == 0 || d_weights == nullptr) return FP8BS_OK;
    // no columns: the weights' gradients are sums of nothing
    if (!aligned(d_weights, 4)) return FP8BS_ERR_ALIGN;
    st = check_device();
    if (st != FP8BS_OK) return st;
    hipError_t e = zero_words(d_weights, (size_t)T * topk * sizeof(float), static_cast<hipStream_t>(stream));
    return e == hipSuccess ? FP8BS_OK : fail_hip(e);
  }
  const bool rows = E > 0 && M_max > 0;  // a layout without rows has no pointers
  if (!d_out || !topk_ids || !slot_of || (rows && (!d_y == !q || !q != !sf || (d_weights && !y)))) return FP8BS_ERR_NULL;
  if (ld_d < N || (q && N % 128 != 0)) return FP8BS_ERR_SHAPE;
  if (misaligned_rows(d_out, ld_d) || !aligned_or_null(y, 16) || !aligned_or_null(d_y, 16) || !aligned_or_null(q, 16) ||
      !aligned_or_null(sf, 4) || !aligned(topk_ids, 4) || !aligned(slot_of, 4) || !aligned_or_null(weights, 4) ||
      !aligned_or_null(d_weights, 4))
    return FP8BS_ERR_ALIGN;
  st = check_device();
  if (st != FP8BS_OK) return st;
  const fp8bs::CombineProblem p = {topk_ids, slot_of, weights, T, E, M_max, N, topk};
  hipError_t e = fp8bs::launch_combine_backward(p, static_cast<const uint16_t*>(d_out), ld_d,
                                                static_cast<const uint16_t*>(y), static_cast<uint16_t*>(d_y),
                                                static_cast<uint8_t*>(q), sf, d_weights,
                                                static_cast<hipStream_t>(stream));
  return e == hipSuccess ? FP8BS_OK : fail_hip(e);
}

int residual_rms_norm(const void* x, int64_t ldx, int32_t residual_f32, const void* y, int64_t ldy, const void* w_post,
                      const void* gate, int64_t ld_gate, const void* w_pre, float residual_scale, float eps,
                      float weight_offset, int64_t T, int64_t N, void* h, int64_t ldh, void* z, int64_t ldz, void* q,
                      int64_t ldq, uint32_t* sf, int64_t ld_sf, void* stream) {
  if (T == 0 && N >= 0) y = w_post = gate = nullptr;  // no rows: their pointers are not looked at
  int st = check_norm(residual_f32, y, ldy, w_post, gate, ld_gate, w_pre, T, N);
  if (st != FP8BS_OK) return st > 0 ? FP8BS_OK : st;
  if (q && N % 128 != 0) return FP8BS_ERR_SHAPE;
  if (T == 0) return FP8BS_OK;
  if (!x || !q != !sf || (!h && !z && !q)) return FP8BS_ERR_NULL;
  if (ldx < N || bad_rows(h, ldh, N) || bad_rows(z, ldz, N) || bad_rows(q, ldq, N) || (sf && ld_sf < T))
    return FP8BS_ERR_SHAPE;
  if (misaligned_rows(x, ldx) || misaligned_rows(h, ldh) || misaligned_rows(z, ldz) || misaligned_rows(q, ldq) ||
      (q && ldq % 16 != 0) || !aligned_or_null(sf, 4))
    return FP8BS_ERR_ALIGN;
  st = check_device();
  if (st != FP8BS_OK) return st;
  const fp8bs::NormProblem p = norm_problem(residual_f32, y, ldy, w_post, gate, ld_gate, w_pre, residual_scale, eps,
                                            weight_offset, T, N);
  hipError_t e = fp8bs::launch_norm(p, x, ldx, h, ldh, static_cast<uint16_t*>(z), ldz, static_cast<uint8_t*>(q), ldq,
                                    sf, ld_sf, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? FP8BS_OK : fail_hip(e);
}

int residual_rms_norm_backward(const void* d_z, int64_t ld_dz, const void* d_h, int64_t ld_dh, const void* h,
                               int64_t ldh, int32_t residual_f32, const void* y, int64_t ldy, const void* w_post,
                               const void* gate, int64_t ld_gate, const void* w_pre, float residual_scale, float eps,
                               float weight_offset, int64_t T, int64_t N, void* d_x, int64_t ld_dx, void* d_y,
                               int64_t ld_dy, float* d_w_pre, float* d_w_post, void* d_gate, int64_t ld_dgate,
                               void* stream) {
  return run_norm_backward(false, nullptr, 0, d_z, ld_dz, d_h, ld_dh, h, ldh, residual_f32, y, ldy, w_post, gate,
                           ld_gate, w_pre, residual_scale, eps, weight_offset, T, N, d_x, ld_dx, d_y, ld_dy, d_w_pre,
                           d_w_post, d_gate, ld_dgate, stream);
}

int64_t residual_rms_norm_backward_scratch_bytes(int64_t T, int64_t N) {
  if (T <= 0 || N <= 0 || N % 8 != 0 || N > fp8bs::kNormMaxN) return 0;
  fp8bs::NormProblem p = {};
  p.T = T;
  p.N = N;
  return (int64_t)fp8bs::norm_backward_scratch_bytes(p);
}

int residual_rms_norm_backward_noalloc(const void* d_z, int64_t ld_dz, const void* d_h, int64_t ld_dh, const void* h,
                                       int64_t ldh, int32_t residual_f32, const void* y, int64_t ldy,
                                       const void* w_post, const void* gate, int64_t ld_gate, const void* w_pre,
                                       float residual_scale, float eps, float weight_offset, int64_t T, int64_t N,
                                       void* d_x, int64_t ld_dx, void* d_y, int64_t ld_dy, float* d_w_pre,
                                       float* d_w_post, void* d_gate, int64_t ld_dgate, void* scratch,
                                       int64_t scratch_bytes, void* stream) {
  return run_norm_backward(true, scratch, scratch_bytes, d_z, ld_dz, d_h, ld_dh, h, ldh, residual_f32, y, ldy, w_post,
                           gate, ld_gate, w_pre, residual_scale, eps, weight_offset, T, N, d_x, ld_dx, d_y, ld_dy, d_w_pre,
                           d_w_post, d_gate, ld_dgate, stream);
}

int silu_mul_quant_group_pack_checkpoint(const void* x, const int32_t* masked_m, int64_t E, int64_t M_max, int64_t H,
                                         void* q, uint32_t* sf, void* cq, uint32_t* csf, void* stream) {
  int st = check_checkpoint(E, M_max, H);
  if (st != FP8BS_OK) return st > 0 ? FP8BS_OK : st;
  if (!x || !masked_m || !q || !sf || !cq || !csf) return FP8BS_ERR_NULL;
  if (!aligned(x, 16) || !aligned(q, 16) || !aligned(cq, 16) || !aligned(sf, 4) || !aligned(csf, 4) ||
      !aligned(masked_m, 4))
    return FP8BS_ERR_ALIGN;
  st = check_device();
  if (st != FP8BS_OK) return st;
  hipError_t e = fp8bs::launch_silu_checkpoint(static_cast<const uint16_t*>(x), masked_m, E, M_max, H,
                                               static_cast<uint8_t*>(q), sf, static_cast<uint8_t*>(cq), csf,
                                               static_cast<hipStream_t>(stream));
  return e == hipSuccess ? FP8BS_OK : fail_hip(e);
}

int silu_mul_backward_from_checkpoint(const void* d_y, const int32_t* masked_m, int64_t E, int64_t M_max, int64_t H,
                                      const void* cq, const uint32_t* csf, void* d_x, void* q, uint32_t* sf,
                                      void* stream) {
  int st = check_checkpoint(E, M_max, H);
  if (st != FP8BS_OK) return st > 0 ? FP8BS_OK : st;
  if (!d_y || !masked_m || !cq || !csf || !d_x == !q || !q != !sf) return FP8BS_ERR_NULL;
  if (!aligned(d_y, 16) || !aligned(cq, 16) || !aligned_or_null(d_x, 16) || !aligned_or_null(q, 16) ||
      !aligned(csf, 4) || !aligned_or_null(sf, 4) || !aligned(masked_m, 4))
    return FP8BS_ERR_ALIGN;
  st = check_device();
  if (st != FP8BS_OK) return st;
  hipError_t e = fp8bs::launch_silu_backward(static_cast<const uint16_t*>(d_y), masked_m, E, M_max, H,
                                             static_cast<const uint8_t*>(cq), csf, static_cast<uint16_t*>(d_x),
                                             static_cast<uint8_t*>(q), sf, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? FP8BS_OK : fail_hip(e);
}

int fp8bs_gemm_config_count(void) { return fp8bs::gemm_config_count(); }

int fp8bs_gemm_config(int masked, int64_t M, int64_t N, int64_t K, int32_t* kernel, int32_t* bm, int32_t* bn,
                      int32_t* splits) {
  if (M < 0 || N < 0 || K < 128 || K % 128 != 0 || N % 64 != 0) return FP8BS_ERR_SHAPE;
  if (!kernel || !bm || !bn || !splits) return FP8BS_ERR_NULL;
  if (masked < 0 || masked > 6) return FP8BS_ERR_SHAPE;
  const fp8bs::GemmProblem p = host_problem(masked, M, N, K);
  const fp8bs::GemmConfig cfg = fp8bs::choose_gemm_config(p);
  if (cfg.kernel < 0) return FP8BS_ERR_SHAPE;  // no entry takes this problem (K past every scale table)
  *kernel = cfg.kernel;
  *bm = cfg.bm;
  *bn = cfg.bn;
  *splits = cfg.splits;
  return FP8BS_OK;
}

int fp8bs_gemm_config_of(int32_t kernel, int masked, int64_t M, int64_t N, int64_t K, int32_t splits, int32_t* bm,
                         int32_t* bn, int32_t* splits_out) {
  if (M < 0 || N < 0 || K < 128 || K % 128 != 0 || N % 64 != 0) return FP8BS_ERR_SHAPE;
  if (!bm || !bn || !splits_out) return FP8BS_ERR_NULL;
  if (masked < 0 || masked > 6) return FP8BS_ERR_SHAPE;
  const fp8bs::GemmProblem p = host_problem(masked, M, N, K);
  fp8bs::GemmConfig cfg;
  if (!fp8bs::gemm_config_by_index(kernel, p, splits < 1 ? 1 : splits, &cfg)) return FP8BS_ERR_SHAPE;
  *bm = cfg.bm;
  *bn = cfg.bn;
  *splits_out = cfg.splits;
  return FP8BS_OK;
}

const char* fp8bs_status_string(int status) {
  switch (status) {
    case FP8BS_OK: return "ok";
    case FP8BS_ERR_NULL: return "null pointer";
    case FP8BS_ERR_SHAPE: return "invalid shape or leading dimension";
    case FP8BS_ERR_ALIGN: return "misaligned pointer or row stride";
    case FP8BS_ERR_DEVICE: return "device is not gfx950";
    case FP8BS_ERR_LAUNCH: return "HIP call failed";
    case FP8BS_ERR_ALLOC: return "workspace allocation failed or refused during graph capture";
    case FP8BS_ERR_SCRATCH: return "the problem needs more scratch than a no-allocation entry has or was given";
    default: return "unknown status";
  }
}

int fp8bs_last_hip_error(void) { return g_last_hip_error; }

}  // extern "C"
