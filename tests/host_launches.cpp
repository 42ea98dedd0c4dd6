// What the library's host code asks of the HIP runtime, call by call, without a GPU: the
// program defines the few runtime functions that libfp8bs.so uses (its own definitions come
// before those of the runtime), writes every launch down and starts nothing.
// `host_launches <scenario>` prints what is wrong and returns 1, or returns 0.
#include <hip/hip_runtime_api.h>

#include <chrono>
#include <condition_variable>
#include <cstdio>
#include <cstring>
#include <functional>
#include <map>
#include <mutex>
#include <string>
#include <thread>
#include <vector>

#include "../include/fp8bs.h"

namespace {

struct Launch {
  std::string kernel;  // mangled name
  dim3 grid, block;
  hipStream_t stream;
  std::thread::id by;
  void** args;  // only inside on_launch
};
std::mutex mu;
std::vector<Launch> launches;
std::function<void(const Launch&)> on_launch;  // called after a launch has been written down
bool capturing = false;
int allocations = 0;

std::map<const void*, std::string>& kernels() {  // filled before main
  static std::map<const void*, std::string> m;
  return m;
}
struct Configuration {
  dim3 grid, block;
  size_t lds;
  hipStream_t stream;
};
thread_local Configuration pushed;

}  // namespace

extern "C" {
void** __hipRegisterFatBinary(const void*) {
  static void* handle = nullptr;
  return &handle;
}
void __hipUnregisterFatBinary(void**) {}
void __hipRegisterFunction(void**, const void* host, char*, const char* name, unsigned, void*, void*, void*, void*,
                           int*) {
  kernels()[host] = name;
}
void __hipRegisterVar(void**, void*, char*, char*, int, size_t, int, int) {}
hipError_t __hipPushCallConfiguration(dim3 grid, dim3 block, size_t lds, hipStream_t stream) {
  pushed = {grid, block, lds, stream};
  return hipSuccess;
}
hipError_t __hipPopCallConfiguration(dim3* grid, dim3* block, size_t* lds, hipStream_t* stream) {
  *grid = pushed.grid;
  *block = pushed.block;
  *lds = pushed.lds;
  *stream = pushed.stream;
  return hipSuccess;
}
hipError_t hipLaunchKernel(const void* f, dim3 grid, dim3 block, void** args, size_t, hipStream_t stream) {
  const Launch l = {kernels()[f], grid, block, stream, std::this_thread::get_id(), args};
  {
    std::lock_guard<std::mutex> lk(mu);
    launches.push_back(l);
  }
  if (on_launch) on_launch(l);
  return hipSuccess;
}
hipError_t hipGetLastError() { return hipSuccess; }
hipError_t hipGetDevice(int* dev) {
  *dev = 0;
  return hipSuccess;
}
hipError_t hipGetDevicePropertiesR0600(hipDeviceProp_tR0600* prop, int) {
  std::memset(prop, 0, sizeof(*prop));
  std::strcpy(prop->gcnArchName, "gfx950");
  return hipSuccess;
}
hipError_t hipMalloc(void** p, size_t) {
  static uintptr_t next = uintptr_t(1) << 40;  // never dereferenced
  std::lock_guard<std::mutex> lk(mu);
  ++allocations;
  next += uintptr_t(1) << 36;
  *p = reinterpret_cast<void*>(next);
  return hipSuccess;
}
hipError_t hipFree(void*) { return hipSuccess; }
hipError_t hipFuncSetAttribute(const void*, hipFuncAttribute, int) { return hipSuccess; }
hipError_t hipGetSymbolAddress(void** p, const void*) { return hipMalloc(p, 0); }
hipError_t hipStreamIsCapturing(hipStream_t, hipStreamCaptureStatus* status) {
  *status = capturing ? hipStreamCaptureStatusActive : hipStreamCaptureStatusNone;
  return hipSuccess;
}
}

namespace {

bool failed = false;
void expect(bool ok, const std::string& what) {
  if (ok) return;
  failed = true;
  std::printf("%s\n", what.c_str());
}
template <typename T = void>
T* at(uintptr_t n) {  // an aligned address that nothing reads
  return reinterpret_cast<T*>(n << 20);
}
void* stream_of(uintptr_t n) { return at(1000 + n); }

int norm_backward(int64_t T, int64_t N, void* stream) {
  return residual_rms_norm_backward(at(1), N, nullptr, 0, at(2), N, 0, at(3), N, at(4), at(5), 0, at(6), 1.0f, 1e-6f,
                                    0.0f, T, N, at(7), N, at(8), N, at<float>(9), at<float>(10), at<float>(11), 0,
                                    stream);
}
int to_experts(void* stream) {
  return fp8_quant_group_pack_to_experts(at(1), 512, 4096, 512, at<int32_t>(2), 8, 32, 64, at(3), at<uint32_t>(4),
                                         at<int32_t>(5), at<int32_t>(6), stream);
}
int noalloc_gemm(void* stream) {
  return fp8_block_gemm_nt_preshuffled_noalloc(at(1), at<uint32_t>(2), 512, at(3), at<float>(4), at(5), 960, 512, 960,
                                               18432, stream);
}
int split_gemm(void* stream) {
  return fp8_block_gemm_nt(at(1), at<uint32_t>(2), 64, at(3), at<float>(4), at(5), 7168, 64, 7168, 18432, stream);
}

// The entry that allocates nothing has one scratch for the GPU: its calls on one stream do not
// break into each other either.
void noalloc_threads() {
  expect(noalloc_gemm(stream_of(0)) == FP8BS_OK, "GEMM without allocation failed");  // clears the counters
  launches.clear();
  std::mutex m;
  std::condition_variable cv;
  bool started = false, answered = false;
  on_launch = [&](const Launch&) {
    std::unique_lock<std::mutex> lk(m);
    if (!started) {
      started = true;
      cv.notify_all();
      cv.wait_for(lk, std::chrono::milliseconds(100), [&] { return answered; });
    } else {
      answered = true;
      cv.notify_all();
    }
  };
  std::thread a([&] { expect(noalloc_gemm(stream_of(0)) == FP8BS_OK, "GEMM without allocation failed"); });
  std::thread b([&] {
    std::unique_lock<std::mutex> lk(m);
    cv.wait(lk, [&] { return started; });
    lk.unlock();
    expect(noalloc_gemm(stream_of(0)) == FP8BS_OK, "GEMM without allocation failed");
  });
  a.join();
  b.join();
  on_launch = nullptr;
  expect(launches.size() == 4 && launches[0].by == launches[1].by && launches[2].by == launches[3].by,
         "a GEMM without allocation breaks into another");
}

// A call whose launches share the stream's workspace is not broken into by another host
// thread's call on that stream, which would overwrite what the first one's later launches
// read; calls on other streams do not wait for it.
void threads() {
  struct Call {
    const char* name;
    std::function<int(void*)> run;
    size_t launches;
  };
  Call calls[] = {{"norm backward", [](void* s) { return norm_backward(512, 2048, s); }, 0},
                  {"quantization into the experts' layout", to_experts, 0},
                  {"split GEMM", split_gemm, 0}};
  for (int turn = 0; turn < 2; ++turn)  // the first allocates, which clears the counters with a launch
    for (Call& c : calls)
      for (int s = 0; s < 2; ++s) {
        launches.clear();
        expect(c.run(stream_of(s)) == FP8BS_OK, std::string(c.name) + " failed");
        c.launches = launches.size();
      }
  for (const Call& first : calls) {
    expect(first.launches == 2, std::string(first.name) + ": not two launches");
    for (const Call& second : calls) {
      for (int other = 0; other < 2; ++other) {
        launches.clear();
        std::mutex m;
        std::condition_variable cv;
        bool started = false, answered = false;
        std::thread::id a_id;
        on_launch = [&](const Launch& l) {
          std::unique_lock<std::mutex> lk(m);
          if (l.by == a_id && !started) {  // the first launch: give the other thread time for its call
            started = true;
            cv.notify_all();
            cv.wait_for(lk, std::chrono::milliseconds(other ? 5000 : 100), [&] { return answered; });
          } else if (l.by != a_id) {
            answered = true;
            cv.notify_all();
          }
        };
        std::thread a([&] {
          {
            std::lock_guard<std::mutex> lk(m);
            a_id = std::this_thread::get_id();
          }
          expect(first.run(stream_of(0)) == FP8BS_OK, std::string(first.name) + " failed");
        });
        std::thread b([&] {
          std::unique_lock<std::mutex> lk(m);
          cv.wait(lk, [&] { return started; });
          lk.unlock();
          expect(second.run(stream_of(other)) == FP8BS_OK, std::string(second.name) + " failed");
        });
        const std::thread::id b_id = b.get_id();
        a.join();
        b.join();
        on_launch = nullptr;
        std::string order;
        for (const Launch& l : launches) order += l.by == b_id ? 'b' : 'a';
        const std::string as(first.launches, 'a'), bs(second.launches, 'b');
        if (other)
          expect(order[1] == 'b', std::string(second.name) + " on another stream waits for " + first.name + ": " + order);
        else
          expect(order == as + bs, std::string(second.name) + " breaks into " + first.name + ": " + order);
      }
    }
  }
}

// The largest sizes of the operators around the experts' products: no launch may have 2^32
// threads in one dimension, and a combine that takes several covers every token once.
void limits() {
  const int64_t T = int64_t(1) << 22;
  struct Size {
    int64_t T, N;
  };
  for (const Size s : {Size{T, 8192}, Size{T, 7168}, Size{T, 6152}, Size{1 << 15, 1 << 20}, Size{(1 << 15) - 1, 1 << 20},
                       Size{5, 8192}}) {
    const int64_t ld = s.N + 8, topk = 3;
    int64_t tokens = 0;
    launches.clear();
    on_launch = [&](const Launch& l) {
      auto arg = [&](int i) { return *static_cast<uintptr_t*>(l.args[i]); };
      // ids, slots, weights, .., base (8), its stride, out (10), its stride, tiles
      for (int i : {0, 1, 2})
        expect(arg(i) - reinterpret_cast<uintptr_t>(at(2 + i)) == uintptr_t(tokens * topk * 4), "pairs of another token");
      for (int i : {8, 10})
        expect(arg(i) - reinterpret_cast<uintptr_t>(at(i)) == uintptr_t(tokens * ld * 2), "rows of another token");
      const unsigned tiles = *static_cast<unsigned*>(l.args[12]);
      expect(int64_t(tiles) * l.block.x * 8 >= s.N, "columns left out");
      expect(l.grid.x % tiles == 0, "part of a token");
      tokens += l.grid.x / tiles;
    };
    expect(moe_combine(at(1), at<int32_t>(2), at<int32_t>(3), at<float>(4), at(8), ld, s.T, topk, 4, 8, s.N, at(10), ld,
                       stream_of(0)) == FP8BS_OK, "combine refused");
    on_launch = nullptr;
    expect(tokens == s.T, "combine of " + std::to_string(tokens) + " tokens for " + std::to_string(s.T));
    expect(s.T > 5 || launches.size() == 1, "more launches than one for a small combine");
    for (const Launch& l : launches)
      expect(uint64_t(l.grid.x) * l.block.x < (uint64_t(1) << 32),
             "combine " + std::to_string(s.T) + " x " + std::to_string(s.N) + ": 2^32 threads");
  }
  expect(moe_combine(at(1), at<int32_t>(2), at<int32_t>(3), nullptr, nullptr, 0, T, 1, 4, 8, 8200, at(5), 8200, nullptr) ==
             FP8BS_ERR_SHAPE, "combine past the stated limit");
  launches.clear();
  expect(moe_route_topk(at(1), 1, 1024, T, 1024, nullptr, FP8BS_SIGMOID, 1, 1, 1, 64, 1, 1.0f, at<int32_t>(2),
                        at<float>(3), nullptr) == FP8BS_OK, "route refused");
  expect(moe_route_topk(at(1), 0, 256, T, 256, nullptr, FP8BS_SOFTMAX, 1, 1, 1, 8, 1, 1.0f, at<int32_t>(2), at<float>(3),
                        nullptr) == FP8BS_OK, "route refused");
  expect(moe_route_topk_backward(at(1), 1, 1024, T, 1024, at<int32_t>(2), at<float>(3), FP8BS_SOFTMAX, 64, 0, 1.0f,
                                 at(4), 1024, nullptr) == FP8BS_OK, "route backward refused");
  expect(moe_combine_backward(at(1), 8192, at(2), at<int32_t>(3), at<int32_t>(4), at<float>(5), T, 64, 4, 8, 8192, at(6),
                              nullptr, nullptr, at<float>(7), nullptr) == FP8BS_OK, "combine backward refused");
  expect(norm_backward(T, 16384, nullptr) == FP8BS_OK, "norm backward refused");
  expect(residual_rms_norm(at(1), 16384, 1, nullptr, 0, nullptr, nullptr, 0, at(2), 1.0f, 1e-6f, 0.0f, T, 16384, at(3),
                           16384, nullptr, 0, nullptr, 0, nullptr, 0, nullptr) == FP8BS_OK, "norm refused");
  for (const Launch& l : launches)
    expect(uint64_t(l.grid.x) * l.block.x < (uint64_t(1) << 32) && l.grid.y <= 65535, l.kernel + ": grid too large");
}

// A dot product over no columns is zero, and is written.
void no_columns() {
  launches.clear();
  uintptr_t cleared = 0;
  int64_t words = 0;
  on_launch = [&](const Launch& l) {
    expect(l.kernel.find("zero_words") != std::string::npos, l.kernel + " over no columns");
    cleared = *static_cast<uintptr_t*>(l.args[0]);
    words = *static_cast<int64_t*>(l.args[1]);
  };
  expect(moe_combine_backward(nullptr, 0, nullptr, at<int32_t>(3), at<int32_t>(4), at<float>(5), 7, 3, 4, 8, 0, nullptr,
                              nullptr, nullptr, at<float>(7), nullptr) == FP8BS_OK, "combine backward refused");
  on_launch = nullptr;
  expect(cleared == reinterpret_cast<uintptr_t>(at(7)) && words == 21, "weights' gradients of no columns not cleared");
  launches.clear();
  expect(moe_combine_backward(nullptr, 0, nullptr, nullptr, nullptr, nullptr, 7, 3, 4, 8, 0, nullptr, nullptr, nullptr,
                              nullptr, nullptr) == FP8BS_OK, "combine backward without weights refused");
  expect(moe_combine_backward(nullptr, 0, nullptr, nullptr, nullptr, nullptr, 0, 3, 4, 8, 0, nullptr, nullptr, nullptr,
                              at<float>(7), nullptr) == FP8BS_OK, "combine backward of nothing refused");
  expect(launches.empty(), "a launch without anything to write");
}

// One row has no partial sums: its norm backward allocates nothing, also under capture.
void one_row() {
  allocations = 0;
  capturing = true;
  launches.clear();
  for (int64_t N : {int64_t(8), int64_t(7168), int64_t(16384)})
    expect(norm_backward(1, N, stream_of(0)) == FP8BS_OK, "norm backward of one row refused under capture");
  expect(launches.size() == 3 && allocations == 0, "norm backward of one row: not one launch and no allocation");
  expect(norm_backward(2, 8, stream_of(0)) == FP8BS_ERR_ALLOC, "an allocation under capture");
  capturing = false;
}

// Norm backward in scratch of the caller's: nothing is allocated, the partial sums lie in it,
// and the call does not wait for one that holds the stream's workspace.
void given_scratch() {
  auto run = [](int64_t T, int64_t N, void* scratch, int64_t bytes) {
    return residual_rms_norm_backward_noalloc(at(1), N, nullptr, 0, at(2), N, 0, at(3), N, at(4), at(5), 0, at(6), 1.0f,
                                              1e-6f, 0.0f, T, N, at(7), N, at(8), N, at<float>(9), at<float>(10),
                                              at<float>(11), 0, scratch, bytes, stream_of(0));
  };
  capturing = true;
  allocations = 0;
  const uintptr_t scratch = reinterpret_cast<uintptr_t>(at(20));
  for (int64_t T : {2, 300, 70000})
    for (int64_t N : {8, 2048, 8200, 16384}) {
      const int64_t need = residual_rms_norm_backward_scratch_bytes(T, N);
      launches.clear();
      int64_t blocks = 0;
      on_launch = [&](const Launch& l) {
        if (l.kernel.find("norm_sums_kernel") != std::string::npos) {
          const uintptr_t from = *static_cast<uintptr_t*>(l.args[0]);
          blocks = *static_cast<int*>(l.args[1]);
          expect(from == scratch, "sums from elsewhere");
          expect(int64_t(l.grid.y) * blocks * N * 4 <= need, "sums past the scratch");
        }
      };
      expect(run(T, N, at(20), need) == FP8BS_OK, "refused with enough scratch");
      on_launch = nullptr;
      expect(launches.size() == 2 && blocks == int64_t(launches[0].grid.x) && launches[1].grid.y == 3, "launches");
      expect(need == 3 * blocks * N * 4, "scratch is not what the sums take");
      expect(run(T, N, at(20), need - 1) == FP8BS_ERR_SCRATCH && run(T, N, nullptr, need) == FP8BS_ERR_NULL &&
                 run(T, N, reinterpret_cast<void*>(scratch + 8), need) == FP8BS_ERR_ALIGN, "bad scratch taken");
    }
  expect(allocations == 0, "an allocation");
  expect(run(1, 2048, nullptr, 0) == FP8BS_OK, "one row refused without scratch");
  for (int64_t N : {-8, 0, 4, 16392}) expect(residual_rms_norm_backward_scratch_bytes(300, N) == 0, "scratch of no rows");
  expect(residual_rms_norm_backward_scratch_bytes(0, 64) == 0 && residual_rms_norm_backward_scratch_bytes(1, 64) == 0 &&
             residual_rms_norm_backward_scratch_bytes(-1, 64) == 0, "scratch of at most one row");
  capturing = false;
  // from inside another call's first launch, whose thread holds the workspace
  expect(norm_backward(300, 2048, stream_of(0)) == FP8BS_OK, "norm backward failed");
  bool inside = false, done = false;
  on_launch = [&](const Launch& l) {
    if (inside) return;
    inside = true;
    std::thread b([&] { done = run(300, 2048, at(20), residual_rms_norm_backward_scratch_bytes(300, 2048)) == FP8BS_OK; });
    b.join();
  };
  expect(norm_backward(300, 2048, stream_of(0)) == FP8BS_OK && done, "waits for the workspace");
  on_launch = nullptr;
}

}  // namespace

int main(int argc, char** argv) {
  const std::map<std::string, void (*)()> scenarios = {{"threads", threads},
                                                       {"noalloc_threads", noalloc_threads},
                                                       {"limits", limits},
                                                       {"no_columns", no_columns},
                                                       {"one_row", one_row},
                                                       {"given_scratch", given_scratch}};
  if (argc != 2 || scenarios.count(argv[1]) == 0) return 2;
  scenarios.at(argv[1])();
  return failed ? 1 : 0;
}
