// Which kernels the calls of the decode step's operators launch, with the stand-in of
// host_launches.cpp: reads a call a line, `layer KIND T TOPK E K H` or `product T N K FORMAT GROUP ZEROS`, and prints
// the kernel of each of its launches; `kernels` prints those that the library has.
#define main host_launches_main
#include "host_launches.cpp"
#undef main

#include <cxxabi.h>

#include <cstdlib>
#include <iostream>

namespace {

std::string plain(const std::string& mangled) {
  char* s = abi::__cxa_demangle(mangled.c_str(), nullptr, nullptr, nullptr);
  const std::string name = s ? s : mangled;
  std::free(s);
  return name;
}

int layer(const std::string& kind, int64_t T, int32_t topk, int64_t E, int64_t K, int64_t H) {
  const int64_t need = moe_decode_layer_scratch_bytes(T, topk, H);
  void* const stream = stream_of(0);
  if (kind == "w4")
    return moe_decode_layer_w4(at(1), K, at<uint32_t>(2), T, at<int32_t>(3), at<float>(4), at(5), at(6), at(7), at(8), at(9),
                               K, T, topk, E, K, H, at(10), K, at(11), need, stream);
  return (kind == "plain" ? moe_decode_layer : moe_decode_layer_preshuffled)(
      at(1), K, at<uint32_t>(2), T, at<int32_t>(3), at<float>(4), at(5), at<float>(6), at(7), at<float>(8), at(9), K, T, topk,
      E, K, H, at(10), K, at(11), need, stream);
}

}  // namespace

int main() {
  for (std::string what; std::cin >> what;) {
    launches.clear();
    if (what == "kernels") {
      for (const auto& k : kernels()) std::printf("%s\n", plain(k.second).c_str());
    } else if (what == "layer") {
      std::string kind;
      int64_t T, E, K, H;
      int32_t topk;
      std::cin >> kind >> T >> topk >> E >> K >> H;
      expect(layer(kind, T, topk, E, K, H) == FP8BS_OK, "layer refused");
    } else {
      std::string format;
      int64_t T, N, K;
      int32_t group;
      bool zeros;
      std::cin >> T >> N >> K >> format >> group >> zeros;
      expect(w4_group_gemv_nt(at(1), K, at(2), at(3), zeros ? at(4) : nullptr, T, N, K, format == "int4" ? FP8BS_INT4 : FP8BS_E2M1,
                              group, at(5), N, stream_of(0)) == FP8BS_OK, "product refused");
    }
    for (const Launch& l : launches) std::printf("%s\n", plain(l.kernel).c_str());
  }
  return failed ? 1 : 0;
}
