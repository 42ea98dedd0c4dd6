// Internal launchers of the operators of a decode step: the mixture-of-experts layer of a
// few tokens and the products with 4-bit weights.  The C-ABI layer validates every argument
// before calling these; the launchers only pick grid shapes and launch on the caller's
// stream.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fp8bs {

// How a product's weights lie in memory.
enum class Weights { kPlain, kShuffled, kW4 };

constexpr int64_t kMoeDecodeMaxT = 64;
constexpr int64_t kMoeDecodeMaxE = 1024;
constexpr int kMoeDecodeMaxTopk = 64;
constexpr int64_t kMoeDecodeMaxK = 65536;  // hidden and half sizes
struct MoeDecodeProblem {
  const uint8_t* q;    // e4m3 [T][ldq]
  const uint32_t* sf;  // [ceil(K / 512)][ld_sf]
  const int32_t* ids;  // [T][topk]
  const float* weights;
  const uint8_t* w13;  // [E][2H][K], or 4-bit tiles of it
  const void* s13;
  const uint8_t* w2;  // [E][K][H]
  const void* s2;
  const uint16_t* base;  // or nullptr
  uint16_t* out;
  int64_t ldq, ld_sf, ld_base, ld_out;
  int T, topk, E, K, H;
};
// scratch: moe_decode_scratch_bytes() of device memory.
hipError_t launch_moe_decode(const MoeDecodeProblem& p, Weights kind, void* scratch, hipStream_t stream);
size_t moe_decode_scratch_bytes(int64_t T, int64_t topk, int64_t H);

// Weights of 4 bits under group scales: e2m1 codes with a UE8M0 byte for 32 columns, or integers
// 0..15 with a bf16 scale (and a zero point, or 8) for 32, 64 or 128 columns.
constexpr int64_t kW4MaxK = 65536;
struct W4Problem {
  const uint16_t* x;  // bf16 [T][ldx]
  int64_t ldx, T, N, K;
  const uint8_t* codes;   // 4-bit tiles
  const void* scales;     // uint8 (e2m1) or bf16 (integers)
  const uint8_t* zeros;   // or nullptr
  bool e2m1;
  int group;
  uint16_t* out;  // bf16 [T][ld_out]
  int64_t ld_out;
};
hipError_t launch_w4_gemv(const W4Problem& p, hipStream_t stream);
hipError_t launch_w4_quant(const uint16_t* w, int64_t rows, int64_t K, bool e2m1, int group, uint8_t* codes,
                           void* scales, uint8_t* zeros, hipStream_t stream);
hipError_t launch_w4_preshuffle(const uint8_t* codes, const void* scales, const uint8_t* zeros, int64_t E, int64_t N,
                                int64_t K, bool e2m1, int group, uint8_t* codes_out, void* scales_out,
                                uint8_t* zeros_out, hipStream_t stream);

}  // namespace fp8bs
