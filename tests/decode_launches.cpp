// What the decode step's operators ask of the HIP runtime, with the stand-in of
// host_launches.cpp: `decode_launches` prints what is wrong and returns 1, or returns 0.
#define main host_launches_main
#include "host_launches.cpp"
#undef main

namespace {

int layer(int64_t T, int32_t topk, int64_t E, int64_t K, int64_t H) {
  return moe_decode_layer(at(1), K, at<uint32_t>(2), T, at<int32_t>(3), at<float>(4), at(5), at<float>(6), at(7),
                          at<float>(8), at(9), K, T, topk, E, K, H, at(10), K, at(11),
                          moe_decode_layer_scratch_bytes(T, topk, H), stream_of(0));
}

int product(int64_t T, int64_t N, int64_t K, int32_t format, int32_t group) {
  return w4_group_gemv_nt(at(1), K, at(2), at(3), format == FP8BS_INT4 ? at(4) : nullptr, T, N, K, format, group, at(5), N,
                          stream_of(0));
}

}  // namespace

int main() {
  capturing = true;  // nothing is allocated, also under capture
  for (int64_t T : {1, 3, 16, 17, 33, 64})
    for (int32_t topk : {1, 8, 64})
      for (int64_t E : {1, 32, 1024})
        for (int64_t K : {128, 7168, 65536})
          for (int64_t H : {128, 2048, 65536}) {
            launches.clear();
            expect(layer(T, topk, E, K, H) == FP8BS_OK, "layer refused");
            expect(launches.size() == 2, "not two launches");
            const int64_t experts = E < T * topk ? E : T * topk;
            // workgroups of 128, 64 or 32 columns of every expert that can be chosen; 16 or 32 output columns
            const int64_t n = launches[0].grid.x;
            expect(n == experts * H / 128 || n == experts * H / 64 || n == experts * H / 32, "columns left out");
            expect(launches[1].grid.x == K / 16 || launches[1].grid.x == K / 32, "output columns left out");
            expect(n == experts * H / 128 || (T <= 16 && T * topk <= 64), "K in parts for many pairs");
          }
  for (int64_t T : {1, 5, 8, 9, 40, 64, 65, 1 << 21})
    for (int64_t N : {1, 16, 4096, 4112, 8192, 8208, 16368, 16384, 1 << 27})
      for (int32_t group : {32, 64, 128})
        for (int format : {FP8BS_E2M1, FP8BS_INT4}) {
          if (format == FP8BS_E2M1 && group != 32) continue;
          launches.clear();
          expect(product(T, N, 7168, format, group) == FP8BS_OK, "product refused");
          expect(launches.size() == 1, "not one launch");
          const int64_t tiles = (N + 15) / 16;
          const Launch& l = launches[0];
          const int64_t per = (tiles + l.grid.x - 1) / l.grid.x;  // tiles a workgroup
          expect(per == 1 || per == 2 || per == 4 || per == 8, "tiles left out");
          expect(l.grid.y == (T + 63) / 64, "tokens left out");
        }
  launches.clear();
  expect(w4_group_quant(at(1), INT64_C(1) << 40, 65536, FP8BS_INT4, 32, at(2), at(3), at(4), nullptr) == FP8BS_OK, "quantization");
  expect(w4_preshuffle(at(1), at(2), at(3), 1 << 13, 1 << 27, 65536, FP8BS_INT4, 32, at(4), at(5), at(6), nullptr) == FP8BS_OK,
         "layout");
  expect(launches.size() == 4, "launches of the weights");
  for (const Launch& l : launches) expect(uint64_t(l.grid.x) * l.block.x < (uint64_t(1) << 32), l.kernel + ": grid too large");
  launches.clear();
  for (int64_t N : {int64_t(1) << 27})
    for (int64_t T : {1, 64, 1 << 21}) expect(product(T, N, 128, FP8BS_E2M1, 32) == FP8BS_OK, "product refused");
  expect(layer(64, 64, 1024, 65536, 65536) == FP8BS_OK, "layer refused");
  for (const Launch& l : launches)
    expect(uint64_t(l.grid.x) * l.block.x < (uint64_t(1) << 32) && l.grid.y <= 65535, l.kernel + ": grid too large");
  launches.clear();
  expect(layer(0, 8, 32, 7168, 2048) == FP8BS_OK && product(0, 64, 128, FP8BS_E2M1, 32) == FP8BS_OK &&
             product(3, 0, 128, FP8BS_E2M1, 32) == FP8BS_OK && launches.empty(), "a launch of nothing");
  expect(allocations == 0, "an allocation");
  return failed ? 1 : 0;
}
