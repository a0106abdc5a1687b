// Two host threads make their first calls of the operators' launches together, on stand-ins of
// the CUDA runtime (_fake_cudart.cpp, no GPU), under ThreadSanitizer: what the launches keep
// between calls has to be published in an order.  Each launch's grid is checked as well.
#include <atomic>
#include <cstdio>
#include <thread>

#include "block.cuh"

extern std::atomic<int> launches, empty_grids;

namespace {
std::atomic<int> waiting{0};
CUresult encode(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill) {
  return CUDA_SUCCESS;
}
}  // namespace

namespace moe {
unsigned long long current_context_id() { return 1; }
EncodeTiledFn get_encode_tiled_fn() { return encode; }
}  // namespace moe

namespace {

int calls() {
  using namespace moe;
  uint16_t* p = reinterpret_cast<uint16_t*>(0x10000);
  float* f = reinterpret_cast<float*>(0x10000);
  int32_t* i = reinterpret_cast<int32_t*>(0x10000);
  int failed = 0;
  // the pair kernel, two pairs a tile, the split kernel (with and without a padded copy)
  const int shapes[][3] = {{4096, 4096, 2048}, {256, 7168, 7168}, {7, 7168, 512}, {4096, 4095, 77}};
  for (const auto& s : shapes) {
    LinearCall a = {};
    a.M = s[0], a.N = s[1], a.K = s[2];
    a.x = a.w = p, a.y = p;
    a.ldx = a.ldw = s[2], a.ldy = s[1];
    if (s[2] % 8) a.x_pad = a.w_pad = p;
    failed += launch_linear(a, nullptr) != cudaSuccess;
  }
  LinearBwdCall b = {};
  b.M = b.N = b.K = 1024;
  b.x = b.w = b.dy = p, b.dx = b.dw = b.dz = p, b.db = b.part = f;
  b.ldx = b.ldw = b.lddy = b.lddx = b.lddw = 1024;
  failed += launch_linear_bwd(b, nullptr) != cudaSuccess;
  for (int cols : {256, 1023, 7168, 8191, 16384}) {
    failed += launch_add_rmsnorm(p, p, false, p, false, 1e-6f, 5000, cols, p, p, nullptr, nullptr,
                                 f, nullptr) != cudaSuccess;
    failed += launch_add_rmsnorm_bwd(p, p, false, p, false, f, 5000, cols, nullptr, p, nullptr, f,
                                     f, nullptr) != cudaSuccess;
  }
  for (int E : {8, 61, 384, 1024})
    failed += launch_balance_bwd(f, i, nullptr, nullptr, i, i, f, f, f, 5000, E, 2, 1, f,
                                 nullptr) != cudaSuccess;
  return failed;
}

}  // namespace

int main() {
  std::atomic<int> failed{0};
  auto run = [&] {
    waiting.fetch_add(1, std::memory_order_relaxed);
    while (waiting.load(std::memory_order_relaxed) < 2) std::this_thread::yield();
    failed.fetch_add(calls(), std::memory_order_relaxed);
  };
  std::thread a(run), b(run);
  a.join(), b.join();
  std::printf("%d launches, %d failed, %d empty grids\n", launches.load(), failed.load(),
              empty_grids.load());
  return launches.load() > 40 && failed.load() == 0 && empty_grids.load() == 0 ? 0 : 1;
}
