// Two host threads make their first calls of the launches together, on stand-ins of
// the CUDA runtime (_fake_cudart.cpp, no GPU), under ThreadSanitizer: what the launches keep
// between calls has to be published in an order.  Each launch's grid is checked as well.
#include <atomic>
#include <cstdio>
#include <thread>

#include "block.cuh"

extern std::atomic<int> launches, empty_grids;

namespace {
std::atomic<int> waiting{0};
}  // namespace

namespace moe {
unsigned long long current_context_id() { return 1; }
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
  // the layer's own: every list of the tile plan, one-SM and SM-pair kernels, both formats
  uint8_t* c = reinterpret_cast<uint8_t*>(0x10000);
  for (int form = 0; form < 4; ++form) {
    GemmLaunch g = {};
    g.w_codes = g.w_scales = g.act = g.act_scales = c, g.y = p;
    g.G = 8, g.N = 512, g.K = 1024, g.rows_total = 4000;
    NvGemmLaunch n = {};
    n.w_codes = n.w_scales = c, n.act = p, n.y = p;
    n.G = 8, n.N = 512, n.K = 1024, n.rows_total = 4000;
    for (int v = 0; v < kNumVariants; ++v) g.max_items[v] = n.max_items[v] = 20;
    g.max_group_rows = n.max_group_rows = 500;
    g.pair_tiles = form == 1;
    if (form == 2) g.hq = g.hs = c;
    failed += (form < 3 ? launch_grouped_gemm(g, nullptr) : launch_grouped_gemm_nv(n, nullptr)) !=
              cudaSuccess;
  }
  failed += launch_router_logits_split(p, p, f, 3000, 1024, 64, nullptr, nullptr) != cudaSuccess;
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
  return launches.load() > 80 && failed.load() == 0 && empty_grids.load() == 0 ? 0 : 1;
}
