// Tokens to the rows of their experts and back, in training: moe_dispatch, its gradient, and
// the gradient of the weighted combine.
//
//   xp[inv[t,j]] = x[t]                       dx[t] = dx_in[t] + sum_j dxp[inv[t,j]] + dxp[R+t]
//   dy2[inv[t,j]] = w[t,j] dout[t]            dw[t,j] = sum_h dout[t][h] y2[inv[t,j]][h]
//
// All three walk the tokens, not the packed rows: a token's row is read (or written) once
// and stays in registers while its k + 1 packed rows are written (or read), so every byte
// crosses HBM once.  Walking the packed rows instead would read x k + 1 times, in expert
// order and from HBM once x is larger than L2.  No two threads write the same place and a
// token's rows are added in one order: no atomics, run-to-run identical.
// A thread moves 8 bf16 values (16 bytes) at a time.  Bound by HBM: of 7168 columns, top-8 and
// shared, the dispatch of 16384 tokens 347 us (6.76 TB/s, the copy rate), its gradient to fp32 423
// (7.2: more reads than writes), the combine's gradient of 8192 tokens with dw 315 (6.7).
// An entry of inv outside [0, R) is a token slot without a row: nothing is written for it,
// it adds nothing, its weight's gradient is zero.
#include "grad.cuh"

namespace moe {

namespace {

constexpr int kMaxK = 16;

// Thread -> (token, 8-column chunk).
struct TokenChunk {
  int t, c;
  bool live;
  __device__ __forceinline__ TokenChunk(int T, int chunks) {
    const long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
    live = i < static_cast<long long>(T) * chunks;
    t = i < (1LL << 32) ? static_cast<int>(static_cast<uint32_t>(i) / chunks)
                        : static_cast<int>(i / chunks);
    c = static_cast<int>(i - static_cast<long long>(t) * chunks);
  }
};

// kWeights: the combine's gradient without the weights' own, dy2 of dout (rounded once; the
// shared row as it is).
template <bool kWeights>
__global__ void __launch_bounds__(256) k_dispatch(const uint16_t* __restrict__ x,
                                                  const int32_t* __restrict__ inv,
                                                  const float* __restrict__ w, int T, int k, int H,
                                                  int R, int shared, uint16_t* __restrict__ xp) {
  pdl_wait();
  pdl_trigger();
  const TokenChunk at(T, H / 8);
  if (!at.live) return;
  uint32_t v[4];
  ld_bf16x8(x + static_cast<size_t>(at.t) * H + at.c * 8, v);
  const size_t slot = static_cast<size_t>(at.t) * k;
  for (int j = 0; j < k; ++j) {
    const int r = __ldg(inv + slot + j);
    if (r < 0 || r >= R) continue;
    uint32_t o[4];
    if (kWeights) {
      const float wj = __ldg(w + slot + j);
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = bf16x2_of(wj * bf16_lo(v[i]), wj * bf16_hi(v[i]));
    }
    st_bf16x8(xp + static_cast<size_t>(r) * H + at.c * 8, kWeights ? o : v);
  }
  if (shared) st_bf16x8(xp + (static_cast<size_t>(R) + at.t) * H + at.c * 8, v);
}

// kF32: dx and dx_in are fp32.  fp32 sum in j order, the shared row last, one rounding.
template <bool kF32>
__global__ void __launch_bounds__(256) k_dispatch_bwd(const uint16_t* __restrict__ dxp,
                                                      const int32_t* __restrict__ inv,
                                                      const void* dx_in, int T, int k, int H,
                                                      int R, int shared, void* dx) {
  pdl_wait();
  pdl_trigger();
  const TokenChunk at(T, H / 8);
  if (!at.live) return;
  const size_t here = static_cast<size_t>(at.t) * H + at.c * 8;
  float acc[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = 0.f;
  if (dx_in) {
    if (kF32) {
      const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(dx_in) + here);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float4 f = p[i];
        acc[4 * i] = f.x, acc[4 * i + 1] = f.y, acc[4 * i + 2] = f.z, acc[4 * i + 3] = f.w;
      }
    } else {
      uint32_t v[4];
      ld_bf16x8(static_cast<const uint16_t*>(dx_in) + here, v);
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[2 * i] = bf16_lo(v[i]), acc[2 * i + 1] = bf16_hi(v[i]);
    }
  }
  const int32_t* slot = inv + static_cast<size_t>(at.t) * k;
  // four rows in flight at a time
  const int n = k + shared;
  for (int j0 = 0; j0 < n; j0 += 4) {
    uint32_t v[4][4];
#pragma unroll
    for (int jj = 0; jj < 4; ++jj) {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[jj][i] = 0;
      const int j = j0 + jj;
      if (j < n) {
        const long long r = j < k ? __ldg(slot + j) : static_cast<long long>(R) + at.t;
        if (r >= 0 && (r < R || j == k)) ld_bf16x8(dxp + r * H + at.c * 8, v[jj]);
      }
    }
#pragma unroll
    for (int jj = 0; jj < 4; ++jj)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[2 * i] += bf16_lo(v[jj][i]);
        acc[2 * i + 1] += bf16_hi(v[jj][i]);
      }
  }
  if (kF32) {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(dx) + here);
#pragma unroll
    for (int i = 0; i < 2; ++i)
      p[i] = make_float4(acc[4 * i], acc[4 * i + 1], acc[4 * i + 2], acc[4 * i + 3]);
  } else {
    uint32_t v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = bf16x2_of(acc[2 * i], acc[2 * i + 1]);
    st_bf16x8(static_cast<uint16_t*>(dx) + here, v);
  }
}

// dw, and dy2 if it is not null (it may be y2's buffer).  A CTA per token, or with kPack `warps`
// warps per token and as many tokens as the CTA's warps do for.
template <bool kPack>
__global__ void __launch_bounds__(kPack ? 256 : 512)
    k_combine_bwd(const uint16_t* __restrict__ dout, const uint16_t* y2,
                  const int32_t* __restrict__ inv, const float* __restrict__ w, int T, int k, int H,
                  int R, int shared, int pack, uint16_t* dy2, float* __restrict__ dw) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // (kPack: the CTA's token, the warp's part of its row)
  const int of = kPack ? warp / pack : 0, part_of = kPack ? warp - of * pack : warp;
  const int t = kPack ? blockIdx.x * (blockDim.x / 32 / pack) + of : blockIdx.x;
  const int first = kPack ? (part_of * 32 + lane) * 8 : threadIdx.x * 8;
  __shared__ float part[16][kMaxK];
  const bool live = !kPack || t < T;
  const int32_t* slot = inv + static_cast<size_t>(t) * k;
  const float* wt = w + static_cast<size_t>(t) * k;
  float dot[kMaxK];
#pragma unroll
  for (int j = 0; j < kMaxK; ++j) dot[j] = 0.f;
  for (int c = first; live && c < H; c += kPack ? pack * 256 : blockDim.x * 8) {
    uint32_t g[4];
    ld_bf16x8(dout + static_cast<size_t>(t) * H + c, g);
#pragma unroll
    for (int j0 = 0; j0 < kMaxK; j0 += 4) {
      if (j0 >= k) break;
      int r[4];
      uint32_t y[4][4];
#pragma unroll
      for (int jj = 0; jj < 4; ++jj) {
        const int j = j0 + jj;
        r[jj] = j < k ? __ldg(slot + j) : -1;
        if (r[jj] >= R) r[jj] = -1;
#pragma unroll
        for (int i = 0; i < 4; ++i) y[jj][i] = 0;
        if (r[jj] >= 0) ld_bf16x8(y2 + static_cast<size_t>(r[jj]) * H + c, y[jj]);
      }
#pragma unroll
      for (int jj = 0; jj < 4; ++jj) {
        if (r[jj] < 0) continue;
        if (dy2) {
          const float wj = __ldg(wt + j0 + jj);
          uint32_t o[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) o[i] = bf16x2_of(wj * bf16_lo(g[i]), wj * bf16_hi(g[i]));
          st_bf16x8(dy2 + static_cast<size_t>(r[jj]) * H + c, o);
        }
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          s = fmaf(bf16_lo(g[i]), bf16_lo(y[jj][i]), s);
          s = fmaf(bf16_hi(g[i]), bf16_hi(y[jj][i]), s);
        }
        dot[j0 + jj] += s;
      }
    }
    if (dy2 && shared) st_bf16x8(dy2 + (static_cast<size_t>(R) + t) * H + c, g);
  }
#pragma unroll
  for (int j = 0; j < kMaxK; ++j) {
    if (j >= k) break;
    float s = dot[j];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    if (lane == 0) part[warp][j] = s;
  }
  __syncthreads();
  if (live && part_of == 0 && lane < k) {
    float s = 0.f;
    const int n = kPack ? pack : blockDim.x / 32;
    for (int i = 0; i < n; ++i) s += part[warp + i][lane];
    dw[static_cast<size_t>(t) * k + lane] = s;
  }
}

cudaError_t chunk_grid(int T, int H, unsigned* grid) {
  const long long n = (static_cast<long long>(T) * (H / 8) + 255) / 256;
  if (n > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
  *grid = static_cast<unsigned>(n);
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_dispatch(const uint16_t* x, const int32_t* inv, int T, int k, int H, int R,
                            int shared, uint16_t* xp, cudaStream_t st) {
  unsigned grid;
  const cudaError_t e = chunk_grid(T, H, &grid);
  if (e != cudaSuccess) return e;
  return launch_k(k_dispatch<false>, grid, 256, 0, st, x, inv, nullptr, T, k, H, R, shared, xp);
}

cudaError_t launch_dispatch_bwd(const uint16_t* dxp, const int32_t* inv, const void* dx_in,
                                bool f32, int T, int k, int H, int R, int shared, void* dx,
                                cudaStream_t st) {
  unsigned grid;
  const cudaError_t e = chunk_grid(T, H, &grid);
  if (e != cudaSuccess) return e;
  return launch_k(f32 ? k_dispatch_bwd<true> : k_dispatch_bwd<false>, grid, 256, 0, st, dxp, inv,
                  dx_in, T, k, H, R, shared, dx);
}

cudaError_t launch_combine_bwd(const uint16_t* dout, const uint16_t* y2, const int32_t* inv,
                               const float* w, int T, int k, int H, int R, int shared,
                               uint16_t* dy2, float* dw, cudaStream_t st) {
  if (!dw) {  // no sums over rows (6881 tokens of 128 columns: 2.4 us, as a CTA a token 7.6)
    unsigned grid;
    const cudaError_t e = chunk_grid(T, H, &grid);
    if (e != cudaSuccess) return e;
    return launch_k(k_dispatch<true>, grid, 256, 0, st, dout, inv, w, T, k, H, R, shared, dy2);
  }
  // as many warps as a token's row has chunks for, in as few rounds as 16 warps allow; of short
  // rows several share a CTA (whose place among the SM's 32 a row of its own would leave half
  // empty)
  const int chunks = H / 8, rounds = (chunks + 511) / 512;
  const int warps = (chunks + rounds * 32 - 1) / (rounds * 32);
  const int tokens = warps < 8 ? 8 / warps : 1;
  return launch_k(tokens > 1 ? k_combine_bwd<true> : k_combine_bwd<false>,
                  (T + tokens - 1) / tokens, warps * tokens * 32, 0, st, dout, y2, inv, w, T, k, H, R,
                  shared, warps, dy2, dw);
}

}  // namespace moe
