// SwiGLU in training: the activation with an 8-bit checkpoint of its inputs, and its gradient.
//
// Forward, y13 = [g | u] in bf16: h = silu(g) u is quantised for W2 as in inference (hq, hs),
// and in the same pass g and u themselves to E4M3 codes with a power-of-two scale per 128
// columns (yq, ys): what stays until the backward pass is 2 I + I bytes a row instead of the
// 4 I of y13 (and the 2 H of y2, which the combine weights' gradient then does not need: see
// below).  One read of y13 for both (a separate quantisation would read it again).
//
// Backward, with s = 1 / (1 + e^-g) and d = w dh (w the row's combine weight):
//     dg = d u s (1 + g (1 - s)),   du = d g s,   dw = sum_i dh_i h_i.
// dw is the gradient of the combine weight: y2 = W2 h, so <dout, y2> = <W2^T dout, h> = <dh, h>
// with dh = W2^T dout of the unweighted row.  h is what W2 took, the values of hq, where they
// are given, else silu(g) u.  Everything in fp32, one rounding to bf16 at the end.
#include "grad.cuh"

namespace moe {

namespace {

// The sigmoid from ex2.approx and rcp.approx (each within 2 units of 2^-23), as the other
// elementwise kernels have it: its error is far below the outputs' bf16 rounding.
__device__ __forceinline__ float sigmoid_of(float z) {
  return __fdividef(1.f, 1.f + __expf(-z));
}

__device__ __forceinline__ void ld_floats16(const uint16_t* p, float (&f)[16]) {
  uint32_t lo[4], hi[4];
  ld_bf16x8(p, lo);
  ld_bf16x8(p + 8, hi);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16_lo(lo[i]), f[2 * i + 1] = bf16_hi(lo[i]);
    f[8 + 2 * i] = bf16_lo(hi[i]), f[9 + 2 * i] = bf16_hi(hi[i]);
  }
}

// The 16 values of one lane of an 8-lane group whose lanes hold a 128-column block: their
// codes and the block's scale exponent.  All lanes of the warp must call it.
__device__ __forceinline__ uint4 codes16(const float (&f)[16], int& e) {
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(f[i]));
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
  e = fp8_scale_exponent(amax);
  const float s = pow2_neg(e);
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    c[i] = e4m3x2(f[4 * i] * s, f[4 * i + 1] * s) |
           static_cast<uint32_t>(e4m3x2(f[4 * i + 2] * s, f[4 * i + 3] * s)) << 16;
  return make_uint4(c[0], c[1], c[2], c[3]);
}

// 2^(b - 127) of a scale byte, exact (2^-127 is an fp32 subnormal).
__device__ __forceinline__ float scale_of(uint32_t b) {
  return b ? __uint_as_float(b << 23) : __uint_as_float(1u << 22);
}

// Four codes (a word) as fp32, without their scale.
__device__ __forceinline__ void codes4(uint32_t w, float (&f)[4]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2(
        static_cast<__nv_fp8x2_storage_t>((w >> (16 * i)) & 0xFFFFu), __NV_E4M3);
    const float2 v = __half22float2(__half2(hr));
    f[2 * i] = v.x, f[2 * i + 1] = v.y;
  }
}
__device__ __forceinline__ void bf16x4(uint32_t lo, uint32_t hi, float (&f)[4]) {
  f[0] = bf16_lo(lo), f[1] = bf16_hi(lo), f[2] = bf16_lo(hi), f[3] = bf16_hi(hi);
}
// The gradient's CTAs: at most so many threads, and so many CTAs of that size per SM.
constexpr int kBwdThreads = 512, kBwdCtas = 4;

// Eight lanes per 128-column block, 16 columns a lane (73728 rows of 2048: 172 us, 0.92 of HBM; 16
// lanes of 8 columns: 193 to 214, their reductions); Idx as wide as the lanes need.
template <typename Idx>
__global__ void __launch_bounds__(256) k_swiglu_save(const uint16_t* __restrict__ y13, int rows,
                                                     int I, uint8_t* __restrict__ hq,
                                                     uint8_t* __restrict__ hs,
                                                     uint8_t* __restrict__ yq,
                                                     uint8_t* __restrict__ ys) {
  pdl_wait();
  pdl_trigger();
  const Idx nblk = I / 128;
  const Idx gid = static_cast<Idx>(blockIdx.x) * blockDim.x + threadIdx.x;
  const Idx blk = gid >> 3;
  const int sub = static_cast<int>(gid & 7);
  const bool live = blk < static_cast<Idx>(rows) * nblk;
  const Idx r = live ? blk / nblk : 0, b = live ? blk - r * nblk : 0;
  float g[16], u[16], h[16];
  const size_t col = static_cast<size_t>(b) * 128 + sub * 16;
  const size_t at = static_cast<size_t>(r) * 2 * I + col;
  if (live) {
    ld_floats16(y13 + at, g);
    ld_floats16(y13 + at + I, u);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) g[i] = u[i] = 0.f;
  }
  // (the same expression as the inference kernel's, so that hq and hs are its, bit for bit)
#pragma unroll
  for (int i = 0; i < 16; ++i) h[i] = __fdividef(g[i], 1.0f + __expf(-g[i])) * u[i];
  int eg, eu, eh;
  const uint4 cg = codes16(g, eg), cu = codes16(u, eu), ch = codes16(h, eh);
  if (!live) return;
  *reinterpret_cast<uint4*>(yq + at) = cg;
  *reinterpret_cast<uint4*>(yq + at + I) = cu;
  *reinterpret_cast<uint4*>(hq + static_cast<size_t>(r) * I + col) = ch;
  if (sub == 0) {
    uint8_t* s = ys + static_cast<size_t>(r) * 2 * nblk + b;
    s[0] = static_cast<uint8_t>(eg + 127);
    s[nblk] = static_cast<uint8_t>(eu + 127);
    hs[static_cast<size_t>(r) * nblk + b] = static_cast<uint8_t>(eh + 127);
  }
}

// A CTA per row, or with kPack `pack` warps per row and as many rows as the CTA's warps do for; 8
// columns a thread at a time; all of a thread's loads are in flight before the first is used,
// and what they bring stays packed until its four columns' turn, so that registers leave room
// for full occupancy (73728 rows of 2048: 224 to 227 us, 0.91 of HBM; with 40 registers a thread 272,
// with 16 columns and 64 registers 254).  kCodes: g and u from the checkpoint; kH: h from hq.
template <bool kCodes, bool kH, bool kPack>
__global__ void __launch_bounds__(kPack ? 256 : kBwdThreads, kPack ? 6 : kBwdCtas)
    k_swiglu_bwd(const SwigluBwdCall a, int pack) {
  pdl_wait();
  pdl_trigger();
  const int I = a.I, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // (kPack: the CTA's row, the warp's part of it)
  const int of = kPack ? warp / pack : 0, part_of = kPack ? warp - of * pack : warp;
  const int r = kPack ? blockIdx.x * (blockDim.x / 32 / pack) + of : blockIdx.x;
  const int first = kPack ? (part_of * 32 + lane) * 8 : threadIdx.x * 8;
  __shared__ float part[kBwdThreads / 32];
  int src = 0;
  bool has = false;  // the row has a combine weight
  if (r < a.R && a.perm_src) {
    src = __ldg(a.perm_src + r);
    has = src >= 0 && src < a.R;
  }
  const float w = a.w && has ? __ldg(a.w + src) : 1.f;
  const size_t row = static_cast<size_t>(r);
  float dot = 0.f;
  for (int c = first; (!kPack || r < a.rows) && c < I; c += kPack ? pack * 256 : blockDim.x * 8) {
    uint32_t dv[4], gv[4], uv[4], hv[2] = {0, 0};
    ld_bf16x8(a.dh + row * I + c, dv);
    float sg = 1.f, su = 1.f, sh = 1.f;
    if (kCodes) {
      const uint8_t* q = a.yq + row * 2 * I + c;
      const uint8_t* s = a.ys + (row * 2 * I + c) / 128;
      const uint2 g = *reinterpret_cast<const uint2*>(q), u = *reinterpret_cast<const uint2*>(q + I);
      gv[0] = g.x, gv[1] = g.y, uv[0] = u.x, uv[1] = u.y;
      sg = scale_of(s[0]), su = scale_of(s[I / 128]);
    } else {
      ld_bf16x8(a.y13 + row * 2 * I + c, gv);
      ld_bf16x8(a.y13 + row * 2 * I + I + c, uv);
    }
    if (kH) {
      const uint2 h = *reinterpret_cast<const uint2*>(a.hq + row * I + c);
      hv[0] = h.x, hv[1] = h.y;
      sh = scale_of(a.hs[(row * I + c) / 128]);
    }
    float sum = 0.f;
    if (kH) {  // (first, so that h's codes hold no registers beside the products below)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float d[4], h[4];
        bf16x4(dv[2 * i], dv[2 * i + 1], d);
        codes4(hv[i], h);
#pragma unroll
        for (int j = 0; j < 4; ++j) sum = fmaf(d[j], h[j], sum);
      }
      dot = fmaf(sum, sh, dot);  // (h's scale is a power of two)
    }
    uint32_t og[4], ou[4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {  // four columns
      float d[4], g[4], u[4], dg[4], du[4];
      bf16x4(dv[2 * i], dv[2 * i + 1], d);
      if (kCodes) {
        codes4(gv[i], g);
        codes4(uv[i], u);
      } else {
        bf16x4(gv[2 * i], gv[2 * i + 1], g);
        bf16x4(uv[2 * i], uv[2 * i + 1], u);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float gj = kCodes ? g[j] * sg : g[j], uj = kCodes ? u[j] * su : u[j];
        const float s = sigmoid_of(gj), silu = gj * s, dd = w * d[j], f = fmaf(silu, 1.f - s, s);
        if (!kH) sum = fmaf(d[j], silu * uj, sum);
        // (where d u is past fp32 both are above 1, and |f| is at most 1.1: d f overflows only if dg
        // does.  In the other order a small d f would lose its bits)
        const float p = dd * uj;
        const bool far = fabsf(p) == INFINITY;
        dg[j] = (far ? dd * f : p) * (far ? uj : f);
        du[j] = dd * silu;
      }
      og[2 * i] = bf16x2_of(dg[0], dg[1]), og[2 * i + 1] = bf16x2_of(dg[2], dg[3]);
      ou[2 * i] = bf16x2_of(du[0], du[1]), ou[2 * i + 1] = bf16x2_of(du[2], du[3]);
    }
    if (!kH) dot += sum;
    st_bf16x8(a.dy13 + row * 2 * I + c, og);
    st_bf16x8(a.dy13 + row * 2 * I + I + c, ou);
  }
  if (!a.dw || (!kPack && !has)) return;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xFFFFFFFFu, dot, o);
  if (lane == 0) part[warp] = dot;
  __syncthreads();
  if (has && part_of == 0 && lane == 0) {
    const int n = kPack ? pack : blockDim.x / 32;
    for (int i = 1; i < n; ++i) dot += part[warp + i];
    a.dw[src] = dot;
  }
}

}  // namespace

cudaError_t launch_swiglu_save(const uint16_t* y13, int rows, int I, uint8_t* hq, uint8_t* hs,
                               uint8_t* yq, uint8_t* ys, cudaStream_t st) {
  const long long blocks = static_cast<long long>(rows) * (I / 128), grid = (blocks + 31) / 32;
  if (grid > 0x7FFFFFFFLL) return cudaErrorInvalidValue;
  return launch_k(grid * 256 <= 0xFFFFFFFFLL ? k_swiglu_save<uint32_t>
                                             : k_swiglu_save<unsigned long long>,
                  static_cast<unsigned>(grid), 256, 0, st, y13, rows, I, hq, hs, yq, ys);
}

cudaError_t launch_swiglu_bwd(const SwigluBwdCall& a, cudaStream_t st) {
  const int chunks = a.I / 8, rounds = (chunks + kBwdThreads - 1) / kBwdThreads;
  const int warps = (chunks + rounds * 32 - 1) / (rounds * 32);
  const int rows = warps < 8 ? 8 / warps : 1;  // of short rows several share a CTA
  using Kernel = void (*)(const SwigluBwdCall, int);
  static const Kernel kernels[2][2][2] = {
      {{k_swiglu_bwd<false, false, false>, k_swiglu_bwd<false, false, true>},
       {k_swiglu_bwd<false, true, false>, k_swiglu_bwd<false, true, true>}},
      {{k_swiglu_bwd<true, false, false>, k_swiglu_bwd<true, false, true>},
       {k_swiglu_bwd<true, true, false>, k_swiglu_bwd<true, true, true>}}};
  const Kernel kern = kernels[a.y13 == nullptr][a.dw && a.hq][rows > 1];
  return launch_k(kern, static_cast<unsigned>((static_cast<long long>(a.rows) + rows - 1) / rows),
                  warps * rows * 32, 0, st, a, warps);
}

}  // namespace moe
