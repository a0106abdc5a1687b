// Shared by the kernels of the routed layer's gradient (moves.cu, swiglu_grad.cu,
// expert_grad.cu) and their C interface (capi_grad.cu).
#pragma once

#include "block.cuh"

namespace moe {

// Whether the library supports these dims (capi.cu).
bool dims_ok(const moe_dims* d);

// ------------------------------------------------------------------ bf16 accesses -----

__device__ __forceinline__ void ld_bf16x8(const uint16_t* p, uint32_t (&w)[4]) {
  const uint4 v = *reinterpret_cast<const uint4*>(p);
  w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
}
__device__ __forceinline__ void st_bf16x8(uint16_t* p, const uint32_t (&w)[4]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t bf16x2_of(float lo, float hi) {
  __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&b);
}

// ------------------------------------------------------------------ launches ----------

// Tokens to their packed rows and back (moves.cu).  R routed rows, Rs packed rows.
cudaError_t launch_dispatch(const uint16_t* x, const int32_t* inv, int T, int k, int H, int R,
                            int shared, uint16_t* xp, cudaStream_t st);
cudaError_t launch_dispatch_bwd(const uint16_t* dxp, const int32_t* inv, const void* dx_in,
                                bool f32, int T, int k, int H, int R, int shared, void* dx,
                                cudaStream_t st);
cudaError_t launch_combine_bwd(const uint16_t* dout, const uint16_t* y2, const int32_t* inv,
                               const float* w, int T, int k, int H, int R, int shared,
                               uint16_t* dy2, float* dw, cudaStream_t st);

// SwiGLU with its 8-bit checkpoint, and its gradient (swiglu_grad.cu).
cudaError_t launch_swiglu_save(const uint16_t* y13, int rows, int I, uint8_t* hq, uint8_t* hs,
                               uint8_t* yq, uint8_t* ys, cudaStream_t st);
struct SwigluBwdCall {
  int rows, R, I;
  const uint16_t* dh;
  const uint16_t* y13;      // or null: yq, ys
  const uint8_t *yq, *ys;
  const uint8_t *hq, *hs;   // or null: h = silu(g) u
  const int32_t* perm_src;  // [R] with w or dw
  const float* w;           // or null: 1
  uint16_t* dy13;
  float* dw;                // or null
};
cudaError_t launch_swiglu_bwd(const SwigluBwdCall& a, cudaStream_t st);

// Gradient products of the experts (expert_grad.cu): for every row r of group g,
// dx[r][f] = sum_c dy[r][c] * deq(w[g])[c][f], with codes w [G][C][F/2] and scales [G][C][F/32]
// (MXFP4) or [G][C][F/16] and gs [G][gs_segments] (NVFP4: a tensor scale per equal part of the C
// rows).
struct ExpertGradCall {
  const uint16_t* dy;       // [rows][C]
  const int32_t* offsets;   // [G + 1]
  const uint8_t *w, *w_s;
  const float* gs;          // or null: 1
  int nv, gs_segments;      // NVFP4; 1 or 2
  uint16_t* dx;             // [rows][F]
  int E, G, routed, rows, C, F;  // G = E, or E + 1 with a shared expert; routed: rows of the E
  uint32_t* status;
};
// CTAs a tile: single ones (1) or SM pairs (2), as the sizes' cost has it.
int expert_grad_ctas(const ExpertGradCall& a);
cudaError_t launch_expert_grad(const ExpertGradCall& a, int ctas, cudaStream_t st);

}  // namespace moe
