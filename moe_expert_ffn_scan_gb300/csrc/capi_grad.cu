// C interface (include/moe.h) of the routed layer's gradient: argument checks and launches.
// No allocation, no host synchronisation.
#include "grad.cuh"

using namespace moe;

namespace {

constexpr size_t kAlign = 256;

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// A pointer that may be null.
bool null_or(const void* p, size_t a) { return !p || aligned(p, a); }

int cuda_rc(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

// (limits that leave room in 32-bit row and column arithmetic)
bool swiglu_ok(int rows, int I) {
  return rows >= 0 && rows <= (1 << 30) && I >= 128 && I % 128 == 0 && I <= (1 << 29);
}

int rows_R(const moe_dims* d) { return d->T * d->k; }
int rows_Rs(const moe_dims* d) { return rows_R(d) + (d->has_shared ? d->T : 0); }

// Weights of C rows of F features: codes w [G][C][F/2], scales w_s [G][C][F/32] or (segments > 0:
// NVFP4) [G][C][F/16] and gs [G][segments].
struct GradWeights {
  const uint8_t *w, *w_s;
  const float* gs;
  int segments;
};

ExpertGradCall sizes_of(const moe_dims* d, int C, int F) {
  ExpertGradCall a = {};
  a.E = d->E, a.G = d->E + d->has_shared, a.routed = rows_R(d), a.rows = rows_Rs(d);
  a.C = C, a.F = F;
  return a;
}

// dx of the rows of dy through those weights, with 1 or 2 CTAs a tile or (0) as the sizes have it.
int expert_grad(const moe_dims* d, int C, int F, const uint16_t* dy, const int32_t* offsets,
                const GradWeights& W, uint16_t* dx, void* ws, size_t ws_bytes, void* stream,
                int ctas = 0) {
  if (!dims_ok(d) || static_cast<long long>(d->E + 1) * C >= (1LL << 31))
    return MOE_ERR_UNSUPPORTED_SHAPE;
  if (W.segments && (d->H % 256 || d->I % 256)) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (!dy || !offsets || !W.w || !W.w_s || !dx || !ws) return MOE_ERR_INVALID_ARG;
  if (!aligned(dy, 16) || !aligned(offsets, 4) || !aligned(W.w, 32) || !aligned(W.w_s, 16) ||
      !null_or(W.gs, 4) || !aligned(dx, 16) || !aligned(ws, kAlign))
    return MOE_ERR_INVALID_ARG;
  if (ws_bytes < moe_gemm_backward_workspace_size(d)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  ExpertGradCall a = sizes_of(d, C, F);
  a.dy = dy, a.offsets = offsets, a.w = W.w, a.w_s = W.w_s, a.dx = dx;
  a.nv = W.segments > 0, a.gs_segments = W.segments, a.gs = W.gs;
  a.status = static_cast<uint32_t*>(ws);
  return cuda_rc(launch_expert_grad(a, ctas ? ctas : expert_grad_ctas(a),
                                    static_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

int moe_dispatch(const moe_dims* d, const uint16_t* x, const int32_t* inv, uint16_t* xp,
                 void* stream) {
  if (!dims_ok(d)) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (!x || !inv || !xp || !aligned(x, 16) || !aligned(inv, 4) || !aligned(xp, 16))
    return MOE_ERR_INVALID_ARG;
  return cuda_rc(launch_dispatch(x, inv, d->T, d->k, d->H, rows_R(d), d->has_shared, xp,
                                 static_cast<cudaStream_t>(stream)));
}

int moe_dispatch_backward(const moe_dims* d, const uint16_t* dxp, const int32_t* inv,
                          const void* dx_in, int32_t dx_dtype, void* dx, void* stream) {
  if (!dims_ok(d)) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (dx_dtype != MOE_DTYPE_BF16 && dx_dtype != MOE_DTYPE_F32) return MOE_ERR_INVALID_ARG;
  if (!dxp || !inv || !dx || !aligned(dxp, 16) || !aligned(inv, 4) || !null_or(dx_in, 16) ||
      !aligned(dx, 16))
    return MOE_ERR_INVALID_ARG;
  return cuda_rc(launch_dispatch_bwd(dxp, inv, dx_in, dx_dtype == MOE_DTYPE_F32, d->T, d->k, d->H,
                                     rows_R(d), d->has_shared, dx,
                                     static_cast<cudaStream_t>(stream)));
}

int moe_combine_backward(const moe_dims* d, const uint16_t* dout, const uint16_t* y2,
                         const int32_t* inv, const float* w, uint16_t* dy2, float* dw,
                         void* stream) {
  if (!dims_ok(d)) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (!dout || !inv || (!dy2 && !dw) || (dy2 && !w) || (dw && !y2)) return MOE_ERR_INVALID_ARG;
  if (!aligned(dout, 16) || !null_or(y2, 16) || !aligned(inv, 4) || !null_or(w, 4) ||
      !null_or(dy2, 16) || !null_or(dw, 4))
    return MOE_ERR_INVALID_ARG;
  return cuda_rc(launch_combine_bwd(dout, y2, inv, w, d->T, d->k, d->H, rows_R(d), d->has_shared,
                                    dy2, dw, static_cast<cudaStream_t>(stream)));
}

int moe_swiglu_quant_save(int32_t rows, int32_t I, const uint16_t* y13, uint8_t* hq, uint8_t* hs,
                          uint8_t* yq, uint8_t* ys, void* stream) {
  if (!swiglu_ok(rows, I)) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (rows == 0) return MOE_OK;
  if (!y13 || !hq || !hs || !yq || !ys || !aligned(y13, 16) || !aligned(hq, 16) ||
      !aligned(yq, 16))
    return MOE_ERR_INVALID_ARG;
  return cuda_rc(launch_swiglu_save(y13, rows, I, hq, hs, yq, ys,
                                    static_cast<cudaStream_t>(stream)));
}

int moe_swiglu_backward(const moe_swiglu_backward_desc* d, const uint16_t* dh, const uint16_t* y13,
                        const uint8_t* yq, const uint8_t* ys, const uint8_t* hq,
                        const uint8_t* hs, const int32_t* perm_src, const float* w,
                        uint16_t* dy13, float* dw, void* stream) {
  if (!d || !swiglu_ok(d->rows, d->I) || d->R < 0 || d->R > d->rows)
    return MOE_ERR_UNSUPPORTED_SHAPE;
  if (d->rows == 0) return MOE_OK;
  // the activations in exactly one form; codes with their scales
  if (!dh || !dy13 || (y13 != nullptr) == (yq != nullptr) || (yq != nullptr) != (ys != nullptr) ||
      (hq != nullptr) != (hs != nullptr) || ((w || dw) && d->R > 0 && !perm_src))
    return MOE_ERR_INVALID_ARG;
  if (!aligned(dh, 16) || !null_or(y13, 16) || !null_or(yq, 16) || !null_or(hq, 16) ||
      !null_or(perm_src, 4) || !null_or(w, 4) || !aligned(dy13, 16) || !null_or(dw, 4))
    return MOE_ERR_INVALID_ARG;
  SwigluBwdCall a = {};
  a.rows = d->rows, a.R = d->R, a.I = d->I;
  a.dh = dh, a.y13 = y13, a.yq = yq, a.ys = ys, a.hq = hq, a.hs = hs;
  a.perm_src = perm_src, a.w = w, a.dy13 = dy13, a.dw = dw;
  return cuda_rc(launch_swiglu_bwd(a, static_cast<cudaStream_t>(stream)));
}

size_t moe_gemm_backward_workspace_size(const moe_dims* d) { return dims_ok(d) ? kAlign : 0; }

int moe_grouped_gemm_w2_backward(const moe_dims* d, const uint16_t* dy2,
                                 const int32_t* group_offsets, const uint8_t* w2,
                                 const uint8_t* w2_s, uint16_t* dh, void* ws, size_t ws_bytes,
                                 void* stream) {
  if (!d) return MOE_ERR_UNSUPPORTED_SHAPE;
  return expert_grad(d, d->H, d->I, dy2, group_offsets, {w2, w2_s, nullptr, 0}, dh, ws, ws_bytes,
                     stream);
}

int moe_grouped_gemm_w13_backward(const moe_dims* d, const uint16_t* dy13,
                                  const int32_t* group_offsets, const uint8_t* w13,
                                  const uint8_t* w13_s, uint16_t* dxp, void* ws, size_t ws_bytes,
                                  void* stream) {
  if (!d || d->I > (1 << 29)) return MOE_ERR_UNSUPPORTED_SHAPE;
  return expert_grad(d, 2 * d->I, d->H, dy13, group_offsets, {w13, w13_s, nullptr, 0}, dxp, ws,
                     ws_bytes, stream);
}

int moe_grouped_gemm_w2_backward_nvfp4(const moe_dims* d, const uint16_t* dy2,
                                       const int32_t* group_offsets, const uint8_t* w2,
                                       const uint8_t* w2_s, const float* w2_gs, uint16_t* dh,
                                       void* ws, size_t ws_bytes, void* stream) {
  if (!d) return MOE_ERR_UNSUPPORTED_SHAPE;
  return expert_grad(d, d->H, d->I, dy2, group_offsets, {w2, w2_s, w2_gs, 1}, dh, ws, ws_bytes,
                     stream);
}

int moe_grouped_gemm_w13_backward_nvfp4(const moe_dims* d, const uint16_t* dy13,
                                        const int32_t* group_offsets, const uint8_t* w13,
                                        const uint8_t* w13_s, const float* w13_gs, uint16_t* dxp,
                                        void* ws, size_t ws_bytes, void* stream) {
  if (!d || d->I > (1 << 29)) return MOE_ERR_UNSUPPORTED_SHAPE;
  return expert_grad(d, 2 * d->I, d->H, dy13, group_offsets, {w13, w13_s, w13_gs, 2}, dxp, ws,
                     ws_bytes, stream);
}

int moe_gemm_backward_ctas(const moe_dims* d, int32_t product) {
  if (!dims_ok(d) || d->I > (1 << 29) || (product != 2 && product != 13)) return 0;
  return expert_grad_ctas(product == 2 ? sizes_of(d, d->H, d->I) : sizes_of(d, 2 * d->I, d->H));
}

int moe_gemm_backward_form(const moe_dims* d, int32_t product, int32_t nvfp4, int32_t ctas,
                           const uint16_t* dy, const int32_t* group_offsets, const uint8_t* w,
                           const uint8_t* w_s, const float* gs, uint16_t* dx, void* ws,
                           size_t ws_bytes, void* stream) {
  if (!d || d->I > (1 << 29)) return MOE_ERR_UNSUPPORTED_SHAPE;
  if ((product != 2 && product != 13) || (nvfp4 != 0 && nvfp4 != 1) || (ctas != 1 && ctas != 2) ||
      (gs && !nvfp4))
    return MOE_ERR_INVALID_ARG;
  const bool two = product == 2;
  const GradWeights W = {w, w_s, gs, !nvfp4 ? 0 : two ? 1 : 2};
  return expert_grad(d, two ? d->H : 2 * d->I, two ? d->I : d->H, dy, group_offsets, W, dx, ws,
                     ws_bytes, stream, ctas);
}

}  // extern "C"
