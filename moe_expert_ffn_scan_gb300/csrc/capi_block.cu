// C interface (include/moe.h) of the operators around the expert FFN: argument checks,
// workspace carving and launches.  No allocation, no host synchronisation.
#include "kernels.cuh"

using namespace moe;

namespace {

constexpr size_t kAlign = 256;

size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// A pointer that may be null.
bool null_or(const void* p, size_t a) { return !p || aligned(p, a); }

bool dtype_ok(int t) { return t == MOE_DTYPE_BF16 || t == MOE_DTYPE_F32; }

int cuda_rc(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

// Bump allocator over a caller-provided workspace (or a size counter when base is null).
struct Carver {
  uint8_t* base;
  size_t used = 0;
  explicit Carver(void* b) : base(static_cast<uint8_t*>(b)) {}
  template <typename T>
  T* take(size_t count) {
    const size_t off = used;
    used = align_up(used + count * sizeof(T));
    return base ? reinterpret_cast<T*>(base + off) : nullptr;
  }
};

constexpr int kMaxTokens = 1 << 30;  // leaves room in 32-bit row arithmetic

bool balance_ok(int T, int E, int k, int S) {
  return T >= 0 && T <= kMaxTokens && E >= 1 && E <= 1024 && k >= 1 && k <= 16 && k <= E &&
         S >= 1 && S <= 65535 && static_cast<long long>(T) * k < (1LL << 31);
}

BalanceWs carve_balance(Carver& c, int T, int E, int S) {
  BalanceWs w;
  const size_t slots = static_cast<size_t>(balance_ctas(T)) + S - 1;
  w.status = c.take<uint32_t>(64);
  w.flags = c.take<uint32_t>(balance_ctas(T));
  w.p = c.take<float>(slots * E);
  w.c = c.take<int32_t>(slots * E);
  w.z = c.take<float>(slots);
  w.n = c.take<int32_t>(slots);
  w.ticket = c.take<int32_t>(S);
  w.terms = c.take<float>(static_cast<size_t>(S) * ((E + 31) / 32));
  return w;
}

}  // namespace

extern "C" {

int moe_add_rmsnorm(int32_t rows, int32_t cols, const uint16_t* x, const void* residual,
                    int32_t res_dtype, const void* gain, int32_t gain_dtype, float eps, void* h,
                    uint16_t* y, uint8_t* q, uint8_t* s, float* rstd, void* stream) {
  if (rows < 0 || cols < 1) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (q && cols % 128) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (!dtype_ok(res_dtype) || !dtype_ok(gain_dtype) || !(eps >= 0.f)) return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  if (!x || !gain || (!h && !y && !q) || (q == nullptr) != (s == nullptr))
    return MOE_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !null_or(residual, 16) || !aligned(gain, 16) || !null_or(h, 16) ||
      !null_or(y, 16) || !null_or(q, 16) || !null_or(rstd, 4))
    return MOE_ERR_INVALID_ARG;
  return cuda_rc(launch_add_rmsnorm(x, residual, res_dtype == MOE_DTYPE_F32, gain,
                                    gain_dtype == MOE_DTYPE_F32, eps, rows, cols, h, y, q, s,
                                    rstd, static_cast<cudaStream_t>(stream)));
}

size_t moe_add_rmsnorm_backward_workspace_size(int32_t rows, int32_t cols) {
  if (rows < 0 || cols < 1) return 0;
  const size_t parts = rows < kNormBwdCtas ? (rows > 0 ? rows : 1) : kNormBwdCtas;
  return align_up(parts * static_cast<size_t>(cols) * sizeof(float));
}

int moe_add_rmsnorm_backward(int32_t rows, int32_t cols, const uint16_t* dy, const void* h,
                             int32_t h_dtype, const void* gain, int32_t gain_dtype,
                             const float* rstd, const void* dh_in, void* dh, uint16_t* dx,
                             float* dgain, void* ws, size_t ws_bytes, void* stream) {
  if (rows < 0 || cols < 1) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (!dtype_ok(h_dtype) || !dtype_ok(gain_dtype)) return MOE_ERR_INVALID_ARG;
  if (!dh && !dx && !dgain) return MOE_ERR_INVALID_ARG;
  if (rows > 0 && (!dy || !h || !gain || !rstd)) return MOE_ERR_INVALID_ARG;
  if (!null_or(dy, 16) || !null_or(h, 16) || !null_or(gain, 16) || !null_or(rstd, 4) ||
      !null_or(dh_in, 16) || !null_or(dh, 16) || !null_or(dx, 16) || !null_or(dgain, 4))
    return MOE_ERR_INVALID_ARG;
  if (dgain) {
    if (!ws || !aligned(ws, kAlign)) return MOE_ERR_INVALID_ARG;
    if (ws_bytes < moe_add_rmsnorm_backward_workspace_size(rows, cols))
      return MOE_ERR_WORKSPACE_TOO_SMALL;
  }
  return cuda_rc(launch_add_rmsnorm_bwd(dy, h, h_dtype == MOE_DTYPE_F32, gain,
                                        gain_dtype == MOE_DTYPE_F32, rstd, rows, cols, dh_in, dh,
                                        dx, dgain, static_cast<float*>(ws),
                                        static_cast<cudaStream_t>(stream)));
}

size_t moe_balance_loss_workspace_size(int32_t T, int32_t E, int32_t k, int32_t S) {
  if (!balance_ok(T, E, k, S)) return 0;
  Carver c(nullptr);
  carve_balance(c, T, E, S);
  return c.used;
}

int moe_balance_loss(int32_t T, int32_t E, int32_t k, int32_t S, const float* logits,
                     const int32_t* idx, const int32_t* seq_offsets, const uint8_t* token_mask,
                     int32_t* counts, int32_t* n_tokens, float* prob, float* loss, float* z_loss,
                     void* ws, size_t ws_bytes, void* stream) {
  if (!balance_ok(T, E, k, S)) return MOE_ERR_UNSUPPORTED_SHAPE;
  if ((T > 0 && (!logits || !idx)) || (S > 1 && !seq_offsets) || !counts || !n_tokens || !prob ||
      !loss || !ws)
    return MOE_ERR_INVALID_ARG;
  if (!null_or(logits, 16) || !null_or(idx, 4) || !null_or(seq_offsets, 4) ||
      !aligned(counts, 4) || !aligned(n_tokens, 4) || !aligned(prob, 4) || !aligned(loss, 4) ||
      !null_or(z_loss, 4) || !aligned(ws, kAlign))
    return MOE_ERR_INVALID_ARG;
  Carver c(ws);
  const BalanceWs w = carve_balance(c, T, E, S);
  if (ws_bytes < c.used) return MOE_ERR_WORKSPACE_TOO_SMALL;
  return cuda_rc(launch_balance_loss(logits, idx, seq_offsets, token_mask, T, E, k, S, w, counts,
                                     n_tokens, prob, loss, z_loss,
                                     static_cast<cudaStream_t>(stream)));
}

int moe_balance_loss_backward(int32_t T, int32_t E, int32_t k, int32_t S, const float* logits,
                              const int32_t* idx, const int32_t* seq_offsets,
                              const uint8_t* token_mask, const int32_t* counts,
                              const int32_t* n_tokens, const float* dloss, const float* dz_loss,
                              const float* dw, float* dlogits, void* stream) {
  if (!balance_ok(T, E, k, S)) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (T == 0) return MOE_OK;
  if (!logits || !idx || (S > 1 && !seq_offsets) || !counts || !n_tokens || !dlogits)
    return MOE_ERR_INVALID_ARG;
  if (!aligned(logits, 16) || !aligned(idx, 4) || !null_or(seq_offsets, 4) ||
      !aligned(counts, 4) || !aligned(n_tokens, 4) || !null_or(dloss, 4) ||
      !null_or(dz_loss, 4) || !null_or(dw, 4) || !aligned(dlogits, 16))
    return MOE_ERR_INVALID_ARG;
  return cuda_rc(launch_balance_bwd(logits, idx, seq_offsets, token_mask, counts, n_tokens, dloss,
                                    dz_loss, dw, T, E, k, S, dlogits,
                                    static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
