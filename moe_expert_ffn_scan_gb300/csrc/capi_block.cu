// C interface (include/moe.h) of the operators around the expert FFN: argument checks,
// workspace carving and launches.  No allocation, no host synchronisation.
#include "block.cuh"

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
constexpr int kMaxCols = 1 << 30;    // and in the norm's column arithmetic

bool balance_ok(int T, int E, int k, int S) {
  return T >= 0 && T <= kMaxTokens && E >= 1 && E <= 1024 && k >= 1 && k <= 16 && k <= E &&
         S >= 1 && S <= 65535 && static_cast<long long>(T) * k < (1LL << 31);
}

BalanceWs carve_balance(Carver& c, int T, int E, int S) {
  BalanceWs w;
  const size_t ctas = balance_ctas_most(T, E), slots = ctas + S - 1;
  w.status = c.take<uint32_t>(64);
  w.flags = c.take<uint32_t>(ctas);
  w.p = c.take<float>(slots * E);
  w.c = c.take<int32_t>(slots * E);
  w.z = c.take<float>(slots);
  w.n = c.take<int32_t>(slots);
  w.acc = c.take<unsigned long long>(S);
  w.terms = c.take<float>(static_cast<size_t>(S) * ((E + 31) / 32));
  return w;
}

// Row strides with their defaults (0: contiguous).  One row: any stride does.
struct LinearLd {
  long long x, w, r, y, z;
};
LinearLd linear_ld(const moe_linear_desc* d) {
  LinearLd l = {d->ldx ? d->ldx : d->K, d->ldw ? d->ldw : d->K, d->ldr ? d->ldr : d->N,
                d->ldy ? d->ldy : d->N, d->ldz ? d->ldz : d->N};
  if (d->M == 1) {
    l.x = linear_padded(d->K);
    l.r = l.y = l.z = linear_padded(d->N);
  }
  if (d->N == 1) l.w = linear_padded(d->K);
  return l;
}

bool linear_ok(const moe_linear_desc* d) {
  if (!d || d->M < 0 || d->N < 1 || d->K < 1) return false;
  const long long most = 1LL << 36;  // elements: TMA strides and tile counts stay in range
  if (d->M > kMaxTokens || d->N > (1 << 22) || d->K > (1 << 22)) return false;
  if (static_cast<long long>(d->M) * d->N > most || static_cast<long long>(d->M) * d->K > most)
    return false;
  const LinearLd l = linear_ld(d);
  return l.x >= d->K && l.w >= d->K && l.r >= d->N && l.y >= d->N && l.z >= d->N &&
         l.x < most && l.w < most && l.r < most && l.y < most && l.z < most;
}

struct LinearWs {
  uint32_t* status;
  uint16_t *x_pad, *w_pad, *dz;
  float* part;
};

LinearWs carve_linear(Carver& c, const moe_linear_desc* d, bool backward) {
  LinearWs w = {};
  const LinearLd l = linear_ld(d);
  w.status = c.take<uint32_t>(64);
  if (l.x % 8) w.x_pad = c.take<uint16_t>(static_cast<size_t>(d->M) * linear_padded(d->K));
  if (l.w % 8) w.w_pad = c.take<uint16_t>(static_cast<size_t>(d->N) * linear_padded(d->K));
  if (backward) {
    if (d->act != MOE_ACT_NONE || l.y % 8)
      w.dz = c.take<uint16_t>(static_cast<size_t>(d->M) * linear_padded(d->N));
    w.part = c.take<float>(static_cast<size_t>(kLinearDbParts) * d->N);
  }
  return w;
}

bool linear_args_ok(const moe_linear_desc* d) {
  return d->act >= MOE_ACT_NONE && d->act <= MOE_ACT_GELU && dtype_ok(d->y_dtype) &&
         dtype_ok(d->bias_dtype);
}

}  // namespace

extern "C" {

size_t moe_linear_workspace_size(const moe_linear_desc* d) {
  if (!linear_ok(d)) return 0;
  Carver c(nullptr);
  carve_linear(c, d, false);
  return c.used;
}

int moe_linear(const moe_linear_desc* d, const uint16_t* x, const uint16_t* w, const void* bias,
               const void* residual, void* y, uint16_t* z, void* ws, size_t ws_bytes,
               void* stream) {
  if (!linear_ok(d)) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (!linear_args_ok(d)) return MOE_ERR_INVALID_ARG;
  if (d->M == 0) return MOE_OK;
  if (!x || !w || !y || !ws || !aligned(x, 16) || !aligned(w, 16) || !null_or(bias, 4) ||
      !null_or(residual, 16) || !aligned(y, 16) || !null_or(z, 16) || !aligned(ws, kAlign))
    return MOE_ERR_INVALID_ARG;
  Carver c(ws);
  const LinearWs s = carve_linear(c, d, false);
  if (ws_bytes < c.used) return MOE_ERR_WORKSPACE_TOO_SMALL;
  const LinearLd l = linear_ld(d);
  LinearCall a = {};
  a.M = d->M, a.N = d->N, a.K = d->K, a.act = d->act;
  a.x = x, a.w = w, a.bias = bias, a.res = residual, a.y = y, a.z = z;
  a.ldx = l.x, a.ldw = l.w, a.ldr = l.r, a.ldy = l.y, a.ldz = l.z;
  a.bias_f32 = d->bias_dtype == MOE_DTYPE_F32;
  a.y_f32 = d->y_dtype == MOE_DTYPE_F32;
  a.x_pad = s.x_pad, a.w_pad = s.w_pad, a.status = s.status;
  return cuda_rc(launch_linear(a, static_cast<cudaStream_t>(stream)));
}

size_t moe_linear_backward_workspace_size(const moe_linear_desc* d) {
  if (!linear_ok(d)) return 0;
  Carver c(nullptr);
  carve_linear(c, d, true);
  return c.used;
}

int moe_linear_backward(const moe_linear_desc* d, const uint16_t* x, const uint16_t* w,
                        const uint16_t* z, const uint16_t* dy, uint16_t* dx, uint16_t* dw,
                        float* dbias, void* ws, size_t ws_bytes, void* stream) {
  if (!linear_ok(d)) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (!linear_args_ok(d) || (!dx && !dw && !dbias)) return MOE_ERR_INVALID_ARG;
  if (d->M > 0 && (!dy || (dx && !w) || (dw && !x) || (d->act != MOE_ACT_NONE && !z)))
    return MOE_ERR_INVALID_ARG;
  if (!ws || !aligned(ws, kAlign) || !null_or(x, 16) || !null_or(w, 16) || !null_or(z, 16) ||
      !null_or(dy, 16) || !null_or(dx, 16) || !null_or(dw, 16) || !null_or(dbias, 4))
    return MOE_ERR_INVALID_ARG;
  Carver c(ws);
  const LinearWs s = carve_linear(c, d, true);
  if (ws_bytes < c.used) return MOE_ERR_WORKSPACE_TOO_SMALL;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (d->M == 0) {  // sums over no rows
    if (dw && cudaMemsetAsync(dw, 0, static_cast<size_t>(d->N) * d->K * 2, st) != cudaSuccess)
      return MOE_ERR_CUDA;
    if (dbias && cudaMemsetAsync(dbias, 0, static_cast<size_t>(d->N) * 4, st) != cudaSuccess)
      return MOE_ERR_CUDA;
    return MOE_OK;
  }
  const LinearLd l = linear_ld(d);
  LinearBwdCall a = {};
  a.M = d->M, a.N = d->N, a.K = d->K, a.act = d->act;
  a.x = x, a.w = w, a.z = z, a.dy = dy, a.dx = dx, a.dw = dw, a.db = dbias;
  a.ldx = l.x, a.ldw = l.w, a.ldz = l.z, a.lddy = l.y, a.lddx = d->K, a.lddw = d->K;
  // without the products only the sums are wanted
  a.dz = dx || dw ? s.dz : nullptr;
  a.part = dbias ? s.part : nullptr;
  a.x_pad = s.x_pad, a.w_pad = s.w_pad, a.status = s.status;
  return cuda_rc(launch_linear_bwd(a, st));
}

int moe_add_rmsnorm(int32_t rows, int32_t cols, const uint16_t* x, const void* residual,
                    int32_t res_dtype, const void* gain, int32_t gain_dtype, float eps, void* h,
                    uint16_t* y, uint8_t* q, uint8_t* s, float* rstd, void* stream) {
  if (rows < 0 || cols < 1 || cols > kMaxCols) return MOE_ERR_UNSUPPORTED_SHAPE;
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
  if (rows < 0 || cols < 1 || cols > kMaxCols) return 0;
  const size_t parts = norm_bwd_parts(rows, cols);
  return kAlign + align_up(parts * static_cast<size_t>(cols) * sizeof(float));
}

int moe_add_rmsnorm_backward(int32_t rows, int32_t cols, const uint16_t* dy, const void* h,
                             int32_t h_dtype, const void* gain, int32_t gain_dtype,
                             const float* rstd, const void* dh_in, void* dh, uint16_t* dx,
                             float* dgain, void* ws, size_t ws_bytes, void* stream) {
  if (rows < 0 || cols < 1 || cols > kMaxCols) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (!dtype_ok(h_dtype) || !dtype_ok(gain_dtype)) return MOE_ERR_INVALID_ARG;
  if (!dh && !dx && !dgain) return MOE_ERR_INVALID_ARG;
  if (rows > 0 && (!dy || !h || !gain || !rstd)) return MOE_ERR_INVALID_ARG;
  if (!null_or(dy, 16) || !null_or(h, 16) || !null_or(gain, 16) || !null_or(rstd, 4) ||
      !null_or(dh_in, 16) || !null_or(dh, 16) || !null_or(dx, 16) || !null_or(dgain, 4))
    return MOE_ERR_INVALID_ARG;
  float* part = nullptr;
  if (dgain) {
    if (!ws || !aligned(ws, kAlign)) return MOE_ERR_INVALID_ARG;
    if (ws_bytes < moe_add_rmsnorm_backward_workspace_size(rows, cols))
      return MOE_ERR_WORKSPACE_TOO_SMALL;
    // behind the first 256 bytes, a status word's place in every other workspace (which the
    // binding's allocation clears on the stream that is current there)
    part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kAlign);
  }
  return cuda_rc(launch_add_rmsnorm_bwd(dy, h, h_dtype == MOE_DTYPE_F32, gain,
                                        gain_dtype == MOE_DTYPE_F32, rstd, rows, cols, dh_in, dh,
                                        dx, dgain, part, static_cast<cudaStream_t>(stream)));
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
