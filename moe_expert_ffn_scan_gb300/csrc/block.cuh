// Shared by the operators around the expert FFN (norm.cu, balance.cu, linear.cu and their C
// interface, capi_block.cu): device helpers beyond common.cuh's and launch declarations.
#pragma once

#include "context_once.cuh"
#include "kernels.cuh"

namespace moe {

// SMs of a GB300.  Grids and cost models go by it (results do not).
constexpr int kSms = 152;

// ------------------------------------------------------------------ cp.async ------

// 16 bytes into shared memory, asynchronously and past L1.
__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src)
               : "memory");
}
__device__ __forceinline__ void cp_async4(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// ------------------------------------------------------------------ tcgen05, TMA --

// kind::f16 MMA (bf16 x bf16 -> fp32) of an SM pair: M = 256 over its two CTAs.
__device__ __forceinline__ void mma_bf16_ss_pair(uint32_t d_tmem, uint64_t a_desc,
                                                 uint64_t b_desc, uint32_t idesc,
                                                 uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Each thread of the warp reads 8 consecutive 32-bit columns of its own TMEM lane ...
__device__ __forceinline__ void tmem_ld_32x32b_x8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7])
      : "r"(taddr)
      : "memory");
}

// ... or 32 of them.
__device__ __forceinline__ void tmem_ld_32x32b_x32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32"
      " {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15,"
      "  %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
        "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
        "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]),
        "=r"(r[31])
      : "r"(taddr)
      : "memory");
}

// A 2D tile whose completion is counted on an mbarrier of either CTA of the pair (bar: a
// shared::cluster address).
__device__ __forceinline__ void tma_load_2d_pair(void* dst, const CUtensorMap* m, uint32_t bar,
                                                 int32_t c0, int32_t c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(c0), "r"(c1)
      : "memory");
}

// A float of another CTA's shared memory (addr: a shared::cluster address).
__device__ __forceinline__ float ld_shared_cluster(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

// ------------------------------------------------------------------ launches ------

// Residual addition + RMS norm and its gradient (norm.cu).  part: the dgain partials,
// [norm_bwd_parts(rows, cols)][cols] fp32 (not read when dgain is null).
int norm_bwd_parts(int rows, int cols);
cudaError_t launch_add_rmsnorm(const uint16_t* x, const void* res, bool res_f32, const void* gain,
                               bool gain_f32, float eps, int rows, int cols, void* h, uint16_t* y,
                               uint8_t* q, uint8_t* s, float* rstd, cudaStream_t st);
cudaError_t launch_add_rmsnorm_bwd(const uint16_t* dy, const void* h, bool h_f32, const void* gain,
                                   bool gain_f32, const float* rstd, int rows, int cols,
                                   const void* dh_in, void* dh, uint16_t* dx, float* dgain,
                                   float* part, cudaStream_t st);

// out[c] = sum over `parts` rows of part[.][cols], in a fixed order (norm.cu).
cudaError_t launch_column_sum(const float* part, int parts, int cols, float* out,
                              cudaStream_t st);

// Dense projection and its gradient (linear.cu).  Row strides in elements.  x_pad / w_pad
// are non-null where that operand's rows are not whole 16-byte vectors: room for a copy
// with rows of linear_padded(columns).
inline long long linear_padded(int cols) { return (static_cast<long long>(cols) + 7) / 8 * 8; }
struct LinearCall {
  int M, N, K, act;
  const uint16_t *x, *w;
  const void *bias, *res;
  void* y;
  uint16_t* z;
  long long ldx, ldw, ldr, ldy, ldz;
  int bias_f32, y_f32;  // the residual has y's type
  uint16_t *x_pad, *w_pad;
  uint32_t* status;
};
cudaError_t launch_linear(const LinearCall& a, cudaStream_t st);
constexpr int kLinearDbParts = 256;  // row blocks of the bias gradient's partial sums
struct LinearBwdCall {
  int M, N, K, act;
  const uint16_t *x, *w, *z, *dy;
  long long ldx, ldw, ldz, lddy, lddx, lddw;
  uint16_t *dx, *dw;  // or null
  float* db;          // or null
  uint16_t* dz;       // [M][linear_padded(N)] where dy itself is not the products' operand
  float* part;        // [kLinearDbParts][N] with db
  uint16_t *x_pad, *w_pad;
  uint32_t* status;
};
cudaError_t launch_linear_bwd(const LinearBwdCall& a, cudaStream_t st);

// Router balance loss and its gradient (balance.cu).  The forward's first kernel runs
// balance_ctas(T, E) <= kBalanceCtas CTAs and writes one partial slot per (CTA, sequence)
// pair that has rows: balance_ctas(T, E) + S - 1 slots.  That count falls by some CTAs
// wherever the rows of a CTA become one more; workspaces have balance_ctas_most(T, E), which
// never falls: one made for the longest step does for every shorter one.
constexpr int kBalanceCtas = 2 * kSms;
struct BalanceWs {
  uint32_t* status;
  uint32_t* flags;   // [balance_ctas_most(T, E)] status bits, by CTA
  float* p;          // [slots][E] sums of p
  int32_t* c;        // [slots][E] counts
  float* z;          // [slots]
  int32_t* n;        // [slots] counted tokens
  unsigned long long* acc;  // [S] loss sums and arrivals
  float* terms;             // [S][E / 32, rounded up] the loss terms too small for acc
};
int balance_ctas(int T, int E);
int balance_ctas_most(int T, int E);
cudaError_t launch_balance_loss(const float* logits, const int32_t* idx, const int32_t* off,
                                const uint8_t* mask, int T, int E, int k, int S,
                                const BalanceWs& w, int32_t* counts, int32_t* n_tokens,
                                float* prob, float* loss, float* z_loss, cudaStream_t st);
cudaError_t launch_balance_bwd(const float* logits, const int32_t* idx, const int32_t* off,
                               const uint8_t* mask, const int32_t* counts,
                               const int32_t* n_tokens, const float* dloss, const float* dz,
                               const float* dw, int T, int E, int k, int S, float* dlogits,
                               cudaStream_t st);

// Lets `kern` take all of a CTA's shared memory that its static arrays leave (at most 1 KB),
// once per context.
constexpr int kSmemMax = 226 * 1024;
template <auto kern>
cudaError_t allow_smem() {
  static OncePerContext once;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= OncePerContext::kDevices) return cudaErrorInvalidDevice;
  if (once.ready(dev, current_context_id())) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax);
  if (e == cudaSuccess) once.set(dev, 0);
  return e;
}

}  // namespace moe
