// Router balance loss with per-expert counts, and the gradient of the logits.
//
// Per sequence s of n counted tokens, p = softmax(logits) over the E experts:
//   count_e = tokens that chose e,  P_e = mean of p_te,  f_e = count_e * E / (k * n),
//   loss = sum_e f_e * P_e,  z = mean of logsumexp(logits_t)^2.
// Gradient (counts are constants), with A_e = dloss * E * count_e / (k * n^2):
//   dlogit_te = p_te * (A_e - sum_j A_j p_tj) + p_te * 2 dz * lse_t / n
//   and for the chosen experts j of the token: += w_j * (dw_j - sum_i w_i dw_i),
//   w = softmax over the chosen logits (moe_route's combine weights).
//
// One pass over the logits: a warp holds a token's E logits in registers (E <= 1024), so
// the maximum, the sum, the probabilities and their products are register work; both
// directions are bound by reading (and in the gradient writing) T x E fp32 values.
// No floating-point atomics: partial sums are added in a fixed order.
#include "kernels.cuh"

namespace moe {

namespace {

constexpr int kWarps = 8;  // per CTA

// A lane's experts: VEC consecutive ones from lane * VEC + i * 32 * VEC.  Missing experts
// read as -inf (probability 0).
template <int NV, int VEC>
struct Row {
  float v[NV][VEC];
  __device__ __forceinline__ static int at(int lane, int i) { return (i * 32 + lane) * VEC; }
  __device__ __forceinline__ void load(const float* p, int E, int lane) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = at(lane, i);
      if constexpr (VEC == 4) {
        float4 f = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
        if (e < E) f = __ldg(reinterpret_cast<const float4*>(p + e));
        v[i][0] = f.x, v[i][1] = f.y, v[i][2] = f.z, v[i][3] = f.w;
      } else {
        v[i][0] = e < E ? __ldg(p + e) : -INFINITY;
      }
    }
  }
  // v becomes the probabilities; returns logsumexp.  A row of -inf alone has no
  // probabilities: zeros, and 0 for its logsumexp.
  __device__ __forceinline__ float softmax() {
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) m = fmaxf(m, v[i][j]);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, off));
    // (a NaN does not reach m, but its exp below does reach the sum)
    const bool none = m == -INFINITY;
    if (none) m = 0.f;
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        v[i][j] = expf(v[i][j] - m);
        sum += v[i][j];
      }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, off);
    if (none && sum == 0.f) return 0.f;
    const float r = 1.f / sum;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[i][j] *= r;
    return m + logf(sum);
  }
};

// Offsets come from memory: read with their bounds (0 <= off <= T).
__device__ __forceinline__ int seq_off(const int32_t* off, int s, int S, int T) {
  if (!off) return s == 0 ? 0 : T;
  const int v = __ldg(off + s);
  return v < 0 ? 0 : v > T ? T : v;
}

// The last sequence s with off[s] <= t (0 if there is none).
__device__ __forceinline__ int seq_of(const int32_t* off, int S, int T, int t) {
  int lo = 0, hi = S - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (seq_off(off, mid, S, T) <= t) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// One CTA sums rows [blockIdx.x * per, + per), for each sequence s that has some of them
// into partial slot blockIdx.x + s.  (Walking the (CTA, sequence) pairs in order, each step
// raises one of the two, so the slots differ; there are CTAs + S - 1 of them.)
template <int NV, int VEC>
__global__ void __launch_bounds__(kWarps * 32)
    k_balance_partial(const float* __restrict__ logits, const int32_t* __restrict__ idx,
                      const int32_t* __restrict__ off, const uint8_t* __restrict__ mask, int T,
                      int E, int k, int S, int per, float* __restrict__ part_p,
                      int32_t* __restrict__ part_c, float* __restrict__ part_z,
                      int32_t* __restrict__ part_n, int32_t* __restrict__ ticket,
                      uint32_t* __restrict__ flags) {
  pdl_wait();
  pdl_trigger();
  extern __shared__ float dyn[];  // [kWarps][E] sums of p, then [E] counts
  __shared__ float zs[kWarps];
  __shared__ int ns[kWarps];
  int32_t* hist = reinterpret_cast<int32_t*>(dyn + kWarps * E);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // the arrival counters of the kernel after this one
  for (int s = blockIdx.x * blockDim.x + threadIdx.x; s < S; s += gridDim.x * blockDim.x)
    ticket[s] = 0;
  const int begin = blockIdx.x * per, end = T - begin < per ? T : begin + per;
  int row = begin;
  uint32_t bad = 0;  // data-dependent checks of this thread (STATUS_*)
  for (int s = seq_of(off, S, T, begin); s < S && row < end; ++s) {
    const int sb = seq_off(off, s, S, T), se = seq_off(off, s + 1, S, T);
    if (se < sb) bad |= STATUS_BAD_PLAN;
    const int r0 = sb > row ? sb : row, r1 = se < end ? se : end;
    if (r0 >= r1) continue;  // (the same for the whole CTA)
    row = r1;
    for (int e = threadIdx.x; e < E; e += blockDim.x) hist[e] = 0;
    __syncthreads();
    float acc[NV][VEC];
    float z = 0.f;
    int n = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) acc[i][j] = 0.f;
    for (int r = r0 + warp; r < r1; r += kWarps) {
      if (mask && !__ldg(mask + r)) continue;
      Row<NV, VEC> x;
      x.load(logits + static_cast<size_t>(r) * E, E, lane);
      if (lane < k) {
        const int e = __ldg(idx + static_cast<size_t>(r) * k + lane);
        if (static_cast<unsigned>(e) < static_cast<unsigned>(E)) atomicAdd(hist + e, 1);
        else bad |= STATUS_BAD_INDEX;
      }
      const float lse = x.softmax();
      z = fmaf(lse, lse, z);
      ++n;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j) acc[i][j] += x.v[i][j];
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const int e = Row<NV, VEC>::at(lane, i) + j;
        if (e < E) dyn[warp * E + e] = acc[i][j];
      }
    if (lane == 0) zs[warp] = z, ns[warp] = n;
    __syncthreads();
    const size_t slot = static_cast<size_t>(blockIdx.x) + s;
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) v += dyn[w * E + e];
      part_p[slot * E + e] = v;
      part_c[slot * E + e] = hist[e];
    }
    if (threadIdx.x == 0) {
      float zt = 0.f;
      int nt = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) zt += zs[w], nt += ns[w];
      part_z[slot] = zt;
      part_n[slot] = nt;
    }
    __syncthreads();
  }
  const int plan = __syncthreads_or(bad & STATUS_BAD_PLAN);
  const int index = __syncthreads_or(bad & STATUS_BAD_INDEX);
  if (threadIdx.x == 0)
    flags[blockIdx.x] = (plan ? STATUS_BAD_PLAN : 0u) | (index ? STATUS_BAD_INDEX : 0u);
}

// Adds up the partials of sequence blockIdx.y for 32 experts; warp w takes the slots
// first + w, + 32, ... and the warps' sums are added in order.  The CTA that finishes its
// sequence last adds the CTAs' loss terms, in CTA order.
__global__ void __launch_bounds__(1024)
    k_balance_final(const int32_t* __restrict__ off, int T, int E, int k, int S, int per,
                    const float* __restrict__ part_p, const int32_t* __restrict__ part_c,
                    const float* __restrict__ part_z, const int32_t* __restrict__ part_n,
                    int32_t* ticket, float* terms, int32_t* __restrict__ counts,
                    int32_t* __restrict__ n_tokens, float* __restrict__ prob,
                    float* __restrict__ loss, float* __restrict__ z_loss,
                    const uint32_t* __restrict__ flags, int nflags, uint32_t* status) {
  pdl_wait();
  pdl_trigger();
  __shared__ float rp[32][33];
  __shared__ int rc[32][33];
  __shared__ float rz[32];
  __shared__ int rn[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int s = blockIdx.y, e = blockIdx.x * 32 + lane;
  if (blockIdx.x == 0 && s == 0) {  // the call's status word (nflags <= 1024)
    const uint32_t f = static_cast<int>(threadIdx.x) < nflags ? flags[threadIdx.x] : 0u;
    const int plan = __syncthreads_or(f & STATUS_BAD_PLAN);
    const int index = __syncthreads_or(f & STATUS_BAD_INDEX);
    if (threadIdx.x == 0)
      *status = (plan ? STATUS_BAD_PLAN : 0u) | (index ? STATUS_BAD_INDEX : 0u);
  }
  const int sb = seq_off(off, s, S, T), se = seq_off(off, s + 1, S, T);
  const int first = sb / per, last = se > sb ? (se - 1) / per : first - 1;  // CTAs
  float p = 0.f;
  int c = 0;
  if (e < E) {
#pragma unroll 4
    for (int b = first + warp; b <= last; b += 32) {
      const size_t slot = static_cast<size_t>(b) + s;
      p += part_p[slot * E + e];
      c += part_c[slot * E + e];
    }
  }
  // token count and z: every CTA needs the first, lane by lane over the slots
  float z = 0.f;
  int n = 0;
  for (int b = first + static_cast<int>(threadIdx.x); b <= last; b += 1024) {
    z += part_z[static_cast<size_t>(b) + s];
    n += part_n[static_cast<size_t>(b) + s];
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    z += __shfl_xor_sync(0xFFFFFFFFu, z, o);
    n += __shfl_xor_sync(0xFFFFFFFFu, n, o);
  }
  rp[warp][lane] = p;
  rc[warp][lane] = c;
  if (lane == 0) rz[warp] = z, rn[warp] = n;
  __syncthreads();
  if (warp != 0) return;
  p = 0.f, z = 0.f;
  c = 0, n = 0;
#pragma unroll
  for (int w = 0; w < 32; ++w) {
    p += rp[w][lane];
    c += rc[w][lane];
    z += rz[w];
    n += rn[w];
  }
  const float inv = n > 0 ? 1.f / static_cast<float>(n) : 0.f;
  p *= inv;
  if (e < E) {
    prob[static_cast<size_t>(s) * E + e] = p;
    counts[static_cast<size_t>(s) * E + e] = c;
  }
  float term = static_cast<float>(c) * inv * p;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) term += __shfl_xor_sync(0xFFFFFFFFu, term, o);
  if (blockIdx.x == 0 && lane == 0) {
    n_tokens[s] = n;
    if (z_loss) z_loss[s] = z * inv;
  }
  int done = 0;
  if (lane == 0) {
    terms[static_cast<size_t>(s) * gridDim.x + blockIdx.x] = term;
    __threadfence();
    done = atomicAdd(ticket + s, 1) == static_cast<int>(gridDim.x) - 1;
    __threadfence();
  }
  if (!__shfl_sync(0xFFFFFFFFu, done, 0)) return;
  float sum = 0.f;  // (gridDim.x <= 32)
  if (lane < static_cast<int>(gridDim.x))
    sum = __ldcg(terms + static_cast<size_t>(s) * gridDim.x + lane);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
  if (lane == 0) loss[s] = sum * (static_cast<float>(E) / static_cast<float>(k));
}

template <int NV, int VEC>
__global__ void __launch_bounds__(kWarps * 32)
    k_balance_bwd(const float* __restrict__ logits, const int32_t* __restrict__ idx,
                  const int32_t* __restrict__ off, const uint8_t* __restrict__ mask,
                  const int32_t* __restrict__ counts, const int32_t* __restrict__ n_tokens,
                  const float* __restrict__ dloss, const float* __restrict__ dz,
                  const float* __restrict__ dw, int T, int E, int k, int S, int per,
                  float* __restrict__ dlogits) {
  pdl_wait();
  pdl_trigger();
  extern __shared__ float dyn[];  // [kWarps][E]: the chosen experts' terms of the warp's row
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float* mine = dyn + warp * E;
  if (dw) {
    for (int e = lane; e < E; e += 32) mine[e] = 0.f;
    __syncwarp();
  }
  // a warp takes `per` consecutive rows, so that its sequence seldom changes
  const long long first = (static_cast<long long>(blockIdx.x) * kWarps + warp) * per;
  const int r0 = first < T ? static_cast<int>(first) : T;
  const int r1 = T - r0 < per ? T : r0 + per;
  if (r0 >= r1) return;
  int s = seq_of(off, S, T, r0), have = -1;
  float a[NV][VEC];
  float zc = 0.f;
  for (int r = r0; r < r1; ++r) {
    while (s + 1 < S && seq_off(off, s + 1, S, T) <= r) ++s;
    float* out = dlogits + static_cast<size_t>(r) * E;
    const bool counted = (!mask || __ldg(mask + r)) && seq_off(off, s, S, T) <= r &&
                         r < seq_off(off, s + 1, S, T);
    Row<NV, VEC> x;
    if (!counted) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j) x.v[i][j] = 0.f;
    } else {
      x.load(logits + static_cast<size_t>(r) * E, E, lane);
      if (have != s) {
        have = s;
        const int n = __ldg(n_tokens + s);
        const float inv = n > 0 ? 1.f / static_cast<float>(n) : 0.f;
        const float f = dloss ? __ldg(dloss + s) * (static_cast<float>(E) /
                                                    static_cast<float>(k)) * inv * inv
                              : 0.f;
        zc = dz ? 2.f * __ldg(dz + s) * inv : 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            const int e = Row<NV, VEC>::at(lane, i) + j;
            a[i][j] = e < E ? f * static_cast<float>(__ldg(counts + static_cast<size_t>(s) * E + e))
                            : 0.f;
          }
      }
      int chosen = 0;
      float delta = 0.f;
      bool use = false;
      if (dw) {
        // lane j < k: the j-th chosen expert's logit, weight and term
        float l = -INFINITY, g = 0.f;
        if (lane < k) {
          chosen = __ldg(idx + static_cast<size_t>(r) * k + lane);
          use = static_cast<unsigned>(chosen) < static_cast<unsigned>(E);
          if (use) {
            l = __ldg(logits + static_cast<size_t>(r) * E + chosen);
            g = __ldg(dw + static_cast<size_t>(r) * k + lane);
          }
        }
        float m = l;
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        float w = use ? expf(l - m) : 0.f;
        if (m == -INFINITY) w = 0.f;
        float ws = w, wg = w * g;
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) {
          ws += __shfl_xor_sync(0xFFFFFFFFu, ws, o);
          wg += __shfl_xor_sync(0xFFFFFFFFu, wg, o);
        }
        const float q = ws != 0.f ? 1.f / ws : 0.f;
        delta = w * q * (g - wg * q);
      }
      const float lse = x.softmax();
      float dot = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j) dot = fmaf(a[i][j], x.v[i][j], dot);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xFFFFFFFFu, dot, o);
      const float shift = zc * lse - dot;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j) x.v[i][j] *= a[i][j] + shift;
      if (dw) {
        for (int j = 0; j < k; ++j) {  // in order: an expert listed twice gets both terms
          if (lane == j && use) mine[chosen] += delta;
          __syncwarp();
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int e = Row<NV, VEC>::at(lane, i);
          if (e < E) {
#pragma unroll
            for (int j = 0; j < VEC; ++j) x.v[i][j] += mine[e + j];
          }
        }
        __syncwarp();
        if (use) mine[chosen] = 0.f;
        __syncwarp();
      }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = Row<NV, VEC>::at(lane, i);
      if (e < E) {
        if constexpr (VEC == 4)
          *reinterpret_cast<float4*>(out + e) =
              make_float4(x.v[i][0], x.v[i][1], x.v[i][2], x.v[i][3]);
        else
          out[e] = x.v[i][0];
      }
    }
  }
}

// Calls f with the (NV, VEC) of E: vectors of 4 when rows are whole 16-byte vectors.
template <int N>
struct Num {
  static constexpr int value = N;
};
template <typename F>
cudaError_t with_row(int E, F f) {
  if (E % 4 == 0) {
    if (E <= 128) return f(Num<1>(), Num<4>());
    if (E <= 256) return f(Num<2>(), Num<4>());
    if (E <= 384) return f(Num<3>(), Num<4>());
    if (E <= 512) return f(Num<4>(), Num<4>());
    return f(Num<8>(), Num<4>());
  }
  if (E <= 32) return f(Num<1>(), Num<1>());
  if (E <= 64) return f(Num<2>(), Num<1>());
  if (E <= 128) return f(Num<4>(), Num<1>());
  if (E <= 256) return f(Num<8>(), Num<1>());
  if (E <= 512) return f(Num<16>(), Num<1>());
  return f(Num<32>(), Num<1>());
}

}  // namespace

// Rows per CTA of the forward's first kernel.
static int balance_rows_per_cta(int T) {
  const int per = static_cast<int>((static_cast<long long>(T) + kBalanceCtas - 1) / kBalanceCtas);
  return per < kWarps ? kWarps : per;
}

int balance_ctas(int T) {
  const int per = balance_rows_per_cta(T);
  const int n = static_cast<int>((static_cast<long long>(T) + per - 1) / per);
  return n < 1 ? 1 : n;  // (T = 0: one CTA, which clears the tickets)
}

cudaError_t launch_balance_loss(const float* logits, const int32_t* idx, const int32_t* off,
                                const uint8_t* mask, int T, int E, int k, int S,
                                const BalanceWs& w, int32_t* counts, int32_t* n_tokens,
                                float* prob, float* loss, float* z_loss, cudaStream_t st) {
  const int per = balance_rows_per_cta(T);
  const int ctas = balance_ctas(T);
  const size_t smem = sizeof(float) * (kWarps + 1) * E;
  cudaError_t e = with_row(E, [&](auto nv, auto vec) {
    return launch_k(k_balance_partial<decltype(nv)::value, decltype(vec)::value>, ctas,
                    kWarps * 32, smem, st, logits, idx, off, mask, T, E, k, S, per, w.p, w.c,
                    w.z, w.n, w.ticket, w.flags);
  });
  if (e != cudaSuccess) return e;
  const dim3 grid((E + 31) / 32, S);
  return launch_k(k_balance_final, grid, 1024, 0, st, off, T, E, k, S, per, w.p, w.c, w.z, w.n,
                  w.ticket, w.terms, counts, n_tokens, prob, loss, z_loss, w.flags, ctas,
                  w.status);
}

cudaError_t launch_balance_bwd(const float* logits, const int32_t* idx, const int32_t* off,
                               const uint8_t* mask, const int32_t* counts,
                               const int32_t* n_tokens, const float* dloss, const float* dz,
                               const float* dw, int T, int E, int k, int S, float* dlogits,
                               cudaStream_t st) {
  if (T == 0) return cudaSuccess;
  // up to 8 CTAs an SM, all resident
  const long long warps = 152 * 8 * kWarps;
  const int per = static_cast<int>((T + warps - 1) / warps);
  const int ctas = static_cast<int>((T + static_cast<long long>(per) * kWarps - 1) /
                                    (static_cast<long long>(per) * kWarps));
  const size_t smem = dw ? sizeof(float) * kWarps * E : 0;
  return with_row(E, [&](auto nv, auto vec) {
    return launch_k(k_balance_bwd<decltype(nv)::value, decltype(vec)::value>, ctas, kWarps * 32,
                    smem, st, logits, idx, off, mask, counts, n_tokens, dloss, dz, dw, T, E, k, S,
                    per, dlogits);
  });
}

}  // namespace moe
