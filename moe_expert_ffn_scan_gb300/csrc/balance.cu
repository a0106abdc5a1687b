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

constexpr int kWarps = 8;  // per CTA of the gradient

// Warps per CTA of the forward, whose CTAs each leave one partial row per sequence: 16 while
// a lane's values leave two such CTAs per SM their registers.
__host__ __device__ constexpr int fwd_warps(int E) { return E <= 512 ? 16 : 8; }

// e^(v - m): the difference first, so that the largest and lowest finite values have one.
// ex2.approx is within 2 units of 2^-23; with the product's rounding that is
// (2 + |v - m|) * 2^-23, and expf's range handling (half of the row's instructions) is saved.
__device__ __forceinline__ float exp_diff(float v, float m) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"((v - m) * 1.44269504f));
  return r;
}
__device__ __forceinline__ float warp_max(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

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
  // v becomes exp(v - max) (a NaN or infinity leaves a NaN in the sum); returns the maximum.
  // A row of -inf alone has no probabilities: zeros.
  __device__ __forceinline__ float exps() {
    float m = v[0][0];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) m = fmaxf(m, v[i][j]);
    m = warp_max(m);
    const float base = m == -INFINITY ? 0.f : m;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[i][j] = exp_diff(v[i][j], base);
    return m;
  }
  __device__ __forceinline__ float total() const {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) sum += v[i][j];
    return sum;
  }
};

// logsumexp and 1 / sum from the maximum and the sum; 0 and 0 for a row of -inf alone.
__device__ __forceinline__ float lse_of(float m, float sum, float& inv) {
  const bool none = m == -INFINITY && sum == 0.f;
  inv = none ? 0.f : __fdividef(1.f, sum);
  return none ? 0.f : m + logf(sum);
}

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
__global__ void __launch_bounds__(fwd_warps(NV * VEC * 32) * 32, 2)
    k_balance_partial(const float* __restrict__ logits, const int32_t* __restrict__ idx,
                      const int32_t* __restrict__ off, const uint8_t* __restrict__ mask, int T,
                      int E, int k, int S, int per, float* __restrict__ part_p,
                      int32_t* __restrict__ part_c, float* __restrict__ part_z,
                      int32_t* __restrict__ part_n, int32_t* __restrict__ ticket,
                      uint32_t* __restrict__ flags) {
  pdl_wait();
  pdl_trigger();
  constexpr int W = fwd_warps(NV * VEC * 32);
  extern __shared__ __align__(16) float dyn[];  // [W][E] sums of p, then [E] counts
  __shared__ float zs[W];
  __shared__ int ns[W];
  int32_t* hist = reinterpret_cast<int32_t*>(dyn + W * E);
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
    // one row ahead: its logits, mask and choices are in flight under this row's softmax
    // (masked rows too: their values are loaded and dropped)
    Row<NV, VEC> nx;
    bool nx_on = false;
    int nx_e = -1;
    auto fetch = [&](int r) {
      nx_on = r < r1;
      if (!nx_on) return;
      nx.load(logits + static_cast<size_t>(r) * E, E, lane);
      if (lane < k) nx_e = __ldg(idx + static_cast<size_t>(r) * k + lane);
      if (mask) nx_on = __ldg(mask + r) != 0;
    };
    fetch(r0 + warp);
    for (int r = r0 + warp; r < r1; r += W) {
      Row<NV, VEC> x = nx;
      const bool on = nx_on;
      const int e = nx_e;
      fetch(r + W);
      if (!on) continue;
      if (lane < k) {
        if (static_cast<unsigned>(e) < static_cast<unsigned>(E)) atomicAdd(hist + e, 1);
        else bad |= STATUS_BAD_INDEX;
      }
      const float m = x.exps();
      float r1s;
      const float lse = lse_of(m, warp_sum(x.total()), r1s);
      z = fmaf(lse, lse, z);
      ++n;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j) acc[i][j] = fmaf(x.v[i][j], r1s, acc[i][j]);
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
      for (int w = 0; w < W; ++w) v += dyn[w * E + e];
      part_p[slot * E + e] = v;
      part_c[slot * E + e] = hist[e];
    }
    if (threadIdx.x == 0) {
      float zt = 0.f;
      int nt = 0;
#pragma unroll
      for (int w = 0; w < W; ++w) zt += zs[w], nt += ns[w];
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
// first + w, + WARPS, ... and the warps' sums are added in order.  The CTA that finishes its
// sequence last adds the CTAs' loss terms, in CTA order.
template <int WARPS>
__global__ void __launch_bounds__(WARPS * 32)
    k_balance_final(const int32_t* __restrict__ off, int T, int E, int k, int S, int per,
                    const float* __restrict__ part_p, const int32_t* __restrict__ part_c,
                    const float* __restrict__ part_z, const int32_t* __restrict__ part_n,
                    int32_t* ticket, float* terms, int32_t* __restrict__ counts,
                    int32_t* __restrict__ n_tokens, float* __restrict__ prob,
                    float* __restrict__ loss, float* __restrict__ z_loss,
                    const uint32_t* __restrict__ flags, int nflags, uint32_t* status) {
  pdl_wait();
  pdl_trigger();
  __shared__ float rp[WARPS][33];
  __shared__ int rc[WARPS][33];
  __shared__ float rz[WARPS];
  __shared__ int rn[WARPS];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int s = blockIdx.y, e = blockIdx.x * 32 + lane;
  const int sb = seq_off(off, s, S, T), se = seq_off(off, s + 1, S, T);
  const int first = sb / per, last = se > sb ? (se - 1) / per : first - 1;  // CTAs
  // the loads of kBatch slots a warp are issued before the first is used
  constexpr int kBatch = 10;
  float p = 0.f, z = 0.f;
  int c = 0, n = 0;
  for (int b0 = first + warp; b0 <= last; b0 += kBatch * WARPS) {
    float pv[kBatch];
    int cv[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int b = b0 + WARPS * i;
      pv[i] = 0.f, cv[i] = 0;
      if (b <= last && e < E) {
        const size_t at = (static_cast<size_t>(b) + s) * E + e;
        pv[i] = part_p[at];
        cv[i] = part_c[at];
      }
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) p += pv[i], c += cv[i];
  }
  for (int b = first + static_cast<int>(threadIdx.x); b <= last; b += WARPS * 32) {
    z += part_z[static_cast<size_t>(b) + s];
    n += part_n[static_cast<size_t>(b) + s];
  }
  if (blockIdx.x == 0 && s == 0) {  // the call's status word
    uint32_t f = 0;
    for (int i = threadIdx.x; i < nflags; i += WARPS * 32) f |= flags[i];
    const int plan = __syncthreads_or(f & STATUS_BAD_PLAN);
    const int index = __syncthreads_or(f & STATUS_BAD_INDEX);
    if (threadIdx.x == 0)
      *status = (plan ? STATUS_BAD_PLAN : 0u) | (index ? STATUS_BAD_INDEX : 0u);
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
  p = 0.f, c = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) p += rp[w][lane], c += rc[w][lane];
  z = lane < WARPS ? rz[lane] : 0.f, n = lane < WARPS ? rn[lane] : 0;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    z += __shfl_xor_sync(0xFFFFFFFFu, z, o);
    n += __shfl_xor_sync(0xFFFFFFFFu, n, o);
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

// CTAs per SM by the registers a lane's values take.
__host__ __device__ constexpr int bwd_ctas_per_sm(int E) {
  return E <= 384 ? 4 : E <= 512 ? 2 : 1;
}

template <int NV, int VEC>
__global__ void __launch_bounds__(kWarps * 32, bwd_ctas_per_sm(NV * VEC * 32))
    k_balance_bwd(const float* __restrict__ logits, const int32_t* __restrict__ idx,
                  const int32_t* __restrict__ off, const uint8_t* __restrict__ mask,
                  const int32_t* __restrict__ counts, const int32_t* __restrict__ n_tokens,
                  const float* __restrict__ dloss, const float* __restrict__ dz,
                  const float* __restrict__ dw, int T, int E, int k, int S, int per,
                  float* __restrict__ dlogits) {
  pdl_wait();
  pdl_trigger();
  extern __shared__ __align__(16) float dyn[];  // with dw: [kWarps][E], terms of the warp's row
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
  int sb = seq_off(off, s, S, T), se = seq_off(off, s + 1, S, T);
  float a[NV][VEC];
  float zc = 0.f;
  for (int r = r0; r < r1; ++r) {
    // (the other warps hide these loads; a row ahead in registers costs more of them: 26 us
    // instead of 24 for 32768 x 384)
    Row<NV, VEC> x;
    x.load(logits + static_cast<size_t>(r) * E, E, lane);
    const bool on = !mask || __ldg(mask + r) != 0;
    int chosen = -1;
    float g = 0.f;
    if (dw && lane < k) {
      chosen = __ldg(idx + static_cast<size_t>(r) * k + lane);
      g = __ldg(dw + static_cast<size_t>(r) * k + lane);
    }
    while (r >= se && s + 1 < S) {
      ++s;
      sb = seq_off(off, s, S, T), se = seq_off(off, s + 1, S, T);
    }
    float* out = dlogits + static_cast<size_t>(r) * E;
    if (!on || r < sb || r >= se) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j) x.v[i][j] = 0.f;
    } else {
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
      const bool use = dw && lane < k && static_cast<unsigned>(chosen) < static_cast<unsigned>(E);
      float delta = 0.f;
      if (dw) {
        // lane j < k: the j-th chosen expert's logit, weight and term
        const float l = use ? __ldg(logits + static_cast<size_t>(r) * E + chosen) : -INFINITY;
        const float m = warp_max(l);
        const float w = use && m != -INFINITY ? exp_diff(l, m) : 0.f;
        float ws = w, wg = use ? w * g : 0.f;
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) {
          ws += __shfl_xor_sync(0xFFFFFFFFu, ws, o);
          wg += __shfl_xor_sync(0xFFFFFFFFu, wg, o);
        }
        const float q = ws != 0.f ? 1.f / ws : 0.f;
        delta = use ? w * q * (g - wg * q) : 0.f;
        // into the row's layout through shared memory (zero between rows); an expert listed
        // twice gets both terms, in order
        const unsigned same = __match_any_sync(0xFFFFFFFFu, use ? chosen : -1 - lane);
        if (__any_sync(0xFFFFFFFFu, same & (same - 1))) {
          for (int j = 0; j < k; ++j) {
            if (lane == j && use) mine[chosen] += delta;
            __syncwarp();
          }
        } else {
          if (use) mine[chosen] = delta;
          __syncwarp();
        }
      }
      const float m = x.exps();
      float dot = 0.f, sum = x.total();
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j) dot = fmaf(a[i][j], x.v[i][j], dot);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        dot += __shfl_xor_sync(0xFFFFFFFFu, dot, o);
      }
      float inv;
      const float lse = lse_of(m, sum, inv);
      const float shift = zc * lse - dot * inv;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j) x.v[i][j] *= (a[i][j] + shift) * inv;
      if (dw) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int e = Row<NV, VEC>::at(lane, i);
          if (e < E) {
            float term[VEC];
            if constexpr (VEC == 4) {
              const float4 f = *reinterpret_cast<const float4*>(mine + e);
              term[0] = f.x, term[1] = f.y, term[2] = f.z, term[3] = f.w;
            } else {
              term[0] = mine[e];
            }
#pragma unroll
            for (int j = 0; j < VEC; ++j) x.v[i][j] += term[j];
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

// Rows per CTA of the forward's first kernel: as many CTAs as are resident at once.
static int balance_rows_per_cta(int T, int E) {
  const int per = static_cast<int>((static_cast<long long>(T) + kBalanceCtas - 1) / kBalanceCtas);
  return per < fwd_warps(E) ? fwd_warps(E) : per;
}

int balance_ctas(int T, int E) {
  const int per = balance_rows_per_cta(T, E);
  const int n = static_cast<int>((static_cast<long long>(T) + per - 1) / per);
  return n < 1 ? 1 : n;  // (T = 0: one CTA, which clears the tickets)
}

cudaError_t launch_balance_loss(const float* logits, const int32_t* idx, const int32_t* off,
                                const uint8_t* mask, int T, int E, int k, int S,
                                const BalanceWs& w, int32_t* counts, int32_t* n_tokens,
                                float* prob, float* loss, float* z_loss, cudaStream_t st) {
  const int per = balance_rows_per_cta(T, E);
  const int ctas = balance_ctas(T, E);
  const size_t smem = sizeof(float) * (fwd_warps(E) + 1) * E;
  cudaError_t e = with_row(E, [&](auto nv, auto vec) {
    return launch_k(k_balance_partial<decltype(nv)::value, decltype(vec)::value>, ctas,
                    fwd_warps(decltype(nv)::value * decltype(vec)::value * 32) * 32, smem, st, logits, idx, off, mask, T, E, k, S, per, w.p, w.c,
                    w.z, w.n, w.ticket, w.flags);
  });
  if (e != cudaSuccess) return e;
  const dim3 grid((E + 31) / 32, S);
  // one sequence has up to kBalanceCtas slots, one of many a share of them (64 sequences of
  // 32768 tokens with 1024 threads each: 28 us instead of 18)
  if (S > 8)
    return launch_k(k_balance_final<8>, grid, 256, 0, st, off, T, E, k, S, per, w.p, w.c, w.z, w.n,
                    w.ticket, w.terms, counts, n_tokens, prob, loss, z_loss, w.flags, ctas,
                    w.status);
  return launch_k(k_balance_final<32>, grid, 1024, 0, st, off, T, E, k, S, per, w.p, w.c, w.z, w.n,
                  w.ticket, w.terms, counts, n_tokens, prob, loss, z_loss, w.flags, ctas,
                  w.status);
}

cudaError_t launch_balance_bwd(const float* logits, const int32_t* idx, const int32_t* off,
                               const uint8_t* mask, const int32_t* counts,
                               const int32_t* n_tokens, const float* dloss, const float* dz,
                               const float* dw, int T, int E, int k, int S, float* dlogits,
                               cudaStream_t st) {
  if (T == 0) return cudaSuccess;
  const long long warps = 152 * bwd_ctas_per_sm(E) * kWarps;  // all resident
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
