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
// One pass over the logits, which stay in the registers of the token's lanes (E <= 1024), so
// the maximum, the sum, the probabilities and their products are register work.  Both
// directions are bound by reading (and in the gradient writing) T x E fp32 values, and at the
// sizes of a training step by what surrounds that: 32768 x 384 takes 16.8 us forward (12 for
// the pass over 50 MB, the rest the second kernel's chain of dependent loads) and 21.3 us
// backward (100 MB; 0.70 of the copy bandwidth).
// No floating-point atomics: partial sums are added in a fixed order, or in fixed point.
#include "block.cuh"

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
template <int LPR>
__device__ __forceinline__ float row_max(float v) {
  if constexpr (LPR == 32) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
  }
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return v;
}
template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// A lane's experts in a row over LPR lanes: VEC consecutive ones from (lane + i * LPR) *
// VEC.  Missing experts read as -inf (probability 0).
template <int NV, int VEC, int LPR>
struct Row {
  float v[NV][VEC];
  __device__ __forceinline__ static int at(int lane, int i) { return (i * LPR + lane) * VEC; }
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
  // The lane's own part of a row into shared memory, asynchronously, and out of it.
  __device__ __forceinline__ static void fetch(float* slot, const float* p, int E, int lane) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (at(lane, i) < E) {
        if constexpr (VEC == 4) cp_async16(slot + at(lane, i), p + at(lane, i));
        else cp_async4(slot + at(lane, i), p + at(lane, i));
      }
  }
  __device__ __forceinline__ void take(const float* slot, int E, int lane) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = at(lane, i);
      if constexpr (VEC == 4) {
        float4 f = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
        if (e < E) f = *reinterpret_cast<const float4*>(slot + e);
        v[i][0] = f.x, v[i][1] = f.y, v[i][2] = f.z, v[i][3] = f.w;
      } else {
        v[i][0] = e < E ? slot[e] : -INFINITY;
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
    m = row_max<LPR>(m);
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

// Beside the STATUS_* bits in a CTA's flags: the offsets decrease somewhere (as seq_off reads
// them).  The slots that the first kernel fills are then not those that the second would add.
constexpr uint32_t kDecreasing = 1u << 31;

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
// raises one of the two, so the slots differ; there are CTAs + S - 1 of them.)  The offsets
// are checked apart from that walk, which need not come past every pair of them: thread i of
// the grid has pairs i, i + threads, ...
template <int NV, int VEC>
__global__ void __launch_bounds__(fwd_warps(NV * VEC * 32) * 32, 2)
    k_balance_partial(const float* __restrict__ logits, const int32_t* __restrict__ idx,
                      const int32_t* __restrict__ off, const uint8_t* __restrict__ mask, int T,
                      int E, int k, int S, int per, float* __restrict__ part_p,
                      int32_t* __restrict__ part_c, float* __restrict__ part_z,
                      int32_t* __restrict__ part_n, unsigned long long* __restrict__ acc,
                      uint32_t* __restrict__ flags) {
  pdl_wait();
  pdl_trigger();
  constexpr int W = fwd_warps(NV * VEC * 32);
  extern __shared__ __align__(16) float dyn[];  // [W][E] sums of p, then [E] counts
  __shared__ float zs[W];
  __shared__ int ns[W];
  int32_t* hist = reinterpret_cast<int32_t*>(dyn + W * E);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t bad = 0;  // data-dependent checks of this thread (STATUS_*, kDecreasing)
  for (int s = blockIdx.x * blockDim.x + threadIdx.x; s < S; s += gridDim.x * blockDim.x) {
    acc[s] = 0;  // the loss sums of the kernel after this one
    if (off) {
      const int lo = __ldg(off + s), hi = __ldg(off + s + 1);
      if (lo < 0 || hi > T || hi < lo) bad |= STATUS_BAD_PLAN;
      if (seq_off(off, s + 1, S, T) < seq_off(off, s, S, T)) bad |= kDecreasing;
    }
  }
  const int begin = blockIdx.x * per, end = T - begin < per ? T : begin + per;
  int row = begin;
  for (int s = seq_of(off, S, T, begin); s < S && row < end; ++s) {
    const int sb = seq_off(off, s, S, T), se = seq_off(off, s + 1, S, T);
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
    // (masked rows too: their values are loaded and dropped).  (16 lanes a token and a ring in
    // shared memory, as in the gradient: the same 17 us for 32768 x 384, slower elsewhere.)
    Row<NV, VEC, 32> nx;
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
      Row<NV, VEC, 32> x = nx;
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
      const float lse = lse_of(m, row_sum<32>(x.total()), r1s);
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
        const int e = Row<NV, VEC, 32>::at(lane, i) + j;
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
  const int decreasing = plan ? __syncthreads_or(bad & kDecreasing) : 0;
  if (threadIdx.x == 0)
    flags[blockIdx.x] = (plan ? STATUS_BAD_PLAN : 0u) | (index ? STATUS_BAD_INDEX : 0u) |
                        (decreasing ? kDecreasing : 0u);
}

// Adds up the partials of sequence blockIdx.y for 32 experts; warp w takes the slots
// first + w, + WARPS, ... and the warps' sums are added in order.  The CTA that finishes its
// sequence last has the sum of the CTAs' loss terms.  Decreasing offsets (the first `nchecks`
// CTAs of the kernel before have looked for them): no slot is added, the sums are NaN.
template <int WARPS>
__global__ void __launch_bounds__(WARPS * 32)
    k_balance_final(const int32_t* __restrict__ off, int T, int E, int k, int S, int per,
                    const float* __restrict__ part_p, const int32_t* __restrict__ part_c,
                    const float* __restrict__ part_z, const int32_t* __restrict__ part_n,
                    unsigned long long* acc, float* terms, int32_t* __restrict__ counts,
                    int32_t* __restrict__ n_tokens, float* __restrict__ prob,
                    float* __restrict__ loss, float* __restrict__ z_loss,
                    const uint32_t* __restrict__ flags, int nflags, int nchecks,
                    uint32_t* status) {
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
  uint32_t checks = 0;
  for (int i = lane; i < nchecks; i += 32) checks |= flags[i];
  float inv = n > 0 ? 1.f / static_cast<float>(n) : 0.f;
  if (__any_sync(0xFFFFFFFFu, checks & kDecreasing)) c = 0, n = 0, inv = NAN, p = 0.f, z = 0.f;
  p *= inv;
  if (e < E) {
    prob[static_cast<size_t>(s) * E + e] = p;
    counts[static_cast<size_t>(s) * E + e] = c;
  }
  float term = static_cast<float>(c) * inv * p;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) term += __shfl_xor_sync(0xFFFFFFFFu, term, o);
  if (lane != 0) return;
  if (blockIdx.x == 0) {
    n_tokens[s] = n;
    if (z_loss) z_loss[s] = z * inv;
  }
  // One atomic does the loss's sum and the arrival: [51:0] the terms in fixed point (each at
  // most k <= 16, to 2^-47: whatever the order, the same sum), [57:52] how many were NaN,
  // [63:58] arrivals.  The last CTA has it all.  Terms of less than 2^-18 (experts were chosen
  // that have next to no probability) are left in fp32 as well: where the sum is that small,
  // all of them are, and it is added up from these, in order.
  constexpr float kSmall = 1.f / (1 << 18);
  terms += static_cast<size_t>(s) * gridDim.x;
  if (n > 0 && term < kSmall) {
    terms[blockIdx.x] = term;
    __threadfence();
  }
  const bool bad = !(term <= 32.f);
  const unsigned long long add =
      (1ull << 58) | (bad ? 1ull << 52 : static_cast<unsigned long long>(
                                             static_cast<double>(term) * 140737488355328.0));
  const unsigned long long all = atomicAdd(acc + s, add) + add;
  if (all >> 58 != gridDim.x) return;
  double sum = static_cast<double>(all & ((1ull << 52) - 1)) / 140737488355328.0;
  if (all >> 52 & 63) {
    sum = nan("");
  } else if (n > 0 && sum < kSmall) {
    __threadfence();
    sum = 0.0;
    for (int i = 0; i < static_cast<int>(gridDim.x); ++i) sum += __ldcg(terms + i);
  }
  loss[s] = static_cast<float>(sum * E / k);
}

// CTAs per SM: by the registers a lane's values take, and no more (32768 x 384 with three 26
// us, with four 30: each row's lanes load their counts first, and few rows follow).
__host__ __device__ constexpr int bwd_ctas_per_sm(int E) {
  return E <= 512 ? 2 : 1;
}

template <int NV, int VEC, int LPR>
__global__ void __launch_bounds__(kWarps * 32, bwd_ctas_per_sm(NV * VEC * LPR))
    k_balance_bwd(const float* __restrict__ logits, const int32_t* __restrict__ idx,
                  const int32_t* __restrict__ off, const uint8_t* __restrict__ mask,
                  const int32_t* __restrict__ counts, const int32_t* __restrict__ n_tokens,
                  const float* __restrict__ dloss, const float* __restrict__ dz,
                  const float* __restrict__ dw, int T, int E, int k, int S, int per,
                  float* __restrict__ dlogits) {
  pdl_wait();
  pdl_trigger();
  using R = Row<NV, VEC, LPR>;
  constexpr int RPW = 32 / LPR;  // rows a warp takes at once
  extern __shared__ __align__(16) float dyn[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = lane / LPR, ll = lane % LPR;
  // this row's lanes': [E] the chosen experts' terms (zero between rows; with dw)
  float* mine = dyn + (warp * RPW + sub) * E;
  // and the row that is on its way
  float* next = dyn + (kWarps * RPW + warp * RPW + sub) * E;
  if (dw) {
    for (int e = ll; e < E; e += LPR) mine[e] = 0.f;
    __syncwarp();
  }
  // a CTA takes `per` * (its rows at once) consecutive rows, its rows at once side by side:
  // few streams for HBM (each row's lanes on a stretch of their own: 26 us instead of 22),
  // and the sequence seldom changes
  constexpr int STEP = kWarps * RPW;
  const long long begin = static_cast<long long>(blockIdx.x) * STEP * per;
  const long long end = begin + static_cast<long long>(STEP) * per;
  const int r0 = static_cast<int>(begin) + warp * RPW + sub;
  const int r1 = end < T ? static_cast<int>(end) : T;
  int s = r0 < r1 ? seq_of(off, S, T, r0) : 0, have = -1;
  int sb = seq_off(off, s, S, T), se = seq_off(off, s + 1, S, T);
  float a[NV][VEC] = {};
  float zc = 0.f;
  auto fetch = [&](int r) {
    if (r < r1) R::fetch(next, logits + static_cast<size_t>(r) * E, E, ll);
    cp_async_commit();
  };
  int nx_e = -1;
  float nx_g = 0.f;
  auto fetch_choice = [&](int r) {
    if (dw && r < r1 && ll < k) {
      nx_e = __ldg(idx + static_cast<size_t>(r) * k + ll);
      nx_g = __ldg(dw + static_cast<size_t>(r) * k + ll);
    }
  };
  fetch(r0);
  fetch_choice(r0);
  // the lanes of a warp stay together: every row of the block, there or not
  for (int i = 0; i < per; ++i) {
    const int r = r0 + i * STEP;
    const bool in = r < r1;
    if (!__any_sync(0xFFFFFFFFu, in)) break;
    while (in && r >= se && s + 1 < S) {
      ++s;
      sb = seq_off(off, s, S, T), se = seq_off(off, s + 1, S, T);
    }
    const bool on = in && r >= sb && r < se && (!mask || __ldg(mask + r) != 0);
    R x;
    const int chosen = on ? nx_e : -1;
    const float g = nx_g;
    const bool use = static_cast<unsigned>(chosen) < static_cast<unsigned>(E);
    float l = -INFINITY;  // lane j < k: the j-th chosen expert's logit
    fetch_choice(r + STEP);
    cp_async_wait<0>();
    __syncwarp();
    x.take(next, E, ll);
    if (dw && use) l = next[chosen];
    __syncwarp();
    fetch(r + STEP);
    if (on) {
      if (have != s) {
        have = s;
        const int n = __ldg(n_tokens + s);
        const float inv = n > 0 ? 1.f / static_cast<float>(n) : 0.f;
        const float f = dloss ? __ldg(dloss + s) * (static_cast<float>(E) /
                                                    static_cast<float>(k)) * inv * inv
                              : 0.f;
        zc = dz ? 2.f * __ldg(dz + s) * inv : 0.f;
#pragma unroll
        for (int q = 0; q < NV; ++q)
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            const int e = R::at(ll, q) + j;
            a[q][j] = e < E ? f * static_cast<float>(__ldg(counts + static_cast<size_t>(s) * E + e))
                            : 0.f;
          }
      }
    } else {
#pragma unroll
      for (int q = 0; q < NV; ++q)
#pragma unroll
        for (int j = 0; j < VEC; ++j) x.v[q][j] = -INFINITY;
    }
    if (dw) {
      // its weight and term
      const float m = row_max<16>(l);
      const float w = use && m != -INFINITY ? exp_diff(l, m) : 0.f;
      const float ws = row_sum<16>(w), wg = row_sum<16>(use ? w * g : 0.f);
      const float q = ws != 0.f ? __fdividef(1.f, ws) : 0.f;
      const float delta = use ? w * q * (g - wg * q) : 0.f;
      // into the row's layout through shared memory; an expert listed twice gets both terms,
      // in order
      const unsigned same = __match_any_sync(0xFFFFFFFFu, use ? sub * 1024 + chosen : -1 - lane);
      if (__any_sync(0xFFFFFFFFu, same & (same - 1))) {
        for (int j = 0; j < k; ++j) {
          if (ll == j && use) mine[chosen] += delta;
          __syncwarp();
        }
      } else {
        if (use) mine[chosen] = delta;
        __syncwarp();
      }
    }
    const float m = x.exps();
    float dot = 0.f;
#pragma unroll
    for (int q = 0; q < NV; ++q)
#pragma unroll
      for (int j = 0; j < VEC; ++j) dot = fmaf(a[q][j], x.v[q][j], dot);
    const float sum = row_sum<LPR>(x.total());
    dot = row_sum<LPR>(dot);
    if (in) {
      float inv;
      const float lse = lse_of(m, sum, inv);
      const float shift = zc * lse - dot * inv;
      float* out = dlogits + static_cast<size_t>(r) * E;
#pragma unroll
      for (int q = 0; q < NV; ++q) {
        const int e = R::at(ll, q);
        if (e < E) {
          float d[VEC];
#pragma unroll
          for (int j = 0; j < VEC; ++j)
            d[j] = on ? x.v[q][j] * ((a[q][j] + shift) * inv) : 0.f;
          if constexpr (VEC == 4) {
            if (dw) {
              const float4 t = *reinterpret_cast<const float4*>(mine + e);
              d[0] += t.x, d[1] += t.y, d[2] += t.z, d[3] += t.w;
            }
            *reinterpret_cast<float4*>(out + e) = make_float4(d[0], d[1], d[2], d[3]);
          } else {
            out[e] = d[0] + (dw ? mine[e] : 0.f);
          }
        }
      }
    }
    if (dw) {
      __syncwarp();
      if (use) mine[chosen] = 0.f;
      __syncwarp();
    }
  }
}

// Calls f with the (NV, VEC, LPR) of E: vectors of 4 when rows are whole 16-byte vectors.
template <int NV_, int VEC_, int LPR_>
struct Shape {
  static constexpr int NV = NV_, VEC = VEC_, LPR = LPR_;
};
// The forward's: a token takes a warp.
template <typename F>
cudaError_t with_fwd_row(int E, F f) {
  if (E % 4 == 0) {
    if (E <= 128) return f(Shape<1, 4, 32>());
    if (E <= 256) return f(Shape<2, 4, 32>());
    if (E <= 384) return f(Shape<3, 4, 32>());
    if (E <= 512) return f(Shape<4, 4, 32>());
    return f(Shape<8, 4, 32>());
  }
  if (E <= 32) return f(Shape<1, 1, 32>());
  if (E <= 64) return f(Shape<2, 1, 32>());
  if (E <= 128) return f(Shape<4, 1, 32>());
  if (E <= 256) return f(Shape<8, 1, 32>());
  if (E <= 512) return f(Shape<16, 1, 32>());
  return f(Shape<32, 1, 32>());
}
// The gradient's: a token takes 16 lanes (the row's sums, logarithm, quotients and the chosen
// experts' terms then cost one instruction for two tokens) up to 512 experts in vectors, a warp
// above.  24000 tokens, 16 lanes and 32: 388 experts 17.5 and 19.3 us, 448 18.6 and 20.4, 512
// 20.8 and 21.5.  Scalar rows, whose accesses are a fourth as wide, go over at 256: 129 experts
// 14.0 and 16.8, 255 18.0 and 18.3, 385 26.9 and 25.8, 511 33.0 and 28.6.
template <typename F>
cudaError_t with_bwd_row(int E, F f) {
  if (E % 4 == 0) {
    if (E <= 64) return f(Shape<1, 4, 16>());
    if (E <= 128) return f(Shape<2, 4, 16>());
    if (E <= 256) return f(Shape<4, 4, 16>());
    if (E <= 384) return f(Shape<6, 4, 16>());
    if (E <= 512) return f(Shape<8, 4, 16>());
    return f(Shape<8, 4, 32>());
  }
  if (E <= 32) return f(Shape<2, 1, 16>());
  if (E <= 64) return f(Shape<4, 1, 16>());
  if (E <= 128) return f(Shape<8, 1, 16>());
  if (E <= 256) return f(Shape<16, 1, 16>());
  if (E <= 512) return f(Shape<16, 1, 32>());
  return f(Shape<32, 1, 32>());
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
  return n < 1 ? 1 : n;  // (T = 0: one CTA, which clears the sums)
}

int balance_ctas_most(int T, int E) {
  const int n = static_cast<int>((static_cast<long long>(T) + fwd_warps(E) - 1) / fwd_warps(E));
  return n < 1 ? 1 : n < kBalanceCtas ? n : kBalanceCtas;
}

cudaError_t launch_balance_loss(const float* logits, const int32_t* idx, const int32_t* off,
                                const uint8_t* mask, int T, int E, int k, int S,
                                const BalanceWs& w, int32_t* counts, int32_t* n_tokens,
                                float* prob, float* loss, float* z_loss, cudaStream_t st) {
  const int per = balance_rows_per_cta(T, E);
  const int ctas = balance_ctas(T, E);
  const size_t smem = sizeof(float) * (fwd_warps(E) + 1) * E;
  cudaError_t e = with_fwd_row(E, [&](auto sh) {
    using H = decltype(sh);
    return launch_k(k_balance_partial<H::NV, H::VEC>, ctas, fwd_warps(E) * 32, smem, st, logits,
                    idx, off, mask, T, E, k, S, per, w.p, w.c, w.z, w.n, w.acc, w.flags);
  });
  if (e != cudaSuccess) return e;
  const dim3 grid((E + 31) / 32, S);
  const int threads = fwd_warps(E) * 32, checking = (S + threads - 1) / threads;
  const int checks = !off ? 0 : checking < ctas ? checking : ctas;
  // one sequence has up to kBalanceCtas slots, one of many a share of them (64 sequences of
  // 32768 tokens with 1024 threads each: 28 us instead of 18)
  if (S > 8)
    return launch_k(k_balance_final<8>, grid, 256, 0, st, off, T, E, k, S, per, w.p, w.c, w.z, w.n,
                    w.acc, w.terms, counts, n_tokens, prob, loss, z_loss, w.flags, ctas,
                    checks, w.status);
  return launch_k(k_balance_final<32>, grid, 1024, 0, st, off, T, E, k, S, per, w.p, w.c, w.z, w.n,
                  w.acc, w.terms, counts, n_tokens, prob, loss, z_loss, w.flags, ctas,
                  checks, w.status);
}

cudaError_t launch_balance_bwd(const float* logits, const int32_t* idx, const int32_t* off,
                               const uint8_t* mask, const int32_t* counts,
                               const int32_t* n_tokens, const float* dloss, const float* dz,
                               const float* dw, int T, int E, int k, int S, float* dlogits,
                               cudaStream_t st) {
  if (T == 0) return cudaSuccess;
  return with_bwd_row(E, [&](auto sh) {
    using H = decltype(sh);
    constexpr int rows = kWarps * (32 / H::LPR);  // a CTA's at once
    const long long all = 1LL * kSms * bwd_ctas_per_sm(H::NV * H::VEC * H::LPR) * rows;  // resident
    const int per = static_cast<int>((T + all - 1) / all);
    const int ctas = static_cast<int>((T + static_cast<long long>(per) * rows - 1) /
                                      (static_cast<long long>(per) * rows));
    constexpr auto kern = k_balance_bwd<H::NV, H::VEC, H::LPR>;
    const size_t smem = sizeof(float) * rows * E * 2;
    const cudaError_t a = allow_smem<kern>();
    if (a != cudaSuccess) return a;
    return launch_k(kern, ctas, kWarps * 32, smem, st, logits, idx, off, mask, counts, n_tokens,
                    dloss, dz, dw, T, E, k, S, per, dlogits);
  });
}

}  // namespace moe
