// Dense projection with its epilogue, y = act(x W^T + bias) + residual, and its gradient.
//
// Every product is out[t][f] = sum_c P[t][c] * Q[f][c] of bf16 operands with fp32 sums:
//   forward   P = x  [M][K]        Q = W [N][K]         c = K
//   dx        P = dz [M][N]        Q = W read as [K][N]  c = N
//   dW        P = dz read as [N][M] Q = x read as [K][M]  c = M
// An operand "read as" its transpose stays where it is: its tiles are loaded with the other
// index contiguous and the MMA takes them as MN-major.  Operands whose rows are not whole
// 16-byte vectors cannot be loaded by TMA and are first copied to padded rows.
//
// Two kernels, chosen per product by their measured costs (choose below):
//   * k_linear_pair: 256 x 256 outputs per SM pair (cta_group::2 MMAs of M = 256, N = 256),
//     64 columns of c a stage in a ring of six, persistent, two accumulators in TMEM so that a
//     tile's epilogue runs under the next tile's MMAs; with few tiles two pairs share one,
//     each summing half of c.  Bound by the tensor cores (16384 x 7168 x 7168 with residual:
//     1.01 to 1.06 ms, 1.59 to 1.67 PFLOP/s under the power cap) or, for short c, by the
//     epilogue's elementwise work (8192 x 4096 x 1024: 42 us plain, with bias and SiLU 52, with
//     bias and GELU 65 to 70).
//   * k_linear_split: for outputs with too few such tiles.  128 features (the MMA's M side:
//     the weights fill its rows even for one token) x NT tokens a tile, c split among the
//     CTAs of a cluster, whose partial sums meet in distributed shared memory and are added
//     in rank order (no atomics, no workspace).  Bound by reading W for few tokens (7 x 7168
//     x 7168: 20 us, 15.4 of them the weights' at the copy bandwidth).
// Every wait is bounded; one that expires sets the workspace's status word.
#include "block.cuh"

#include <math.h>

namespace moe {

namespace {

constexpr int kBK = 64;            // contraction columns per stage: one 128-byte swizzle row
constexpr int kRowBytes = kBK * 2;

// One operand: its matrix in memory and which index is contiguous.
struct Operand {
  const uint16_t* p;
  long long ld;  // elements; ld % 8 == 0
  int rows;      // t or f extent
  int mn;        // 1: [c][rows] (rows contiguous), 0: [rows][c]
};

struct Epi {
  const void* bias;  // [F] or null
  const void* res;   // [R][ldr] or null
  void* out;         // [R][ldo]
  uint16_t* z;       // [R][ldz] or null: the value in front of the activation
  long long ldr, ldo, ldz;
  int bias_f32, out_f32, act;  // residual has the output's type
  int whole;         // rows of out, res and z are whole 32-byte sectors
};

struct LinearParams {
  int R, F, C;  // out rows, out columns, contraction
  int p_mn, q_mn;
  Epi e;
  uint32_t* status;
};

__device__ __forceinline__ float bf16_up(uint16_t v) {
  return __uint_as_float(static_cast<uint32_t>(v) << 16);
}
__device__ __forceinline__ uint16_t bf16_down(float v) {
  return __bfloat16_as_ushort(__float2bfloat16_rn(v));
}
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&b);
}

// Activations and their slopes, in fp32.  The sigmoid from ex2.approx and rcp.approx (each
// within 2 units of 2^-23; the argument's rounding adds |z| * 2^-24): expf and the IEEE
// quotient would double the gradient pass's instructions, which bound it.
__device__ __forceinline__ float sigmoid(float z) { return __fdividef(1.f, 1.f + __expf(-z)); }
__device__ __forceinline__ float act_value(float z, int act) {
  if (act == MOE_ACT_RELU) return z > 0.f ? z : (z != z ? z : 0.f);
  if (act == MOE_ACT_SILU) return z * sigmoid(z);
  if (act == MOE_ACT_GELU) return 0.5f * z * (1.f + erff(z * 0.70710678f));
  return z;
}
__device__ __forceinline__ float act_slope(float z, int act) {
  if (act == MOE_ACT_RELU) return z > 0.f ? 1.f : (z != z ? z : 0.f);
  if (act == MOE_ACT_SILU) {
    const float s = sigmoid(z);
    return s * fmaf(z, 1.f - s, 1.f);
  }
  if (act == MOE_ACT_GELU)
    return 0.5f * (1.f + erff(z * 0.70710678f)) + z * 0.39894228f * __expf(-0.5f * z * z);
  return 1.f;
}
// dy * act'(z); a ReLU that is off passes nothing on, an infinity or NaN neither
__device__ __forceinline__ float act_grad(float dy, float z, int act) {
  return act == MOE_ACT_RELU && z <= 0.f ? 0.f : dy * act_slope(z, act);
}

__device__ __forceinline__ float bias_at(const Epi& e, int f) {
  return e.bias_f32 ? __ldg(static_cast<const float*>(e.bias) + f)
                    : bf16_up(__ldg(static_cast<const uint16_t*>(e.bias) + f));
}

// Column f of N rows t0, t0 + step, ... (those with on[i]) in two steps, so that the
// residuals (which the output might alias) can be loaded long before they are needed and all
// before the first store.  b: the column's bias.
template <int N>
__device__ __forceinline__ void load_column(const Epi& e, int t0, int step, int f,
                                            const bool (&on)[N], float (&r)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) r[i] = 0.f;
  if (!e.res) return;
  const long long at = t0 * e.ldr + f, inc = step * e.ldr;
  if (e.out_f32) {
    const float* p = static_cast<const float*>(e.res) + at;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (on[i]) r[i] = p[i * inc];
  } else {
    const uint16_t* p = static_cast<const uint16_t*>(e.res) + at;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (on[i]) r[i] = bf16_up(p[i * inc]);
  }
}
template <int N>
__device__ __forceinline__ void emit_column(const Epi& e, int t0, int step, int f, float b,
                                            const bool (&on)[N], const float (&r)[N],
                                            float (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] += b;
  if (e.z) {
    uint16_t* p = e.z + t0 * e.ldz + f;
    const long long inc = step * e.ldz;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (on[i]) p[i * inc] = bf16_down(v[i]);
  }
  if (e.act != MOE_ACT_NONE) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = act_value(v[i], e.act);
  }
  const long long at = t0 * e.ldo + f, inc = step * e.ldo;
  if (e.out_f32) {
    float* p = static_cast<float*>(e.out) + at;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (on[i]) p[i * inc] = v[i] + r[i];
  } else {
    uint16_t* p = static_cast<uint16_t*>(e.out) + at;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (on[i]) p[i * inc] = bf16_down(v[i] + r[i]);
  }
}

// 32 bytes at once: a whole sector of a row (p 32-byte aligned).
__device__ __forceinline__ void ld_sector(const void* p, uint32_t (&w)[8]) {
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]),
                 "=r"(w[6]), "=r"(w[7])
               : "l"(p)
               : "memory");
}
__device__ __forceinline__ void st_sector(void* p, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]),
               "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}
// 32 columns from f0 of a row of F: n = how many of them there are, whole sectors.
__device__ __forceinline__ void st_bf16x32(uint16_t* p, const float (&v)[32], int n) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = bf16_pair(v[16 * h + 2 * i], v[16 * h + 2 * i + 1]);
    if (16 * h < n) st_sector(p + 16 * h, w);
  }
}

// The next 32 columns' residual, loaded ahead where it is bf16 (two sectors) ...
struct RowRes {
  uint32_t w[2][8];
};
__device__ __forceinline__ void load_row32(const Epi& e, int t, int f0, int n, RowRes& r) {
  if (!e.res || e.out_f32) return;
  const uint16_t* p = static_cast<const uint16_t*>(e.res) + static_cast<size_t>(t) * e.ldr + f0;
#pragma unroll
  for (int h = 0; h < 2; ++h)
    if (16 * h < n) ld_sector(p + 16 * h, r.w[h]);
}
// ... and the outputs.
__device__ __forceinline__ void emit_row32(const Epi& e, int t, int f0, int n, const RowRes& r,
                                           const float* bias, float (&v)[32]) {
  if (e.bias) {  // bias: the 32 columns', in shared memory (16-byte aligned)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float4 b = reinterpret_cast<const float4*>(bias)[i];
      v[4 * i] += b.x, v[4 * i + 1] += b.y, v[4 * i + 2] += b.z, v[4 * i + 3] += b.w;
    }
  }
  if (e.z) st_bf16x32(e.z + static_cast<size_t>(t) * e.ldz + f0, v, n);
  if (e.act == MOE_ACT_RELU) {
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = act_value(v[i], MOE_ACT_RELU);
  } else if (e.act == MOE_ACT_SILU) {
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = act_value(v[i], MOE_ACT_SILU);
  } else if (e.act == MOE_ACT_GELU) {
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = act_value(v[i], MOE_ACT_GELU);
  }
  const size_t at = static_cast<size_t>(t) * e.ldo + f0;
  if (e.out_f32) {
    const float* rp = static_cast<const float*>(e.res) + static_cast<size_t>(t) * e.ldr + f0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t w[8];
      if (8 * i < n) {
        if (e.res) ld_sector(rp + 8 * i, w);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          w[j] = __float_as_uint(v[8 * i + j] + (e.res ? __uint_as_float(w[j]) : 0.f));
        st_sector(static_cast<float*>(e.out) + at + 8 * i, w);
      }
    }
  } else {
    if (e.res) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          v[16 * i + 2 * j] += __uint_as_float(r.w[i][j] << 16);
          v[16 * i + 2 * j + 1] += __uint_as_float(r.w[i][j] & 0xFFFF0000u);
        }
    }
    st_bf16x32(static_cast<uint16_t*>(e.out) + at, v, n);
  }
}

// Instruction descriptor, kind::f16: D fp32, A and B bf16, M x n, transposed operands.
__device__ __forceinline__ uint32_t idesc_bf16(int m, int n, int a_mn, int b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(a_mn) << 15) |
         (static_cast<uint32_t>(b_mn) << 16) | (static_cast<uint32_t>(n >> 3) << 17) |
         (static_cast<uint32_t>(m >> 4) << 24);
}

// A stage's tile of `rows` (a multiple of 64, or 16 / 32 when K-major) x 64 c:
//   K-major:  [rows][64 c], 128-byte swizzled rows; 16 c further is 32 bytes further.
//   MN-major: [rows / 64][64 c][64 rows], 128-byte swizzled rows; 8 c are 1024 bytes (the
//             stride offset), 64 rows 8192 (the leading offset), 16 c 2048 further.
__device__ __forceinline__ uint64_t tile_desc(uint32_t base, int mn, int kk) {
  return mn ? smem_desc(base + kk * 16 * kRowBytes, kBK * kRowBytes, 1024, kLayoutSw128)
            : smem_desc(base + kk * 32, 0, 1024, kLayoutSw128);
}

// ---------------------------------------------------------------- SM pairs ----------

constexpr int kPTile = 256;                      // output rows and columns per pair
constexpr int kPOpBytes = 128 * kRowBytes;       // one operand's stage in one CTA
constexpr int kPStageBytes = 2 * kPOpBytes;
template <bool kWhole>
struct PairCfg {
  // Rows that are no whole sectors cost the epilogue more: twice the warps, a stage less (2000
  // x 3001 x 1504 33 us, with eight warps 47).
  static constexpr int kStages = kWhole ? 6 : 5;
  static constexpr int kWarps = kWhole ? 8 : 16;              // epilogue warps
  static constexpr int kCols = kPTile / (kWarps / 4);         // a warp's columns of the tile
  static constexpr int kThreads = 128 + 32 * kWarps;          // TMA, MMA, two idle warps
  static constexpr int kOffBar = kStages * kPStageBytes;
  // full[S], empty[S], acc_full[2], acc_empty[2], drain
  static constexpr int kOffMisc = kOffBar + (2 * kStages + 5) * 8;
  // per epilogue warp: its columns' bias (kWhole), or a 32 x 33 block
  static constexpr int kOffTurn = (kOffMisc + 16 + 15) / 16 * 16;
  static constexpr int kSmem = kOffTurn + kWarps * (kWhole ? kCols * 4 : 32 * 33 * 4);
  static_assert(kSmem <= 232448, "dynamic shared memory of one CTA");
};
// Tiles are walked in bands of this many output rows' tiles, column by column, so that the
// tiles in flight share both operands' blocks in L2.
constexpr int kPBand = 8;

struct PairTile {
  int t0, f0;
};
__device__ __forceinline__ PairTile pair_tile(int L, int tiles_t, int tiles_f) {
  const int per = kPBand * tiles_f;
  const int band = L / per, in = L - band * per;
  const int first = band * kPBand;
  const int h = tiles_t - first < kPBand ? tiles_t - first : kPBand;
  PairTile r;
  r.t0 = (first + in % h) * kPTile;
  r.f0 = (in / h) * kPTile;
  return r;
}

// CTA r of a pair: output rows 128 r.. of the tile (its P rows and accumulator lanes) and Q
// rows 128 r.. (half of the MMA's N side).
// kWhole: the output's rows (and the residual's and z's) are whole 32-byte sectors.
// S > 1 (few tiles): one tile per cluster of S pairs, each of which sums an S-th of c; the
// partial sums meet in distributed shared memory (the drained rings), where pair i finishes
// the i-th part of the tile's columns, adding in pair order.
template <bool kWhole, int S>
__global__ void __launch_bounds__(PairCfg<kWhole>::kThreads, 1)
    k_linear_pair(const __grid_constant__ CUtensorMap tmP, const __grid_constant__ CUtensorMap tmQ,
                  const LinearParams p) {
  using C = PairCfg<kWhole>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t crank = cluster_ctarank(), rank = crank & 1, pair = crank >> 1;
  const bool leader = rank == 0;
  const uint16_t both = static_cast<uint16_t>(3u << (crank & ~1u));  // this pair's CTAs
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint64_t* empty = full + C::kStages;
  uint64_t* acc_full = empty + C::kStages;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* drain = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 2 * C::kWarps);  // two CTAs' epilogue warps
    }
    mbar_init(drain, 1);
    // swizzled tiles need a 1024-byte aligned base: a misaligned one makes every role a
    // no-op (the CTA still takes part in the pair's set-up and teardown)
    const bool bad = (smem_u32(smem) & 1023u) != 0;
    *abort_flag = bad ? 1 : 0;
    if (bad) set_status(p.status, STATUS_BAD_PLAN);
    fence_mbar_init();
    tma_prefetch_desc(&tmP);
    tma_prefetch_desc(&tmQ);
  }
  if (warp == 1) tmem_alloc_pair(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  pdl_wait();
  const uint32_t tmem = *tmem_slot;
  const int tiles_t = (p.R + kPTile - 1) / kPTile, tiles_f = (p.F + kPTile - 1) / kPTile;
  const int total = tiles_t * tiles_f;
  const int nk = (p.C + kBK - 1) / kBK;
  const int kb0 = static_cast<int>(static_cast<long long>(nk) * pair / S);
  const int kb1 = static_cast<int>(static_cast<long long>(nk) * (pair + 1) / S);
  const int cl = blockIdx.x / (2 * S), ncl = gridDim.x / (2 * S);
  auto leader_addr = [&](const uint64_t* b) -> uint32_t {
    return mapa_shared(smem_u32(b), crank & ~1u);
  };
  // 32 columns f.. of the warp's 32 rows t - lane.., not whole sectors: turned in shared
  // memory, so that a warp stores 32 consecutive values of a row
  auto ragged = [&](const float (&v32)[32], int t, int f) {
    float* turn = reinterpret_cast<float*>(smem + C::kOffTurn) + (warp - 4) * 32 * 33;
#pragma unroll
    for (int i = 0; i < 32; ++i) turn[lane * 33 + i] = v32[i];
    __syncwarp();
    const int tw = t - lane, fc = f + lane;
    const int rows = fc < p.F ? p.R - tw : 0;  // this lane's, from tw
    const float bias = p.e.bias && rows > 0 ? bias_at(p.e, fc) : 0.f;
    constexpr int kRows = 16;  // (8: a sixth slower; 32: out of registers)
#pragma unroll 1
    for (int i = 0; i < 32; i += kRows) {
      float v[kRows], rr[kRows];
      bool on[kRows];
#pragma unroll
      for (int j = 0; j < kRows; ++j) on[j] = i + j < rows;
      load_column<kRows>(p.e, tw + i, 1, fc, on, rr);
#pragma unroll
      for (int j = 0; j < kRows; ++j) v[j] = turn[(i + j) * 33 + lane];
      emit_column<kRows>(p.e, tw + i, 1, fc, bias, on, rr, v);
    }
    __syncwarp();
  };

  if (warp == 0) {
    // ---------------------------------------------------------------- TMA
    if (lane == 0) {
      uint32_t it = 0;
      bool ok = true;
      for (int L = cl; L < total && ok && !*abort_flag; L += ncl) {
        const PairTile tl = pair_tile(L, tiles_t, tiles_f);
        const int t0 = tl.t0 + static_cast<int>(rank) * 128;
        const int f0 = tl.f0 + static_cast<int>(rank) * 128;
        for (int kb = kb0; kb < kb1; ++kb, ++it) {
          const int s = it % C::kStages;
          if (it >= C::kStages &&
              !mbar_wait(&empty[s], ((it / C::kStages) & 1u) ^ 1u, p.status, abort_flag)) {
            ok = false;
            break;
          }
          if (leader) mbar_arrive_expect_tx(&full[s], 2 * kPStageBytes);
          const uint32_t fb = leader_addr(&full[s]);
          uint8_t* a = smem + s * kPStageBytes;
          uint8_t* b = a + kPOpBytes;
          if (p.p_mn) {
            tma_load_2d_pair(a, &tmP, fb, t0, kb * kBK);
            tma_load_2d_pair(a + kPOpBytes / 2, &tmP, fb, t0 + 64, kb * kBK);
          } else {
            tma_load_2d_pair(a, &tmP, fb, kb * kBK, t0);
          }
          if (p.q_mn) {
            tma_load_2d_pair(b, &tmQ, fb, f0, kb * kBK);
            tma_load_2d_pair(b + kPOpBytes / 2, &tmQ, fb, f0 + 64, kb * kBK);
          } else {
            tma_load_2d_pair(b, &tmQ, fb, kb * kBK, f0);
          }
        }
      }
      // after an abort: the pair's loads still in flight (all counted on these barriers)
      if (leader && *abort_flag) {
        const uint32_t from = it > C::kStages ? it - C::kStages : 0;
        for (uint32_t i = from; i < it; ++i)
          mbar_wait_drain(&full[i % C::kStages], (i / C::kStages) & 1u);
      }
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA
    if (leader && lane == 0) {
      uint32_t it = 0, tc = 0;
      const uint32_t idesc = idesc_bf16(256, 256, p.p_mn, p.q_mn);
      bool ok = true;
      for (int L = cl; L < total && ok && !*abort_flag; L += ncl, ++tc) {
        const uint32_t b = tc & 1u, use = tc >> 1;
        if (tc >= 2 && !mbar_wait(&acc_empty[b], (use - 1) & 1u, p.status, abort_flag)) break;
        tc_fence_after();
        const uint32_t d = tmem + b * kPTile;
        for (int kb = kb0; kb < kb1; ++kb, ++it) {
          const int s = it % C::kStages;
          if (!mbar_wait(&full[s], (it / C::kStages) & 1u, p.status, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a0 = smem_u32(smem + s * kPStageBytes);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_bf16_ss_pair(d, tile_desc(a0, p.p_mn, kk), tile_desc(a0 + kPOpBytes, p.q_mn, kk),
                             idesc, kb > kb0 || kk > 0);
          tc_commit_pair_mc(&empty[s], both);
        }
        if (ok) tc_commit_pair_mc(&acc_full[b], both);
      }
      // after an abort: the MMAs already issued
      if (*abort_flag) {
        tc_commit_pair_mc(drain, static_cast<uint16_t>(1u << crank));
        mbar_wait_drain(drain, 0);
      }
    }
  } else if (warp >= 4 && S == 1) {
    // ---------------------------------------------------------------- epilogue
    // four warps for the accumulator's lanes, and so for each share of its columns
    const int q = warp & 3, share = (warp - 4) >> 2;
    uint32_t tc = 0;
    for (int L = cl; L < total; L += ncl, ++tc) {  // (an abort makes the wait fail)
      const PairTile tl = pair_tile(L, tiles_t, tiles_f);
      const uint32_t b = tc & 1u, use = tc >> 1;
      const int t = tl.t0 + static_cast<int>(rank) * 128 + q * 32 + lane;
      const int f0 = tl.f0 + share * C::kCols;
      const int cols = p.F - f0 < C::kCols ? p.F - f0 : C::kCols;
      // the next 32 columns' residual is in flight under these columns' stores, the first
      // ones' under the tile's last MMAs
      RowRes res;
      float* bias = reinterpret_cast<float*>(smem + C::kOffTurn) + (warp - 4) * C::kCols;
      if constexpr (kWhole) {
        if (t < p.R) load_row32(p.e, t, f0, cols, res);
        if (p.e.bias) {
          __syncwarp();  // (the last tile's has been read)
          for (int c = lane; c < cols; c += 32) bias[c] = bias_at(p.e, f0 + c);
          __syncwarp();
        }
      }
      int w_ok = 1;
      if (lane == 0) w_ok = mbar_wait(&acc_full[b], use & 1u, p.status, abort_flag);
      if (!__shfl_sync(0xFFFFFFFFu, w_ok, 0)) break;
      tc_fence_after();
      const uint32_t acc =
          tmem + (static_cast<uint32_t>(q * 32) << 16) + b * kPTile + share * C::kCols;
      for (int c = 0; c < cols; c += 32) {
        uint32_t r[32];
        tmem_ld_32x32b_x32(acc + c, r);
        tmem_ld_wait();
        if constexpr (kWhole) {
          const RowRes now = res;
          if (t < p.R) {
            if (c + 32 < cols) load_row32(p.e, t, f0 + c + 32, cols - c - 32, res);
            float v[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
            emit_row32(p.e, t, f0 + c, cols - c, now, bias + c, v);
          }
        } else {
          float v[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
          ragged(v, t, f0 + c);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (leader) mbar_arrive(&acc_empty[b]);
        else mbar_arrive_cluster(leader_addr(&acc_empty[b]));
      }
    }
  }
  if constexpr (S > 1) {
    // ---------------------------------------------------------------- joined epilogue
    constexpr int CW = kPTile / S;  // columns a pair finishes
    const PairTile tl = pair_tile(cl, tiles_t, tiles_f);
    const int q = warp & 3, share = (warp - 4) >> 2;
    constexpr int kStep = 32 * (C::kWarps / 4);  // columns from a warp's block to its next
    const int row = q * 32 + lane, t = tl.t0 + static_cast<int>(rank) * 128 + row;
    const uint32_t acc = tmem + (static_cast<uint32_t>(q * 32) << 16);
    float* sums = reinterpret_cast<float*>(smem);  // [column of the tile][128 rows]
    int w_ok = 0;
    if (warp >= 4) {
      if (lane == 0) w_ok = mbar_wait(&acc_full[0], 0, p.status, abort_flag);
      w_ok = __shfl_sync(0xFFFFFFFFu, w_ok, 0);
      tc_fence_after();
      for (int c = share * 32; c < kPTile && w_ok; c += kStep) {
        if (c / CW == static_cast<int>(pair) || tl.f0 + c >= p.F) continue;
        uint32_t r[32];
        tmem_ld_32x32b_x32(acc + c, r);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 32; ++i) sums[(c + i) * 128 + row] = __uint_as_float(r[i]);
      }
    }
    __syncwarp();
    cluster_sync();  // every pair's sums are in place
    if (warp >= 4) {
      for (int c = static_cast<int>(pair) * CW + share * 32;
           c < (static_cast<int>(pair) + 1) * CW; c += kStep) {
        const int f = tl.f0 + c;
        if (!w_ok || f >= p.F) break;
        RowRes res;
        float* bias = reinterpret_cast<float*>(smem + C::kOffTurn) + (warp - 4) * C::kCols;
        if constexpr (kWhole) {
          if (t < p.R) load_row32(p.e, t, f, p.F - f, res);
          if (p.e.bias) {
            __syncwarp();
            if (f + lane < p.F) bias[lane] = bias_at(p.e, f + lane);
            __syncwarp();
          }
        }
        uint32_t r[32];
        tmem_ld_32x32b_x32(acc + c, r);
        float v[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = 0.f;
        tmem_ld_wait();
#pragma unroll
        for (int o = 0; o < S; ++o) {
          const uint32_t at = mapa_shared(smem_u32(sums + c * 128 + row), 2 * o + rank);
          float u[32];
#pragma unroll
          for (int i = 0; i < 32; ++i)
            u[i] = o == static_cast<int>(pair) ? __uint_as_float(r[i])
                                               : ld_shared_cluster(at + i * 512);
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] += u[i];
        }
        if constexpr (kWhole) {
          if (t < p.R) emit_row32(p.e, t, f, p.F - f, res, bias, v);
        } else {
          ragged(v, t, f);
        }
      }
    }
    __syncwarp();
  }
  pdl_trigger();
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // neither CTA releases TMEM or shared memory the pair still uses
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

// ---------------------------------------------------------------- split contraction --

constexpr int kSFeat = 128;  // features per tile

template <int NT>
struct SplitCfg {
  static constexpr int kQBytes = kSFeat * kRowBytes;
  static constexpr int kPBytes = NT * kRowBytes;
  static constexpr int kStageBytes = kQBytes + kPBytes;
  static constexpr int kStages = 100 * 1024 / kStageBytes;  // two CTAs per SM
  static constexpr int kOffBar = kStages * kStageBytes;
  static constexpr int kOffMisc = kOffBar + (2 * kStages + 2) * 8;
  static constexpr int kSmem = kOffMisc + 16;
  static constexpr int kTmemCols = NT < 32 ? 32 : NT;
  static_assert(NT * kSFeat * 4 <= kOffBar, "the partial sums reuse the ring");
};

// grid (splits, feature tiles, token tiles), cluster (splits, 1, 1).  CTA r sums its share
// of the contraction blocks; then token j of the tile is finished by CTA j % splits.
template <int NT>
__global__ void __launch_bounds__(256, 2)
    k_linear_split(const __grid_constant__ CUtensorMap tmP, const __grid_constant__ CUtensorMap tmQ,
                   const LinearParams p) {
  using C = SplitCfg<NT>;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint64_t* empty = full + C::kStages;
  uint64_t* acc_full = empty + C::kStages;
  uint64_t* drain = acc_full + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(acc_full, 1);
    mbar_init(drain, 1);
    const bool bad = (smem_u32(smem) & 1023u) != 0;
    *abort_flag = bad ? 1 : 0;
    if (bad) set_status(p.status, STATUS_BAD_PLAN);
    fence_mbar_init();
    tma_prefetch_desc(&tmP);
    tma_prefetch_desc(&tmQ);
  }
  if (warp == 1) tmem_alloc(tmem_slot, C::kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_wait();
  pdl_trigger();  // (after the TMEM allocation: a successor's cannot come in between)
  const uint32_t tmem = *tmem_slot;
  const int splits = gridDim.x, part = blockIdx.x;
  const int f0 = blockIdx.y * kSFeat, t0 = blockIdx.z * NT;
  const int nk = (p.C + kBK - 1) / kBK;
  const int kb0 = static_cast<int>(static_cast<long long>(nk) * part / splits);
  const int kb1 = static_cast<int>(static_cast<long long>(nk) * (part + 1) / splits);

  if (warp == 0) {
    if (lane == 0) {
      uint32_t it = 0;
      for (int kb = kb0; kb < kb1; ++kb, ++it) {
        const int s = it % C::kStages;
        if (*abort_flag ||
            (it >= C::kStages &&
             !mbar_wait(&empty[s], ((it / C::kStages) & 1u) ^ 1u, p.status, abort_flag)))
          break;
        uint8_t* a = smem + s * C::kStageBytes;
        uint8_t* b = a + C::kQBytes;
        mbar_arrive_expect_tx(&full[s], C::kStageBytes);
        if (p.q_mn) {
          tma_load_2d(a, &tmQ, &full[s], f0, kb * kBK);
          tma_load_2d(a + C::kQBytes / 2, &tmQ, &full[s], f0 + 64, kb * kBK);
        } else {
          tma_load_2d(a, &tmQ, &full[s], kb * kBK, f0);
        }
        if (NT >= 64 && p.p_mn) {
          tma_load_2d(b, &tmP, &full[s], t0, kb * kBK);
          if (NT == 128) tma_load_2d(b + C::kPBytes / 2, &tmP, &full[s], t0 + 64, kb * kBK);
        } else {
          tma_load_2d(b, &tmP, &full[s], kb * kBK, t0);
        }
      }
      if (*abort_flag) {
        const uint32_t from = it > C::kStages ? it - C::kStages : 0;
        for (uint32_t i = from; i < it; ++i)
          mbar_wait_drain(&full[i % C::kStages], (i / C::kStages) & 1u);
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t idesc = idesc_bf16(kSFeat, NT, p.q_mn, NT >= 64 ? p.p_mn : 0);
      uint32_t it = 0;
      bool ok = !*abort_flag;
      for (int kb = kb0; kb < kb1 && ok; ++kb, ++it) {
        const int s = it % C::kStages;
        if (!mbar_wait(&full[s], (it / C::kStages) & 1u, p.status, abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t a0 = smem_u32(smem + s * C::kStageBytes);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          mma_bf16_ss(tmem, tile_desc(a0, p.q_mn, kk),
                      tile_desc(a0 + C::kQBytes, NT >= 64 ? p.p_mn : 0, kk), idesc,
                      kb > kb0 || kk > 0);
        tc_commit(&empty[s]);
      }
      if (ok) {
        tc_commit(acc_full);
      } else {
        tc_commit(drain);
        mbar_wait_drain(drain, 0);
      }
    }
  }
  __syncwarp();
  // Epilogue: a thread has one feature, four warps the tile's 128, eight warps two sets of
  // tokens.  What the contraction does not decide (bias, the first residuals) is loaded
  // before the wait for it.
  const int q = warp & 3, set = warp >> 2;
  const int fl = q * 32 + lane, f = f0 + fl;
  const bool live = f < p.F;
  const int nt = p.R - t0 < NT ? p.R - t0 : NT;
  const float bias = p.e.bias && live ? bias_at(p.e, f) : 0.f;
  const uint32_t acc = tmem + (static_cast<uint32_t>(q * 32) << 16);
  // one CTA: tokens in blocks of kTok, alternating between the sets
  // a cluster: tokens part + splits * (set + 2 i), kTok of them at a time
  // (kTok = 16 makes the code so long that fetching it costs a single token 2 us)
  constexpr int kTok = 8;
  const bool alone = splits == 1;
  const int step = alone ? 1 : 2 * splits, first = alone ? set * kTok : part + set * splits;
  const int block = alone ? 2 * kTok : kTok * step;
  float res[kTok];
  bool on[kTok];
  auto fetch = [&](int j0) {
#pragma unroll
    for (int i = 0; i < kTok; ++i) on[i] = live && j0 + i * step < nt;
    load_column<kTok>(p.e, t0 + j0, step, f, on, res);
  };
  fetch(first);
  int w_ok = 1;
  if (lane == 0) w_ok = mbar_wait(acc_full, 0, p.status, abort_flag);
  w_ok = __shfl_sync(0xFFFFFFFFu, w_ok, 0);
  tc_fence_after();
  float* sums = reinterpret_cast<float*>(smem);  // [NT][128], in the drained ring
  if (!alone) {
    for (int c = set * 8; c < nt && w_ok; c += 16) {
      uint32_t r[8];
      tmem_ld_32x32b_x8(acc + c, r);
      tmem_ld_wait();
#pragma unroll
      for (int i = 0; i < 8; ++i) sums[(c + i) * kSFeat + fl] = __uint_as_float(r[i]);
    }
    cluster_sync();  // every CTA's partial sums are in place
  }
  for (int j0 = first; j0 < nt && w_ok; j0 += block) {
    float v[kTok];
    if (alone) {
      uint32_t r[8];
      tmem_ld_32x32b_x8(acc + j0, r);
      tmem_ld_wait();
#pragma unroll
      for (int i = 0; i < kTok; ++i) v[i] = __uint_as_float(r[i]);
    } else {
#pragma unroll
      for (int i = 0; i < kTok; ++i) v[i] = 0.f;
      const uint32_t mine = smem_u32(sums + j0 * kSFeat + fl);
      for (int r0 = 0; r0 < splits; r0 += 4) {  // four CTAs' sums in flight
        float u[4][kTok];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const uint32_t at = mapa_shared(mine, r0 + r < splits ? r0 + r : 0);
#pragma unroll
          for (int i = 0; i < kTok; ++i) {
            u[r][i] = 0.f;
            if (r0 + r < splits && j0 + i * step < nt)
              u[r][i] = ld_shared_cluster(at + i * step * kSFeat * 4);
          }
        }
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int i = 0; i < kTok; ++i) v[i] += u[r][i];
      }
    }
    emit_column<kTok>(p.e, t0 + j0, step, f, bias, on, res, v);
    if (j0 + block < nt) fetch(j0 + block);
  }
  if (!alone) cluster_sync();  // no CTA leaves while its sums are read
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// ---------------------------------------------------------------- elementwise --------

// Rows copied to a row length that TMA can load (the columns past `cols` are never read);
// blockIdx.y: which of up to two matrices.
struct Repack {
  const uint16_t* src;
  uint16_t* dst;
  long long lds, ldd;
  int rows, cols;
};
__global__ void __launch_bounds__(256) k_repack(const Repack a, const Repack b) {
  pdl_wait();
  pdl_trigger();
  const Repack m = blockIdx.y ? b : a;
  // two values a thread: a destination word from one source word, or where the row starts on
  // an odd value from the halves of two (5001 x 5001: 30 us; value by value 50)
  const int full = (m.cols - 1) / 2;  // words with a value of the row behind them
  for (int r = blockIdx.x; r < m.rows; r += gridDim.x) {
    const uint16_t* src = m.src + static_cast<size_t>(r) * m.lds;
    uint32_t* dst = reinterpret_cast<uint32_t*>(m.dst + static_cast<size_t>(r) * m.ldd);
    const bool odd = (reinterpret_cast<uintptr_t>(src) & 2) != 0;
    const uint32_t* words = reinterpret_cast<const uint32_t*>(src - (odd ? 1 : 0));
    if (odd) {
#pragma unroll 4
      for (int w = threadIdx.x; w < full; w += 256)
        dst[w] = __funnelshift_r(words[w], words[w + 1], 16);
    } else {
#pragma unroll 4
      for (int w = threadIdx.x; w < full; w += 256) dst[w] = words[w];
    }
    if (threadIdx.x == 0)  // the last one or two values, and nothing past the row
      for (int c = full * 2; c < m.cols; ++c) reinterpret_cast<uint16_t*>(dst)[c] = src[c];
  }
}

// dz = bf16(dy * act'(z)) (the products take bf16 operands; the rounding is 2^-9 of each
// element), and with part the column sums of the unrounded values over rows [blockIdx.y *
// per, + per): a thread owns VEC columns.  dz null: only the sums.  Memory-bound: VEC = 8
// where all rows are whole 16-byte vectors (4096 x 6144: 30 us; two columns a thread 63).
template <int VEC>
__global__ void __launch_bounds__(128)
    k_linear_dz(const uint16_t* __restrict__ dy, long long ldy, const uint16_t* __restrict__ z,
                long long ldz, int act, int M, int N, int per, uint16_t* __restrict__ dz,
                long long ldd, float* __restrict__ part) {
  pdl_wait();
  pdl_trigger();
  const int c0 = (blockIdx.x * 128 + threadIdx.x) * VEC;
  if (c0 >= N) return;
  const int r0 = blockIdx.y * per, r1 = M - r0 < per ? M : r0 + per;
  float sum[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) sum[i] = 0.f;
#pragma unroll 4
  for (int r = r0; r < r1; ++r) {
    float a[VEC], s[VEC];
    if constexpr (VEC == 8) {
      const uint4 u = __ldg(reinterpret_cast<const uint4*>(dy + r * ldy + c0));
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a[2 * i] = __uint_as_float(w[i] << 16);
        a[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      }
      if (z) {
        const uint4 t = __ldg(reinterpret_cast<const uint4*>(z + r * ldz + c0));
        const uint32_t y[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          s[2 * i] = __uint_as_float(y[i] << 16);
          s[2 * i + 1] = __uint_as_float(y[i] & 0xFFFF0000u);
        }
      }
    } else {
      a[0] = bf16_up(__ldg(dy + r * ldy + c0));
      if (z) s[0] = bf16_up(__ldg(z + r * ldz + c0));
    }
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      if (z) a[i] = act_grad(a[i], s[i], act);
      sum[i] += a[i];
    }
    if (dz) {
      if constexpr (VEC == 8)
        *reinterpret_cast<uint4*>(dz + r * ldd + c0) =
            make_uint4(bf16_pair(a[0], a[1]), bf16_pair(a[2], a[3]), bf16_pair(a[4], a[5]),
                       bf16_pair(a[6], a[7]));
      else
        dz[r * ldd + c0] = bf16_down(a[0]);
    }
  }
  if (part) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) part[static_cast<size_t>(blockIdx.y) * N + c0 + i] = sum[i];
  }
}

// ---------------------------------------------------------------- host side ----------

bool on32(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 31) == 0; }

bool encode(CUtensorMap* m, const Operand& o, int C, int box_rows) {
  EncodeTiledFn enc = get_encode_tiled_fn();
  if (!enc) return false;
  const cuuint64_t inner = o.mn ? o.rows : C, outer = o.mn ? C : o.rows;
  cuuint64_t dims[2] = {inner, outer};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(o.ld) * 2};
  cuuint32_t box[2] = {64, static_cast<cuuint32_t>(o.mn ? kBK : box_rows)};
  cuuint32_t es[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<uint16_t*>(o.p), dims, strides, box,
             es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// ks: of a persistent kernel, how many of its clusters fit the GPU at once.
cudaError_t launch_cluster(const void* kern, OncePerContext& ks, int smem, int cluster, dim3 grid,
                           int threads, bool persistent, cudaStream_t st, void** args) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= OncePerContext::kDevices) return cudaErrorInvalidDevice;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  int clusters = 0;
  if (ks.ready(dev, current_context_id())) {
    clusters = ks.value(dev);
  } else {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    if (persistent) {
      int sms = 0;
      e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
      if (e != cudaSuccess) return e;
      cfg.gridDim = dim3(sms / cluster * cluster);
      cfg.numAttrs = 1;
      e = cudaOccupancyMaxActiveClusters(&clusters, kern, &cfg);
      if (e != cudaSuccess) return e;
      if (clusters < 1) return cudaErrorInvalidConfiguration;
    }
    ks.set(dev, clusters);
  }
  if (persistent && grid.x > static_cast<unsigned>(clusters) * cluster) grid.x = clusters * cluster;
  cfg.gridDim = grid;
  cfg.numAttrs = 2;
  return cudaLaunchKernelExC(&cfg, kern, args);
}

template <int NT>
cudaError_t launch_split(const Operand& P, const Operand& Q, const LinearParams& p, int splits,
                         cudaStream_t st) {
  static OncePerContext ks;
  CUtensorMap tmP, tmQ;
  if (!encode(&tmP, P, p.C, NT) || !encode(&tmQ, Q, p.C, kSFeat)) return cudaErrorInvalidValue;
  const dim3 grid(splits, (p.F + kSFeat - 1) / kSFeat, (p.R + NT - 1) / NT);
  if (grid.y > 65535 || grid.z > 65535) return cudaErrorInvalidValue;
  void* args[] = {&tmP, &tmQ, const_cast<LinearParams*>(&p)};
  return launch_cluster(reinterpret_cast<const void*>(k_linear_split<NT>), ks, SplitCfg<NT>::kSmem,
                        splits, grid, 256, false, st, args);
}

template <bool kWhole, int S>
cudaError_t launch_pair_tiles(const Operand& P, const Operand& Q, const LinearParams& p,
                              cudaStream_t st) {
  static OncePerContext ks;
  CUtensorMap tmP, tmQ;
  if (!encode(&tmP, P, p.C, 128) || !encode(&tmQ, Q, p.C, 128)) return cudaErrorInvalidValue;
  const long long tiles = static_cast<long long>((p.R + kPTile - 1) / kPTile) *
                          ((p.F + kPTile - 1) / kPTile);
  if (tiles > (1LL << 28)) return cudaErrorInvalidValue;
  void* args[] = {&tmP, &tmQ, const_cast<LinearParams*>(&p)};
  return launch_cluster(reinterpret_cast<const void*>(k_linear_pair<kWhole, S>), ks,
                        PairCfg<kWhole>::kSmem, 2 * S,
                        dim3(static_cast<unsigned>(2 * S * tiles)), PairCfg<kWhole>::kThreads,
                        S == 1, st, args);
}
template <bool kWhole>
cudaError_t launch_pairs(const Operand& P, const Operand& Q, const LinearParams& p, int splits,
                         cudaStream_t st) {
  if (splits == 2) return launch_pair_tiles<kWhole, 2>(P, Q, p, st);
  return launch_pair_tiles<kWhole, 1>(P, Q, p, st);
}

// One product, on the kernel and tile that should take the least time, by costs measured on
// GB300 (us).  A pair tile: 0.29 per 64 columns of c, 76 tiles at a time, a tile's epilogue
// (6.3 with whole rows, 9 without) under the next tile's MMAs.  Split tiles: their loads
// together at 12.5 TB/s from L2, W's at 6.9 from HBM, a CTA's stages 0.27 to 0.41 each; per
// wave of 304 CTAs 3 for launch and first load, 0.87 per 16 tokens of a CTA's epilogue and
// 0.02 per token that a cluster exchanges.  Clusters of 3, 5 and 6 fit the GPU's partitions
// badly (7 x 7168 x 7168 in 4 parts 20.2, in 5 20.9, in 6 27.4) and are not used.
// Both sides (pairs, two pairs a tile, split): 7168 x 7168 weights, 128 rows: 38, 28, 26.5;
// 256: 39, 28, 41; 512: 40, -, 67; 1024 x 1024 x 8192: 42, 26, 24; 1024 x 2048 x 2048: 15.5,
// 13.2, 18.7; 300 x 1024 x 256: 7.6, -, 4.4; 8192 x 256 x 1024: 11.5, -, 17.8.
struct Choice {
  double us;
  int nt, splits;  // nt = 0: SM pairs
};
Choice choose(int R, int F, int C, bool p_mn, bool whole) {
  constexpr int kPairs = kSms / 2;  // pair tiles at a time; split CTAs: two per SM
  const int nk = (C + kBK - 1) / kBK;
  const long long tiles =
      static_cast<long long>((R + kPTile - 1) / kPTile) * ((F + kPTile - 1) / kPTile);
  const double waves = static_cast<double>((tiles + kPairs - 1) / kPairs);
  const double mma = 0.29 * nk, epi = whole ? 6.3 : 9.0;
  Choice best = {(waves - 1) * (mma > epi ? mma : epi) + mma + epi, 0, 1};
  // two pairs a tile, while all their clusters fit (four: clusters of eight CTAs with an SM
  // each fit badly, 7168 x 7168 weights and 256 rows 40 us)
  const double two_us = 0.16 * nk + (whole ? 8.5 : 10.0);
  if (tiles <= 36 && nk >= 2 && two_us < best.us) best = {two_us, 0, 2};
  const long long ft = (F + kSFeat - 1) / kSFeat;
  for (int nt = p_mn ? 64 : 16; nt <= 128; nt *= 2) {
    const long long tt = (R + nt - 1) / nt;
    if (tt > 65535 || ft > 65535) continue;
    const int rows = R < nt ? R : nt;
    const double l2 = ft * tt * static_cast<double>(nk) * (kSFeat + nt) * kRowBytes / 12.5e6;
    const double hbm = static_cast<double>(F) * C * 2 / 6.9e6;
    const double stage = nt == 128 ? 0.41 : nt == 64 ? 0.31 : 0.27;
    for (int splits = 1; splits <= 8 && splits <= nk; splits *= 2) {
      const double w = static_cast<double>((ft * tt * splits + 2 * kSms - 1) / (2 * kSms));
      const double chain = w * stage * ((nk + splits - 1) / splits);
      double us = l2 > hbm ? l2 : hbm;
      us = (us > chain ? us : chain) + 0.1 * chain + (splits == 8 ? 2.0 : 0.0) +
           w * (3.0 + 0.87 * ((rows + 16 * splits - 1) / (16 * splits)) +
                (splits > 1 ? 0.2 + 0.02 * rows : 0.0));
      if (us < best.us) best = {us, nt, splits};
    }
  }
  return best;
}

cudaError_t product(const Operand& P, const Operand& Q, const LinearParams& p, cudaStream_t st) {
  const Choice c = choose(p.R, p.F, p.C, p.p_mn, p.e.whole);
  switch (c.nt) {
    case 0:
      return p.e.whole ? launch_pairs<true>(P, Q, p, c.splits, st)
                       : launch_pairs<false>(P, Q, p, c.splits, st);
    case 16: return launch_split<16>(P, Q, p, c.splits, st);
    case 32: return launch_split<32>(P, Q, p, c.splits, st);
    case 64: return launch_split<64>(P, Q, p, c.splits, st);
    default: return launch_split<128>(P, Q, p, c.splits, st);
  }
}

// Points o at its copy in `to` (null: it stays where it is); returns the copy to make.
Repack repack(Operand& o, int C, uint16_t* to) {
  Repack r = {};
  if (!to) return r;
  r.src = o.p, r.lds = o.ld;
  r.rows = o.mn ? C : o.rows, r.cols = o.mn ? o.rows : C;
  r.dst = to, r.ldd = linear_padded(r.cols);
  o.p = to, o.ld = r.ldd;
  return r;
}
cudaError_t run_repack(Repack a, Repack b, cudaStream_t st) {
  if (!a.rows) a = b, b = Repack{};
  if (!a.rows) return cudaSuccess;
  const int rows = a.rows > b.rows ? a.rows : b.rows;
  const dim3 grid(rows < 4096 ? rows : 4096, b.rows ? 2 : 1);
  return launch_k(k_repack, grid, 256, 0, st, a, b);
}

}  // namespace

cudaError_t launch_linear(const LinearCall& a, cudaStream_t st) {
  Operand P = {a.x, a.ldx, a.M, 0}, Q = {a.w, a.ldw, a.N, 0};
  const Repack rp = repack(P, a.K, a.x_pad), rq = repack(Q, a.K, a.w_pad);
  const cudaError_t e = run_repack(rp, rq, st);
  if (e != cudaSuccess) return e;
  LinearParams p = {a.M, a.N, a.K, 0, 0, {}, a.status};
  p.e = {a.bias, a.res, a.y, a.z, a.ldr, a.ldy, a.ldz, a.bias_f32, a.y_f32, a.act, 0};
  const int ow = a.y_f32 && !a.z ? 8 : 16;  // columns in whole sectors of every matrix
  p.e.whole = a.N % ow == 0 && a.ldy % ow == 0 && on32(a.y) &&
              (!a.res || (a.ldr % ow == 0 && on32(a.res))) &&
              (!a.z || (a.ldz % ow == 0 && on32(a.z)));
  return product(P, Q, p, st);
}

cudaError_t launch_linear_bwd(const LinearBwdCall& a, cudaStream_t st) {
  cudaError_t e = cudaSuccess;
  Operand x = {a.x, a.ldx, a.K, 1};   // dW's Q: [c = M][K]
  Operand w = {a.w, a.ldw, a.K, 1};   // dx's Q: [c = N][K]
  const uint16_t* dz = a.dy;
  long long ldz = a.lddy;
  if (a.dz || a.part) {
    const uint16_t* z = a.act == MOE_ACT_NONE ? nullptr : a.z;
    const bool vec = a.N % 8 == 0 && a.lddy % 8 == 0 && (!z || a.ldz % 8 == 0);
    const int blocks = (a.N + (vec ? 1023 : 127)) / (vec ? 1024 : 128);
    // row blocks: about 8 CTAs of 128 threads per SM (4: 53 us)
    int parts = (kSms * 8 + blocks - 1) / blocks;
    parts = parts > kLinearDbParts ? kLinearDbParts : parts;
    const int per = (a.M + parts - 1) / parts;
    parts = (a.M + per - 1) / per;
    const dim3 grid(blocks, parts);
    e = vec ? launch_k(k_linear_dz<8>, grid, 128, 0, st, a.dy, a.lddy, z, a.ldz, a.act, a.M, a.N,
                       per, a.dz, linear_padded(a.N), a.part)
            : launch_k(k_linear_dz<1>, grid, 128, 0, st, a.dy, a.lddy, z, a.ldz, a.act, a.M, a.N,
                       per, a.dz, linear_padded(a.N), a.part);
    if (e != cudaSuccess) return e;
    if (a.part) {
      e = launch_column_sum(a.part, parts, a.N, a.db, st);
      if (e != cudaSuccess) return e;
    }
    if (a.dz) dz = a.dz, ldz = linear_padded(a.N);
  }
  const Repack rw = repack(w, a.N, a.dx ? a.w_pad : nullptr);
  const Repack rx = repack(x, a.M, a.dw ? a.x_pad : nullptr);
  e = run_repack(rw, rx, st);
  if (e != cudaSuccess) return e;
  if (a.dx) {
    LinearParams p = {a.M, a.K, a.N, 0, 1, {}, a.status};
    p.e = {nullptr, nullptr, a.dx, nullptr, 0, a.lddx, 0, 0, 0, MOE_ACT_NONE,
           a.K % 16 == 0 && on32(a.dx)};
    e = product({dz, ldz, a.M, 0}, w, p, st);
    if (e != cudaSuccess) return e;
  }
  if (a.dw) {
    LinearParams p = {a.N, a.K, a.M, 1, 1, {}, a.status};
    p.e = {nullptr, nullptr, a.dw, nullptr, 0, a.lddw, 0, 0, 0, MOE_ACT_NONE,
           a.K % 16 == 0 && on32(a.dw)};
    e = product({dz, ldz, a.N, 1}, x, p, st);
  }
  return e;
}

}  // namespace moe
