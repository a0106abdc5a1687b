// Gradient products of the experts: for every packed row r of group g
//     dx[r][f] = sum_c dy[r][c] * deq(w[g])[c][f]
// with codes w [G][C][F/2] (E2M1) and scales [G][C][F/32] (MXFP4) or [G][C][F/16] (NVFP4) as the
// forward has them: W2 is [H][I] (C = H, F = I), W13 [2I][H] (C = 2I, F = H).
//
// The contraction runs over the weight's ROWS, so its scales (one per 32 or 16 elements of a
// row) lie along the output axis: the block-scaled MMA kinds, whose scales go along the
// contraction, cannot apply them, and a transposed copy would be a second set of weights.  The
// kernel multiplies in bf16 instead: E2M1 times a power of two or an E4M3 scale is exact there (2
// or 6 significant bits), dy is bf16 as it comes, the products are exact in fp32 and are summed in
// fp32; NVFP4's tensor scales multiply the sums.
//
// The codes become bf16 straight in tensor memory, the MMA's A operand: the features are its M
// side, one per TMEM lane.  The weights lie with the features contiguous, so a transpose is
// needed, and ldmatrix makes it on the codes: read as 16-bit values (four features of one c),
// transposed, a thread's 32-bit register holds four features of two consecutive c, and the codes
// of one feature are 16 bits apart: two masks and a product put them into the two halves of one
// TMEM column, one multiplication by the two c's scales finishes them.  (Through shared memory
// the converted weights cost 328 of the 773 cycles of its bandwidth that 64 c took, and bound
// the kernel.)
//
// Two forms of one kernel, P CTAs a tile:
//   * P = 2, SM pairs (cta_group::2 MMAs of M = 256): 256 features x up to 256 rows of one group.
//     Each CTA converts its 128 features and loads half of the rows, so a stage costs an SM half
//     of the shared-memory traffic for dy that a tile of its own would.  Bound by the tensor
//     cores: w13 of 7168 x 2048, 16 groups of 1024 rows 496 us, 1.94 PFLOP/s; in long runs by the
//     power cap, w13 1.62 to 1.67, w2 1.52 to 1.57.  (NVFP4's W13, whose halves have a scale each: 541 us, 1.78.)
//   * P = 1, two CTAs an SM: 128 features x up to 32 rows, for groups of few rows, where the
//     weights' way from HBM and their conversion are the work.  Bound by the conversion's
//     instructions: 32 groups of 16 rows 114 us, the weights at 4.5 TB/s (NVFP4 126, 4.3).
// In each CTA, a stage at a time:
//   * warp 2 brings the codes of 128 weight rows x 128 features (8 KB, TMA) and their scales
//     (cp.async) into a ring, so that many stages of the weights are on their way;
//   * warp 3, of NVFP4 with the last warp, makes the scales what the converters multiply by;
//   * three groups of four converter warps, a stage each in turn; a warp has 32 features, so
//     one scale a row (its wait on the factors covers the codes too: warp 3 waited for both);
//   * warp 0 brings dy's rows (K-major, TMA), warp 1 (of the pair's first CTA) issues the MMAs;
//   * four or twelve warps store the sums of the last tile under the next one's MMAs.
// Persistent; every CTA finds its tiles from the group offsets by itself (no plan kernel).
// Every wait is bounded; one that expires sets the workspace's status word.
#include "grad.cuh"

#include <math.h>

namespace moe {

namespace {

// c per stage.  With 64 the warps that issue and wait spend twice the instructions on it (SM
// pairs, 32 groups of w13, 7168 x 2048: 64 rows each 214 us in place of 170, 128 rows 229 in place
// of 194; 256 rows 262 in place of 268; few rows on single CTAs 156 in place of 127).
constexpr int kBK = 128;
constexpr int kFeat = 128;       // features per CTA
constexpr int kMaxGroups = 1025;

// Weight formats: MXFP4, and NVFP4 with one tensor scale for all of a weight's rows or one for
// each half of them (W13's gate and up projection).  The halves' sums are kept apart until the
// end where tensor memory has room for two: up to 32 rows, or 128 of a pair.  In a pair's tile of
// more rows the half of the smaller scale is summed first, that sum is then multiplied in place by
// the scales' quotient, and the other half added to it (w13 of 7168 x 2048, 32 groups of 256 rows:
// 281 us, by two tiles of 128 rows 388; 16 groups of 1024: 541, 758).
enum Format { kMx = 0, kNv = 1, kNvHalves = 2 };

template <int P, int F>
struct Cfg {
  static constexpr int kOcc = P == 2 ? 1 : 2;         // CTAs per SM
  static constexpr int kBlock = F == kMx ? 32 : 16;   // features per scale byte
  static constexpr int kACols = kBK / 2;              // TMEM columns of a stage of A
  static constexpr int kRawCodes = kFeat / 2 * kBK;
  static constexpr int kRawScales = 16 * kBK;         // 16 bytes a weight row, 4 or 8 the CTA's
  // The scales of a stage as the converters multiply by them: [32 c][block of the features]
  // [lane % 4][register of ldmatrix], two bf16 each; behind them, whether a byte is above 128.
  static constexpr int kFactors = kBK * 2 * (kFeat / kBlock) + 16;
  // Epilogue warps.  A pair's hold a tile's sums in registers: of eight warps with 128 rows each these
  // were too many, and spilled ones go to L2, as shared memory leaves hardly any L1 (w13 of
  // 7168 x 2048, 32 groups of 64, 128, 192 rows: 174, 195, 217 us in place of 167, 187, 209; twelve
  // warps spill none with MXFP4 and up to 28 bytes a thread with NVFP4).
  static constexpr int kEpi = P == 2 ? 12 : 4;
  static constexpr int kGroups = 3;                   // converter groups of four warps
  // Warps that make factors: NVFP4's are twice as many and take a conversion each (32 groups of
  // 64 rows, w13 by one warp 206 us, without their work 178, by two 184; w2 117, 103).
  static constexpr int kScalers = F == kMx ? 1 : 2;
  static constexpr int kConv0 = 4 + kEpi, kScaler1 = kConv0 + 4 * kGroups;  // warps
  static constexpr int kThreads = 32 * (kScaler1 + kScalers - 1);
  static constexpr int kSums = F == kNvHalves && P == 1 ? 2 : 1;  // of a tile
  static constexpr bool kHalves = F == kNvHalves && P == 2;
  // parts of the contraction, in loops of their own: of the loads, of the sums
  static constexpr int kLoads = kHalves ? 2 : 1, kParts = F == kNvHalves ? 2 : 1;
  static constexpr int kTwoMax = F != kNvHalves ? 0 : P == 2 ? 128 : 32;  // rows that have two
  static constexpr int kRowsMax = P == 2 ? 256 : 32;  // rows per tile
  static constexpr int kUnit = 16 * P;                // its N is a multiple of this
  static constexpr int kBox = kRowsMax / P, kBoxSmall = P == 2 ? 32 : 16;  // rows a TMA load
  static constexpr int kAcc = P == 2 ? 1 : 2 / kSums; // accumulators (each of kSums sums)
  static constexpr int kAccCols = kSums * kRowsMax;
  static constexpr int kSt = P == 2 ? 4 : 3;          // stages of both operands
  static constexpr int kRaw = P == 1 && F != kMx ? 6 : 7;       // of codes and scales
  static constexpr int kTmemCols = P == 2 ? 512 : 256;
  static constexpr int kTmemA = kAcc * kAccCols;      // A's stages behind the accumulators
  static constexpr int kBBytes = kRowsMax / P * kBK * 2;
  static constexpr int kOffRaw = kSt * kBBytes;
  static constexpr int kOffScale = kOffRaw + kRaw * kRawCodes;
  static constexpr int kOffFactor = kOffScale + kRaw * kRawScales;
  static constexpr int kOffBar = kOffFactor + kRaw * kFactors;
  // full, empty [St], raw_full, raw_empty, fac_full [R], acc_full, acc_empty [2], drain, half,
  // scaled
  static constexpr int kOffMisc = kOffBar + (2 * kSt + 3 * kRaw + 7) * 8;
  static constexpr int kOffGroups = kOffMisc + 16;  // tmem slot, abort flag; then off[], first[]
  static constexpr int kSmem = kOffGroups + 2 * (kMaxGroups + 1) * 4 + kThreads / 32 * 4;
  static_assert(kTmemA + kSt * kACols <= kTmemCols, "tensor memory");
  static_assert(kOffBar % 8 == 0 && kSmem <= kSmemMax / kOcc, "dynamic shared memory");
};

struct GradParams {
  const int32_t* offsets;
  const uint8_t* scales;
  const float* gs;  // NVFP4: [G] or, for two halves, [G][2] tensor scales; null: 1
  uint16_t* dx;
  int G, rows, C, F;
  uint32_t* status;
};

// Work item (chunk of a group's rows) and its tiles.
struct GradTile {
  int g, row0, rows, f0;
};

// Instruction descriptor, kind::f16: D fp32, A and B bf16 and K-major, M x n.
__device__ __forceinline__ uint32_t idesc_bf16(int m, int n) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n >> 3) << 17) |
         (static_cast<uint32_t>(m >> 4) << 24);
}

// kind::f16 MMA of an SM pair with A (each CTA's 128 rows) in tensor memory.
__device__ __forceinline__ void mma_bf16_ts_pair(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                                 uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Four 8 x 8 matrices of 16-bit values, transposed: lane l gives the address of row l % 8 of
// matrix l / 8; its register m then holds (low, high) rows 2 (l % 4), + 1 of column l / 4.
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// 16 TMEM lanes x 16 columns: lane l's registers 2 m, 2 m + 1 go to lanes l / 4, l / 4 + 8 of
// column 4 m + l % 4.
__device__ __forceinline__ void tmem_st_16x128b_x4(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
      : "memory");
}

// Arrive on an mbarrier of the pair's other CTA.  What it announces is in tensor memory,
// complete since tcgen05.wait, so the arrival orders no more than this thread's CTA sees: with a
// release for the cluster each took 1700 cycles.
__device__ __forceinline__ void mbar_arrive_other(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// One lane of a converged warp, always the same.  The warps that issue TMA loads and MMAs run
// their loops as a whole and branch to one lane for the issue alone: their addresses and
// descriptors then live in uniform registers, as those instructions take them.  (A loop that one
// lane runs alone spent 660 cycles on four MMAs and their commit.)
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r)
      :
      : "memory");
  return r != 0;
}

// A ring's slot and its phase, every `step`-th from `first` on.
template <int N, int step = 1>
struct Ring {
  static_assert(N >= step, "at most one round a step");
  uint32_t s, phase = 0, round = 0;  // round: 0 while the slots are used for the first time
  __device__ __forceinline__ explicit Ring(uint32_t first = 0) : s(first) {}
  __device__ __forceinline__ void next() {
    s += step;
    if (s >= N) s -= N, phase ^= 1u, round = 1;
  }
};

// Tile L: chunks of a group's rows (at most kRowsMax, near-equal multiples of kUnit) inside a
// block of features, so that a weight tile is read for all of its group's chunks at about the
// same time.
template <int P, int F>
__device__ __forceinline__ int chunks_of(int m) {
  return (m + Cfg<P, F>::kRowsMax - 1) / Cfg<P, F>::kRowsMax;
}
template <int P, int F>
__device__ __forceinline__ GradTile tile_at(long long L, int f_tiles, int G, const int* off,
                                            const int* first) {
  const int item = static_cast<int>(L / f_tiles);
  int lo = 0, hi = G;  // first[lo] <= item < first[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= item) lo = mid;
    else hi = mid;
  }
  const int m = off[lo + 1] - off[lo], nch = first[lo + 1] - first[lo];
  const int in = static_cast<int>(L - static_cast<long long>(first[lo]) * f_tiles);
  constexpr int U = Cfg<P, F>::kUnit;
  const int per = ((m + nch - 1) / nch + U - 1) / U * U;
  const int chunk = in % nch;
  GradTile t;
  t.g = lo;
  t.row0 = off[lo] + chunk * per;
  t.rows = m - chunk * per < per ? m - chunk * per : per;
  t.f0 = in / nch * (kFeat * P);
  return t;
}

// A register of ldmatrix: feature i's codes of two c at bits 4 i and 4 i + 16, scales s the two
// c's bytes (low, high half).  A code s e e m at bits 15 and 8..6 of a bf16 is its value times
// 2^-126, subnormals included; the factor 2^(s - 127 + 126) is a bf16 up to s = 128.
// (The product puts a copy of the code below bit 15 and one below bit 9; what the two leave
// besides sign and magnitude is masked.  Shifts and joins would double the instructions.)
__device__ __forceinline__ void codes_to_bf16(uint32_t w, uint32_t factor, uint32_t (&o)[4]) {
#pragma unroll
  for (int i = 0; i < 4; i += 2) {
    const uint32_t x = i ? w >> 8 : w;
    uint32_t v[2];
    v[0] = ((x & 0x000F000Fu) * (64 + 4096)) & 0x81C081C0u;
    v[1] = ((x & 0x00F000F0u) * (4 + 256)) & 0x81C081C0u;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const __nv_bfloat162 r = __hmul2(*reinterpret_cast<__nv_bfloat162*>(&v[j]),
                                       *reinterpret_cast<__nv_bfloat162*>(&factor));
      o[i + j] = *reinterpret_cast<const uint32_t*>(&r);
    }
  }
}
// The factor where a scale byte is above 128: 2^127 in its place, and what is left of it
// (255: NaN).
__device__ __forceinline__ uint32_t factor_most(uint32_t s) {
  const uint32_t lo = s & 0xFFFFu, hi = s >> 16;
  return (((lo < 128 ? lo : 128) + 126) << 7) | (((hi < 128 ? hi : 128) + 126) << 23);
}
__device__ __forceinline__ uint32_t factor_rest(uint32_t s) {
  const uint32_t lo = s & 0xFFFFu, hi = s >> 16;
  const uint32_t a = lo == 255 ? 0x7FC0u : (lo < 128 ? 127u : lo - 1) << 7;
  const uint32_t b = hi == 255 ? 0x7FC0u : (hi < 128 ? 127u : hi - 1) << 7;
  return a | (b << 16);
}
// TMEM lane l of a warp's 32 holds feature 4 (l % 8) + l / 8, so lanes l, l + 8, l + 16, l + 24
// have four neighbours.  Of rows (r0, r0 + 1) and (r0 + 2, r0 + 3) of its feature each lane gets
// row r0 + l / 8 of all four, for one store of 8 bytes (a store of 2 bytes a row and lane made
// the epilogue of a tile 8 us).
__device__ __forceinline__ uint2 four_rows(uint32_t r01, uint32_t r23, int lane) {
  const bool high = lane & 16, odd = lane & 8;
  const uint32_t own = high ? r23 : r01;
  const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, high ? r01 : r23, 16);
  // features (l / 8) % 2 and that + 2 of the same two rows
  const uint32_t f0 = high ? got : own, f2 = high ? own : got;
  const uint32_t mine = __byte_perm(f0, f2, odd ? 0x7632 : 0x5410);
  const uint32_t other = __shfl_xor_sync(0xFFFFFFFFu, __byte_perm(f0, f2, odd ? 0x5410 : 0x7632), 8);
  const uint32_t even = odd ? other : mine, odds = odd ? mine : other;
  return make_uint2(__byte_perm(even, odds, 0x5410), __byte_perm(even, odds, 0x7632));
}

__device__ __forceinline__ void cp_async_wait_all() {
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// A tile's scales, from weight row c (of all groups) on, kBK a stage: lane l has rows l, l + 32, ...  Of each row the CTA's
// four or eight bytes are loaded with the aligned 16 around them (which end inside the tensor: its
// size is a multiple of 512 bytes), because copies of 16 bytes pass L1 by: with 4 bytes a row 32 groups
// of one row took 158 us in place of 132.  Their arrival counts on the stage's barrier.
template <int P, int F>
struct ScaleLoad {
  const uint8_t* at;
  size_t row;
  bool there;  // (a pair's second half may lie past the last feature)
  __device__ __forceinline__ ScaleLoad(const GradParams& p, int c, int f0, int lane)
      : row(p.F / Cfg<P, F>::kBlock), there(f0 < p.F) {
    at = p.scales + (static_cast<size_t>(c) + lane) * row + f0 / Cfg<P, F>::kBlock;
  }
  __device__ __forceinline__ void stage(uint8_t* to, uint64_t* bar, int lane) {
    if (there) {
#pragma unroll
      for (int i = 0; i < kBK / 32; ++i) {
        cp_async16(to + (32 * i + lane) * 16,
                   reinterpret_cast<const void*>(reinterpret_cast<uintptr_t>(at) & ~uintptr_t(15)));
        at += 32 * row;
      }
    }
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
  }
};
// Where row c of a stage has them (`own` bytes): a stage's first row, and so a group's, starts at
// a multiple of 16 bytes.
__device__ __forceinline__ int scale_at(int c, int f0, int features, int own) {
  return c * 16 + ((c * (features / kFeat) + f0 / kFeat) & (16 / own - 1)) * own;
}
// Two E4M3 scales as bf16 factors, times 2^119 (448 * 2^119 is below bf16's largest value); the
// codes come times 2^-126, so products are short of 2^7, which the epilogue makes up for (Scaled).
__device__ __forceinline__ uint32_t factor_e4m3(uint32_t lo_hi) {
  const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2(
      static_cast<__nv_fp8x2_storage_t>(lo_hi & 0xFFFFu), __NV_E4M3);
  const float2 v = __half22float2(__half2(hr));
  return bf16x2_of(v.x * 0x1p119f, v.y * 0x1p119f);
}

// A sum short of 2^7 times its tensor scale.  The 2^7 goes to the scale where that is below 1, else
// to the sum: 128 * scale would overflow from 2^121 on, and a sum that overflows in 128 * sum does so
// with a scale of 1 or more anyway.
struct Scaled {
  float up, scale;
  __device__ __forceinline__ explicit Scaled(float gs)
      : up(fabsf(gs) >= 1.f ? 128.f : 1.f), scale(fabsf(gs) >= 1.f ? gs : 128.f * gs) {}
  __device__ __forceinline__ float of(float sum) const { return scale * (up * sum); }
};

// The halves of a group's contraction in the order of their tensor scales' magnitudes, so that the
// quotient overflows nowhere: last * (quotient * first sum + second sum).  (Of scales more than
// 2^126 apart the smaller one's half is lost.)  A NaN is the first scale or makes the quotient one,
// also where the other scale is 0; of two infinite scales the quotient is NaN.
struct Halves {
  bool swap;  // the second half first
  float quotient, last;
  __device__ __forceinline__ Halves(const float* gs, int g) {
    const float a = gs ? __ldg(gs + 2 * g) : 1.f, b = gs ? __ldg(gs + 2 * g + 1) : 1.f;
    swap = fabsf(a) > fabsf(b);
    last = swap ? a : b;
    const float other = swap ? b : a;
    quotient = last == 0.f ? other : other / last;  // (0, or the other one's NaN)
  }
};
template <int P, int F>
__device__ __forceinline__ bool rescaled(const GradTile& t) {
  return Cfg<P, F>::kHalves && t.rows > Cfg<P, F>::kTwoMax;
}
template <int P, int F>
__device__ __forceinline__ bool swapped(const GradParams& p, const GradTile& t) {
  return Cfg<P, F>::kHalves && Halves(p.gs, t.g).swap;
}
template <int P, int F>
__global__ void __launch_bounds__(Cfg<P, F>::kThreads, Cfg<P, F>::kOcc)
    k_expert_grad(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmB,
                  const __grid_constant__ CUtensorMap tmBs, const GradParams p) {
  using C = Cfg<P, F>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t rank = P == 2 ? cluster_ctarank() : 0;
  const bool leader = rank == 0;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  uint64_t* empty = full + C::kSt;
  uint64_t* raw_full = empty + C::kSt;
  uint64_t* raw_empty = raw_full + C::kRaw;
  uint64_t* fac_full = raw_empty + C::kRaw;
  uint64_t* acc_full = fac_full + C::kRaw;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* drain = acc_empty + 2;
  uint64_t* half = drain + 1;   // of a rescaled tile the first half is summed,
  uint64_t* scaled = half + 1;  // and multiplied
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);
  int* off = reinterpret_cast<int*>(smem + C::kOffGroups);
  int* first = off + kMaxGroups + 1;
  int* sums = first + kMaxGroups + 1;  // a warp's
  const int warp = __shfl_sync(0xFFFFFFFFu, static_cast<int>(threadIdx.x >> 5), 0);
  const int lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kSt; ++s) {
      mbar_init(&full[s], 1 + 4 * P);  // dy's loads, the stage's converter warps
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < C::kRaw; ++s) {
      mbar_init(&raw_full[s], 1 + 32);
      mbar_init(&raw_empty[s], 4);
      mbar_init(&fac_full[s], C::kScalers);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], C::kEpi * P);
    }
    mbar_init(drain, 1);
    mbar_init(half, 1);
    mbar_init(scaled, C::kEpi * P);
    const bool bad = (smem_u32(smem) & 1023u) != 0;
    *abort_flag = bad ? 1 : 0;
    if (bad) set_status(p.status, STATUS_BAD_PLAN);
    fence_mbar_init();
    tma_prefetch_desc(&tmW);
    tma_prefetch_desc(&tmB);
    tma_prefetch_desc(&tmBs);
  }
  if (warp == 1) {
    if (P == 2) tmem_alloc_pair(tmem_slot, C::kTmemCols);
    else tmem_alloc(tmem_slot, C::kTmemCols);
  }
  pdl_wait();
  // group offsets, and the number of chunks in front of each group
  const int G = p.G;
  for (int g = threadIdx.x; g <= G; g += C::kThreads) off[g] = p.offsets[g];
  __syncthreads();
  {
    constexpr int kPer = (kMaxGroups + C::kThreads) / C::kThreads;
    int n[kPer], total = 0;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int g = threadIdx.x * kPer + i;
      n[i] = total;
      if (g < G) {
        const int a = off[g], b = off[g + 1];
        if (a < 0 || b < a || b > p.rows) bad = true;
        else total += chunks_of<P, F>(b - a);
      }
    }
    int scan = total;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xFFFFFFFFu, scan, o);
      if (lane >= o) scan += v;
    }
    if (lane == 31) sums[warp] = scan;
    // offsets that are no plan: nothing is computed from them
    if (bad) {
      set_status(p.status, STATUS_BAD_PLAN);
      *abort_flag = 1;
    }
    __syncthreads();
    int before = scan - total;
    for (int i = 0; i < warp; ++i) before += sums[i];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int g = threadIdx.x * kPer + i;
      if (g <= G) first[g] = before + n[i];
    }
  }
  tc_fence_before();
  __syncthreads();
  if (P == 2) cluster_sync();
  tc_fence_after();
  pdl_trigger();
  const uint32_t tmem = *tmem_slot;
  const int f_tiles = (p.F + kFeat * P - 1) / (kFeat * P);
  const int nk = p.C / kBK;  // stages
  const long long total = *abort_flag ? 0 : static_cast<long long>(first[G]) * f_tiles;
  const int cl = blockIdx.x / P, ncl = gridDim.x / P;
  auto leader_addr = [&](const uint64_t* b) -> uint32_t { return mapa_shared(smem_u32(b), 0); };

  if (warp == 0) {
    // ---------------------------------------------------------------- dy
    Ring<C::kSt> st;
    bool ok = true;
    uint32_t issued = 0;
    const uint32_t bar0 = P == 2 ? leader_addr(&full[0]) : 0;
    for (long long L = cl; L < total && ok; L += ncl) {
      const GradTile t = tile_at<P, F>(L, f_tiles, G, off, first);
      const int mine = (t.rows + C::kUnit - 1) / C::kUnit * C::kUnit / P;  // rows in this CTA
      const int row0 = t.row0 + static_cast<int>(rank) * mine;
      const bool small = mine <= P * C::kBoxSmall;  // (at most P loads)
      const int box = small ? C::kBoxSmall : C::kBox, boxes = (mine + box - 1) / box;
      const CUtensorMap* map = small ? &tmBs : &tmB;
      const uint32_t bytes = P * boxes * box * kBK * 2;
      const bool swap = swapped<P, F>(p, t);
      for (int part = 0; part < C::kLoads; ++part) {
        int c = (part != 0) != swap ? p.C / 2 : 0;
        for (int kb = 0; kb < nk / C::kLoads; ++kb, c += kBK, ++issued, st.next()) {
          if (st.round) ok = mbar_wait(&empty[st.s], st.phase ^ 1u, p.status, abort_flag);
          ok = __all_sync(0xFFFFFFFFu, ok);  // (the lanes part only together)
          if (!ok) break;
          uint8_t* b = smem + st.s * C::kBBytes;
          if (elect_one()) {
            if (leader) mbar_arrive_expect_tx(&full[st.s], bytes);
#pragma unroll
            for (int h = 0; h < kBK / 64; ++h)  // 64 c, one 128-byte swizzle row, each
              for (int i = 0; i < boxes; ++i) {
                uint8_t* to = b + (h * (C::kRowsMax / P) + i * box) * 128;
                if (P == 2)
                  tma_load_2d_pair(to, map, bar0 + st.s * 8, c + h * 64, row0 + i * box);
                else
                  tma_load_2d(to, map, &full[st.s], c + h * 64, row0 + i * box);
              }
          }
        }
        if (!ok) break;
      }
    }
    // after an abort: the loads still in flight (all counted on the first CTA's barriers)
    if (leader && *abort_flag) {
      const uint32_t from = issued > C::kSt ? issued - C::kSt : 0;
      for (uint32_t i = from; i < issued; ++i)
        mbar_wait_drain(&full[i % C::kSt], (i / C::kSt) & 1u);
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA
    if (leader) {
      Ring<C::kSt> st;
      uint32_t tc = 0, rescales = 0;
      bool ok = true;
      // (of a descriptor only the address, the low 14 bits, moves)
      const uint64_t db0 = smem_desc(smem_u32(smem), 0, 1024, kLayoutSw128);
      for (long long L = cl; L < total && ok; L += ncl, ++tc) {
        const GradTile t = tile_at<P, F>(L, f_tiles, G, off, first);
        const uint32_t idesc =
            idesc_bf16(kFeat * P, (t.rows + C::kUnit - 1) / C::kUnit * C::kUnit);
        const uint32_t b = tc % C::kAcc, use = tc / C::kAcc;
        if (use) ok = mbar_wait(&acc_empty[b], (use - 1) & 1u, p.status, abort_flag);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) break;
        tc_fence_after();
        const uint32_t d0 = tmem + b * C::kAccCols;
        const bool twice = rescaled<P, F>(t), two = C::kTwoMax && !twice;
        for (int part = 0; part < C::kParts; ++part) {
          if (part && twice) {
            if (elect_one()) tc_commit_pair_mc(half, 3);
            __syncwarp();
            ok = mbar_wait(scaled, rescales++ & 1u, p.status, abort_flag);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) break;
            tc_fence_after();
          }
          const uint32_t d = d0 + (part && two ? C::kTwoMax : 0);
          const bool add = part && twice;
          for (int kb = 0; kb < nk / C::kParts; ++kb, st.next()) {
            ok = __all_sync(0xFFFFFFFFu, mbar_wait(&full[st.s], st.phase, p.status, abort_flag));
            if (!ok) break;
            tc_fence_after();
            const uint32_t at = tmem + C::kTmemA + st.s * C::kACols;
            const uint32_t db = static_cast<uint32_t>(db0) + st.s * (C::kBBytes / 16);
            if (elect_one()) {
#pragma unroll
              for (int kk = 0; kk < kBK / 16; ++kk) {
                const uint64_t dk = (db0 >> 32) << 32 |
                                    (db + kk / 4 * (C::kRowsMax / P * 128 / 16) + kk % 4 * 2);
                if (P == 2) mma_bf16_ts_pair(d, at + kk * 8, dk, idesc, add || kb > 0 || kk > 0);
                else mma_bf16_ts(d, at + kk * 8, dk, idesc, add || kb > 0 || kk > 0);
              }
              if (P == 2) tc_commit_pair_mc(&empty[st.s], 3);
              else tc_commit(&empty[st.s]);
            }
            __syncwarp();
          }
          if (!ok) break;
        }
        if (ok && elect_one()) {
          if (P == 2) tc_commit_pair_mc(&acc_full[b], 3);
          else tc_commit(&acc_full[b]);
        }
        __syncwarp();
      }
      // after an abort: the MMAs already issued
      if (__any_sync(0xFFFFFFFFu, *abort_flag != 0)) {
        if (elect_one()) {
          if (P == 2) tc_commit_pair_mc(drain, 1);
          else tc_commit(drain);
        }
        mbar_wait_drain(drain, 0);
      }
    }
  } else if (warp == 2) {
    // ---------------------------------------------------------------- codes and scales
    Ring<C::kRaw> st;
    bool ok = true;
    uint32_t issued = 0;
    for (long long L = cl; L < total && ok; L += ncl) {
      const GradTile t = tile_at<P, F>(L, f_tiles, G, off, first);
      const int f0 = t.f0 + static_cast<int>(rank) * kFeat;
      const bool swap = swapped<P, F>(p, t);
      for (int part = 0; part < C::kLoads; ++part) {
        int c = t.g * p.C + ((part != 0) != swap ? p.C / 2 : 0);  // of all the groups' weight rows
        ScaleLoad<P, F> sc(p, c, f0, lane);
        for (int kb = 0; kb < nk / C::kLoads; ++kb, c += kBK, ++issued, st.next()) {
          if (st.round) ok = mbar_wait(&raw_empty[st.s], st.phase ^ 1u, p.status, abort_flag);
          ok = __all_sync(0xFFFFFFFFu, ok);
          if (!ok) break;
          if (elect_one()) {
            mbar_arrive_expect_tx(&raw_full[st.s], C::kRawCodes);
            tma_load_2d(smem + C::kOffRaw + st.s * C::kRawCodes, &tmW, &raw_full[st.s], f0 / 2, c);
          }
          __syncwarp();
          sc.stage(smem + C::kOffScale + st.s * C::kRawScales, &raw_full[st.s], lane);
        }
        if (!ok) break;
      }
    }
    cp_async_wait_all();
    __syncwarp();
    if (*abort_flag) {
      const uint32_t from = issued > C::kRaw ? issued - C::kRaw : 0;
      for (uint32_t i = from; i < issued; ++i)
        mbar_wait_drain(&raw_full[i % C::kRaw], (i / C::kRaw) & 1u);
    }
  } else if (warp == 3 || warp >= C::kScaler1) {
    // ---------------------------------------------------------------- factors
    // lane l has c = 2 l, 2 l + 1 of every 64: a bf16 factor each for every block of features,
    // of an E8M0 byte s 2^(s - 127 + 126); of two warps each has every other 64
    const int h0 = C::kScalers > 1 && warp != 3;
    constexpr int kBlocks = kFeat / C::kBlock, kOwn = kBlocks;  // bytes a row
    Ring<C::kRaw> st;
    bool ok = true;
    uint32_t* to = reinterpret_cast<uint32_t*>(smem + C::kOffFactor) + (lane >> 4) * (kBlocks * 16) +
                   (lane & 3) * 4 + ((lane >> 2) & 3);
    for (long long L = cl; L < total && ok; L += ncl) {
      const GradTile t = tile_at<P, F>(L, f_tiles, G, off, first);
      const int f0 = t.f0 + static_cast<int>(rank) * kFeat;
      const uint8_t* lo = smem + C::kOffScale + scale_at(2 * lane, f0, p.F, kOwn);
      const uint8_t* hi = smem + C::kOffScale + scale_at(2 * lane + 1, f0, p.F, kOwn);
      for (int kb = 0; kb < nk; ++kb, st.next()) {
        ok = __all_sync(0xFFFFFFFFu, mbar_wait(&raw_full[st.s], st.phase, p.status, abort_flag));
        if (!ok) break;
        uint32_t over = 0;
#pragma unroll
        for (int i = 0; i < kBK / 64 / C::kScalers; ++i) {
          const int h = h0 + i * C::kScalers;
          // (64 rows further the bytes' place in their 16 is the same)
          const int at = st.s * C::kRawScales + h * 1024;
          uint32_t* out = to + st.s * (C::kFactors / 4) + h * (kBlocks * 32);
#pragma unroll
          for (int v = 0; v < kOwn / 4; ++v) {
            const uint32_t x = *reinterpret_cast<const uint32_t*>(lo + at + 4 * v);
            const uint32_t y = *reinterpret_cast<const uint32_t*>(hi + at + 4 * v);
            if (F == kMx)  // a byte above 128 has its highest bit and another
              over |= (((x & 0x7F7F7F7Fu) + 0x7F7F7F7Fu) & x) |
                      (((y & 0x7F7F7F7Fu) + 0x7F7F7F7Fu) & y);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              if (F == kMx)
                out[q * 16] =
                    (__byte_perm(x, y, q | (4 + q) << 8) & 0x00FF00FFu) * 128 + 0x3F003F00u;
              else
                out[(4 * v + q) * 16] = factor_e4m3(__byte_perm(x, y, q | (4 + q) << 4));
            }
          }
        }
        const bool any = __any_sync(0xFFFFFFFFu, (over & 0x80808080u) != 0);
        if (F == kMx && lane == 0) {
          *reinterpret_cast<uint32_t*>(smem + C::kOffFactor + st.s * C::kFactors + C::kFactors - 16) =
              any;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&fac_full[st.s]);
      }
    }
  } else if (warp >= C::kConv0) {
    // ---------------------------------------------------------------- converters
    const int q = warp & 3;  // its features' quarter, and TMEM lanes
    // (64-byte swizzle: eight rows' 16-byte chunks fall on all the banks)
    const uint32_t src =
        smem_u32(smem + C::kOffRaw) + lane * 64 + ((q ^ ((lane >> 1) & 3)) << 4);
    // (a lane's four features: in the warp's one block of 32, or the first or second of 16)
    constexpr int kStep = 64 * (kFeat / C::kBlock);  // bytes of factors per 32 c
    const uint8_t* factors =
        smem + C::kOffFactor + (F == kMx ? q : 2 * q + (lane >> 4)) * 64 + (lane & 3) * 16;
    const uint32_t dst = tmem + (static_cast<uint32_t>(q * 32) << 16) + C::kTmemA;
    const uint32_t tiles = cl < total ? static_cast<uint32_t>((total - cl + ncl - 1) / ncl) : 0;
    const unsigned long long end = static_cast<unsigned long long>(tiles) * nk;
    const uint32_t group = (warp - C::kConv0) >> 2;
    const uint32_t full0 = P == 2 ? leader_addr(&full[0]) : 0;
    Ring<C::kSt, C::kGroups> ra(group);
    Ring<C::kRaw, C::kGroups> rr(group);
    for (unsigned long long n = group; n < end; n += C::kGroups, ra.next(), rr.next()) {
      bool w_ok = mbar_wait(&fac_full[rr.s], rr.phase, p.status, abort_flag);
      if (w_ok && ra.round) w_ok = mbar_wait(&empty[ra.s], ra.phase ^ 1u, p.status, abort_flag);
      if (!__all_sync(0xFFFFFFFFu, w_ok)) break;
      tc_fence_after();
      const uint32_t over = *reinterpret_cast<const uint32_t*>(
          smem + C::kOffFactor + rr.s * C::kFactors + C::kFactors - 16);
      constexpr int kH = kBK / 32;  // 32 c each
      const uint32_t to = dst + ra.s * C::kACols;
      if (F != kMx || !over) {
#pragma unroll
        for (int h = 0; h < kH; ++h) {
          uint32_t w[4], lo[8], hi[8];  // features 0, 1 and 2, 3 of the thread's four
          ldmatrix_x4_trans(src + rr.s * C::kRawCodes + h * 2048, w);
          const uint4 f = *reinterpret_cast<const uint4*>(factors + rr.s * C::kFactors + h * kStep);
          if (h == kH - 1) {
            __syncwarp();
            if (lane == 0) mbar_arrive(&raw_empty[rr.s]);
          }
          const uint32_t f4[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            uint32_t o[4];
            codes_to_bf16(w[m], f4[m], o);
            lo[2 * m] = o[0], lo[2 * m + 1] = o[1], hi[2 * m] = o[2], hi[2 * m + 1] = o[3];
          }
          tmem_st_16x128b_x4(to + h * 16, lo);
          tmem_st_16x128b_x4(to + h * 16 + (16u << 16), hi);
        }
      } else {  // a scale byte above 128: two factors, from the bytes
#pragma unroll 1
        for (int h = 0; h < kH; ++h) {
          uint32_t w[4], lo[8], hi[8];
          ldmatrix_x4_trans(src + rr.s * C::kRawCodes + h * 2048, w);
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            // the two bytes again, of what the factor's arithmetic made of them
            const uint32_t f = *reinterpret_cast<const uint32_t*>(
                factors + rr.s * C::kFactors + h * kStep + m * 4);
            const uint32_t sc = ((f - 0x3F003F00u) >> 7) & 0x01FF01FFu;
            uint32_t o[4], rest = factor_rest(sc);
            codes_to_bf16(w[m], factor_most(sc), o);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const __nv_bfloat162 r = __hmul2(*reinterpret_cast<__nv_bfloat162*>(&o[i]),
                                               *reinterpret_cast<__nv_bfloat162*>(&rest));
              o[i] = *reinterpret_cast<const uint32_t*>(&r);
            }
            lo[2 * m] = o[0], lo[2 * m + 1] = o[1], hi[2 * m] = o[2], hi[2 * m + 1] = o[3];
          }
          __syncwarp();
          tmem_st_16x128b_x4(to + h * 16, lo);
          tmem_st_16x128b_x4(to + h * 16 + (16u << 16), hi);
        }
        if (lane == 0) mbar_arrive(&raw_empty[rr.s]);
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (P == 2 && !leader) mbar_arrive_other(full0 + ra.s * 8);
        else mbar_arrive(&full[ra.s]);
      }
    }
  } else if (warp >= 4) {
    // ---------------------------------------------------------------- epilogue
    // P = 2: one accumulator, so the sums are first all taken to registers (twelve warps, three
    // for the same lanes with a part of the tile's rows each) and stored under the next tile's MMAs.
    const int q = warp & 3;
    constexpr int kShares = P == 2 ? C::kEpi / 4 : 1;
    constexpr int kCols = P == 2 ? (C::kRowsMax + kShares * 8 - 1) / (kShares * 8) * 8 : 16;
    uint32_t tc = 0, rescales = 0;
    for (long long L = cl; L < total; L += ncl, ++tc) {
      const GradTile t = tile_at<P, F>(L, f_tiles, G, off, first);
      const uint32_t b = tc % C::kAcc, use = tc / C::kAcc;
      // the warp's rows of the tile (columns of the sums)
      const int part = P == 2 ? (t.rows + kShares * 8 - 1) / (kShares * 8) * 8 : t.rows;
      const int c0 = P == 2 ? ((warp - 4) >> 2) * part : 0;
      const int own = t.rows - c0 < part ? t.rows - c0 : part;
      const uint32_t acc = tmem + (static_cast<uint32_t>(q * 32) << 16) + b * C::kAccCols + c0;
      int w_ok = 1;
      Scaled gs0(1.f), gs1(1.f);
      const bool twice = rescaled<P, F>(t);
      if (C::kHalves) {  // the first sum times the quotient, plus the second if that is apart
        const Halves h(p.gs, t.g);
        gs0 = Scaled(h.last);
        if (lane == 0) {
          if (twice) w_ok = mbar_wait(half, rescales & 1u, p.status, abort_flag);
          else w_ok = mbar_wait(&acc_full[b], use & 1u, p.status, abort_flag);
        }
        rescales += twice;
        if (!__shfl_sync(0xFFFFFFFFu, w_ok, 0)) break;
        tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < own; c += 8) {
          uint32_t x[8], y[8] = {};
          tmem_ld_32x32b_x8(acc + c, x);
          if (!twice) tmem_ld_32x32b_x8(acc + C::kTwoMax + c, y);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 8; ++i)
            x[i] = __float_as_uint(
                fmaf(h.quotient, __uint_as_float(x[i]), __uint_as_float(y[i])));
          tmem_st_32x32b_x8(acc + c, x);
        }
        tmem_st_wait();
        if (twice) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            if (!leader) mbar_arrive_other(leader_addr(scaled));
            else mbar_arrive(scaled);
          }
        }
      } else if (F != kMx) {
        gs0 = Scaled(p.gs ? __ldg(p.gs + t.g * C::kSums) : 1.f);
        if (C::kSums == 2) gs1 = Scaled(p.gs ? __ldg(p.gs + t.g * 2 + 1) : 1.f);
      }
      if (lane == 0) w_ok = mbar_wait(&acc_full[b], use & 1u, p.status, abort_flag);
      if (!__shfl_sync(0xFFFFFFFFu, w_ok, 0)) break;
      tc_fence_after();
      const int f = t.f0 + static_cast<int>(rank) * kFeat + q * 32;
      const int rows = f < p.F ? own : 0;
      uint16_t* out = p.dx + static_cast<size_t>(t.row0 + c0 + (lane >> 3)) * p.F + f + 4 * (lane & 7);
      auto release = [&] {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (P == 2 && !leader) mbar_arrive_other(leader_addr(&acc_empty[b]));
          else mbar_arrive(&acc_empty[b]);
        }
      };
      // two rows a register (without the zeros they count as live from tile to tile)
      uint32_t v[kCols / 2] = {};
      for (int r0 = 0; r0 < (P == 2 ? 1 : rows); r0 += kCols) {
#pragma unroll
        for (int c = 0; c < kCols; c += 8) {
          if (r0 + c < rows) {
            uint32_t x[8];
            tmem_ld_32x32b_x8(acc + r0 + c, x);
            if (C::kSums == 2) {
              uint32_t y[8];
              tmem_ld_32x32b_x8(acc + C::kTwoMax + r0 + c, y);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 8; ++i)
                x[i] = __float_as_uint(fmaf(gs0.scale, gs0.up * __uint_as_float(x[i]),
                                            gs1.of(__uint_as_float(y[i]))));
            } else {
              tmem_ld_wait();
              if (F != kMx) {
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = __float_as_uint(gs0.of(__uint_as_float(x[i])));
              }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
              v[c / 2 + i] = bf16x2_of(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1]));
          }
        }
        if (P == 2) release();
#pragma unroll
        for (int c = 0; c < kCols; c += 4)
          if (r0 + c < rows) {
            const uint2 o = four_rows(v[c / 2], v[c / 2 + 1], lane);
            if (r0 + c + (lane >> 3) < rows)
              *reinterpret_cast<uint2*>(out + static_cast<size_t>(r0 + c) * p.F) = o;
          }
      }
      if (P == 1) release();
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (P == 2) cluster_sync();  // neither CTA releases what the pair still uses
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    if (P == 2) tmem_dealloc_pair(tmem, C::kTmemCols);
    else tmem_dealloc(tmem, C::kTmemCols);
  }
}

bool encode_w(CUtensorMap* m, const ExpertGradCall& a, int box_rows) {
  EncodeTiledFn enc = get_encode_tiled_fn();
  if (!enc) return false;
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(a.F) / 2, static_cast<cuuint64_t>(a.G) * a.C};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(a.F) / 2};
  cuuint32_t box[2] = {kFeat / 2, static_cast<cuuint32_t>(box_rows)}, es[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(a.w), dims, strides, box,
             es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
         CUDA_SUCCESS;
}

bool encode_dy(CUtensorMap* m, const ExpertGradCall& a, int box_rows) {
  EncodeTiledFn enc = get_encode_tiled_fn();
  if (!enc) return false;
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(a.C), static_cast<cuuint64_t>(a.rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(a.C) * 2};
  cuuint32_t box[2] = {64, static_cast<cuuint32_t>(box_rows)}, es[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<uint16_t*>(a.dy), dims, strides,
             box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
         CUDA_SUCCESS;
}

template <int P, int F>
cudaError_t launch_grad(const ExpertGradCall& a, cudaStream_t st) {
  using C = Cfg<P, F>;
  static OncePerContext once;  // how many of its clusters fit the GPU at once
  int dev = 0, clusters = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= OncePerContext::kDevices) return cudaErrorInvalidDevice;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = P;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = st;
  if (once.ready(dev, current_context_id())) {
    clusters = once.value(dev);
  } else {
    e = cudaFuncSetAttribute(k_expert_grad<P, F>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             C::kSmem);
    if (e != cudaSuccess) return e;
    int sms = 0;
    e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    if (P == 2) {
      cfg.gridDim = dim3(sms / P * P);
      cfg.attrs = attr + 1;
      cfg.numAttrs = 1;
      e = cudaOccupancyMaxActiveClusters(&clusters, k_expert_grad<P, F>, &cfg);
      if (e != cudaSuccess) return e;
      if (clusters < 1) return cudaErrorInvalidConfiguration;
    } else {
      clusters = sms * C::kOcc;  // (the query says one CTA per SM of any kernel with tensor memory)
    }
    once.set(dev, clusters);
  }
  CUtensorMap tmW, tmB, tmBs;
  if (!encode_w(&tmW, a, kBK) || !encode_dy(&tmB, a, C::kBox) || !encode_dy(&tmBs, a, C::kBoxSmall))
    return cudaErrorInvalidValue;
  const GradParams p = {a.offsets, a.w_s, a.gs, a.dx, a.G, a.rows, a.C, a.F, a.status};
  cfg.gridDim = dim3(clusters * P);
  cfg.attrs = attr;
  cfg.numAttrs = P == 2 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, k_expert_grad<P, F>, tmW, tmB, tmBs, p);
}

// The form that should take less time, from what the host knows: the dims, not the routing.  Of
// a form's tiles as many run at once as CTAs or pairs fit, each a stage's time per stage and a
// tile's own besides.  A group of R / E rows is taken to have one chunk up to three quarters of a
// tile's rows, above that what its rows fill and 0.4 (the groups' sizes vary).  Costs as measured
// on GB300, weights from HBM (us; P = 1 and 2): w13 of 7168 x 2048, 32 groups of 24, 33, 40 rows:
// 113, 223, 224 and 167, 168, 168; 8 groups of 30, 64: 41, 62 and 48, 48; 2 groups of 32, 100: 17, 41
// and 19, 21; w13 and w2 of 2048 x 1024, 16 groups of 50: 25, 15.2 and 21, 13.7; w2 of 1024 x 1024,
// 64 groups of 20, 40: 17, 27 and 23, 23; w2 of 1280 x 768, 13 groups of 60, 179: 11.1, 18.0 and
// 10.8, 12.8 (NVFP4 up to a tenth more of each).
// (The formats' tiles have the same rows, features and stages.)
template <int P>
double cost_us(const ExpertGradCall& a) {
  using C = Cfg<P, kMx>;
  const double M = C::kRowsMax, groups = a.routed < a.E ? a.routed : a.E;
  auto chunks = [&](double rows) { return rows <= 0.75 * M ? 1.0 : rows / M + 0.4; };
  double items = groups * chunks(a.routed / groups);
  if (a.G > a.E) items += chunks(a.rows - a.routed);
  const double tiles = items * ((a.F + kFeat * P - 1) / (kFeat * P));
  const double waves = ceil(tiles * P / (kSms * C::kOcc));
  const double stages = a.C / kBK;
  // (a CTA that has its SM for itself is faster: w2 of 2048 x 1024, 16 groups of 24 rows 11.4 us; a
  // pair's MMAs take longer for more rows)
  const bool alone = tiles <= kSms;
  if (P == 1) return (alone ? 3.8 : 4.5) + waves * (stages * (alone ? 0.38 : 0.56) + 1.2);
  const double rows = a.rows / items;
  return 6.2 + waves * (stages * (0.36 + 0.28 * (rows < M ? rows / M : 1.0)) + 0.7);
}

template <int F>
cudaError_t launch_form(const ExpertGradCall& a, int ctas, cudaStream_t st) {
  return ctas == 1 ? launch_grad<1, F>(a, st) : launch_grad<2, F>(a, st);
}

}  // namespace

int expert_grad_ctas(const ExpertGradCall& a) {
  return cost_us<1>(a) <= cost_us<2>(a) ? 1 : 2;
}

cudaError_t launch_expert_grad(const ExpertGradCall& a, int ctas, cudaStream_t st) {
  if (!a.nv) return launch_form<kMx>(a, ctas, st);
  return a.gs_segments == 2 ? launch_form<kNvHalves>(a, ctas, st) : launch_form<kNv>(a, ctas, st);
}

}  // namespace moe
