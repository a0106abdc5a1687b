// Gradient products of the MXFP4 experts: for every packed row r of group g
//     dx[r][f] = sum_c dy[r][c] * deq(w[g])[c][f]
// with w [G][C][F/2] (E2M1 codes) and scales [G][C][F/32] as the forward has them: W2 is
// [H][I] (C = H, F = I), W13 [2I][H] (C = 2I, F = H).
//
// The contraction runs over the weight's ROWS, so its scales (one per 32 elements of a row)
// lie along the output axis: the block-scaled MMA kinds, whose scales go along the
// contraction, cannot apply them, and a transposed copy would be a second set of weights.  The
// kernel multiplies in bf16 instead: E2M1 times a power of two is exact there (2 significant
// bits), dy is bf16 as it comes, the products are exact in fp32 and are summed in fp32.
//
// A tile is 128 features (the MMA's M side) x up to 256 rows of one group (its N side, a
// multiple of 16); a stage is 64 values of c:
//   * warp 2 brings the codes of 64 weight rows x 128 features (4 KB, TMA) and their scales
//     (cp.async: 4 bytes a row) into a ring of their own, so that many stages of the weights
//     are on their way from HBM;
//   * eight converter warps turn them into bf16 in shared memory, MN-major with the 128-byte
//     swizzle (64 features of one c are a 128-byte row): a thread has 32 codes of one weight
//     row and so one scale;
//   * warp 0 brings dy's rows (K-major, TMA), warp 1 issues the MMAs;
//   * four warps store the fp32 sums of the last tile from TMEM under the next one's MMAs.
// Persistent CTAs; every CTA finds its tiles from the group offsets by itself (no plan kernel).
// Every wait is bounded; one that expires sets the workspace's status word.
#include "grad.cuh"

namespace moe {

namespace {

constexpr int kBK = 64;          // c per stage: one 128-byte row of dy
constexpr int kFeat = 128;       // features per tile
constexpr int kRowsMax = 256;    // rows per tile
constexpr int kMaxGroups = 1025;
constexpr int kConvWarps = 8;
constexpr int kThreads = 32 * (8 + kConvWarps);

constexpr int kABytes = kFeat * kBK * 2;
constexpr int kBBytes = kRowsMax * kBK * 2;
constexpr int kStageBytes = kABytes + kBBytes;
constexpr int kStages = 3;
constexpr int kRawCodes = kFeat / 2 * kBK;
constexpr int kRawScales = kFeat / 32 * kBK;
constexpr int kRaw = 12;
constexpr int kOffRaw = kStages * kStageBytes;
constexpr int kOffScale = kOffRaw + kRaw * kRawCodes;
constexpr int kOffBar = kOffScale + kRaw * kRawScales;
// full[S], empty[S], raw_full[R], raw_empty[R], acc_full[2], acc_empty[2], drain
constexpr int kOffMisc = kOffBar + (2 * kStages + 2 * kRaw + 5) * 8;
constexpr int kOffGroups = kOffMisc + 16;  // tmem slot, abort flag; then off[], first[]
constexpr int kSmem = kOffGroups + 2 * (kMaxGroups + 1) * 4 + 64;
static_assert(kSmem <= kSmemMax, "dynamic shared memory of one CTA");

struct GradParams {
  const int32_t* offsets;
  const uint8_t* scales;
  uint16_t* dx;
  int G, rows, C, F;
  uint32_t* status;
};

// Work item (chunk of a group's rows) and its tiles.
struct GradTile {
  int g, row0, rows, f0;
};

__device__ __forceinline__ uint32_t idesc_a_mn(int n) {  // bf16, A MN-major, M = 128
  return (1u << 4) | (1u << 7) | (1u << 10) | (1u << 15) | (static_cast<uint32_t>(n >> 3) << 17) |
         (static_cast<uint32_t>(128 >> 4) << 24);
}

// Rows of a group in chunks of at most kRowsMax, near-equal multiples of 16.
__device__ __forceinline__ int chunks_of(int m) { return (m + kRowsMax - 1) / kRowsMax; }

// Tile L: items chunk by chunk inside a group, for one block of features after the other, so
// that a weight tile is read for all of its group's chunks at about the same time.
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
  const int per = ((m + nch - 1) / nch + 15) & ~15;
  const int chunk = in % nch;
  GradTile t;
  t.g = lo;
  t.row0 = off[lo] + chunk * per;
  t.rows = m - chunk * per < per ? m - chunk * per : per;
  t.f0 = in / nch * kFeat;
  return t;
}

// Eight codes (a word, the code of feature i in bits 4 i..) to bf16 at memory positions
// 0..7 = features 0, 4, 1, 5, 2, 6, 3, 7 (codes 16 bits apart share a register).  A code
// s e e m put at bits 15 and 8..6 of a bf16 is its value times 2^-126, subnormals included;
// mul is the scale times 2^126.
__device__ __forceinline__ void codes_to_bf16(uint32_t w, __nv_bfloat162 mul, uint32_t (&o)[4]) {
  const uint32_t s[4] = {w << 12, w << 8, w << 4, w};
  const uint32_t m[4] = {w << 6, w << 2, w >> 2, w >> 6};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t v = (s[j] & 0x80008000u) | (m[j] & 0x01C001C0u);
    const __nv_bfloat162 r = __hmul2(*reinterpret_cast<__nv_bfloat162*>(&v), mul);
    o[j] = *reinterpret_cast<const uint32_t*>(&r);
  }
}
// Position p of those eight holds feature:
__device__ __forceinline__ int feature_at(int p) {
  return (p & ~7) | ((p & 1) << 2) | ((p & 7) >> 1);
}

__global__ void __launch_bounds__(kThreads, 1)
    k_expert_grad(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmB,
                  const __grid_constant__ CUtensorMap tmBs, const GradParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kOffBar);
  uint64_t* empty = full + kStages;
  uint64_t* raw_full = empty + kStages;
  uint64_t* raw_empty = raw_full + kRaw;
  uint64_t* acc_full = raw_empty + kRaw;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* drain = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kOffMisc + 4);
  int* off = reinterpret_cast<int*>(smem + kOffGroups);
  int* first = off + kMaxGroups + 1;
  int* sums = first + kMaxGroups + 1;  // of 16 warps
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1 + kConvWarps);
      mbar_init(&empty[s], 1);
    }
    for (int s = 0; s < kRaw; ++s) {
      mbar_init(&raw_full[s], 1 + 32);
      mbar_init(&raw_empty[s], kConvWarps);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 4);
    }
    mbar_init(drain, 1);
    const bool bad = (smem_u32(smem) & 1023u) != 0;
    *abort_flag = bad ? 1 : 0;
    if (bad) set_status(p.status, STATUS_BAD_PLAN);
    fence_mbar_init();
    tma_prefetch_desc(&tmW);
    tma_prefetch_desc(&tmB);
    tma_prefetch_desc(&tmBs);
  }
  if (warp == 1) tmem_alloc(tmem_slot, 512);
  pdl_wait();
  // group offsets, and the number of chunks in front of each group
  const int G = p.G;
  for (int g = threadIdx.x; g <= G; g += kThreads) off[g] = p.offsets[g];
  __syncthreads();
  {
    constexpr int kPer = (kMaxGroups + kThreads - 1) / kThreads;
    int n[kPer], total = 0;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int g = threadIdx.x * kPer + i;
      n[i] = total;
      if (g < G) {
        const int a = off[g], b = off[g + 1];
        if (a < 0 || b < a || b > p.rows) bad = true;
        else total += chunks_of(b - a);
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
  tc_fence_after();
  pdl_trigger();
  const uint32_t tmem = *tmem_slot;
  const int f_tiles = p.F / kFeat, nk = p.C / kBK;
  const long long total = *abort_flag ? 0 : static_cast<long long>(first[G]) * f_tiles;

  if (warp == 0) {
    // ---------------------------------------------------------------- dy
    if (lane == 0) {
      uint32_t it = 0;
      bool ok = true;
      for (long long L = blockIdx.x; L < total && ok; L += gridDim.x) {
        const GradTile t = tile_at(L, f_tiles, G, off, first);
        const bool small = t.rows <= 64;  // boxes of 32 rows, else of 128
        const int box = small ? 32 : 128, boxes = (t.rows + box - 1) / box;
        for (int kb = 0; kb < nk; ++kb, ++it) {
          const int s = it % kStages;
          if (it >= kStages &&
              !mbar_wait(&empty[s], ((it / kStages) & 1u) ^ 1u, p.status, abort_flag)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&full[s], boxes * box * kBK * 2);
          uint8_t* b = smem + s * kStageBytes + kABytes;
          for (int i = 0; i < boxes; ++i)
            tma_load_2d(b + i * box * kBK * 2, small ? &tmBs : &tmB, &full[s], kb * kBK,
                        t.row0 + i * box);
        }
      }
      if (*abort_flag) {
        const uint32_t from = it > kStages ? it - kStages : 0;
        for (uint32_t i = from; i < it; ++i) mbar_wait_drain(&full[i % kStages], (i / kStages) & 1u);
      }
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA
    if (lane == 0) {
      uint32_t it = 0, tc = 0;
      bool ok = true;
      for (long long L = blockIdx.x; L < total && ok; L += gridDim.x, ++tc) {
        const GradTile t = tile_at(L, f_tiles, G, off, first);
        const uint32_t idesc = idesc_a_mn((t.rows + 15) & ~15);
        const uint32_t b = tc & 1u, use = tc >> 1;
        if (tc >= 2 && !mbar_wait(&acc_empty[b], (use - 1) & 1u, p.status, abort_flag)) break;
        tc_fence_after();
        const uint32_t d = tmem + b * kRowsMax;
        for (int kb = 0; kb < nk; ++kb, ++it) {
          const int s = it % kStages;
          if (!mbar_wait(&full[s], (it / kStages) & 1u, p.status, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a0 = smem_u32(smem + s * kStageBytes);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_bf16_ss(d, smem_desc(a0 + kk * 2048, kBK * 128, 1024, kLayoutSw128),
                        smem_desc(a0 + kABytes + kk * 32, 0, 1024, kLayoutSw128), idesc,
                        kb > 0 || kk > 0);
          tc_commit(&empty[s]);
        }
        if (ok) tc_commit(&acc_full[b]);
      }
      if (*abort_flag) {
        tc_commit(drain);
        mbar_wait_drain(drain, 0);
      }
    }
  } else if (warp == 2) {
    // ---------------------------------------------------------------- codes and scales
    uint32_t it = 0;
    bool ok = true;
    for (long long L = blockIdx.x; L < total && ok; L += gridDim.x) {
      const GradTile t = tile_at(L, f_tiles, G, off, first);
      const uint8_t* sc = p.scales + static_cast<size_t>(t.g) * p.C * (p.F / 32) + t.f0 / 32;
      for (int kb = 0; kb < nk; ++kb, ++it) {
        const int s = it % kRaw;
        int w_ok = 1;
        if (it >= kRaw) {
          if (lane == 0)
            w_ok = mbar_wait(&raw_empty[s], ((it / kRaw) & 1u) ^ 1u, p.status, abort_flag);
          w_ok = __shfl_sync(0xFFFFFFFFu, w_ok, 0);
        }
        if (!w_ok) {
          ok = false;
          break;
        }
        if (lane == 0) {
          mbar_arrive_expect_tx(&raw_full[s], kRawCodes);
          tma_load_2d(smem + kOffRaw + s * kRawCodes, &tmW, &raw_full[s], t.f0 / 2,
                      t.g * p.C + kb * kBK);
        }
        uint8_t* ds = smem + kOffScale + s * kRawScales;
#pragma unroll
        for (int i = 0; i < kBK; i += 32)
          cp_async4(ds + (i + lane) * 4, sc + static_cast<size_t>(kb * kBK + i + lane) * (p.F / 32));
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(
                         smem_u32(&raw_full[s]))
                     : "memory");
      }
    }
    cp_async_commit();
    cp_async_wait<0>();
    __syncwarp();
    if (lane == 0 && *abort_flag) {
      const uint32_t from = it > kRaw ? it - kRaw : 0;
      for (uint32_t i = from; i < it; ++i) mbar_wait_drain(&raw_full[i % kRaw], (i / kRaw) & 1u);
    }
  } else if (warp >= 8) {
    // ---------------------------------------------------------------- converters
    // A warp has 32 weight rows x 32 features of the stage: with a row a lane, a quarter
    // warp's 16-byte accesses fall on all the banks on both sides.
    const int cw = warp - 8, q = cw & 3, row = (cw >> 2) * 32 + lane;
    const uint32_t src = row * 64 + ((q ^ ((row >> 1) & 3)) << 4);  // 64-byte swizzle
    const uint32_t dst = (q >> 1) * (kBK * 128) + row * 128;
    const int j0 = (q & 1) * 4;
    const uint32_t steps_per_tile = nk;
    uint32_t it = 0;
    bool ok = true;
    for (long long L = blockIdx.x; L < total && ok; L += gridDim.x) {
      for (uint32_t kb = 0; kb < steps_per_tile; ++kb, ++it) {
        const int rs = it % kRaw, s = it % kStages;
        bool w_ok = mbar_wait(&raw_full[rs], (it / kRaw) & 1u, p.status, abort_flag);
        if (w_ok && it >= kStages)
          w_ok = mbar_wait(&empty[s], ((it / kStages) & 1u) ^ 1u, p.status, abort_flag);
        if (!__all_sync(0xFFFFFFFFu, w_ok)) {
          ok = false;
          break;
        }
        const uint4 c = *reinterpret_cast<const uint4*>(smem + kOffRaw + rs * kRawCodes + src);
        const uint32_t sb = smem[kOffScale + rs * kRawScales + row * 4 + q];
        __syncwarp();
        if (lane == 0) mbar_arrive(&raw_empty[rs]);
        // 2^(sb - 127) * 2^126 as one bf16 factor up to sb = 128; what is above goes into a
        // second one (255: NaN)
        const uint32_t e1 = sb + 126 < 254 ? sb + 126 : 254;
        const __nv_bfloat162 mul = __bfloat162bfloat162(__ushort_as_bfloat16(e1 << 7));
        const uint32_t cw4[4] = {c.x, c.y, c.z, c.w};
        uint32_t o[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) codes_to_bf16(cw4[i], mul, o[i]);
        if (sb > 128) {
          const uint32_t e2 = sb == 255 ? 0x7FC0u : (sb - 128 + 127) << 7;
          const __nv_bfloat162 more = __bfloat162bfloat162(__ushort_as_bfloat16(e2));
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const __nv_bfloat162 r =
                  __hmul2(*reinterpret_cast<__nv_bfloat162*>(&o[i][j]), more);
              o[i][j] = *reinterpret_cast<const uint32_t*>(&r);
            }
        }
        uint8_t* a = smem + s * kStageBytes + dst;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<uint4*>(a + (((j0 + i) ^ (row & 7)) << 4)) =
              make_uint4(o[i][0], o[i][1], o[i][2], o[i][3]);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[s]);
      }
    }
  } else if (warp >= 4) {
    // ---------------------------------------------------------------- epilogue
    const int q = warp & 3;
    uint32_t tc = 0;
    for (long long L = blockIdx.x; L < total; L += gridDim.x, ++tc) {
      const GradTile t = tile_at(L, f_tiles, G, off, first);
      const uint32_t b = tc & 1u, use = tc >> 1;
      int w_ok = 1;
      if (lane == 0) w_ok = mbar_wait(&acc_full[b], use & 1u, p.status, abort_flag);
      if (!__shfl_sync(0xFFFFFFFFu, w_ok, 0)) break;
      tc_fence_after();
      const uint32_t acc = tmem + (static_cast<uint32_t>(q * 32) << 16) + b * kRowsMax;
      uint16_t* out = p.dx + static_cast<size_t>(t.row0) * p.F + t.f0 + q * 32 + feature_at(lane);
      for (int c = 0; c < t.rows; c += 16) {
        uint32_t v[16];
        tmem_ld_32x32b_x16(acc + c, v);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (c + i < t.rows)
            out[static_cast<size_t>(c + i) * p.F] =
                __bfloat16_as_ushort(__float2bfloat16_rn(__uint_as_float(v[i])));
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&acc_empty[b]);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

bool encode_w(CUtensorMap* m, const ExpertGradCall& a) {
  EncodeTiledFn enc = get_encode_tiled_fn();
  if (!enc) return false;
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(a.F) / 2, static_cast<cuuint64_t>(a.G) * a.C};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(a.F) / 2};
  cuuint32_t box[2] = {kFeat / 2, kBK}, es[2] = {1, 1};
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
  cuuint32_t box[2] = {kBK, static_cast<cuuint32_t>(box_rows)}, es[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<uint16_t*>(a.dy), dims, strides,
             box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
         CUDA_SUCCESS;
}

}  // namespace

cudaError_t launch_expert_grad(const ExpertGradCall& a, cudaStream_t st) {
  cudaError_t e = allow_smem<k_expert_grad>();
  if (e != cudaSuccess) return e;
  CUtensorMap tmW, tmB, tmBs;
  if (!encode_w(&tmW, a) || !encode_dy(&tmB, a, 128) || !encode_dy(&tmBs, a, 32))
    return cudaErrorInvalidValue;
  const GradParams p = {a.offsets, a.w_s, a.dx, a.G, a.rows, a.C, a.F, a.status};
  return launch_k(k_expert_grad, kSms, kThreads, kSmem, st, tmW, tmB, tmBs, p);
}

}  // namespace moe
