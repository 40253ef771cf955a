// y = x . W^T + bias with both operands in microscaled 4 bits, on the block-scaled
// tensor-core path (tcgen05.mma kind::mxf4 / kind::mxf4nvf4): the scales are applied
// inside the MMA, sums are fp32.
//
// A CTA computes 128 tokens x NT features; with many tokens a pair of CTAs (cta_group::2)
// computes 256 x 256, each loading half of the weights' rows, since the traffic from L2
// bounds a single CTA's tile.  A stage is 256 values of K: 128-byte packed
// rows of both operands by TMA (128-byte swizzle) and their scales as whole 512-byte
// tiles, which tcgen05.cp spreads over the four TMEM lane quadrants as the MMA wants
// them.  A lane of one warp issues the loads, a lane of another the scale copies and MMAs; eight
// warps write results.
//
// Rows of y that are not whole 16-byte units would be written value by value, a row a lane.
// There the operands change places: a lane then has a feature, and a warp writes 32 neighbours
// of one token (388 x 9839 x 1472: 12 us, 75 by rows).
//
// Work: one CTA per output tile, persistent over the SMs; where there are fewer tiles
// than SMs a cluster of CTAs shares a tile along K and adds the fp32 partial tiles through
// distributed shared memory, in rank order, so results do not depend on timing.
#include "mx4_device.cuh"

namespace aqlm {
namespace {

constexpr int kRows = 128;           // tokens of a tile (MMA M)
constexpr int kStageK = 256;         // values of K in a stage
constexpr int kRowBytes = kStageK / 2;
constexpr int kStepK = 64;           // values of K in one MMA
constexpr int kThreads = 320;        // load warp, MMA warp, 8 epilogue warps
constexpr int kMaxSmem = 227 * 1024;

constexpr int round_pow2(int v) { return v <= 32 ? 32 : v <= 64 ? 64 : v <= 128 ? 128 : v <= 256 ? 256 : 512; }

// Shapes that follow from the format and the tile width.
template <int FORMAT, int NT, int CG>
struct Plan {
  static constexpr int kTilesK = kStageK / (4 * mx4_block(FORMAT));  // scale tiles of a stage along K
  static constexpr int kTilesN = NT > 128 ? 2 : 1;                   // and along the features
  static constexpr int kA = kRows * kRowBytes, kB = NT / CG * kRowBytes;
  static constexpr int kSa = kTilesK * 512, kSb = kTilesN * kTilesK * 512;
  static constexpr int kStage = kA + kB + ((kSa + kSb + 1023) & ~1023);
  static constexpr int kFit = (kMaxSmem - 2048) / kStage;
  static constexpr int kStages = kFit > 8 ? 8 : kFit;
  // TMEM columns: accumulators (two where they fit beside two stages' scales), then scales
  static constexpr int kScaleCols = kTilesK * 4 * (1 + kTilesN);
  static constexpr int kAccs = 2 * NT + 2 * kScaleCols <= 512 ? 2 : 1;
  static constexpr int kFitScales = (512 - kAccs * NT) / kScaleCols;
  static constexpr int kScaleBufs = kFitScales > kStages ? kStages : kFitScales;
  static constexpr int kCols = round_pow2(kAccs * NT + kScaleBufs * kScaleCols);
  static constexpr int kRedPitch = NT + 4;  // floats of a partial row: 16-byte stores of 8 lanes hit all banks
  static_assert(CG == 1 || NT == 256, "a pair's halves are whole scale tiles");
  static constexpr size_t kSmem = static_cast<size_t>(kStages) * kStage + 2048;
  static_assert((NT / 2) % 32 == 0, "a warp's columns");
  static_assert(kStages >= 3 && kScaleBufs >= 2 && kCols <= 512, "");
  static_assert(kRows * kRedPitch * 4 <= kStages * kStage, "");
};

struct ProductParams {
  const uint8_t* xs;
  const uint8_t* ws;
  const float* gx;
  const float* gw;
  const void* bias;
  void* y;
  uint32_t* status;
  int batch, N, K, tiles;  // rows of the first and second operand; scale tiles along K
  int m_tiles, n_tiles, splits, y_type;
  bool swapped;            // the first operand is the weights: y is [N][batch]
};

// Shared-memory descriptor of a 512-byte scale tile: 32 rows of 16 bytes, 8-row groups 128
// bytes apart, no swizzle.
__device__ __forceinline__ uint64_t scales_desc(uint32_t smem) {
  return static_cast<uint64_t>((smem >> 4) & 0x3FFFu) | static_cast<uint64_t>(128u >> 4) << 32 |
         static_cast<uint64_t>(1u) << 46;
}
template <int CG>
__device__ __forceinline__ void tmem_copy_scales(uint32_t taddr, uint64_t desc) {
  if constexpr (CG == 1) asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
  else asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

// Instruction descriptor of the block-scaled MMA: e2m1 operands (code 1), both K-major.
//   bits 4-5 / 29-30 byte of the scale word that B's / A's scales start at
//   bits 7-9 / 10-12 operand types, 17-22 N >> 3, 23 scale type (1: e8m0), 24-28 M >> 4
template <int FORMAT, int CG>
__host__ __device__ constexpr uint32_t mx4_idesc(uint32_t n, uint32_t sf) {
  return sf << 4 | 1u << 7 | 1u << 10 | (n >> 3) << 17 | (FORMAT == kMxfp4 ? 1u : 0u) << 23 | (kRows * CG >> 4) << 24 |
         sf << 29;
}

template <int FORMAT, int CG>
__device__ __forceinline__ void umma_mx4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa, uint32_t sb,
                                         uint32_t accumulate) {
#define MX4_MMA(group, kind)                                                                       \
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"                                  \
               "tcgen05.mma.cta_group::" group "." kind " [%0], %1, %2, %3, [%4], [%5], p;\n\t}"    \
               ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate) : "memory")
  if constexpr (FORMAT == kMxfp4 && CG == 1) MX4_MMA("1", "kind::mxf4.block_scale.scale_vec::2X");
  else if constexpr (FORMAT == kMxfp4) MX4_MMA("2", "kind::mxf4.block_scale.scale_vec::2X");
  else if constexpr (CG == 1) MX4_MMA("1", "kind::mxf4nvf4.block_scale.scale_vec::4X");
  else MX4_MMA("2", "kind::mxf4nvf4.block_scale.scale_vec::4X");
#undef MX4_MMA
}

// Both tensor scales as factors of a sum, v * first * second: 1 and their product, unless that
// leaves fp32's normal range.  Then one after the other: the larger first where it is too small, so
// that only a result that is too small itself loses bits on the way, the smaller first where it is
// too large.  Results are written by straight code that runs once or twice, whose fetching counts:
// the first factor has a branch of its own (multiplying every value by both took 0.1 us more of 9.5,
// 64 x 14336 x 4096).
struct TensorScales {
  float first = 1.0f, second;
  __device__ __forceinline__ explicit TensorScales(const ProductParams& p) {
    const float x = p.gx ? *p.gx : 1.0f, w = p.gw ? *p.gw : 1.0f;
    second = w * x;
    const float a = fabsf(second);
    if ((a < 1.17549435e-38f || a > 3.402823466e38f) && x != 0.0f && w != 0.0f) {
      const bool x_first = (fabsf(x) > fabsf(w)) == (a < 1.0f);
      first = x_first ? x : w;
      second = x_first ? w : x;
    }
  }
  template <int N>
  __device__ __forceinline__ void apply_first(float (&v)[N]) const {
    if (first != 1.0f)
#pragma unroll
      for (float& f : v) f *= first;
  }
};

// bias[c .. c + 8) as fp32; `c` in whole 16-byte units
__device__ __forceinline__ void bias8(const void* bias, int type, size_t c, float (&b)[8]) {
  if (type == kF32) {
    const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(bias) + c);
    const float4 u = q[0], v = q[1];
    b[0] = u.x, b[1] = u.y, b[2] = u.z, b[3] = u.w, b[4] = v.x, b[5] = v.y, b[6] = v.z, b[7] = v.w;
  } else {
    const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(bias) + c);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = type == kF16 ? h2_to_f2(w[i]) : b2_to_f2(w[i]);
      b[2 * i] = f.x, b[2 * i + 1] = f.y;
    }
  }
}

// One value of a swapped product: y[c][row].
__device__ __forceinline__ void put_swapped(const ProductParams& p, int row, int c, float v, float scale, float bias) {
  const size_t at = static_cast<size_t>(c) * p.batch + row;
  const float r = fmaf(v, scale, bias);
  if (p.y_type == kF32) store_value<kF32>(p.y, at, r);
  else if (p.y_type == kF16) store_value<kF16>(p.y, at, r);
  else store_value<kBf16>(p.y, at, r);
}
__device__ __forceinline__ float bias_of(const ProductParams& p, int i) {
  return !p.bias ? 0.0f
         : p.y_type == kF32 ? load_value<kF32>(p.bias, i)
         : p.y_type == kF16 ? load_value<kF16>(p.bias, i)
                            : load_value<kBf16>(p.bias, i);
}

// v[0..8) * scale + bias to y[row][c ..).  Rows of y are whole 16-byte units (else the operands have
// changed places): eight values, or the last four of an fp32 row.
__device__ __forceinline__ void put8(const ProductParams& p, int row, int c, const float* v, float scale) {
  const size_t at = static_cast<size_t>(row) * p.N + c;
  if (c + 8 > p.N) {
    float4 b = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (p.bias) b = *reinterpret_cast<const float4*>(static_cast<const float*>(p.bias) + c);
    *reinterpret_cast<float4*>(static_cast<float*>(p.y) + at) =
        make_float4(fmaf(v[0], scale, b.x), fmaf(v[1], scale, b.y), fmaf(v[2], scale, b.z), fmaf(v[3], scale, b.w));
    return;
  }
  float b[8] = {}, o[8];
  if (p.bias) bias8(p.bias, p.y_type, c, b);
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] = fmaf(v[i], scale, b[i]);
  if (p.y_type == kF32) {
    float4* q = reinterpret_cast<float4*>(static_cast<float*>(p.y) + at);
    q[0] = make_float4(o[0], o[1], o[2], o[3]);
    q[1] = make_float4(o[4], o[5], o[6], o[7]);
  } else {
    uint4 q;
    if (p.y_type == kF16)
      q = make_uint4(f2_to_h2_rn(o[0], o[1]), f2_to_h2_rn(o[2], o[3]), f2_to_h2_rn(o[4], o[5]), f2_to_h2_rn(o[6], o[7]));
    else
      q = make_uint4(f2_to_b2_rn(o[0], o[1]), f2_to_b2_rn(o[2], o[3]), f2_to_b2_rn(o[4], o[5]), f2_to_b2_rn(o[6], o[7]));
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.y) + at) = q;
  }
}

template <int FORMAT, int NT, int CG>
__global__ void __launch_bounds__(kThreads, 1) product_kernel(const __grid_constant__ CUtensorMap x_map,
                                                              const __grid_constant__ CUtensorMap w_map,
                                                              const ProductParams p) {
  using P = Plan<FORMAT, NT, CG>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* stages = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ uint64_t full[P::kStages], empty[P::kStages], acc_full[P::kAccs], acc_empty[P::kAccs];
  __shared__ uint32_t tmem_slot;
  __shared__ volatile uint32_t failed;

  const int warp = uniform_warp(), lane = threadIdx.x & 31;
  const int rank = CG > 1 || p.splits > 1 ? static_cast<int>(cluster_rank()) : 0;
  if (threadIdx.x == 0) {
    failed = 0;
    for (int i = 0; i < P::kStages; ++i) {
      mbar_init(&full[i], CG > 1 && rank == 0 ? 2 : 1);  // a pair's first CTA also waits for its second
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < P::kAccs; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], 8 * CG);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 0 && lane == 0) prefetch_map(&x_map), prefetch_map(&w_map);
  if (warp == 1) tmem_alloc_cg<CG>(&tmem_slot, P::kCols);
  tc_fence_before_sync();
  __syncthreads();
  if (CG > 1) cluster_sync();  // the pair's barriers are ready before either arrives on them
  tc_fence_after_sync();
  const uint32_t tmem = tmem_slot;
  const uint32_t scale_tmem = tmem + P::kAccs * NT;

  const int k_stages = (p.K + kStageK - 1) / kStageK;
  const int k_rank = CG > 1 ? 0 : rank, pair_rank = CG > 1 ? rank : 0;
  const int s0 = k_stages * k_rank / p.splits, s1 = k_stages * (k_rank + 1) / p.splits;
  const int total = p.m_tiles * p.n_tiles;
  const int per = CG > 1 ? CG : p.splits;
  const int first = blockIdx.x / per, step = gridDim.x / per;

  grid_dependency_wait();
  grid_dependents_launch();

  // a wait that gives up makes every later one of this CTA that is not over end soon
  const auto wait = [&](uint64_t* bar, uint32_t parity, uint32_t site) {
    if (mbar_wait_sleeping<false>(bar, parity, p.status, site, &failed)) return true;
    failed = 1;
    return false;
  };
  const auto wait_pair = [&](uint64_t* bar, uint32_t parity, uint32_t site) {
    if (mbar_wait_sleeping<(CG > 1)>(bar, parity, p.status, site, &failed)) return true;
    failed = 1;
    return false;
  };

  if (warp == 0) {
    // ---- loads: the whole warp walks the stages, one lane issues
    const bool issuer = elect_one();
    const uint64_t keep = l2_policy_evict_last(), pass = l2_policy_evict_first();
    const int w_row_tiles = (p.N + 127) / 128, x_row_tiles = (p.batch + 127) / 128;
    Ring<P::kStages> r;
    bool ok = true;
    for (int t = first; t < total && ok; t += step) {
      const int m = (t % p.m_tiles) * CG + pair_rank, n0 = (t / p.m_tiles) * NT;
      for (int s = s0; s < s1; ++s, r.next()) {
        ok = __all_sync(0xFFFFFFFFu, wait(&empty[r.slot], r.phase ^ 1, kSitePipeEmpty));
        if (!ok) break;
        uint64_t* bar = &full[r.slot];
        const uint32_t base = smem_addr(stages + r.slot * P::kStage);
        const int c0 = s * P::kTilesK;
        const uint32_t run = static_cast<uint32_t>(min(P::kTilesK, p.tiles - c0)) * 512;
        const int wt = n0 / 128;
        const int w_tiles = min(P::kTilesN, w_row_tiles - wt);
        const int x_tiles = m < x_row_tiles;  // a pair's second CTA may have no tokens: it reads zeros
        if (issuer) {
          mbar_arrive_expect_tx(bar, P::kA + P::kB + run * (x_tiles + w_tiles));
          tma_load_2d(base, &x_map, s * kRowBytes, m * kRows, bar, keep);
          tma_load_2d(base + P::kA, &w_map, s * kRowBytes, n0 + pair_rank * (NT / CG), bar, p.m_tiles > 1 ? keep : pass);
          const uint32_t sa = base + P::kA + P::kB, sb = sa + P::kSa;
          if (x_tiles) bulk_load(sa, p.xs + (static_cast<size_t>(m) * p.tiles + c0) * 512, run, bar);
          for (int j = 0; j < w_tiles; ++j)
            bulk_load(sb + j * P::kSa, p.ws + (static_cast<size_t>(wt + j) * p.tiles + c0) * 512, run, bar);
        }
      }
    }
  } else if (warp == 1 && CG > 1 && rank > 0) {
    // ---- the pair's second CTA tells the first when its part of a stage is there
    Ring<P::kStages> r;
    bool ok = true;
    for (int t = first; t < total && ok; t += step)
      for (int s = s0; s < s1 && ok; ++s, r.next()) {
        ok = __all_sync(0xFFFFFFFFu, wait(&full[r.slot], r.phase, kSitePipeFull));
        if (ok && lane == 0) mbar_arrive_leader(&full[r.slot]);
      }
  } else if (warp == 1) {
    // ---- scale copies and MMAs: the whole warp walks the stages, so that descriptors stay
    // in uniform registers; one lane issues.  The lanes wait by themselves, since no whole-warp
    // instruction follows within a tile, and agree at its end
    const bool issuer = elect_one();
    const uint64_t a_desc = umma_desc_sw128_kmajor(smem_addr(stages)), s_desc = scales_desc(smem_addr(stages) + P::kA + P::kB);
    Ring<P::kStages> r;
    Ring<P::kScaleBufs> sc;
    uint32_t acc_it = 0, it = 0;
    bool ok = true;
    for (int t = first; t < total && ok; t += step, ++acc_it) {
      const int n0 = (t / p.m_tiles) * NT;
      const uint32_t shift = (n0 & 127) / 32;  // the tile's first scale column
      const uint32_t acc = acc_it % P::kAccs;
      ok = wait_pair(&acc_empty[acc], ((acc_it / P::kAccs) & 1) ^ 1, kSitePipeAcc);
      tc_fence_after_sync();
      const uint32_t d = tmem + acc * NT;
      uint32_t go = 0;
      for (int s = s0; s < s1 && ok; ++s, r.next(), sc.next(), ++it) {
        ok = wait_pair(&full[r.slot], r.phase, kSitePipeFull);
        // the scale columns' last readers: the MMAs kScaleBufs stages ago
        if (P::kScaleBufs < P::kStages && ok && it >= P::kScaleBufs) {
          const uint32_t old = it - P::kScaleBufs;
          ok = wait(&empty[old % P::kStages], (old / P::kStages) & 1, kSitePipeEmpty);
        }
        if (!ok) break;
        tc_fence_after_sync();
        const uint64_t da = a_desc + r.slot * (P::kStage >> 4), db = da + (P::kA >> 4);
        const uint64_t sa = s_desc + r.slot * (P::kStage >> 4), sb = sa + (P::kSa >> 4);
        const uint32_t ta = scale_tmem + sc.slot * P::kScaleCols, tb = ta + P::kTilesK * 4;
        const int steps = (p.K - s * kStageK + kStepK - 1) / kStepK;
        if (issuer) {
#pragma unroll
          for (int c = 0; c < P::kTilesK; ++c) {
            tmem_copy_scales<CG>(ta + c * 4, sa + c * (512 >> 4));
#pragma unroll
            for (int j = 0; j < P::kTilesN; ++j)
              tmem_copy_scales<CG>(tb + (c * P::kTilesN + j) * 4, sb + (j * P::kSa + c * 512) / 16);
          }
#pragma unroll
          for (int k = 0; k < kStageK / kStepK; ++k) {
            // 64 values: two MXFP4 scales of a word, or all four NVFP4 scales of one
            const int c = FORMAT == kMxfp4 ? k / 2 : k;
            const uint32_t sf = FORMAT == kMxfp4 ? (k & 1) * 2 : 0;
            if (k < steps)
              umma_mx4<FORMAT, CG>(d, da + k * 2, db + k * 2, mx4_idesc<FORMAT, CG>(NT, sf), ta + c * 4,
                               tb + c * P::kTilesN * 4 + shift, k > 0 ? 1 : go);
          }
          umma_commit_cg<CG>(&empty[r.slot]);
        }
        go = 1;
      }
      ok = __all_sync(0xFFFFFFFFu, ok);
      if (ok && issuer) umma_commit_cg<CG>(&acc_full[acc]);
    }
  } else if (warp >= 2) {
    // ---- results
    const int quad = warp & 3, half = (warp - 2) >> 2;  // TMEM lanes, half of the columns
    const TensorScales scales(p);
    uint32_t acc_it = 0;
    bool ok = true;
    for (int t = first; t < total && ok; t += step, ++acc_it) {
      const int m0 = ((t % p.m_tiles) * CG + pair_rank) * kRows, n0 = (t / p.m_tiles) * NT;
      const uint32_t acc = acc_it % P::kAccs;
      ok = __all_sync(0xFFFFFFFFu, wait(&acc_full[acc], (acc_it / P::kAccs) & 1, kSitePipeAcc));
      if (!ok) break;
      tc_fence_after_sync();
      const int row = m0 + quad * 32 + lane;
      const uint32_t lane_base = tmem + acc * NT + (static_cast<uint32_t>(quad * 32) << 16);
      // the warp's columns into registers at once, so that the next tile's MMAs can begin
      constexpr int kMine = NT / 2, kParts = (kMine + 31) / 32;
      uint32_t v[kParts][32];
#pragma unroll
      for (int i = 0; i < kParts; ++i) tmem_ld_x32_start(lane_base + half * kMine + i * 32, v[i]);
      tmem_ld_wait(v);
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) {
        if constexpr (CG == 1) mbar_arrive(&acc_empty[acc]);
        else mbar_arrive_leader(&acc_empty[acc]);
      }
#pragma unroll
      for (int i = 0; i < kParts; ++i) {
        const int c = half * kMine + i * 32;
        float(&f)[32] = reinterpret_cast<float(&)[32]>(v[i]);
        if (p.splits == 1) scales.apply_first(f);
        if (p.splits > 1) {
          float4* q = reinterpret_cast<float4*>(reinterpret_cast<float*>(stages) + (quad * 32 + lane) * P::kRedPitch + c);
#pragma unroll
          for (int e = 0; e < 8; ++e) q[e] = make_float4(f[4 * e], f[4 * e + 1], f[4 * e + 2], f[4 * e + 3]);
        } else if (p.swapped) {
          if (row < p.batch) {
            const float bias = bias_of(p, row);
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (n0 + c + e < p.N) put_swapped(p, row, n0 + c + e, f[e], scales.second, bias);
          }
        } else if (row < p.batch) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (n0 + c + 8 * e < p.N) put8(p, row, n0 + c + 8 * e, f + 8 * e, scales.second);
        }
      }
    }
  }

  __syncwarp();
  settle_after_failure(failed);
  if (p.splits > 1) {
    // the partial tiles of the cluster, added in rank order: eight columns of a row a thread
    __syncwarp();
    cluster_sync();
    const int m0 = (first % p.m_tiles) * kRows, n0 = (first / p.m_tiles) * NT;
    const int rows = min(kRows, p.batch - m0), cols = min(NT, p.N - n0);
    const TensorScales scales(p);
    const uint32_t red = smem_addr(stages);
    for (int e = rank * kThreads + threadIdx.x; e < rows * (NT / 8); e += kThreads * p.splits) {
      const int r = p.swapped ? e % rows : e / (NT / 8), c = (p.swapped ? e / rows : e % (NT / 8)) * 8;
      if (c >= cols) continue;
      float v[8] = {};
      for (int s = 0; s < p.splits; ++s) {
        const uint32_t at = red + (r * P::kRedPitch + c) * 4;
        const float4 a = ld_cluster_f4(at, s), b = ld_cluster_f4(at + 16, s);
        v[0] += a.x, v[1] += a.y, v[2] += a.z, v[3] += a.w;
        v[4] += b.x, v[5] += b.y, v[6] += b.z, v[7] += b.w;
      }
      scales.apply_first(v);
      if (p.swapped) {
        const float bias = bias_of(p, m0 + r);
        for (int i = 0; i < 8; ++i)
          if (c + i < cols) put_swapped(p, m0 + r, n0 + c + i, v[i], scales.second, bias);
      } else {
        put8(p, m0 + r, n0 + c, v, scales.second);
      }
    }
    cluster_sync();  // no CTA leaves while another reads its partial tile
  }
  tc_fence_before_sync();
  __syncwarp();
  __syncthreads();
  if (CG > 1) cluster_sync();
  tc_fence_after_sync();
  if (warp == 1) tmem_dealloc_cg<CG>(tmem, P::kCols);
}

// Packed rows as a 2-D map of bytes: boxes of 128 bytes x `box` rows, 128-byte swizzle.
cudaError_t packed_map(CUtensorMap* map, const Mx4& t, int K, int box) {
  EncodeTiledFn encode = encode_tiled();
  if (!encode) return cudaErrorNotSupported;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(K / 2), static_cast<cuuint64_t>(t.rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(K / 2)};
  const cuuint32_t boxes[2] = {kRowBytes, static_cast<cuuint32_t>(box)};
  const cuuint32_t ones[2] = {1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(t.packed), dims, strides, boxes, ones,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? cudaSuccess
             : cudaErrorInvalidValue;
}

constexpr int kSms = 148;

// a: the operand of 128-row tiles, b: that of NT; the activations and the weights, or swapped.
template <int FORMAT, int NT, int CG = 1>
cudaError_t product_as(const Mx4Product& p, const Mx4& a, const Mx4& b, bool swapped, int splits, uint32_t* status,
                       cudaStream_t stream) {
  using P = Plan<FORMAT, NT, CG>;
  CUtensorMap a_map, b_map;
  cudaError_t e = packed_map(&a_map, a, p.K, kRows);
  if (e == cudaSuccess) e = packed_map(&b_map, b, p.K, NT / CG);
  if (e != cudaSuccess) return e;
  ProductParams q{};
  q.xs = a.scales;
  q.ws = b.scales;
  q.gx = p.x.tensor_scale;
  q.gw = p.w.tensor_scale;
  q.bias = p.bias;
  q.y = p.y;
  q.status = status;
  q.batch = a.rows;
  q.N = b.rows;
  q.K = p.K;
  q.tiles = mx4_scale_tiles(p.K, FORMAT);
  q.m_tiles = (q.batch + kRows * CG - 1) / (kRows * CG);
  q.n_tiles = (q.N + NT - 1) / NT;
  q.splits = splits;
  q.y_type = p.y_type;
  q.swapped = swapped;
  auto* kernel = product_kernel<FORMAT, NT, CG>;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(P::kSmem));
  if (e != cudaSuccess) return e;
  const long long tiles = static_cast<long long>(q.m_tiles) * q.n_tiles;
  if (tiles > 0x7FFFFFFF / 8) return cudaErrorInvalidValue;
  const long long ctas = tiles * CG * splits;
  const unsigned grid = static_cast<unsigned>(splits > 1 || ctas < kSms ? ctas : kSms);
  return launch_overlapped(kernel, grid, kThreads, P::kSmem, stream, CG * splits, a_map, b_map, q);
}

// Tile width and K split.  A tile's time is its MMAs (2 cycles per column and 64 values of K at
// a rate of 128 x 256 x 64 in 128 cycles) or its loads, plus filling and draining.  Forcing each
// width and split on 1 to 1000 tokens of 4096 to 14336 features found nothing more than 15 %
// faster than what this picks (64 x 14336 x 4096: 128 wide 9.4 us, 64 wide 13.5, 256 wide 12.5;
// 64 x 4096 x 14336: 128 wide, K in four, 11.5, unsplit 20.7); the kernel now takes 8.8 for the
// first.  Reading the weights from HBM, which bounds fewer tokens, is not in the costs.
//
// Pairs are outside the costs too: they are taken wherever they make at least 37 tiles (4096 x
// 28672 x 8192: 400 us, single tiles 508; 354 now).  Where their tiles fill the 74 places badly
// (5120 features: 40 tiles at 512 tokens, 14.7 us; 80 at 1024, 22.7) single ones have not been
// compared.
template <int FORMAT>
cudaError_t product_planned(const Mx4Product& p, uint32_t* status, cudaStream_t stream) {
  const bool swapped = p.w.rows % (p.y_type == kF32 ? 4 : 8) != 0;
  const Mx4 &a = swapped ? p.w : p.x, &b = swapped ? p.x : p.w;
  const long long m_tiles = (a.rows + kRows - 1) / kRows;
  const int k_stages = (p.K + kStageK - 1) / kStageK;
  int best_nt = 256, best_split = 1;
  double best = 1e300;
  for (int nt : {64, 128, 192, 256}) {
    const long long tiles = m_tiles * ((b.rows + nt - 1) / nt);
    for (int split : {1, 2, 4, 8}) {
      if (split > 1 && (tiles * split > kSms || k_stages < 2 * split || nt > 128)) continue;
      const double waves = static_cast<double>((tiles * split + kSms - 1) / kSms);
      const double stages = static_cast<double>((k_stages + split - 1) / split);
      const double stage = 4 * (nt < 128 ? 64.0 : nt / 2.0);
      const double drain = nt * 6.0, fill = 2500 + (split > 1 ? 1500 : 0);
      const double cost = waves * (stages * stage + (nt == 256 ? drain : 0)) + drain + fill;
      if (cost < best) best = cost, best_nt = nt, best_split = split;
    }
  }
  const long long pairs = (m_tiles + 1) / 2 * ((b.rows + 255) / 256);
  if (m_tiles > 1 && pairs >= kSms / 4) return product_as<FORMAT, 256, 2>(p, a, b, swapped, 1, status, stream);
  switch (best_nt) {
    case 64: return product_as<FORMAT, 64>(p, a, b, swapped, best_split, status, stream);
    case 128: return product_as<FORMAT, 128>(p, a, b, swapped, best_split, status, stream);
    case 192: return product_as<FORMAT, 192>(p, a, b, swapped, best_split, status, stream);
    default: return product_as<FORMAT, 256>(p, a, b, swapped, best_split, status, stream);
  }
}

}  // namespace

cudaError_t launch_mx4_product(const Mx4Product& p, uint32_t* status, cudaStream_t stream) {
  return p.format == kMxfp4 ? product_planned<kMxfp4>(p, status, stream) : product_planned<kNvfp4>(p, status, stream);
}

}  // namespace aqlm
