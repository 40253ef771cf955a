// y = x . W^T + bias with 16-bit x and microscaled 4-bit W, for up to eight tokens.  The weights
// are decoded in registers and multiplied by mma.sync (16 rows x 8 tokens x 16 values), which
// keeps the arithmetic per weight well below fp32 FMAs.
//
// Persistent CTAs, one an SM, walk units of 32 weight rows.  A stage is 1024 values of them:
// four 128-byte-swizzled TMA boxes and the scale tiles, in a ring that runs across units, so
// that the reads never pause (loads by the lanes that use the values were slower, from
// registers or by cp.async: 1 x 28672 x 8192 52 and 62 us).  Two sets of eight warps take stages
// in turn, a warp 128 values of the 32 rows; lane (g, t) has 32 of them in four rows.  Which of
// the 128 values an MMA takes is free as long as x is taken alike.  The partial sums of a unit
// are fp32, added in a fixed order by a warp of their own; with few units a cluster of CTAs
// splits the reduction.
//
// Decoding is a table lookup: a byte of two codes gives their pair.  The table has a copy
// for every lane, each in its own bank, 256 bytes a row, so that one byte permute makes
// the address and no lookup conflicts.  Eight weights cost a lane four of each.  The decoded
// weight is exact: e2m1 times 2^e or e4m3 fits bf16, e2m1 times e4m3 fits fp16.  fp16 x with
// MXFP4 weights is split into two bf16 parts.
//
// One token leaves seven of an MMA's eight columns free.  They take the blocks apart: column
// 2 t + h holds x where lane t has half h of its 32 values and zeros elsewhere, so that the
// sums come out per 16 values, and the scales multiply four fp32 sums a step instead of
// every pair of weights.  16 products of unscaled weights with bf16 x could pass the end of fp32
// where the scale would bring them back: there the table holds the weights times 2^-7 (16 times 6
// is below 2^7), which fp32 sums do not lose, and the sum of all is multiplied by 2^7.
//
// Measured (NVFP4 bf16): 1 token 4096 x 4096 5.2 us, 11008 x 4096 10.4, 28672 x 8192 33.6 (3.9
// TB/s); 8 tokens 52 us on the last.  While a CTA's warps are active the shared-memory and L1 pipe
// is at 78 % (64 of a warp step's 88 wavefronts are lookups) and 58 % of the issue slots are taken.
// When the kernel took 36.5 us for one token there, its loads alone took 25 and its arithmetic
// alone 34.6; decoding a quarter or half of the words by logic instead was slower (37 and 43 us),
// as were three sets of warps (37.7).
#include "mx4_device.cuh"

namespace aqlm {
namespace {

constexpr int kSet = 8, kWarps = 2 * kSet, kThreads = (kWarps + 2) * 32;  // and a warp that loads, one that adds
constexpr int kRows = 32, kStage = 1024, kBox = 256, kStep = 128;
constexpr int kStageBytes = kRows * kStage / 2;
constexpr int kTableBytes = 65536;
constexpr int kSms = 148;

template <int FORMAT, bool ONE>
struct Shape {
  static constexpr int kTiles = kStage / (4 * mx4_block(FORMAT));  // scale tiles of a stage
  static constexpr int kSlot = kStageBytes + kTiles * 512;
  static constexpr int kTokens = ONE ? 1 : 8;
  static constexpr int kPitch = 36;  // floats of a token's 32 sums: a warp's writes hit all banks
  static constexpr int kSums = kTokens * kPitch;
  static constexpr int kSets = 2;
  static constexpr int kPart = kSets * kWarps * kSums * 4;
  static constexpr int kFit = (227 * 1024 - 1024 - kTableBytes - kPart - 256) / kSlot;
  // An even number, so that a slot's stages are all of one set of warps: a set that skipped a phase of
  // a slot's barrier could take the phase before it for the one it waits for.
  static constexpr int kSlots = kFit / 2 * 2;
  static constexpr size_t kSmem = 1024 + kTableBytes + kPart + kSlots * kSlot;
  static_assert(kSlots >= 4 && kSlots <= 8, "");
};

struct GemvParams {
  const uint8_t* scales;
  const float* gamma;
  const void* x;
  const void* bias;
  void* y;
  uint32_t* status;
  int N, K, batch, tiles, units;
  int splits;  // CTAs of a cluster that share a unit
};

template <int TYPE>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  if constexpr (TYPE == kF16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Eight codes as four pairs, in order, times `scale` (SCALED); `lane4`: 4 * lane.
template <int TYPE, bool SCALED>
__device__ __forceinline__ void decode_pairs(const uint8_t* table, uint32_t lane4, uint32_t w, uint32_t scale,
                                             uint32_t (&h)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    h[j] = *reinterpret_cast<const uint32_t*>(table + prmt(w, lane4, 0x5504 | j << 4));
    if constexpr (SCALED) {
      if constexpr (TYPE == kF16) asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(h[j]) : "r"(h[j]), "r"(scale));
      else asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(h[j]) : "r"(h[j]), "r"(scale));
    }
  }
}

// Two bf16 parts of a pair of fp16 values, hi + lo exactly: hi keeps 8 significant bits.  A NaN's
// bits are made those of one that keeps some of them in hi; a second part of an infinity or a
// NaN is some finite value.
__device__ __forceinline__ void split_pair(uint32_t x, uint32_t& hi, uint32_t& lo) {
  // the maximum with minus infinity: x, or 0x7FFF for a NaN
  asm("max.NaN.f16x2 %0, %0, %1;" : "+r"(x) : "r"(0xFC00FC00u));
  const uint32_t top = x & 0xFFF8FFF8u;
  const __half2 rest = __hmin2(__hsub2(*reinterpret_cast<const __half2*>(&x), *reinterpret_cast<const __half2*>(&top)),
                               __half2half2(__ushort_as_half(0x7BFF)));
  const float2 h = h2_to_f2(top), l = __half22float2(rest);
  hi = f2_to_b2_rn(h.x, h.y);
  lo = f2_to_b2_rn(l.x, l.y);
}

// The one-token kernel's factor of the table (above).
template <int XT>
constexpr float kOneUp = XT == kBf16 ? 128.0f : 1.0f;

// ONE: one token; else up to eight.
template <int FORMAT, int XT, bool ONE>
__global__ void __launch_bounds__(kThreads, 1) gemv_kernel(const __grid_constant__ CUtensorMap w_map, const GemvParams p) {
  using S = Shape<FORMAT, ONE>;
  constexpr bool kSplit = !ONE && FORMAT == kMxfp4 && XT == kF16;
  constexpr int TYPE = kSplit ? kBf16 : XT;
  extern __shared__ __align__(16) uint8_t table[];  // first, so that its address is a constant of the lookups
  float* part = reinterpret_cast<float*>(table + kTableBytes);  // [sets][warps][tokens][32 rows, padded]
  const uint32_t ring = (smem_addr(table) + kTableBytes + S::kPart + 1023) & ~1023u;
  __shared__ uint64_t full[S::kSlots], empty[S::kSlots], sums_full[S::kSets], sums_empty[S::kSets];
  __shared__ volatile uint32_t failed;

  const int warp = uniform_warp(), lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int rank = p.splits > 1 ? static_cast<int>(cluster_rank()) : 0;
  if (threadIdx.x == 0) {
    failed = 0;
    for (int i = 0; i < S::kSlots; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], kSet);
    }
    for (int i = 0; i < S::kSets; ++i) {
      mbar_init(&sums_full[i], kWarps);
      mbar_init(&sums_empty[i], 1);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kWarps && lane == 0) prefetch_map(&w_map);
  const uint32_t lane4 = lane * 4;
  if (warp < kWarps) {  // the table: each warp's 16 bytes, decoded by a lane each
    uint32_t h[4];
    e2m1x8_decode<TYPE>(warp * 16 + (lane & 15), h);
    if constexpr (ONE && XT == kBf16) asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(h[0]) : "r"(0x3C003C00u));  // 2^-7
#pragma unroll
    for (int b = 0; b < 16; ++b)
      *reinterpret_cast<uint32_t*>(table + (warp * 16 + b) * 256 + lane4) = __shfl_sync(0xFFFFFFFFu, h[0], b);
  }
  __syncthreads();

  const int stages = (p.K + kStage - 1) / kStage, chunks = p.K / 32;
  const int s0 = stages * rank / p.splits, s1 = stages * (rank + 1) / p.splits;
  const int first = blockIdx.x / p.splits, step = gridDim.x / p.splits;

  grid_dependency_wait();
  grid_dependents_launch();

  const auto wait = [&](uint64_t* bar, uint32_t parity, uint32_t site) {
    if (mbar_wait_sleeping<false>(bar, parity, p.status, site, &failed)) return true;
    failed = 1;
    return false;
  };

  if (warp == kWarps) {
    // ---- copies
    const uint64_t pol = l2_policy_evict_first();
    const bool issuer = elect_one();
    Ring<S::kSlots> r;
    bool ok = true;
    for (int u = first; u < p.units && ok; u += step)
      for (int s = s0; s < s1; ++s, r.next()) {
        ok = __all_sync(0xFFFFFFFFu, wait(&empty[r.slot], r.phase ^ 1, kSitePipeEmpty));
        if (!ok) break;
        const uint32_t at = ring + r.slot * S::kSlot;
        const int boxes = min(kStage / kBox, (p.K - s * kStage + kBox - 1) / kBox);
        const uint32_t run = static_cast<uint32_t>(min(S::kTiles, p.tiles - s * S::kTiles)) * 512;
        if (issuer) {
          mbar_arrive_expect_tx(&full[r.slot], boxes * (kRows * kBox / 2) + run);
#pragma unroll
          for (int b = 0; b < kStage / kBox; ++b)
            if (b < boxes)
              tma_load_2d(at + b * (kRows * kBox / 2), &w_map, s * (kStage / 2) + b * (kBox / 2), u * kRows, &full[r.slot], pol);
          bulk_load(at + kStageBytes, p.scales + (static_cast<size_t>(u >> 2) * p.tiles + s * S::kTiles) * 512, run,
                    &full[r.slot]);
        }
      }
  } else if (warp == kWarps + 1) {
    // ---- the sums of the warps, in their order, while those go on with the next unit: a lane
    // a row
    const float gamma = p.gamma ? *p.gamma : 1.0f, up = ONE ? kOneUp<XT> : 1.0f;
    Ring<S::kSets> r;
    for (int u = first; u < p.units; u += step, r.next()) {
      if (!__all_sync(0xFFFFFFFFu, wait(&sums_full[r.slot], r.phase, kSitePipeAcc))) break;
      const int row = u * kRows + lane;
      const float bias = p.bias && row < p.N ? load_value<XT>(p.bias, row) : 0.0f;
      float* sums = part + r.slot * kWarps * S::kSums + lane;
      for (int token = 0; token < p.batch; ++token) {
        float sum = 0.0f;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) sum += sums[k * S::kSums + token * S::kPitch];
        if (p.splits > 1) sums[token * S::kPitch] = sum;  // of this CTA's part of the reduction
        else if (row < p.N) store_value<XT>(p.y, static_cast<size_t>(token) * p.N + row, fmaf(sum * up, gamma, bias));
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sums_empty[r.slot]);
    }
  } else {
    // ---- products: the 32 rows, values 128 kw .. of a stage.  An MMA's row g is row
    // g / 2 + 4 (g % 2) of its eight: the eight lanes of a 16-byte read then have two rows
    // whose swizzled chunks lie in different banks.
    const int set = warp / kSet, kw = warp % kSet, rr = (g >> 1) | ((g & 1) << 2);
    const uint32_t from = (kw >> 1) * (kRows * kBox / 2) + rr * 128 + (((((kw & 1) << 2) | t) ^ rr) << 4);
    // MXFP4: 128 values are one scale tile, the lane's block byte t; NVFP4: two tiles, the
    // lane's two blocks a half word of tile t / 2
    const uint32_t from_s = kStageBytes + (FORMAT == kMxfp4 ? kw : 2 * kw + (t >> 1)) * 512 + rr * 16;
    // what a lane holds of x in a step: its 32 values of a token, or half of them or none
    uint4 x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = make_uint4(0, 0, 0, 0);
    // the lane's values in stage 0; a token past the last has zeros
    const bool x_real = ONE ? g >> 1 == t : g < p.batch;
    const uint4* x_from = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.x) +
                                                         static_cast<size_t>(!ONE && x_real ? g : 0) * p.K + (kw * 4 + t) * 32);
    const auto load_x = [&](int s) {
      if (!x_real) return;
      const bool in = s * (kStage / 32) + kw * 4 + t < chunks;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (!ONE || i >> 1 == (g & 1)) x[i] = in ? ldg_nc_v4(x_from + s * (kStage / 8) + i) : make_uint4(0, 0, 0, 0);
    };
    // eight rows' scale words as the lane's two factors
    const auto scales_of = [&](uint32_t word, bool in, float& f0, float& f1) {
      if constexpr (FORMAT == kMxfp4) {
        f0 = f1 = mx4_scale_value<kMxfp4>(word >> (8 * t) & 0xFF);
      } else {
        uint32_t f;
        asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(f) : "r"(in ? word >> (16 * (t & 1)) : 0));
        const float2 v = h2_to_f2(f);
        f0 = v.x, f1 = v.y;
      }
    };
    Ring<S::kSlots> r;
    Ring<S::kSets> sums;
    int turn = 0;
    bool ok = true;
    for (int u = first; u < p.units && ok; u += step, sums.next()) {
      float acc[2][4] = {};
      for (int s = s0; s < s1; ++s, r.next(), turn ^= 1) {
        if (turn != set) continue;
        const bool any = s * kStage + kw * kStep < p.K;
        if (any) load_x(s);
        ok = __all_sync(0xFFFFFFFFu, wait(&full[r.slot], r.phase, kSitePipeFull));
        if (!ok) break;
        if (any) {
          const uint32_t at = ring + r.slot * S::kSlot;
          uint32_t w[4][4], sw[4];  // rows rr + 8 h
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                         : "=r"(w[h][0]), "=r"(w[h][1]), "=r"(w[h][2]), "=r"(w[h][3]) : "r"(at + from + h * 1024));
            asm volatile("ld.shared.u32 %0, [%1];" : "=r"(sw[h]) : "r"(at + from_s + (u & 3) * 4 + h * 128));
          }
          const bool in = s * (kStage / 32) + kw * 4 + t < chunks;  // there may be no scales there
          float f[4][2];
#pragma unroll
          for (int h = 0; h < 4; ++h) scales_of(sw[h], in, f[h][0], f[h][1]);
          if constexpr (ONE) {
            float sum[2][2][4] = {};
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
              for (int m = 0; m < 2; ++m) {
                uint32_t up[4], down[4];
                decode_pairs<TYPE, false>(table, lane4, w[2 * m][i], 0, up);
                decode_pairs<TYPE, false>(table, lane4, w[2 * m + 1][i], 0, down);
                mma16816<TYPE>(sum[m][0], up[0], down[0], up[1], down[1], x[i].x, x[i].y);
                mma16816<TYPE>(sum[m][1], up[2], down[2], up[3], down[3], x[i].z, x[i].w);
              }
            // columns 2 t, 2 t + 1: the lane's own blocks
#pragma unroll
            for (int h = 0; h < 4; ++h)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int m = h >> 1, c = 2 * (h & 1) + e;
                acc[m][c] = fmaf(sum[m][0][c] + sum[m][1][c], f[h][e], acc[m][c]);
              }
          } else {
            uint32_t scale[4][2];  // of the row's two 16-value halves, as pairs
#pragma unroll
            for (int h = 0; h < 4; ++h)
#pragma unroll
              for (int e = 0; e < 2; ++e) scale[h][e] = f2_to_pair<TYPE>(f[h][e], f[h][e]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t b[4] = {x[i].x, x[i].y, x[i].z, x[i].w}, lo[4];
              if constexpr (kSplit) {
#pragma unroll
                for (int k = 0; k < 4; ++k) split_pair(b[k], b[k], lo[k]);
              }
#pragma unroll
              for (int m = 0; m < 2; ++m) {
                uint32_t up[4], down[4];
                decode_pairs<TYPE, true>(table, lane4, w[2 * m][i], scale[2 * m][i >> 1], up);
                decode_pairs<TYPE, true>(table, lane4, w[2 * m + 1][i], scale[2 * m + 1][i >> 1], down);
                mma16816<TYPE>(acc[m], up[0], down[0], up[1], down[1], b[0], b[1]);
                mma16816<TYPE>(acc[m], up[2], down[2], up[3], down[3], b[2], b[3]);
                if constexpr (kSplit) {
                  mma16816<TYPE>(acc[m], up[0], down[0], up[1], down[1], lo[0], lo[1]);
                  mma16816<TYPE>(acc[m], up[2], down[2], up[3], down[3], lo[2], lo[3]);
                }
              }
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[r.slot]);
      }
      if (!ok || !(ok = __all_sync(0xFFFFFFFFu, wait(&sums_empty[sums.slot], sums.phase ^ 1, kSitePipeAcc)))) break;
      float* mine = part + (sums.slot * kWarps + warp) * S::kSums;
      if constexpr (ONE) {  // the columns of a row are in its four lanes
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          float v = acc[h >> 1][2 * (h & 1)] + acc[h >> 1][2 * (h & 1) + 1];
          v += __shfl_xor_sync(0xFFFFFFFFu, v, 1);
          v += __shfl_xor_sync(0xFFFFFFFFu, v, 2);
          if (t == 0) mine[h * 8 + rr] = v;
        }
      } else {
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int e = 0; e < 4; ++e)  // row 16 m + 8 (e / 2) + rr, token 2 t + e % 2
            mine[(2 * t + (e & 1)) * S::kPitch + m * 16 + (e >> 1) * 8 + rr] = acc[m][e];
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sums_full[sums.slot]);
    }
  }
  __syncwarp();
  settle_after_failure(failed);
  if (p.splits > 1) {  // of the one unit
    cluster_sync();
    const float gamma = p.gamma ? *p.gamma : 1.0f, up = ONE ? kOneUp<XT> : 1.0f;
    for (int e = rank * kThreads + threadIdx.x; e < kRows * p.batch; e += kThreads * p.splits) {
      const int row = e % kRows, token = e / kRows;
      if (first * kRows + row >= p.N) continue;
      const uint32_t at = smem_addr(part + token * S::kPitch + row);
      float sum = 0.0f;
      for (int c = 0; c < p.splits; ++c) {
        float v;
        asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %1, %2;\n\tld.shared::cluster.f32 %0, [a];\n\t}"
                     : "=f"(v) : "r"(at), "r"(c) : "memory");
        sum += v;
      }
      const float bias = p.bias ? load_value<XT>(p.bias, first * kRows + row) : 0.0f;
      store_value<XT>(p.y, static_cast<size_t>(token) * p.N + first * kRows + row, fmaf(sum * up, gamma, bias));
    }
    cluster_sync();  // no CTA leaves while another reads its sums
  }
}

template <int FORMAT, int XT, bool ONE>
cudaError_t gemv_as(const Mx4Linear& c, uint32_t* status, cudaStream_t stream) {
  using S = Shape<FORMAT, ONE>;
  EncodeTiledFn encode = encode_tiled();
  if (!encode) return cudaErrorNotSupported;
  CUtensorMap map;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(c.K / 2), static_cast<cuuint64_t>(c.w.rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(c.K / 2)};
  const cuuint32_t box[2] = {kBox / 2, kRows}, ones[2] = {1, 1};
  if (encode(&map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(c.w.packed), dims, strides, box, ones,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  GemvParams p{};
  p.scales = c.w.scales;
  p.gamma = c.w.tensor_scale;
  p.x = c.x;
  p.bias = c.bias;
  p.y = c.y;
  p.status = status;
  p.N = c.w.rows;
  p.K = c.K;
  p.batch = c.batch;
  p.tiles = mx4_scale_tiles(c.K, FORMAT);
  p.units = (c.w.rows + kRows - 1) / kRows;
  p.splits = 1;
  while (p.splits < 8 && p.units * p.splits * 2 <= kSms && (c.K + kStage - 1) / kStage >= p.splits * 2) p.splits *= 2;
  auto* kernel = gemv_kernel<FORMAT, XT, ONE>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(S::kSmem));
  if (e != cudaSuccess) return e;
  const int ctas = p.units * p.splits;
  return launch_overlapped(kernel, p.splits > 1 || ctas < kSms ? ctas : kSms, kThreads, S::kSmem, stream, p.splits, map, p);
}

template <int FORMAT, int XT>
cudaError_t gemv_tokens(const Mx4Linear& c, uint32_t* status, cudaStream_t stream) {
  return c.batch == 1 ? gemv_as<FORMAT, XT, true>(c, status, stream) : gemv_as<FORMAT, XT, false>(c, status, stream);
}

}  // namespace

// Up to the eight tokens of one MMA, where this kernel is the faster (NVFP4 bf16, against the
// decoding tensor-core kernel: 1 token 4096 x 4096 5.2 us, 9.1; 28672 x 8192 33.6, 53.6; 8 tokens
// 6.6, 9.2 and 52, 53.8).  With two groups of tokens it was the slower of the two on large layers
// (16 tokens: 8.7, 9.6 and 61.2, 55.5).
bool mx4_gemv_takes(int batch) { return batch <= 8; }

cudaError_t launch_mx4_gemv(const Mx4Linear& c, uint32_t* status, cudaStream_t stream) {
  if (c.format == kMxfp4) return c.type == kF16 ? gemv_tokens<kMxfp4, kF16>(c, status, stream) : gemv_tokens<kMxfp4, kBf16>(c, status, stream);
  return c.type == kF16 ? gemv_tokens<kNvfp4, kF16>(c, status, stream) : gemv_tokens<kNvfp4, kBf16>(c, status, stream);
}

}  // namespace aqlm
