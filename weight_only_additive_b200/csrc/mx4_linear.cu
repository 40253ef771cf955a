// Products of 16-bit activations with a microscaled 4-bit weight matrix, for more than a
// few tokens: y = x . W^T + bias and the input gradient dx = dy . W, on the fp16 / bf16
// tensor-core path with the weights decoded on chip.
//
// The MMA's rows (TMEM lanes) are 128 output features a CTA, its columns a tile of up to
// 256 tokens.  Eight warps, or sixteen with a lookup table where a tile has few tokens, decode
// the weights of a stage (128 values of the reduction for y, 64 for dx) exactly: e2m1 times an
// e4m3 scale fits fp16 and bf16, e2m1 times a power of two fits bf16.  For y a lane's values go
// to tensor memory, which takes the decoded operand off the shared-memory ports; for dx, where
// the reduction runs over weight rows, they go to shared memory with the features contiguous
// (MN-major).  Packed weights and scales arrive by TMA in a ring of 256-deep slots,
// activations in one of stages.
//
// With many tokens two CTAs form a pair (cta_group::2): 256 features x 256 tokens, each
// decoding its own 128 features and loading half of the tokens, which halves the L2 traffic
// that bounds a single CTA's tile.  With few, a cluster of CTAs splits the reduction and
// adds the fp32 partial tiles through distributed shared memory in rank order.
//
// fp16 activations with MXFP4 weights fit neither type together: x is split into two bf16
// parts, x = hi + lo exactly (11 bits into 8 + 8), and every stage is multiplied twice.
#include "mx4_device.cuh"

namespace aqlm {
namespace {

constexpr int kF = 128;          // features of a CTA
constexpr int kSlotDepth = 256;  // reduction depth of a weight slot
constexpr int kRing = 4;         // stages in flight
constexpr int kSlotBytes = 16384, kSlotScales = 2048;
constexpr int kTableBytes = 65536;
constexpr int kSms = 148;

// TABLE: decoding by lookup and by sixteen warps, for the tiles of few tokens, whose small stages
// leave room for both (11008 x 4096 and 37 tokens: 17.4 us; 24.6 by eight warps without the table.
// Of sixteen without it, 16 tokens and 28672 x 8192 took 59.6 us, 55.4 with; 128 and 11008 x 4096
// 22.7, 20.9).
template <bool GRAD, bool TABLE>
struct Shape {
  static constexpr int kGroups = TABLE ? 4 : 2;  // of four decoding warps, which take stages in turn
  static constexpr int kWarpX = 0, kWarpMma = 1, kWarpDecode = 2, kWarpOut = 2 + 4 * kGroups, kWarpW = kWarpOut + 4;
  static constexpr int kThreads = (kWarpW + 1) * 32;
  // Reduction depth of a stage.  Every stage costs the warp that issues a wait and a commit, so
  // deep ones; dx's decoded stages lie in shared memory, which has room for 64.
  static constexpr int kDepth = GRAD ? 64 : 128;
  static constexpr int kSlotStages = kSlotDepth / kDepth;
  static constexpr int kABytes = GRAD ? kF * kDepth * 2 : 0;
  static constexpr uint32_t kACols = kDepth / 2;  // TMEM columns of a decoded stage (not GRAD)
  static constexpr int kWSlots = GRAD ? 3 : 4;
  static constexpr int kXBytes = (TABLE ? GRAD ? 32 : 64 : GRAD ? 96 : 128) * 1024;
  static constexpr int kX = kRing * kABytes;
  static constexpr int kW = kX + kXBytes;
  static constexpr int kS = kW + kWSlots * kSlotBytes;
  static constexpr size_t kSmem = (TABLE ? kTableBytes : 0) + kS + kWSlots * kSlotScales + 1024;
  // With more groups than stages in a slot, sets of groups take slots in turn.
  static constexpr int kSets = kGroups > kSlotStages ? kGroups / kSlotStages : 1;
  static constexpr int kSetGroups = kGroups / kSets;
  // A group's stages and slots are the same ones every time round: it waits for every phase of their
  // barriers, and none passes unseen.
  static_assert(kRing % kGroups == 0 && kSlotStages % kSetGroups == 0 && kWSlots % kSets == 0, "");
};
constexpr uint32_t kATmem = 256;  // first TMEM column of the decoded stages

struct LinearParams {
  const uint8_t* scales;
  const float* gamma;
  const void* bias;
  void* out;
  uint32_t* status;
  int features, depth, batch;  // of the output, of the reduction
  int tiles;                   // scale tiles along K
  int nt, f_tiles, t_tiles;    // tokens of a tile; tiles
  int splits, parts, out_type;
};

// Instruction descriptor of kind::f16 with fp32 sums; bit 15: A is MN-major.
template <int TYPE, bool GRAD>
__device__ __forceinline__ uint32_t linear_idesc(uint32_t m, uint32_t n) {
  const uint32_t t = TYPE == kBf16 ? 1u : 0u;
  return 1u << 4 | t << 7 | t << 10 | (GRAD ? 1u << 15 : 0u) | (n >> 3) << 17 | (m >> 4) << 24;
}

template <int CG>
__device__ __forceinline__ void umma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  if constexpr (CG == 1)
    umma_f16_ss(d, a, b, idesc, accumulate);
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate) : "memory");
}
template <int CG>
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  if constexpr (CG == 1)
    umma_f16_ts(d, a, b, idesc, accumulate);
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
        ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(accumulate) : "memory");
}

// MN-major 128-byte-swizzled stage: 64 reduction rows of 128 features; atoms of 8 rows x
// 64 features (1 KB), 8-row groups 1024 bytes apart, feature halves 8192.
__device__ __forceinline__ uint32_t mn_offset(int n, int chunk) {
  return static_cast<uint32_t>((chunk >> 3) * 8192 + (n >> 3) * 1024 + (n & 7) * 128 + (((chunk & 7) ^ (n & 7)) << 4));
}
__device__ __forceinline__ uint64_t mn_desc(uint32_t addr) {
  return static_cast<uint64_t>((addr >> 4) & 0x3FFFu) | static_cast<uint64_t>(8192u >> 4) << 16 |
         static_cast<uint64_t>(1024u >> 4) << 32 | static_cast<uint64_t>(1u) << 46 | static_cast<uint64_t>(2u) << 61;
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t bmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// The scale of a block whose scale byte is `b` as a pair of the decoded type (exact).
template <int FORMAT, int TYPE>
__device__ __forceinline__ uint32_t scale_pair(uint32_t b) {
  if constexpr (FORMAT == kMxfp4) {
    // bf16 exponent field; 2^-127 is subnormal
    const uint32_t e = b == 255 ? 0x7FC0u : max(b << 7, 0x40u);
    return e * 0x10001u;
  } else if constexpr (TYPE == kF16) {
    uint32_t h;
    asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(h) : "r"(b | b << 8));
    return h;
  } else {
    return (__float_as_uint(mx4_scale_value<kNvfp4>(b)) >> 16) * 0x10001u;
  }
}

// Eight codes times the scale as four pairs.  TABLE: a byte of two codes is looked up in the
// lane's copy of the table (256 bytes a row, a bank a lane; lane4 = 4 * lane).
template <int TYPE, bool TABLE>
__device__ __forceinline__ void decode_scaled(const uint8_t* table, uint32_t lane4, uint32_t codes, uint32_t scale,
                                              uint32_t (&h)[4]) {
  if constexpr (TABLE) {
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = *reinterpret_cast<const uint32_t*>(table + prmt(codes, lane4, 0x5504 | i << 4));
  } else {
    e2m1x8_decode<TYPE>(codes, h);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = TYPE == kF16 ? hmul2(h[i], scale) : bmul2(h[i], scale);
}

__device__ __forceinline__ void tmem_st_x32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};"
      ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
        "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]),
        "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}

template <int FORMAT, int TYPE, bool GRAD, int CG, bool TABLE>
__global__ void __launch_bounds__(Shape<GRAD, TABLE>::kThreads, 1) linear_kernel(const __grid_constant__ CUtensorMap x_map,
                                                             const __grid_constant__ CUtensorMap w_map,
                                                             const LinearParams p) {
  using S = Shape<GRAD, TABLE>;
  constexpr int kWarpX = S::kWarpX, kWarpMma = S::kWarpMma, kWarpDecode = S::kWarpDecode, kWarpOut = S::kWarpOut,
                kWarpW = S::kWarpW, kThreads = S::kThreads;
  extern __shared__ __align__(16) uint8_t table[];  // first, so that its address is a constant of the lookups
  const uint32_t smem = (smem_addr(table) + (TABLE ? kTableBytes : 0) + 1023) & ~1023u;
  uint8_t* smem_ptr = table + (smem - smem_addr(table));
  // ready: a stage's activations (one arrival and their bytes) and its decoded weights (4
  // warps); the first CTA of a pair also waits for its second's.  done: it is multiplied.
  __shared__ uint64_t ready[kRing], done[kRing], w_full[S::kWSlots], w_empty[S::kWSlots], acc_full[2], acc_empty[2];
  __shared__ uint32_t tmem_slot;
  __shared__ volatile uint32_t failed;

  const int warp = uniform_warp(), lane = threadIdx.x & 31;
  const int rank = CG > 1 || p.splits > 1 ? static_cast<int>(cluster_rank()) : 0;
  if (threadIdx.x == 0) {
    failed = 0;
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&ready[i], CG > 1 && rank == 0 ? 6 : 5);
      mbar_init(&done[i], 1);
    }
    for (int i = 0; i < S::kWSlots; ++i) {
      mbar_init(&w_full[i], 1);
      mbar_init(&w_empty[i], 4 * S::kSetGroups);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], 4 * CG);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kWarpMma) tmem_alloc_cg<CG>(&tmem_slot, 512);
  if (warp == kWarpX && lane == 0) prefetch_map(&x_map);
  if (warp == kWarpW && lane == 0) prefetch_map(&w_map);
  const uint32_t lane4 = lane * 4;
  if (TABLE && warp >= kWarpDecode && warp < kWarpOut) {  // a warp's 16 bytes, decoded by a lane each
    const int b0 = (warp - kWarpDecode) * 16;
    uint32_t h[4];
    e2m1x8_decode<TYPE>(b0 + (lane & 15), h);
#pragma unroll
    for (int b = 0; b < 16; ++b)
      *reinterpret_cast<uint32_t*>(table + (b0 + b) * 256 + lane4) = __shfl_sync(0xFFFFFFFFu, h[0], b);
  }
  tc_fence_before_sync();
  __syncthreads();
  if (CG > 1) cluster_sync();  // the pair's barriers are ready before either arrives on them
  tc_fence_after_sync();
  const uint32_t tmem = tmem_slot;

  const int slots = (p.depth + kSlotDepth - 1) / kSlotDepth;
  const int k_rank = CG > 1 ? 0 : rank;
  const int s0 = slots * k_rank / p.splits, s1 = slots * (k_rank + 1) / p.splits;
  const int total = p.f_tiles * p.t_tiles;
  const int per = CG > 1 ? CG : p.splits;
  const int first = blockIdx.x / per, step = gridDim.x / per;
  const int accs = GRAD || p.nt <= 128 ? 2 : 1;
  const uint32_t acc_cols = GRAD ? 256 : 128;
  const uint32_t x_box = static_cast<uint32_t>(p.nt / CG) * 128;          // bytes of 64 values of the tile's tokens
  const uint32_t x_part = x_box * (S::kDepth / 64), x_stage = x_part * p.parts;
  grid_dependency_wait();
  grid_dependents_launch();

  const auto features_at = [&](int t) { return (t / p.t_tiles) * kF * CG + (CG > 1 ? rank * kF : 0); };
  const auto tokens_at = [&](int t) { return (t % p.t_tiles) * p.nt; };
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
  // a warp waits as one
  const auto warp_ok = [&](auto&& waits) { return __all_sync(0xFFFFFFFFu, waits()) != 0; };

  if (warp == kWarpX) {
    // ---- activations; the whole warp walks the stages here too, and one lane issues
    const bool issuer = elect_one();
    const uint64_t keep = l2_policy_evict_last();
    Ring<kRing> r;
    bool ok = true;
    for (int t = first; t < total && ok; t += step) {
      const int row = tokens_at(t) + (CG > 1 ? rank * (p.nt / CG) : 0);
      for (int s = s0; s < s1 && ok; ++s)
        for (int j = 0; j < S::kSlotStages; ++j, r.next()) {
          ok = warp_ok([&] { return wait(&done[r.slot], r.phase ^ 1, kSitePipeEmpty); });
          if (!ok) break;
          uint32_t at = smem + S::kX + r.slot * x_stage;
          if (issuer) {
            mbar_arrive_expect_tx(&ready[r.slot], x_stage);
            for (int q = 0; q < p.parts; ++q)
#pragma unroll
              for (int h = 0; h < S::kDepth / 64; ++h, at += x_box)
                tma_load_2d(at, &x_map, s * kSlotDepth + j * S::kDepth + h * 64, row + q * p.batch, &ready[r.slot], keep);
          }
        }
    }
  } else if (warp == kWarpW) {
    // ---- packed weights and scales
    const bool issuer = elect_one();
    const uint64_t pol = p.t_tiles > 1 ? l2_policy_evict_last() : l2_policy_evict_first();
    const int row_tiles = ((GRAD ? p.depth : p.features) + 127) / 128;
    Ring<S::kWSlots> r;
    bool ok = true;
    for (int t = first; t < total && ok; t += step) {
      const int f0 = features_at(t);
      for (int s = s0; s < s1; ++s, r.next()) {
        ok = warp_ok([&] { return wait(&w_empty[r.slot], r.phase ^ 1, kSitePipeCodes); });
        if (!ok) break;
        const uint32_t at = smem + S::kW + r.slot * kSlotBytes, sc = smem + S::kS + r.slot * kSlotScales;
        // scale tiles: along K (y), or those of the CTA's features in two row tiles (dx)
        const int c0 = GRAD ? f0 / (4 * mx4_block(FORMAT)) : s * kSlotDepth / (4 * mx4_block(FORMAT));
        const int most = (GRAD ? kF : kSlotDepth) / (4 * mx4_block(FORMAT));
        const int r0 = GRAD ? s * 2 : f0 / 128, r_most = GRAD ? 2 : 1;
        // a pair's second CTA may have no features: its rows are read as zeros
        const uint32_t run = static_cast<uint32_t>(max(0, min(most, p.tiles - c0))) * 512;
        const int rows = run ? max(0, min(r_most, row_tiles - r0)) : 0;
        uint64_t* full = &w_full[r.slot];
        if (issuer) {
          mbar_arrive_expect_tx(full, kSlotBytes + rows * run);
          if constexpr (GRAD) tma_load_2d(at, &w_map, f0 / 2, s * kSlotDepth, full, pol);
          else tma_load_2d(at, &w_map, s * (kSlotDepth / 2), f0, full, pol);
          for (int q = 0; q < rows; ++q)
            bulk_load(sc + q * (kSlotScales / 2), p.scales + (static_cast<size_t>(r0 + q) * p.tiles + c0) * 512, run, full);
        }
      }
    }
  } else if (warp == kWarpMma && CG > 1 && rank > 0) {
    // ---- the pair's second CTA tells the first when its part of a stage is there
    Ring<kRing> r;
    bool ok = true;
    for (int t = first; t < total && ok; t += step)
      for (int s = s0; s < s1 && ok; ++s)
        for (int j = 0; j < S::kSlotStages && ok; ++j, r.next()) {
          ok = warp_ok([&] { return wait(&ready[r.slot], r.phase, kSitePipeFull); });
          if constexpr (!GRAD) {  // a link between the decoding warps' tcgen05.st and the first CTA's MMAs
            tc_fence_after_sync();
            tc_fence_before_sync();
          }
          if (ok && lane == 0) mbar_arrive_leader(&ready[r.slot]);
        }
  } else if (warp == kWarpMma) {
    // ---- MMAs: the whole warp walks the stages, so that descriptors stay in uniform
    // registers; one lane issues.  The lanes wait by themselves, since no whole-warp instruction
    // follows within a tile, and agree at its end (agreeing at every stage: 1 to 2 % of the time
    // of few tokens)
    const uint32_t idesc = linear_idesc<TYPE, GRAD>(kF * CG, p.nt);
    const bool issuer = elect_one();
    const uint64_t x_desc = umma_desc_sw128_kmajor(smem + S::kX), a_desc = mn_desc(smem);
    Ring<kRing> r;
    uint32_t n_acc = 0;
    bool ok = true;
    for (int t = first; t < total && ok; t += step, ++n_acc) {
      const uint32_t acc = accs == 2 ? n_acc & 1 : 0, acc_phase = accs == 2 ? (n_acc >> 1) & 1 : n_acc & 1;
      ok = wait_pair(&acc_empty[acc], acc_phase ^ 1, kSitePipeAcc);
      tc_fence_after_sync();
      const uint32_t d = tmem + acc * acc_cols;
      uint32_t go = 0;
      for (int s = s0; s < s1 && ok; ++s)
        for (int j = 0; j < S::kSlotStages; ++j, r.next()) {
          ok = wait_pair(&ready[r.slot], r.phase, kSitePipeFull);
          if (!ok) break;
          tc_fence_after_sync();
          uint64_t b = x_desc + ((r.slot * x_stage) >> 4);
          const uint64_t a = a_desc + r.slot * (S::kABytes >> 4);
          const uint32_t ta = tmem + kATmem + r.slot * S::kACols;
          if (issuer) {
            for (int q = 0; q < p.parts; ++q) {
#pragma unroll
              for (int h = 0; h < S::kDepth / 64; ++h, b += x_box >> 4) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  // 16 values: 32 bytes of a swizzled row; of A two 8-row groups, or 8 columns
                  if constexpr (GRAD) umma_ss<CG>(d, a + k * (2048 >> 4), b + k * 2, idesc, go);
                  else umma_ts<CG>(d, ta + h * 32 + k * 8, b + k * 2, idesc, go);
                  go = 1;
                }
              }
            }
            umma_commit_cg<CG>(&done[r.slot]);
          }
          go = 1;
        }
      ok = __all_sync(0xFFFFFFFFu, ok);
      if (ok && issuer) umma_commit_cg<CG>(&acc_full[acc]);
    }
  } else if (warp >= kWarpDecode && warp < kWarpOut) {
    // ---- decoding
    const uint32_t group = (warp - kWarpDecode) >> 2, quad = warp & 3;
    const uint32_t set = group / S::kSetGroups, j0 = group % S::kSetGroups;
    const int tid = quad * 32 + lane;
    Ring<S::kWSlots> w;
    uint32_t seq = 0;  // slots so far
    bool ok = true;
    for (int t = first; t < total && ok; t += step)
      for (int s = s0; s < s1 && ok; ++s, ++seq, w.next()) {
        if (S::kSets > 1 && seq % S::kSets != set) continue;
        ok = warp_ok([&] { return wait(&w_full[w.slot], w.phase, kSitePipeCodes); });
        if (!ok) break;
        const uint32_t at = smem + S::kW + w.slot * kSlotBytes, sc = smem + S::kS + w.slot * kSlotScales;
#pragma unroll 1
        for (uint32_t j = j0; j < S::kSlotStages; j += S::kSetGroups) {
          const uint32_t stage = (seq * S::kSlotStages + j) % kRing, phase = (seq * S::kSlotStages + j) / kRing & 1;
          constexpr int kWords = mx4_block(FORMAT) / 8;  // words of a block
          if constexpr (GRAD) {
            // weight row nl of the stage, 64 of its 128 features: eight lanes of a phase
            // have eight rows, so their 16-byte stores hit all banks
            const int nl = tid & 63, half = tid >> 6, row = static_cast<int>(j) * S::kDepth + nl;
            const uint32_t base = at + row * 64, turn = (row >> 1) & 3;
            const uint4 w0 = lds128(base + (((2 * half) ^ turn) << 4)), w1 = lds128(base + (((2 * half + 1) ^ turn) << 4));
            const uint32_t words[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
            const uint32_t chunk = FORMAT == kMxfp4 ? 0 : half;
            uint32_t four = lds32(sc + (row >> 7) * (kSlotScales / 2) + chunk * 512 + (row & 31) * 16 + ((row >> 5) & 3) * 4);
            if (FORMAT == kMxfp4) four >>= half * 16;
            const bool real = s * kSlotDepth + row < p.depth;  // scales of rows past the end may be anything
            uint8_t* a = smem_ptr + stage * S::kABytes;
            ok = warp_ok([&] { return wait(&done[stage], phase ^ 1, kSitePipeEmpty); });
            if (!ok) break;
#pragma unroll
            for (int b = 0; b < 8 / kWords; ++b) {
              const uint32_t scale = real ? scale_pair<FORMAT, TYPE>(four >> (8 * b) & 0xFF) : 0;
#pragma unroll
              for (int k = 0; k < kWords; ++k) {
                uint32_t h[4];
                decode_scaled<TYPE, TABLE>(table, lane4, words[b * kWords + k], scale, h);
                *reinterpret_cast<uint4*>(a + mn_offset(nl, half * 8 + b * kWords + k)) = make_uint4(h[0], h[1], h[2], h[3]);
              }
            }
            fence_proxy_async_smem();
          } else {
            // lane = feature: 64 values of its row at a time
            const uint32_t base = at + tid * 128;
            uint4 words[S::kDepth / 64][2];
            uint32_t fours[S::kDepth / 64];
#pragma unroll
            for (int h = 0; h < S::kDepth / 64; ++h) {
              const int c = j * (S::kDepth / 64) + h;  // 64 values: 32 bytes, a tile of NVFP4 scales, half an MXFP4 one
              words[h][0] = lds128(base + (((2 * c) ^ (tid & 7)) << 4));
              words[h][1] = lds128(base + (((2 * c + 1) ^ (tid & 7)) << 4));
              fours[h] = lds32(sc + (FORMAT == kMxfp4 ? c >> 1 : c) * 512 + lane * 16 + quad * 4);
            }
            ok = warp_ok([&] { return wait(&done[stage], phase ^ 1, kSitePipeEmpty); });
            if (!ok) break;
            tc_fence_after_sync();  // the stage's release (MMA commit) -> these tcgen05.st
#pragma unroll
            for (int h = 0; h < S::kDepth / 64; ++h) {
              const int c = j * (S::kDepth / 64) + h;
              const uint32_t word[8] = {words[h][0].x, words[h][0].y, words[h][0].z, words[h][0].w,
                                        words[h][1].x, words[h][1].y, words[h][1].z, words[h][1].w};
              const uint32_t four = FORMAT == kMxfp4 ? fours[h] >> ((c & 1) * 16) : fours[h];
              const bool real = s * kSlotDepth + c * 64 < p.depth;  // there may be no scales there
              uint32_t out[32];
#pragma unroll
              for (int b = 0; b < 8 / kWords; ++b) {
                const uint32_t scale = real ? scale_pair<FORMAT, TYPE>(four >> (8 * b) & 0xFF) : 0;
#pragma unroll
                for (int k = 0; k < kWords; ++k)
                  decode_scaled<TYPE, TABLE>(table, lane4, word[b * kWords + k], scale,
                                             *reinterpret_cast<uint32_t(*)[4]>(out + (b * kWords + k) * 4));
              }
              tmem_st_x32(tmem + kATmem + stage * S::kACols + h * 32 + (quad << 21), out);
            }
            tmem_st_wait();
            tc_fence_before_sync();
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&ready[stage]);
        }
        __syncwarp();
        if (ok && lane == 0) mbar_arrive(&w_empty[w.slot]);
      }
  } else if (warp >= kWarpOut && warp < kWarpW) {
    // ---- results
    const int quad = warp & 3;
    const float gamma = p.gamma ? *p.gamma : 1.0f;
    const bool out_f16 = TYPE == kF16 || (FORMAT == kMxfp4 && p.out_type == kF16);
    uint32_t n_acc = 0;
    for (int t = first; t < total; t += step, ++n_acc) {
      const uint32_t acc = accs == 2 ? n_acc & 1 : 0, acc_phase = accs == 2 ? (n_acc >> 1) & 1 : n_acc & 1;
      const int f = features_at(t) + quad * 32 + lane, t0 = tokens_at(t);
      const int tokens = min(p.nt, p.batch - t0);
      const bool real = f < p.features;
      float bias = 0.0f;
      if (p.bias && real) bias = p.out_type == kF16 ? load_value<kF16>(p.bias, f) : load_value<kBf16>(p.bias, f);
      if (!warp_ok([&] { return wait(&acc_full[acc], acc_phase, kSitePipeAcc); })) break;
      tc_fence_after_sync();
      const uint32_t d = tmem + acc * acc_cols + (static_cast<uint32_t>(quad * 32) << 16);
#pragma unroll 1
      for (int c = 0; c < p.nt; c += 16) {
        float v[16];
        tmem_ld_32x32b_x16(d + c, v);
        if (p.splits > 1) {
          float* red = reinterpret_cast<float*>(smem_ptr + S::kX) + quad * 32 + lane;
#pragma unroll
          for (int k = 0; k < 16; ++k) red[(c + k) * kF] = v[k];
        } else if (real) {
          uint16_t* o = static_cast<uint16_t*>(p.out) + static_cast<size_t>(t0 + c) * p.features + f;
#pragma unroll
          for (int k = 0; k < 16; ++k, o += p.features) {
            const float r = fmaf(v[k], gamma, bias);
            if (c + k < tokens) *o = out_f16 ? __half_as_ushort(__float2half_rn(r)) : __bfloat16_as_ushort(__float2bfloat16_rn(r));
          }
        }
      }
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) {
        if constexpr (CG == 1) mbar_arrive(&acc_empty[acc]);
        else mbar_arrive_leader(&acc_empty[acc]);
      }
    }
  }

  __syncwarp();
  settle_after_failure(failed);
  if (CG == 1 && p.splits > 1) {
    cluster_sync();
    const int f0 = features_at(first), t0 = tokens_at(first);
    const int tokens = min(p.nt, p.batch - t0);
    const float gamma = p.gamma ? *p.gamma : 1.0f;
    const uint32_t red = smem + S::kX;
    for (int e = rank * kThreads + threadIdx.x; e < tokens * (kF / 4); e += kThreads * p.splits) {
      const int c = e / (kF / 4), k = e % (kF / 4) * 4;
      float v[4] = {};
      for (int s = 0; s < p.splits; ++s) {
        const float4 a = ld_cluster_f4(red + (c * kF + k) * 4, s);
        v[0] += a.x, v[1] += a.y, v[2] += a.z, v[3] += a.w;
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int f = f0 + k + q;
        if (f >= p.features) break;
        const size_t at = static_cast<size_t>(t0 + c) * p.features + f;
        if (p.out_type == kF16) store_value<kF16>(p.out, at, fmaf(v[q], gamma, p.bias ? load_value<kF16>(p.bias, f) : 0.0f));
        else store_value<kBf16>(p.out, at, fmaf(v[q], gamma, p.bias ? load_value<kBf16>(p.bias, f) : 0.0f));
      }
    }
    cluster_sync();  // no CTA leaves while another reads its partial tile
  }
  tc_fence_before_sync();
  __syncthreads();
  if (CG > 1) cluster_sync();
  tc_fence_after_sync();
  if (warp == kWarpMma) tmem_dealloc_cg<CG>(tmem, 512);
}

// Activations laid out for the kernel: rows of `pitch` values (a multiple of 8), copied, or
// split into two bf16 parts, the second `total` values further on.
template <bool SPLIT>
__global__ void __launch_bounds__(256) restage_kernel(const uint16_t* __restrict__ x, uint16_t* __restrict__ out,
                                                      long long total, int cols, int pitch) {
  grid_dependency_wait();
  grid_dependents_launch();
  for (long long e = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x; e < total;
       e += static_cast<long long>(gridDim.x) * 256) {
    const long long r = e / pitch;
    const int c = static_cast<int>(e - r * pitch);
    const uint16_t raw = c < cols ? x[r * cols + c] : 0;
    if constexpr (SPLIT) {
      const float v = __half2float(__ushort_as_half(raw));
      const __nv_bfloat16 hi = __float2bfloat16_rn(v);
      const float rest = v - __bfloat162float(hi);
      out[e] = __bfloat16_as_ushort(hi);
      out[total + e] = __bfloat16_as_ushort(__float2bfloat16_rn(isfinite(v) ? rest : 0.0f));
    } else {
      out[e] = raw;
    }
  }
}

struct Call {
  const void* x;  // [batch, depth]
  Mx4 w;
  const void* bias;
  void* out;
  int type, features, depth, K, batch, format;
  void* workspace;
};

bool split_parts(int type, int format) { return type == kF16 && format == kMxfp4; }
size_t restaged_bytes(int type, int format, long long depth, long long batch) {
  if (!split_parts(type, format) && depth % 8 == 0) return 0;
  return static_cast<size_t>(batch) * ((depth + 7) / 8 * 8) * 2 * (split_parts(type, format) ? 2 : 1);
}

struct Tiling {
  int nt, cg, splits;
  bool table;
};

// Tokens of a tile, pairs, lookup decoding and the split of the reduction: the least time of
// rounds over the SMs, in cycles, by what 128 values of the reduction take and what the launch
// and a tile take besides.  Measured with 4096 to 14336 features: 5.3 cycles a token of the tile,
// but at least 840 with the table and 1400 without (dx: 1200 and 1550), which is the
// decoding, and 250 more for x in two parts.
// So pairs with the table take the middle (512 tokens, 4096 x 4096: 19 us, 28 without, 33 by
// single CTAs), wide tiles without it the large batches (2048 x 4096 x 11008: 124 us, 149 with).
Tiling plan(int features, int depth, int batch, int parts, bool grad) {
  const int slots = (depth + kSlotDepth - 1) / kSlotDepth;
  Tiling best{};
  double least = 0;
  for (int cg = 1; cg <= 2; ++cg) {
    const long long f_tiles = (features + kF * cg - 1) / (kF * cg);
    for (int table = 0; table <= 1; ++table) {
      const int most = (table ? 64 : grad && cg == 1 ? 192 : 128) * cg / parts;
      const double decode = (table ? grad ? 1200 : 840 : grad ? 1550 : 1400) + (parts > 1 ? 250 : 0);
      for (int t_tiles = (batch + most - 1) / most, more = 0; more < 6; ++more, ++t_tiles) {
        const int unit = 16 * cg, nt = ((batch + t_tiles - 1) / t_tiles + unit - 1) / unit * unit;
        const long long tiles = f_tiles * ((batch + nt - 1) / nt);
        const double mma = 5.3 * nt * parts, stage = mma > decode ? mma : decode;
        for (int splits = 1; splits <= (cg == 1 ? 8 : 1); splits *= 2) {
          if (splits > 1 && (tiles * splits > kSms || slots < 2 * splits)) break;
          const long long rounds = (tiles * cg * splits + kSms - 1) / kSms;
          const double cost = rounds * (2.0 * ((slots + splits - 1) / splits) * stage + 1500) + 9000 + (splits > 1 ? 1500 : 0);
          if (least == 0 || cost < least) least = cost, best = Tiling{nt, cg, splits, table != 0};
        }
      }
    }
  }
  return best;
}

cudaError_t map_2d(CUtensorMap* map, CUtensorMapDataType type, const void* p, uint64_t cols, uint64_t rows, uint64_t pitch,
                   uint32_t box_cols, uint32_t box_rows, CUtensorMapSwizzle swizzle) {
  EncodeTiledFn encode = encode_tiled();
  if (!encode) return cudaErrorNotSupported;
  const cuuint64_t dims[2] = {cols, rows}, strides[1] = {pitch};
  const cuuint32_t box[2] = {box_cols, box_rows}, ones[2] = {1, 1};
  return encode(map, type, 2, const_cast<void*>(p), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? cudaSuccess
             : cudaErrorInvalidValue;
}

template <int FORMAT, int TYPE, bool GRAD, int CG, bool TABLE>
cudaError_t launch_linear(const Call& c, const Tiling& tl, uint32_t* status, cudaStream_t stream) {
  using S = Shape<GRAD, TABLE>;
  const int parts = split_parts(c.type, c.format) ? 2 : 1;
  const int pitch = (c.depth + 7) / 8 * 8;
  const void* x = c.x;
  cudaError_t e;
  if (restaged_bytes(c.type, c.format, c.depth, c.batch)) {
    const long long total = static_cast<long long>(c.batch) * pitch;
    const long long blocks = (total + 255) / 256;
    auto* out = static_cast<uint16_t*>(c.workspace);
    e = launch_overlapped(parts > 1 ? restage_kernel<true> : restage_kernel<false>,
                          static_cast<unsigned>(blocks < kSms * 64 ? blocks : kSms * 64), 256, 0, stream, 1,
                          static_cast<const uint16_t*>(c.x), out, total, c.depth, pitch);
    if (e != cudaSuccess) return e;
    x = out;
  }
  CUtensorMap x_map, w_map;
  e = map_2d(&x_map, TYPE == kF16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, x, c.depth,
             static_cast<uint64_t>(c.batch) * parts, static_cast<uint64_t>(pitch) * 2, 64, tl.nt / CG,
             CU_TENSOR_MAP_SWIZZLE_128B);
  if (e != cudaSuccess) return e;
  e = map_2d(&w_map, CU_TENSOR_MAP_DATA_TYPE_UINT8, c.w.packed, c.K / 2, c.w.rows, c.K / 2, GRAD ? 64 : 128,
             GRAD ? 256 : 128, GRAD ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B);
  if (e != cudaSuccess) return e;
  LinearParams q{};
  q.scales = c.w.scales;
  q.gamma = c.w.tensor_scale;
  q.bias = c.bias;
  q.out = c.out;
  q.status = status;
  q.features = c.features;
  q.depth = c.depth;
  q.batch = c.batch;
  q.tiles = mx4_scale_tiles(c.K, FORMAT);
  q.nt = tl.nt;
  q.f_tiles = (c.features + kF * CG - 1) / (kF * CG);
  q.t_tiles = (c.batch + tl.nt - 1) / tl.nt;
  q.splits = tl.splits;
  q.parts = parts;
  q.out_type = c.type;
  const long long tiles = static_cast<long long>(q.f_tiles) * q.t_tiles;
  if (tiles > 0x7FFFFFFF / 8) return cudaErrorInvalidValue;
  auto* kernel = linear_kernel<FORMAT, TYPE, GRAD, CG, TABLE>;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(S::kSmem));
  if (e != cudaSuccess) return e;
  const long long ctas = tiles * CG * tl.splits;
  const unsigned grid = static_cast<unsigned>(tl.splits > 1 || ctas < kSms ? ctas : kSms);
  return launch_overlapped(kernel, grid, S::kThreads, S::kSmem, stream, CG * tl.splits, x_map, w_map, q);
}

template <bool GRAD>
cudaError_t run(const Call& c, uint32_t* status, cudaStream_t stream) {
  const Tiling tl = plan(c.features, c.depth, c.batch, split_parts(c.type, c.format) ? 2 : 1, GRAD);
#define MX4_CASE(f, t)                                                                     \
  if (tl.table)                                                                            \
    return tl.cg == 2 ? launch_linear<f, t, GRAD, 2, true>(c, tl, status, stream)          \
                      : launch_linear<f, t, GRAD, 1, true>(c, tl, status, stream);         \
  return tl.cg == 2 ? launch_linear<f, t, GRAD, 2, false>(c, tl, status, stream)           \
                    : launch_linear<f, t, GRAD, 1, false>(c, tl, status, stream);
  if (c.format == kMxfp4) { MX4_CASE(kMxfp4, kBf16) }
  if (c.type == kF16) { MX4_CASE(kNvfp4, kF16) }
  MX4_CASE(kNvfp4, kBf16)
#undef MX4_CASE
}

}  // namespace

size_t mx4_linear_workspace(int type, int format, long long K, long long batch) {
  return mx4_gemv_takes(static_cast<int>(batch)) ? 0 : restaged_bytes(type, format, K, batch);
}
size_t mx4_grad_workspace(int type, int format, long long N, long long batch) {
  return restaged_bytes(type, format, N, batch);
}

cudaError_t launch_mx4_linear(const Mx4Linear& p, uint32_t* status, cudaStream_t stream) {
  if (mx4_gemv_takes(p.batch)) return launch_mx4_gemv(p, status, stream);
  return run<false>(Call{p.x, p.w, p.bias, p.y, p.type, p.w.rows, p.K, p.K, p.batch, p.format, p.workspace}, status, stream);
}

cudaError_t launch_mx4_grad(const Mx4Grad& p, uint32_t* status, cudaStream_t stream) {
  return run<true>(Call{p.dy, p.w, nullptr, p.dx, p.type, p.K, p.w.rows, p.K, p.batch, p.format, p.workspace}, status, stream);
}

}  // namespace aqlm
