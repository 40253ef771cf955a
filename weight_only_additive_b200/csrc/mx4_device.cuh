// Device-side pieces shared by the mx4 kernels: where a block's scale lies, scale and
// e2m1 decoding, and conversions of the 16-bit types.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "aqlm_device.cuh"
#include "mx4_internal.h"

namespace aqlm {

// Byte of block c of row r in tiled scales with `tiles` 512-byte tiles along K.
__device__ __forceinline__ size_t mx4_scale_at(int r, int c, int tiles) {
  return (static_cast<size_t>(r >> 7) * tiles + (c >> 2)) * 512 + (r & 31) * 16 + ((r >> 5) & 3) * 4 + (c & 3);
}

// The fp32 value of a scale byte (exact; NaN codes give NaN).
template <int FORMAT>
__device__ __forceinline__ float mx4_scale_value(uint32_t b) {
  if constexpr (FORMAT == kMxfp4) {
    // 2^(b - 127): the exponent field; code 0 is the subnormal 2^-127
    const uint32_t bits = b == 255 ? 0x7FFFFFFFu : max(b << 23, 0x00400000u);
    return __uint_as_float(bits);
  } else {
    uint32_t h2;
    asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(h2) : "r"(b));
    return __half2float(__ushort_as_half(static_cast<unsigned short>(h2 & 0xFFFF)));
  }
}

// Eight e2m1 codes (low four bits first) as four pairs of fp16 or bf16 values, in order:
// byte lookups by the magnitude bits (in fp16 the low byte is always 0), the sign from a
// lookup whose codes with the sign bit repeat the top bit of 0x80.  The conversion
// instruction for e2m1 runs at 4 lanes a clock and SM (measured: it held the decoding
// products at 80 % of that pipe); these 15 to 17 logic instructions run at 64.
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
  return r;
}
template <int TYPE>
__device__ __forceinline__ void e2m1x8_decode(uint32_t w, uint32_t (&h)[4]) {
  constexpr uint32_t kHi0 = TYPE == kF16 ? 0x3E3C3800u : 0x3F3F3F00u, kHi1 = TYPE == kF16 ? 0x46444240u : 0x40404040u;
  const uint32_t m = w & 0x77777777u;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t mi = m >> (16 * i), wi = w >> (16 * i);
    const uint32_t sign = prmt(0x80808080u, 0x80808080u, wi);  // 0xFF or 0x80
    const uint32_t hi = prmt(kHi0, kHi1, mi) | ((sign << 7) & 0x80808080u);
    if constexpr (TYPE == kF16) {
      h[2 * i] = prmt(hi, 0, 0x1404);
      h[2 * i + 1] = prmt(hi, 0, 0x3424);
    } else {
      const uint32_t lo = prmt(0xC0800000u, 0xC0804000u, mi);
      h[2 * i] = prmt(lo, hi, 0x5140);
      h[2 * i + 1] = prmt(lo, hi, 0x7362);
    }
  }
}

__device__ __forceinline__ float2 b2_to_f2(uint32_t v) {
  return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
}

__device__ __forceinline__ uint32_t f2_to_b2_rn(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// A pair of 16-bit values of `TYPE` (kF16, kBf16) to and from fp32.
template <int TYPE>
__device__ __forceinline__ float2 pair_to_f2(uint32_t v) {
  return TYPE == kF16 ? h2_to_f2(v) : b2_to_f2(v);
}
template <int TYPE>
__device__ __forceinline__ uint32_t f2_to_pair(float lo, float hi) {
  return TYPE == kF16 ? f2_to_h2_rn(lo, hi) : f2_to_b2_rn(lo, hi);
}

// One value at index i of an array of `TYPE`.
template <int TYPE>
__device__ __forceinline__ float load_value(const void* p, size_t i) {
  if constexpr (TYPE == kF16) return __half2float(static_cast<const __half*>(p)[i]);
  else if constexpr (TYPE == kBf16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  else return static_cast<const float*>(p)[i];
}
template <int TYPE>
__device__ __forceinline__ void store_value(void* p, size_t i, float v) {
  if constexpr (TYPE == kF16) static_cast<__half*>(p)[i] = __float2half_rn(v);
  else if constexpr (TYPE == kBf16) static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
  else static_cast<float*>(p)[i] = v;
}

// ---------------------------------------------------------------------------
// CTA clusters and CTA pairs
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// All threads of all CTAs of the cluster; orders their shared memory accesses.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr, uint32_t rank) {
  float4 v;
  asm volatile(
      "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %4, %5;\n\t"
      "ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [a];\n\t}"
      : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr), "r"(rank) : "memory");
  return v;
}

// Bounded wait of the pipelined kernels for phase `parity` of `bar` (CLUSTER: other CTAs
// arrive on it).  The thread sleeps in the barrier unit, up to 10 ms at a time: warps that
// poll take shared-memory and issue slots from the ones that work (2048 x 4096 x 11008:
// 350 us polling, 300 us polling with clock reads between).
template <bool CLUSTER>
__device__ __forceinline__ bool mbar_sleep(uint64_t* bar, uint32_t parity) {
  uint32_t done;
  if constexpr (CLUSTER)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done) : "r"(smem_addr(bar)), "r"(parity), "r"(10000000u) : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done) : "r"(smem_addr(bar)), "r"(parity), "r"(10000000u) : "memory");
  return done != 0;
}
// `failed` (shared): another wait of this CTA has given up, so this one does too.
template <bool CLUSTER>
__device__ __forceinline__ bool mbar_wait_sleeping(uint64_t* bar, uint32_t parity, uint32_t* status, uint32_t site,
                                                   volatile uint32_t* failed) {
  if (mbar_sleep<CLUSTER>(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  while (!mbar_sleep<CLUSTER>(bar, parity)) {
    if (*failed) return false;
    if (global_timer_ns() - t0 > kWaitTimeoutNs) {
      record_failure(status, site);
      return false;
    }
  }
  return true;
}

// The end of all roles of a CTA.  After a wait that gave up, the copies and MMAs still in flight
// get a millisecond to end before the shared and tensor memory go away.
__device__ __forceinline__ void settle_after_failure(volatile uint32_t& failed) {
  __syncthreads();
  if (failed) {
    const uint64_t t0 = global_timer_ns();
    while (global_timer_ns() - t0 < 1000000) {
    }
  }
}

// One lane of a converged warp, the same one every time.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}
// A warp's index as a value that the compiler knows to be the same in all lanes.
__device__ __forceinline__ int uniform_warp() { return __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0); }

// Place in a ring of N slots and the parity of the phase that is running there.
template <int N>
struct Ring {
  uint32_t slot = 0, phase = 0;
  __device__ __forceinline__ void next() {
    if (++slot == N) slot = 0, phase ^= 1;
  }
};

// Arrive on the same barrier of the cluster's CTA 0, after this thread's shared-memory
// accesses and those it has waited for.  The fence is restricted to shared memory: a release
// of global memory too took about 1000 cycles a stage (2048 x 4096 x 11008: 172 -> 139 us).
// Tensor memory is not its matter: tc_fence_before_sync() comes before the call where tcgen05
// accesses are handed on.
__device__ __forceinline__ void mbar_arrive_leader(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %0, 0;\n\t"
      "fence.release.sync_restrict::shared::cta.cluster;\n\t"
      "mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [a];\n\t}" ::"r"(smem_addr(bar)) : "memory");
}

// tcgen05 instructions of one CTA (CG 1) or of a pair (CG 2: the even CTA issues for both;
// allocation is by a warp of each).
template <int CG>
__device__ __forceinline__ void tmem_alloc_cg(uint32_t* slot, uint32_t cols) {
  if constexpr (CG == 1) {
    tmem_alloc(slot, cols);
  } else {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(slot)), "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
}
template <int CG>
__device__ __forceinline__ void tmem_dealloc_cg(uint32_t taddr, uint32_t cols) {
  if constexpr (CG == 1) tmem_dealloc(taddr, cols);
  else asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(cols) : "memory");
}
// Arrive on `bar` (in both CTAs of a pair) when the MMAs issued so far have completed.
template <int CG>
__device__ __forceinline__ void umma_commit_cg(uint64_t* bar) {
  if constexpr (CG == 1) {
    umma_commit(bar);
  } else {
    const uint16_t both = 3;
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
        ::"r"(smem_addr(bar)), "h"(both) : "memory");
  }
}

// Load 32 consecutive 32-bit columns of this warp's 32 TMEM lanes; the values are there
// after tmem_ld_wait().
__device__ __forceinline__ void tmem_ld_x32_start(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr) : "memory");
}
template <int N>
__device__ __forceinline__ void tmem_ld_wait(uint32_t (&v)[N][32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
  // the values are used after the wait, not between
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int j = 0; j < 32; ++j) asm volatile("" : "+r"(v[i][j]));
}

// Fetches a tensor map ahead of the first copy that uses it.
__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// Launch with programmatic stream serialisation: the kernel's start overlaps the end of
// the one before it, and its grid_dependency_wait() orders its memory accesses after it.
template <typename... Params, typename... Args>
inline cudaError_t launch_overlapped(void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem,
                                     cudaStream_t stream, int cluster, Args... args) {
  cudaLaunchAttribute attr[2] = {};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
}

}  // namespace aqlm
