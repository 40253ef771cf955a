// y = x . W^T + bias with 16-bit x and microscaled 4-bit W, for a few tokens: bound by
// reading the weights, so they go from global memory to registers, are decoded there and
// multiplied by mma.sync (16 rows x 8 tokens x 16 values), which keeps the arithmetic per
// weight well below what fp32 FMAs would take.
//
// A warp has 32 weight rows, eight neighbours in each of the four 32-row parts of a scale
// tile, so that one 16-byte load brings the four rows' scales of four blocks.  In a step of
// 128 values lane (g, t) reads 32 of them (16 bytes) in rows g of the four parts.  Which of
// the 128 values an MMA takes is free as long as x is taken alike: a word's nibbles j and
// j + 4 make a pair, which costs two shifts and two logic operations to form.
//
// The decoded weight is exact: bf16 holds e2m1 times 2^e or e4m3, fp16 holds e2m1 * e4m3 *
// 2^-14 (a multiple of 2^-24).  fp16 x with MXFP4 weights is split into two bf16 parts.
//
// Warps of a CTA and CTAs of a cluster share the reduction; partial sums are fp32, added in
// a fixed order.
#include "mx4_device.cuh"

namespace aqlm {
namespace {

constexpr int kWarps = 8, kThreads = kWarps * 32;
constexpr int kStep = 128;
constexpr int kSms = 148;

struct GemvParams {
  const uint8_t* packed;
  const uint8_t* scales;
  const float* gamma;
  const void* x;
  const void* bias;
  void* y;
  int N, K, batch, tiles;
  int split_warps;   // warps of a CTA that share rows
  int split_ctas;    // CTAs of a cluster that do
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

// Eight codes as the pairs (j, j + 4), j = 0..3, times `scale`.
//   fp16: the code's three magnitude bits as the low exponent and top mantissa bits are
//         e2m1 * 2^-14; the scale comes without that factor, which the caller takes out.
//   bf16: likewise e2m1 * 2^-126; times 2^126, then times the scale.
template <int TYPE>
__device__ __forceinline__ void decode_pairs(uint32_t w, uint32_t scale, uint32_t (&h)[4]) {
  constexpr int kUp = TYPE == kF16 ? 9 : 6;
  constexpr uint32_t kMask = TYPE == kF16 ? 0x0E000E00u : 0x01C001C0u;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int by = kUp - 4 * j;
    const uint32_t mag = (by >= 0 ? w << by : w >> -by) & kMask;
    const uint32_t v = mag | ((w << (12 - 4 * j)) & 0x80008000u);
    if constexpr (TYPE == kF16) {
      asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(h[j]) : "r"(v), "r"(scale));
    } else {
      uint32_t u;
      asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(u) : "r"(v), "r"(0x7E807E80u));  // 2^126
      asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(h[j]) : "r"(u), "r"(scale));
    }
  }
}

// Two bf16 parts of a pair of fp16 values, hi + lo exactly: hi keeps 8 significant bits.
// An infinity's second part is some finite value.
__device__ __forceinline__ void split_pair(uint32_t x, uint32_t& hi, uint32_t& lo) {
  const uint32_t top = x & 0xFFF8FFF8u;
  const __half2 rest = __hmin2(__hsub2(*reinterpret_cast<const __half2*>(&x), *reinterpret_cast<const __half2*>(&top)),
                               __half2half2(__ushort_as_half(0x7BFF)));
  const float2 h = h2_to_f2(top), l = __half22float2(rest);
  hi = f2_to_b2_rn(h.x, h.y);
  lo = f2_to_b2_rn(l.x, l.y);
}

struct Weights {
  uint4 w[4];  // rows of the four parts
  uint4 s;     // their scale words
};

template <int FORMAT, int XT, int NB>
__global__ void __launch_bounds__(kThreads, NB > 2 ? 1 : 2) gemv_kernel(const GemvParams p) {
  constexpr bool kSplit = FORMAT == kMxfp4 && XT == kF16;
  constexpr int TYPE = kSplit ? kBf16 : XT;
  constexpr int kX = NB * 8;  // tokens
  __shared__ __align__(16) float part[kWarps * 32 * kX];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int rank = p.split_ctas > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int groups = kWarps / p.split_warps;  // 32-row groups of a CTA
  const int group = (blockIdx.x / p.split_ctas) * groups + warp / p.split_warps;
  const int tile = group >> 2, row0 = tile * 128 + (group & 3) * 8 + g;  // + 32 q
  const int first = rank * p.split_warps + warp % p.split_warps, stride = p.split_warps * p.split_ctas;
  const int steps = (p.K + kStep - 1) / kStep, chunks = p.K / 32;

  grid_dependency_wait();
  grid_dependents_launch();

  const uint64_t stream = l2_policy_evict_first();
  const uint8_t* rows[4];
  bool real[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int row = row0 + 32 * q;
    real[q] = row < p.N;
    rows[q] = p.packed + static_cast<size_t>(real[q] ? row : 0) * (p.K / 2) + t * 16;
  }
  // MXFP4: a step is one scale tile, lane t's block its byte t; NVFP4: two tiles, lane t's
  // two blocks a half word of tile t / 2
  const uint8_t* scale_at = p.scales + static_cast<size_t>(tile) * p.tiles * 512 + (row0 & 31) * 16;
  const auto load = [&](Weights& v, int s) {
    const bool in = s < steps && s * 4 + t < chunks;
#pragma unroll
    for (int q = 0; q < 4; ++q)
      v.w[q] = in && real[q] ? ldg_stream_v4(rows[q] + static_cast<size_t>(s) * 64, stream) : make_uint4(0, 0, 0, 0);
    const int c = FORMAT == kMxfp4 ? s : 2 * s + (t >> 1);
    v.s = in && tile * 128 < p.N ? ldg_nc_v4(scale_at + static_cast<size_t>(c) * 512) : make_uint4(0, 0, 0, 0);
  };

  float acc[2][NB][4] = {};
  const auto multiply = [&](const Weights& v, int s) {
    // x, permuted like the weights
    uint32_t b[NB][16], lo[kSplit ? NB : 1][16];
    const bool in = s * 4 + t < chunks;
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      const int token = n * 8 + g;
      const uint4* at = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.x) + static_cast<size_t>(token) * p.K +
                                                       s * kStep + t * 32);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint4 r = make_uint4(0, 0, 0, 0);
        if (in && token < p.batch) r = ldg_nc_v4(at + i);
        uint32_t u[4] = {r.x, r.y, r.z, r.w};
        if constexpr (kSplit) {
          uint32_t l[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) split_pair(u[k], u[k], l[k]);
          lo[n][4 * i] = prmt(l[0], l[2], 0x5410), lo[n][4 * i + 1] = prmt(l[0], l[2], 0x7632);
          lo[n][4 * i + 2] = prmt(l[1], l[3], 0x5410), lo[n][4 * i + 3] = prmt(l[1], l[3], 0x7632);
        }
        b[n][4 * i] = prmt(u[0], u[2], 0x5410), b[n][4 * i + 1] = prmt(u[0], u[2], 0x7632);
        b[n][4 * i + 2] = prmt(u[1], u[3], 0x5410), b[n][4 * i + 3] = prmt(u[1], u[3], 0x7632);
      }
    }
    const uint32_t words[4] = {v.s.x, v.s.y, v.s.z, v.s.w};
    uint32_t scale[4][2];  // of the row's two 16-value halves
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if constexpr (FORMAT == kMxfp4) {
        const uint32_t e = words[q] >> (8 * t) & 0xFF;
        scale[q][0] = scale[q][1] = (e == 255 ? 0x7FC0u : max(e << 7, 0x40u)) * 0x10001u;
      } else {
        uint32_t h;  // two fp16 scales
        asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(h) : "r"(words[q] >> (16 * (t & 1))));
        if constexpr (TYPE == kBf16) {
          const float2 f = h2_to_f2(h);
          h = f2_to_b2_rn(f.x, f.y);
        }
        scale[q][0] = prmt(h, h, 0x1010);
        scale[q][1] = prmt(h, h, 0x3232);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        uint32_t up[4], down[4];
        const auto word = [&](const uint4& r) { return i == 0 ? r.x : i == 1 ? r.y : i == 2 ? r.z : r.w; };
        decode_pairs<TYPE>(word(v.w[2 * m]), scale[2 * m][i >> 1], up);
        decode_pairs<TYPE>(word(v.w[2 * m + 1]), scale[2 * m + 1][i >> 1], down);
#pragma unroll
        for (int n = 0; n < NB; ++n) {
          mma16816<TYPE>(acc[m][n], up[0], down[0], up[1], down[1], b[n][4 * i], b[n][4 * i + 1]);
          mma16816<TYPE>(acc[m][n], up[2], down[2], up[3], down[3], b[n][4 * i + 2], b[n][4 * i + 3]);
          if constexpr (kSplit) {
            mma16816<TYPE>(acc[m][n], up[0], down[0], up[1], down[1], lo[n][4 * i], lo[n][4 * i + 1]);
            mma16816<TYPE>(acc[m][n], up[2], down[2], up[3], down[3], lo[n][4 * i + 2], lo[n][4 * i + 3]);
          }
        }
      }
  };

  // two steps of weights in flight
  Weights v0, v1;
  load(v0, first);
  load(v1, first + stride);
  for (int s = first; s < steps; s += 2 * stride) {
    multiply(v0, s);
    load(v0, s + 2 * stride);
    if (s + stride < steps) {
      multiply(v1, s + stride);
      load(v1, s + 3 * stride);
    }
  }

  // ---- partial sums of the warps, then of the CTAs
  float* mine = part + warp * 32 * kX;
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e)  // row part 2 m + e / 2, row g, token 8 n + 2 t + e % 2
        mine[((2 * m + (e >> 1)) * 8 + g) * kX + n * 8 + 2 * t + (e & 1)] = acc[m][n][e];
  __syncthreads();
  if (p.split_ctas > 1) {
    if (p.split_warps > 1) {
      // into the first warp's place; each element is read and written by one thread
      for (int e = threadIdx.x; e < groups * 32 * kX; e += kThreads) {
        float* at = part + e / (32 * kX) * p.split_warps * 32 * kX + e % (32 * kX);
        float sum = at[0];
        for (int w = 1; w < p.split_warps; ++w) sum += at[w * 32 * kX];
        at[0] = sum;
      }
    }
    cluster_sync();
  }
  const float factor = (FORMAT == kNvfp4 && TYPE == kF16 ? 16384.0f : 1.0f) * (p.gamma ? *p.gamma : 1.0f);
  const uint32_t base = smem_addr(part);
  for (int e = rank * kThreads + threadIdx.x; e < groups * 32 * p.batch; e += kThreads * p.split_ctas) {
    const int r = e % 32, token = e / 32 % p.batch, gr = e / 32 / p.batch;
    const int id = (blockIdx.x / p.split_ctas) * groups + gr;
    const int row = (id >> 2) * 128 + (id & 3) * 8 + (r & 7) + (r >> 3) * 32;
    if (row >= p.N) continue;
    const int at = gr * p.split_warps * 32 * kX + r * kX + token;
    float sum = 0.0f;
    if (p.split_ctas > 1) {
      for (int c = 0; c < p.split_ctas; ++c) {
        float v;
        asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %1, %2;\n\tld.shared::cluster.f32 %0, [a];\n\t}"
                     : "=f"(v) : "r"(base + at * 4), "r"(c) : "memory");
        sum += v;
      }
    } else {
      for (int w = 0; w < p.split_warps; ++w) sum += part[at + w * 32 * kX];
    }
    const float bias = p.bias ? load_value<XT>(p.bias, row) : 0.0f;
    store_value<XT>(p.y, static_cast<size_t>(token) * p.N + row, fmaf(sum, factor, bias));
  }
  if (p.split_ctas > 1) cluster_sync();  // no CTA leaves while another reads its sums
}

template <int FORMAT, int XT, int NB>
cudaError_t gemv_as(const Mx4Linear& c, cudaStream_t stream) {
  GemvParams p{};
  p.packed = c.w.packed;
  p.scales = c.w.scales;
  p.gamma = c.w.tensor_scale;
  p.x = c.x;
  p.bias = c.bias;
  p.y = c.y;
  p.N = c.w.rows;
  p.K = c.K;
  p.batch = c.batch;
  p.tiles = mx4_scale_tiles(c.K, FORMAT);
  // all warps of a CTA on one row group, then clusters, until there are CTAs for the SMs
  const int steps = (c.K + kStep - 1) / kStep;
  const long long row_groups = (static_cast<long long>(c.w.rows) + 127) / 128 * 4;
  p.split_warps = kWarps;
  while (p.split_warps > 1 && (steps < 2 * p.split_warps || row_groups / (kWarps / p.split_warps) >= 16 * kSms)) p.split_warps /= 2;
  p.split_ctas = 1;
  const int groups = kWarps / p.split_warps;
  const long long ctas = (row_groups + groups - 1) / groups;
  while (p.split_ctas < 8 && ctas * p.split_ctas < kSms && steps >= 4 * p.split_warps * p.split_ctas) p.split_ctas *= 2;
  return launch_overlapped(gemv_kernel<FORMAT, XT, NB>, static_cast<unsigned>(ctas * p.split_ctas), kThreads, 0, stream,
                           p.split_ctas, p);
}

template <int FORMAT, int XT>
cudaError_t gemv_tokens(const Mx4Linear& c, cudaStream_t stream) {
  if (c.batch <= 8) return gemv_as<FORMAT, XT, 1>(c, stream);
  if (c.batch <= 16) return gemv_as<FORMAT, XT, 2>(c, stream);
  return gemv_as<FORMAT, XT, 4>(c, stream);
}

}  // namespace

bool mx4_gemv_takes(int batch) { return batch <= 32; }

cudaError_t launch_mx4_gemv(const Mx4Linear& c, cudaStream_t stream) {
  if (c.format == kMxfp4) return c.type == kF16 ? gemv_tokens<kMxfp4, kF16>(c, stream) : gemv_tokens<kMxfp4, kBf16>(c, stream);
  return c.type == kF16 ? gemv_tokens<kNvfp4, kF16>(c, stream) : gemv_tokens<kNvfp4, kBf16>(c, stream);
}

}  // namespace aqlm
