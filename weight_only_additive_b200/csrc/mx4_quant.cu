// Quantisation to and dequantisation from microscaled 4-bit floating point.
//
// Both are one pass bound by HBM: a thread takes 32 consecutive values of a
// row at a time.
#include "mx4_device.cuh"

namespace aqlm {
namespace {

constexpr int kThreads = 256;
constexpr int kSms = 148;

// A thread's way through rows of `units` pieces, `stride` pieces at a time: one division at
// the start, then additions.
struct Walk {
  int row, u;  // piece u of a row
  int rows_on, units_on, units;
  __device__ __forceinline__ Walk(long long first, long long stride, int units_) : units(units_) {
    row = static_cast<int>(first / units);
    u = static_cast<int>(first - static_cast<long long>(row) * units);
    rows_on = static_cast<int>(stride / units);
    units_on = static_cast<int>(stride - static_cast<long long>(rows_on) * units);
  }
  __device__ __forceinline__ void next() {
    row += rows_on;
    u += units_on;
    if (u >= units) u -= units, ++row;
  }
};

// 32 bytes at p (16-byte aligned; `wide`: 32-byte aligned).
__device__ __forceinline__ void load32(const void* p, bool wide, uint32_t (&v)[8]) {
  uint4 a, b;
  if (wide) {
    ldg_nc_v8(p, a, b);
  } else {
    a = ldg_nc_v4(p);
    b = ldg_nc_v4(static_cast<const uint8_t*>(p) + 16);
  }
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}

__device__ __forceinline__ void store32(void* p, bool wide, const uint32_t (&v)[8]) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]) : "memory");
  } else {
    uint4* q = static_cast<uint4*>(p);
    q[0] = make_uint4(v[0], v[1], v[2], v[3]);
    q[1] = make_uint4(v[4], v[5], v[6], v[7]);
  }
}

// Two bytes of e2m1 pairs: (a0, a1) in the low byte, (a2, a3) in the next, and so on.
__device__ __forceinline__ uint32_t to_e2m1x8(const float (&a)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(a[0]), "f"(a[1]), "f"(a[2]), "f"(a[3]), "f"(a[4]), "f"(a[5]), "f"(a[6]), "f"(a[7]));
  return r;
}

__device__ __forceinline__ uint32_t to_e4m3(float v) {
  uint32_t r;
  asm("{\n\t.reg .b16 t;\n\tcvt.rn.satfinite.e4m3x2.f32 t, %1, %1;\n\tcvt.u32.u16 %0, t;\n\t}" : "=r"(r) : "f"(v));
  return r & 0xFF;
}

// The e2m1 code of x / unit from exact products in 64 bits (a midpoint has 3 bits, the
// unit at most 28): one more for every midpoint below |x|, ties to the even code.
__device__ __forceinline__ uint32_t exact_e2m1(float x, double unit) {
  const double a = fabs(static_cast<double>(x));
  uint32_t code = 0;
#pragma unroll
  for (int i = 0; i < 7; ++i) {
    const double mid = i < 4 ? 0.25 + 0.5 * i : i < 6 ? i - 1.5 : 5.0;
    const double border = mid * unit;
    code += a > border || (a == border && (i & 1)) ? 1u : 0u;
  }
  return code | (__float_as_uint(x) >> 31 << 3);
}

// `codes` of the eight values at x, those whose nibble is set in `doubt` decided exactly.
template <int TYPE>
__device__ __noinline__ uint32_t settle(const void* x, uint32_t codes, uint32_t doubt, float s, float gamma) {
  const double unit = static_cast<double>(s) * static_cast<double>(gamma);
  while (doubt) {
    const int i = (__ffs(doubt) - 1) >> 2;
    const uint32_t at = 0xFu << (4 * i);
    codes = (codes & ~at) | exact_e2m1(load_value<TYPE>(x, i), unit) << (4 * i);
    doubt &= ~at;
  }
  return codes;
}

// The sign of x - b c for a product within a few units in the last place of x, exact: the
// difference to the rounded product and that product's error have few bits each.  The error's
// last bit has to be one that fp32 holds: with b in multiples of 2^-9 (borders of e4m3 scales) c is
// at least 2^-117, with whole b (borders of values) at least 2^-126.  `c_low` is what c lacks.
__device__ __forceinline__ float beyond(float x, float b, float c, float c_low) {
  const float p = b * c;
  return (x - p) - fmaf(b, c_low, fmaf(b, c, -p));
}

// e4m3 of amax / (6 gamma) that lies next to the border between the neighbours `low` and
// low + 1: by the exact comparison of amax with it, ties to the even code.
__device__ __forceinline__ uint32_t settle_scale(float amax, float gamma, uint32_t low) {
  const float border = 3.0f * (mx4_scale_value<kNvfp4>(low) + mx4_scale_value<kNvfp4>(low + 1));  // 6 bits
  const float d = beyond(amax, border, gamma, 0.0f);
  return low + (d > 0.0f || (d == 0.0f && (low & 1)) ? 1 : 0);
}

// The same for a gamma whose quotients or borders fp32 does not hold.  The 64-bit quotient is within 2^-52 of
// the exact one, which stays 2^-33 away from every tie unless it is one (its terms have 24 and
// 27 bits), so what lies within 2^-40 of an fp32 value is that value, and anything else goes to
// the odd fp32 neighbour: the conversion then rounds it as it would the quotient.
__device__ __noinline__ uint32_t scale_of_extreme(float amax, float gamma) {
  const double v = fmin(static_cast<double>(amax) / (6.0 * static_cast<double>(gamma)), 1024.0);
  const float f = __double2float_rn(v);
  const double r = v - static_cast<double>(f);
  uint32_t bits = __float_as_uint(f);
  if (fabs(r) > v * 0x1p-40) {
    if (r < 0) --bits;
    bits |= 1u;
  }
  return to_e4m3(__uint_as_float(bits));
}

// Which way the 16-bit values go that lie next to a border of a block.  The borders are 1, 3, 5
// and 7 units times powers of two, and at most one value of the type is that close to each: all
// ones for up.  A value on the border goes to the even code: up at 3 and 7 units.
struct Ways {
  uint32_t up[4];
  template <int TYPE>
  __device__ __forceinline__ void find(float unit, float unit_low) {
    constexpr int kDrop = TYPE == kBf16 ? 16 : 13;  // fp32 bits below the type's last
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float m = 2 * i + 1;
      const float x = __uint_as_float((__float_as_uint(m * unit) + (1u << (kDrop - 1))) & ~((1u << kDrop) - 1));
      const float d = beyond(x, m, unit, unit_low);
      up[i] = d > 0.0f || (d == 0.0f && (i & 1)) ? 0xFFFFFFFFu : 0;
    }
  }
  // eight codes of which those that differ are next to a border, `low` below it
  __device__ __forceinline__ uint32_t choose(uint32_t low, uint32_t high) const {
    const uint32_t d = low ^ high;
    const uint32_t differ = (d | d >> 1 | d >> 2) & 0x11111111u, odd = low, above = low >> 1 | low >> 2;
    // code 0: 1 unit; 1: 3; 2, 4, 6: 5; 3, 5: 7
    const uint32_t way = (odd & ((above & up[3]) | (~above & up[1]))) | (~odd & ((above & up[2]) | (~above & up[0])));
    return low + (way & differ);
  }
};

// CTAs of the quantisation on an SM, by the registers that a thread's values take.
template <int TYPE>
constexpr int kQuantizeCtas = TYPE == kF32 ? 3 : 4;

// 16 values and the largest of their magnitudes.
template <int TYPE>
struct Values {
  uint32_t raw[TYPE == kF32 ? 16 : 8];

  __device__ __forceinline__ void load(const void* x, size_t at, bool wide) {
    uint32_t(*half)[8] = reinterpret_cast<uint32_t(*)[8]>(raw);
    const uint8_t* p = static_cast<const uint8_t*>(x) + at * (TYPE == kF32 ? 4 : 2);
    load32(p, wide, half[0]);
    if constexpr (TYPE == kF32) load32(p + 32, wide, half[1]);
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (uint32_t& r : raw) r = 0;
  }
  // magnitudes compare as whole numbers; infinities and NaN come out on top
  __device__ __forceinline__ uint32_t amax_bits() const {
    if constexpr (TYPE == kF32) {
      uint32_t m = 0;
#pragma unroll
      for (uint32_t r : raw) m = max(m, r & 0x7FFFFFFFu);
      return m;
    } else {
      uint32_t m = 0;
#pragma unroll
      for (uint32_t r : raw) m = __vmaxu2(m, r & 0x7FFF7FFFu);
      return max(m & 0xFFFFu, m >> 16);
    }
  }
  static __device__ __forceinline__ float as_float(uint32_t bits) {
    if constexpr (TYPE == kF32) return __uint_as_float(bits);
    else return pair_to_f2<TYPE>(bits).x;
  }
  __device__ __forceinline__ void eight(int h, float (&f)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (TYPE == kF32) {
        f[i] = __uint_as_float(raw[8 * h + i]);
      } else {
        const float2 p = pair_to_f2<TYPE>(raw[4 * h + i / 2]);
        f[i] = i & 1 ? p.y : p.x;
      }
    }
  }
};

// Rows of `units` pieces of 32 values (one MXFP4 or two NVFP4 blocks), the last ones past K
// filling the row's last scale tile.
template <int FORMAT, int TYPE>
__global__ void __launch_bounds__(kThreads, kQuantizeCtas<TYPE>) quantize_kernel(
    const void* __restrict__ x, uint8_t* __restrict__ packed, uint8_t* __restrict__ scales,
    const float* __restrict__ tensor_scale, int rows, int units, int K, int tiles, bool wide) {
  grid_dependency_wait();
  grid_dependents_launch();
  const float gamma = FORMAT == kNvfp4 && tensor_scale ? *tensor_scale : 1.0f;
  const bool gamma_bad = !(gamma >= 0.0f && gamma <= 3.402823466e38f);
  // 1 / (6 gamma), or 0 where fp32 does not hold it well, or the errors of gamma's products with
  // the scales' borders (beyond(): from 2^-117)
  const float inv6 = gamma > 0x1p-100f && gamma < 0x1p100f ? 1.0f / (6.0f * gamma) : 0.0f;
  const int lane = threadIdx.x & 31;
  // 16-bit values are loaded a piece ahead; the lanes of a warp, whose pieces are neighbours,
  // go on together while any has one
  constexpr bool kAhead = TYPE != kF32;
  Walk way(static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x, static_cast<long long>(gridDim.x) * kThreads, units);
  const auto fetch = [&](Values<TYPE>(&v)[2]) {
    if (way.row < rows && way.u * 32 < K) {
      const size_t at = static_cast<size_t>(way.row) * K + static_cast<size_t>(way.u) * 32;
      v[0].load(x, at, wide);
      v[1].load(x, at + 16, wide);
    } else {
      v[0].zero();
      v[1].zero();
    }
  };
  Values<TYPE> ahead[2];
  if (kAhead) fetch(ahead);
  while (__any_sync(0xFFFFFFFFu, way.row < rows)) {
    if (!kAhead) fetch(ahead);
    const Values<TYPE> v[2] = {ahead[0], ahead[1]};
    const int row = way.row, u = way.u;
    const bool inside = row < rows && u * 32 < K;
    const size_t at = static_cast<size_t>(row) * K + static_cast<size_t>(u) * 32;
    way.next();
    if (kAhead) fetch(ahead);

    uint32_t code = 0;     // the scales, one byte or two
    uint32_t q[4] = {};    // 32 e2m1 codes
    float f[8];
    constexpr uint32_t kInfinity = TYPE == kF32 ? 0x7F800000u : TYPE == kBf16 ? 0x7F80u : 0x7C00u;
    if constexpr (FORMAT == kMxfp4) {
      const uint32_t top = max(v[0].amax_bits(), v[1].amax_bits());
      if (top < kInfinity) {
        const uint32_t e = __float_as_uint(Values<TYPE>::as_float(top)) >> 23;
        code = e > 2 ? e - 2 : 0;
        const float inv = __uint_as_float((254u - code) << 23);  // 2^(127 - code), exact
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          v[h >> 1].eight(h & 1, f);
#pragma unroll
          for (int i = 0; i < 8; ++i) f[i] *= inv;
          q[h] = to_e2m1x8(f);
        }
      } else {
        code = 0xFF;
      }
    } else {
      // Scales: fp32 quotients are within 2^-21; where that much to either side gives two
      // codes, or fp32 cannot hold them, the exact comparison decides.
      bool bad[2];
      float amax[2];
      uint32_t c[2];
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const uint32_t top = v[b].amax_bits();
        bad[b] = top >= kInfinity || gamma_bad;
        amax[b] = bad[b] ? 0.0f : Values<TYPE>::as_float(top);
        const float v6 = amax[b] * inv6;
        uint32_t both;
        asm("{\n\t.reg .b16 t;\n\tcvt.rn.satfinite.e4m3x2.f32 t, %1, %2;\n\tcvt.u32.u16 %0, t;\n\t}"
            : "=r"(both) : "f"(v6 * (1.0f + 0x1p-20f)), "f"(v6 * (1.0f - 0x1p-20f)));
        c[b] = both & 0xFF;
        if (both >> 8 != c[b]) c[b] = settle_scale(amax[b], gamma, c[b]);
        if (inv6 == 0.0f && gamma > 0.0f) c[b] = scale_of_extreme(amax[b], gamma);
      }
      // Values, likewise.
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const float s = mx4_scale_value<kNvfp4>(c[b]);
        const float unit = s * gamma;
        const bool plain = unit > 0x1p-100f && unit < 0x1p100f, zero = bad[b] || c[b] == 0;
        const float inv = plain && !zero ? __fdividef(1.0f, unit) : 0.0f;
        const float below = inv * (1.0f - 0x1p-20f), above = inv * (1.0f + 0x1p-20f);
        uint32_t low[2], high[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float g[8];
          v[b].eight(h, f);
#pragma unroll
          for (int i = 0; i < 8; ++i) g[i] = f[i] * above;
          high[h] = to_e2m1x8(g);
#pragma unroll
          for (int i = 0; i < 8; ++i) g[i] = f[i] * below;
          low[h] = to_e2m1x8(g);
        }
        if (TYPE != kF32 && low[0] == high[0] && low[1] == high[1] && (plain || zero)) {
          // nothing next to a border
        } else if (TYPE != kF32 && plain) {
          Ways ways;
          ways.find<TYPE>(unit, fmaf(s, gamma, -unit));
          low[0] = ways.choose(low[0], high[0]);
          low[1] = ways.choose(low[1], high[1]);
        } else if (!zero && inside) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t doubt = plain ? low[h] ^ high[h] : 0xFFFFFFFFu;
            if (doubt) low[h] = settle<TYPE>(static_cast<const uint8_t*>(x) + (at + 16 * b + 8 * h) * (TYPE == kF32 ? 4 : 2),
                                             low[h], doubt, s, gamma);
          }
        }
        q[2 * b] = zero ? 0 : low[0];
        q[2 * b + 1] = zero ? 0 : low[1];
        code |= (bad[b] ? 0x7Fu : c[b]) << (8 * b);
      }
    }
    if (inside) *reinterpret_cast<uint4*>(packed + at / 2) = make_uint4(q[0], q[1], q[2], q[3]);

    // the four scales of a tile's row together
    if (!inside) code = 0;
    uint32_t four;
    if constexpr (FORMAT == kMxfp4) {
      four = code << (8 * (lane & 3));
      four |= __shfl_xor_sync(0xFFFFFFFFu, four, 1);
      four |= __shfl_xor_sync(0xFFFFFFFFu, four, 2);
    } else {
      four = code << (16 * (lane & 1));
      four |= __shfl_xor_sync(0xFFFFFFFFu, four, 1);
    }
    constexpr int kPer = FORMAT == kMxfp4 ? 4 : 2;  // threads of a tile's row
    if (row < rows && lane % kPer == 0)
      *reinterpret_cast<uint32_t*>(scales + mx4_scale_at(row, u * (4 / kPer), tiles)) = four;
  }
}

// Rows of K / 32 pieces of 32 values.
template <int FORMAT, int TYPE>
__global__ void __launch_bounds__(kThreads) dequantize_kernel(const uint8_t* __restrict__ packed,
                                                              const uint8_t* __restrict__ scales,
                                                              const float* __restrict__ tensor_scale,
                                                              void* __restrict__ out, int rows, int units, int tiles,
                                                              bool wide) {
  grid_dependency_wait();
  grid_dependents_launch();
  const float gamma = tensor_scale ? *tensor_scale : 1.0f;
  Walk way(static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x, static_cast<long long>(gridDim.x) * kThreads, units);
  for (; way.row < rows; way.next()) {
    const int row = way.row, u = way.u;
    const size_t idx = static_cast<size_t>(row) * units + u;
    const uint4 w = ldg_nc_v4(packed + idx * 16);
    float s[2];
    if constexpr (FORMAT == kMxfp4) {
      s[0] = s[1] = mx4_scale_value<FORMAT>(scales[mx4_scale_at(row, u, tiles)]);
    } else {
      const uint32_t two = *reinterpret_cast<const uint16_t*>(scales + mx4_scale_at(row, 2 * u, tiles));
      s[0] = mx4_scale_value<FORMAT>(two & 0xFF);
      s[1] = mx4_scale_value<FORMAT>(two >> 8);
    }
    const uint32_t words[4] = {w.x, w.y, w.z, w.w};
    uint8_t* o = static_cast<uint8_t*>(out) + idx * 32 * (TYPE == kF32 ? 4 : 2);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t v[TYPE == kF32 ? 16 : 8];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        uint32_t pairs[4];
        e2m1x8_decode<kF16>(words[2 * h + j], pairs);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 q = h2_to_f2(pairs[i]);
          const float lo = __fmul_rn(__fmul_rn(q.x, s[h]), gamma), hi = __fmul_rn(__fmul_rn(q.y, s[h]), gamma);
          if constexpr (TYPE == kF32) {
            v[8 * j + 2 * i] = __float_as_uint(lo);
            v[8 * j + 2 * i + 1] = __float_as_uint(hi);
          } else {
            v[4 * j + i] = f2_to_pair<TYPE>(lo, hi);
          }
        }
      }
      uint32_t(*part)[8] = reinterpret_cast<uint32_t(*)[8]>(v);
      if constexpr (TYPE == kF32) {
        store32(o + 64 * h, wide, part[0]);
        store32(o + 64 * h + 32, wide, part[1]);
      } else {
        store32(o + 32 * h, wide, part[0]);
      }
    }
  }
}

// CTAs for `total` pieces, at most `most` an SM.
unsigned blocks_for(long long total, int most) {
  const long long b = (total + kThreads - 1) / kThreads, cap = static_cast<long long>(kSms) * most;
  return static_cast<unsigned>(b < cap ? b : cap);
}

bool aligned32(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 31) == 0; }

template <int FORMAT, int TYPE>
cudaError_t quantize_as(const void* x, uint8_t* packed, uint8_t* scales, const float* tensor_scale, int rows, int K,
                        cudaStream_t stream) {
  const int tiles = mx4_scale_tiles(K, FORMAT);
  const int units = tiles * 4 * mx4_block(FORMAT) / 32;
  const long long total = static_cast<long long>(rows) * units;
  return launch_overlapped(quantize_kernel<FORMAT, TYPE>, blocks_for(total, kQuantizeCtas<TYPE>), kThreads, 0, stream, 1,
                           x, packed, scales, tensor_scale, rows, units, K, tiles, aligned32(x));
}

template <int FORMAT, int TYPE>
cudaError_t dequantize_as(const Mx4& t, void* out, int K, cudaStream_t stream) {
  const int units = K / 32;
  const long long total = static_cast<long long>(t.rows) * units;
  return launch_overlapped(dequantize_kernel<FORMAT, TYPE>, blocks_for(total, 64), kThreads, 0, stream, 1, t.packed,
                           t.scales, t.tensor_scale, out, t.rows, units, mx4_scale_tiles(K, FORMAT), aligned32(out));
}

}  // namespace

cudaError_t launch_mx4_quantize(const void* x, int x_type, uint8_t* packed, uint8_t* scales,
                                const float* tensor_scale, int rows, int K, int format, cudaStream_t stream) {
#define MX4_CASE(f, t) \
  if (format == f && x_type == t) return quantize_as<f, t>(x, packed, scales, tensor_scale, rows, K, stream);
  MX4_CASE(kMxfp4, kF16) MX4_CASE(kMxfp4, kBf16) MX4_CASE(kMxfp4, kF32)
  MX4_CASE(kNvfp4, kF16) MX4_CASE(kNvfp4, kBf16) MX4_CASE(kNvfp4, kF32)
#undef MX4_CASE
  return cudaErrorInvalidValue;
}

cudaError_t launch_mx4_dequantize(const Mx4& t, void* out, int out_type, int K, int format, cudaStream_t stream) {
#define MX4_CASE(f, ty) \
  if (format == f && out_type == ty) return dequantize_as<f, ty>(t, out, K, stream);
  MX4_CASE(kMxfp4, kF16) MX4_CASE(kMxfp4, kBf16) MX4_CASE(kMxfp4, kF32)
  MX4_CASE(kNvfp4, kF16) MX4_CASE(kNvfp4, kBf16) MX4_CASE(kNvfp4, kF32)
#undef MX4_CASE
  return cudaErrorInvalidValue;
}

}  // namespace aqlm
