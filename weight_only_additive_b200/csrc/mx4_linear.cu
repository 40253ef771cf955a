// Products with a 4-bit weight matrix: 64 x 64 output tiles, both operands decoded to
// fp32 in shared memory, 4 x 4 outputs a thread.
#include "mx4_device.cuh"

namespace aqlm {
namespace {

constexpr int kTile = 64, kStep = 32;

// Value (r, k) of a 4-bit tensor, its tensor scale left out.
template <int FORMAT>
__device__ __forceinline__ float mx4_value(const Mx4& t, int r, int k, int K, int tiles) {
  const uint32_t byte = t.packed[static_cast<size_t>(r) * (K / 2) + k / 2];
  uint32_t h[4];
  e2m1x8_to_f16(byte >> ((k & 1) * 4), h);
  return h2_to_f2(h[0]).x * mx4_scale_value<FORMAT>(t.scales[mx4_scale_at(r, k / mx4_block(FORMAT), tiles)]);
}

// out[i][j] = sum_k a(i, k) b(j, k): a from 16-bit rows (A_TYPE) or a 4-bit tensor (-1),
// b the weight (GRAD: its transpose).
template <int FORMAT, int A_TYPE, int OUT_TYPE, bool GRAD>
__global__ void __launch_bounds__(256) product_kernel(const void* a16, Mx4 a4, Mx4 w, const void* bias, void* out,
                                                      int rows, int cols, int depth, int K) {
  __shared__ float As[kStep][kTile + 1], Bs[kStep][kTile + 1];
  grid_dependency_wait();
  grid_dependents_launch();
  const int tiles = (K / mx4_block(FORMAT) + 3) / 4;
  const int i0 = blockIdx.y * kTile, j0 = blockIdx.x * kTile, tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  float acc[4][4] = {};
  for (int k0 = 0; k0 < depth; k0 += kStep) {
    for (int e = threadIdx.x; e < kTile * kStep; e += 256) {
      const int i = e / kStep, k = e % kStep;
      float v = 0.0f;
      if (i0 + i < rows && k0 + k < depth) {
        if constexpr (A_TYPE >= 0) v = load_value<A_TYPE>(a16, static_cast<size_t>(i0 + i) * depth + k0 + k);
        else v = mx4_value<FORMAT>(a4, i0 + i, k0 + k, K, tiles);
      }
      As[k][i] = v;
    }
    for (int e = threadIdx.x; e < kTile * kStep; e += 256) {
      const int j = GRAD ? e % kTile : e / kStep, k = GRAD ? e / kTile : e % kStep;
      float v = 0.0f;
      if (j0 + j < cols && k0 + k < depth)
        v = GRAD ? mx4_value<FORMAT>(w, k0 + k, j0 + j, K, tiles) : mx4_value<FORMAT>(w, j0 + j, k0 + k, K, tiles);
      Bs[k][j] = v;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kStep; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] += As[k][ty * 4 + i] * Bs[k][tx + 16 * j];
    __syncthreads();
  }
  float scale = w.tensor_scale ? *w.tensor_scale : 1.0f;
  if (A_TYPE < 0 && a4.tensor_scale) scale *= *a4.tensor_scale;
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int r = i0 + ty * 4 + i, c = j0 + tx + 16 * j;
      if (r >= rows || c >= cols) continue;
      const float b = bias ? load_value<OUT_TYPE>(bias, c) : 0.0f;
      store_value<OUT_TYPE>(out, static_cast<size_t>(r) * cols + c, acc[i][j] * scale + b);
    }
}

template <int FORMAT, int A_TYPE, int OUT_TYPE, bool GRAD>
cudaError_t product(const void* a16, const Mx4& a4, const Mx4& w, const void* bias, void* out, int rows, int cols,
                    int depth, int K, cudaStream_t stream) {
  const dim3 grid((cols + kTile - 1) / kTile, (rows + kTile - 1) / kTile);
  return launch_overlapped(product_kernel<FORMAT, A_TYPE, OUT_TYPE, GRAD>, grid, 256, 0, stream, 1, a16, a4, w, bias,
                           out, rows, cols, depth, K);
}

}  // namespace

cudaError_t launch_mx4_linear(const Mx4Linear& p, uint32_t*, cudaStream_t stream) {
#define MX4_CASE(f, t) \
  if (p.format == f && p.type == t) \
    return product<f, t, t, false>(p.x, Mx4{}, p.w, p.bias, p.y, p.batch, p.w.rows, p.K, p.K, stream);
  MX4_CASE(kMxfp4, kF16) MX4_CASE(kMxfp4, kBf16) MX4_CASE(kNvfp4, kF16) MX4_CASE(kNvfp4, kBf16)
#undef MX4_CASE
  return cudaErrorInvalidValue;
}

cudaError_t launch_mx4_grad(const Mx4Grad& p, uint32_t*, cudaStream_t stream) {
#define MX4_CASE(f, t) \
  if (p.format == f && p.type == t) \
    return product<f, t, t, true>(p.dy, Mx4{}, p.w, nullptr, p.dx, p.batch, p.K, p.w.rows, p.K, stream);
  MX4_CASE(kMxfp4, kF16) MX4_CASE(kMxfp4, kBf16) MX4_CASE(kNvfp4, kF16) MX4_CASE(kNvfp4, kBf16)
#undef MX4_CASE
  return cudaErrorInvalidValue;
}

}  // namespace aqlm
