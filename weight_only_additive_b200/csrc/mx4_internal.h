// Internal interface between the mx4 entry points (mx4_api.cu) and their kernels.
// Host code only calls these after the checks of mx4_api.cu have passed.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "aqlm_internal.h"

namespace aqlm {

// Values of mx4_format and mx4_type (include/mx4.h).
enum : int { kMxfp4 = 0, kNvfp4 = 1 };
enum : int { kF16 = 0, kBf16 = 1, kF32 = 2 };

constexpr int mx4_block(int format) { return format == kMxfp4 ? 32 : 16; }
// 512-byte scale tiles along K: each holds 4 blocks of 128 rows.
inline int mx4_scale_tiles(int K, int format) { return (K / mx4_block(format) + 3) / 4; }

// A 4-bit tensor in device memory.
struct Mx4 {
  const uint8_t* packed;
  const uint8_t* scales;
  const float* tensor_scale;  // or null
  int rows;
};

cudaError_t launch_mx4_quantize(const void* x, int x_type, uint8_t* packed, uint8_t* scales,
                                const float* tensor_scale, int rows, int K, int format, cudaStream_t stream);
cudaError_t launch_mx4_dequantize(const Mx4& t, void* out, int out_type, int K, int format, cudaStream_t stream);

// y = x . W^T with x in 16 bits.
struct Mx4Linear {
  const void* x;
  Mx4 w;
  const void* bias;  // or null
  void* y;
  int type;  // of x, bias and y
  int K, batch, format;
  void* workspace;
};
cudaError_t launch_mx4_linear(const Mx4Linear& p, uint32_t* status, cudaStream_t stream);
// The kernel for a few tokens, and whether a batch is one for it.
bool mx4_gemv_takes(int batch);
cudaError_t launch_mx4_gemv(const Mx4Linear& p, uint32_t* status, cudaStream_t stream);
size_t mx4_linear_workspace(int type, int format, long long K, long long batch);

// y = x . W^T with both operands in 4 bits.
struct Mx4Product {
  Mx4 x, w;
  const void* bias;  // or null
  void* y;
  int y_type;
  int K, format;
};
cudaError_t launch_mx4_product(const Mx4Product& p, uint32_t* status, cudaStream_t stream);

// dx = dy . W
struct Mx4Grad {
  const void* dy;
  Mx4 w;
  void* dx;
  int type;
  int K, batch, format;
  void* workspace;
};
cudaError_t launch_mx4_grad(const Mx4Grad& p, uint32_t* status, cudaStream_t stream);
size_t mx4_grad_workspace(int type, int format, long long N, long long batch);

// Device address of the library's status word on the current device (null on failure).
uint32_t* status_word();
// The status of a launch result; a CUDA error is recorded for aqlm_last_cuda_error.
int status_of(cudaError_t e);

}  // namespace aqlm
