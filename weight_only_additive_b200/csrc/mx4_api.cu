// C ABI of the microscaled 4-bit operators: argument checks and dispatch.  The contract
// lives in include/mx4.h.
#include <cuda_runtime.h>

#include "mx4.h"
#include "mx4_internal.h"

namespace {

constexpr long long kMaxRows = 1ll << 24, kMaxK = 1ll << 20;

struct Range {
  const void* p;
  size_t bytes;
};

bool apart(const Range& a, const Range& b) {
  if (!a.p || !b.p) return true;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x + a.bytes <= y || y + b.bytes <= x;
}

bool aligned(const void* p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

bool format_ok(mx4_format f) { return f == MX4_MXFP4 || f == MX4_NVFP4; }
bool rows_ok(long long rows) { return rows >= 1 && rows <= kMaxRows; }
bool K_ok(long long K) { return K >= 32 && K <= kMaxK && K % 32 == 0; }
size_t type_bytes(mx4_type t) { return t == MX4_F32 ? 4 : 2; }
bool type16(mx4_type t) { return t == MX4_F16 || t == MX4_BF16; }
bool type_any(mx4_type t) { return type16(t) || t == MX4_F32; }

// A 4-bit operand of a call.
aqlm_status check_tensor(const void* packed, const void* scales, const void* tensor_scale) {
  if (!packed || !scales) return AQLM_ERR_INVALID_ARG;
  if (!aligned(packed, 16) || !aligned(scales, 16) || !aligned(tensor_scale, 4)) return AQLM_ERR_MISALIGNED;
  return AQLM_OK;
}

// The call writes `out` and reads the others; the workspace is written too.
aqlm_status check_apart(const Range& out, const Range& workspace, const Range* in, int count) {
  if (!apart(out, workspace)) return AQLM_ERR_INVALID_ARG;
  for (int i = 0; i < count; ++i)
    if (!apart(out, in[i]) || !apart(workspace, in[i])) return AQLM_ERR_INVALID_ARG;
  return AQLM_OK;
}

aqlm_status check_workspace(const void* ws, size_t bytes, size_t need) {
  if (need == 0) return AQLM_OK;
  if (!ws || bytes < need) return AQLM_ERR_INVALID_ARG;
  return aligned(ws, 16) ? AQLM_OK : AQLM_ERR_MISALIGNED;
}

aqlm_status as_status(cudaError_t e) { return static_cast<aqlm_status>(aqlm::status_of(e)); }

aqlm::Mx4 tensor(const void* packed, const void* scales, const void* tensor_scale, long long rows) {
  return aqlm::Mx4{static_cast<const uint8_t*>(packed), static_cast<const uint8_t*>(scales),
                   static_cast<const float*>(tensor_scale), static_cast<int>(rows)};
}

size_t scales_size(long long rows, long long K, mx4_format format) {
  return static_cast<size_t>((rows + 127) / 128) * aqlm::mx4_scale_tiles(static_cast<int>(K), format) * 512;
}
size_t packed_size(long long rows, long long K) { return static_cast<size_t>(rows) * K / 2; }

}  // namespace

extern "C" {

size_t mx4_scales_bytes(long long rows, long long K, mx4_format format) {
  return rows_ok(rows) && K_ok(K) && format_ok(format) ? scales_size(rows, K, format) : 0;
}

aqlm_status mx4_quantize(const void* x, mx4_type x_type, void* packed, void* scales, const void* tensor_scale,
                         long long rows, long long K, mx4_format format, aqlm_stream_t stream) {
  if (!x || !rows_ok(rows) || !K_ok(K) || !format_ok(format) || !type_any(x_type)) return AQLM_ERR_INVALID_ARG;
  if (format == MX4_MXFP4 && tensor_scale) return AQLM_ERR_INVALID_ARG;
  aqlm_status st = check_tensor(packed, scales, tensor_scale);
  if (st != AQLM_OK) return st;
  if (!aligned(x, 16)) return AQLM_ERR_MISALIGNED;
  const Range xr{x, static_cast<size_t>(rows) * K * type_bytes(x_type)};
  const Range in[] = {xr, {tensor_scale, 4}};
  st = check_apart(Range{packed, packed_size(rows, K)}, Range{scales, scales_size(rows, K, format)}, in, 2);
  if (st != AQLM_OK) return st;
  return as_status(aqlm::launch_mx4_quantize(x, x_type, static_cast<uint8_t*>(packed), static_cast<uint8_t*>(scales),
                                             static_cast<const float*>(tensor_scale), static_cast<int>(rows),
                                             static_cast<int>(K), format, reinterpret_cast<cudaStream_t>(stream)));
}

aqlm_status mx4_dequantize(const void* packed, const void* scales, const void* tensor_scale, void* out,
                           mx4_type out_type, long long rows, long long K, mx4_format format,
                           aqlm_stream_t stream) {
  if (!out || !rows_ok(rows) || !K_ok(K) || !format_ok(format) || !type_any(out_type)) return AQLM_ERR_INVALID_ARG;
  aqlm_status st = check_tensor(packed, scales, tensor_scale);
  if (st != AQLM_OK) return st;
  if (!aligned(out, 16)) return AQLM_ERR_MISALIGNED;
  const Range in[] = {{packed, packed_size(rows, K)}, {scales, scales_size(rows, K, format)}, {tensor_scale, 4}};
  st = check_apart(Range{out, static_cast<size_t>(rows) * K * type_bytes(out_type)}, Range{nullptr, 0}, in, 3);
  if (st != AQLM_OK) return st;
  return as_status(aqlm::launch_mx4_dequantize(tensor(packed, scales, tensor_scale, rows), out, out_type,
                                               static_cast<int>(K), format, reinterpret_cast<cudaStream_t>(stream)));
}

size_t mx4_matmul_workspace_size(mx4_type type, long long N, long long K, long long batch, mx4_format format) {
  if (!rows_ok(N) || !rows_ok(batch) || !K_ok(K) || !format_ok(format) || !type16(type)) return 0;
  return aqlm::mx4_linear_workspace(type, format, K, batch);
}

aqlm_status mx4_matmul(const void* x, mx4_type type, const void* w_packed, const void* w_scales,
                       const void* w_tensor_scale, const void* bias, void* y, long long N, long long K,
                       long long batch, mx4_format format, void* workspace, size_t workspace_bytes,
                       aqlm_stream_t stream) {
  if (!x || !y || !rows_ok(N) || !rows_ok(batch) || !K_ok(K) || !format_ok(format) || !type16(type))
    return AQLM_ERR_INVALID_ARG;
  aqlm_status st = check_tensor(w_packed, w_scales, w_tensor_scale);
  if (st != AQLM_OK) return st;
  if (!aligned(x, 16) || !aligned(y, 16) || !aligned(bias, 16)) return AQLM_ERR_MISALIGNED;
  const size_t need = mx4_matmul_workspace_size(type, N, K, batch, format);
  st = check_workspace(workspace, workspace_bytes, need);
  if (st != AQLM_OK) return st;
  const Range in[] = {{x, static_cast<size_t>(batch) * K * 2}, {w_packed, packed_size(N, K)},
                      {w_scales, scales_size(N, K, format)}, {w_tensor_scale, 4},
                      {bias, static_cast<size_t>(N) * 2}};
  st = check_apart(Range{y, static_cast<size_t>(batch) * N * 2}, Range{need ? workspace : nullptr, need}, in, 5);
  if (st != AQLM_OK) return st;
  uint32_t* status = aqlm::status_word();
  if (!status) return as_status(cudaErrorInvalidDevice);
  const aqlm::Mx4Linear p{x, tensor(w_packed, w_scales, w_tensor_scale, N), bias, y, type,
                          static_cast<int>(K), static_cast<int>(batch), format, workspace};
  return as_status(aqlm::launch_mx4_linear(p, status, reinterpret_cast<cudaStream_t>(stream)));
}

aqlm_status mx4_matmul_mx4(const void* x_packed, const void* x_scales, const void* x_tensor_scale,
                           const void* w_packed, const void* w_scales, const void* w_tensor_scale,
                           const void* bias, void* y, mx4_type y_type, long long N, long long K, long long batch,
                           mx4_format format, aqlm_stream_t stream) {
  if (!y || !rows_ok(N) || !rows_ok(batch) || !K_ok(K) || !format_ok(format) || !type_any(y_type))
    return AQLM_ERR_INVALID_ARG;
  aqlm_status st = check_tensor(x_packed, x_scales, x_tensor_scale);
  if (st == AQLM_OK) st = check_tensor(w_packed, w_scales, w_tensor_scale);
  if (st != AQLM_OK) return st;
  if (!aligned(y, 16) || !aligned(bias, 16)) return AQLM_ERR_MISALIGNED;
  const Range in[] = {{x_packed, packed_size(batch, K)}, {x_scales, scales_size(batch, K, format)},
                      {x_tensor_scale, 4}, {w_packed, packed_size(N, K)}, {w_scales, scales_size(N, K, format)},
                      {w_tensor_scale, 4}, {bias, static_cast<size_t>(N) * type_bytes(y_type)}};
  st = check_apart(Range{y, static_cast<size_t>(batch) * N * type_bytes(y_type)}, Range{nullptr, 0}, in, 7);
  if (st != AQLM_OK) return st;
  uint32_t* status = aqlm::status_word();
  if (!status) return as_status(cudaErrorInvalidDevice);
  const aqlm::Mx4Product p{tensor(x_packed, x_scales, x_tensor_scale, batch),
                           tensor(w_packed, w_scales, w_tensor_scale, N), bias, y, y_type, static_cast<int>(K),
                           format};
  return as_status(aqlm::launch_mx4_product(p, status, reinterpret_cast<cudaStream_t>(stream)));
}

size_t mx4_input_grad_workspace_size(mx4_type type, long long N, long long K, long long batch, mx4_format format) {
  if (!rows_ok(N) || !rows_ok(batch) || !K_ok(K) || !format_ok(format) || !type16(type)) return 0;
  return aqlm::mx4_grad_workspace(type, format, N, batch);
}

aqlm_status mx4_input_grad(const void* dy, mx4_type type, const void* w_packed, const void* w_scales,
                           const void* w_tensor_scale, void* dx, long long N, long long K, long long batch,
                           mx4_format format, void* workspace, size_t workspace_bytes, aqlm_stream_t stream) {
  if (!dy || !dx || !rows_ok(N) || !rows_ok(batch) || !K_ok(K) || !format_ok(format) || !type16(type))
    return AQLM_ERR_INVALID_ARG;
  aqlm_status st = check_tensor(w_packed, w_scales, w_tensor_scale);
  if (st != AQLM_OK) return st;
  if (!aligned(dy, 16) || !aligned(dx, 16)) return AQLM_ERR_MISALIGNED;
  const size_t need = mx4_input_grad_workspace_size(type, N, K, batch, format);
  st = check_workspace(workspace, workspace_bytes, need);
  if (st != AQLM_OK) return st;
  const Range in[] = {{dy, static_cast<size_t>(batch) * N * 2}, {w_packed, packed_size(N, K)},
                      {w_scales, scales_size(N, K, format)}, {w_tensor_scale, 4}};
  st = check_apart(Range{dx, static_cast<size_t>(batch) * K * 2}, Range{need ? workspace : nullptr, need}, in, 4);
  if (st != AQLM_OK) return st;
  uint32_t* status = aqlm::status_word();
  if (!status) return as_status(cudaErrorInvalidDevice);
  const aqlm::Mx4Grad p{dy, tensor(w_packed, w_scales, w_tensor_scale, N), dx, type, static_cast<int>(K),
                        static_cast<int>(batch), format, workspace};
  return as_status(aqlm::launch_mx4_grad(p, status, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
