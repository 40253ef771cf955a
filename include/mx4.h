/*
 * mx4.h -- microscaled 4-bit floating point (MXFP4, NVFP4) in libaqlm.so, beside the
 * AQLM layer of aqlm.h: quantisation, dequantisation, the linear layer with 4-bit
 * weights and 16-bit or 4-bit activations, and its input gradient (B200, sm_100a).
 *
 * A 4-bit tensor of `rows` x `K` values is (packed, scales, tensor_scale):
 *   packed  uint8 [rows, K/2]: two e2m1 values a byte, even k in the low four bits.
 *           An e2m1 code is sign (bit 3) and magnitude 0, 0.5, 1, 1.5, 2, 3, 4, 6 (bits 0-2).
 *   scales  uint8, one per block of consecutive k in a row, in tiles of 128 rows x 4
 *           blocks, 512 bytes a tile, tiles row-major [ceil(rows/128)][ceil(K/block/4)]:
 *           block c of row r is byte (r % 32) * 16 + (r % 128) / 32 * 4 + c % 4 of tile
 *           (r / 128, c / 4) -- the order in which the tensor cores take scales.
 *           The blocks after K/block in the last tile of a row hold 0 (they are read, and
 *           not checked); rows after the last one may hold anything.
 *     MX4_MXFP4  block 32, e8m0: code c is 2^(c - 127), 255 is NaN
 *     MX4_NVFP4  block 16, e4m3 (no sign): 0x7F is NaN
 *   tensor_scale  one fp32 on the device, or NULL for 1
 * The value of element (r, k) is e2m1 * block scale * tensor_scale.
 *
 * Sizes: K a positive multiple of 32, at most 2^20; rows, N, batch in 1 .. 2^24, in any
 * multiple.  A value whose magnitude leaves the range of fp32 (e8m0 codes above 252) is
 * not supported.  Every pointer is caller-owned DEVICE memory, 16-byte aligned
 * (tensor_scale: 4-byte), row-major and dense; outputs must not overlap inputs.
 * Status codes, streams, graph capture, ownership and errors are those of aqlm.h, with
 * one difference: a call reads all its inputs, the weights too, only after the kernel
 * before it on the stream has completed, so a tensor may be used right after the call
 * that quantises it.
 */
#ifndef MX4_H_
#define MX4_H_

#include "aqlm.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { MX4_MXFP4 = 0, MX4_NVFP4 = 1 } mx4_format;
typedef enum { MX4_F16 = 0, MX4_BF16 = 1, MX4_F32 = 2 } mx4_type;

/* Bytes of the tiled scales of a rows x K tensor; 0 for invalid arguments.  Host logic. */
size_t mx4_scales_bytes(long long rows, long long K, mx4_format format);

/*
 * Quantises x [rows, K] (fp16, bf16 or fp32).  With amax the block's largest magnitude:
 *   MXFP4  scale = 2^max(floor(log2 amax) - 2, -127)
 *   NVFP4  scale = e4m3(amax / (6 tensor_scale)), at most 448
 *   code   = e2m1(x / (scale * tensor_scale)), magnitudes above 6 becoming 6
 * where e4m3() and e2m1() round the exact quotient to the nearest value, ties to the even
 * code.  A block of zeros, or one whose e4m3 scale rounds to 0, becomes zeros (MXFP4:
 * scale 2^-127).  A block that holds an infinity or a NaN gets the NaN scale and zero
 * codes: its values read back as NaN.  The same holds for every NVFP4 block if
 * tensor_scale is negative or not finite; if it is 0 every block becomes zeros.
 * tensor_scale is read by NVFP4 alone; MXFP4 takes NULL (else AQLM_ERR_INVALID_ARG).
 *   packed, scales  written; scales of mx4_scales_bytes() bytes.  The bytes of rows after
 *                   the last one are left as they were.
 */
aqlm_status mx4_quantize(const void* x, mx4_type x_type, void* packed, void* scales, const void* tensor_scale,
                         long long rows, long long K, mx4_format format, aqlm_stream_t stream);

/* out [rows, K] (fp16, bf16 or fp32): (e2m1 * block scale) * tensor_scale in fp32, rounded
 * once more (to nearest even) for the 16-bit types. */
aqlm_status mx4_dequantize(const void* packed, const void* scales, const void* tensor_scale, void* out,
                           mx4_type out_type, long long rows, long long K, mx4_format format,
                           aqlm_stream_t stream);

/*
 * y [batch, N] = x . W^T + bias with x [batch, K] in fp16 or bf16 (`type`, also that of
 * y and bias) and W a 4-bit N x K tensor.  The weights are taken exactly; sums in fp32,
 * the tensor scale and the bias in fp32 at the end, one rounding.  bias may be NULL.
 *   workspace  device memory of mx4_matmul_workspace_size() bytes (NULL if 0), 16-byte
 *              aligned, of any contents, not shared by calls that may run at once.
 */
size_t mx4_matmul_workspace_size(mx4_type type, long long N, long long K, long long batch, mx4_format format);
aqlm_status mx4_matmul(const void* x, mx4_type type, const void* w_packed, const void* w_scales,
                       const void* w_tensor_scale, const void* bias, void* y, long long N, long long K,
                       long long batch, mx4_format format, void* workspace, size_t workspace_bytes,
                       aqlm_stream_t stream);

/*
 * The same product of two 4-bit tensors of one format, x batch x K and W N x K, on the
 * block-scaled tensor-core path: products of the 4-bit values and block scales are exact,
 * sums in fp32, then both tensor scales and the bias in fp32, one rounding to y_type
 * (fp16, bf16 or fp32, also bias's type).
 */
aqlm_status mx4_matmul_mx4(const void* x_packed, const void* x_scales, const void* x_tensor_scale,
                           const void* w_packed, const void* w_scales, const void* w_tensor_scale,
                           const void* bias, void* y, mx4_type y_type, long long N, long long K, long long batch,
                           mx4_format format, aqlm_stream_t stream);

/*
 * Input gradient of mx4_matmul for frozen weights: dx [batch, K] = dy [batch, N] . W,
 * dy and dx fp16 or bf16 (`type`).  The weights are taken exactly, sums in fp32, the
 * tensor scale in fp32 at the end, one rounding.  workspace as for mx4_matmul.
 */
size_t mx4_input_grad_workspace_size(mx4_type type, long long N, long long K, long long batch, mx4_format format);
aqlm_status mx4_input_grad(const void* dy, mx4_type type, const void* w_packed, const void* w_scales,
                           const void* w_tensor_scale, void* dx, long long N, long long K, long long batch,
                           mx4_format format, void* workspace, size_t workspace_bytes, aqlm_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MX4_H_ */
