// MXFP4 operands as the kernels see them (layout: fp4.cu), shared by the
// quantization, the product and the expert layer.
#pragma once

#include "bi_internal.h"

namespace bi {

// Contraction length of the codes' rows: a multiple of 256.
__host__ __device__ __forceinline__ int64_t fp4_padded(int64_t c) { return (c + 255) / 256 * 256; }

// Byte of the scale of row r, block b (32 values) of an operand padded to Cp.
__host__ __device__ __forceinline__ int64_t fp4_scale_at(int64_t r, int64_t b, int64_t Cp) {
    return ((r >> 7) * (Cp >> 7) + (b >> 2)) * 512 + (r & 31) * 16 + ((r >> 5) & 3) * 4 + (b & 3);
}

#ifdef __CUDACC__
// 2^(byte - 127); byte 255 is NaN, byte 0 the subnormal 2^-127.
__device__ __forceinline__ float fp4_scale_value(uint32_t byte) {
    return __uint_as_float(byte == 255u ? 0x7fc00000u : byte == 0u ? 0x00400000u : byte << 23);
}
// The value of a code 0..15: sign, two exponent bits, one mantissa bit.
__device__ __forceinline__ float fp4_code_value(uint32_t code) {
    // the three magnitude bits at an f32's exponent and first mantissa bit are the
    // value * 2^-126 (0 and 0.5 being its zero and subnormal, as in e2m1)
    return __uint_as_float(((code & 8u) << 28) | ((code & 7u) << 22)) * 8.507059173023462e37f;  // * 2^126, exact
}
#endif

// out [rows][cols] (out_dt) = a [rows][depth] * b [cols][depth]^T (+ bias [cols]),
// both in MXFP4 along depth; f32 results over more than TC_PIECE_ROWS depth in
// pieces added in order (fp4_tc.cu).
cudaError_t tc_fp4_product(const LaunchCtx& c, bi_dtype out_dt, void* out, const uint8_t* a, const uint8_t* as, const uint8_t* b,
                           const uint8_t* bs, const void* bias, int64_t rows, int64_t cols, int64_t depth);

}  // namespace bi
