// Device helpers of the MXFP4 kernels (gfx950 / CDNA4 only).
//
// A block is 32 consecutive values of a row: one scale byte e (the factor 2^(e - 127), 255 is
// NaN) and 32 codes of 4 bits (sign, two exponent bits, one mantissa bit), two per byte with the
// lower index in the low half, so a block's codes are 16 bytes: one lane's load.
//
// Operand layouts of the scaled MFMA with 4-bit operands (checked on the MI355X with an in-bounds
// probe); D is as in the bf16 shape of the same rows and columns:
//   32x32x64:   lane l holds row (column) l % 32, k = 32 (l / 32) .. + 31 in four registers
//   16x16x128:  lane l holds row (column) l % 16, k = 32 (l / 16) .. + 31
// so a lane's operand is exactly one block, and byte `sel` of its scale register is that block's e.
// The converters with a scale operand use only the exponent field of the fp32 scale, the e of the
// format: e << 23 as a float decodes every block exactly (e = 255 to NaN; a value of 2^128 or more,
// which e = 253 and 254 can give, to an infinity of its sign in bf16) and encodes with round to nearest even, saturating at 6 (all borders, both
// signs and scales 0 to 254 checked on the MI355X).
#pragma once

#include "device_common.h"

namespace w4a16 {

typedef int i32x8_t __attribute__((ext_vector_type(8)));

constexpr uint32_t kOutside = 0x80000000u;   // a buffer offset that no resource here reaches: loads give 0

// A buffer over `bytes` from base, cut at 2 GiB (offsets inside a tile stay below that).
__device__ __forceinline__ __amdgpu_buffer_rsrc_t mx_resource(const void* base, int64_t bytes) {
    const int64_t n = bytes < 0 ? 0 : (bytes > 0x7FFFFFFFll ? 0x7FFFFFFFll : bytes);
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, static_cast<int>(n), 0x00020000);
}

__device__ __forceinline__ float mx_scale(uint32_t e) { return __uint_as_float(e << 23); }

// Eight codes of one word as bf16, in order (four instructions).
__device__ __forceinline__ u32x4_t mx_decode_word(uint32_t w, float scale) {
    u32x4_t r;
    r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0));
    r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1));
    r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2));
    r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3));
    return r;
}

__device__ __forceinline__ i32x8_t mx_operand(const u32x4_t& v) {
    return i32x8_t{static_cast<int>(v[0]), static_cast<int>(v[1]), static_cast<int>(v[2]), static_cast<int>(v[3]),
                   0, 0, 0, 0};
}

// acc += A . B^T over one block per lane, the scales in byte SEL of sa and sb (4 = the 4-bit format).
template <int SEL>
__device__ __forceinline__ f32x16_t mx_mfma32(const u32x4_t& a, uint32_t sa, const u32x4_t& b, uint32_t sb,
                                              const f32x16_t& c) {
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(mx_operand(a), mx_operand(b), c, 4, 4, SEL,
                                                           static_cast<int>(sa), SEL, static_cast<int>(sb));
}

// Two fp32 as packed bf16 (each rounded to nearest even).
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const bf16x2_t v = {static_cast<__bf16>(lo), static_cast<__bf16>(hi)};
    return __builtin_bit_cast(uint32_t, v);
}

// 1 / (1 + 2^(-z log2 e)) from the hardware's exponential and reciprocal, each within a step of fp32.
// The exponent is off by the constant's rounding (0.23 2^-24 of it) and the product's (2^-24), which
// makes 1.23 |z| 2^-24 of the result: (4 + |z|) 2^-23 covers all of it.  2^large is infinite and its
// reciprocal 0, the limit; from z = -87.3 down the hardware's reciprocal flushes a result under 2^-126
// to 0, an error below 2^-126.
__device__ __forceinline__ float mx_sigmoid(float z) {
    return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(z * -1.44269504088896341f));
}

// Orders a wave's LDS writes before its own lanes' later reads (no other wave takes part).
__device__ __forceinline__ void wave_lds_fence() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

}  // namespace w4a16
