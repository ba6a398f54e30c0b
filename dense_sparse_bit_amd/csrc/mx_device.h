// Device helpers of the microscaled 4-bit operators.
#pragma once

#include <hip/hip_bf16.h>
#include <hip/hip_fp16.h>
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/mq.h"

namespace mq {

typedef int mx_i4 __attribute__((ext_vector_type(4)));
typedef int mx_i8 __attribute__((ext_vector_type(8)));
typedef float mx_f4 __attribute__((ext_vector_type(4)));
typedef float mx_f16 __attribute__((ext_vector_type(16)));

template <int DT> struct MxType;
template <> struct MxType<MQ_F32> { using type = float; };
template <> struct MxType<MQ_BF16> { using type = __bf16; };
template <> struct MxType<MQ_F16> { using type = _Float16; };

// Scale byte of a block whose largest magnitude has the fp32 bits `peak`:
// X = 2^(byte - 127) = 2^(floor(log2(peak)) - 2), at least 2^-127. The exponent field
// of `peak` is floor(log2) + 127 (0 for subnormals, whose X is the least anyway). A
// block with an infinity or a NaN has byte 255, the format's NaN: all of it reads back
// as NaN, so the fault is seen in the product instead of being clamped away.
__device__ inline int mx_scale_byte(uint32_t peak) {
    const int e = static_cast<int>(peak >> 23);
    return e == 255 ? 255 : (e > 2 ? e - 2 : 0);
}

// Two values to two 4-bit codes in byte `SEL` of `old`: v * 2^shift rounded to the
// nearest code, ties to even, magnitudes above 6 to 6. The scaling is exact (a power
// of two; a result below the normal range rounds to code 0 either way).
template <int SEL>
__device__ inline uint32_t mx_codes2(uint32_t old, float a, float b, int shift) {
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(old, ldexpf(a, shift), ldexpf(b, shift), 1.0f, SEL);
}

// Eight values of one block to a word of codes (first value in the low nibble); zero
// codes for a block with byte 255.
__device__ inline uint32_t mx_codes8(const float (&v)[8], int byte) {
    if (byte == 255) return 0;
    const int shift = 127 - byte;
    uint32_t w = mx_codes2<0>(0, v[0], v[1], shift);
    w = mx_codes2<1>(w, v[2], v[3], shift);
    w = mx_codes2<2>(w, v[4], v[5], shift);
    return mx_codes2<3>(w, v[6], v[7], shift);
}

// value of a 4-bit code: 0, 0.5, 1, 1.5, 2, 3, 4, 6 with the sign in bit 3
__device__ inline float mx_code_value(uint32_t c) {
    const uint32_t m = c & 7;
    const float v = m < 4 ? 0.5f * m : (m < 6 ? m - 2.0f : 2.0f * m - 8.0f);
    return c & 8 ? -v : v;
}

template <typename T>
__device__ inline T mx_round(float v) { return static_cast<T>(v); }

}  // namespace mq
