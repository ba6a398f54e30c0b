// Device helpers of the microscaled 4-bit operators.
#pragma once

#include <hip/hip_bf16.h>
#include <hip/hip_fp16.h>
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/mq.h"

namespace mq {

typedef int mx_i2 __attribute__((ext_vector_type(2)));
typedef int mx_i4 __attribute__((ext_vector_type(4)));
typedef int mx_i8 __attribute__((ext_vector_type(8)));
typedef float mx_f4 __attribute__((ext_vector_type(4)));
typedef float mx_f16 __attribute__((ext_vector_type(16)));
typedef float mx_f2 __attribute__((ext_vector_type(2)));
typedef __bf16 mx_b2 __attribute__((ext_vector_type(2)));
typedef _Float16 mx_h2 __attribute__((ext_vector_type(2)));
typedef unsigned int mx_u4 __attribute__((ext_vector_type(4)));
typedef unsigned short mx_u16x2 __attribute__((ext_vector_type(2)));

// Scale byte of a block whose largest magnitude has the fp32 bits `peak`:
// X = 2^(byte - 127) = 2^(floor(log2(peak)) - 2), at least 2^-127. The exponent field
// of `peak` is floor(log2) + 127 (0 for subnormals, whose X is the least anyway). A
// block with an infinity or a NaN has byte 255, the format's NaN: all of it reads back
// as NaN, so the fault is seen in the product instead of being clamped away.
__device__ inline int mx_scale_byte(uint32_t peak) {
    const int e = static_cast<int>(peak >> 23);
    return e == 255 ? 255 : (e > 2 ? e - 2 : 0);
}

// The scale as the fp32 operand of the conversion instructions, which take its
// exponent alone (2^-127 has no normal fp32 form: its subnormal stands for it).
__device__ inline float mx_scale_value(int byte) {
    return __uint_as_float(byte ? static_cast<uint32_t>(byte) << 23 : 0x00400000u);
}

// Eight consecutive values in registers, in the form the conversions take: four fp32
// pairs, or four words of two 16-bit values.
template <typename T> struct MxRaw8;

template <> struct MxRaw8<float> {
    float v[8];
    __device__ void push(float x) {              // x becomes the first, the others move up
#pragma unroll
        for (int i = 7; i > 0; --i) v[i] = v[i - 1];
        v[0] = x;
    }
    __device__ void drop(int s) {                // the first s go, zeros follow the last
#pragma unroll
        for (int b = 4; b > 0; b >>= 1)
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = (s & b) ? (i + b < 8 ? v[i + b] : 0.0f) : v[i];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = s >= 8 ? 0.0f : v[i];
    }
    __device__ uint32_t peak() const {           // fp32 bits of the largest magnitude
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
        return m;
    }
    // v / scale rounded to the nearest code, ties to even, magnitudes above 6 to 6;
    // first value in the low nibble
    __device__ uint32_t codes(float scale) const {
        uint32_t w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0, v[0], v[1], scale, 0);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2], v[3], scale, 1);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4], v[5], scale, 2);
        return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6], v[7], scale, 3);
    }
};

template <typename T> struct MxRaw16 {
    uint32_t w[4];
    __device__ void push(T x) {
#pragma unroll
        for (int i = 3; i > 0; --i) w[i] = w[i] << 16 | w[i - 1] >> 16;
        w[0] = w[0] << 16 | __builtin_bit_cast(unsigned short, x);
    }
    __device__ void drop(int s) {
#pragma unroll
        for (int b = 2; b > 0; b >>= 1)
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = (s & 2 * b) ? (i + b < 4 ? w[i + b] : 0) : w[i];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            w[i] = (s & 1) ? w[i] >> 16 | (i < 3 ? w[i + 1] << 16 : 0) : w[i];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = s >= 8 ? 0 : w[i];
    }
    __device__ mx_u16x2 peak2() const {           // magnitudes compare as whole numbers
        mx_u16x2 m = __builtin_bit_cast(mx_u16x2, w[0] & 0x7fff7fffu);
#pragma unroll
        for (int i = 1; i < 4; ++i) m = __builtin_elementwise_max(m, __builtin_bit_cast(mx_u16x2, w[i] & 0x7fff7fffu));
        return m;
    }
    __device__ uint32_t peak_bits() const {
        const mx_u16x2 m = peak2();
        return max(m.x, m.y);
    }
};

template <> struct MxRaw8<__bf16> : MxRaw16<__bf16> {
    __device__ uint32_t peak() const { return peak_bits() << 16; }
    __device__ uint32_t codes(float scale) const {
        uint32_t c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(0, __builtin_bit_cast(mx_b2, w[0]), scale, 0);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(mx_b2, w[1]), scale, 1);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(mx_b2, w[2]), scale, 2);
        return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(mx_b2, w[3]), scale, 3);
    }
};

template <> struct MxRaw8<_Float16> : MxRaw16<_Float16> {
    __device__ uint32_t peak() const {
        return __float_as_uint(static_cast<float>(__builtin_bit_cast(_Float16, static_cast<unsigned short>(peak_bits()))));
    }
    __device__ uint32_t codes(float scale) const {
        uint32_t c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(0, __builtin_bit_cast(mx_h2, w[0]), scale, 0);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(mx_h2, w[1]), scale, 1);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(mx_h2, w[2]), scale, 2);
        return __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(mx_h2, w[3]), scale, 3);
    }
};

// `have` of eight values from p (any number; below 8 the rest are zero, at 0 and below
// nothing is read). Rows need no alignment beyond their type's.
template <typename T>
__device__ inline MxRaw8<T> mx_load8(const T* p, int have) {
    MxRaw8<T> r;
    if (have >= 8) {
        if constexpr (sizeof(T) == 4) {
            typedef uint32_t Words __attribute__((ext_vector_type(4), aligned(4)));
            const Words a = *reinterpret_cast<const Words*>(p), b = *reinterpret_cast<const Words*>(p + 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                r.v[i] = __uint_as_float(a[i]);
                r.v[4 + i] = __uint_as_float(b[i]);
            }
        } else {
            typedef uint32_t Words __attribute__((ext_vector_type(4), aligned(2)));
            const Words a = *reinterpret_cast<const Words*>(p);
#pragma unroll
            for (int i = 0; i < 4; ++i) r.w[i] = a[i];
        }
    } else {
        r = MxRaw8<T>{};
#pragma clang loop unroll(disable)
        for (int i = have - 1; i >= 0; --i) r.push(p[i]);   // rare: kept small
    }
    return r;
}

// The values k .. k + 7 of a row of K >= 8; those from `lim` <= K on (a multiple of 8, or
// K) are zero. Always one whole load within the row, moved down where it had to start
// earlier: no branch, so that the loads of several rows are in flight together.
template <typename T>
__device__ inline MxRaw8<T> mx_load8_tail(const T* row, int k, int K, int lim) {
    const int at = min(k, K - 8), s = k < lim ? k - at : 8;
    MxRaw8<T> r = mx_load8(row + at, 8);
    r.drop(s);
    return r;
}

// Between LDS accesses of a wave's lanes where one lane's stores are another's loads, or the
// other way round. A wave's LDS accesses complete in the order of its instructions, so the
// fences cost none of their own; they keep the compiler, which sees one lane, from moving
// an access across. (The wave barrier alone orders no memory accesses.)
__device__ __forceinline__ void mx_wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
}

// max over the four lanes of a block
__device__ inline uint32_t mx_quad_max(uint32_t m) {
    m = max(m, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(m), 0xB1, 0xf, 0xf, true)));
    return max(m, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(m), 0x4E, 0xf, 0xf, true)));
}

// Eight values of a block whose other values are in the lane's quad: their word of
// codes (zero codes where the block has a NaN or an infinity) and the block's byte.
template <typename T>
__device__ inline uint32_t mx_quant8(const MxRaw8<T>& v, int& byte) {
    byte = mx_scale_byte(mx_quad_max(v.peak()));
    return byte == 255 ? 0 : v.codes(mx_scale_value(byte));
}

template <typename T>
__device__ inline T mx_round(float v) { return static_cast<T>(v); }

// Two values rounded to a 16-bit type, the first in the low half.
template <typename T>
__device__ inline uint32_t mx_pack2(float a, float b) {
    typedef T V2 __attribute__((ext_vector_type(2)));
    const V2 v = {static_cast<T>(a), static_cast<T>(b)};
    return __builtin_bit_cast(uint32_t, v);
}

// Four neighbouring outputs y[at .. at + 3] of type `dtype`; `have` of them exist, and
// `vec` says that `at` is a multiple of 4 wherever all four do.
__device__ inline void mx_store4(void* y, int dtype, int64_t at, int have, bool vec, float a, float b, float c, float d) {
    if (vec && have >= 4) {
        if (dtype == MQ_F32) {
            *reinterpret_cast<float4*>(static_cast<float*>(y) + at) = make_float4(a, b, c, d);
        } else {
            const uint2 p = dtype == MQ_BF16 ? make_uint2(mx_pack2<__bf16>(a, b), mx_pack2<__bf16>(c, d))
                                             : make_uint2(mx_pack2<_Float16>(a, b), mx_pack2<_Float16>(c, d));
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(y) + at) = p;
        }
        return;
    }
    const float v[4] = {a, b, c, d};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (i >= have) return;
        if (dtype == MQ_F32) static_cast<float*>(y)[at + i] = v[i];
        else if (dtype == MQ_BF16) static_cast<__bf16*>(y)[at + i] = static_cast<__bf16>(v[i]);
        else static_cast<_Float16*>(y)[at + i] = static_cast<_Float16>(v[i]);
    }
}

// Buffer loads: reads past the operand's end give zero.
__device__ inline __amdgpu_buffer_rsrc_t buffer(const void* base, int64_t bytes) {
    // wave-uniform by construction; said so here, or every load becomes a loop over lanes
    const uint64_t p = reinterpret_cast<uint64_t>(base);
    const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(p));
    const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(p >> 32));
    const int n = __builtin_amdgcn_readfirstlane(static_cast<int>(bytes < 0 ? 0 : (bytes < 0xffffffff ? bytes : 0xffffffff)));
    return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(static_cast<uint64_t>(hi) << 32 | lo), 0, n, 0x00020000);
}
__device__ inline mx_i4 load16(__amdgpu_buffer_rsrc_t r, int lane_at, int at) {
    return __builtin_bit_cast(mx_i4, __builtin_amdgcn_raw_buffer_load_b128(r, lane_at, at, 0));
}
__device__ inline int load4(__amdgpu_buffer_rsrc_t r, int lane_at, int at) {
    return static_cast<int>(__builtin_amdgcn_raw_buffer_load_b32(r, lane_at, at, 0));
}

// g / (1 + exp(-g)), by the hardware's exponential of 2 and reciprocal, each within a unit in
// the last place. The exponential's argument is rounded to fp32 before, which turns into a
// relative error of up to 1.25 |g| 2^-24: with the rest, up to (1.25 |g| + 8) 2^-24 of the
// result. Below g = -87.3 the reciprocal leaves fp32's normal range and the result is 0 (the
// value is above -1e-36 there). Beside the 4-bit operands' own rounding and a 16-bit h
// none of this shows; an exact exponential and a division would cost twice the
// instructions of all the rest.
__device__ inline float mx_silu(float g) { return g * __builtin_amdgcn_rcpf(1.0f + __expf(-g)); }

}  // namespace mq
