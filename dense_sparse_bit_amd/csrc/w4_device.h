// Device helpers of the group-scaled 4-bit operators.
#pragma once

#include "mx_device.h"

namespace mq {

typedef __bf16 w4_b8 __attribute__((ext_vector_type(8)));
typedef _Float16 w4_h8 __attribute__((ext_vector_type(8)));
typedef uint32_t w4_u4 __attribute__((ext_vector_type(4)));

// A 16-bit scale or zero point. Both conversions and a select: the type is the same for
// all, but a branch would keep loads from being in flight together.
__device__ __forceinline__ float w4_float(uint32_t bits, bool bf) {
    const float h = static_cast<float>(__builtin_bit_cast(_Float16, static_cast<unsigned short>(bits)));
    return bf ? __uint_as_float(bits << 16) : h;
}

__device__ __forceinline__ uint32_t w4_bits(float v, bool bf) {
    return bf ? __builtin_bit_cast(unsigned short, static_cast<__bf16>(v)) : __builtin_bit_cast(unsigned short, static_cast<_Float16>(v));
}

template <typename T>
__device__ __forceinline__ void w4_values(const MxRaw8<T>& r, float (&v)[8]) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = r.v[i];
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (__is_same(T, __bf16)) {
                v[2 * i] = __uint_as_float(r.w[i] << 16);
                v[2 * i + 1] = __uint_as_float(r.w[i] & 0xffff0000u);
            } else {
                const mx_h2 h = __builtin_bit_cast(mx_h2, r.w[i]);
                v[2 * i] = static_cast<float>(h.x);
                v[2 * i + 1] = static_cast<float>(h.y);
            }
        }
    }
}

// `have` of eight values to p, rounded; rows need no alignment beyond their type's.
template <typename T>
__device__ __forceinline__ void w4_store8(T* p, int have, const float (&v)[8]) {
    if (have >= 8) {
        if constexpr (sizeof(T) == 4) {
            typedef float Out __attribute__((ext_vector_type(4), aligned(4)));
            *reinterpret_cast<Out*>(p) = Out{v[0], v[1], v[2], v[3]};
            *reinterpret_cast<Out*>(p + 4) = Out{v[4], v[5], v[6], v[7]};
        } else {
            typedef uint32_t Out __attribute__((ext_vector_type(4), aligned(2)));
            *reinterpret_cast<Out*>(p) = Out{mx_pack2<T>(v[0], v[1]), mx_pack2<T>(v[2], v[3]), mx_pack2<T>(v[4], v[5]),
                                             mx_pack2<T>(v[6], v[7])};
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < have) p[j] = mx_round<T>(v[j]);
    }
}

// Reductions over the lanes of a group: 4, 8 or 16 neighbours hold 32, 64 or 128 inputs.
// (Lane moves within four, then across halves of eight and of sixteen by mirroring.)
template <typename F>
__device__ __forceinline__ int w4_over_group(int v, int group, F f) {
    v = f(v, __builtin_amdgcn_mov_dpp(v, 0xB1, 0xf, 0xf, true));
    v = f(v, __builtin_amdgcn_mov_dpp(v, 0x4E, 0xf, 0xf, true));
    if (group >= 64) v = f(v, __builtin_amdgcn_mov_dpp(v, 0x141, 0xf, 0xf, true));
    if (group >= 128) v = f(v, __builtin_amdgcn_mov_dpp(v, 0x140, 0xf, 0xf, true));
    return v;
}

// The word of eight codes: input i in the low half of byte i, or the high half of byte i - 4.
__device__ __forceinline__ uint32_t w4_word(const uint32_t (&c)[8]) {
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) w |= c[i] << (i < 4 ? 8 * i : 8 * (i - 4) + 4);
    return w;
}

// The scales or zero points of a code tile's groups in one word.
template <int GS> struct W4Scales { typedef uint32_t T; };
template <> struct W4Scales<4> { typedef uint64_t T; };
template <int GS>
__device__ __forceinline__ typename W4Scales<GS>::T w4_scales(const uint16_t* p) {
    if constexpr (GS == 1) return *p;
    else return *reinterpret_cast<const typename W4Scales<GS>::T*>(p);
}

// The scales or zero points of a quad of code tiles (4 GS of them).
template <int GS> struct W4Quad {
    uint32_t w[2 * GS];
    __device__ __forceinline__ void load(const uint16_t* p) {
        if constexpr (GS == 1) {
            const uint2 v = *reinterpret_cast<const uint2*>(p);
            w[0] = v.x;
            w[1] = v.y;
        } else {
#pragma unroll
            for (int i = 0; i < GS / 2; ++i) {
                const uint4 v = reinterpret_cast<const uint4*>(p)[i];
                w[4 * i] = v.x;
                w[4 * i + 1] = v.y;
                w[4 * i + 2] = v.z;
                w[4 * i + 3] = v.w;
            }
        }
    }
    __device__ __forceinline__ float get(int i, bool bf) const { return w4_float(i & 1 ? w[i >> 1] >> 16 : w[i >> 1] & 0xffff, bf); }
};

// Eight codes as bf16 or fp16, exactly, in the order of the inputs: as e4m3 bytes they are
// c * 2^-9. A mask of 0 makes them zeros.
template <typename E>
__device__ __forceinline__ auto w4_codes(uint32_t w, uint32_t mask = 0x0f0f0f0fu) {
    const uint32_t lo = w & mask, hi = w >> 4 & mask;
    if constexpr (__is_same(E, _Float16)) {
        const mx_h2 v[4] = {__builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 512.0f, false), __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 512.0f, true),
                            __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 512.0f, false), __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 512.0f, true)};
        return __builtin_bit_cast(w4_h8, v);
    } else {
        const mx_b2 v[4] = {__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 512.0f, false), __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 512.0f, true),
                            __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 512.0f, false), __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 512.0f, true)};
        return __builtin_bit_cast(w4_b8, v);
    }
}

}  // namespace mq
