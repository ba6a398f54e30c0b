// Group-scaled 4-bit quantization, packing of given codes, and the way back.
#include "w4_device.h"
#include "w4_internal.h"

namespace mq {
namespace {

constexpr int kThreads = 256;

// Words of 16 rows x 512 inputs in LDS, in the order in which the tiles hold them:
// [tile][quarter of the lanes][row][word]. Quarters are 4 words and tiles 16 words further
// apart than they are long, so that a row's 64 words fall into different banks.
constexpr int kQuarter = 64 + 4, kTile = 4 * kQuarter;
__device__ __forceinline__ int lds_word(int row, int lane) {
    return (lane >> 4) * kTile + (lane & 3) * kQuarter + row * 4 + (lane >> 2 & 3);
}
__device__ __forceinline__ int lds_unit(int t) { return (t >> 6) * kTile + (t >> 4 & 3) * kQuarter + (t & 15) * 4; }

// Codes of eight values that share the scale s > 0 (finite), from 0 to 15 with z added.
// Quotients go by a reciprocal, which is off by less than 1e-5 of a step where the code is
// not clamped anyway; where one comes within 1e-4 of a border, the remainder v - q s (exact: a
// multiple of the lesser of v's and s's last places, and less than s) tells on which side it is.
__device__ __forceinline__ void round8(float (&v)[8], float s, float z, uint32_t (&c)[8]) {
    const float up = s < 0x1p-64f ? 0x1p64f : 1.0f;   // away from subnormal reciprocals' loss
    s *= up;
    const float inv = 1.0f / s;
    float q[8], far = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        v[i] *= up;
        const float t = v[i] * inv;
        q[i] = __builtin_rintf(t);
        far = fmaxf(far, fabsf(t - q[i]));
    }
    if (far > 0.4999f) {
        const float half = 0.5f * s;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float d = __builtin_fmaf(-q[i], s, v[i]), e = fabsf(d) - half;
            const bool odd = 0.5f * q[i] != __builtin_rintf(0.5f * q[i]);
            if (e > 0 || (e == 0 && odd)) q[i] += copysignf(1.0f, d);
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = static_cast<uint32_t>(__builtin_amdgcn_fmed3f(q[i] + z, 0.0f, 15.0f));
}

// rne(v / s), s > 0, between 0 and 15
__device__ __forceinline__ float round1(float v, float s) {
    const float up = s < 0x1p-64f ? 0x1p64f : 1.0f;
    s *= up;
    v *= up;
    float q = __builtin_rintf(v / s);
    const float d = __builtin_fmaf(-q, s, v), e = fabsf(d) - 0.5f * s;
    const bool odd = 0.5f * q != __builtin_rintf(0.5f * q);
    if (e > 0 || (e == 0 && odd)) q += copysignf(1.0f, d);
    return __builtin_amdgcn_fmed3f(q, 0.0f, 15.0f);
}

// The word of codes, the scale and the zero point of eight values of a group whose others
// are in neighbouring lanes.
template <bool Z>
__device__ __forceinline__ uint32_t quant8(float (&v)[8], int group, bool bf, uint32_t& scale, uint32_t& zero) {
    int peak = 0;
    float lo = 0, hi = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        peak = max(peak, static_cast<int>(__float_as_uint(v[i]) & 0x7fffffffu));
        if constexpr (Z) {
            lo = fminf(lo, v[i]);
            hi = fmaxf(hi, v[i]);
        }
    }
    peak = w4_over_group(peak, group, [](int a, int b) { return max(a, b); });
    float s = __int_as_float(peak) / 7.0f;
    if constexpr (Z) {
        const auto least = [](int a, int b) { return __float_as_int(fminf(__int_as_float(a), __int_as_float(b))); };
        const auto most = [](int a, int b) { return __float_as_int(fmaxf(__int_as_float(a), __int_as_float(b))); };
        lo = __int_as_float(w4_over_group(__float_as_int(lo), group, least));
        hi = __int_as_float(w4_over_group(__float_as_int(hi), group, most));
        s = (hi - lo) / 15.0f;
    }
    s = fminf(s, bf ? __uint_as_float(0x7f7f0000u) : 65504.0f);
    scale = w4_bits(s, bf);
    s = w4_float(scale, bf);
    float z = Z ? 0.0f : 8.0f;
    const bool bad = peak >= 0x7f800000;
    if (bad) scale = bf ? 0x7fc0 : 0x7e00;
    uint32_t c[8];
    if (s > 0 && !bad) {
        if constexpr (Z) z = round1(-lo, s);
        round8(v, s, z, c);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) c[i] = static_cast<uint32_t>(z);
    }
    zero = w4_bits(z, bf);
    return w4_word(c);
}

// One workgroup: 16 rows x 512 inputs (four code tiles). Wave w reads rows 4w .. 4w + 3, 1 KB
// of a 16-bit type at a time; lane l holds inputs 8l .. 8l + 7. Codes go through LDS, because a
// tile keeps the rows of a few inputs together: they leave as 4 KB runs. Bound by the
// read of x.
template <typename T, bool Z>
__global__ __launch_bounds__(kThreads) void k_w4_quant(W4QuantArgs a) {
    __shared__ __align__(16) uint32_t lds[4 * kTile];
    const int G = (a.K + 127) / 128, Q = (a.K + 511) / 512, per = 512 / a.group;
    const int64_t RT = (a.R + 15) / 16, b = blockIdx.z;
    const int q = blockIdx.x, t = threadIdx.x, wave = t >> 6, lane = t & 63;
    const int k0 = q * 512 + 8 * lane;
    const bool bf = a.scale_dtype == MQ_BF16;
    const T* const x = static_cast<const T*>(a.x) + b * a.stride_b + k0;
    for (int64_t rt = blockIdx.y; rt < RT; rt += gridDim.y) {
        MxRaw8<T> raw[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t r = rt * 16 + 4 * wave + i;
            raw[i] = mx_load8(x + r * a.stride_r, r < a.R ? a.K - k0 : 0);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = 4 * wave + i;
            float v[8];
            w4_values(raw[i], v);
            uint32_t scale, zero;
            uint32_t word = quant8<Z>(v, a.group, bf, scale, zero);
            // what is behind the matrix's end holds zeros
            if (rt * 16 + row >= a.R || k0 / a.group * a.group >= a.K) word = scale = zero = 0;
            else if (k0 + 8 > a.K) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (k0 + j >= a.K) word &= ~(15u << (j < 4 ? 8 * j : 8 * (j - 4) + 4));
            }
            lds[lds_word(row, lane)] = word;
            const int unit = a.group / 8;
            if ((lane & (unit - 1)) == 0) {
                const int64_t at = (((b * RT + rt) * Q + q) * 16 + row) * per + lane / unit;
                a.scales[at] = static_cast<uint16_t>(scale);
                if constexpr (Z) a.zeros[at] = static_cast<uint16_t>(zero);
            }
        }
        __syncthreads();
        if (q * 4 + wave < G)
            *reinterpret_cast<uint4*>(a.codes + ((b * RT + rt) * G + q * 4) * 1024 + t * 16) =
                *reinterpret_cast<const uint4*>(&lds[lds_unit(t)]);
        __syncthreads();
    }
}

// Given codes, scales and zero points into the same places.
__global__ __launch_bounds__(kThreads) void k_w4_pack(W4QuantArgs a) {
    __shared__ __align__(16) uint32_t lds[4 * kTile];
    const int G = (a.K + 127) / 128, Q = (a.K + 511) / 512, per = 512 / a.group, n = (a.K + a.group - 1) / a.group;
    const int64_t RT = (a.R + 15) / 16, b = blockIdx.z;
    const int q = blockIdx.x, t = threadIdx.x, wave = t >> 6, lane = t & 63;
    const int k0 = q * 512 + 8 * lane;
    const uint8_t* const x = static_cast<const uint8_t*>(a.x) + b * a.stride_b + k0;
    for (int64_t rt = blockIdx.y; rt < RT; rt += gridDim.y) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = 4 * wave + i;
            const int64_t r = rt * 16 + row;
            uint32_t c[8] = {};
            if (r < a.R) {
                const uint8_t* const p = x + r * a.stride_r;
                if (k0 + 8 <= a.K) {
                    typedef uint32_t Bytes __attribute__((ext_vector_type(2), aligned(1)));
                    const Bytes w = *reinterpret_cast<const Bytes*>(p);
#pragma unroll
                    for (int j = 0; j < 8; ++j) c[j] = w[j >> 2] >> 8 * (j & 3) & 15;
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (k0 + j < a.K) c[j] = p[j] & 15;
                }
            }
            lds[lds_word(row, lane)] = w4_word(c);
            const int unit = a.group / 8;
            if ((lane & (unit - 1)) == 0) {
                const int g = k0 / a.group;
                const bool there = r < a.R && g < n;
                const int64_t from = (b * a.R + r) * n + g, at = (((b * RT + rt) * Q + q) * 16 + row) * per + lane / unit;
                a.scales[at] = there ? a.s[from] : 0;
                if (a.z) a.zeros[at] = there ? a.z[from] : 0;
            }
        }
        __syncthreads();
        if (q * 4 + wave < G)
            *reinterpret_cast<uint4*>(a.codes + ((b * RT + rt) * G + q * 4) * 1024 + t * 16) =
                *reinterpret_cast<const uint4*>(&lds[lds_unit(t)]);
        __syncthreads();
    }
}

// The way back, tile by tile: codes come in as one run, change places in LDS and leave as
// rows. Bound by the writes.
template <typename T>
__global__ __launch_bounds__(kThreads) void k_w4_dequant(W4QuantArgs a, T* y) {
    __shared__ __align__(16) uint32_t lds[4 * kTile];
    const int G = (a.K + 127) / 128, Q = (a.K + 511) / 512, per = 512 / a.group;
    const int64_t RT = (a.R + 15) / 16, b = blockIdx.z;
    const int q = blockIdx.x, t = threadIdx.x, wave = t >> 6, lane = t & 63;
    const int k0 = q * 512 + 8 * lane, have = a.K - k0;
    const bool bf = a.scale_dtype == MQ_BF16;
    for (int64_t rt = blockIdx.y; rt < RT; rt += gridDim.y) {
        if (q * 4 + wave < G)
            *reinterpret_cast<uint4*>(&lds[lds_unit(t)]) =
                *reinterpret_cast<const uint4*>(a.codes + ((b * RT + rt) * G + q * 4) * 1024 + t * 16);
        float s[4], z[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t at = (((b * RT + rt) * Q + q) * 16 + 4 * wave + i) * per + lane / (a.group / 8);
            s[i] = w4_float(a.scales[at], bf);
            z[i] = a.zeros ? w4_float(a.zeros[at], bf) : 8.0f;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = 4 * wave + i;
            const int64_t r = rt * 16 + row;
            if (r >= a.R || have <= 0) continue;
            const uint32_t w = lds[lds_word(row, lane)], lo = w & 0x0f0f0f0fu, hi = w >> 4 & 0x0f0f0f0fu;
            float v[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[j] = (static_cast<float>(lo >> 8 * j & 255) - z[i]) * s[i];
                v[4 + j] = (static_cast<float>(hi >> 8 * j & 255) - z[i]) * s[i];
            }
            w4_store8(y + (b * a.R + r) * a.K + k0, have, v);
        }
        __syncthreads();
    }
}

dim3 grid_of(const W4QuantArgs& a) {
    const int64_t RT = w4_row_tiles(a.R);
    return dim3(static_cast<unsigned>(w4_quads(a.K)), static_cast<unsigned>(RT < 32768 ? RT : 32768), static_cast<unsigned>(a.B));
}

template <typename T>
hipError_t quant(const W4QuantArgs& a, hipStream_t st) {
    if (a.zeros) k_w4_quant<T, true><<<grid_of(a), kThreads, 0, st>>>(a);
    else k_w4_quant<T, false><<<grid_of(a), kThreads, 0, st>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_w4_quant(const W4QuantArgs& a, hipStream_t st) {
    switch (a.dtype) {
        case MQ_F32: return quant<float>(a, st);
        case MQ_BF16: return quant<__bf16>(a, st);
        default: return quant<_Float16>(a, st);
    }
}

hipError_t launch_w4_pack(const W4QuantArgs& a, hipStream_t st) {
    k_w4_pack<<<grid_of(a), kThreads, 0, st>>>(a);
    return hipGetLastError();
}

hipError_t launch_w4_dequant(const W4QuantArgs& a, void* y, int y_dtype, hipStream_t st) {
    switch (y_dtype) {
        case MQ_F32: k_w4_dequant<float><<<grid_of(a), kThreads, 0, st>>>(a, static_cast<float*>(y)); break;
        case MQ_BF16: k_w4_dequant<__bf16><<<grid_of(a), kThreads, 0, st>>>(a, static_cast<__bf16*>(y)); break;
        default: k_w4_dequant<_Float16><<<grid_of(a), kThreads, 0, st>>>(a, static_cast<_Float16*>(y)); break;
    }
    return hipGetLastError();
}

}  // namespace mq
