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

// v / D, rounded once: a product by the reciprocal and its exact remainder's (Markstein),
// which needs that no part of it is subnormal.
template <int D>
__device__ __forceinline__ float over(float v) {
    constexpr float kInv = 1.0f / D;
    float q = v * kInv;
    q = __builtin_fmaf(__builtin_fmaf(-static_cast<float>(D), q, v), kInv, q);
    if (v < 0x1p-90f || v > 0x1p127f) q = v / D;           // (infinities among them)
    return q;
}

// v / s rounded once, likewise: inv is 1 / s rounded once, and s has no more than 11 bits, so
// that the remainder is exact however the first product was rounded. To round that again to a
// whole number changes nothing: v and s times half a whole number differ by a last place of v
// at least, or not at all.
__device__ __forceinline__ float quotient(float v, float s, float inv) {
    const float q = v * inv;
    return __builtin_fmaf(__builtin_fmaf(-q, s, v), inv, q);
}

// The word of codes, the scale and the zero point of eight values of a group whose others
// are in neighbouring lanes.
template <bool Z, typename T>
__device__ __forceinline__ uint32_t quant8(const MxRaw8<T>& raw, int group, bool bf, uint32_t& scale, uint32_t& zero) {
    constexpr float kWhole = 12582912.0f;                // 1.5 * 2^23: the last place is 1
    float v[8];
    w4_values(raw, v);
    const int peak = w4_over_group(static_cast<int>(raw.peak()), group, [](int a, int b) { return max(a, b); });
    float s, lo = 0;
    if constexpr (Z) {
        float hi = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            lo = fminf(lo, v[i]);
            hi = fmaxf(hi, v[i]);
        }
        const auto least = [](int a, int b) { return __float_as_int(fminf(__int_as_float(a), __int_as_float(b))); };
        const auto most = [](int a, int b) { return __float_as_int(fmaxf(__int_as_float(a), __int_as_float(b))); };
        lo = __int_as_float(w4_over_group(__float_as_int(lo), group, least));
        hi = __int_as_float(w4_over_group(__float_as_int(hi), group, most));
        s = over<15>(hi - lo);
    } else {
        s = over<7>(__int_as_float(peak));
    }
    scale = w4_bits(fminf(s, bf ? __uint_as_float(0x7f7f0000u) : 65504.0f), bf);
    s = w4_float(scale, bf);
    const bool bad = peak >= 0x7f800000, live = s > 0 && !bad;
    if (bad) scale = bf ? 0x7fc0 : 0x7e00;
    if (s < 0x1p-64f || s > 0x1p64f) {                   // reciprocals and remainders to normal numbers
        const float to = s < 1.0f ? 0x1p64f : 0x1p-64f;
        s *= to;
        lo *= to;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= to;
    }
    float inv = __builtin_amdgcn_rcpf(s);
    inv = __builtin_fmaf(__builtin_fmaf(-s, inv, 1.0f), inv, inv);
    // Quotients are rounded, ties to even, by adding a number whose last place is 1 and even;
    // an odd zero point's last bit is added to the codes of both halves of a byte at once.
    float z = 8.0f, odd = 0.0f;
    if constexpr (Z) {
        z = __builtin_amdgcn_fmed3f(__builtin_rintf(quotient(-lo, s, inv)), 0.0f, 15.0f);
        if (!live) z = 0.0f;
        odd = z - 2.0f * floorf(0.5f * z);
    }
    zero = w4_bits(z, bf);
    const float base = kWhole + (z - odd);
    uint32_t c[8], p[4];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        c[i] = __float_as_uint(__builtin_amdgcn_fmed3f(quotient(v[i], s, inv) + base, kWhole - odd, kWhole + 15.0f - odd));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        p[i] = (c[i + 4] << 4) + c[i];                   // the low byte: codes i and i + 4
        if constexpr (Z) p[i] += odd > 0 ? 17 : 0;
    }
    const uint32_t ab = __builtin_amdgcn_perm(p[1], p[0], 0x0c0c0400u), cd = __builtin_amdgcn_perm(p[3], p[2], 0x0c0c0400u);
    return live ? ab | cd << 16 : (Z ? 0 : 0x88888888u);
}

// One workgroup: 16 rows x 512 inputs (four code tiles). Wave w reads rows 4w .. 4w + 3, 1 KB
// of a 16-bit type at a time; lane l holds inputs 8l .. 8l + 7. Codes go through LDS, because a
// tile keeps the rows of a few inputs together: they leave as 4 KB runs, scales as runs of 128 B
// or more. Bound by memory, closely followed by the arithmetic: with a division a value, and
// scales stored two bytes at a time, it took 92 us for 17408 x 5120 of bf16, with quotients by
// the reciprocal 44 us (5.1 TB/s read and written), 59 us with zero points (two more
// reductions).
template <typename T, bool Z>
__global__ __launch_bounds__(kThreads) void k_w4_quant(W4QuantArgs a) {
    __shared__ __align__(16) uint32_t lds[4 * kTile];
    __shared__ __align__(16) uint16_t lds_s[16 * 16], lds_z[Z ? 16 * 16 : 1];
    const int G = (a.K + 127) / 128, Q = (a.K + 511) / 512, bits = __builtin_ctz(a.group), per = 512 >> bits;
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
            uint32_t scale, zero;
            uint32_t word = quant8<Z>(raw[i], a.group, bf, scale, zero);
            // what is behind the matrix's end holds zeros
            if (rt * 16 + row >= a.R || k0 >> bits << bits >= a.K) word = scale = zero = 0;
            else if (k0 + 8 > a.K) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (k0 + j >= a.K) word &= ~(15u << (j < 4 ? 8 * j : 8 * (j - 4) + 4));
            }
            lds[lds_word(row, lane)] = word;
            if ((8 * lane & (a.group - 1)) == 0) {
                const int at = row * per + (8 * lane >> bits);
                lds_s[at] = static_cast<uint16_t>(scale);
                if constexpr (Z) lds_z[at] = static_cast<uint16_t>(zero);
            }
        }
        __syncthreads();
        if (t < 8 * per) {
            const int64_t at = ((b * RT + rt) * Q + q) * 16 * per + 2 * t;
            *reinterpret_cast<uint32_t*>(a.scales + at) = *reinterpret_cast<const uint32_t*>(&lds_s[2 * t]);
            if constexpr (Z) *reinterpret_cast<uint32_t*>(a.zeros + at) = *reinterpret_cast<const uint32_t*>(&lds_z[2 * t]);
        }
        if (q * 4 + wave < G)
            *reinterpret_cast<uint4*>(a.codes + ((b * RT + rt) * G + q * 4) * 1024 + t * 16) =
                *reinterpret_cast<const uint4*>(&lds[lds_unit(t)]);
        __syncthreads();
    }
}

// Given codes, scales and zero points into the same places. Bound by its accesses, 8 bytes of codes and
// 2 of a scale or zero point a lane: 17408 x 5120 in groups of 128 38 us, and 51 from codes that no cache
// holds (read and written at the rate of a large copy: 26); 64 matrices 4096 x 1024 in groups of 64 with
// zero points 175 (84).
__global__ __launch_bounds__(kThreads) void k_w4_pack(W4QuantArgs a) {
    __shared__ __align__(16) uint32_t lds[4 * kTile];
    const int G = (a.K + 127) / 128, Q = (a.K + 511) / 512, bits = __builtin_ctz(a.group), per = 512 >> bits;
    const int n = (a.K + a.group - 1) >> bits;
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
            if ((8 * lane & (a.group - 1)) == 0) {
                const int g = k0 >> bits;
                const bool there = r < a.R && g < n;
                const int64_t from = (b * a.R + r) * n + g, at = (((b * RT + rt) * Q + q) * 16 + row) * per + (8 * lane >> bits);
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
// rows. Bound by the writes: 17408 x 5120 to bf16 in 38 us (4.7 TB/s written).
template <typename T>
__global__ __launch_bounds__(kThreads) void k_w4_dequant(W4QuantArgs a, T* y) {
    __shared__ __align__(16) uint32_t lds[4 * kTile];
    const int G = (a.K + 127) / 128, Q = (a.K + 511) / 512, bits = __builtin_ctz(a.group), per = 512 >> bits;
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
            const int64_t at = (((b * RT + rt) * Q + q) * 16 + 4 * wave + i) * per + (8 * lane >> bits);
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
