// Products of unquantized rows with group-scaled 4-bit weights.
//
// y[m][n] = sum over groups g of s[n][g] * (P - z[n][g] * X), P = sum over the group of
// x[m][k] * c[n][k] and X = sum of x[m][k]. The codes 0 .. 15 become bf16 or fp16 in one
// conversion of two at a time: as e4m3 bytes they are c * 2^-9. They are exact in either type,
// so P is a sum of exact products on the matrix instructions, held in fp32, and the scales,
// which 16 bits would round, come in once a group in fp32. X comes from the same
// instructions, against ones.
#include "w4_device.h"
#include "w4_internal.h"

namespace mq {
namespace {

// The type the matrix instructions take, and how many of it make one value of x.
template <typename XT> struct W4Op {                  // bf16
    typedef __bf16 E;
    typedef w4_b8 V;
    static constexpr int kPieces = 1;
    static __device__ __forceinline__ mx_f4 mfma16(V a, V b, mx_f4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0); }
    static __device__ __forceinline__ V ones() { return __builtin_bit_cast(V, w4_u4{0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u}); }
};
template <> struct W4Op<_Float16> {
    typedef _Float16 E;
    typedef w4_h8 V;
    static constexpr int kPieces = 1;
    static __device__ __forceinline__ mx_f4 mfma16(V a, V b, mx_f4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0); }
    static __device__ __forceinline__ V ones() { return __builtin_bit_cast(V, w4_u4{0x3c003c00u, 0x3c003c00u, 0x3c003c00u, 0x3c003c00u}); }
};
// fp32 is the sum of three bf16 values: the first eight significant bits, the next eight
// and the rest, each cut off and not rounded, so that each remainder is exact.
template <> struct W4Op<float> : W4Op<__bf16> {
    static constexpr int kPieces = 3;
};

// Eight values of LDS (of a row: 16-byte units, fp32 two of them) as matrix operands.
template <typename XT>
__device__ __forceinline__ void pieces(const uint8_t* from, typename W4Op<XT>::V (&a)[W4Op<XT>::kPieces]) {
    typedef typename W4Op<XT>::V V;
    const w4_u4 lo = *reinterpret_cast<const w4_u4*>(from);
    if constexpr (sizeof(XT) == 2) {
        a[0] = __builtin_bit_cast(V, lo);
    } else {
        const w4_u4 hi = *reinterpret_cast<const w4_u4*>(from + 16);
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(i < 4 ? lo[i & 3] : hi[i & 3]);
#pragma unroll
        for (int p = 0; p < 3; ++p) {
            w4_u4 w;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[i] = __builtin_amdgcn_perm(__float_as_uint(v[2 * i + 1]), __float_as_uint(v[2 * i]), 0x07060302u);
            a[p] = __builtin_bit_cast(V, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] -= __uint_as_float(__float_as_uint(v[i]) & 0xffff0000u);
        }
    }
}

// expert of a plan's row, or -1 past the last expert's rows: every lane counts the
// experts that end at or before it
__device__ inline int expert_of(const int32_t* offsets, int E, int row) {
    const int lane = threadIdx.x & 63;
    int n = 0;
    for (int e0 = 0; e0 < E; e0 += 64) {
        const int e = e0 + lane;
        n += __popcll(__ballot(e < E && offsets[e + 1] <= row));
    }
    return n < E ? n : -1;
}

__device__ __forceinline__ void store1(void* y, int dtype, int64_t at, float v) {
    if (dtype == MQ_F32) static_cast<float*>(y)[at] = v;
    else if (dtype == MQ_BF16) static_cast<__bf16*>(y)[at] = static_cast<__bf16>(v);
    else static_cast<_Float16*>(y)[at] = static_cast<_Float16>(v);
}

// GS consecutive scales or zero points
template <int GS>
__device__ __forceinline__ uint64_t load_scales(const uint16_t* p) {
    if constexpr (GS == 1) return *p;
    else if constexpr (GS == 2) return *reinterpret_cast<const uint32_t*>(p);
    else return *reinterpret_cast<const uint64_t*>(p);
}

// ------------------------------------------------------------------- few rows
// A wave's rows of one code tile (128 inputs) in LDS; rows are 16 bytes further apart than
// they are long, so that 16 rows' units of 16 bytes lie in different banks.
template <typename XT> constexpr int kRowPitch = 128 * sizeof(XT) + 16;

// One workgroup: 16 MT rows x NT column tiles of 16, its waves each a run of K; their
// partial sums are added through LDS in the order of the waves. GS: groups in 128 inputs.
template <typename XT, int GS, bool Z, int NT, int MT>
__global__ __launch_bounds__(512) void k_w4_few(W4GemmArgs a) {
    typedef W4Op<XT> Op;
    typedef typename Op::V V;
    constexpr int kPieces = Op::kPieces, kPitch = kRowPitch<XT>, kUnit = 8 * sizeof(XT);
    extern __shared__ __align__(16) uint8_t lds[];    // each wave's rows, then the waves' sums
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
    const int G = (a.K + 127) / 128, Q = (G + 3) / 4, n_tiles = (a.N + 15) / 16, ct = blockIdx.x * NT;
    const int blocks = (a.M + 16 * MT - 1) / (16 * MT);
    const bool bf = a.scale_dtype == MQ_BF16;
    uint8_t* const mine = lds + wave * 16 * MT * kPitch;
    for (int rb = blockIdx.y; rb < blocks; rb += gridDim.y) {
        const int row0 = rb * 16 * MT, rows = min(16 * MT, a.M - row0);
        int e = 0;
        uint64_t alive = ~0ull;                        // which of a plan's rows have a token
        // lane l loads inputs 8 (l % 16) .. of rows 4j + l / 16
        const XT* from[4 * MT];
        if (a.offsets) {
            const int token = a.row_token[row0 + (lane & 15)];                     // (MT = 1)
            alive = __ballot(static_cast<unsigned>(token) < static_cast<unsigned>(a.T)) & 0xffff;
            e = __builtin_amdgcn_readfirstlane(expert_of(a.offsets, a.E, row0));
            if (e < 0) alive = 0;
        }
#pragma unroll
        for (int j = 0; j < 4 * MT; ++j) {
            int64_t r = row0 + min(4 * j + (lane >> 4), rows - 1);
            if (a.by_token) {
                const int t = a.row_token[r];
                r = static_cast<unsigned>(t) < static_cast<unsigned>(a.T) ? t : 0;
            }
            from[j] = static_cast<const XT*>(a.x) + r * a.stride_x + 8 * (lane & 15);
        }
        mx_f4 acc[NT][MT] = {};
        if (alive) {
            const uint8_t* w[NT];
            const uint16_t *ws[NT], *wz[NT];
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const int64_t tile = static_cast<int64_t>(e) * n_tiles + min(ct + j, n_tiles - 1);
                w[j] = a.codes + tile * G * 1024 + lane * 16;
                ws[j] = a.scales + (tile * Q * 16 + (lane & 15)) * 4 * GS;
                wz[j] = Z ? a.zeros + (tile * Q * 16 + (lane & 15)) * 4 * GS : nullptr;
            }
            const int h0 = static_cast<int>(static_cast<int64_t>(G) * wave / waves);
            const int h1 = static_cast<int>(static_cast<int64_t>(G) * (wave + 1) / waves);
            for (int h = h0; h < h1; ++h) {
                MxRaw8<XT> v[4 * MT];
                mx_i4 wc[NT];
                uint64_t sc[NT], zc[NT] = {};
#pragma unroll
                for (int j = 0; j < 4 * MT; ++j) v[j] = mx_load8(from[j] + h * 128, a.K - h * 128 - 8 * (lane & 15));
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    wc[j] = *reinterpret_cast<const mx_i4*>(w[j] + static_cast<int64_t>(h) * 1024);
                    const int at = ((h >> 2) * 16 * 4 + (h & 3)) * GS;
                    sc[j] = load_scales<GS>(ws[j] + at);
                    if constexpr (Z) zc[j] = load_scales<GS>(wz[j] + at);
                }
                mx_wave_sync();                        // the last tile's reads come first
#pragma unroll
                for (int j = 0; j < 4 * MT; ++j) {
                    uint8_t* const to = mine + (4 * j + (lane >> 4)) * kPitch + (lane & 15) * kUnit;
                    if constexpr (sizeof(XT) == 2) {
                        *reinterpret_cast<w4_u4*>(to) = w4_u4{v[j].w[0], v[j].w[1], v[j].w[2], v[j].w[3]};
                    } else {
                        *reinterpret_cast<mx_f4*>(to) = mx_f4{v[j].v[0], v[j].v[1], v[j].v[2], v[j].v[3]};
                        *reinterpret_cast<mx_f4*>(to + 16) = mx_f4{v[j].v[4], v[j].v[5], v[j].v[6], v[j].v[7]};
                    }
                }
                mx_wave_sync();
#pragma unroll
                for (int g = 0; g < GS; ++g) {
                    mx_f4 P[NT][MT] = {}, X[MT] = {};
#pragma unroll
                    for (int s = g * 4 / GS; s < (g + 1) * 4 / GS; ++s) {
                        V b[NT];
#pragma unroll
                        for (int j = 0; j < NT; ++j) b[j] = w4_codes<typename Op::E>(wc[j][s]);
#pragma unroll
                        for (int i = 0; i < MT; ++i) {
                            V x[kPieces];
                            pieces<XT>(mine + (16 * i + (lane & 15)) * kPitch + (4 * s + (lane >> 4)) * kUnit, x);
#pragma unroll
                            for (int p = 0; p < kPieces; ++p) {
                                X[i] = Op::mfma16(x[p], Op::ones(), X[i]);
#pragma unroll
                                for (int j = 0; j < NT; ++j) P[j][i] = Op::mfma16(x[p], b[j], P[j][i]);
                            }
                        }
                    }
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        const float sv = w4_float(static_cast<uint32_t>(sc[j] >> 16 * g) & 0xffff, bf);
                        const float zv = Z ? w4_float(static_cast<uint32_t>(zc[j] >> 16 * g) & 0xffff, bf) : 8.0f;
#pragma unroll
                        for (int i = 0; i < MT; ++i)
#pragma unroll
                            for (int r = 0; r < 4; ++r) acc[j][i][r] += sv * (P[j][i][r] - zv * X[i][r]);
                    }
                }
            }
        }
        float* const red = reinterpret_cast<float*>(lds);   // [waves][NT][MT][64][4]
        __syncthreads();
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int i = 0; i < MT; ++i) reinterpret_cast<mx_f4*>(red)[((wave * NT + j) * MT + i) * 64 + lane] = acc[j][i];
        __syncthreads();
        // output o: column o % (16 NT) of row o / (16 NT)
        for (int o = threadIdx.x; o < NT * MT * 256; o += blockDim.x) {
            const int c = o % (16 * NT), r = o / (16 * NT), m = row0 + r, n = ct * 16 + c;
            if (m >= a.M || n >= a.N) continue;
            const int at = (((c >> 4) * MT + (r >> 4)) * 64 + (r >> 2 & 3) * 16 + (c & 15)) * 4 + (r & 3);
            float v = 0;
            for (int s = 0; s < waves; ++s) v += red[s * NT * MT * 256 + at];
            if (a.bias) v += a.bias[n];
            if (a.offsets && !(alive >> (r & 15) & 1)) v = 0;
            store1(a.y, a.y_dtype, static_cast<int64_t>(m) * a.N + n, v);
        }
        __syncthreads();
    }
}

template <typename XT, int GS, bool Z, int NT, int MT>
hipError_t few(const W4GemmArgs& a, hipStream_t st) {
    const int G = (a.K + 127) / 128;
    const int most = MT == 1 ? 8 : 4, want = G >= 32 ? 8 : (G >= 8 ? 4 : (G >= 4 ? 2 : 1)), waves = want < most ? want : most;
    const unsigned cols = static_cast<unsigned>(((a.N + 15) / 16 + NT - 1) / NT);
    const int blocks = (a.M + 16 * MT - 1) / (16 * MT);
    const size_t one = 16 * MT * kRowPitch<XT>, sums = NT * MT * 1024;
    k_w4_few<XT, GS, Z, NT, MT><<<dim3(cols, blocks < 65535 ? blocks : 65535), 64 * waves, waves * (one > sums ? one : sums), st>>>(a);
    return hipGetLastError();
}

template <typename XT, int GS, bool Z>
hipError_t few_rows(const W4GemmArgs& a, hipStream_t st) {
    if constexpr (sizeof(XT) == 2) {
        if (!a.offsets && a.M > 16) return few<XT, GS, Z, 2, 2>(a, st);
    }
    return few<XT, GS, Z, 1, 1>(a, st);
}

template <typename XT>
hipError_t few_groups(const W4GemmArgs& a, hipStream_t st) {
    if (a.group == 128) return a.zeros ? few_rows<XT, 1, true>(a, st) : few_rows<XT, 1, false>(a, st);
    if (a.group == 64) return a.zeros ? few_rows<XT, 2, true>(a, st) : few_rows<XT, 2, false>(a, st);
    return a.zeros ? few_rows<XT, 4, true>(a, st) : few_rows<XT, 4, false>(a, st);
}

}  // namespace

hipError_t launch_w4_few(const W4GemmArgs& a, hipStream_t st) {
    switch (a.x_dtype) {
        case MQ_F32: return few_groups<float>(a, st);
        case MQ_BF16: return few_groups<__bf16>(a, st);
        default: return few_groups<_Float16>(a, st);
    }
}

}  // namespace mq
