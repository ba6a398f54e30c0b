// Microscaled 4-bit quantization and its reverse.
//
// A block is 32 consecutive inputs of a row. X = 2^(floor(log2(max |v|)) - 2) puts the
// largest magnitude into [4, 8) X; each value becomes the nearest of
// 0, 0.5, 1, 1.5, 2, 3, 4, 6 times X.
#include "mx_device.h"
#include "mx_internal.h"
#include "plan_tiles.h"

namespace mq {
namespace {

constexpr int kThreads = 256;

// One workgroup: 16 rows x 512 inputs (four code tiles, one scale entry per lane).
// Wave w reads rows 4w .. 4w + 3, 1 KB of bf16 at a time; lane l holds inputs
// 8l .. 8l + 7, four lanes a block. Codes and scales go through LDS, because a tile
// keeps the rows of a block together and a row's blocks apart: they leave as 4 KB and
// 256 B runs. Bound by memory: 17408 x 5120 of bf16 in 50 us (4.5 TB/s read and written).
template <typename T>
__global__ __launch_bounds__(kThreads) void k_mx_quant(const T* x, int64_t stride_b, int64_t R, int64_t stride_r, int K,
                                                       uint8_t* codes, uint8_t* scales, MxTilesArgs plan) {
    constexpr int kRun = 16 * 4 + 4;                // words of a block's 16 rows, and 4 more: other banks
    __shared__ __align__(16) uint32_t lds_codes[16 * kRun];
    __shared__ uint8_t lds_scales[256];
    const int G = (K + 127) / 128, G4 = (G + 3) / 4;
    const int64_t RT = (R + 15) / 16;
    const int q = blockIdx.x;                       // quad of tiles
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int k0 = q * 512 + 8 * lane;
    const int64_t b = blockIdx.z;
    static_assert(16 * kRun >= kTilesLds);
    const int first = plan.offsets ? 1 : 0;         // workgroups (0, 0): the plan's row blocks alone
    if (static_cast<int>(blockIdx.y) < first) {
        if (blockIdx.x == 0) plan_tiles<kBlockTiles>(plan, reinterpret_cast<int*>(lds_codes));
        return;
    }
    for (int64_t rt = blockIdx.y - first; rt < RT; rt += gridDim.y - first) {
        MxRaw8<T> v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t r = rt * 16 + 4 * wave + i;
            v[i] = mx_load8(x + b * stride_b + r * stride_r + k0, r < R ? K - k0 : 0);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = 4 * wave + i;
            int byte;
            lds_codes[(lane >> 2) * kRun + row * 4 + (lane & 3)] = mx_quant8(v[i], byte);
            // blocks beyond K hold zeros, so their byte is 0
            if ((lane & 3) == 0) lds_scales[(((lane >> 2) & 3) * 16 + row) * 4 + (lane >> 4)] = byte;
        }
        __syncthreads();
        const int t = threadIdx.x;
        if (q * 4 + (t >> 6) < G)
            *reinterpret_cast<uint4*>(codes + ((b * RT + rt) * G + q * 4) * 1024 + t * 16) =
                *reinterpret_cast<const uint4*>(&lds_codes[(t >> 4) * kRun + (t & 15) * 4]);
        if (t < 64)
            *reinterpret_cast<uint32_t*>(scales + ((b * RT + rt) * G4 + q) * 256 + t * 4) =
                *reinterpret_cast<const uint32_t*>(&lds_scales[4 * t]);
        __syncthreads();
    }
}

// The same blocks row by row: a wave takes 512 inputs of kRows rows, each row's codes
// leave as one run of 256 bytes. 4096 x 4096 of bf16: 12 us.
constexpr int kRows = 4;
template <typename T>
__global__ __launch_bounds__(kThreads) void k_mx_quant_rows(const T* x, int64_t R, int64_t stride_r, int K, uint8_t* codes,
                                                            uint8_t* scales, MxTilesArgs plan) {
    __shared__ int lds[kTilesLds];
    const int first = plan.offsets ? 1 : 0;         // workgroups (0, 0): the plan's row blocks alone
    if (static_cast<int>(blockIdx.x) < first) {
        if (blockIdx.y == 0) plan_tiles<kBlockTiles>(plan, lds);
        return;
    }
    const int G = (K + 127) / 128, G2 = (G + 1) / 2, G4 = (G + 3) / 4;
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int64_t r0 = (static_cast<int64_t>(blockIdx.x - first) * 4 + wave) * kRows;
    const int q = blockIdx.y, k0 = q * 512 + 8 * lane;
    MxRaw8<T> v[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) v[i] = mx_load8(x + (r0 + i) * stride_r + k0, r0 + i < R ? K - k0 : 0);
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        int byte;
        const uint32_t word = mx_quant8(v[i], byte);
        const int64_t r = r0 + i;
        if (r >= R) return;
        if (q * 4 + (lane >> 5) * 2 < G) *reinterpret_cast<uint32_t*>(codes + r * G2 * 128 + q * 256 + lane * 4) = word;
        if ((lane & 3) == 0) scales[(r * G4 + q) * 16 + (lane >> 2 & 3) * 4 + (lane >> 4)] = byte;
    }
}

// The way back, tile by tile as k_mx_quant: the codes of 16 rows x 512 inputs come in as
// one run, change places in LDS (runs of 16 rows 16 bytes apart, so that a row's words
// lie in different banks) and leave as rows, 16 bytes of bf16 a lane. The instruction's
// value times scale is exact in fp32 and rounded once to T. Bound by the writes: 17408 x
// 5120 to bf16 in 34 us (5.2 TB/s written).
template <typename T>
__global__ __launch_bounds__(kThreads) void k_mx_dequant(const uint8_t* codes, const uint8_t* scales, int64_t R, int K,
                                                         T* y) {
    constexpr int kRun = 16 * 4 + 4;                // words of a block's 16 rows, and 4 more
    __shared__ __align__(16) uint32_t lds_codes[16 * kRun];
    __shared__ uint32_t lds_scales[64];
    const int G = (K + 127) / 128, G4 = (G + 3) / 4;
    const int64_t RT = (R + 15) / 16, b = blockIdx.z;
    const int q = blockIdx.x, t = threadIdx.x, wave = t >> 6, lane = t & 63;
    const int k0 = q * 512 + 8 * lane, have = K - k0;
    for (int64_t rt = blockIdx.y; rt < RT; rt += gridDim.y) {
        if (q * 4 + wave < G)
            *reinterpret_cast<uint4*>(&lds_codes[(t >> 4) * kRun + (t & 15) * 4]) =
                *reinterpret_cast<const uint4*>(codes + ((b * RT + rt) * G + q * 4) * 1024 + t * 16);
        if (t < 64) lds_scales[t] = *reinterpret_cast<const uint32_t*>(scales + ((b * RT + rt) * G4 + q) * 256 + t * 4);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = 4 * wave + i;
            const int64_t r = rt * 16 + row;
            if (r >= R || have <= 0) continue;
            const uint32_t w = lds_codes[(lane >> 2) * kRun + row * 4 + (lane & 3)];
            const int byte = lds_scales[(lane >> 2 & 3) * 16 + row] >> 8 * (lane >> 4) & 255;
            const float scale = mx_scale_value(byte);
            float v[8];
            const mx_f2 p0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 0), p1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 1),
                        p2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 2), p3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 3);
            v[0] = p0[0]; v[1] = p0[1]; v[2] = p1[0]; v[3] = p1[1];
            v[4] = p2[0]; v[5] = p2[1]; v[6] = p3[0]; v[7] = p3[1];
            if (byte == 255) {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(0x7fc00000u);
            }
            T* out = y + (b * R + r) * K + k0;
            if (have >= 8) {
                if constexpr (sizeof(T) == 4) {
                    typedef float Out __attribute__((ext_vector_type(4), aligned(4)));
                    *reinterpret_cast<Out*>(out) = Out{v[0], v[1], v[2], v[3]};
                    *reinterpret_cast<Out*>(out + 4) = Out{v[4], v[5], v[6], v[7]};
                } else {
                    typedef uint32_t Out __attribute__((ext_vector_type(4), aligned(2)));
                    *reinterpret_cast<Out*>(out) = Out{mx_pack2<T>(v[0], v[1]), mx_pack2<T>(v[2], v[3]), mx_pack2<T>(v[4], v[5]),
                                                       mx_pack2<T>(v[6], v[7])};
                }
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (j < have) out[j] = mx_round<T>(v[j]);
            }
        }
        __syncthreads();
    }
}

template <typename T>
hipError_t quant(const MxQuantArgs& a, hipStream_t st) {
    const int64_t RT = mx_row_tiles(a.R);
    const int quads = static_cast<int>(mx_quads(a.K));
    const T* x = static_cast<const T*>(a.x);
    const unsigned first = a.plan.offsets ? 1 : 0;     // workgroups for the plan's row blocks
    if (a.by_row) {
        const dim3 grid(static_cast<unsigned>((a.R + 4 * kRows - 1) / (4 * kRows)) + first, quads);
        k_mx_quant_rows<T><<<grid, kThreads, 0, st>>>(x, a.R, a.stride_r, a.K, a.codes, a.scales, a.plan);
    } else {
        const dim3 grid(quads, static_cast<unsigned>(RT < 32768 ? RT : 32768) + first, static_cast<unsigned>(a.B));
        k_mx_quant<T><<<grid, kThreads, 0, st>>>(x, a.stride_b, a.R, a.stride_r, a.K, a.codes, a.scales, a.plan);
    }
    return hipGetLastError();
}

template <typename T>
hipError_t dequant(const uint8_t* codes, const uint8_t* scales, int64_t B, int64_t R, int64_t K, void* y, hipStream_t st) {
    const int64_t RT = mx_row_tiles(R);
    const dim3 grid(static_cast<unsigned>(mx_quads(K)), static_cast<unsigned>(RT < 32768 ? RT : 32768), static_cast<unsigned>(B));
    k_mx_dequant<T><<<grid, kThreads, 0, st>>>(codes, scales, R, static_cast<int>(K), static_cast<T*>(y));
    return hipGetLastError();
}

}  // namespace

hipError_t launch_mx_quant(const MxQuantArgs& a, hipStream_t st) {
    switch (a.dtype) {
        case MQ_F32: return quant<float>(a, st);
        case MQ_BF16: return quant<__bf16>(a, st);
        default: return quant<_Float16>(a, st);
    }
}

hipError_t launch_mx_dequant(const uint8_t* codes, const uint8_t* scales, int64_t B, int64_t R, int64_t K, void* y,
                             int y_dtype, hipStream_t st) {
    switch (y_dtype) {
        case MQ_F32: return dequant<float>(codes, scales, B, R, K, y, st);
        case MQ_BF16: return dequant<__bf16>(codes, scales, B, R, K, y, st);
        default: return dequant<_Float16>(codes, scales, B, R, K, y, st);
    }
}

}  // namespace mq
