// Products of microscaled 4-bit operands on the scaled 16x16x128 matrix instruction.
//
// y[m][n] = sum over blocks b of 32 inputs of Xx[m][b] Xw[n][b] * sum over the block of
// the 4-bit codes' products. The instruction takes the codes and one scale byte per lane
// (a lane holds one row's block) and adds into fp32.
#include "mx_device.h"
#include "mx_internal.h"

namespace mq {
namespace {

// c += A B^T over one 128-input tile; scale bytes at byte S of sa and sb
template <int S>
__device__ inline mx_f4 mfma16(mx_i4 a, mx_i4 b, mx_f4 c, int sa, int sb) {
    const mx_i8 a8 = {a[0], a[1], a[2], a[3], 0, 0, 0, 0}, b8 = {b[0], b[1], b[2], b[3], 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a8, b8, c, 4, 4, S, sa, S, sb);
}

template <int S, int NT>
__device__ inline void step16(const uint8_t* const (&w)[NT], const uint8_t* x, int g, const int (&sw)[NT], int sx,
                              mx_f4 (&acc)[NT]) {
    const mx_i4 b = *reinterpret_cast<const mx_i4*>(x + static_cast<int64_t>(g) * 1024);
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        const mx_i4 a = *reinterpret_cast<const mx_i4*>(w[i] + static_cast<int64_t>(g) * 1024);
        acc[i] = mfma16<S>(a, b, acc[i], sw[i], sx);
    }
}

// expert of a plan's row tile, or -1 past the last expert's rows
__device__ inline int expert_of(const int32_t* offsets, int E, int row) {
    int lo = 0, hi = E;                 // offsets[lo] <= row < offsets[hi]
    if (row >= offsets[E]) return -1;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (offsets[mid] <= row) lo = mid; else hi = mid;
    }
    return lo;
}

__device__ inline float silu(float g) { return g / (1.0f + __expf(-g)); }

// One wave: 16 rows x 64 columns (32 of gate and 32 of up). Weights are the A operand,
// so a lane ends with four neighbouring columns of one row.
template <typename T, bool GATED>
__global__ __launch_bounds__(64) void k_mx_gemm(MxGemmArgs a) {
    constexpr int NT = 4;
    constexpr int NC = GATED ? 2 : 4;                // 16-column tiles of the output
    const int lane = threadIdx.x;
    const int G = (a.K + 127) / 128, G4 = (G + 3) / 4;
    const int NTiles = (a.N + 15) / 16;
    const int rt = blockIdx.y, ct = blockIdx.x * NC;
    const int m = rt * 16 + (lane & 15);
    T* y = static_cast<T*>(a.y);
    int e = 0;
    bool live = m < a.M;
    if (a.offsets) {
        e = expert_of(a.offsets, a.E, rt * 16);
        live = live && e >= 0 && (!a.row_token || static_cast<unsigned>(a.row_token[m]) < static_cast<unsigned>(a.T));
    }
    mx_f4 acc[NT] = {};
    if (e >= 0) {
        const uint8_t *w[NT], *ws[NT];
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            const int c = GATED ? i >> 1 : i;
            const int tile = ct + c < NTiles ? ct + c : NTiles - 1;
            const int64_t at = static_cast<int64_t>(e) * NTiles + tile;
            w[i] = ((GATED && (i & 1)) ? a.w2q : a.wq) + at * G * 1024 + lane * 16;
            ws[i] = ((GATED && (i & 1)) ? a.w2s : a.ws) + at * G4 * 256 + lane * 4;
        }
        const uint8_t* x = a.xq + static_cast<int64_t>(rt) * G * 1024 + lane * 16;
        const uint8_t* xs = a.xs + static_cast<int64_t>(rt) * G4 * 256 + lane * 4;
        for (int q = 0; q < G4; ++q) {
            int sw[NT];
#pragma unroll
            for (int i = 0; i < NT; ++i) sw[i] = *reinterpret_cast<const int*>(ws[i] + q * 256);
            const int sx = *reinterpret_cast<const int*>(xs + q * 256);
            const int g = 4 * q;
            step16<0>(w, x, g, sw, sx, acc);
            if (g + 1 < G) step16<1>(w, x, g + 1, sw, sx, acc);
            if (g + 2 < G) step16<2>(w, x, g + 2, sw, sx, acc);
            if (g + 3 < G) step16<3>(w, x, g + 3, sw, sx, acc);
        }
    }
    if (m >= a.M) return;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int n = (ct + c) * 16 + 4 * (lane >> 4) + i;
            if (n >= a.N) continue;
            float v = GATED ? silu(acc[2 * c][i]) * acc[2 * c + 1][i] : acc[c][i];
            if (a.bias) v += a.bias[n];
            y[static_cast<int64_t>(m) * a.N + n] = mx_round<T>(live ? v : 0.0f);
        }
    }
}

template <typename T>
hipError_t gemm(const MxGemmArgs& a, hipStream_t st) {
    const unsigned rows = (a.M + 15) / 16, cols = (a.N + 15) / 16;
    if (a.w2q)
        k_mx_gemm<T, true><<<dim3((cols + 1) / 2, rows), 64, 0, st>>>(a);
    else
        k_mx_gemm<T, false><<<dim3((cols + 3) / 4, rows), 64, 0, st>>>(a);
    return hipGetLastError();
}

template <typename T>
__global__ __launch_bounds__(256) void k_combine(const float* rows, int64_t n_rows, const int32_t* row_of,
                                                 const float* weights, int64_t T_, int k, int64_t D, T* y) {
    const int64_t d = static_cast<int64_t>(blockIdx.y) * 256 + threadIdx.x;
    const int64_t t = blockIdx.x;
    if (d >= D) return;
    float acc = 0.0f;
    for (int j = 0; j < k; ++j) {
        const int p = row_of[t * k + j];
        const float r = p >= 0 && p < n_rows ? rows[p * D + d] : 0.0f;
        acc += weights[t * k + j] * r;
    }
    y[t * D + d] = mx_round<T>(acc);
}

template <typename T>
hipError_t combine(const float* rows, int64_t n_rows, const int32_t* row_of, const float* weights, int64_t T_, int k,
                   int64_t D, void* y, hipStream_t st) {
    k_combine<T><<<dim3(static_cast<unsigned>(T_), static_cast<unsigned>((D + 255) / 256)), 256, 0, st>>>(
        rows, n_rows, row_of, weights, T_, k, D, static_cast<T*>(y));
    return hipGetLastError();
}

}  // namespace

hipError_t launch_mx_gemm(const MxGemmArgs& a, hipStream_t st) {
    switch (a.y_dtype) {
        case MQ_F32: return gemm<float>(a, st);
        case MQ_BF16: return gemm<__bf16>(a, st);
        default: return gemm<_Float16>(a, st);
    }
}

hipError_t launch_combine(const float* rows, int64_t n_rows, const int32_t* row_of, const float* weights, int64_t T,
                          int k, int64_t D, void* y, int y_dtype, hipStream_t st) {
    switch (y_dtype) {
        case MQ_F32: return combine<float>(rows, n_rows, row_of, weights, T, k, D, y, st);
        case MQ_BF16: return combine<__bf16>(rows, n_rows, row_of, weights, T, k, D, y, st);
        default: return combine<_Float16>(rows, n_rows, row_of, weights, T, k, D, y, st);
    }
}

}  // namespace mq
