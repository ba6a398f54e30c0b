// Tokens to the rows of their experts and back, over a plan.
//
// Both go token by token: a token's row is in registers once while its k rows are written
// (gather) or read (combine). Nothing is computed beyond a product per element, so both are
// bound by memory: (T + P) D elements of gather, (T k + T) D of combine, and the same again
// of `other` where the dots are wanted.
#include "w4_device.h"
#include "w4_internal.h"

namespace mq {
namespace {

constexpr int kThreads = 256;
constexpr int kSlots = 8;                              // slots of a token that are in flight together

// Sums over the workgroup of each thread's n <= kSlots values; thread i < n has the i-th.
__device__ __forceinline__ float sums(const float (&v)[kSlots], int n, float* lds) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int j = 0; j < kSlots; ++j) {
        float s = v[j];
        for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o);
        if (lane == 0) lds[wave * kSlots + j] = s;
    }
    __syncthreads();
    float s = 0;
    if (static_cast<int>(threadIdx.x) < n)
        for (int w = 0; w < kThreads / 64; ++w) s += lds[w * kSlots + threadIdx.x];
    __syncthreads();
    return s;
}

// Workgroups (y): the tokens, then one for every 16 rows of the plan, which zeroes those of
// no token. DOTS: a workgroup takes a token's whole row; else (x) 8 inputs a thread of it.
template <typename XT, typename RT, bool DOTS>
__global__ __launch_bounds__(kThreads) void k_gather(RowsArgs a) {
    __shared__ float lds[kThreads / 64 * kSlots];
    RT* const rows = static_cast<RT*>(const_cast<void*>(a.rows));
    const int first = DOTS ? 0 : blockIdx.x * kThreads * 8, end = DOTS ? a.D : min(a.D, first + kThreads * 8);
    const int64_t blocks = a.T + (a.P + 15) / 16;
    for (int64_t t = blockIdx.y; t < blocks; t += gridDim.y) {
        if (t >= a.T) {
            const float none[8] = {};
            for (int64_t p = (t - a.T) * 16; p < min(a.P, (t - a.T) * 16 + 16); ++p) {
                if (static_cast<uint64_t>(static_cast<int64_t>(a.row_token[p])) < static_cast<uint64_t>(a.T)) continue;
                for (int d = first + 8 * threadIdx.x; d < end; d += kThreads * 8) w4_store8(rows + p * a.D + d, a.D - d, none);
            }
            continue;
        }
        const XT* const x = static_cast<const XT*>(a.x) + t * a.stride_t;
        for (int j0 = 0; j0 < a.k; j0 += kSlots) {
            const int n = min(kSlots, a.k - j0);
            float dot[kSlots] = {};
            for (int d = first + 8 * threadIdx.x; d < end; d += kThreads * 8) {
                float v[8];
                w4_values(mx_load8(x + d, a.D - d), v);
#pragma unroll
                for (int j = 0; j < kSlots; ++j) {
                    if (j >= n) break;
                    const int64_t p = a.row_of[t * a.k + j0 + j];
                    if (p < 0 || p >= a.P) continue;
                    const float f = a.weights ? a.weights[t * a.k + j0 + j] : 1.0f;
                    float r[8];
                    if constexpr (DOTS) {
                        w4_values(mx_load8(static_cast<const RT*>(a.other) + p * a.D + d, a.D - d), r);
#pragma unroll
                        for (int i = 0; i < 8; ++i) dot[j] += v[i] * r[i];
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) r[i] = f * v[i];
                    w4_store8(rows + p * a.D + d, a.D - d, r);
                }
            }
            if constexpr (DOTS) {
                const float s = sums(dot, n, lds);
                if (static_cast<int>(threadIdx.x) < n) a.dots[t * a.k + j0 + threadIdx.x] = s;
            }
        }
    }
}

template <typename XT, typename RT, bool DOTS>
__global__ __launch_bounds__(kThreads) void k_combine(RowsArgs a) {
    __shared__ float lds[kThreads / 64 * kSlots];
    const int first = DOTS ? 0 : blockIdx.x * kThreads * 8, end = DOTS ? a.D : min(a.D, first + kThreads * 8);
    const RT* const rows = static_cast<const RT*>(a.rows);
    for (int64_t t = blockIdx.y; t < a.T; t += gridDim.y) {
        XT* const x = static_cast<XT*>(const_cast<void*>(a.x)) + t * a.stride_t;
        for (int j0 = 0; DOTS && j0 < a.k; j0 += kSlots) {
            const int n = min(kSlots, a.k - j0);
            float dot[kSlots] = {};
            for (int d = 8 * threadIdx.x; d < a.D; d += kThreads * 8) {
                float v[8];
                w4_values(mx_load8(static_cast<const XT*>(a.other) + t * a.stride_o + d, a.D - d), v);
#pragma unroll
                for (int j = 0; j < kSlots; ++j) {
                    if (j >= n) break;
                    const int64_t p = a.row_of[t * a.k + j0 + j];
                    if (p < 0 || p >= a.P) continue;
                    float r[8];
                    w4_values(mx_load8(rows + p * a.D + d, a.D - d), r);
#pragma unroll
                    for (int i = 0; i < 8; ++i) dot[j] += v[i] * r[i];
                }
            }
            const float s = sums(dot, n, lds);
            if (static_cast<int>(threadIdx.x) < n) a.dots[t * a.k + j0 + threadIdx.x] = s;
        }
        for (int d = first + 8 * threadIdx.x; d < end; d += kThreads * 8) {
            float sum[8] = {};
            for (int j = 0; j < a.k; ++j) {
                const int64_t p = a.row_of[t * a.k + j];
                const float f = a.weights ? a.weights[t * a.k + j] : 1.0f;
                float r[8] = {};
                if (p >= 0 && p < a.P) w4_values(mx_load8(rows + p * a.D + d, a.D - d), r);
#pragma unroll
                for (int i = 0; i < 8; ++i) sum[i] += f * r[i];
            }
            w4_store8(x + d, a.D - d, sum);
        }
    }
}

template <typename XT, typename RT>
hipError_t gather(const RowsArgs& a, hipStream_t st) {
    const int64_t blocks = a.T + (a.P + 15) / 16;
    const unsigned y = static_cast<unsigned>(blocks < 65535 ? blocks : 65535);
    if (a.dots) k_gather<XT, RT, true><<<dim3(1, y), kThreads, 0, st>>>(a);
    else k_gather<XT, RT, false><<<dim3((a.D + kThreads * 8 - 1) / (kThreads * 8), y), kThreads, 0, st>>>(a);
    return hipGetLastError();
}

template <typename XT, typename RT>
hipError_t combine(const RowsArgs& a, hipStream_t st) {
    const unsigned y = static_cast<unsigned>(a.T < 65535 ? a.T : 65535);
    if (a.dots) k_combine<XT, RT, true><<<dim3(1, y), kThreads, 0, st>>>(a);
    else k_combine<XT, RT, false><<<dim3((a.D + kThreads * 8 - 1) / (kThreads * 8), y), kThreads, 0, st>>>(a);
    return hipGetLastError();
}

// f<tokens' type, rows' type>
template <typename F>
hipError_t with_types(const RowsArgs& a, F f) {
    auto rows = [&](auto x) {
        switch (a.rows_dtype) {
            case MQ_F32: return f(x, 0.0f);
            case MQ_BF16: return f(x, __bf16{});
            default: return f(x, _Float16{});
        }
    };
    switch (a.x_dtype) {
        case MQ_F32: return rows(0.0f);
        case MQ_BF16: return rows(__bf16{});
        default: return rows(_Float16{});
    }
}

}  // namespace

hipError_t launch_rows_gather(const RowsArgs& a, hipStream_t st) {
    return with_types(a, [&](auto x, auto r) { return gather<decltype(x), decltype(r)>(a, st); });
}

hipError_t launch_rows_combine(const RowsArgs& a, hipStream_t st) {
    return with_types(a, [&](auto x, auto r) { return combine<decltype(x), decltype(r)>(a, st); });
}

}  // namespace mq
