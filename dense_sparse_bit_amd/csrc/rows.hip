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

// Eight columns of row p from d on as bits that `there` lets through; not by a branch where the
// columns are whole units of eight (p of no row: any row of the memory, its bits cut off).
// Rows are read once: past the caches (60.0 us with them, 56.5 without).
template <bool V> struct Whole { static constexpr bool value = V; };
template <bool WHOLE, typename RT>
__device__ __forceinline__ MxRaw8<RT> row8(const RT* rows, int64_t p, bool there, int D, int d) {
    const RT* const from = rows + (there ? p : 0) * D + d;
    MxRaw8<RT> r;
    if constexpr (!WHOLE) {
        r = mx_load8(from, D - d);
    } else if constexpr (sizeof(RT) == 4) {
        typedef float Words __attribute__((ext_vector_type(4), aligned(4)));
        const Words lo = __builtin_nontemporal_load(reinterpret_cast<const Words*>(from));
        const Words hi = __builtin_nontemporal_load(reinterpret_cast<const Words*>(from) + 1);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            r.v[i] = lo[i];
            r.v[4 + i] = hi[i];
        }
    } else {
        typedef uint32_t Words __attribute__((ext_vector_type(4), aligned(2)));
        const Words w = __builtin_nontemporal_load(reinterpret_cast<const Words*>(from));
#pragma unroll
        for (int i = 0; i < 4; ++i) r.w[i] = w[i];
    }
    const uint32_t mask = there ? ~0u : 0;
    if constexpr (sizeof(RT) == 4) {
#pragma unroll
        for (int i = 0; i < 8; ++i) r.v[i] = __uint_as_float(__float_as_uint(r.v[i]) & mask);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) r.w[i] &= mask;
    }
    return r;
}

// Workgroups (y): the tokens, then one for every 16 rows of the plan, which zeroes those of
// no token. DOTS: a workgroup takes a token's whole row, and loads its rows of `other` before the
// first is used; else (x) 8 columns a thread of it. 4096 tokens of 8 slots, 4096 columns of bf16: 58 us
// (5.2 TB/s; 77 to rows that no cache holds any of), with dots 117 (4.9 TB/s). Narrow rows leave lanes
// idle: 8192 tokens, 64 / 512 / 1024 columns 19 / 28 / 41 us, where their bytes take 1.8 / 15 / 29.
template <typename XT, typename RT, bool DOTS>
__global__ __launch_bounds__(kThreads) void k_gather(RowsArgs a) {
    __shared__ float lds[kThreads / 64 * kSlots];
    RT* const rows = static_cast<RT*>(const_cast<void*>(a.rows));
    const RT* const other = static_cast<const RT*>(a.other);
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
            const int32_t* const row_of = a.row_of + t * a.k + j0;
            const float* const weights = a.weights ? a.weights + t * a.k + j0 : nullptr;
            float dot[kSlots] = {};
            auto columns = [&](auto whole, int d) __attribute__((always_inline)) {
                constexpr bool kWhole = decltype(whole)::value;
                MxRaw8<RT> raw[kSlots];
                float v[8], r[8];
                const MxRaw8<XT> mine = mx_load8(x + d, kWhole ? 8 : a.D - d);
                if constexpr (DOTS) {
#pragma unroll
                    for (int j = 0; j < kSlots; ++j) {
                        const int64_t p = row_of[min(j, n - 1)];
                        raw[j] = row8<kWhole>(other, p, j < n && p >= 0 && p < a.P, a.D, d);
                    }
                }
                w4_values(mine, v);
#pragma unroll
                for (int j = 0; j < kSlots; ++j) {
                    if (j >= n) break;
                    const int64_t p = row_of[j];
                    if (p < 0 || p >= a.P) continue;
                    if constexpr (DOTS) {
                        w4_values(raw[j], r);
#pragma unroll
                        for (int i = 0; i < 8; ++i) dot[j] += v[i] * r[i];
                    }
                    const float f = weights ? weights[j] : 1.0f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) r[i] = f * v[i];
                    w4_store8(rows + p * a.D + d, kWhole ? 8 : a.D - d, r);
                }
            };
            for (int d = first + 8 * threadIdx.x; d < end; d += kThreads * 8) {
                if (a.D % 8 == 0) columns(Whole<true>{}, d);
                else columns(Whole<false>{}, d);
            }
            if constexpr (DOTS) {
                const float s = sums(dot, n, lds);
                if (static_cast<int>(threadIdx.x) < n) a.dots[t * a.k + j0 + threadIdx.x] = s;
            }
        }
    }
}

// Workgroups (y): the tokens. The rows of up to SLOTS (2, 4 or 8) slots are loaded before the
// first is added: 4096 tokens of 8 slots and 4096 columns 57 us (65 from rows that no cache
// holds), with each row added as it comes 76; 8192 tokens, 64 / 512 / 1024 columns 15 / 20 / 35 us.
// DOTS: a workgroup takes a token's whole row, and each of its rows serves the sum and the dot (k <=
// SLOTS; with more slots they are read twice); else (x) 8 columns a thread of it.
template <typename XT, typename RT, int SLOTS, bool DOTS>
__global__ __launch_bounds__(kThreads) void k_combine(RowsArgs a) {
    __shared__ float lds[kThreads / 64 * kSlots];
    const int first = DOTS ? 0 : blockIdx.x * kThreads * 8, end = DOTS ? a.D : min(a.D, first + kThreads * 8);
    const RT* const rows = static_cast<const RT*>(a.rows);
    for (int64_t t = blockIdx.y; t < a.T; t += gridDim.y) {
        XT* const x = static_cast<XT*>(const_cast<void*>(a.x)) + t * a.stride_t;
        const int32_t* const row_of = a.row_of + t * a.k;
        const float* const weights = a.weights ? a.weights + t * a.k : nullptr;
        // the sums (and, with `both`, the dots) of the slots j0 .. j0 + SLOTS - 1
        auto slots = [&](auto whole, int j0, int d, const float (&v)[8], float (&sum)[8], float (&dot)[kSlots]) __attribute__((always_inline)) {
            MxRaw8<RT> raw[SLOTS];
            float f[SLOTS];
#pragma unroll
            for (int j = 0; j < SLOTS; ++j) {
                const int jj = min(j0 + j, a.k - 1);
                const int64_t p = row_of[jj];
                f[j] = j0 + j < a.k ? (weights ? weights[jj] : 1.0f) : 0.0f;
                raw[j] = row8<decltype(whole)::value>(rows, p, j0 + j < a.k && p >= 0 && p < a.P, a.D, d);
            }
#pragma unroll
            for (int j = 0; j < SLOTS; ++j) {
                float r[8];
                w4_values(raw[j], r);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    sum[i] += f[j] * r[i];
                    if constexpr (DOTS) dot[j] += v[i] * r[i];
                }
            }
        };
        auto put_dots = [&](const float (&dot)[kSlots], int j0) __attribute__((always_inline)) {
            const int j = j0 + threadIdx.x, n = min(SLOTS, a.k - j0);
            const float s = sums(dot, n, lds);
            if (static_cast<int>(threadIdx.x) < n) a.dots[t * a.k + j] = row_of[j] >= 0 && row_of[j] < a.P ? s : 0.0f;
        };
        auto other8 = [&](int d, float (&v)[8]) __attribute__((always_inline)) {
            if constexpr (DOTS) w4_values(mx_load8(static_cast<const XT*>(a.other) + t * a.stride_o + d, a.D - d), v);
        };
        if (DOTS && a.k > SLOTS) {
            for (int j0 = 0; j0 < a.k; j0 += SLOTS) {
                float dot[kSlots] = {}, none[8] = {};
                for (int d = 8 * threadIdx.x; d < a.D; d += kThreads * 8) {
                    float v[8];
                    other8(d, v);
                    slots(Whole<false>{}, j0, d, v, none, dot);
                }
                put_dots(dot, j0);
            }
        }
        float dot[kSlots] = {};
        for (int d = first + 8 * threadIdx.x; d < end; d += kThreads * 8) {
            float sum[8] = {}, v[8] = {};
            other8(d, v);
            if (a.D % 8 == 0) {
                for (int j0 = 0; j0 < a.k; j0 += SLOTS) slots(Whole<true>{}, j0, d, v, sum, dot);
            } else {
                for (int j0 = 0; j0 < a.k; j0 += SLOTS) slots(Whole<false>{}, j0, d, v, sum, dot);
            }
            w4_store8(x + d, a.D - d, sum);
        }
        if (DOTS && a.k <= SLOTS) put_dots(dot, 0);
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

template <typename XT, typename RT, int SLOTS>
hipError_t combine_slots(const RowsArgs& a, hipStream_t st) {
    const unsigned y = static_cast<unsigned>(a.T < 65535 ? a.T : 65535);
    if (a.dots) k_combine<XT, RT, SLOTS, true><<<dim3(1, y), kThreads, 0, st>>>(a);
    else k_combine<XT, RT, SLOTS, false><<<dim3((a.D + kThreads * 8 - 1) / (kThreads * 8), y), kThreads, 0, st>>>(a);
    return hipGetLastError();
}

template <typename XT, typename RT>
hipError_t combine(const RowsArgs& a, hipStream_t st) {
    if (a.k <= 2) return combine_slots<XT, RT, 2>(a, st);
    return a.k <= 4 ? combine_slots<XT, RT, 4>(a, st) : combine_slots<XT, RT, 8>(a, st);
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
