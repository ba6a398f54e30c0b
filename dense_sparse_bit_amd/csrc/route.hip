// Routing of tokens to experts, and the plan that orders a batch's rows by expert.
//
// score[e] = softmax or sigmoid of the logits. Experts are chosen by
// key[e] = score[e] + bias[e] (without a bias by the logit, whose order both scores
// keep), after only the best groups of experts are kept; ties go to the lower index.
// Scores and keys are held in 64 bits: experts are chosen by comparing them, and at 32
// bits two neighbouring experts swap with the rounding of the exponential.
#include <math.h>

#include <type_traits>

#include "mx_device.h"
#include "mx_internal.h"

namespace mq {
namespace {

constexpr int kMaxExperts = 1024;
constexpr int kTokens = 4;                 // tokens, one a wave, of a routing workgroup

// Reductions over a wave by lane moves within the vector unit: the result is in lane 63
// (row_shr 1, 2, 4, 8 within 16 lanes, then the last lanes of rows are added across).
template <int CTRL, int ROWS>
__device__ inline uint32_t moved(uint32_t v, uint32_t none) {
    return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(static_cast<int>(none), static_cast<int>(v), CTRL, ROWS, 0xf, false));
}
template <int CTRL, int ROWS>
__device__ inline double moved(double v) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint64_t m = static_cast<uint64_t>(moved<CTRL, ROWS>(static_cast<uint32_t>(b >> 32), 0)) << 32 |
                       moved<CTRL, ROWS>(static_cast<uint32_t>(b), 0);
    return __builtin_bit_cast(double, m);
}
__device__ inline uint32_t last_lane(uint32_t v) {
    return static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(v), 63));
}

__device__ inline uint32_t wave_max(uint32_t v) {
    v = max(v, moved<0x111, 0xf>(v, 0));
    v = max(v, moved<0x112, 0xf>(v, 0));
    v = max(v, moved<0x114, 0xf>(v, 0));
    v = max(v, moved<0x118, 0xf>(v, 0));
    v = max(v, moved<0x142, 0xa>(v, 0));
    v = max(v, moved<0x143, 0xc>(v, 0));
    return last_lane(v);
}

__device__ inline double wave_sum(double v) {
    v += moved<0x111, 0xf>(v);
    v += moved<0x112, 0xf>(v);
    v += moved<0x114, 0xf>(v);
    v += moved<0x118, 0xf>(v);
    v += moved<0x142, 0xa>(v);
    v += moved<0x143, 0xc>(v);
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    return __builtin_bit_cast(double, static_cast<uint64_t>(last_lane(static_cast<uint32_t>(b >> 32))) << 32 |
                                          last_lane(static_cast<uint32_t>(b)));
}

// Whole numbers in the order of the floating values (-0 as +0); 0 is below every value
// but NaN, which never gets here, and -inf has the least of the others' places.
__device__ inline uint32_t ordered(float v) {
    const uint32_t b = __float_as_uint(v + 0.0f);
    return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ inline uint64_t ordered(double v) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v + 0.0);
    return b ^ ((b >> 63) ? ~0ull : 1ull << 63);
}

// The first lane that holds the wave's largest key, or -1 where all keys are 0.
__device__ inline int first_best(uint32_t key) {
    const uint32_t top = wave_max(key);
    return top ? __builtin_ctzll(__ballot(key == top)) : -1;
}
__device__ inline int first_best(uint64_t key) {
    const uint32_t hi = static_cast<uint32_t>(key >> 32), top = wave_max(hi);
    const uint64_t some = __ballot(hi == top);
    if (top && !(some & (some - 1))) return __builtin_ctzll(some);      // most often one lane alone
    const uint32_t lo = hi == top ? static_cast<uint32_t>(key) : 0, low = wave_max(lo);
    return top || low ? __builtin_ctzll(__ballot(hi == top && lo == low)) : -1;
}

// One wave per token; lane l holds the experts V l .. V l + V - 1, so that the first
// lane, and in it the first expert, of a tie is the lowest index. BIAS: keys are scores
// with their bias, in 64 bits; else the logits themselves, and only the chosen experts'
// scores are computed (softmax: and the sum). A key of 0 is a masked expert. One token is
// bound by the latency of k rounds of a maximum over the wave: lane moves in the vector unit
// keep a round near 200 cycles (through LDS permutes, 64-bit values: 1500). Batches are bound
// by vector instructions, 64-bit exponentials and divisions most of all: 4096 tokens of 256
// experts in 8 groups, sigmoid and bias, take 983 a token, and the vector units are busy for
// 71% of the 11.7 us. One token of 128 experts: 3.5 us.
template <typename T, int V, bool BIAS>
__global__ __launch_bounds__(64 * kTokens) void k_route(RouteArgs a) {
    using Key = typename std::conditional<BIAS, uint64_t, uint32_t>::type;
    extern __shared__ __align__(16) double lds[];     // (groups) keys, and scores where they are computed
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * kTokens + wave; t < a.T; t += static_cast<int64_t>(gridDim.x) * kTokens) {
        const T* logits = static_cast<const T*>(a.logits) + t * a.stride_t;
        const bool softmax = a.score == MQ_SCORE_SOFTMAX;
        float x[V], bias[V];
        bool fault = false;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = min(lane * V + i, a.E - 1);      // lanes past the last expert: its values, masked
            x[i] = static_cast<float>(logits[e]);
            bias[i] = BIAS ? a.bias[e] : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if (lane * V + i >= a.E) x[i] = -INFINITY;
            fault |= !(x[i] == x[i]) || (softmax && x[i] == INFINITY);
        }
        double sum = 1.0, base = 0.0;
        double score[V];
        if (softmax) {
            float top = x[0];
#pragma unroll
            for (int i = 1; i < V; ++i) top = fmaxf(top, x[i]);
            const uint32_t best = wave_max(ordered(top));
            base = __uint_as_float(best ^ ((best >> 31) ? 0x80000000u : 0xffffffffu));
            if (!(base > -INFINITY)) base = 0.0;
            sum = 0.0;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                score[i] = exp(static_cast<double>(x[i]) - base);
                sum += score[i];
            }
            sum = wave_sum(sum);
            if (!(sum > 0.0)) sum = 1.0;
        }
        auto score_of = [&](float v) __attribute__((always_inline)) -> double {
            return softmax ? exp(static_cast<double>(v) - base) / sum : 1.0 / (1.0 + exp(-static_cast<double>(v)));
        };
        Key key[V];
        if constexpr (BIAS) {
            if (softmax) {
#pragma unroll
                for (int i = 0; i < V; ++i) score[i] /= sum;
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i) score[i] = 1.0 / (1.0 + exp(-static_cast<double>(x[i])));
            }
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const double v = x[i] == -INFINITY ? -HUGE_VAL : score[i] + static_cast<double>(bias[i]);
                fault |= !(v == v);
                key[i] = v == -HUGE_VAL ? 0 : ordered(v);
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) key[i] = x[i] == -INFINITY ? 0 : ordered(x[i]);
        }
        float* weights = a.weights + t * a.k;
        int32_t* ids = a.ids + t * a.k;
        if (__any(fault)) {
            // a NaN among the logits or biases: no expert, and weights that show it
            if (lane < a.k) { ids[lane] = -1; weights[lane] = NAN; }
            continue;
        }
        if (a.top_groups < a.groups) {
            // a run of lanes weighs a group, whose experts it finds in LDS: each lane the two
            // best of some, then the run's by exchanges (one lane a group: 1.2 us more, at
            // 4096 tokens of 8 groups of 32)
            const int per = a.E / a.groups;
            const bool two = a.group_score == MQ_GROUP_TOP2;
            const int shift = a.groups > 1 ? __builtin_clz(a.groups - 1) - 26 : 6, run = 1 << shift;
            const int group = lane >> shift;
            double* mine = lds + wave * 64 * V;
            mx_wave_sync();                              // the last token's reads come first
#pragma unroll
            for (int i = 0; i < V; ++i) {
                double v = -HUGE_VAL;
                if (key[i]) {
                    if constexpr (BIAS) v = score[i] + static_cast<double>(bias[i]);
                    else v = x[i];
                }
                mine[lane * V + i] = v;
            }
            mx_wave_sync();
            double first = -HUGE_VAL, second = -HUGE_VAL;
            if (group < a.groups) {
#pragma unroll 4
                for (int i = lane & (run - 1); i < per; i += run) {
                    const double v = mine[group * per + i];
                    if (v > first) { second = first; first = v; } else if (v > second) second = v;
                }
            }
            for (int o = 1; o < run; o <<= 1) {
                const double f = __shfl_xor(first, o);
                if (two) second = fmax(fmin(first, f), fmax(second, __shfl_xor(second, o)));
                first = fmax(first, f);
            }
            double worth = first;
            if (two && first > -HUGE_VAL) {
                if constexpr (BIAS) {
                    if (second > -HUGE_VAL) worth += second;
                } else {
                    worth = score_of(static_cast<float>(first)) + (second > -HUGE_VAL ? score_of(static_cast<float>(second)) : 0.0);
                }
            }
            const uint64_t wb = ordered(worth);
            int rank = 0;
            for (int g = 0; g < a.groups; ++g) {
                const uint64_t other = static_cast<uint64_t>(static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(wb >> 32), g << shift))) << 32 |
                                       static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(wb), g << shift));
                rank += other > wb || (other == wb && g < group);
            }
            const uint64_t keep = __ballot(rank < a.top_groups);         // a bit for each lane of a run
            const float share = 1.0f / per;
#pragma unroll
            for (int i = 0; i < V; ++i)                    // (e + 1/2) / per is never near a whole number
                if (!(keep >> ((static_cast<int>((lane * V + i + 0.5f) * share) << shift) & 63) & 1)) key[i] = 0;
        }
        int mine = -1;
        double w = 0.0;
        float logit = 0.0f;
        for (int j = 0; j < a.k; ++j) {
            Key best = key[0];
            int at = 0;
#pragma unroll
            for (int i = 1; i < V; ++i)
                if (key[i] > best) { best = key[i]; at = i; }
            const int from = first_best(best);
            if (from < 0) break;                           // no expert is left
            const int i0 = __builtin_amdgcn_readlane(at, from);
            if (lane == j) mine = from * V + i0;
            // the chosen expert's logit (its score, where scores are computed)
            double s = 0.0;
            float l = 0.0f;
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (i == i0) {
                    if constexpr (BIAS) s = score[i];
                    l = x[i];
                    if (lane == from) key[i] = 0;
                }
            if constexpr (BIAS) {
                const uint64_t b = __builtin_bit_cast(uint64_t, s);
                const uint64_t r = static_cast<uint64_t>(static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(b >> 32), from))) << 32 |
                                   static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(b), from));
                if (lane == j) w = __builtin_bit_cast(double, r);
            } else {
                const float r = __uint_as_float(static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(__float_as_uint(l)), from)));
                if (lane == j) logit = r;
            }
        }
        if constexpr (!BIAS) w = mine >= 0 ? score_of(logit) : 0.0;
        if (a.renormalize) {
            const double total = wave_sum(w);
            w = total > 0.0 ? w / total : 0.0;
        }
        if (lane < a.k) {
            ids[lane] = mine;
            weights[lane] = static_cast<float>(w * static_cast<double>(a.scale));
        }
    }
}

template <typename T, int V>
hipError_t route(const RouteArgs& a, hipStream_t st) {
    const int64_t wgs = (a.T + kTokens - 1) / kTokens;
    const unsigned grid = static_cast<unsigned>(wgs < (1 << 22) ? wgs : 1 << 22);
    const size_t lds = a.top_groups < a.groups ? kTokens * 64 * V * sizeof(double) : 0;
    if (a.bias) k_route<T, V, true><<<grid, 64 * kTokens, lds, st>>>(a);
    else k_route<T, V, false><<<grid, 64 * kTokens, lds, st>>>(a);
    return hipGetLastError();
}

template <typename T>
hipError_t route(const RouteArgs& a, hipStream_t st) {
    if (a.E <= 64) return route<T, 1>(a, st);
    if (a.E <= 128) return route<T, 2>(a, st);
    if (a.E <= 256) return route<T, 4>(a, st);
    if (a.E <= 512) return route<T, 8>(a, st);
    return route<T, 16>(a, st);
}

// ------------------------------------------------------------------- plan
constexpr int kPlanThreads = 1024;
constexpr int kPlanWaves = kPlanThreads / 64;

// Slots up to which a plan takes one launch. Measured, one / three, in us (64 and 1024
// experts): 2^15 slots 8.0 / 22.6 and 8.5 / 29.7, 2^17 17.7 / 22.3 and 17.3 / 30.8, 2^18 30.6 / 23.7
// and 30.1 / 33.2, 2^19 103 / 28 and 83 / 39.
constexpr int64_t kOneLaunchSlots = 1 << 18;

struct PlanLds {
    int before[kMaxExperts];                       // first the experts' counts, then their next rows
    int count[kMaxExperts];
    int first[kMaxExperts + 1];                    // offsets
    int wave_sum[kPlanWaves];
    unsigned short in_wave[kPlanWaves][kMaxExperts];
};

// first[] from count[]: each expert's rows, rounded up to 16, one after the other
__device__ void plan_scan(PlanLds& s) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    int n = (s.count[tid] + 15) & ~15;
    for (int o = 1; o < 64; o <<= 1) {
        const int v = __shfl_up(n, o);
        if (lane >= o) n += v;
    }
    if (lane == 63) s.wave_sum[wave] = n;
    __syncthreads();
    for (int w = 0; w < wave; ++w) n += s.wave_sum[w];
    s.first[tid + 1] = n;
    if (tid == 0) s.first[0] = 0;
    __syncthreads();
}

// Rows for the slots [from, to), in their order: a slot's row is its expert's next row
// (before[], which moves on) plus the slots of the same expert before it among the
// workgroup's 1024: in its wave by comparing ids bit by bit across the lanes, in earlier
// waves by their counts.
__device__ void plan_place(const PlanArgs& a, PlanLds& s, int64_t from, int64_t to) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int bits = 32 - __builtin_clz(a.E);       // ids 0 .. E (E: no expert)
    const int rows = static_cast<int>(a.rows);
    for (int64_t i0 = from; i0 < to; i0 += kPlanThreads) {
        for (int i = tid; i < kPlanWaves * kMaxExperts / 2; i += kPlanThreads)
            if ((i & (kMaxExperts / 2 - 1)) * 2 < a.E) reinterpret_cast<uint32_t*>(s.in_wave)[i] = 0;
        __syncthreads();
        const int64_t i = i0 + tid;
        int e = a.E;
        if (i < to) {
            e = a.ids[i];
            if (e < 0 || e >= a.E) e = a.E;
        }
        unsigned long long same = ~0ull;
        for (int b = 0; b < bits; ++b) {
            const unsigned long long m = __ballot(e >> b & 1);
            same &= (e >> b & 1) ? m : ~m;
        }
        const int rank = __popcll(same & ((1ull << lane) - 1));
        if (e < a.E && rank == 0) s.in_wave[wave][e] = static_cast<unsigned short>(__popcll(same));
        __syncthreads();
        if (i < to) {
            int row = -1;
            if (e < a.E) {
                row = s.before[e] + rank;
                for (int w = 0; w < wave; ++w) row += s.in_wave[w][e];
                if (row < rows) a.row_token[row] = static_cast<int32_t>(i / a.k);
            }
            a.row_of[i] = row;
        }
        __syncthreads();
        if (i0 + kPlanThreads < to && tid < a.E) {
            int n = 0;
            for (int w = 0; w < kPlanWaves; ++w) n += s.in_wave[w][tid];
            s.before[tid] += n;
        }
        __syncthreads();                              // before the counts are cleared
    }
}

// offsets, and the rows of no token after each expert's last (fewer than 16); shared out
// over the grid
__device__ void plan_ends(const PlanArgs& a, const PlanLds& s) {
    const int tid = threadIdx.x;
    if (blockIdx.x == 0) {
        if (tid < a.E) a.offsets[tid] = s.first[tid];
        if (tid == 0) a.offsets[a.E] = s.first[a.E];
    }
    for (int i = blockIdx.x * kPlanThreads + tid; i < a.E * 16; i += gridDim.x * kPlanThreads) {
        const int row = s.first[i >> 4] + s.count[i >> 4] + (i & 15);
        if (row < s.first[(i >> 4) + 1]) a.row_token[row] = -1;
    }
}

// the rows after the last expert's
__device__ void plan_tail(const PlanArgs& a, int64_t end) {
    const int64_t step = static_cast<int64_t>(gridDim.x) * kPlanThreads;
    for (int64_t r = end + static_cast<int64_t>(blockIdx.x) * kPlanThreads + threadIdx.x; r < a.rows; r += step) a.row_token[r] = -1;
}

// One launch: workgroup b counts the ids of all slots, and of those before its own 1024,
// which it then places. The ids are read once a workgroup, from L2, and counted by LDS
// atomics (whose order changes nothing), which take most of the time: 8 slots 4.1 us, 32768
// slots of 256 experts 8.2 us.
__global__ __launch_bounds__(kPlanThreads) void k_plan(PlanArgs a) {
    __shared__ PlanLds s;
    const int tid = threadIdx.x;
    s.before[tid] = 0;
    s.count[tid] = 0;
    __syncthreads();
    const int n = static_cast<int>(a.T * a.k), from = blockIdx.x * kPlanThreads;
    for (int i0 = tid; i0 < n; i0 += 8 * kPlanThreads) {
        int e[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) e[j] = i0 + j * kPlanThreads < n ? a.ids[i0 + j * kPlanThreads] : -1;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (e[j] >= 0 && e[j] < a.E) atomicAdd(i0 + j * kPlanThreads < from ? &s.before[e[j]] : &s.count[e[j]], 1);
    }
    __syncthreads();
    s.count[tid] += s.before[tid];
    __syncthreads();
    plan_scan(s);
    s.before[tid] += s.first[tid];
    __syncthreads();
    plan_ends(a, s);
    plan_tail(a, s.first[a.E]);
    plan_place(a, s, from, min(from + kPlanThreads, n));
}

// Many slots: chunks of `chunk` slots (the last up to twice that) are counted, the
// counts summed over the chunks, and the chunks placed. A chunk's counts lie at the
// start of its own part of row_of until it is placed (chunk >= kMaxExperts).
__global__ __launch_bounds__(kPlanThreads) void k_plan_count(PlanArgs a, int64_t chunk) {
    __shared__ int count[kMaxExperts];
    const int tid = threadIdx.x;
    count[tid] = 0;
    __syncthreads();
    const int64_t n = a.T * a.k, from = blockIdx.x * chunk, to = blockIdx.x + 1 == gridDim.x ? n : from + chunk;
    for (int64_t i = from + tid; i < to; i += kPlanThreads) {
        const int e = a.ids[i];
        if (e >= 0 && e < a.E) atomicAdd(&count[e], 1);
    }
    __syncthreads();
    if (tid < a.E) a.row_of[from + tid] = count[tid];
}

__global__ __launch_bounds__(kPlanThreads) void k_plan_sum(PlanArgs a, int64_t chunk, int chunks) {
    __shared__ PlanLds s;
    const int tid = threadIdx.x;
    int n = 0;
    if (tid < a.E) {
#pragma unroll 8
        for (int c = 0; c < chunks; ++c) n += a.row_of[c * chunk + tid];
    }
    s.count[tid] = n;
    __syncthreads();
    plan_scan(s);
    plan_ends(a, s);
    if (tid < a.E) {
        int row = s.first[tid];
        for (int c = 0; c < chunks; ++c) {
            const int here = a.row_of[c * chunk + tid];
            a.row_of[c * chunk + tid] = row;
            row += here;
        }
    }
}

__global__ __launch_bounds__(kPlanThreads) void k_plan_chunks(PlanArgs a, int64_t chunk) {
    __shared__ PlanLds s;
    const int tid = threadIdx.x;
    const int64_t n = a.T * a.k, from = blockIdx.x * chunk, to = blockIdx.x + 1 == gridDim.x ? n : from + chunk;
    if (tid < a.E) s.before[tid] = a.row_of[from + tid];
    __syncthreads();
    plan_place(a, s, from, to);
    plan_tail(a, a.offsets[a.E]);
}

}  // namespace

hipError_t launch_route(const RouteArgs& a, hipStream_t st) {
    switch (a.dtype) {
        case MQ_F32: return route<float>(a, st);
        case MQ_BF16: return route<__bf16>(a, st);
        default: return route<_Float16>(a, st);
    }
}

hipError_t launch_plan(const PlanArgs& a, hipStream_t st) {
    const int64_t n = a.T * a.k;
    if (n <= kOneLaunchSlots) {
        k_plan<<<static_cast<unsigned>(n ? (n + kPlanThreads - 1) / kPlanThreads : 1), kPlanThreads, 0, st>>>(a);
        return hipGetLastError();
    }
    // at most 1024 chunks: their counts are summed by one workgroup
    int64_t chunk = 8 * kPlanThreads;
    while (n / chunk > 1024) chunk *= 2;
    const int chunks = static_cast<int>(n / chunk);
    k_plan_count<<<chunks, kPlanThreads, 0, st>>>(a, chunk);
    k_plan_sum<<<1, kPlanThreads, 0, st>>>(a, chunk, chunks);
    k_plan_chunks<<<chunks, kPlanThreads, 0, st>>>(a, chunk);
    return hipGetLastError();
}

}  // namespace mq
