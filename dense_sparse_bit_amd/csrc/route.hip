// Routing of tokens to experts, and the plan that orders a batch's rows by expert.
//
// score[e] = softmax or sigmoid of the logits. Experts are chosen by
// key[e] = score[e] + bias[e] (without a bias by the logit, whose order both scores
// keep), after only the best groups of experts are kept; ties go to the lower index.
// Scores and keys are held in 64 bits: experts are chosen by comparing them, and at 32
// bits two neighbouring experts swap with the rounding of the exponential.
#include <math.h>

#include "mx_device.h"
#include "mx_internal.h"

namespace mq {
namespace {

constexpr int kMaxExperts = 1024;
constexpr int kMaxGroups = 64;

__device__ inline double wave_sum(double v) {
    for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o);
    return v;
}

__device__ inline double wave_max(double v) {
    for (int o = 32; o; o >>= 1) v = fmax(v, __shfl_xor(v, o));
    return v;
}

// largest key of the wave and its lowest index
__device__ inline void wave_best(double& v, int& i) {
    for (int o = 32; o; o >>= 1) {
        const double v2 = __shfl_xor(v, o);
        const int i2 = __shfl_xor(i, o);
        if (v2 > v || (v2 == v && i2 < i)) { v = v2; i = i2; }
    }
}

// One wave per token; lane l holds the experts l, l + 64, ...
template <typename T, int V>
__global__ __launch_bounds__(64) void k_route(RouteArgs a) {
    __shared__ double lds_key[64 * V];
    __shared__ double lds_score[64 * V];
    __shared__ int lds_keep[kMaxGroups];
    const int lane = threadIdx.x;
    const int64_t t = blockIdx.x;
    const T* logits = static_cast<const T*>(a.logits) + t * a.stride_t;
    const double none = -HUGE_VAL;
    double x[V], score[V], key[V];
    double top = none;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = lane + 64 * i;
        x[i] = e < a.E ? static_cast<double>(static_cast<float>(logits[e])) : none;
        top = fmax(top, x[i]);
    }
    double sum = 0.0;
    bool fault = false;
    if (a.score == MQ_SCORE_SOFTMAX) {
        top = wave_max(top);
        const double base = top == none ? 0.0 : top;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            score[i] = exp(x[i] - base);     // 0 for a masked expert, NaN for a NaN or +inf logit
            sum += score[i];
        }
        sum = wave_sum(sum);
        const double inv = sum > 0.0 ? sum : 1.0;
#pragma unroll
        for (int i = 0; i < V; ++i) score[i] /= inv;
        fault = !(sum == sum);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            score[i] = 1.0 / (1.0 + exp(-x[i]));
            fault |= !(score[i] == score[i]);
        }
    }
    fault = __any(fault);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = lane + 64 * i;
        key[i] = x[i];
        if (a.bias && e < a.E) {
            key[i] = x[i] == none ? none : score[i] + static_cast<double>(a.bias[e]);
            fault |= !(key[i] == key[i]);
        }
    }
    fault = __any(fault);
    float* weights = a.weights + t * a.k;
    int32_t* ids = a.ids + t * a.k;
    if (fault) {
        // a NaN among the logits or biases: no expert, and weights that show it
        if (lane < a.k) { ids[lane] = -1; weights[lane] = NAN; }
        return;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        lds_key[lane + 64 * i] = key[i];
        lds_score[lane + 64 * i] = score[i];
    }
    __syncthreads();
    if (a.top_groups < a.groups) {
        const int per = a.E / a.groups;
        double worth = none;
        if (lane < a.groups) {
            double first = none, second = none;
            for (int i = 0; i < per; ++i) {
                const int e = lane * per + i;
                double v = lds_key[e];
                if (v != none && a.group_score == MQ_GROUP_TOP2 && !a.bias) v = lds_score[e];
                if (v > first) { second = first; first = v; } else if (v > second) second = v;
            }
            worth = first;
            if (a.group_score == MQ_GROUP_TOP2 && second != none) worth += second;
        }
        int rank = 0;
        for (int g = 0; g < a.groups; ++g) {
            const double other = __shfl(worth, g);
            rank += other > worth || (other == worth && g < lane);
        }
        lds_keep[lane] = rank < a.top_groups;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = lane + 64 * i;
            if (e < a.E && !lds_keep[e / per]) key[i] = none;
        }
    }
    int mine = -1;
    for (int j = 0; j < a.k; ++j) {
        double best = none;
        int at = kMaxExperts * 2;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (key[i] > best) { best = key[i]; at = lane + 64 * i; }
        wave_best(best, at);
        const int e = best == none ? -1 : at;
        if (lane == j) mine = e;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (lane + 64 * i == e) key[i] = none;
    }
    double w = lane < a.k && mine >= 0 ? lds_score[mine] : 0.0;
    if (a.renormalize) {
        const double total = wave_sum(w);
        w = total > 0.0 ? w / total : 0.0;
    }
    if (lane < a.k) {
        ids[lane] = mine;
        weights[lane] = static_cast<float>(w * static_cast<double>(a.scale));
    }
}

template <typename T>
hipError_t route(const RouteArgs& a, hipStream_t st) {
    const unsigned grid = static_cast<unsigned>(a.T);
    if (a.E <= 64) k_route<T, 1><<<grid, 64, 0, st>>>(a);
    else if (a.E <= 128) k_route<T, 2><<<grid, 64, 0, st>>>(a);
    else if (a.E <= 256) k_route<T, 4><<<grid, 64, 0, st>>>(a);
    else if (a.E <= 512) k_route<T, 8><<<grid, 64, 0, st>>>(a);
    else k_route<T, 16><<<grid, 64, 0, st>>>(a);
    return hipGetLastError();
}

constexpr int kPlanThreads = 1024;

// Rows of each expert, and the experts' first rows. One workgroup.
__global__ __launch_bounds__(kPlanThreads) void k_plan_offsets(PlanArgs a) {
    __shared__ int count[kMaxExperts];
    __shared__ int scan[kMaxExperts];
    const int tid = threadIdx.x;
    count[tid] = 0;
    __syncthreads();
    const int64_t n = a.T * a.k;
    for (int64_t i = tid; i < n; i += kPlanThreads) {
        const int e = a.ids[i];
        if (e >= 0 && e < a.E) atomicAdd(&count[e], 1);
    }
    __syncthreads();
    const int own = (count[tid] + 15) & ~15;
    scan[tid] = own;
    for (int o = 1; o < kMaxExperts; o <<= 1) {
        __syncthreads();
        const int v = tid >= o ? scan[tid - o] : 0;
        __syncthreads();
        scan[tid] += v;
    }
    if (tid < a.E) a.offsets[tid + 1] = scan[tid];
    if (tid == 0) a.offsets[0] = 0;
}

// Workgroup e < E: the slots of expert e in order, each with the next row of e.
// Workgroup E: slots of no expert, and the rows after the last expert's.
__global__ __launch_bounds__(kPlanThreads) void k_plan_place(PlanArgs a) {
    __shared__ int wave_count[kPlanThreads / 64];
    const int e = blockIdx.x, tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
    const int64_t n = a.T * a.k;
    if (e == a.E) {
        for (int64_t i = tid; i < n; i += kPlanThreads)
            if (a.ids[i] < 0 || a.ids[i] >= a.E) a.row_of[i] = -1;
        for (int64_t r = a.offsets[a.E] + tid; r < a.rows; r += kPlanThreads) a.row_token[r] = -1;
        return;
    }
    int row = a.offsets[e];
    const int end = a.offsets[e + 1];
    for (int64_t i0 = 0; i0 < n && row < end; i0 += kPlanThreads) {
        const int64_t i = i0 + tid;
        const bool hit = i < n && a.ids[i] == e;
        const unsigned long long mask = __ballot(hit);
        if (lane == 0) wave_count[wave] = __popcll(mask);
        __syncthreads();
        int before = row, total = 0;
        for (int w = 0; w < kPlanThreads / 64; ++w) {
            if (w < wave) before += wave_count[w];
            total += wave_count[w];
        }
        if (hit) {
            const int r = before + __popcll(mask & ((1ull << lane) - 1));
            a.row_of[i] = r;
            a.row_token[r] = static_cast<int32_t>(i / a.k);
        }
        row += total;
        __syncthreads();
    }
    if (row + tid < end) a.row_token[row + tid] = -1;     // fewer than 16
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
    k_plan_offsets<<<1, kPlanThreads, 0, st>>>(a);
    k_plan_place<<<a.E + 1, kPlanThreads, 0, st>>>(a);
    return hipGetLastError();
}

}  // namespace mq
