// Row blocks of an expert plan, for products that take many rows at a time.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mx_internal.h"

namespace mq {

// By one workgroup of 256 threads: thread t counts the blocks (of at most BLOCK 16-row tiles, an
// even number) of the entries 4t .. 4t + 3 (experts, and one for the rows after the last's), whose
// sums give each entry its place. It goes with a launch over the rows, which takes longer: a
// launch of its own took 5 us.
constexpr int kTilesLds = 1024 + 256 / 64 + 1;
template <int BLOCK>
__device__ void plan_tiles(const MxTilesArgs& p, int* lds) {
    int* const last = lds;                     // blocks up to and with entry i; then waves' sums
    const int tid = threadIdx.x, lane = tid & 63;
    auto start = [&](int e) { return min(max(p.offsets[e] >> 4, 0), p.P16); };
    auto end = [&](int e) { return e < p.E ? start(e + 1) : p.P16; };
    int n[4], sum = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int e = 4 * tid + i, c = e <= p.E ? end(e) - start(e) : 0;
        n[i] = sum += c > 0 ? (c + BLOCK - 1) / BLOCK : 0;
    }
    for (int o = 1; o < 64; o <<= 1) {
        const int v = __shfl_up(sum, o);
        if (lane >= o) sum += v;
    }
    if (lane == 63) lds[1024 + (tid >> 6)] = sum;
    __syncthreads();
    sum -= n[3];
    for (int w = 0; w < (tid >> 6); ++w) sum += lds[1024 + w];
#pragma unroll
    for (int i = 0; i < 4; ++i) last[4 * tid + i] = sum + n[i];
    __syncthreads();
    // 1024 experts: the rows after the last one's have no thread of their own
    const int rest = p.E == 1024 ? p.P16 - start(1024) : 0;
    const int experts = last[1023], count = min(experts + (rest + BLOCK - 1) / BLOCK, p.cap);
    if (tid == 0) p.tiles[0] = count;
    for (int i = tid; i < count; i += 256) {
        int lo = 0, hi = 1024;                  // first e with last[e] > i
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (last[mid] > i) hi = mid; else lo = mid + 1;
        }
        const int f = start(lo), c = end(lo) - f, before = lo ? last[lo - 1] : 0;
        const int parts = (c + BLOCK - 1) / BLOCK, j = i - before;
        // pieces of 32 rows are whole; the parts differ by one piece at most
        const int pieces = (c + 1) / 2;
        const int p0 = static_cast<int>(static_cast<int64_t>(pieces) * j / parts);
        const int p1 = static_cast<int>(static_cast<int64_t>(pieces) * (j + 1) / parts);
        *reinterpret_cast<int4*>(p.tiles + 4 + 4 * i) = make_int4(lo < p.E ? lo : -1, f + 2 * p0, min(2 * p1, c) - 2 * p0, 0);
    }
    __syncthreads();
}

}  // namespace mq
