// Products of many unquantized rows with group-scaled 4-bit weights, by tiles.
//
// As in w4_gemm.hip, y = sum over groups of s * (P - z * X). Here P - z * X is one chain of matrix
// instructions: X, the sum of a row's group, is known before (a pass over x) as three
// bf16 pieces, and one instruction more a group multiplies them by -z. fp32 x comes as
// three bf16 planes, which are as many runs of K over the same weights.
#include "plan_tiles.h"
#include "w4_device.h"
#include "w4_internal.h"
#include "w4_tiles.h"

namespace mq {
namespace {

constexpr int kThreads = 256;

// ------------------------------------------------------------------- rows
// The sums of each row's groups, [stage][group][row] units of 16 bytes: bf16 hi, mid, lo, hi,
// mid, lo, 0, 0 (the second three meet the low part of z), and where `copy` is given the
// rows themselves, [row][stage][128], zeros past K. A stage is 128 inputs; of fp32 rows, of
// one of their planes (stage 3h + plane). One wave: 512 inputs of four rows. Once for all the tiles
// that take a row, which would else each make its sums again. 2048 x 5120
// of bf16 6 us, 33000 x 1024 19 us (3.5 TB/s): bound by the reads; 22 us where it looks at the
// bf16 scales of 64 matrices 4096 x 1024 beside (8 MB).
constexpr int kRows = 4;

// One wave, four 16-row tiles of W from `tile` on, a row a lane: all bits of wild[tile] where a row's scales
// (bf16) that are not 0 are more than 2^40 apart or outside 2^-126 .. 2^126 (NaN among them).
// With fp16's scales no two are further apart, and the tiles do not ask.
template <int GS>
__device__ void wild_scales(const uint16_t* scales, int64_t tile, int64_t tiles, int Q, int* wild) {
    const int lane = threadIdx.x & 63;
    tile += lane >> 4;
    uint32_t least = 0x7f800000u, most = 0;                // bits of magnitudes, in order
    const uint16_t* const from = scales + ((tile < tiles ? tile : tiles - 1) * Q * 16 + (lane & 15)) * 4 * GS;
#pragma unroll 2
    for (int q = 0; q < Q; ++q) {
        W4Quad<GS> s;
        s.load(from + static_cast<int64_t>(q) * 64 * GS);
#pragma unroll
        for (int i = 0; i < 4 * GS; ++i) {
            const uint32_t a = __float_as_uint(s.get(i, true)) & 0x7fffffffu;
            most = max(most, a);
            least = min(least, a ? a : 0x7f800000u);
        }
    }
    // (rows of zeros: least is infinity)
    const bool far = most && (least < 0x00800000u || most > 0x7e800000u || most - least > 40u << 23);
    const uint64_t which = __ballot(far);
    if ((lane & 15) == 0 && tile < tiles) wild[tile] = which >> lane & 0xffff ? ~0 : 0;
}

template <typename XT>
__global__ __launch_bounds__(kThreads) void k_w4_rows(const XT* x, int64_t R, int64_t stride, int K, int group, uint4* sums,
                                                      uint16_t* copy, MxTilesArgs plan, int rt, int row_blocks, const uint16_t* scales,
                                                      int64_t tiles, int* wild) {
    __shared__ int lds[kTilesLds];
    const int first = plan.offsets ? 1 : 0;            // workgroups (0, 0): the plan's row blocks alone
    if (static_cast<int>(blockIdx.x) < first) {
        if (blockIdx.y == 0) {
            if (rt == 4) plan_tiles<8>(plan, lds);
            else if (rt == 3) plan_tiles<6>(plan, lds);
            else if (rt == 2) plan_tiles<4>(plan, lds);
            else plan_tiles<2>(plan, lds);
        }
        return;
    }
    if (static_cast<int>(blockIdx.x) >= first + row_blocks) {               // the scales
        const int64_t tile = ((static_cast<int64_t>(blockIdx.x - first - row_blocks) * gridDim.y + blockIdx.y) * 4 + (threadIdx.x >> 6)) * 4;
        const int Q = (K + 511) / 512;
        if (tile >= tiles) return;
        if (group == 128) wild_scales<1>(scales, tile, tiles, Q, wild);
        else if (group == 64) wild_scales<2>(scales, tile, tiles, Q, wild);
        else wild_scales<4>(scales, tile, tiles, Q, wild);
        return;
    }
    constexpr int kPlanes = sizeof(XT) == 4 ? 3 : 1;
    const int G = (K + 127) / 128, per = 128 / group, unit = group / 8;
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int64_t r0 = (static_cast<int64_t>(blockIdx.x - first) * 4 + wave) * kRows;
    const int h = blockIdx.y * 4 + (lane >> 4), k0 = blockIdx.y * 512 + 8 * lane;
    MxRaw8<XT> raw[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) raw[i] = mx_load8(x + (r0 + i) * stride + k0, r0 + i < R ? K - k0 : 0);
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int64_t r = r0 + i;
        float v[8];
        w4_values(raw[i], v);
#pragma unroll
        for (int p = 0; p < kPlanes; ++p) {
            if constexpr (kPlanes == 3) {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = raw[i].v[j];
            }
            float s = 0;
            w4_u4 words;
            if constexpr (kPlanes == 3) {
                float cut[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) cut[j] = __uint_as_float(__float_as_uint(v[j]) & 0xffff0000u);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    words[j] = __builtin_amdgcn_perm(__float_as_uint(cut[2 * j + 1]), __float_as_uint(cut[2 * j]), 0x07060302u);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    s += cut[j];
                    raw[i].v[j] = v[j] - cut[j];
                }
            } else {
                words = w4_u4{raw[i].w[0], raw[i].w[1], raw[i].w[2], raw[i].w[3]};
#pragma unroll
                for (int j = 0; j < 8; ++j) s += v[j];
            }
            s = __int_as_float(w4_over_group(__float_as_int(s), group, [](int a, int b) {
                return __float_as_int(__int_as_float(a) + __int_as_float(b));
            }));
            if (r >= R || h >= G) continue;
            const int64_t stage = static_cast<int64_t>(h) * kPlanes + p;
            if ((lane & (unit - 1)) == 0) {
                const uint32_t hi = __float_as_uint(s) >> 16;
                const float rest = s - __uint_as_float(hi << 16);
                const uint32_t mid = __float_as_uint(rest) >> 16;
                const uint32_t lo = __float_as_uint(rest - __uint_as_float(mid << 16)) >> 16;
                sums[(stage * per + (lane & 15) / unit) * R + r] = make_uint4(hi | mid << 16, lo | hi << 16, mid | lo << 16, 0);
            }
            if (copy) *reinterpret_cast<w4_u4*>(copy + (r * G * kPlanes + stage) * 128 + (lane & 15) * 8) = words;
        }
    }
}

template <typename XT>
hipError_t rows(const W4RowsArgs& a, hipStream_t st) {
    const int64_t first = a.plan.offsets ? 1 : 0, row_blocks = (a.R + 4 * kRows - 1) / (4 * kRows), quads = w4_quads(a.K);
    const int64_t blocks = first + row_blocks + ((a.tiles + 15) / 16 + quads - 1) / quads;
    if (blocks >= int64_t(1) << 24) return hipErrorInvalidConfiguration;     // a grid's axis holds 2^32 threads
    k_w4_rows<XT><<<dim3(static_cast<unsigned>(blocks), static_cast<unsigned>(quads)), kThreads, 0, st>>>(
        static_cast<const XT*>(a.x), a.R, a.stride, a.K, a.group, static_cast<uint4*>(a.sums), static_cast<uint16_t*>(a.copy), a.plan, a.rt,
        static_cast<int>(row_blocks), a.scales, a.tiles, a.wild);
    return hipGetLastError();
}

// ------------------------------------------------------------------- tiles
template <typename E> struct Op;
template <> struct Op<__bf16> {
    typedef w4_b8 V;
    static __device__ __forceinline__ mx_f16 mfma(V a, V b, mx_f16 c) { return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0); }
};
template <> struct Op<_Float16> {
    typedef w4_h8 V;
    static __device__ __forceinline__ mx_f16 mfma(V a, V b, mx_f16 c) { return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0); }
};

// 16 bytes a lane to lane * 16 behind `to` (wave-uniform)
__device__ __forceinline__ void to_lds(__amdgpu_buffer_rsrc_t r, int lane_at, int at, uint8_t* to) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)to, 16, lane_at, at, 0, 0);
}

// The kernel's arguments where the launch put them: as a parameter that three branches use
// they went to scratch memory, and their loads waited for those of the weights.
typedef __attribute__((address_space(4))) W4WideArgs Args;

// Stages in LDS: one at work, the others on their way. Small tiles have little to do in a
// stage and wait for memory with one on its way (64 rows of 4096 x 4096, weights from memory:
// 31.3 us with one, 26.6 with three); large ones have no registers for more weights.
template <int RT, int CT> constexpr int kDepth = RT <= 2 ? (RT * CT == 1 ? 4 : 3) : 2;
template <int RT, int GS, int D> struct WideLds {
    static constexpr int kX = 32 * RT * 256, kSums = GS * 32 * RT * 16, kStage = kX + kSums;
    static constexpr int kOut = 32 * (64 * 4 + 16);      // a wave's results on their way out
    static constexpr int kBytes = D * kStage > 4 * kOut ? D * kStage : 4 * kOut;
};
template <int N> struct Count { static constexpr int value = N; };
// Every wave's loads but the last N are done, and so are all waves' reads before.
template <int N>
__device__ __forceinline__ void loads_and_barrier() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// The scale of a code tile's group g; -z of it as the matrix instructions take it: the sums' pieces
// meet its high part, then its low part (`none`: 0, for the lanes of the other inputs).
template <typename S>
__device__ __forceinline__ float scale_of(S s, int g, bool bf) { return w4_float(static_cast<uint32_t>(s >> 16 * g) & 0xffff, bf); }
template <typename S>
__device__ __forceinline__ w4_b8 zero_of(S z, int g, bool bf, bool has_zeros, bool none) {
    const float given = -scale_of(z, g, bf), v = has_zeros ? given : -8.0f;
    const uint32_t hi = none ? 0 : __float_as_uint(v) >> 16;
    const uint32_t lo = none ? 0 : __float_as_uint(v - __uint_as_float(__float_as_uint(v) & 0xffff0000u)) >> 16;
    return __builtin_bit_cast(w4_b8, w4_u4{hi | hi << 16, hi | lo << 16, lo | lo << 16, 0});
}

// x's row of row r of a block; those past its end read the last one's.
__device__ __forceinline__ int row_at(const Args& a, int row0, int rows, int r) {
    const int p = min(r, rows - 1);
    if (!a.by_token) return p;
    const int token = a.row_token[row0 + p];
    return static_cast<unsigned>(token) < static_cast<unsigned>(a.T) ? token : 0;
}

// 32 rows from p0 on, `rows` of them there, leave through LDS (`tile`, a wave's own): a lane holds one
// column of rows 8 (r / 4) + 4 (l / 32) + r % 4 in value(j, r), read back it holds eight columns of a row.
// True where one of a row that counts is not finite.
template <int CT, typename Value>
__device__ __forceinline__ bool leave(const Args& a, uint8_t* tile, int p0, int rows, int n0, int have, Value value) {
    constexpr int kPitch = 32 * CT * 4 + 16, kLanes = 4 * CT, kRound = 64 / kLanes;
    const int lane = threadIdx.x & 63, half = lane >> 5, N = a.N, column = (lane % kLanes) * 8, block = column / 32, n = n0 + column;
    // a part of K: its sums go to its own fp32 rows, and become outputs with the others'
    const bool parted = a.partial != nullptr;
    const int T = a.T, y_dtype = parted ? MQ_F32 : a.y_dtype;
    const int32_t* const row_token = a.row_token;
    const float* const bias = parted ? nullptr : a.bias;
    void* const y = parted ? a.partial + static_cast<int64_t>(blockIdx.y) * a.M * N : a.y;
    float peak = 0;
    mx_wave_sync();
#pragma unroll
    for (int j = 0; j < CT; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r)
            *reinterpret_cast<float*>(tile + (8 * (r >> 2) + 4 * half + (r & 3)) * kPitch + (32 * j + (lane & 31)) * 4) = value(j, r);
    mx_wave_sync();
    // (the second block's columns begin at its first tile)
    const uint8_t* const from = tile + (32 * block + column - 16 * w4_block_tile(block, 2, have)) * 4;
#pragma unroll
    for (int q = 0; q < 32 / kRound; ++q) {
        const int r = q * kRound + lane / kLanes, p = p0 + r;
        if (r >= rows || n >= N) continue;
        const mx_f4 lo = *reinterpret_cast<const mx_f4*>(from + r * kPitch);
        const mx_f4 hi = *reinterpret_cast<const mx_f4*>(from + r * kPitch + 16);
        float v[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
        if (row_token && static_cast<unsigned>(row_token[p]) >= static_cast<unsigned>(T)) {
#pragma unroll
            for (int c = 0; c < 8; ++c) v[c] = 0.0f;
        }
#pragma unroll
        for (int c = 0; c < 8; ++c) peak = __builtin_elementwise_maximum(peak, fabsf(v[c]));         // (NaN stays)
        if (bias) {
#pragma unroll
            for (int c = 0; c < 8; ++c) v[c] += n + c < N ? bias[n + c] : 0.0f;
        }
        const int64_t at = static_cast<int64_t>(p) * N + n;
        if (y_dtype == MQ_F32) w4_store8(static_cast<float*>(y) + at, N - n, v);
        else if (y_dtype == MQ_BF16) w4_store8(static_cast<__bf16*>(y) + at, N - n, v);
        else w4_store8(static_cast<_Float16*>(y) + at, N - n, v);
    }
    return !(peak < __builtin_inff());
}

// One wave's part of a tile of 32 RT rows: 32 CT columns. The rows of a stage (128 inputs) go
// from memory to LDS, units of 16 bytes in an order that has a row's sixteen and sixteen
// rows' alike in different banks; the weights go to registers, each wave its own, a stage
// ahead.
//
// The sums stand in units of the column's present scale: where a group begins, they are
// multiplied by the last scale over the new one, and go on through the matrix instructions.
// Beside them a second set, to be added to once a group, has no room in the registers of
// a tile of this size. Not all sums have a value in all units. Where a scale falls they may leave
// fp32's range, and end as infinities or NaN; where it rises they lose what is below 2^-126 of the
// new unit. So 32 rows with a result that is not finite are computed again with a second set
// (wide_again), and all of them where k_w4_rows found the columns' scales too far apart.
// Returns which: bit i for the rows 32 i on.
template <typename E, int GS, int RT, int CT, int D>
__device__ __forceinline__ uint32_t wide_tile(const Args& a, uint8_t* lds, int e, int row0, int rows, int n0) {
    typedef typename Op<E>::V V;
    typedef WideLds<RT, GS, D> L;
    constexpr int kSteps = 8 / GS;
    const int lane = threadIdx.x & 63, half = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int N = a.N, planes = a.planes, G = (a.K + 127) / 128, Q = (G + 3) / 4, stages = G * planes, n_tiles = (N + 15) / 16;
    const bool bf = a.scale_dtype == MQ_BF16, has_zeros = a.zeros != nullptr, by_token = a.by_token != 0;
    const int64_t rows_x = a.rows_x;
    const uint4* const all_sums = a.sums;
    // (there are no more parts than stages: each has one at least)
    const int first_stage = static_cast<int>(static_cast<int64_t>(stages) * blockIdx.y / gridDim.y);
    const int last = static_cast<int>(static_cast<int64_t>(stages) * (blockIdx.y + 1) / gridDim.y) - 1;
    const int64_t first_row = by_token ? 0 : row0;
    // this lane's places: rows 4 (2 RT wave + i) + lane / 16, unit lane % 16 of LDS is unit
    // (lane % 16) ^ (row % 16) of the row
    uint32_t xat[2 * RT];
#pragma unroll
    for (int i = 0; i < 2 * RT; ++i) {
        const int r = 4 * (2 * RT * wave + i) + (lane >> 4);
        xat[i] = static_cast<uint32_t>(row_at(a, row0, rows, r)) * static_cast<uint32_t>(a.ldx) * 2 + 16 * ((lane & 15) ^ (r & 15));
    }
    // and the wave's fourth of the sums' units
    constexpr int kUnits = 8 * GS * RT, kSumsPer = (kUnits + 63) / 64;
    uint32_t sat[kSumsPer];
#pragma unroll
    for (int i = 0; i < kSumsPer; ++i) {
        const int u = wave * kUnits + min(i * 64 + lane, kUnits - 1);
        sat[i] = (static_cast<uint32_t>(u / (32 * RT)) * static_cast<uint32_t>(rows_x) + row_at(a, row0, rows, u % (32 * RT))) * 16;
    }
    const uint16_t* const x0 = a.x + first_row * a.ldx;
    const int64_t x_bytes = ((by_token ? a.T : rows) - 1) * a.ldx * 2 + 256;         // behind a stage's first input
    // Loads of a stage, in every wave. A stage's rows are waited for by the number of loads issued
    // after them, so all of a stage's are issued before the next stage's first: the barriers
    // within run() see to that, and the fences between the stages that come before it.
    constexpr int kLoads = 2 * RT + kSumsPer + 4 * CT;
    static_assert(D == 2 || kUnits <= 64);
    // (the stage is said to be the same in all lanes, or the tiles of three stages take it for a vector,
    // and each load of the weights for one of many)
    auto load_x = [&](int at, int buf) __attribute__((always_inline)) {
        const int stage = __builtin_amdgcn_readfirstlane(at);
        uint8_t* const to = lds + buf * L::kStage;
        const __amdgpu_buffer_rsrc_t xr = buffer(x0 + static_cast<int64_t>(stage) * 128, x_bytes);
        const __amdgpu_buffer_rsrc_t sr = buffer(all_sums + static_cast<int64_t>(stage) * GS * rows_x + first_row,
                                                 (GS * rows_x - first_row) * 16);
#pragma unroll
        for (int i = 0; i < 2 * RT; ++i) to_lds(xr, xat[i], 0, to + (2 * RT * wave + i) * 1024);
#pragma unroll
        for (int i = 0; i < kSumsPer; ++i)
            if (i * 64 + lane < kUnits) to_lds(sr, sat[i], 0, to + L::kX + (wave * kUnits + i * 64) * 16);
    };
    // weights: a wave with no column of its own (past N) reads the last tile's and writes nothing
    const int tile0 = min(n0 / 16, n_tiles - 1), have = min(n_tiles - tile0, 2 * CT);
    const int64_t first = static_cast<int64_t>(e) * n_tiles + tile0;
    const int scale_bytes = w4_scale_bytes(Q, GS);       // of a row tile
    const __amdgpu_buffer_rsrc_t wr = buffer(a.codes + first * G * 1024, static_cast<int64_t>(have) * G * 1024);
    const __amdgpu_buffer_rsrc_t scr = buffer(a.scales + first * (scale_bytes / 2), static_cast<int64_t>(have) * scale_bytes);
    const __amdgpu_buffer_rsrc_t zr = has_zeros ? buffer(a.zeros + first * (scale_bytes / 2), static_cast<int64_t>(have) * scale_bytes) : scr;
    uint32_t redo = 0;                                   // all, where the columns' scales are too far apart
    if (bf) {
#pragma unroll
        for (int t = 0; t < 2 * CT; ++t) redo |= a.wild[first + min(t, have - 1)];
    }
    const int wat = w4_pair_code(lane, have, G), scat = w4_pair_scale(lane, have, Q, GS);
    int block[CT];                                       // the first tiles of the blocks of 32 columns
#pragma unroll
    for (int j = 0; j < CT; ++j) block[j] = __builtin_amdgcn_readfirstlane(w4_block_tile(j, 2, have));
    // words w of [j][0] are steps 2w, of [j][1] steps 2w + 1
    typedef typename W4Scales<GS>::T Scales;
    struct Weights {
        mx_i4 c[CT][2];
        Scales s[CT], z[CT];
    } W[D - 1];
    auto scales_at = [&](__amdgpu_buffer_rsrc_t r, int at) __attribute__((always_inline)) -> Scales {
        if constexpr (GS == 1) return __builtin_amdgcn_raw_buffer_load_b16(r, scat, at, 0);
        else if constexpr (GS == 2) return __builtin_amdgcn_raw_buffer_load_b32(r, scat, at, 0);
        else return __builtin_bit_cast(uint64_t, __builtin_amdgcn_raw_buffer_load_b64(r, scat, at, 0));
    };
    auto load_w = [&](int which, Weights& to) __attribute__((always_inline)) {
        const int stage = __builtin_amdgcn_readfirstlane(which);
        const int h = planes == 1 ? stage : stage / 3;
#pragma unroll
        for (int j = 0; j < CT; ++j) {
            const int at = w4_code_at(block[j], h, G);
            to.c[j][0] = load16(wr, wat, at);
            to.c[j][1] = load16(wr, wat, at + 512);
            to.s[j] = scales_at(scr, w4_scale_at(block[j], h, Q, GS));
            to.z[j] = scales_at(zr, w4_scale_at(block[j], h, Q, GS));
        }
    };
    mx_f16 acc[RT][CT] = {};
    // A group's: the factor from the last unit to its own, its unit, -z as the matrix instructions
    // take it. A scale of 0 leaves the unit as it is and its codes out: by their mask, or, in the
    // tiles of 128 rows, whose registers are all in use, by clearing them where one is met, and with
    // one unit instead of the last and the next (groups of 64 spill 12 registers else: 4096 tokens of 8
    // of 64, 4096 x 1024, 414 us and 379 so; 64 x 256 tiles take 3% longer so).
    constexpr bool kTight = RT == 4;
    float unit[CT] = {}, by[CT], next[CT];
    w4_b8 zb[CT];
    uint32_t mask[CT];
    // there: not a stage past the last one
    auto begin = [&](Weights& w, int g, bool there) __attribute__((always_inline)) {
        bool any = false;
#pragma unroll
        for (int j = 0; j < CT; ++j) {
            const float s = scale_of(w.s[j], g, bf);
            const bool none = s == 0;
            const float to = none ? 1.0f : s, from = none ? 1.0f : unit[j], inv = __builtin_amdgcn_rcpf(to), q = from * inv;
            by[j] = __builtin_fmaf(__builtin_fmaf(-q, to, from), inv, q);
            if constexpr (kTight) unit[j] = none || !there ? unit[j] : s;
            else next[j] = none ? unit[j] : s;
            any |= none;
            mask[j] = !kTight && none ? 0 : 0x0f0f0f0fu;
            zb[j] = zero_of(w.z[j], g, bf, has_zeros, none || half);
        }
        if (kTight && __ballot(any)) {
#pragma unroll
            for (int j = 0; j < CT; ++j) {
                const uint32_t keep = scale_of(w.s[j], g, bf) == 0 ? 0 : ~0u;
#pragma unroll
                for (int s = g * kSteps; s < (g + 1) * kSteps; ++s) w.c[j][s & 1][s >> 1] &= keep;
            }
        }
    };
    V x_of[2][RT], b[2][CT];
    // a row tile's share of the conversions of a step
    auto convert = [&](const Weights& w, int step, int i) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < CT; ++j)
            if (j * RT / CT == i) b[step & 1][j] = w4_codes<E>(w.c[j][step & 1][step >> 1], mask[j]);
    };
#pragma unroll
    for (int d = 0; d < D - 1; ++d) {
        load_x(min(first_stage + d, last), d);
        load_w(min(first_stage + d, last), W[d]);
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
    }
    begin(W[0], 0, true);
#pragma unroll
    for (int i = 0; i < RT; ++i) convert(W[0], 0, i);
    const int swap = (half ^ (lane & 15)) * 16;
    // Stage `stage` (whose weights are in `now`, the next one's in `after`). Loads past the last
    // stage are of that again, and not used: a wave's loads are counted. `later`: how many of them
    // may still be on their way.
    int buf = 0;
    auto run = [&](auto later, int stage, Weights& now, Weights& after) __attribute__((always_inline)) {
        loads_and_barrier<decltype(later)::value>();     // stage's rows are there, reads of the buffer to be filled are done
        Weights w = now;
        load_x(min(stage + D - 1, last), buf == 0 ? D - 1 : buf - 1);
        load_w(min(stage + D - 1, last), now);
        const uint8_t* const x = lds + buf * L::kStage + (lane & 31) * 256;
        const uint8_t* const sums = lds + buf * L::kStage + L::kX + (lane & 31) * 16;
        buf = buf == D - 1 ? 0 : buf + 1;
        w4_b8 sum[RT];
        auto read = [&](int step, int i) __attribute__((always_inline)) {
            x_of[step & 1][i] = *reinterpret_cast<const V*>(x + 32 * i * 256 + (swap ^ step * 32));
        };
        auto read_sum = [&](int g, int i) __attribute__((always_inline)) {
            sum[i] = *reinterpret_cast<const w4_b8*>(sums + (g * 32 * RT + 32 * i) * 16);
        };
        // A step's operands are read and converted during the step before, a group's begun
        // during the last one's end; the scheduling barriers keep each row tile's products
        // with its share of that. Left alone, the compiler reads operands right before
        // their use, and the matrix units wait for them and for the conversions.
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            read_sum(0, i);
            read(0, i);
        }
#pragma unroll
        for (int g = 0; g < GS; ++g) {
#pragma unroll
            for (int j = 0; j < CT; ++j) unit[j] = kTight ? unit[j] : next[j];
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                const int step = g * kSteps + s;
#pragma unroll
                for (int i = 0; i < RT; ++i) {
                    if (s == 0) {
#pragma unroll
                        for (int j = 0; j < CT; ++j) acc[i][j] *= by[j];
#pragma unroll
                        for (int j = 0; j < CT; ++j) acc[i][j] = Op<__bf16>::mfma(sum[i], zb[j], acc[i][j]);
                    }
#pragma unroll
                    for (int j = 0; j < CT; ++j) acc[i][j] = Op<E>::mfma(x_of[step & 1][i], b[step & 1][j], acc[i][j]);
                    if (s + 1 < kSteps) {
                        read(step + 1, i);
                        convert(w, step + 1, i);
                    } else if (g + 1 < GS) {
                        if (i == 0) begin(w, g + 1, true);
                        read_sum(g + 1, i);
                        read(step + 1, i);
                        convert(w, step + 1, i);
                    } else {                             // (past the last stage: of its own again, not used)
                        if (i == 0) {
#pragma unroll
                            for (int j = 0; j < CT; ++j) asm volatile("" : "+v"(after.s[j]), "+v"(after.z[j]));    // no use of these loads sooner
                            begin(after, 0, stage < last);
                        }
                        convert(after, 0, i);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
        }
    };
    constexpr Count<(D - 2) * kLoads> kLater{};
    int stage = first_stage;
    for (; stage + D - 2 <= last; stage += D - 1) {
#pragma unroll
        for (int d = 0; d < D - 1; ++d) run(kLater, stage + d, W[d], W[d + 1 == D - 1 ? 0 : d + 1]);
    }
    // (nothing uses the weights that the first of these loads, and the compiler leaves them out: the
    // second cannot count on them, and has nothing but loads of the last stage again behind it)
    static_assert(D <= 4);
    if (D > 2 && stage <= last) run(kLater, stage, W[0], W[D > 2 ? 1 : 0]);
    if (D > 3 && stage + 1 <= last) run(Count<0>{}, stage + 1, W[D > 3 ? 1 : 0], W[D > 3 ? 2 : 0]);

    uint8_t* const tile = lds + wave * L::kOut;
    loads_and_barrier<0>();                              // nothing is on its way to LDS any more
#pragma unroll
    for (int i = 0; i < RT; ++i)
        if (__ballot(leave<CT>(a, tile, row0 + 32 * i, rows - 32 * i, n0, have, [&](int j, int r) __attribute__((always_inline)) { return acc[i][j][r] * unit[j]; })))
            redo |= 1u << i;
    return redo;
}

// Rows of a wave's part of a tile once more (the bits of `redo`, 32 each): a group's products in sums
// of their own, which its scale multiplies. Operands come from memory as they are used: the rare
// way, for inputs that few products see. All rows of 2048 x 17408 x 5120 again: 1100 us where the tiles
// alone take 355 (groups of 32: 1630, 505); one row with a NaN, which is among 32 in all columns: 490.
// A lane writes the outputs that it wrote before.
template <typename E, int GS, int CT>
__device__ __forceinline__ void wide_again(const Args& a, uint8_t* tile, int e, int row0, int rows, int n0, uint32_t redo) {
    typedef typename Op<E>::V V;
    constexpr int kSteps = 8 / GS;
    const int lane = threadIdx.x & 63, half = lane >> 5;
    const int planes = a.planes, G = (a.K + 127) / 128, Q = (G + 3) / 4, stages = G * planes, n_tiles = (a.N + 15) / 16;
    const bool bf = a.scale_dtype == MQ_BF16, has_zeros = a.zeros != nullptr;
    const int first_stage = static_cast<int>(static_cast<int64_t>(stages) * blockIdx.y / gridDim.y);
    const int last = static_cast<int>(static_cast<int64_t>(stages) * (blockIdx.y + 1) / gridDim.y) - 1;
    const int64_t first_row = a.by_token ? 0 : row0;
    const int tile0 = min(n0 / 16, n_tiles - 1), have = min(n_tiles - tile0, 2 * CT);
    const int64_t first = static_cast<int64_t>(e) * n_tiles + tile0;
    const uint8_t* const codes = a.codes + first * G * 1024 + w4_pair_code(lane, have, G);
    const int64_t scales_at = first * (w4_scale_bytes(Q, GS) / 2) + w4_pair_scale(lane, have, Q, GS) / 2;
#pragma unroll 1
    for (int i = 0; 32 * i < rows; ++i) {
        if (!(redo >> i & 1)) continue;
        const int row = row_at(a, row0, rows, 32 * i + (lane & 31));
        const uint16_t* const x = a.x + (first_row + row) * a.ldx + 8 * half;
        mx_f16 sum[CT] = {};
#pragma unroll 1
        for (int stage = first_stage; stage <= last; ++stage) {
            const int h = planes == 1 ? stage : stage / 3;
            mx_i4 c[CT][2];
            typename W4Scales<GS>::T s[CT], z[CT];
#pragma unroll
            for (int j = 0; j < CT; ++j) {
                const int t = w4_block_tile(j, 2, have);
                const int64_t at = scales_at + w4_scale_at(t, h, Q, GS) / 2;
                c[j][0] = *reinterpret_cast<const mx_i4*>(codes + w4_code_at(t, h, G));
                c[j][1] = *reinterpret_cast<const mx_i4*>(codes + w4_code_at(t, h, G) + 512);
                s[j] = w4_scales<GS>(a.scales + at);
                z[j] = has_zeros ? w4_scales<GS>(a.zeros + at) : s[j];
            }
#pragma unroll
            for (int g = 0; g < GS; ++g) {
                const w4_b8 rows_sum = __builtin_bit_cast(w4_b8, a.sums[(static_cast<int64_t>(stage) * GS + g) * a.rows_x + first_row + row]);
                mx_f16 P[CT] = {};
#pragma unroll
                for (int j = 0; j < CT; ++j) P[j] = Op<__bf16>::mfma(rows_sum, zero_of(z[j], g, bf, has_zeros, half), P[j]);
#pragma unroll
                for (int step = g * kSteps; step < (g + 1) * kSteps; ++step) {
                    const V v = *reinterpret_cast<const V*>(x + static_cast<int64_t>(stage) * 128 + 16 * step);
#pragma unroll
                    for (int j = 0; j < CT; ++j) P[j] = Op<E>::mfma(v, w4_codes<E>(c[j][step & 1][step >> 1]), P[j]);
                }
#pragma unroll
                for (int j = 0; j < CT; ++j) sum[j] += scale_of(s[j], g, bf) * P[j];
            }
        }
        leave<CT>(a, tile, row0 + 32 * i, rows - 32 * i, n0, have, [&](int j, int r) __attribute__((always_inline)) { return sum[j][r]; });
    }
}

// zeros for rows after the last expert's
template <int COLS>
__device__ void zero_rows(const Args& a, int row0, int rows, int n0) {
    void* const y = a.y;                                 // (a plan's rows have no parts of K)
    const int y_dtype = a.y_dtype;
    const float none[8] = {};
    for (int i = threadIdx.x; i < rows * (COLS / 8); i += kThreads) {
        const int n = n0 + i % (COLS / 8) * 8;
        const int64_t at = static_cast<int64_t>(row0 + i / (COLS / 8)) * a.N + n;
        if (n >= a.N) continue;
        if (y_dtype == MQ_F32) w4_store8(static_cast<float*>(y) + at, a.N - n, none);
        else if (y_dtype == MQ_BF16) w4_store8(static_cast<__bf16*>(y) + at, a.N - n, none);
        else w4_store8(static_cast<_Float16*>(y) + at, a.N - n, none);
    }
}

// y = the parts' sums, in the order of the parts, and the bias.
// Eight outputs a thread. A launch, and about 0.4 us for each MB of sums written and read.
template <typename T>
__global__ __launch_bounds__(kThreads) void k_w4_add(const float* partial, int parts, int64_t M, int N, const float* bias, T* y) {
    const int n = (blockIdx.x * kThreads + threadIdx.x) * 8;
    if (n >= N) return;
    for (int64_t m = blockIdx.y; m < M; m += gridDim.y) {
        float sum[8] = {};
        for (int p0 = 0; p0 < parts; p0 += 4) {
            MxRaw8<float> v[4];
#pragma unroll
            for (int p = 0; p < 4; ++p) v[p] = mx_load8(partial + ((p0 + p) * M + m) * N + n, p0 + p < parts ? N - n : 0);
#pragma unroll
            for (int p = 0; p < 4; ++p)
#pragma unroll
                for (int i = 0; i < 8; ++i) sum[i] += v[p].v[i];
        }
        if (bias) {
#pragma unroll
            for (int i = 0; i < 8; ++i) sum[i] += n + i < N ? bias[n + i] : 0.0f;
        }
        w4_store8(y + m * N + n, N - n, sum);
    }
}

template <typename T>
hipError_t add_parts(const W4WideArgs& a, hipStream_t st) {
    const dim3 grid((a.N + 8 * kThreads - 1) / (8 * kThreads), a.M < 65535 ? a.M : 65535);
    k_w4_add<T><<<grid, kThreads, 0, st>>>(a.partial, a.parts, a.M, a.N, a.bias, static_cast<T*>(a.y));
    return hipGetLastError();
}

// Four waves side by side, on blocks of at most 32 RT rows. Bound by the matrix units, whose power
// holds the clock near 1.9 GHz, and by the changes of units: 2048 x 17408 x 5120 of bf16, groups of
// 128 / 64 / 32: 355 / 410 / 515 us, up to a tenth more on some cards (1.03 / 0.89 / 0.71 PFLOP/s; a
// bf16 library product of the size 0.92). Which tile a product takes is fitted in api_w4.hip.
template <typename E, int GS, int RT, int CT>
__global__ __launch_bounds__(kThreads, 2) void k_w4_wide(W4WideArgs) {
    const Args& a = *(const Args*)__builtin_amdgcn_kernarg_segment_ptr();
    constexpr int D = kDepth<RT, CT>;
    __shared__ __align__(16) uint8_t lds[WideLds<RT, GS, D>::kBytes];
    constexpr int kCols = 128 * CT, kSlots = 64;           // workgroups that a die holds at a time
    const int ncol = (a.N + kCols - 1) / kCols, blocks = (a.M + 32 * RT - 1) / (32 * RT);
    const int count = a.tiles ? a.tiles[0] : blocks;
    // Workgroups go to the eight dies in turn: each die takes a run of neighbouring tiles,
    // which share rows and weights in its L2. The tiles that would be left for a last round of
    // few workgroups are split by rows, so that they fill it.
    const int total = count * ncol, share = (total + 7) / 8;
    const int die = blockIdx.x & 7, mine = min(share, total - die * share);
    int u = blockIdx.x >> 3, part = 0, parts = 1;
    if (!a.tiles && mine > kSlots) {
        const int whole = mine / kSlots * kSlots, rest = mine - whole;
        parts = rest * 4 <= kSlots && RT == 4 ? 4 : (rest * 2 <= kSlots && RT > 1 ? 2 : 1);
        if (u >= whole) {
            part = (u - whole) % parts;
            u = whole + (u - whole) / parts;
        } else {
            parts = 1;
        }
    }
    const int t = die * share + u;
    if (u >= mine) return;
    int e = 0, row0, rows, col;
    if (a.tiles) {
        const int4 tile = *reinterpret_cast<const int4*>(a.tiles + 4 + 4 * (t / ncol));
        e = __builtin_amdgcn_readfirstlane(tile.x);
        row0 = __builtin_amdgcn_readfirstlane(tile.y) * 16;
        rows = min(__builtin_amdgcn_readfirstlane(tile.z) * 16, a.M - row0);
        col = t % ncol;
    } else {
        // neighbours: eight row blocks, then the next columns of these, so that the 64 tiles at
        // work on a die share eight blocks of rows and eight of columns
        const int group = t / (8 * ncol), in_group = min(8, blocks - 8 * group), i = t - group * 8 * ncol;
        const int pieces = (RT + parts - 1) / parts;       // of 32 rows
        row0 = ((8 * group + i % in_group) * RT + part * pieces) * 32;
        rows = min(32 * min(pieces, RT - part * pieces), a.M - row0);
        col = i / in_group;
        if (rows <= 0) return;
    }
    if (e < 0) {
        zero_rows<kCols>(a, row0, rows, col * kCols);
        return;
    }
    const int n0 = col * kCols + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) * 32 * CT;
    uint32_t redo;
    if (RT >= 4 && rows > 96) redo = wide_tile<E, GS, RT, CT, D>(a, lds, e, row0, rows, n0);
    else if (RT >= 3 && rows > 64) redo = wide_tile<E, GS, RT < 3 ? RT : 3, CT, D>(a, lds, e, row0, rows, n0);
    else if (RT >= 2 && rows > 32) redo = wide_tile<E, GS, RT < 2 ? RT : 2, CT, D>(a, lds, e, row0, rows, n0);
    else redo = wide_tile<E, GS, 1, CT, D>(a, lds, e, row0, rows, n0);
    if (__builtin_expect(redo != 0, 0))
        wide_again<E, GS, CT>(a, lds + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) * WideLds<RT, GS, D>::kOut, e, row0, rows, n0, redo);
}

template <typename E, int GS, int RT, int CT>
hipError_t wide(const W4WideArgs& a, hipStream_t st) {
    const int64_t ncol = (a.N + 128 * CT - 1) / (128 * CT);
    const int64_t n = a.tiles ? w4_blocks_cap(a.M, a.E, RT) : (a.M + 32 * RT - 1) / (32 * RT);
    // split tiles make up to 64 workgroups on each die
    const int64_t want = ((n * ncol + 7) / 8 + (a.tiles || n * ncol <= 8 * 64 ? 0 : 64)) * 8;
    if (want >= int64_t(1) << 24) return hipErrorInvalidConfiguration;       // a grid holds 2^32 threads
    k_w4_wide<E, GS, RT, CT><<<dim3(static_cast<unsigned>(want), a.parts), kThreads, 0, st>>>(a);
    return hipGetLastError();
}

template <typename E, int GS>
hipError_t wide_tiles(const W4WideArgs& a, int rt, int ct, hipStream_t st) {
    if (ct == 1) return rt == 1 ? wide<E, GS, 1, 1>(a, st) : wide<E, GS, 2, 1>(a, st);
    if constexpr (GS < 4) {                                // (groups of 32: only 96 rows, w4_has_tile)
        if (rt == 2) return wide<E, GS, 2, 2>(a, st);
        if (rt == 4) return wide<E, GS, 4, 2>(a, st);
    }
    return wide<E, GS, 3, 2>(a, st);
}

template <typename E>
hipError_t wide_groups(const W4WideArgs& a, int rt, int ct, hipStream_t st) {
    if (a.group == 128) return wide_tiles<E, 1>(a, rt, ct, st);
    return a.group == 64 ? wide_tiles<E, 2>(a, rt, ct, st) : wide_tiles<E, 4>(a, rt, ct, st);
}

}  // namespace

hipError_t launch_w4_rows(const W4RowsArgs& a, hipStream_t st) {
    switch (a.dtype) {
        case MQ_F32: return rows<float>(a, st);
        case MQ_BF16: return rows<__bf16>(a, st);
        default: return rows<_Float16>(a, st);
    }
}

hipError_t launch_w4_wide(const W4WideArgs& a, int rt, int ct, hipStream_t st) {
    const hipError_t rc = a.x_dtype == MQ_F16 ? wide_groups<_Float16>(a, rt, ct, st) : wide_groups<__bf16>(a, rt, ct, st);
    if (rc != hipSuccess || !a.partial) return rc;
    switch (a.y_dtype) {
        case MQ_F32: return add_parts<float>(a, st);
        case MQ_BF16: return add_parts<__bf16>(a, st);
        default: return add_parts<_Float16>(a, st);
    }
}

}  // namespace mq
