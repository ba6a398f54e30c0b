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
#include "w4_tiles.h"

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

// Eight values as matrix operands.
template <typename XT>
__device__ __forceinline__ void pieces(const MxRaw8<XT>& r, typename W4Op<XT>::V (&a)[W4Op<XT>::kPieces]) {
    typedef typename W4Op<XT>::V V;
    if constexpr (sizeof(XT) == 2) {
        a[0] = __builtin_bit_cast(V, w4_u4{r.w[0], r.w[1], r.w[2], r.w[3]});
    } else {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = r.v[i];
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
__device__ __forceinline__ typename W4Scales<GS>::T load_scales(__amdgpu_buffer_rsrc_t r, int lane_at, int at) {
    if constexpr (GS == 1) return __builtin_amdgcn_raw_buffer_load_b16(r, lane_at, at, 0);
    else if constexpr (GS == 2) return __builtin_amdgcn_raw_buffer_load_b32(r, lane_at, at, 0);
    else return __builtin_bit_cast(uint64_t, __builtin_amdgcn_raw_buffer_load_b64(r, lane_at, at, 0));
}

// ------------------------------------------------------------------- few rows
constexpr int kMaxWaves = 8;
// 16 rows of one code tile (128 inputs) in LDS, 16 bytes further apart than they are long, so
// that their units of 16 bytes lie in different banks.
template <typename XT> constexpr int kRowPitch = 128 * sizeof(XT) + 16;

template <typename XT>
__device__ __forceinline__ void put8(uint8_t* to, const MxRaw8<XT>& v) {
    if constexpr (sizeof(XT) == 2) {
        *reinterpret_cast<w4_u4*>(to) = w4_u4{v.w[0], v.w[1], v.w[2], v.w[3]};
    } else {
        *reinterpret_cast<mx_f4*>(to) = mx_f4{v.v[0], v.v[1], v.v[2], v.v[3]};
        *reinterpret_cast<mx_f4*>(to + 16) = mx_f4{v.v[4], v.v[5], v.v[6], v.v[7]};
    }
}
template <typename XT>
__device__ __forceinline__ MxRaw8<XT> get8(const uint8_t* from) {
    MxRaw8<XT> r;
    const mx_f4 lo = *reinterpret_cast<const mx_f4*>(from);
    if constexpr (sizeof(XT) == 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i) r.w[i] = __float_as_uint(lo[i]);
    } else {
        const mx_f4 hi = *reinterpret_cast<const mx_f4*>(from + 16);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            r.v[i] = lo[i];
            r.v[4 + i] = hi[i];
        }
    }
    return r;
}

// The products of one code tile, all in this wave: acc += s (P - z X) for each of its groups.
// `from`: this lane's operands of step 0 in LDS, row tiles 16 pitches apart; scale(g, j) and
// zero(g, j).
template <typename XT, int GS, int NT, int MT, typename Scale, typename Zero>
__device__ __forceinline__ void tile_products(const mx_i4 (&c)[NT], const uint8_t* from, int pitch, Scale scale, Zero zero,
                                              mx_f4 (&acc)[NT][MT]) {
    typedef W4Op<XT> Op;
    typedef typename Op::V V;
    constexpr int kPieces = Op::kPieces, kUnit = 8 * sizeof(XT);
#pragma unroll
    for (int g = 0; g < GS; ++g) {
        mx_f4 P[NT][MT] = {}, X[MT] = {};
#pragma unroll
        for (int s = g * 4 / GS; s < (g + 1) * 4 / GS; ++s) {
            V b[NT];
#pragma unroll
            for (int j = 0; j < NT; ++j) b[j] = w4_codes<typename Op::E>(c[j][s]);
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                V v[kPieces];
                pieces<XT>(get8<XT>(from + 16 * i * pitch + 4 * s * kUnit), v);
#pragma unroll
                for (int p = 0; p < kPieces; ++p) {
                    X[i] = Op::mfma16(v[p], Op::ones(), X[i]);
#pragma unroll
                    for (int j = 0; j < NT; ++j) P[j][i] = Op::mfma16(v[p], b[j], P[j][i]);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const float sv = scale(g, j), zv = zero(g, j);
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) acc[j][i][r] += sv * (P[j][i][r] - zv * X[i][r]);
        }
        // One group's products at a time, the sums made right after them: put off to the end
        // they keep many groups' products in registers, and the waves that would hide the
        // loads out.
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int i = 0; i < MT; ++i) asm volatile("" : "+v"(acc[j][i]));
        __builtin_amdgcn_sched_barrier(0);
    }
}

// The waves' sums added in the order of the waves, and stored: columns from n0 on of the rows
// first .. first + count - 1 of the MT row tiles at row0. live(r): not a row of no token.
template <int NT, int MT, typename Live>
__device__ __forceinline__ void add_and_store(const W4GemmArgs& a, float* red, const mx_f4 (&acc)[NT][MT], int row0, int first,
                                              int count, int n0, Live live) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
    __syncthreads();                                       // [waves][NT][MT][64][4]
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < MT; ++i) reinterpret_cast<mx_f4*>(red)[((wave * NT + j) * MT + i) * 64 + lane] = acc[j][i];
    __syncthreads();
    for (int o = threadIdx.x; o < NT * 16 * count; o += blockDim.x) {
        const int c = o % (16 * NT), r = first + o / (16 * NT), m = row0 + r, n = n0 + c;
        if (n >= a.N) continue;
        const int at = (((c >> 4) * MT + (r >> 4)) * 64 + (r >> 2 & 3) * 16 + (c & 15)) * 4 + (r & 3);
        float v = 0;
        for (int s = 0; s < waves; ++s) v += red[s * NT * MT * 256 + at];
        if (a.bias) v += a.bias[n];
        store1(a.y, a.y_dtype, static_cast<int64_t>(m) * a.N + n, live(r) ? v : 0.0f);
    }
    __syncthreads();
}

// Eight values of a row from k on, zeros past K; not by a branch where K >= 8.
template <typename XT>
__device__ __forceinline__ MxRaw8<XT> load8(const XT* row, int k, int K, bool whole) {
    if (whole) return mx_load8(row + k, 8);
    return K >= 8 ? mx_load8_tail(row, k, K, K) : mx_load8(row + k, K - k);
}

// At most RB (1 or 4) rows and 16 columns a workgroup, its waves each a run of K in quads of
// code tiles (512 inputs), which are loaded while the quad before is multiplied. A row reaches
// the matrix instructions through LDS, one load of 1 KB a quad; the sums of its groups come
// from the lanes that loaded it. The instructions' rows 0 .. RB - 1 (lanes 0 .. 15 of the
// result) are the rows, the others repeat the last. GS: groups in 128 inputs. Bound by latency: a
// launch, the row, a batch of loads; 1 x 4096 x 4096 takes 4.4 to 4.7 us, one token by 8 experts of
// 1024 x 4096 6.1 to 6.7 (reading their weights at the rate of a large copy: 1.7 and 3.4); 1 x 17408 x
// 5120 15.9 with the weights from memory (8.8).
template <typename XT, int GS, bool Z, int RB>
__global__ __launch_bounds__(64 * kMaxWaves) void k_w4_one(W4GemmArgs a) {
    typedef W4Op<XT> Op;
    typedef typename Op::V V;
    constexpr int kUnit = 8 * sizeof(XT), kPieces = Op::kPieces;
    // rows a quad at a time, 16 bytes apart in the banks
    constexpr int kPitch = 512 * sizeof(XT) + 16;
    __shared__ __align__(16) uint8_t lds[kMaxWaves * RB * kPitch];
    __shared__ float sums[kMaxWaves][RB][16];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
    const int G = (a.K + 127) / 128, Q = (G + 3) / 4, n_tiles = (a.N + 15) / 16;
    const bool bf = a.scale_dtype == MQ_BF16;
    uint8_t* const mine = lds + wave * RB * kPitch;
    const int q0 = static_cast<int>(static_cast<int64_t>(Q) * wave / waves);
    const int q1 = static_cast<int>(static_cast<int64_t>(Q) * (wave + 1) / waves);
    // dense: RB rows; of a plan, 16 rows of one expert
    const int per = a.offsets ? 16 : RB;
    for (int row0 = blockIdx.y * per; row0 < a.M; row0 += gridDim.y * per) {
        int e = 0, rows = min(RB, a.M - row0);
        uint64_t alive = ~0ull;                            // which of a plan's rows have a token
        if (a.offsets) {
            const int token = a.row_token[row0 + (lane & 15)];
            alive = __ballot(static_cast<unsigned>(token) < static_cast<unsigned>(a.T)) & 0xffff;
            e = __builtin_amdgcn_readfirstlane(expert_of(a.offsets, a.E, row0));
            if (e < 0) alive = 0;
            rows = alive ? 64 - __builtin_clzll(alive) : 0;
            for (int o = threadIdx.x; o < 256; o += blockDim.x)                    // zeros for the others
                if (!(alive >> (o >> 4) & 1) && blockIdx.x * 16 + (o & 15) < a.N)
                    store1(a.y, a.y_dtype, static_cast<int64_t>(row0 + (o >> 4)) * a.N + blockIdx.x * 16 + (o & 15), 0.0f);
        }
        const int64_t tile = static_cast<int64_t>(e) * n_tiles + blockIdx.x;
        const uint8_t* const w = a.codes + tile * G * 1024 + lane * 16;
        const uint16_t* const ws = a.scales + (tile * Q * 16 + (lane & 15)) * 4 * GS;
        const uint16_t* const wz = Z ? a.zeros + (tile * Q * 16 + (lane & 15)) * 4 * GS : nullptr;
        for (int r0 = 0; r0 < rows; r0 += RB) {
            const int here = min(RB, rows - r0);
            const XT* from[RB];
#pragma unroll
            for (int i = 0; i < RB; ++i) {
                int64_t r = row0 + r0 + min(i, here - 1);
                if (a.by_token) {
                    const int t = a.row_token[r];
                    r = static_cast<unsigned>(t) < static_cast<unsigned>(a.T) ? t : 0;
                }
                from[i] = static_cast<const XT*>(a.x) + r * a.stride_x;
            }
            MxRaw8<XT> v[RB];
            mx_i4 c[4], cc[4];
            W4Quad<GS> sc, zc, ss, zz;
            auto load = [&](int q) __attribute__((always_inline)) {
#pragma unroll
                for (int i = 0; i < RB; ++i)
                    if (i < here) v[i] = load8(from[i], 512 * q + 8 * lane, a.K, 512 * (q + 1) <= a.K);
#pragma unroll
                for (int u = 0; u < 4; ++u)                // past K: the last tile, times zeros
                    c[u] = *reinterpret_cast<const mx_i4*>(w + static_cast<int64_t>(min(4 * q + u, G - 1)) * 1024);
                sc.load(ws + static_cast<int64_t>(q) * 64 * GS);
                if constexpr (Z) zc.load(wz + static_cast<int64_t>(q) * 64 * GS);
            };
            float acc[RB] = {};
            const uint8_t* const mine_at = mine + min(lane & 15, here - 1) * kPitch + (lane >> 4) * kUnit;
            if (q0 < q1) load(q0);
            for (int q = q0; q < q1; ++q) {
                int X[RB];                                 // a lane's group's sum
                mx_wave_sync();                            // the last quad's reads come first
#pragma unroll
                for (int i = 0; i < RB; ++i) {
                    X[i] = 0;
                    if (i >= here) continue;
                    put8(mine + i * kPitch + lane * kUnit, v[i]);
                    float f[8];
                    w4_values(v[i], f);
                    X[i] = w4_over_group(__float_as_int(((f[0] + f[1]) + (f[2] + f[3])) + ((f[4] + f[5]) + (f[6] + f[7]))), 128 / GS,
                                         [](int p, int r) { return __float_as_int(__int_as_float(p) + __int_as_float(r)); });
                }
                mx_wave_sync();
#pragma unroll
                for (int u = 0; u < 4; ++u) cc[u] = c[u];
                ss = sc;
                zz = zc;
                if (q + 1 < q1) load(q + 1);
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    mx_f4 P[GS] = {};
#pragma unroll
                    for (int s = 0; s < 4; ++s) {
                        V x[kPieces];
                        pieces<XT>(get8<XT>(mine_at + (16 * u + 4 * s) * kUnit), x);
                        const V b = w4_codes<typename Op::E>(cc[u][s]);
#pragma unroll
                        for (int p = 0; p < kPieces; ++p) P[s * GS / 4] = Op::mfma16(x[p], b, P[s * GS / 4]);
                    }
#pragma unroll
                    for (int g = 0; g < GS; ++g) {
                        const float sv = ss.get(u * GS + g, bf), zv = Z ? zz.get(u * GS + g, bf) : 8.0f;
#pragma unroll
                        for (int i = 0; i < RB; ++i)
                            acc[i] += sv * (P[g][i] - zv * __int_as_float(__builtin_amdgcn_readlane(X[i], (u * GS + g) * (16 / GS))));
                    }
                    // Two tiles' products at a time, the sums made right after them: put off to the
                    // end they keep a quad's products in registers, and the waves that would
                    // hide the loads out.
                    if (u & 1) {
#pragma unroll
                        for (int i = 0; i < RB; ++i) asm volatile("" : "+v"(acc[i]));
                        __builtin_amdgcn_sched_barrier(0);
                    }
                }
            }
            // the waves' sums, in the order of the waves
            if (lane < 16) {
#pragma unroll
                for (int i = 0; i < RB; ++i) sums[wave][i][lane] = acc[i];
            }
            __syncthreads();
            const int n = blockIdx.x * 16 + (threadIdx.x & 15), i = threadIdx.x >> 4;
            if (i < here && n < a.N && (alive >> (r0 + i) & 1)) {
                float y = 0;
                for (int s = 0; s < waves; ++s) y += sums[s][i][threadIdx.x & 15];
                if (a.bias) y += a.bias[n];
                store1(a.y, a.y_dtype, static_cast<int64_t>(row0 + r0 + i) * a.N + n, y);
            }
            __syncthreads();
        }
    }
}

// One workgroup: 16 MT rows x NT column tiles of 16, its waves each a run of K, tile by tile;
// rows reach the matrix instructions through LDS (256 bytes of four rows a load; lanes that
// read their own operands, 64 bytes of 16 rows, take twice the time). Bound by latency: 32 rows,
// 14336 x 4096 take 17.2 us with the weights from memory and 15.0 us from caches, where reading them
// takes 6. 32 x 64 workgroups have two waves a SIMD (212 registers, and 36 scalars in their lanes),
// which wait for half of their time; vector instructions fill 38% of the cycles (64 conversions of two
// codes and 64 sums of groups a code tile), matrix instructions 16%.
template <typename XT, int GS, bool Z, int NT, int MT, int W>
__global__ __launch_bounds__(64 * W) void k_w4_few(W4GemmArgs a) {
    constexpr int kPitch = kRowPitch<XT>, kUnit = 8 * sizeof(XT);
    // The next code tile is loaded during this one's products where registers are left for it
    // (64 tokens' rows of 64 experts, 1024 x 4096: 44 us, 48 without); 32 rows and 64 columns
    // have none (32 x 14336 x 4096: 18.7 us, 17.4 without).
    constexpr bool kAhead = NT * MT <= 4;
    // each wave's rows, then the waves' sums
    __shared__ __align__(16) uint8_t lds[W * (16 * MT * kPitch > NT * MT * 1024 ? 16 * MT * kPitch : NT * MT * 1024)];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
    const int G = (a.K + 127) / 128, Q = (G + 3) / 4, n_tiles = (a.N + 15) / 16, ct = blockIdx.x * NT;
    const int blocks = (a.M + 16 * MT - 1) / (16 * MT);
    const bool bf = a.scale_dtype == MQ_BF16;
    uint8_t* const mine = lds + wave * 16 * MT * kPitch;
    for (int rb = blockIdx.y; rb < blocks; rb += gridDim.y) {
        const int row0 = rb * 16 * MT;
        int rows = min(16 * MT, a.M - row0), e = 0;
        uint64_t alive = ~0ull;                            // which of a plan's rows have a token
        if (a.offsets) {                                   // (MT = 1) lane l % 16 is row l % 16
            const int token = a.row_token[row0 + (lane & 15)];
            alive = __ballot(static_cast<unsigned>(token) < static_cast<unsigned>(a.T)) & 0xffff;
            e = __builtin_amdgcn_readfirstlane(expert_of(a.offsets, a.E, row0));
            if (e < 0) alive = 0;
            rows = 64 - __builtin_clzll(alive | 1);
        }
        mx_f4 acc[NT][MT] = {};
        if (alive) {
            // lane l brings inputs 8 (l % 16) .. of rows 4i + l / 16
            const XT* from[4 * MT];
#pragma unroll
            for (int i = 0; i < 4 * MT; ++i) {
                int64_t r = row0 + min(4 * i + (lane >> 4), rows - 1);
                if (a.by_token) {
                    const int t = a.row_token[r];
                    r = static_cast<unsigned>(t) < static_cast<unsigned>(a.T) ? t : 0;
                }
                from[i] = static_cast<const XT*>(a.x) + r * a.stride_x;
            }
            // (through buffers, whose addresses take no vector registers)
            const int have = min(NT, n_tiles - ct), scale_bytes = w4_scale_bytes(Q, GS);
            const int64_t tile = static_cast<int64_t>(e) * n_tiles + ct;
            const __amdgpu_buffer_rsrc_t wr = buffer(a.codes + tile * G * 1024, static_cast<int64_t>(have) * G * 1024);
            const __amdgpu_buffer_rsrc_t scr = buffer(a.scales + tile * (scale_bytes / 2), static_cast<int64_t>(have) * scale_bytes);
            const __amdgpu_buffer_rsrc_t zr = Z ? buffer(a.zeros + tile * (scale_bytes / 2), static_cast<int64_t>(have) * scale_bytes) : scr;
            const int h0 = static_cast<int>(static_cast<int64_t>(G) * wave / waves);
            const int h1 = static_cast<int>(static_cast<int64_t>(G) * (wave + 1) / waves);
            MxRaw8<XT> v[4 * MT];
            mx_i4 next[NT];
            typename W4Scales<GS>::T next_s[NT], next_z[NT] = {};
            auto load = [&](int h) __attribute__((always_inline)) {
#pragma unroll
                for (int i = 0; i < 4 * MT; ++i)
                    if (4 * i < rows) v[i] = load8(from[i], 128 * h + 8 * (lane & 15), a.K, 128 * (h + 1) <= a.K);
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    const int t = w4_block_tile(j, 1, have), at = w4_scale_at(t, h, Q, GS);
                    next[j] = load16(wr, w4_lane_code(lane), w4_code_at(t, h, G));
                    next_s[j] = load_scales<GS>(scr, w4_lane_scale(lane, GS), at);
                    if constexpr (Z) next_z[j] = load_scales<GS>(zr, w4_lane_scale(lane, GS), at);
                }
            };
            if (kAhead && h0 < h1) load(h0);
            for (int h = h0; h < h1; ++h) {
                if (!kAhead) load(h);
                mx_wave_sync();                            // the last tile's reads come first
#pragma unroll
                for (int i = 0; i < 4 * MT; ++i)
                    if (4 * i < rows) put8(mine + (4 * i + (lane >> 4)) * kPitch + (lane & 15) * kUnit, v[i]);
                mx_wave_sync();
                mx_i4 c[NT];
                typename W4Scales<GS>::T sc[NT], zc[NT];
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    c[j] = next[j];
                    sc[j] = next_s[j];
                    zc[j] = next_z[j];
                }
                if (kAhead && h + 1 < h1) load(h + 1);
                if (kAhead) __builtin_amdgcn_sched_barrier(0);
                tile_products<XT, GS>(c, mine + (lane & 15) * kPitch + (lane >> 4) * kUnit, kPitch,
                                      [&](int g, int j) __attribute__((always_inline)) { return w4_float(static_cast<uint32_t>(sc[j] >> 16 * g) & 0xffff, bf); },
                                      [&](int g, int j) __attribute__((always_inline)) {
                                          return Z ? w4_float(static_cast<uint32_t>(zc[j] >> 16 * g) & 0xffff, bf) : 8.0f;
                                      },
                                      acc);
            }
        }
        add_and_store(a, reinterpret_cast<float*>(lds), acc, row0, 0, min(16 * MT, a.M - row0), ct * 16,
                      [&](int r) { return !a.offsets || (alive >> (r & 15) & 1); });
    }
}

template <typename XT, int GS, bool Z, int NT, int MT, int W>
hipError_t few(const W4GemmArgs& a, hipStream_t st) {
    const unsigned cols = static_cast<unsigned>(((a.N + 15) / 16 + NT - 1) / NT);
    const int blocks = (a.M + 16 * MT - 1) / (16 * MT);
    const int waves = static_cast<int>(w4_few_waves(static_cast<int64_t>(cols) * blocks, a.K, NT * MT));
    k_w4_few<XT, GS, Z, NT, MT, W><<<dim3(cols, blocks < 65535 ? blocks : 65535), 64 * waves, 0, st>>>(a);
    return hipGetLastError();
}

template <typename XT, int GS, bool Z, int RB>
hipError_t one(const W4GemmArgs& a, hipStream_t st) {
    const int Q = (a.K + 511) / 512, each = (Q + kMaxWaves - 1) / kMaxWaves, waves = (Q + each - 1) / each;
    const int blocks = a.offsets ? a.M / 16 : (a.M + RB - 1) / RB;
    k_w4_one<XT, GS, Z, RB><<<dim3((a.N + 15) / 16, blocks < 65535 ? blocks : 65535), 64 * waves, 0, st>>>(a);
    return hipGetLastError();
}

template <typename XT, int GS, bool Z>
hipError_t few_rows(const W4GemmArgs& a, W4Few kind, hipStream_t st) {
    if (kind == kW4One) return a.offsets || a.M == 1 ? one<XT, GS, Z, 1>(a, st) : one<XT, GS, Z, 4>(a, st);
    if constexpr (sizeof(XT) == 2) {
        if (kind == kW4Rows16x64) return few<XT, GS, Z, 4, 1, 8>(a, st);
        if (kind == kW4Rows32x32) return few<XT, GS, Z, 2, 2, 8>(a, st);
        if (kind == kW4Rows32x64) return few<XT, GS, Z, 4, 2, 8>(a, st);
    }
    return kind == kW4Rows16 ? few<XT, GS, Z, 1, 1, 8>(a, st) : few<XT, GS, Z, 2, 1, 8>(a, st);
}

template <typename XT>
hipError_t few_groups(const W4GemmArgs& a, W4Few kind, hipStream_t st) {
    if (a.group == 128) return a.zeros ? few_rows<XT, 1, true>(a, kind, st) : few_rows<XT, 1, false>(a, kind, st);
    if (a.group == 64) return a.zeros ? few_rows<XT, 2, true>(a, kind, st) : few_rows<XT, 2, false>(a, kind, st);
    return a.zeros ? few_rows<XT, 4, true>(a, kind, st) : few_rows<XT, 4, false>(a, kind, st);
}

}  // namespace

hipError_t launch_w4_few(const W4GemmArgs& a, W4Few kind, hipStream_t st) {
    switch (a.x_dtype) {
        case MQ_F32: return few_groups<float>(a, kind, st);
        case MQ_BF16: return few_groups<__bf16>(a, kind, st);
        default: return few_groups<_Float16>(a, kind, st);
    }
}

}  // namespace mq
