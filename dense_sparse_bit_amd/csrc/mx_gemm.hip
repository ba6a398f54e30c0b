// Products of microscaled 4-bit operands on the scaled matrix instructions.
//
// y[m][n] = sum over blocks b of 32 inputs of Xx[m][b] Xw[n][b] * sum over the block of
// the 4-bit codes' products. The instructions take the codes and one scale byte per lane
// (a lane holds one row's block) and add into fp32. Weights are the A operand, so a lane
// ends with neighbouring columns of one row of y.
#include "mx_device.h"
#include "mx_internal.h"

namespace mq {
namespace {

typedef unsigned int mx_u4 __attribute__((ext_vector_type(4)));

__device__ inline mx_i8 wide8(mx_i4 v) { return __builtin_shufflevector(v, v, 0, 1, 2, 3, -1, -1, -1, -1); }

// c += A B^T over one 128-input tile of 16 x 16; the scales are the low bytes
__device__ inline mx_f4 mfma16(mx_i4 a, mx_i4 b, mx_f4 c, int sa, int sb) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wide8(a), wide8(b), c, 4, 4, 0, sa, 0, sb);
}

// c += A B^T over 64 inputs of 32 x 32; the scales are byte S
template <int S>
__device__ inline mx_f16 mfma32(mx_i4 a, mx_i4 b, mx_f16 c, int sa, int sb) {
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(wide8(a), wide8(b), c, 4, 4, S, sa, S, sb);
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

// ------------------------------------------------------------------- few rows
// The matrix of rows as it is found: codes and scales of a quantized operand (MxReady),
// or rows of a type that are quantized here, block by block, in the lane that feeds the
// block to the matrix instruction.
struct MxReady {};

template <typename XT, int U>
struct XBlocks {                                   // blocks of U groups of one lane's row
    MxRaw8<XT> v[U][4];
    __device__ void load(const MxGemmArgs& a, int64_t row, int, int kc, int g, int end) {
        const XT* p = static_cast<const XT*>(a.x) + row * a.stride_x;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int k = (g + u) * 128 + kc * 32;
            const int have = g + u < end ? a.K - k : 0;
            if (have >= 32) {
#pragma unroll
                for (int i = 0; i < 4; ++i) v[u][i] = mx_load8(p + k + 8 * i, 8);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) v[u][i] = mx_load8(p + k + 8 * i, have - 8 * i);
            }
        }
    }
    __device__ void take(int u, mx_i4& codes, int& byte) const { codes = mx_quant32<XT>(v[u], byte); }
};

template <int U>
struct XBlocks<MxReady, U> {
    mx_i4 c[U];
    int b[U];
    __device__ void load(const MxGemmArgs& a, int64_t row, int G4, int kc, int g, int end) {
        const int G = (a.K + 127) / 128;
        const int at = kc * 16 + static_cast<int>(row & 15);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int h = g + u < end ? g + u : end - 1;
            const mx_i4 t = *reinterpret_cast<const mx_i4*>(a.xq + (((row >> 4) * G + h) * 64 + at) * 16);
            c[u] = g + u < end ? t : mx_i4{0, 0, 0, 0};
            b[u] = g + u < end ? a.xs[(((row >> 4) * G4 + (h >> 2)) * 64 + at) * 4 + (h & 3)] : 0;
        }
    }
    __device__ void take(int u, mx_i4& codes, int& byte) const { codes = c[u]; byte = b[u]; }
};

// One workgroup: 16 MT rows x NT column tiles of 16 (GATED: NT / 2 of each matrix), its
// waves each a run of K; the partial sums are added through LDS in the order of the
// waves. Bound by the weights' read: every load of a wave's run is issued before its
// first product, the rows' first, so that they are quantized while the weights arrive.
template <typename XT, int NT, int MT, bool GATED>
__global__ __launch_bounds__(512) void k_mx_few(MxGemmArgs a) {
    constexpr int U = sizeof(XT) == 4 || MT > 1 ? 2 : 4;     // groups loaded together
    constexpr int NC = GATED ? NT / 2 : NT;
    extern __shared__ mx_f4 red[];                            // [waves][NT * MT][64]
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
    const int G = (a.K + 127) / 128, G4 = (G + 3) / 4;
    const int n_tiles = (a.N + 15) / 16;
    const int row0 = blockIdx.y * 16 * MT, ct = blockIdx.x * NC;
    int e = 0;
    if (a.offsets) e = __builtin_amdgcn_readfirstlane(expert_of(a.offsets, a.E, row0));
    bool live[MT];
    int64_t xrow[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const int m = row0 + 16 * i + (lane & 15);
        live[i] = m < a.M && e >= 0;
        xrow[i] = m < a.M ? m : a.M - 1;
        if (a.row_token) {
            const int t = a.row_token[xrow[i]];
            const bool ok = static_cast<unsigned>(t) < static_cast<unsigned>(a.T);
            live[i] = live[i] && ok;
            if (a.x) xrow[i] = ok ? t : 0;
        }
    }
    mx_f4 acc[NT][MT] = {};
    if (e >= 0) {
        const uint8_t *w[NT], *ws[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const int c = GATED ? j >> 1 : j;
            const int64_t tile = static_cast<int64_t>(e) * n_tiles + (ct + c < n_tiles ? ct + c : n_tiles - 1);
            w[j] = ((GATED && (j & 1)) ? a.w2q : a.wq) + tile * G * 1024 + lane * 16;
            ws[j] = ((GATED && (j & 1)) ? a.w2s : a.ws) + tile * G4 * 256 + lane * 4;
        }
        const int end = static_cast<int>(static_cast<int64_t>(G) * (wave + 1) / waves);
        for (int g = static_cast<int>(static_cast<int64_t>(G) * wave / waves); g < end; g += U) {
            XBlocks<XT, U> x[MT];
#pragma unroll
            for (int i = 0; i < MT; ++i) x[i].load(a, xrow[i], G4, lane >> 4, g, end);
            mx_i4 wc[U][NT];
            int wb[U][NT];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int h = g + u < end ? g + u : end - 1;
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    wc[u][j] = *reinterpret_cast<const mx_i4*>(w[j] + static_cast<int64_t>(h) * 1024);
                    wb[u][j] = ws[j][(h >> 2) * 256 + (h & 3)];
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    mx_i4 c;
                    int b;
                    x[i].take(u, c, b);
                    // past the run's end both operands are there, and the rows' codes zero
                    if (g + u >= end) { c = mx_i4{0, 0, 0, 0}; b = 0; }
#pragma unroll
                    for (int j = 0; j < NT; ++j)
                        acc[j][i] = mfma16(wc[u][j], c, acc[j][i], wb[u][j], b);
                }
            }
        }
    }
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < MT; ++i) red[(wave * NT * MT + j * MT + i) * 64 + lane] = acc[j][i];
    // which rows are live, for the threads that write them
    __shared__ unsigned short alive[MT];
    if (wave == 0) {
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const unsigned long long mask = __ballot(live[i]);
            if (lane == 0) alive[i] = static_cast<unsigned short>(mask & 0xffff);
        }
    }
    __syncthreads();
    for (int o = threadIdx.x; o < NC * MT * 64; o += blockDim.x) {
        const int l = o & 63, i = (o >> 6) % MT, c = (o >> 6) / MT;
        const int m = row0 + 16 * i + (l & 15), n = (ct + c) * 16 + 4 * (l >> 4);
        if (m >= a.M || n >= a.N) continue;
        mx_f4 v = {}, u = {};
        for (int s = 0; s < waves; ++s) {
            v += red[(s * NT * MT + (GATED ? 2 * c : c) * MT + i) * 64 + l];
            if (GATED) u += red[(s * NT * MT + (2 * c + 1) * MT + i) * 64 + l];
        }
        if (GATED) {
#pragma unroll
            for (int r = 0; r < 4; ++r) v[r] = mx_silu(v[r]) * u[r];
        }
        if (a.bias) {
#pragma unroll
            for (int r = 0; r < 4; ++r) v[r] += n + r < a.N ? a.bias[n + r] : 0.0f;
        }
        if (!(alive[i] >> (l & 15) & 1)) v = mx_f4{0, 0, 0, 0};
        mx_store4(a.y, a.y_dtype, static_cast<int64_t>(m) * a.N + n, a.N - n, a.N % 4 == 0, v[0], v[1], v[2], v[3]);
    }
}

template <typename XT>
hipError_t few(const MxGemmArgs& a, hipStream_t st) {
    const unsigned tiles = static_cast<unsigned>((a.N + 15) / 16);
    const int G = (a.K + 127) / 128;
    const int waves = G >= 16 ? 8 : (G >= 4 ? 4 : 1);
    const unsigned rows = static_cast<unsigned>((a.M + 15) / 16);
    if (a.w2q) {
        k_mx_few<XT, 2, 1, true><<<dim3(tiles, rows), 64 * waves, waves * 2 * 1024, st>>>(a);
    } else if (a.offsets || a.M <= 16) {
        k_mx_few<XT, 1, 1, false><<<dim3(tiles, rows), 64 * waves, waves * 1024, st>>>(a);
    } else {
        k_mx_few<XT, 2, 2, false><<<dim3((tiles + 1) / 2, (rows + 1) / 2), 64 * waves, waves * 4 * 1024, st>>>(a);
    }
    return hipGetLastError();
}

// ------------------------------------------------------------------- many rows
template <int S> struct Phase { static constexpr int value = S; };
constexpr int kMaxSub = 6;                    // 32-row pieces of a row block
constexpr int kBlockTiles = 2 * kMaxSub;      // its 16-row tiles

__device__ inline __amdgpu_buffer_rsrc_t buffer(const void* base, int64_t bytes) {
    // wave-uniform by construction; said so here, or every load becomes a loop over lanes
    const uint64_t p = reinterpret_cast<uint64_t>(base);
    const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(p));
    const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(p >> 32));
    const int n = __builtin_amdgcn_readfirstlane(static_cast<int>(bytes < 0 ? 0 : (bytes < 0x7fffffff ? bytes : 0x7fffffff)));
    return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(static_cast<uint64_t>(hi) << 32 | lo), 0, n, 0x00020000);
}
__device__ inline mx_i4 load16(__amdgpu_buffer_rsrc_t r, int lane_at, int at) {
    return __builtin_bit_cast(mx_i4, __builtin_amdgcn_raw_buffer_load_b128(r, lane_at, at, 0));
}
__device__ inline int load4(__amdgpu_buffer_rsrc_t r, int lane_at, int at) {
    return static_cast<int>(__builtin_amdgcn_raw_buffer_load_b32(r, lane_at, at, 0));
}

// One wave's part of a tile of SUB * 32 rows: 64 columns (GATED: 32 of gate and 32 of
// up). Its weights go from memory straight to registers, three steps of 128 inputs
// ahead (the layout is the instruction's own); the rows, which the four waves share, go
// through two LDS stages, one barrier a step. Reads beyond the operands' ends give zero
// (buffer loads with the operands' sizes).
template <int SUB, bool GATED>
__device__ __forceinline__ void wide_tile(const MxGemmArgs& a, uint8_t* lds, int rt0, int n16, int e, int col16) {
    constexpr int XL = (SUB + 1) / 2;                // 16-row tiles that a wave fetches a step
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int G = (a.K + 127) / 128, G4 = (G + 3) / 4;
    const int n_tiles = (a.N + 15) / 16;
    // a wave with no column of its own (past N) reads the last one's and writes nothing
    const int col_there = min(col16, n_tiles - 1);
    const int64_t first = static_cast<int64_t>(e) * n_tiles + col_there;
    const int have = min(n_tiles - col_there, GATED ? 2 : 4);
    const int lane_pair = (lane >> 4 & 1) * G * 1024 + (lane >> 5) * 256 + (lane & 15) * 16;
    const int scale_pair = (lane >> 4 & 1) * G4 * 256 + (lane >> 5) * 64 + (lane & 15) * 4;
    const __amdgpu_buffer_rsrc_t wr = buffer(a.wq + first * G * 1024, static_cast<int64_t>(have) * G * 1024);
    const __amdgpu_buffer_rsrc_t wsr = buffer(a.ws + first * G4 * 256, static_cast<int64_t>(have) * G4 * 256);
    const __amdgpu_buffer_rsrc_t w2r = GATED ? buffer(a.w2q + first * G * 1024, static_cast<int64_t>(have) * G * 1024) : wr;
    const __amdgpu_buffer_rsrc_t w2sr = GATED ? buffer(a.w2s + first * G4 * 256, static_cast<int64_t>(have) * G4 * 256) : wsr;
    const int pair1 = GATED ? 0 : 2 * G * 1024, spair1 = GATED ? 0 : 2 * G4 * 256;
    const __amdgpu_buffer_rsrc_t xr = buffer(a.xq + static_cast<int64_t>(rt0) * G * 1024, static_cast<int64_t>(n16) * G * 1024);
    const __amdgpu_buffer_rsrc_t xsr = buffer(a.xs + static_cast<int64_t>(rt0) * G4 * 256, static_cast<int64_t>(n16) * G4 * 256);

    mx_i4 W[4][2][2];                                // [step % 4][column pair][half]
    // The scalar part of an offset stays within the buffer (the range check subtracts
    // it): steps past the last read the last again, and are not used.
    auto load_w = [&](int step, mx_i4 (&w)[2][2]) __attribute__((always_inline)) {
        const int g = min(step, G - 1);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            w[0][h] = load16(wr, lane_pair + h * 512, g * 1024);
            w[1][h] = load16(w2r, lane_pair + pair1 + h * 512, g * 1024);
        }
    };
    mx_i4 X[2][XL];                                  // rows on the way to LDS
    auto load_x = [&](int step, mx_i4 (&x)[XL]) __attribute__((always_inline)) {
        const int g = min(step, G - 1);
#pragma unroll
        for (int i = 0; i < XL; ++i) x[i] = load16(xr, (i * 4 + wave) * G * 1024 + lane * 16, g * 1024);
    };
    auto store_x = [&](int stage, const mx_i4 (&x)[XL]) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < XL; ++i)
            if ((i * 4 + 3 < 2 * SUB) || i * 4 + wave < 2 * SUB)
                *reinterpret_cast<mx_i4*>(lds + (stage * kBlockTiles + i * 4 + wave) * 1024 + lane * 16) = x[i];
    };
    int sw[2][2], sx[SUB][2], swn[2][2], sxn[SUB][2];
    auto load_s = [&](int quad, int (&w)[2][2], int (&x)[SUB][2]) __attribute__((always_inline)) {
        const int q = min(quad, G4 - 1);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            w[0][h] = load4(wsr, scale_pair + h * 128, q * 256);
            w[1][h] = load4(w2sr, scale_pair + spair1 + h * 128, q * 256);
#pragma unroll
            for (int i = 0; i < SUB; ++i) x[i][h] = load4(xsr, scale_pair + h * 128, (2 * i * G4 + q) * 256);
        }
    };
    mx_f16 acc[SUB][2] = {};
    const uint8_t* xl = lds + (lane >> 4 & 1) * 1024 + (lane >> 5) * 256 + (lane & 15) * 16;
    // step g (S = g % 4): products of group g; the weights of g + 3 and rows of g + 3
    // leave memory, rows of g + 1 enter LDS
    auto step = [&](auto phase, int g) __attribute__((always_inline)) {
        constexpr int S = decltype(phase)::value;
        load_w(g + 3, W[(S + 3) & 3]);
        const int stage = S & 1;
#pragma unroll
        for (int i = 0; i < SUB; ++i) {
            const mx_i4 b0 = *reinterpret_cast<const mx_i4*>(xl + (stage * kBlockTiles + 2 * i) * 1024);
            const mx_i4 b1 = *reinterpret_cast<const mx_i4*>(xl + (stage * kBlockTiles + 2 * i) * 1024 + 512);
#pragma unroll
            for (int j = 0; j < 2; ++j) acc[i][j] = mfma32<S>(W[S][j][0], b0, acc[i][j], sw[j][0], sx[i][0]);
#pragma unroll
            for (int j = 0; j < 2; ++j) acc[i][j] = mfma32<S>(W[S][j][1], b1, acc[i][j], sw[j][1], sx[i][1]);
        }
        store_x(stage ^ 1, X[stage ^ 1]);
        load_x(g + 3, X[stage ^ 1]);
        __syncthreads();
    };
    load_x(0, X[0]);
    load_w(0, W[0]);
    load_s(0, sw, sx);
    load_x(1, X[1]);
    load_w(1, W[1]);
    load_w(2, W[2]);
    store_x(0, X[0]);
    load_x(2, X[0]);
    __syncthreads();
    int g = 0;
    for (; g + 4 <= G; g += 4) {
        load_s((g >> 2) + 1, swn, sxn);
        step(Phase<0>{}, g);
        step(Phase<1>{}, g + 1);
        step(Phase<2>{}, g + 2);
        step(Phase<3>{}, g + 3);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int j = 0; j < 2; ++j) sw[j][h] = swn[j][h];
#pragma unroll
            for (int i = 0; i < SUB; ++i) sx[i][h] = sxn[i][h];
        }
    }
    if (g < G) {
        step(Phase<0>{}, g);
        if (g + 1 < G) step(Phase<1>{}, g + 1);
        if (g + 2 < G) step(Phase<2>{}, g + 2);
    }

    // lane: row m = l % 32 of a piece; register r: column 8 (r / 4) + 4 (l / 32) + r % 4
    const int lm = lane & 31;
#pragma unroll
    for (int i = 0; i < SUB; ++i) {
        const int64_t m = rt0 * 16 + 32 * i + lm;
        const bool row_there = 32 * i + lm < n16 * 16 && m < a.M;
        bool live = row_there;
        if (GATED && row_there) live = static_cast<unsigned>(a.row_token[m]) < static_cast<unsigned>(a.T);
#pragma unroll
        for (int j = 0; j < (GATED ? 1 : 2); ++j) {
            const int n0 = col16 * 16 + 32 * j;
            float v[16];
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                v[r] = GATED ? mx_silu(acc[i][0][r]) * acc[i][1][r] : acc[i][j][r];
                if (GATED && !live) v[r] = 0.0f;
            }
            if (a.bias) {
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int n = n0 + 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3);
                    v[r] += n < a.N ? a.bias[n] : 0.0f;
                }
            }
            if (a.y_dtype != MQ_F32 && a.N % 8 == 0) {
                // halves of the wave trade pieces: eight neighbouring columns a lane
#pragma unroll
                for (int c = 0; c < 4; c += 2) {
                    uint32_t p[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        p[k] = a.y_dtype == MQ_BF16 ? mx_pack2<__bf16>(v[4 * c + 2 * k], v[4 * c + 2 * k + 1])
                                                    : mx_pack2<_Float16>(v[4 * c + 2 * k], v[4 * c + 2 * k + 1]);
                    const auto s0 = __builtin_amdgcn_permlane32_swap(p[0], p[2], false, false);
                    const auto s1 = __builtin_amdgcn_permlane32_swap(p[1], p[3], false, false);
                    const int n = n0 + 8 * c + 8 * (lane >> 5);
                    if (row_there && n < a.N)
                        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.y) + m * a.N + n) = make_uint4(s0[0], s1[0], s0[1], s1[1]);
                }
            } else {
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const int n = n0 + 8 * c + 4 * (lane >> 5);
                    if (row_there && n < a.N)
                        mx_store4(a.y, a.y_dtype, m * a.N + n, a.N - n, a.N % 4 == 0, v[4 * c], v[4 * c + 1], v[4 * c + 2],
                                  v[4 * c + 3]);
                }
            }
        }
    }
}

// zeros for rows after the last expert's
__device__ inline void zero_rows(const MxGemmArgs& a, int rt0, int n16, int n0, int cols) {
    const int c = n0 + cols < a.N ? cols : a.N - n0;
    for (int i = threadIdx.x; i < n16 * 16 * ((c + 3) / 4); i += blockDim.x) {
        const int64_t m = rt0 * 16 + i / ((c + 3) / 4);
        const int n = n0 + 4 * (i % ((c + 3) / 4));
        if (m < a.M) mx_store4(a.y, a.y_dtype, m * a.N + n, a.N - n, a.N % 4 == 0, 0.0f, 0.0f, 0.0f, 0.0f);
    }
}

// Four waves, each 64 columns (GATED: 32), of one row block. Workgroups go to the eight
// dies in turn, so each die takes a run of neighbouring tiles: they share rows and
// weights in its L2.
template <bool GATED>
__global__ __launch_bounds__(256) void k_mx_wide(MxGemmArgs a, int blocks, int block_tiles) {
    __shared__ __align__(16) uint8_t lds[2 * kBlockTiles * 1024];
    constexpr int kCols = GATED ? 128 : 256;
    const int ncol = (a.N + kCols - 1) / kCols;
    const int count = a.tiles ? a.tiles[0] : blocks;
    const int total = count * ncol, share = (total + 7) / 8;
    const int t = static_cast<int>(blockIdx.x & 7) * share + static_cast<int>(blockIdx.x >> 3);
    if (static_cast<int>(blockIdx.x >> 3) >= share || t >= total) return;
    int e = 0, rt0, n16, col;
    if (a.tiles) {
        const int4 tile = *reinterpret_cast<const int4*>(a.tiles + 4 + 4 * (t / ncol));
        e = __builtin_amdgcn_readfirstlane(tile.x);
        rt0 = __builtin_amdgcn_readfirstlane(tile.y);
        n16 = __builtin_amdgcn_readfirstlane(tile.z);
        col = t % ncol;
    } else {
        rt0 = (t % blocks) * block_tiles;
        n16 = min(block_tiles, (a.M + 15) / 16 - rt0);
        col = t / blocks;
    }
    if (e < 0) {
        if (GATED) zero_rows(a, rt0, n16, col * kCols, kCols);
        return;
    }
    const int col16 = col * (kCols / 16) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) * (kCols / 64);
    switch ((n16 + 1) / 2) {
        case 1: wide_tile<1, GATED>(a, lds, rt0, n16, e, col16); break;
        case 2: wide_tile<2, GATED>(a, lds, rt0, n16, e, col16); break;
        case 3: wide_tile<3, GATED>(a, lds, rt0, n16, e, col16); break;
        case 4: wide_tile<4, GATED>(a, lds, rt0, n16, e, col16); break;
        case 5: wide_tile<5, GATED>(a, lds, rt0, n16, e, col16); break;
        default: wide_tile<6, GATED>(a, lds, rt0, n16, e, col16); break;
    }
}

// Row blocks of a plan: each expert's rows in blocks of at most kBlockTiles 16-row
// tiles, of even sizes; then the rows after the last expert's, with expert -1.
// tiles: [0] their number, then (expert, first 16-row tile, 16-row tiles, 0) each.
__global__ __launch_bounds__(1024) void k_mx_tiles(const int32_t* offsets, int E, int P16, int32_t* tiles, int cap) {
    __shared__ int last[1024 + 1];             // blocks up to and with expert e
    __shared__ int wave_sum[16];
    const int tid = threadIdx.x, lane = tid & 63;
    int from = 0, to = 0;
    if (tid <= E) {
        from = min(max(offsets[tid] >> 4, 0), P16);
        to = tid < E ? min(max(offsets[tid + 1] >> 4, 0), P16) : P16;
    }
    int n = to > from ? (to - from + kBlockTiles - 1) / kBlockTiles : 0;
    for (int o = 1; o < 64; o <<= 1) {
        const int v = __shfl_up(n, o);
        if (lane >= o) n += v;
    }
    if (lane == 63) wave_sum[tid >> 6] = n;
    __syncthreads();
    for (int w = 0; w < (tid >> 6); ++w) n += wave_sum[w];
    last[tid] = n;
    // E = 1024: the rows after the last expert's have no thread of their own
    if (tid == 1023) {
        const int rest = E == 1024 ? max(0, P16 - min(max(offsets[1024] >> 4, 0), P16)) : 0;
        last[1024] = n + (rest + kBlockTiles - 1) / kBlockTiles;
    }
    __syncthreads();
    const int count = min(last[1024], cap);
    if (tid == 0) tiles[0] = count;
    for (int i = tid; i < count; i += 1024) {
        int lo = 0, hi = 1024;                  // first e with last[e] > i
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (last[mid] > i) hi = mid; else lo = mid + 1;
        }
        const int f = min(max(offsets[lo] >> 4, 0), P16);
        const int l = lo < E ? min(max(offsets[lo + 1] >> 4, 0), P16) : P16;
        const int c = l - f, before = lo ? last[lo - 1] : 0;
        const int parts = (c + kBlockTiles - 1) / kBlockTiles, j = i - before;
        // pieces of 32 rows are whole; the parts differ by one piece at most
        const int pieces = (c + 1) / 2;
        const int p0 = static_cast<int>(static_cast<int64_t>(pieces) * j / parts);
        const int p1 = static_cast<int>(static_cast<int64_t>(pieces) * (j + 1) / parts);
        int4* at = reinterpret_cast<int4*>(tiles + 4 + 4 * i);
        *at = make_int4(lo < E ? lo : -1, f + 2 * p0, min(2 * p1, c) - 2 * p0, 0);
    }
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

int64_t tiles_cap(int64_t P, int64_t E) { return P / 16 / kBlockTiles + E + 2; }

}  // namespace

bool mx_few_rows(int64_t M, int64_t N, int64_t K) { return M <= 32; }

hipError_t launch_mx_few(const MxGemmArgs& a, hipStream_t st) {
    if (!a.x) return few<MxReady>(a, st);
    switch (a.x_dtype) {
        case MQ_F32: return few<float>(a, st);
        case MQ_BF16: return few<__bf16>(a, st);
        default: return few<_Float16>(a, st);
    }
}

hipError_t launch_mx_wide(const MxGemmArgs& a, hipStream_t st) {
    const int rt = (a.M + 15) / 16;
    const bool gated = a.w2q != nullptr;
    const int64_t ncol = (a.N + (gated ? 127 : 255)) / (gated ? 128 : 256);
    int blocks = 0, block_tiles = 0;
    if (!a.tiles) {
        blocks = (rt + kBlockTiles - 1) / kBlockTiles;
        block_tiles = ((rt + blocks - 1) / blocks + 1) / 2 * 2;
        blocks = (rt + block_tiles - 1) / block_tiles;
    }
    const int64_t n = a.tiles ? tiles_cap(a.M, a.E) : blocks;
    const unsigned grid = static_cast<unsigned>((n * ncol + 7) / 8 * 8);
    if (gated)
        k_mx_wide<true><<<grid, 256, 0, st>>>(a, blocks, block_tiles);
    else
        k_mx_wide<false><<<grid, 256, 0, st>>>(a, blocks, block_tiles);
    return hipGetLastError();
}

int64_t mx_tiles_size(int64_t P, int64_t E) { return 4 + 4 * tiles_cap(P, E); }

hipError_t launch_mx_tiles(const int32_t* offsets, int E, int64_t P, int32_t* tiles, hipStream_t st) {
    k_mx_tiles<<<1, 1024, 0, st>>>(offsets, E, static_cast<int>(P / 16), tiles, static_cast<int>(tiles_cap(P, E)));
    return hipGetLastError();
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
