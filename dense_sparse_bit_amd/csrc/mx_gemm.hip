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
// A batch is four groups (512 inputs) of a wave's run of K.
constexpr int kBatch = 4;
// The rows' codes of a batch in LDS, per 16 rows: [16 blocks][16 rows][16 B]; blocks are
// 16 B further apart than they are long, so that a row's 16 blocks, written by one
// instruction, fall into different banks. Then a word of scales per (block % 4, row).
constexpr int kBlockPitch = 16 * 16 + 16;
constexpr int kRowsLds = 16 * kBlockPitch + 256;

struct MxReady {};                                   // rows that are quantized already

// Quantizes rows 0 .. rows - 1 (row i of x: row_at(i), wave-uniform) of the groups
// [g, min(g + 4, end)) into the wave's LDS: a row's 512 inputs are one 16-byte load a
// lane, four lanes a block. RB rows are loaded before the first is converted; `between`
// runs after the first loads are issued (the weights' loads, which must come after them:
// loads complete in order).
template <typename XT, int RB, typename Row, typename Between>
__device__ __forceinline__ void rows_to_lds(const XT* x, int64_t stride, int K, int rows, Row row_at, int g, int end,
                                            uint8_t* lds, Between between) {
    const int lane = threadIdx.x & 63;
    const int k = g * 128 + 8 * lane;
    auto put = [&](int r, const MxRaw8<XT>& v) __attribute__((always_inline)) {
        int byte;
        const uint32_t word = mx_quant8(v, byte);
        uint8_t* to = lds + (r >> 4) * kRowsLds;
        *reinterpret_cast<uint32_t*>(to + (lane >> 2) * kBlockPitch + (r & 15) * 16 + (lane & 3) * 4) = word;
        if ((lane & 3) == 0) to[16 * kBlockPitch + ((lane >> 2 & 3) * 16 + (r & 15)) * 4 + (lane >> 4)] = byte;
    };
    auto all = [&](auto load) __attribute__((always_inline)) {
        MxRaw8<XT> v[RB];
#pragma unroll
        for (int i = 0; i < RB; ++i) v[i] = load(min(i, rows - 1));
        between();
#pragma unroll
        for (int i = 0; i < RB; ++i)
            if (RB == 1 || i < rows) put(i, v[i]);
        for (int r = RB; r < rows; r += RB) {
#pragma unroll
            for (int i = 0; i < RB; ++i) v[i] = load(min(r + i, rows - 1));
#pragma unroll
            for (int i = 0; i < RB; ++i)
                if (r + i < rows) put(r + i, v[i]);
        }
    };
    const int lim = min(K, end * 128);
    if ((g + kBatch) * 128 <= lim) {
        all([&](int r) __attribute__((always_inline)) { return mx_load8(x + row_at(r) * stride + k, 8); });
    } else if (K >= 8) {                                   // the end of the run or of the rows
        all([&](int r) __attribute__((always_inline)) { return mx_load8_tail(x + row_at(r) * stride, k, K, lim); });
    } else {
        between();
        for (int r = 0; r < rows; ++r) put(r, mx_load8(x + row_at(r) * stride + k, K - k));
    }
}

// One wave's share of 16 MT rows x NT weight tiles: the products of the groups
// [g0, end). w and ws: the tiles' codes and scales, at this lane. Bound by the weights'
// read: a batch's loads are all issued before its first product.
template <typename XT, int NT, int MT, int RB, typename Row>
__device__ __forceinline__ void few_run(const MxGemmArgs& a, const uint8_t* const (&w)[NT], const uint8_t* const (&ws)[NT],
                                        int rows, Row row_at, int g0, int end, uint8_t* lds, mx_f4 (&acc)[NT][MT]) {
    const int lane = threadIdx.x & 63;
    for (int g = g0; g < end; g += kBatch) {
        mx_i4 wc[kBatch][NT];
        int wb[kBatch][NT];
        auto load_w = [&]() __attribute__((always_inline)) {
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const int h = min(g + u, end - 1);         // past the run's end: its last, times codes of zero
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    wc[u][j] = *reinterpret_cast<const mx_i4*>(w[j] + static_cast<int64_t>(h) * 1024);
                    wb[u][j] = ws[j][(h >> 2) * 256 + (h & 3)];
                }
            }
        };
        if constexpr (__is_same(XT, MxReady)) {
            const int G = (a.K + 127) / 128, G4 = (G + 3) / 4;
            mx_i4 c[kBatch][MT];
            int b[kBatch][MT];
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    const int h = min(g + u, end - 1);
                    const int64_t m = row_at(min(16 * i + (lane & 15), rows - 1));
                    const int at = (lane & 48) + static_cast<int>(m & 15);
                    c[u][i] = *reinterpret_cast<const mx_i4*>(a.xq + (((m >> 4) * G + h) * 64 + at) * 16);
                    b[u][i] = a.xs[(((m >> 4) * G4 + (h >> 2)) * 64 + at) * 4 + (h & 3)];
                    if (g + u >= end) { c[u][i] = mx_i4{0, 0, 0, 0}; b[u][i] = 0; }
                }
            }
            load_w();
#pragma unroll
            for (int u = 0; u < kBatch; ++u)
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int j = 0; j < NT; ++j) acc[j][i] = mfma16(wc[u][j], c[u][i], acc[j][i], wb[u][j], b[u][i]);
        } else {
            mx_wave_sync();                                // the last batch's reads come first
            rows_to_lds<XT, RB>(static_cast<const XT*>(a.x), a.stride_x, a.K, rows, row_at, g, end, lds, load_w);
            mx_wave_sync();
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const uint8_t* from = lds + i * kRowsLds;
                const uint32_t b = *reinterpret_cast<const uint32_t*>(from + 16 * kBlockPitch + lane * 4);
#pragma unroll
                for (int u = 0; u < kBatch; ++u) {
                    const mx_i4 c = *reinterpret_cast<const mx_i4*>(from + (u * 4 + (lane >> 4)) * kBlockPitch + (lane & 15) * 16);
#pragma unroll
                    for (int j = 0; j < NT; ++j) acc[j][i] = mfma16(wc[u][j], c, acc[j][i], wb[u][j], b >> 8 * u);
                }
            }
        }
    }
}

// One workgroup: 16 MT rows x NT column tiles of 16 (GATED: NT / 2 of each matrix), its
// waves each a run of K; the partial sums are added through LDS in the order of the
// waves. Bound by the weights' read where there are enough of them, in us, on weights that no
// cache holds / that the last-level cache does: one row of 28672 x 8192 23.6 (5.3 TB/s) / 20.8,
// 14336 x 4096 8.4 / 5.6, 17408 x 5120 12.9 / 10.6; of 4096 x 4096 4.7 / 3.6, most of it the
// latency of a launch, the rows' quantization and one batch of loads. Sixteen quantized rows
// of 28672 x 8192 30.2 (4.1 TB/s), of 17408 x 5120 17.5 (2.7 TB/s: eight waves have five groups
// each, so every second batch is mostly repeats).
template <typename XT, int NT, int MT, int RB, bool GATED>
__global__ __launch_bounds__(512) void k_mx_few(MxGemmArgs a) {
    constexpr int NC = GATED ? NT / 2 : NT;
    extern __shared__ __align__(16) uint8_t lds[];    // each wave's rows, then the waves' sums
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
    const int G = (a.K + 127) / 128, G4 = (G + 3) / 4;
    const int n_tiles = (a.N + 15) / 16;
    const int row0 = blockIdx.y * 16 * MT, ct = blockIdx.x * NC;
    int rows = min(16 * MT, a.M - row0), e = 0, token = 0;
    uint64_t alive = ~0ull;                            // which of the rows have a token
    if constexpr (GATED) {
        // (MT = 1) lane l % 16 is row l % 16 of the plan's tile
        token = a.row_token[row0 + (lane & 15)];
        alive = __ballot(static_cast<unsigned>(token) < static_cast<unsigned>(a.T)) & 0xffff;
        e = __builtin_amdgcn_readfirstlane(expert_of(a.offsets, a.E, row0));
        if (e < 0) alive = 0;
        rows = 64 - __builtin_clzll(alive | 1);
    }
    mx_f4 acc[NT][MT] = {};
    if (alive) {
        const uint8_t *w[NT], *ws[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const int c = GATED ? j >> 1 : j;
            const int64_t tile = static_cast<int64_t>(e) * n_tiles + (ct + c < n_tiles ? ct + c : n_tiles - 1);
            w[j] = ((GATED && (j & 1)) ? a.w2q : a.wq) + tile * G * 1024 + lane * 16;
            ws[j] = ((GATED && (j & 1)) ? a.w2s : a.ws) + tile * G4 * 256 + lane * 4;
        }
        auto row_at = [&](int i) __attribute__((always_inline)) -> int64_t {
            if (!GATED) return row0 + i;
            const int t = __builtin_amdgcn_readlane(token, i & 15);
            return static_cast<unsigned>(t) < static_cast<unsigned>(a.T) ? t : 0;
        };
        const int g0 = static_cast<int>(static_cast<int64_t>(G) * wave / waves);
        const int end = static_cast<int>(static_cast<int64_t>(G) * (wave + 1) / waves);
        if constexpr (__is_same(XT, MxReady)) {
            few_run<XT, NT, MT, RB>(a, w, ws, rows, row_at, g0, end, nullptr, acc);
        } else {
            few_run<XT, NT, MT, RB>(a, w, ws, rows, row_at, g0, end, lds + wave * MT * kRowsLds, acc);
        }
    }
    mx_f4* red = reinterpret_cast<mx_f4*>(lds);        // [waves][NT * MT][64]
    __syncthreads();
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < MT; ++i) red[(wave * NT * MT + j * MT + i) * 64 + lane] = acc[j][i];
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
        if (GATED && !(alive >> (l & 15) & 1)) v = mx_f4{0, 0, 0, 0};
        mx_store4(a.y, a.y_dtype, static_cast<int64_t>(m) * a.ldy + n, a.N - n, a.ldy % 4 == 0, v[0], v[1], v[2], v[3]);
    }
}

template <typename XT, int NT, int MT, int RB, bool GATED>
hipError_t few(const MxGemmArgs& a, hipStream_t st) {
    constexpr int NC = GATED ? NT / 2 : NT;
    const unsigned cols = static_cast<unsigned>(((a.N + 15) / 16 + NC - 1) / NC);
    const unsigned rows = static_cast<unsigned>((a.M + 16 * MT - 1) / (16 * MT));
    const int G = (a.K + 127) / 128;
    // A wave has at least two groups, from four waves on. Eight waves or four from K = 4096 on:
    // 4.2 / 4.4 us (1 x 4096 x 4096), 8.5 / 8.9 (N = 14336); sixteen change nothing.
    const int waves = G >= 32 ? 8 : (G >= 8 ? 4 : (G >= 4 ? 2 : 1));
    constexpr int kRowsBytes = __is_same(XT, MxReady) ? 0 : kRowsLds;
    const size_t lds = static_cast<size_t>(waves) * (kRowsBytes > NT * 1024 ? kRowsBytes : NT * 1024) * MT;
    k_mx_few<XT, NT, MT, RB, GATED><<<dim3(cols, rows), 64 * waves, lds, st>>>(a);
    return hipGetLastError();
}

// Rows that are quantized on the way: at most 16 a workgroup. RB (rows whose loads are in
// flight together) follows their number; two column tiles a wave, which share the rows'
// quantization, where there are enough tiles for two rounds of workgroups without.
// Measured (K = 4096): 4 rows, N = 4096: RB 4 / 8: 4.1 / 4.5 us; 16 rows, one tile / two:
// N = 4096 6.7 / 7.2 us, N = 14336 15.5 / 11.4 us.
template <typename XT>
hipError_t few_raw(const MxGemmArgs& a, int64_t rows, hipStream_t st) {
    if (a.w2q) {
        if (rows == 1) return few<XT, 2, 1, 1, true>(a, st);
        return rows <= 4 ? few<XT, 2, 1, 4, true>(a, st) : few<XT, 2, 1, 8, true>(a, st);
    }
    if (rows == 1) return few<XT, 1, 1, 1, false>(a, st);
    if (rows <= 4) return few<XT, 1, 1, 4, false>(a, st);
    return a.N > 8192 ? few<XT, 2, 1, 8, false>(a, st) : few<XT, 1, 1, 8, false>(a, st);
}

// The experts' down products of few tokens, each token by itself: workgroup (16 NT
// columns, token), a wave for each slot (of up to kDownWaves; fewer slots: several waves
// split a slot's K). The slots' sums meet in LDS and are added in their order, so the
// rows need no memory of their own and no second launch. Experts that tokens share are
// read once a token: for few tokens there are few of those. One token, 8 experts of 4096 x
// 1024: 6.0 us, bound by the chain of loads (slot's row, its expert, the row, the weights).
constexpr int kDownWaves = 16;

template <typename XT, int NT>
__global__ __launch_bounds__(64 * kDownWaves) void k_mx_down_few(MxGemmArgs a, const int32_t* row_of, const float* weights, int k,
                                                                 int parts, int64_t P) {
    extern __shared__ __align__(16) uint8_t lds[];        // each wave's rows; the sums [k * parts][16 NT]
    mx_f4* sums = reinterpret_cast<mx_f4*>(lds + kDownWaves * kRowsLds);
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int G = (a.K + 127) / 128, G4 = (G + 3) / 4;
    const int n_tiles = (a.N + 15) / 16, ct = blockIdx.x * NT;
    const int64_t t = blockIdx.y;
    for (int u = wave; u < k * parts; u += kDownWaves) {
        const int part = u % parts;
        const int p = __builtin_amdgcn_readfirstlane(row_of[t * k + u / parts]);
        const int e = p >= 0 && p < P ? __builtin_amdgcn_readfirstlane(expert_of(a.offsets, a.E, p)) : -1;
        mx_f4 acc[NT][1] = {};
        if (e >= 0) {
            const uint8_t *w[NT], *ws[NT];
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const int64_t tile = static_cast<int64_t>(e) * n_tiles + min(ct + j, n_tiles - 1);
                w[j] = a.wq + tile * G * 1024 + lane * 16;
                ws[j] = a.ws + tile * G4 * 256 + lane * 4;
            }
            few_run<XT, NT, 1, 1>(a, w, ws, 1, [&](int) __attribute__((always_inline)) -> int64_t { return p; },
                                  G * part / parts, G * (part + 1) / parts, lds + wave * kRowsLds, acc);
        }
        if ((lane & 15) == 0) {
#pragma unroll
            for (int j = 0; j < NT; ++j) sums[(u * NT + j) * 4 + (lane >> 4)] = acc[j][0];
        }
    }
    __syncthreads();
    if (threadIdx.x < 4 * NT) {
        const int n = ct * 16 + 4 * threadIdx.x;
        mx_f4 y = {};
        for (int j = 0; j < k; ++j) {
            mx_f4 v = sums[j * parts * NT * 4 + threadIdx.x];
            for (int i = 1; i < parts; ++i) v += sums[(j * parts + i) * NT * 4 + threadIdx.x];
            y += weights[t * k + j] * v;
        }
        if (n < a.N) mx_store4(a.y, a.y_dtype, t * a.N + n, a.N - n, a.N % 4 == 0, y[0], y[1], y[2], y[3]);
    }
}

template <typename XT>
hipError_t down_few(const MxGemmArgs& a, const int32_t* row_of, const float* weights, int k, int64_t P, hipStream_t st) {
    const int G = (a.K + 127) / 128;
    int parts = kDownWaves / k > 1 ? kDownWaves / k : 1;
    if (parts > G) parts = G;
    const size_t lds = kDownWaves * kRowsLds + static_cast<size_t>(k) * parts * 64;
    k_mx_down_few<XT, 1><<<dim3(static_cast<unsigned>((a.N + 15) / 16), static_cast<unsigned>(a.T)), 64 * kDownWaves, lds, st>>>(
        a, row_of, weights, k, parts, P);
    return hipGetLastError();
}

// ------------------------------------------------------------------- many rows
template <int S> struct Phase { static constexpr int value = S; };
constexpr int kMaxSub = kBlockTiles / 2;      // 32-row pieces of a row block
// Its rows' scales for four steps: words of four bytes, one for each block % 4 and row;
// blocks are a row block and 32 words apart, so that neighbouring rows' words, and with
// them two blocks', lie in different banks.
constexpr int kScaleBlock = 128 * kMaxSub + 128;
constexpr int kScaleBytes = 4 * kScaleBlock;
constexpr int kOutBytes = 32 * (64 * 4 + 16); // a wave's results on their way out: 32 rows, 16 B apart in the banks

// Pieces of 32 rows in a row block, for `rows32` pieces in all over `cols` column blocks:
// the least time of n workgroups of s pieces each, two to a CU. Measured in us (K = 1024,
// 4096, 14336): a round of 512 takes from 6.2, 15.4, 50 (s = 1) to 12.4, 34.8, 104 (s = 4),
// one of at most 256, alone on their CUs, from 5.3, 11.7, 30 to 11.5, 21.6, 57. Rounds
// after the first run into one another; the last one's end costs about 0.15 of one.
int wide_pieces(int64_t rows32, int64_t cols, int64_t K, double* time) {
    const double g = static_cast<double>((K + 127) / 128);
    int best = 1;
    double least = 0.0;
    for (int s = 1; s <= kMaxSub; ++s) {
        const int64_t n = (rows32 + s - 1) / s * cols;
        const double round = 2.0 + 0.8 * s + g * (0.255 + 0.157 * s), alone = 2.0 + 1.4 * s + g * (0.155 + 0.07 * s);
        const double t = n <= 256 ? alone : (n <= 512 ? round : (static_cast<double>(n) / 512 + 0.15) * round);
        if (s == 1 || t < least) {
            least = t;
            best = s;
        }
    }
    if (time) *time = least;
    return best;
}

// One wave's part of a tile of SUB * 32 rows: 64 columns (GATED: 32 of gate and 32 of
// up). Its weights go from memory straight to registers, two steps of 128 inputs ahead
// (the layout is the instruction's own); the rows and their scales, which the four waves
// share, go through four LDS stages, one barrier a step. Reads beyond the operands' ends
// give zero (buffer loads with the operands' sizes). Two workgroups share a CU: one's
// products fill the other's barriers, first loads and stores (against one workgroup of 192
// rows a CU, whose waves have twice the registers: 32768 x 4096 x 1024 97 / 124 us, 8192^3
// 262 / 286, 2048 x 17408 x 5120 106 / 105).
// Measured: 8192^3 4.2 PFLOP/s, where products fed from registers reach 6.6 on such codes.
// The matrix units are busy for half the cycles, LDS for a third; with all codes alike the
// same products run at 5.3, so the clock that the power leaves is a good part of it.
template <typename T, int SUB, bool GATED>
__device__ __forceinline__ void wide_tile(const MxGemmArgs& a, uint8_t* lds, int rt0, int n16, int e, int col16) {
    constexpr int XL = (SUB + 1) / 2;                // 16-row tiles that a wave fetches a step
    // LDS: a tile's four runs of 16 blocks; gathered rows are written across the runs, and
    // 64 bytes between these keep eight lanes on different banks
    constexpr int kBlock = GATED ? 320 : 256, kTile = 4 * kBlock, kStage = kBlockTiles * kTile + (GATED ? 16 : 0);
    static_assert(4 * XL <= kBlockTiles);            // (odd SUB: two tiles of zeros too, and no branch)
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int G = (a.K + 127) / 128, G4 = (G + 3) / 4;
    const int n_tiles = (a.N + 15) / 16;
    // a wave with no column of its own (past N) reads the last one's and writes nothing
    const int col_there = min(col16, n_tiles - 1);
    const int64_t first = static_cast<int64_t>(e) * a.w_tiles + a.w_tile0 + col_there;
    const int have = min(n_tiles - col_there, GATED ? 2 : 4);
    const int lane_pair = (lane >> 4 & 1) * G * 1024 + (lane >> 5) * 256 + (lane & 15) * 16;
    const int scale_pair = (lane >> 4 & 1) * G4 * 256 + (lane >> 5) * 64 + (lane & 15) * 4;
    const __amdgpu_buffer_rsrc_t wr = buffer(a.wq + first * G * 1024, static_cast<int64_t>(have) * G * 1024);
    const __amdgpu_buffer_rsrc_t wsr = buffer(a.ws + first * G4 * 256, static_cast<int64_t>(have) * G4 * 256);
    const __amdgpu_buffer_rsrc_t w2r = GATED ? buffer(a.w2q + first * G * 1024, static_cast<int64_t>(have) * G * 1024) : wr;
    const __amdgpu_buffer_rsrc_t w2sr = GATED ? buffer(a.w2s + first * G4 * 256, static_cast<int64_t>(have) * G4 * 256) : wsr;
    const int pair1 = GATED ? 0 : 2 * G * 1024, spair1 = GATED ? 0 : 2 * G4 * 256;
    // rows: tiles in the weights' layout, or (GATED) rows of their own, picked by token:
    const int pitch = (G + 1) / 2 * 128;
    const __amdgpu_buffer_rsrc_t xr = GATED ? buffer(a.xq, static_cast<int64_t>(a.T) * pitch)
                                            : buffer(a.xq + static_cast<int64_t>(rt0) * G * 1024, static_cast<int64_t>(n16) * G * 1024);
    const __amdgpu_buffer_rsrc_t xsr = GATED ? buffer(a.xs, static_cast<int64_t>(a.T) * G4 * 16)
                                             : buffer(a.xs + static_cast<int64_t>(rt0) * G4 * 256, static_cast<int64_t>(n16) * G4 * 256);
    auto token = [&](int r) __attribute__((always_inline)) -> uint32_t {          // of no row: token 0's, never written
        const int t = r < n16 * 16 ? a.row_token[rt0 * 16 + r] : 0;
        return static_cast<uint32_t>(t) < static_cast<uint32_t>(a.T) ? t : 0;
    };
    uint32_t xat[2][XL], xsat;                       // this lane's places in xr and xsr
#pragma unroll
    for (int p = 0; p < 2 * XL; ++p)
        xat[p / XL][p % XL] = GATED ? token((p % XL * 4 + wave) * 16 + 8 * (p / XL) + (lane >> 3)) * pitch + (lane & 7) * 16
                                    : (p % XL * 4 + wave) * G * 1024 + lane * 16;
    // a quad of steps' scales, 8 bytes a thread
    if constexpr (GATED) xsat = token(threadIdx.x >> 1) * G4 * 16 + (threadIdx.x & 1) * 8;
    else xsat = (threadIdx.x >> 5) * G4 * 256 + (threadIdx.x & 31) * 8;

    mx_i4 W[4][2][2];                                // [step % 4][column pair][half]
    // The scalar part of an offset stays within the buffer (the range check subtracts
    // it): steps past the last read the last again, and are not used.
    auto load_w = [&](int step, int piece) __attribute__((always_inline)) {       // a fourth of a step's weights
        const int g = min(step, G - 1), h = piece & 1;
        return piece < 2 ? load16(wr, lane_pair + h * 512, g * 1024) : load16(w2r, lane_pair + pair1 + h * 512, g * 1024);
    };
    // Rows on the way to LDS, two steps' worth: X[s][p] is piece p of step g + s of a pair
    // of steps; of gathered rows, rows 8 s to 8 s + 7 of a tile for both steps (eight lanes
    // read 128 bytes of a row: a whole line, where one step's 64 were half of one).
    mx_i4 X[2][XL];
    auto load_x = [&](int step, int s, int i) __attribute__((always_inline)) {     // step: the pair's first
        if constexpr (GATED) return load16(xr, xat[s][i], min(step, (G - 1) & ~1) * 64);
        else return load16(xr, xat[0][i], min(step + s, G - 1) * 1024);
    };
    auto store_x = [&](int stage, int s, int i, mx_i4 x) __attribute__((always_inline)) {   // stage: the pair's first
        uint8_t* to = lds + (i * 4 + wave) * kTile;
        if constexpr (GATED) to += (stage + (lane >> 2 & 1)) * kStage + (lane & 3) * kBlock + (8 * s + (lane >> 3)) * 16;
        else to += (stage + s) * kStage + lane * 16;
        *reinterpret_cast<mx_i4*>(to) = x;
    };
    // The rows' scales, in two buffers that take turns by quads of steps. A thread brings two
    // words: two rows' of one block (GATED: two blocks' of one row).
    uint8_t* scales = lds + 4 * kStage;
    mx_i2 XS;
    auto load_xs = [&](int quad) __attribute__((always_inline)) {
        const int q = min(quad, G4 - 1);
        return __builtin_bit_cast(mx_i2, __builtin_amdgcn_raw_buffer_load_b64(xsr, xsat, q * (GATED ? 16 : 256), 0));
    };
    uint8_t* const scales_to = scales + (GATED ? (threadIdx.x & 1) * 2 * kScaleBlock + (threadIdx.x >> 1) * 4
                                               : (threadIdx.x >> 3 & 3) * kScaleBlock + (threadIdx.x >> 5) * 64 + (threadIdx.x & 7) * 8);
    auto store_xs = [&](int at, mx_i2 v) __attribute__((always_inline)) {
        if constexpr (GATED) {
            *reinterpret_cast<int*>(scales_to + at) = v[0];
            *reinterpret_cast<int*>(scales_to + at + kScaleBlock) = v[1];
        } else {
            *reinterpret_cast<mx_i2*>(scales_to + at) = v;
        }
    };
    int sw[2][2], swn[2][2];
    auto load_s = [&](int quad, int (&w)[2][2]) __attribute__((always_inline)) {
        const int q = min(quad, G4 - 1);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            w[0][h] = load4(wsr, scale_pair + h * 128, q * 256);
            w[1][h] = load4(w2sr, scale_pair + spair1 + h * 128, q * 256);
        }
    };
    mx_f16 acc[SUB][2] = {};
    if (!GATED && a.bias) {                          // the sums start from the bias
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int c = col16 * 16 + 32 * j + 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3);
                const float b = c < a.N ? a.bias[c] : 0.0f;
#pragma unroll
                for (int i = 0; i < SUB; ++i) acc[i][j][r] = b;
            }
    }
    // Fragment q of a step: half q / SUB of piece q % SUB, and its scales. All first halves
    // come before the second ones: products that add to the same sums are 2 SUB apart
    // (two apart, the instructions alone run at 5.9 PFLOP/s, eight apart at 6.5).
    struct Fragment { mx_i4 c; int s; };
    const uint8_t* xl = lds + (lane >> 4 & 1) * kTile + (lane >> 5) * kBlock + (lane & 15) * 16;
    const uint8_t* sl = scales + (lane >> 5) * kScaleBlock + (lane & 31) * 4;
    auto read = [&](int stage, int at, int q) __attribute__((always_inline)) {
        const int i = q % SUB, h = q / SUB;
        return Fragment{*reinterpret_cast<const mx_i4*>(xl + stage * kStage + 2 * i * kTile + 2 * h * kBlock),
                        *reinterpret_cast<const int*>(sl + at + i * 128 + h * 2 * kScaleBlock)};
    };
    // Step g (S = g % 4): the products of group g. Even steps: rows of g + 2 and g + 3 enter
    // LDS (the barrier before step g + 1 shows them to it, which reads its successor's
    // first pieces), those of g + 4 and g + 5 leave memory; weights of g + 2 do in each.
    // In step 2 the next quad's scales enter LDS. Fragments are read kAhead ahead, across
    // the step's end. The scheduling barriers keep each fragment's products with its reads:
    // left alone, the compiler moves all reads of four steps, and their waits, before the
    // first product.
    constexpr int NF = 2 * SUB, kAhead = SUB < 2 ? 2 : 3;
    Fragment F[kAhead];
    int now = 0;                                     // the quad's scale buffer
    auto step = [&](auto phase, int g) __attribute__((always_inline)) {
        constexpr int S = decltype(phase)::value;
        Fragment f[NF + kAhead];
#pragma unroll
        for (int q = 0; q < kAhead; ++q) f[q] = F[q];
#pragma unroll
        for (int q = 0; q < NF; ++q) {
            // the step's loads are spread over its products: issued together by four waves
            // that just left a barrier, they hold up the products behind them
#pragma unroll
            for (int p = 0; p < 4; ++p)
                if (p * NF / 4 == q) W[(S + 2) & 3][p >> 1][p & 1] = load_w(g + 2, p);
            if (!(S & 1)) {
#pragma unroll
                for (int p = 0; p < 2 * XL; ++p)
                    if (NF - 1 - p * NF / (2 * XL) == q) {
                        store_x((S + 2) & 3, p / XL, p % XL, X[p / XL][p % XL]);
                        X[p / XL][p % XL] = load_x(g + 4, p / XL, p % XL);
                    }
            }
            if (S == 2 && q == 0) {
                store_xs(now ^ kScaleBytes, XS);
                XS = load_xs((g >> 2) + 2);
            }
            f[q + kAhead] = q + kAhead < NF ? read(S, now, q + kAhead)
                                            : read((S + 1) & 3, S == 3 ? now ^ kScaleBytes : now, q + kAhead - NF);
#pragma unroll
            for (int j = 0; j < 2; ++j)
                acc[q % SUB][j] = mfma32<S>(W[S][j][q / SUB], f[q].c, acc[q % SUB][j], sw[j][q / SUB], f[q].s);
            __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int q = 0; q < kAhead; ++q) F[q] = f[NF + q];
        __syncthreads();
        __builtin_amdgcn_sched_barrier(0);
    };
#pragma unroll
    for (int p = 0; p < 2 * XL; ++p) X[p / XL][p % XL] = load_x(0, p / XL, p % XL);
    XS = load_xs(0);
#pragma unroll
    for (int p = 0; p < 4; ++p) W[0][p >> 1][p & 1] = load_w(0, p);
    load_s(0, sw);
#pragma unroll
    for (int p = 0; p < 4; ++p) W[1][p >> 1][p & 1] = load_w(1, p);
#pragma unroll
    for (int p = 0; p < 2 * XL; ++p) {
        store_x(0, p / XL, p % XL, X[p / XL][p % XL]);
        X[p / XL][p % XL] = load_x(2, p / XL, p % XL);
    }
    store_xs(0, XS);
    XS = load_xs(1);
    __syncthreads();
#pragma unroll
    for (int q = 0; q < kAhead; ++q) F[q] = read(0, 0, q);
    int g = 0;
    for (; g + 4 <= G; g += 4) {
        load_s((g >> 2) + 1, swn);
        step(Phase<0>{}, g);
        step(Phase<1>{}, g + 1);
        step(Phase<2>{}, g + 2);
        step(Phase<3>{}, g + 3);
        now ^= kScaleBytes;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < 2; ++j) sw[j][h] = swn[j][h];
    }
    if (g < G) {
        step(Phase<0>{}, g);
        if (g + 1 < G) step(Phase<1>{}, g + 1);
        if (g + 2 < G) step(Phase<2>{}, g + 2);
    }

    // The results leave through LDS, piece by piece: a lane holds one row's columns
    // 8 (r / 4) + 4 (l / 32) + r % 4, four neighbours; read back, eight lanes (fp32:
    // sixteen) hold 128 (256) bytes of a row, and a store covers whole lines.
    constexpr int kWaveCols = GATED ? 32 : 64;
    constexpr int kPitch = kWaveCols * sizeof(T) + 16;           // rows 16 B apart in the banks
    constexpr int kPer = 16 / sizeof(T);                         // columns of a lane's 16 bytes
    constexpr int kLanes = kWaveCols / kPer;                     // lanes of a row
    constexpr int kRound = 64 / kLanes;                          // rows of a store
    static_assert(32 * kPitch <= kOutBytes);
    uint8_t* tile = lds + wave * kOutBytes;                      // every wave is past the last barrier
    const int n = col16 * 16 + (lane & (kLanes - 1)) * kPer;
    const int rows = min(n16 * 16, a.M - rt0 * 16);
    T* y = static_cast<T*>(a.y) + static_cast<int64_t>(rt0) * 16 * a.ldy;
    // 16-byte stores, those beyond the block's rows or N dropped by their offset
    const bool vec = a.ldy % kPer == 0 && a.ldy <= (1 << 21);
    const __amdgpu_buffer_rsrc_t yr = buffer(y, static_cast<int64_t>(rows) * a.ldy * sizeof(T));
    uint32_t at = n < a.N ? ((lane / kLanes) * a.ldy + n) * sizeof(T) : 0x80000000u;
#pragma unroll
    for (int i = 0; i < SUB; ++i) {
        bool live = true;
        if (GATED) {
            const int m = 32 * i + (lane & 31);
            live = m < rows && static_cast<unsigned>(a.row_token[rt0 * 16 + m]) < static_cast<unsigned>(a.T);
        }
        mx_wave_sync();                                          // the last piece's reads come first
#pragma unroll
        for (int j = 0; j < (GATED ? 1 : 2); ++j) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                float v[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int q = 4 * c + r;
                    v[r] = GATED ? (live ? mx_silu(acc[i][0][q]) * acc[i][1][q] : 0.0f) : acc[i][j][q];
                }
                uint8_t* to = tile + (lane & 31) * kPitch + (32 * j + 8 * c + 4 * (lane >> 5)) * sizeof(T);
                if constexpr (sizeof(T) == 4)
                    *reinterpret_cast<float4*>(to) = make_float4(v[0], v[1], v[2], v[3]);
                else
                    *reinterpret_cast<uint2*>(to) = make_uint2(mx_pack2<T>(v[0], v[1]), mx_pack2<T>(v[2], v[3]));
            }
        }
        mx_wave_sync();
        if (vec) {
#pragma unroll
            for (int s = 0; s < 32 / kRound; ++s) {
                const mx_u4 v = *reinterpret_cast<const mx_u4*>(tile + (s * kRound + lane / kLanes) * kPitch + (lane & (kLanes - 1)) * 16);
                __builtin_amdgcn_raw_buffer_store_b128(v, yr, at, 0, 0);
                at += kRound * a.ldy * sizeof(T);
            }
        } else {
            const T* from = reinterpret_cast<const T*>(tile);
            const int cols = min(kWaveCols, a.N - col16 * 16);
#pragma clang loop unroll(disable)
            for (int o = lane; o < 32 * kWaveCols; o += 64) {
                const int r = o / kWaveCols, c = o % kWaveCols;
                if (32 * i + r < rows && c < cols)
                    y[static_cast<int64_t>(32 * i + r) * a.ldy + col16 * 16 + c] = from[r * (kPitch / sizeof(T)) + c];
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
        if (m < a.M) mx_store4(a.y, a.y_dtype, m * a.ldy + n, a.N - n, a.ldy % 4 == 0, 0.0f, 0.0f, 0.0f, 0.0f);
    }
}

// Four waves, each 64 columns (GATED: 32), of one row block. Workgroups go to the eight
// dies in turn, so each die takes a run of neighbouring tiles: they share rows and
// weights in its L2.
template <typename T, bool GATED>
__global__ __launch_bounds__(256, 2) void k_mx_wide(MxGemmArgs a, int blocks, int block_tiles) {
    constexpr int kStages = 4 * kBlockTiles * (GATED ? 1280 : 1024) + (GATED ? 64 : 0) + 2 * kScaleBytes;
    static_assert(kStages >= 4 * kOutBytes);
    __shared__ __align__(16) uint8_t lds[kStages];
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
        case 1: wide_tile<T, 1, GATED>(a, lds, rt0, n16, e, col16); break;
        case 2: wide_tile<T, 2, GATED>(a, lds, rt0, n16, e, col16); break;
        case 3: wide_tile<T, 3, GATED>(a, lds, rt0, n16, e, col16); break;
        default: wide_tile<T, 4, GATED>(a, lds, rt0, n16, e, col16); break;
    }
}

// y[t][d0 + d] = sum over j of weights[t][j] * rows[row_of[t][j]][d], d < cols, rows before
// *end (the last expert's end). Four columns
// a thread; a token's rows are read eight at a time. Bound by that read: 201 MB of rows in
// 40 us, 134 MB in 24.
template <typename T>
__global__ __launch_bounds__(256) void k_combine(const float* rows, int64_t n_rows, const int32_t* end, const int32_t* row_of,
                                                 const float* weights, int64_t T_, int k, int pitch, int cols, int64_t d0,
                                                 int64_t D, T* y) {
    const int d = (blockIdx.y * 256 + threadIdx.x) * 4;
    if (d >= cols) return;
    const int live = *end < n_rows ? *end : static_cast<int>(n_rows);      // no product wrote the rows from here on
    for (int64_t t = blockIdx.x; t < T_; t += gridDim.x) {
        mx_f4 acc = {};
        for (int j0 = 0; j0 < k; j0 += 8) {
            mx_f4 r[8];
            float w[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const bool there = j0 + j < k;
                const int p = there ? row_of[t * k + j0 + j] : -1;
                w[j] = there ? weights[t * k + j0 + j] : 0.0f;
                r[j] = mx_f4{0, 0, 0, 0};
                if (p >= 0 && p < live) r[j] = *reinterpret_cast<const mx_f4*>(rows + static_cast<int64_t>(p) * pitch + d);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) acc += w[j] * r[j];
        }
        mx_store4(y, sizeof(T) == 4 ? MQ_F32 : (__is_same(T, __bf16) ? MQ_BF16 : MQ_F16), t * D + d0 + d, cols - d,
                  D % 4 == 0 && d0 % 4 == 0, acc[0], acc[1], acc[2], acc[3]);
    }
}

template <typename T>
hipError_t combine(const float* rows, int64_t n_rows, const int32_t* end, const int32_t* row_of, const float* weights,
                   int64_t T_, int k, int pitch, int cols, int64_t d0, int64_t D, void* y, hipStream_t st) {
    const unsigned grid = static_cast<unsigned>(T_ < (1 << 20) ? T_ : 1 << 20);
    k_combine<T><<<dim3(grid, static_cast<unsigned>((cols + 1023) / 1024)), 256, 0, st>>>(
        rows, n_rows, end, row_of, weights, T_, k, pitch, cols, d0, D, static_cast<T*>(y));
    return hipGetLastError();
}

template <typename T>
hipError_t wide(const MxGemmArgs& a, hipStream_t st) {
    const int rt = (a.M + 15) / 16;
    const bool gated = a.w2q != nullptr;
    const int64_t ncol = (a.N + (gated ? 127 : 255)) / (gated ? 128 : 256);
    int blocks = 0, block_tiles = 0;
    if (!a.tiles) {
        block_tiles = 2 * mx_wide_pieces(a.M, a.N, a.K);
        blocks = (rt + block_tiles - 1) / block_tiles;
    }
    const int64_t n = a.tiles ? mx_tiles_cap(a.M, a.E) : blocks;
    const int64_t want = (n * ncol + 7) / 8 * 8;
    if (want >= int64_t(1) << 24) return hipErrorInvalidConfiguration;       // a grid holds 2^32 threads
    const unsigned grid = static_cast<unsigned>(want);
    if (gated)
        k_mx_wide<T, true><<<grid, 256, 0, st>>>(a, blocks, block_tiles);
    else
        k_mx_wide<T, false><<<grid, 256, 0, st>>>(a, blocks, block_tiles);
    return hipGetLastError();
}

}  // namespace

// The least of the ways' costs, fits of measured times (us) in rounds of 256 workgroups:
// 16 rows and one column tile a workgroup, 32 rows and one, two or four, and tiles of many
// rows (the fourth way's workgroups are two to a CU by their LDS, so it goes by whole rounds
// of 512). Few workgroups of the last take a third of a us or more for a step of K: the
// latency of weights that no cache holds. Over the 110 sizes that the fits were made of (10 to
// 800 rows, K = 512 to 14336) the choice is within 13% of the fastest way, 0.6% on average. E.g. (in this order) 64 x 1024 x 4096: 3.9, 4.4,
// 6.0, 7.7, 11.0; 256 x 4096 x 14336: 66.7, 53.1, 41.6, 33.6, 47.0; 96 x 14336 x 4096: 27.2, 23.0,
// 20.9, 21.6, 16.4.
int mx_plan(int64_t M, int64_t N, int64_t K) {
    if (M <= 16) return kMxOneTile;
    const int64_t rows16 = (M + 15) / 16, rows32 = (M + 31) / 32, tiles = (N + 15) / 16;
    const double g = static_cast<double>((K + 127) / 128) / 32;
    const double v = static_cast<double>(rows16 * tiles) / 256, u = static_cast<double>(rows32 * tiles) / 256;
    const double cost[4] = {0.65 + 0.53 * g + fmax(v, 1.0) * (0.73 + 0.83 * g),
                            2.3 + 0.6 * g + fmax(u, 1.0) * (0.58 + 1.49 * g),
                            2.53 + 1.7 * g + fmax(u / 2, 1.0) * (0.77 + 2.12 * g),
                            3.91 + 2.5 * g + (u <= 8 ? fmax(u / 4, 0.75) : 2 * ceil(u / 8)) * (0.35 + 3.45 * g)};
    int best = 0;
    for (int i = 1; i < 4; ++i)
        if (cost[i] < cost[best]) best = i;
    double wide;
    wide_pieces(rows32, (N + 255) / 256, K, &wide);
    wide = fmax(wide, 2.0 + 0.37 * 32 * g);
    return cost[best] < wide && rows16 <= 65535 ? best + kMxOneTile : kMxWide;
}

int mx_wide_pieces(int64_t M, int64_t N, int64_t K) { return wide_pieces((M + 31) / 32, (N + 255) / 256, K, nullptr); }

hipError_t launch_mx_few(const MxGemmArgs& a, int plan, hipStream_t st) {
    if (a.x) {
        const int64_t rows = a.w2q ? a.T : a.M;
        switch (a.x_dtype) {
            case MQ_F32: return few_raw<float>(a, rows, st);
            case MQ_BF16: return few_raw<__bf16>(a, rows, st);
            default: return few_raw<_Float16>(a, rows, st);
        }
    }
    switch (plan) {
        case kMxOneTile: return few<MxReady, 1, 1, 8, false>(a, st);
        case 0: return few<MxReady, 1, 2, 8, false>(a, st);
        case 1: return few<MxReady, 2, 2, 8, false>(a, st);
        default: return few<MxReady, 4, 2, 8, false>(a, st);
    }
}

hipError_t launch_mx_down_few(const MxGemmArgs& a, const int32_t* row_of, const float* weights, int k, int64_t P,
                              hipStream_t st) {
    switch (a.x_dtype) {
        case MQ_F32: return down_few<float>(a, row_of, weights, k, P, st);
        case MQ_BF16: return down_few<__bf16>(a, row_of, weights, k, P, st);
        default: return down_few<_Float16>(a, row_of, weights, k, P, st);
    }
}

hipError_t launch_mx_wide(const MxGemmArgs& a, hipStream_t st) {
    switch (a.y_dtype) {
        case MQ_F32: return wide<float>(a, st);
        case MQ_BF16: return wide<__bf16>(a, st);
        default: return wide<_Float16>(a, st);
    }
}

hipError_t launch_combine(const float* rows, int64_t n_rows, const int32_t* end, const int32_t* row_of, const float* weights,
                          int64_t T, int k, int pitch, int cols, int64_t d0, int64_t D, void* y, int y_dtype, hipStream_t st) {
    switch (y_dtype) {
        case MQ_F32: return combine<float>(rows, n_rows, end, row_of, weights, T, k, pitch, cols, d0, D, y, st);
        case MQ_BF16: return combine<__bf16>(rows, n_rows, end, row_of, weights, T, k, pitch, cols, d0, D, y, st);
        default: return combine<_Float16>(rows, n_rows, end, row_of, weights, T, k, pitch, cols, d0, D, y, st);
    }
}

}  // namespace mq
