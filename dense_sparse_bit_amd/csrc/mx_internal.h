// Internal interface of the microscaled 4-bit operators and the routing
// (api_mx.hip checks arguments; mx_quant.hip, mx_gemm.hip and route.hip launch).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mq {

// Layout of a microscaled matrix [R][K] (mq.h): 16-row x 128-input tiles in the lane
// order of the 16x16x128 matrix instruction, one scale byte per lane and tile.
constexpr int kMxGroup = 128;      // inputs per code tile
constexpr int kMxTileBytes = 1024;
inline int64_t mx_row_tiles(int64_t R) { return (R + 15) / 16; }
inline int64_t mx_groups(int64_t K) { return (K + kMxGroup - 1) / kMxGroup; }
inline int64_t mx_quads(int64_t K) { return (mx_groups(K) + 3) / 4; }
inline int64_t mx_codes_size(int64_t R, int64_t K) { return mx_row_tiles(R) * mx_groups(K) * kMxTileBytes; }
inline int64_t mx_scales_size(int64_t R, int64_t K) { return mx_row_tiles(R) * mx_quads(K) * 256; }

// rows of an expert plan: every expert's rows start at a multiple of 16
inline int64_t plan_rows(int64_t T, int64_t k, int64_t E) {
    const int64_t n = T * k;
    return (n + 15 * (n < E ? n : E)) / 16 * 16;
}

// Row by row, for rows that are picked one by one (experts' tokens): a row's codes are
// whole runs of 128 bytes (256 inputs) in the order of the inputs; its scales 16 bytes per 512 inputs, the byte
// of block b at (b / 16) * 16 + (b % 4) * 4 + b / 4 % 4.
inline int64_t mx_row_codes_size(int64_t R, int64_t K) { return R * ((mx_groups(K) + 1) / 2) * 128; }
inline int64_t mx_row_scales_size(int64_t R, int64_t K) { return R * mx_quads(K) * 16; }

// Row blocks of an expert plan, for launch_mx_wide: each expert's rows in blocks of at most
// kBlockTiles 16-row tiles, of even sizes; then the rows after the last expert's, with
// expert -1. tiles: [0] their number, then (expert, first 16-row tile, 16-row tiles, 0)
// each.
constexpr int kBlockTiles = 8;
inline int64_t mx_tiles_cap(int64_t P, int64_t E) { return P / 16 / kBlockTiles + E + 2; }
inline int64_t mx_tiles_size(int64_t P, int64_t E) { return 4 + 4 * mx_tiles_cap(P, E); }
struct MxTilesArgs {
    const int32_t* offsets;          // of a plan of P16 16-row tiles; null: no tiles are wanted
    int E, P16;
    int32_t* tiles;
    int cap;
};

// x[b][r][c] of a strided matrix, as it is read by the quantizer. by_row (B = 1): the
// row by row layout.
struct MxQuantArgs {
    const void* x;
    int dtype;
    int64_t B, stride_b, R, stride_r;
    int K;
    bool by_row;
    uint8_t* codes;
    uint8_t* scales;
    MxTilesArgs plan;                // row blocks that the launch makes too
};

// Y = X W^T over microscaled operands. Dense: M x N outputs. With offsets (expert
// products): rows are a plan's rows, the expert e with offsets[e] <= row < offsets[e + 1]
// picks the weights, and rows of no token are zero. With w2q: silu(X W^T) * (X W2^T)
// (gate and up).
struct MxGemmArgs {
    const uint8_t *xq, *xs;          // quantized operand (w2q: row by row, picked by row_token), or
    const void* x;                   // rows to be quantized on the way (null: xq, xs)
    int x_dtype;
    int64_t stride_x;
    const uint8_t *wq, *ws, *w2q, *w2s;
    int M, N, K;
    const float* bias;
    void* y;                         // rows ldy apart
    int y_dtype, ldy;
    int w_tile0, w_tiles;            // N is a run of the weights' rows: from 16-row tile w_tile0 of w_tiles
    const int32_t* offsets;
    const int32_t* row_token;        // x's row of each of the plan's rows (x given), and which rows are live
    int E, T;
    int32_t* tiles;                  // row blocks of the plan (MxTilesArgs)
};

struct RouteArgs {
    const void* logits;
    int dtype;
    int64_t T, stride_t;
    int E;
    const float* bias;
    int score, groups, top_groups, group_score, k, renormalize;
    float scale;
    int32_t* ids;
    float* weights;
};

struct PlanArgs {
    const int32_t* ids;
    int64_t T;
    int k, E;
    int32_t *offsets, *row_token, *row_of;
    int64_t rows;
};

hipError_t launch_mx_quant(const MxQuantArgs& a, hipStream_t st);
hipError_t launch_mx_dequant(const uint8_t* codes, const uint8_t* scales, int64_t B, int64_t R, int64_t K, void* y,
                             int y_dtype, hipStream_t st);
// The kernel of a product of M rows: split over K with 16 rows a workgroup, or 32 rows and
// one, two or four column tiles (0, 1, 2), or tiles of many rows.
constexpr int kMxOneTile = -1, kMxWide = 3;
int mx_plan(int64_t M, int64_t N, int64_t K);
// 32-row pieces of a row block of such tiles
int mx_wide_pieces(int64_t M, int64_t N, int64_t K);
// a.x given: rows are quantized on the way (plan kMxOneTile, or rows of a plan's tiles)
hipError_t launch_mx_few(const MxGemmArgs& a, int plan, hipStream_t st);
// y[t] = sum over j of weights[t][j] * (Q(x[row_of[t][j]]) . w[expert of the row]), in one
// launch, for few tokens (P: rows of x; k <= 32)
hipError_t launch_mx_down_few(const MxGemmArgs& a, const int32_t* row_of, const float* weights, int k, int64_t P,
                              hipStream_t st);
hipError_t launch_mx_wide(const MxGemmArgs& a, hipStream_t st);
hipError_t launch_route(const RouteArgs& a, hipStream_t st);
hipError_t launch_plan(const PlanArgs& a, hipStream_t st);
// y[t][d0 + d] = sum over j of weights[t][j] * rows[row_of[t][j]][d], d < cols (fp32 rows,
// a multiple of 4 apart; those from *end on, on the device, are no rows)
hipError_t launch_combine(const float* rows, int64_t n_rows, const int32_t* end, const int32_t* row_of, const float* weights,
                          int64_t T, int k, int pitch, int cols, int64_t d0, int64_t D, void* y, int y_dtype, hipStream_t st);

}  // namespace mq
