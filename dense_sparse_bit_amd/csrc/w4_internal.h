// Internal interface of the group-scaled 4-bit operators and of the calls between tokens
// and their experts' rows (api_w4.hip checks arguments; w4_quant.hip, w4_gemm.hip and
// rows.hip launch).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mx_internal.h"

namespace mq {

// Layout of a matrix [R][K] (mq.h): 16-row x 128-input code tiles in the lane order of the
// 16x16x32 matrix instructions, scales by row in quads of tiles.
inline int64_t w4_row_tiles(int64_t R) { return (R + 15) / 16; }
inline int64_t w4_tiles(int64_t K) { return (K + 127) / 128; }
inline int64_t w4_quads(int64_t K) { return (K + 511) / 512; }
inline int64_t w4_codes_size(int64_t R, int64_t K) { return w4_row_tiles(R) * w4_tiles(K) * 1024; }
inline int64_t w4_scales_size(int64_t R, int64_t K, int group) { return w4_row_tiles(R) * w4_quads(K) * 16 * (512 / group) * 2; }

struct W4QuantArgs {
    const void* x;                   // values, or codes one to a byte (pack)
    int dtype;
    const uint16_t *s, *z;           // pack: scales and zero points [B][R][ceil(K/group)]
    int64_t B, stride_b, R, stride_r;
    int K, group, scale_dtype;
    uint8_t* codes;
    uint16_t *scales, *zeros;
};

// Y = X W^T. Dense: M x N outputs. With offsets: M rows of a plan, each with its expert's
// matrix; by_token: row p is x's row row_token[p].
struct W4GemmArgs {
    const void* x;
    int x_dtype;
    int64_t stride_x;
    const uint8_t* codes;
    const uint16_t *scales, *zeros;
    int scale_dtype, group;
    int M, N, K;
    const float* bias;
    void* y;
    int y_dtype;
    const int32_t *offsets, *row_token;
    int by_token, E, T;
};


// Row blocks of a plan for launch_w4_wide, as MxTilesArgs' but of at most 2 rt 16-row tiles.
inline int64_t w4_blocks_cap(int64_t P, int64_t E, int rt) { return P / 16 / (2 * rt) + E + 2; }

// What launch_w4_wide takes of x: the sums of its groups, and a copy where x itself does not
// do (fp32, or rows that are not made of aligned 16-byte units). And of the scales: which 16-row tiles
// of W have rows whose scales are too far apart for sums in units of them.
struct W4RowsArgs {
    const void* x;
    int dtype;
    int64_t R, stride;
    int K, group;
    void *sums, *copy;
    MxTilesArgs plan;                // row blocks that the launch makes too,
    int rt;                          // of 32 rt rows (1 to 4)
    const uint16_t* scales;          // bf16
    int64_t tiles;                   // of all matrices, 0 for fp16 scales
    int* wild;                       // [tiles], not 0 for those
};
inline int w4_planes(int x_dtype) { return x_dtype == 0 ? 3 : 1; }
inline int64_t w4_sums_size(int64_t R, int64_t K, int planes, int group) { return w4_tiles(K) * planes * (128 / group) * R * 16; }
inline int64_t w4_copy_size(int64_t R, int64_t K, int planes) { return R * w4_tiles(K) * planes * 256; }

struct W4WideArgs {
    const uint16_t* x;               // 16-bit rows in whole runs of 128 inputs, ldx apart
    int x_dtype;
    int64_t ldx, rows_x;             // rows of x
    int planes;                      // runs of 128 inputs for each 128 of K
    const uint4* sums;
    const int* wild;
    const uint8_t* codes;
    const uint16_t *scales, *zeros;
    int scale_dtype, group;
    int M, N, K;
    const float* bias;
    void* y;
    int y_dtype;
    const int32_t *row_token, *tiles;
    int by_token, E, T;
    int parts;                       // of K, at most its stages (w4_tiles(K) * planes)
    float* partial;                  // [parts][M][N] where there are more than one
};

struct RowsArgs {
    const void* x;                   // [T][D], the tokens' side
    int x_dtype;
    int64_t stride_t;
    const void* rows;                // [P][D], the experts' side
    int rows_dtype;
    int64_t T, P;
    int k, D;
    const int32_t *row_token, *row_of;
    const float* weights;
    const void* other;               // of the output's size; combine: rows stride_o apart
    int64_t stride_o;
    float* dots;
};

hipError_t launch_w4_quant(const W4QuantArgs& a, hipStream_t st);
hipError_t launch_w4_pack(const W4QuantArgs& a, hipStream_t st);
hipError_t launch_w4_dequant(const W4QuantArgs& a, void* y, int y_dtype, hipStream_t st);
// The kernels of few rows: up to 4 rows and 16 columns a workgroup, a quad of code tiles at a
// time, or 16 or 32 rows and these columns, tile by tile; each splits K over its waves. fp32
// and a plan's rows: at most 16 rows, at most 32 columns for fp32, 64 else.
enum W4Few { kW4One, kW4Rows16, kW4Rows16x32, kW4Rows16x64, kW4Rows32x32, kW4Rows32x64 };

// Waves of a workgroup of few rows, which share its code tiles: eight where there are so many.
// Where workgroups fill the chip, four find them short of nothing and have half the sums to add:
// 100 rows, 2048 x 2048, by 16 rows and 16 columns (896 workgroups) 8.4 us against 10.3; 64 tokens'
// rows of 64 experts, 4096 x 1024 (6000) 49 against 96. Where they do not, eight are faster: 20 rows,
// 512 x 2048 (64) 4.5 us against 5.0; 100 rows, 2048 x 2048 by 16 and 32 (448) 7.9 against 8.2.
inline int64_t w4_few_waves(int64_t workgroups, int64_t K, int tiles) {
    const int64_t G = w4_tiles(K), most = workgroups > (tiles == 1 ? 256 : 512) && G < 32 ? 4 : 8;
    return G < most ? G : most;
}
hipError_t launch_w4_few(const W4GemmArgs& a, W4Few kind, hipStream_t st);
hipError_t launch_w4_rows(const W4RowsArgs& a, hipStream_t st);
// tiles of 32 rt rows and 128 ct columns: rt <= 2 with ct = 1, 2 <= rt <= 4 with ct = 2 (a plan's rows: 1 or
// 2 with 1, 3 or 4 with 2). Groups of 32 take no 64 x 256, which the costs never choose for them, and no 128
// x 256, whose registers do not hold them (96 x 256 keeps one of them in scratch memory while its loop runs).
inline bool w4_has_tile(int rt, int ct, int group) { return group > 32 || ct == 1 || rt == 3; }
hipError_t launch_w4_wide(const W4WideArgs& a, int rt, int ct, hipStream_t st);
hipError_t launch_rows_gather(const RowsArgs& a, hipStream_t st);
hipError_t launch_rows_combine(const RowsArgs& a, hipStream_t st);

}  // namespace mq
