// C ABI of the microscaled 4-bit operators and the routing: argument checks, then
// kernel launches. Declarations and the meaning of every argument are in include/mq.h.
#include <stdint.h>

#include "../../include/mq.h"
#include "mx_internal.h"

namespace {

int status_of(hipError_t e) { return e == hipSuccess ? MQ_OK : MQ_ERR_HIP; }
bool bad_type(int d) { return d != MQ_F32 && d != MQ_BF16 && d != MQ_F16; }
int64_t type_size(int d) { return d == MQ_F32 ? 4 : 2; }
bool off(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; }

constexpr int64_t kMaxRows = int64_t(1) << 24;
constexpr int64_t kMaxCols = int64_t(1) << 20;
constexpr int64_t kMaxElements = int64_t(1) << 40;
constexpr int64_t kMaxBatch = 65535;
constexpr int64_t kMaxSlots = int64_t(1) << 27;
constexpr int kMaxTop = 32;

// sizes of a microscaled matrix (or batch of them)
int check_matrix(int64_t B, int64_t R, int64_t K) {
    if (B < 0 || R < 0 || K <= 0) return MQ_ERR_INVALID_ARG;
    if (B > kMaxBatch || R > kMaxRows || K > kMaxCols || B * R > kMaxElements / K) return MQ_ERR_UNSUPPORTED;
    return MQ_OK;
}

int check_codes(const void* codes, const void* scales) {
    return !codes || !scales || off(codes, 16) || off(scales, 4) ? MQ_ERR_INVALID_ARG : MQ_OK;
}

int check_product(int64_t M, int64_t N, int64_t K) {
    if (M < 0 || N <= 0 || K <= 0) return MQ_ERR_INVALID_ARG;
    if (M > kMaxRows || N > kMaxRows || K > kMaxCols || N > kMaxElements / K || (M && N > kMaxElements / M))
        return MQ_ERR_UNSUPPORTED;
    return MQ_OK;
}

// the up products find a token's quantized row by a 32-bit offset
int check_row_offsets(int64_t T, int64_t D) {
    return mq::mx_row_codes_size(T, D) > int64_t(0xffffffff) ? MQ_ERR_UNSUPPORTED : MQ_OK;
}

int check_slots(int64_t T, int64_t k, int64_t E) {
    if (T < 0 || k <= 0 || E <= 0) return MQ_ERR_INVALID_ARG;
    if (E > MQ_MAX_EXPERTS || T > kMaxSlots / k) return MQ_ERR_UNSUPPORTED;
    return MQ_OK;
}

// sizes of the experts' products of T tokens: N outputs of K inputs a row and expert
int check_experts(int64_t T, int64_t k, int64_t E, int64_t N, int64_t K) {
    const int rc = check_slots(T, k, E);
    if (rc) return rc;
    const int product = check_product(mq::plan_rows(T, k, E), N, K);
    return product ? product : check_matrix(E, N, K);
}

size_t round16(int64_t n) { return static_cast<size_t>((n + 15) / 16 * 16); }

// codes, then scales, of an R x K matrix in a workspace
size_t mx_bytes(int64_t R, int64_t K) { return round16(mq::mx_codes_size(R, K)) + round16(mq::mx_scales_size(R, K)); }

mq::MxGemmArgs product(const uint8_t* xq, const uint8_t* xs, const uint8_t* wq, const uint8_t* ws, int64_t M, int64_t N,
                       int64_t K, void* y, int y_dtype) {
    mq::MxGemmArgs a = {};
    a.xq = xq;
    a.xs = xs;
    a.wq = wq;
    a.ws = ws;
    a.M = static_cast<int>(M);
    a.N = static_cast<int>(N);
    a.K = static_cast<int>(K);
    a.y = y;
    a.y_dtype = y_dtype;
    a.ldy = static_cast<int>(N);
    a.w_tiles = static_cast<int>(mq::mx_row_tiles(N));
    return a;
}

mq::MxQuantArgs rows_of(const void* x, int dtype, int64_t R, int64_t stride, int64_t K, uint8_t* codes, uint8_t* scales) {
    mq::MxQuantArgs a = {};
    a.x = x;
    a.dtype = dtype;
    a.B = 1;
    a.R = R;
    a.stride_r = stride;
    a.K = static_cast<int>(K);
    a.codes = codes;
    a.scales = scales;
    return a;
}

mq::MxTilesArgs blocks_of(const int32_t* offsets, int64_t E, int64_t P, int32_t* tiles) {
    return {offsets, static_cast<int>(E), static_cast<int>(P / 16), tiles, static_cast<int>(mq::mx_tiles_cap(P, E))};
}

size_t row_bytes(int64_t R, int64_t K) {
    return round16(mq::mx_row_codes_size(R, K)) + round16(mq::mx_row_scales_size(R, K));
}

// Whether a product quantizes its rows on the way. It saves a launch (about 3 us) and
// costs each workgroup the whole matrix of rows. Measured, on the way / apart, in us:
// 16 rows, 4096 x 4096: 6.9 / 7.6, N = 14336: 13.2 / 13.8, N = 4096, K = 14336: 20 / 14.8;
// N = 28672, K = 8192: 8 rows 28.8 / 31.9, 16 rows 37 / 31.7. Where K leaves a wave a batch and
// part of one the rows cost it twice, which the rule does not see: N = 17408, K = 5120, on
// weights that no cache holds, 8 rows 20.7 / 20.7, 10 25.4 / 20.9, 16 28.7 / 21.0.
bool on_the_way(int64_t M, int64_t N, int64_t K) { return M <= 16 && M * K <= 1 << 17 && M * K <= (int64_t(1) << 31) / N; }

hipError_t launch_product(const mq::MxGemmArgs& a, hipStream_t st) {
    const int plan = mq::mx_plan(a.M, a.N, a.K);
    return plan == mq::kMxWide ? mq::launch_mx_wide(a, st) : mq::launch_mx_few(a, plan, st);
}

// Whether the up products split K, quantizing on the way, instead of taking tiles of many
// rows. Measured, split / tiles, in us: 64 experts of 4096 x 1024, 8 a token: 1 token 6.8 /
// 16.3, 8 30.7 / 32.6, 16 30.7 / 32.9, 24 38.1 / 35.5; 8 experts of 4096 x 4096, 2 a token:
// 1 token 6.7 / 15.5, 16 24.9 / 24.8, 24 29.7 / 26.7. (All up to 4096 columns.)
bool few_tokens(int64_t T, int64_t k) { return T <= 16 && k <= 1024; }
// Whether the down products go token by token. As above, by token / tiles: 1 token 6.0 /
// 13.5, 4 13.8 / 20.3, 8 25.1 / 25.1, 16 44.3 / 25.3; 5.3 / 15.3, 14.2 / 18.7, 21.2 / 18.6,
// 37.8 / 19.4; 128 experts of 2048 x 768, 8 a token: 5.8 / 12.5, 8.0 / 13.2, 13.5 / 15.9,
// 24.2 / 20.1. So 8 tokens lose 14% where experts are few and large, and win as much where
// they are many and small.
bool one_by_one(int64_t T, int64_t k) { return T <= 8 && k <= 32; }
// Columns of the down products that are made, and summed, at a time: even parts, in whole
// blocks of 256 columns, of at most kDownBytes of fp32 rows, which the last-level cache
// (256 MB) holds. Where that is less than two blocks (from 102401 rows on) the cache no
// longer helps, and narrow parts cost more launches: parts of at most 1024 columns then,
// which also keep the workspace below that of all at once. Measured (8 of 64 experts, 4096
// columns), in us, parts of 256 / 512 / 1024 / 1536 / 2048 / all at once: 4096 tokens (33728
// rows) 529 / 403 / 328 / 319 / 325 / 335, 10000 847 / 769 / 770 / 790 / 773 / 767, 16384
// (132032) 1260 / 1340 / 1276 / 1291 / 1250 / 1233, 32768 2795 / 2601 / 2510 / 2528 / 2450 /
// 2434, 65536 5275 / 5043 / 4885 / 4920 / 4812 / 4871.
constexpr int64_t kDownBytes = int64_t(200) << 20;
int64_t down_cols(int64_t P, int64_t D) {
    const int64_t fit = P ? kDownBytes / (P * 4) / 256 * 256 : D + 255;
    const int64_t most = fit >= 512 ? fit : 1024;
    const int64_t parts = (D + most - 1) / most;
    const int64_t cols = ((D + parts - 1) / parts + 255) / 256 * 256;
    return cols < D ? cols : (D + 3) / 4 * 4;
}
size_t tiles_bytes(int64_t P, int64_t E) { return round16(mq::mx_tiles_size(P, E) * 4); }

}  // namespace

extern "C" {

size_t mq_mx_codes_bytes(int64_t R, int64_t K) {
    return check_matrix(1, R, K) ? 0 : static_cast<size_t>(mq::mx_codes_size(R, K));
}

size_t mq_mx_scales_bytes(int64_t R, int64_t K) {
    return check_matrix(1, R, K) ? 0 : static_cast<size_t>(mq::mx_scales_size(R, K));
}

int mq_mx_quantize(const void* x, int x_dtype, int64_t B, int64_t stride_b, int64_t R, int64_t stride_r, int64_t K,
                   uint8_t* codes, uint8_t* scales, void* stream) {
    int rc = check_matrix(B, R, K);
    if (rc) return rc;
    if (bad_type(x_dtype) || stride_b < 0 || stride_r < 0) return MQ_ERR_INVALID_ARG;
    if (B == 0 || R == 0) return MQ_OK;
    if (!x || off(x, type_size(x_dtype))) return MQ_ERR_INVALID_ARG;
    if ((rc = check_codes(codes, scales))) return rc;
    mq::MxQuantArgs a = rows_of(x, x_dtype, R, stride_r, K, codes, scales);
    a.B = B;
    a.stride_b = stride_b;
    return status_of(mq::launch_mx_quant(a, static_cast<hipStream_t>(stream)));
}

int mq_mx_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t B, int64_t R, int64_t K, void* y, int y_dtype,
                     void* stream) {
    int rc = check_matrix(B, R, K);
    if (rc) return rc;
    if (bad_type(y_dtype)) return MQ_ERR_INVALID_ARG;
    if (B == 0 || R == 0) return MQ_OK;
    if ((rc = check_codes(codes, scales))) return rc;
    if (!y || off(y, 16)) return MQ_ERR_INVALID_ARG;
    return status_of(mq::launch_mx_dequant(codes, scales, B, R, K, y, y_dtype, static_cast<hipStream_t>(stream)));
}

int mq_mx_gemm(const uint8_t* xq, const uint8_t* xs, const uint8_t* wq, const uint8_t* ws, int64_t M, int64_t N,
               int64_t K, const float* bias, void* y, int y_dtype, void* stream) {
    int rc = check_product(M, N, K);
    if (rc) return rc;
    if (bad_type(y_dtype) || off(bias, 4)) return MQ_ERR_INVALID_ARG;
    if (M == 0) return MQ_OK;
    if ((rc = check_codes(xq, xs)) || (rc = check_codes(wq, ws))) return rc;
    if (!y || off(y, 16)) return MQ_ERR_INVALID_ARG;
    mq::MxGemmArgs a = product(xq, xs, wq, ws, M, N, K, y, y_dtype);
    a.bias = bias;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    return status_of(launch_product(a, st));
}

int mq_mx_gemm_way(int64_t M, int64_t N, int64_t K) {
    const int rc = check_product(M, N, K);
    if (rc) return rc;
    const int plan = mq::mx_plan(M, N, K);
    return plan == mq::kMxWide ? 3 + mq::mx_wide_pieces(M, N, K) : plan - mq::kMxOneTile;
}

size_t mq_mx_linear_workspace_bytes(int64_t M, int64_t N, int64_t K) {
    return check_product(M, N, K) || on_the_way(M, N, K) ? 0 : mx_bytes(M, K);
}

int mq_mx_linear(const void* x, int x_dtype, int64_t stride_m, const uint8_t* wq, const uint8_t* ws, int64_t M,
                 int64_t N, int64_t K, const float* bias, void* y, int y_dtype, void* workspace, size_t workspace_bytes,
                 void* stream) {
    int rc = check_product(M, N, K);
    if (rc) return rc;
    if (bad_type(x_dtype) || bad_type(y_dtype) || stride_m < 0 || off(bias, 4)) return MQ_ERR_INVALID_ARG;
    if (M == 0) return MQ_OK;
    if (!x || off(x, type_size(x_dtype)) || !y || off(y, 16)) return MQ_ERR_INVALID_ARG;
    if ((rc = check_codes(wq, ws))) return rc;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    mq::MxGemmArgs a = product(nullptr, nullptr, wq, ws, M, N, K, y, y_dtype);
    a.bias = bias;
    if (on_the_way(M, N, K)) {
        a.x = x;
        a.x_dtype = x_dtype;
        a.stride_x = stride_m;
        return status_of(mq::launch_mx_few(a, mq::kMxOneTile, st));
    }
    if (workspace_bytes < mx_bytes(M, K) || !workspace || off(workspace, 16)) return MQ_ERR_INVALID_ARG;
    uint8_t* xq = static_cast<uint8_t*>(workspace);
    uint8_t* xs = xq + round16(mq::mx_codes_size(M, K));
    if (mq::launch_mx_quant(rows_of(x, x_dtype, M, stride_m, K, xq, xs), st) != hipSuccess) return MQ_ERR_HIP;
    a.xq = xq;
    a.xs = xs;
    return status_of(launch_product(a, st));
}

int mq_route(const void* logits, int dtype, int64_t T, int64_t stride_t, int64_t E, const float* bias, int score,
             int64_t groups, int64_t top_groups, int group_score, int64_t k, int renormalize, float scale, int32_t* ids,
             float* weights, void* stream) {
    int rc = check_slots(T, k, E);
    if (rc) return rc;
    if (bad_type(dtype) || stride_t < 0 || off(bias, 4)) return MQ_ERR_INVALID_ARG;
    if (score != MQ_SCORE_SOFTMAX && score != MQ_SCORE_SIGMOID) return MQ_ERR_INVALID_ARG;
    if (group_score != MQ_GROUP_MAX && group_score != MQ_GROUP_TOP2) return MQ_ERR_INVALID_ARG;
    if (groups <= 0 || E % groups || top_groups <= 0 || top_groups > groups) return MQ_ERR_INVALID_ARG;
    if (k > top_groups * (E / groups)) return MQ_ERR_INVALID_ARG;
    if (k > kMaxTop || groups > 64) return MQ_ERR_UNSUPPORTED;
    if (T == 0) return MQ_OK;
    if (!logits || off(logits, type_size(dtype)) || !ids || off(ids, 4) || !weights || off(weights, 4))
        return MQ_ERR_INVALID_ARG;
    mq::RouteArgs a;
    a.logits = logits;
    a.dtype = dtype;
    a.T = T;
    a.stride_t = stride_t;
    a.E = static_cast<int>(E);
    a.bias = bias;
    a.score = score;
    a.groups = static_cast<int>(groups);
    a.top_groups = static_cast<int>(top_groups);
    a.group_score = group_score;
    a.k = static_cast<int>(k);
    a.renormalize = renormalize != 0;
    a.scale = scale;
    a.ids = ids;
    a.weights = weights;
    return status_of(mq::launch_route(a, static_cast<hipStream_t>(stream)));
}

int64_t mq_plan_rows(int64_t T, int64_t k, int64_t E) { return check_slots(T, k, E) ? -1 : mq::plan_rows(T, k, E); }

int mq_expert_plan(const int32_t* ids, int64_t T, int64_t k, int64_t E, int32_t* offsets, int32_t* row_token,
                   int32_t* row_of, void* stream) {
    int rc = check_slots(T, k, E);
    if (rc) return rc;
    if (!offsets || off(offsets, 4)) return MQ_ERR_INVALID_ARG;
    if (T > 0 && (!ids || off(ids, 4) || !row_of || off(row_of, 4) || !row_token || off(row_token, 4)))
        return MQ_ERR_INVALID_ARG;
    mq::PlanArgs a;
    a.ids = ids;
    a.T = T;
    a.k = static_cast<int>(k);
    a.E = static_cast<int>(E);
    a.offsets = offsets;
    a.row_token = row_token;
    a.row_of = row_of;
    a.rows = mq::plan_rows(T, k, E);
    return status_of(mq::launch_plan(a, static_cast<hipStream_t>(stream)));
}

size_t mq_mx_experts_up_workspace_bytes(int64_t T, int64_t k, int64_t E, int64_t D, int64_t I) {
    if (check_experts(T, k, E, I, D) || check_row_offsets(T, D) || few_tokens(T, k)) return 0;
    const int64_t P = mq::plan_rows(T, k, E);
    return row_bytes(T, D) + tiles_bytes(P, E);
}

int mq_mx_experts_up(const void* x, int x_dtype, int64_t stride_t, int64_t T, int64_t k, int64_t E, int64_t D, int64_t I,
                     const int32_t* offsets, const int32_t* row_token, const int32_t* row_of, const uint8_t* gate_q,
                     const uint8_t* gate_s, const uint8_t* up_q, const uint8_t* up_s, void* h, int h_dtype,
                     void* workspace, size_t workspace_bytes, void* stream) {
    int rc = check_experts(T, k, E, I, D);
    if (rc || (rc = check_row_offsets(T, D))) return rc;
    if (bad_type(x_dtype) || bad_type(h_dtype) || stride_t < 0) return MQ_ERR_INVALID_ARG;
    if (T == 0) return MQ_OK;
    if (!x || off(x, type_size(x_dtype)) || !h || off(h, 16)) return MQ_ERR_INVALID_ARG;
    if (!offsets || off(offsets, 4) || !row_token || off(row_token, 4) || !row_of || off(row_of, 4))
        return MQ_ERR_INVALID_ARG;
    if ((rc = check_codes(gate_q, gate_s)) || (rc = check_codes(up_q, up_s))) return rc;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    const int64_t P = mq::plan_rows(T, k, E);
    mq::MxGemmArgs a = product(nullptr, nullptr, gate_q, gate_s, P, I, D, h, h_dtype);
    a.w2q = up_q;
    a.w2s = up_s;
    a.offsets = offsets;
    a.row_token = row_token;
    a.E = static_cast<int>(E);
    a.T = static_cast<int>(T);
    if (few_tokens(T, k)) {
        a.x = x;
        a.x_dtype = x_dtype;
        a.stride_x = stride_t;
        return status_of(mq::launch_mx_few(a, mq::kMxOneTile, st));
    }
    if (workspace_bytes < mq_mx_experts_up_workspace_bytes(T, k, E, D, I) || !workspace || off(workspace, 16))
        return MQ_ERR_INVALID_ARG;
    uint8_t* xq = static_cast<uint8_t*>(workspace);
    uint8_t* xs = xq + round16(mq::mx_row_codes_size(T, D));
    a.xq = xq;
    a.xs = xs;
    a.tiles = reinterpret_cast<int32_t*>(xs + round16(mq::mx_row_scales_size(T, D)));
    mq::MxQuantArgs q = rows_of(x, x_dtype, T, stride_t, D, xq, xs);
    q.by_row = true;
    q.plan = blocks_of(offsets, E, P, a.tiles);
    if (mq::launch_mx_quant(q, st) != hipSuccess) return MQ_ERR_HIP;
    return status_of(mq::launch_mx_wide(a, st));
}

size_t mq_mx_experts_down_workspace_bytes(int64_t T, int64_t k, int64_t E, int64_t D, int64_t I) {
    if (check_experts(T, k, E, D, I) || one_by_one(T, k)) return 0;
    const int64_t P = mq::plan_rows(T, k, E);
    const size_t rows = round16(P * down_cols(P, D) * 4);
    return rows + mx_bytes(P, I) + tiles_bytes(P, E);
}

int mq_mx_experts_down(const void* h, int h_dtype, int64_t T, int64_t k, int64_t E, int64_t D, int64_t I,
                       const int32_t* offsets, const int32_t* row_of, const float* weights, const uint8_t* wq,
                       const uint8_t* ws, void* y, int y_dtype, void* workspace, size_t workspace_bytes, void* stream) {
    int rc = check_experts(T, k, E, D, I);
    if (rc) return rc;
    if (bad_type(h_dtype) || bad_type(y_dtype)) return MQ_ERR_INVALID_ARG;
    if (T == 0) return MQ_OK;
    if (!h || off(h, type_size(h_dtype)) || !y || off(y, 16)) return MQ_ERR_INVALID_ARG;
    if (!offsets || off(offsets, 4) || !row_of || off(row_of, 4) || !weights || off(weights, 4)) return MQ_ERR_INVALID_ARG;
    if ((rc = check_codes(wq, ws))) return rc;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    const int64_t P = mq::plan_rows(T, k, E);
    if (one_by_one(T, k)) {
        mq::MxGemmArgs a = product(nullptr, nullptr, wq, ws, P, D, I, y, y_dtype);
        a.offsets = offsets;
        a.E = static_cast<int>(E);
        a.T = static_cast<int>(T);
        a.x = h;
        a.x_dtype = h_dtype;
        a.stride_x = I;
        return status_of(mq::launch_mx_down_few(a, row_of, weights, static_cast<int>(k), P, st));
    }
    if (workspace_bytes < mq_mx_experts_down_workspace_bytes(T, k, E, D, I) || !workspace || off(workspace, 16))
        return MQ_ERR_INVALID_ARG;
    float* rows = static_cast<float*>(workspace);
    const int64_t step = down_cols(P, D);
    mq::MxGemmArgs a = product(nullptr, nullptr, wq, ws, P, D, I, rows, MQ_F32);
    a.offsets = offsets;
    a.E = static_cast<int>(E);
    a.T = static_cast<int>(T);
    a.ldy = static_cast<int>(step);
    uint8_t* hq = static_cast<uint8_t*>(workspace) + round16(P * step * 4);
    uint8_t* hs = hq + round16(mq::mx_codes_size(P, I));
    a.xq = hq;
    a.xs = hs;
    a.tiles = reinterpret_cast<int32_t*>(hs + round16(mq::mx_scales_size(P, I)));
    mq::MxQuantArgs q = rows_of(h, h_dtype, P, I, I, hq, hs);
    q.plan = blocks_of(offsets, E, P, a.tiles);
    if (mq::launch_mx_quant(q, st) != hipSuccess) return MQ_ERR_HIP;
    for (int64_t d = 0; d < D; d += step) {
        a.N = static_cast<int>(D - d < step ? D - d : step);
        a.w_tile0 = static_cast<int>(d / 16);
        if (mq::launch_mx_wide(a, st) != hipSuccess) return MQ_ERR_HIP;
        if (mq::launch_combine(rows, P, offsets + E, row_of, weights, T, static_cast<int>(k), static_cast<int>(step), a.N, d, D,
                               y, y_dtype, st) != hipSuccess)
            return MQ_ERR_HIP;
    }
    return MQ_OK;
}

}  // extern "C"
