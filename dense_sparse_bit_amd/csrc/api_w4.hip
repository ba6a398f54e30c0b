// C ABI of the group-scaled 4-bit operators and of the calls between tokens and their
// experts' rows: argument checks, then kernel launches. Declarations and the meaning of
// every argument are in include/mq.h.
#include <math.h>
#include <stdint.h>

#include "../../include/mq.h"
#include "mx_internal.h"
#include "w4_internal.h"

namespace {

int status_of(hipError_t e) { return e == hipSuccess ? MQ_OK : MQ_ERR_HIP; }
bool bad_type(int d) { return d != MQ_F32 && d != MQ_BF16 && d != MQ_F16; }
bool bad_scales(int d) { return d != MQ_BF16 && d != MQ_F16; }
bool bad_group(int g) { return g != 32 && g != 64 && g != 128; }
int64_t type_size(int d) { return d == MQ_F32 ? 4 : 2; }
bool off(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; }

constexpr int64_t kMaxRows = int64_t(1) << 24;
constexpr int64_t kMaxCols = int64_t(1) << 20;
constexpr int64_t kMaxElements = int64_t(1) << 40;
constexpr int64_t kMaxBatch = 65535;
constexpr int64_t kMaxOffset = 0xffffffff;             // of x's rows in the tiles: of a block's, or of all tokens'
constexpr int64_t kMaxSlots = int64_t(1) << 27;

int check_matrix(int64_t B, int64_t R, int64_t K, int group) {
    if (B < 0 || R < 0 || K <= 0 || bad_group(group)) return MQ_ERR_INVALID_ARG;
    if (B > kMaxBatch || R > kMaxRows || K > kMaxCols || B * R > kMaxElements / K) return MQ_ERR_UNSUPPORTED;
    return MQ_OK;
}

// zeros may be NULL
int check_weights(const void* codes, const void* scales, const void* zeros, int scale_dtype) {
    return !codes || !scales || off(codes, 16) || off(scales, 16) || off(zeros, 16) || bad_scales(scale_dtype)
               ? MQ_ERR_INVALID_ARG
               : MQ_OK;
}

int check_product(int64_t M, int64_t N, int64_t K, int group) {
    if (M < 0 || N <= 0 || K <= 0 || bad_group(group)) return MQ_ERR_INVALID_ARG;
    if (M > kMaxRows || N > kMaxRows || K > kMaxCols || N > kMaxElements / K || (M && N > kMaxElements / M))
        return MQ_ERR_UNSUPPORTED;
    return MQ_OK;
}

int check_slots(int64_t T, int64_t k, int64_t E) {
    if (T < 0 || k <= 0 || E <= 0) return MQ_ERR_INVALID_ARG;
    if (E > MQ_MAX_EXPERTS || T > kMaxSlots / k) return MQ_ERR_UNSUPPORTED;
    return MQ_OK;
}

int check_experts(int64_t T, int64_t k, int64_t E, int64_t N, int64_t K, int group) {
    const int rc = check_slots(T, k, E);
    if (rc) return rc;
    const int product = check_product(mq::plan_rows(T, k, E), N, K, group);
    return product ? product : check_matrix(E, N, K, group);
}

int check_rows(int64_t T, int64_t k, int64_t E, int64_t D) {
    const int rc = check_slots(T, k, E);
    if (rc) return rc;
    if (D <= 0) return MQ_ERR_INVALID_ARG;
    return D > kMaxCols ? MQ_ERR_UNSUPPORTED : MQ_OK;
}

mq::W4QuantArgs matrix(int64_t B, int64_t R, int64_t K, int group, const uint8_t* codes, const void* scales, const void* zeros) {
    mq::W4QuantArgs a = {};
    a.B = B;
    a.R = R;
    a.K = static_cast<int>(K);
    a.group = group;
    a.codes = const_cast<uint8_t*>(codes);
    a.scales = static_cast<uint16_t*>(const_cast<void*>(scales));
    a.zeros = static_cast<uint16_t*>(const_cast<void*>(zeros));
    return a;
}

mq::W4GemmArgs product(const void* x, int x_dtype, int64_t stride_x, const uint8_t* codes, const void* scales, const void* zeros,
                       int scale_dtype, int group, int64_t M, int64_t N, int64_t K, void* y, int y_dtype) {
    mq::W4GemmArgs a = {};
    a.x = x;
    a.x_dtype = x_dtype;
    a.stride_x = stride_x;
    a.codes = codes;
    a.scales = static_cast<const uint16_t*>(scales);
    a.zeros = static_cast<const uint16_t*>(zeros);
    a.scale_dtype = scale_dtype;
    a.group = group;
    a.M = static_cast<int>(M);
    a.N = static_cast<int>(N);
    a.K = static_cast<int>(K);
    a.y = y;
    a.y_dtype = y_dtype;
    return a;
}

mq::RowsArgs rows_of(int64_t T, int64_t k, int64_t E, int64_t D, const void* x, int x_dtype, int64_t stride_t, const void* rows,
                     int rows_dtype, const int32_t* row_of, const float* weights, const void* other, float* dots) {
    mq::RowsArgs a = {};
    a.x = x;
    a.x_dtype = x_dtype;
    a.stride_t = stride_t;
    a.rows = rows;
    a.rows_dtype = rows_dtype;
    a.T = T;
    a.P = mq::plan_rows(T, k, E);
    a.k = static_cast<int>(k);
    a.D = static_cast<int>(D);
    a.row_of = row_of;
    a.weights = weights;
    a.other = other;
    a.dots = dots;
    return a;
}

size_t round16(int64_t n) { return static_cast<size_t>((n + 15) / 16 * 16); }

// The way of a product: a kernel of few rows, or (rt > 0) tiles of 32 rt rows and 128 ct columns
// with K in `parts`.
struct Way {
    mq::W4Few few;
    int rt, ct, parts;
};

// Parts of K are whole stages of the tiles, one at least.
Way tiles_way(int rt, int ct, int64_t parts, int64_t stages) {
    return {mq::kW4One, rt, ct, static_cast<int>(parts < 1 ? 1 : (parts < stages ? parts : stages))};
}

// The costs below are fits, in us, of times measured on weights that no cache holds: 23 sizes
// from 512 x 512 to 17408 x 5120, 5 to 2048 rows, every way. Over 298 of those with up to 256
// rows the choice is within 23% of the fastest way, 0.9% on average (fp32 rows, 88 sizes: 26% and
// 1.5%).
//
// A kernel of few rows: in rounds of workgroups (`per` rounds for each 256 of eight waves), a start
// and each wave's code tiles, whose time grows with the groups in them.
struct FewCost {
    int rows, cols;
    double start, round, tile, per, groups;
};
double few_cost(const FewCost& c, int64_t M, int64_t N, int64_t K, int group) {
    const int64_t wgs = ((N + c.cols - 1) / c.cols) * ((M + c.rows - 1) / c.rows);
    const double waves = static_cast<double>(mq::w4_few_waves(wgs, K, c.rows * c.cols / 256));
    const double tiles = static_cast<double>(mq::w4_tiles(K)) / waves * (1 + c.groups * (128 / group - 1));
    return c.start + (c.round + c.tile * tiles) * fmax(1.0, c.per * static_cast<double>(wgs) / 256 * waves / 8);
}

// Tiles: the sums of the rows' groups, then the stages, each as long as its chain of
// instructions where a CU has one workgroup (alone) and as its products where it has more;
// the parts' sums written, read and added.
struct TileCost {
    int rt, ct;
    double start, alone, busy, join, moved, groups;
};
constexpr TileCost kTiles[] = {{1, 1, 8.13, 0.59, 0.40, 2.48, 0.57, 0.17},
                               {2, 1, 8.44, 0.68, 0.59, 2.65, 0.42, 0.22},
                               {2, 2, 9.63, 1.04, 1.09, 3.06, 0.35, 0.28},
                               {3, 2, 9.93, 1.41, 1.20, 2.57, 0.35, 0.27},
                               {4, 2, 10.8, 1.72, 1.52, 2.16, 0.35, 0.22}};
double tile_cost(const TileCost& c, int64_t M, int64_t N, int64_t K, int planes, int group, int parts) {
    const double tiles = static_cast<double>((M + 32 * c.rt - 1) / (32 * c.rt)) * static_cast<double>((N + 128 * c.ct - 1) / (128 * c.ct));
    const double n = tiles * parts / 256, stages = static_cast<double>(mq::w4_tiles(K) * planes) / parts;
    const double stage = fmax(c.alone, c.busy * (c.rt >= 3 && n > 1 ? ceil(n) : n));
    const double rows = static_cast<double>(M) * static_cast<double>(K) * planes * 0.67e-6;
    const double join = parts > 1 ? c.join + c.moved * parts * static_cast<double>(M) * static_cast<double>(N) * 4e-6 : 0;
    return c.start + rows + stages * stage * (1 + c.groups * (128 / group - 1)) + join;
}

Way dense_way(int64_t M, int64_t N, int64_t K, int x_dtype, int group) {
    const int planes = mq::w4_planes(x_dtype);
    const int64_t stages = mq::w4_tiles(K) * planes;
    // Four rows, 4096 x 4096: by four 5.8 us, by 16 7.7; 14336 x 4096: 17.8, 12.2.
    if (M == 1 || (M <= 4 && N <= 8192)) return {mq::kW4One, 0, 0, 1};
    Way best = {mq::kW4Rows16, 0, 0, 1};
    double least = 1e300;
    auto take = [&](Way w, double cost) {
        if (cost < least) {
            least = cost;
            best = w;
        }
    };
    if (M <= 256) {
        const double more = planes == 1 ? 1 : 2;           // fp32 rows: three times the products
        take({mq::kW4Rows16, 0, 0, 1}, few_cost({16, 16, 2.88, 0.63, more * 0.72, 0.85, 0.20}, M, N, K, group));
        take({mq::kW4Rows16x32, 0, 0, 1}, few_cost({16, 32, 3.68, 0.24, more * 0.85, 1.12, 0.22}, M, N, K, group));
        if (M <= 16) return best;
        if (planes == 1) {
            take({mq::kW4Rows32x32, 0, 0, 1}, few_cost({32, 32, 2.18, 2.50, 1.34, 1.21, 0.23}, M, N, K, group));
            take({mq::kW4Rows32x64, 0, 0, 1}, few_cost({32, 64, 3.06, 2.77, 1.71, 1.42, 0.33}, M, N, K, group));
        }
    }
    for (const TileCost& c : kTiles) {
        if (!mq::w4_has_tile(c.rt, c.ct, group)) continue;
        const int64_t tiles = ((M + 32 * c.rt - 1) / (32 * c.rt)) * ((N + 128 * c.ct - 1) / (128 * c.ct));
        for (int parts = 1; parts <= 8; parts *= 2)
            if (parts == 1 || (stages >= 4 * parts && tiles * parts <= 1100))
                take(tiles_way(c.rt, c.ct, parts, stages), tile_cost(c, M, N, K, planes, group, parts));
    }
    return best;
}

// 64 experts, 8 a token, 1024 x 4096 / 4096 x 1024, in us: 1 token one row at a time 5.9 / 5.7, by
// 16 rows 6.8 / 7.0; 64 tokens by 16 rows 42 / 49, by tiles 44 / 41; 128 tokens 57 / 82 and 50 / 49.
// By 16 rows, 32 columns a workgroup / 64: 1024 x 4096 41 / 49, 4096 x 1024 55 / 45. Where the
// smallest tiles leave CUs idle 16 rows serve longer: 64 tokens of 2 of 8, 4096 x 4096 34 against 38.
// Tiles of 32 or 64 rows and 128 columns where they make few workgroups, the largest else: 512 tokens
// of 8 of 64, 1024 x 4096 (512) 83 against 102; 256 of 2 of 8, 4096 x 4096 (256) 50 against 77; 4096
// of 8 of 64 (4096) 342 against 317. K in parts for 256 tokens: 65 / 61 / 59 in 1, 2, 4
// (1024 x 4096) and 51 / 77 / 124.
Way experts_way(int64_t T, int64_t k, int64_t E, int64_t N, int64_t K, bool by_token, int x_dtype, int group) {
    if (T == 1) return {mq::kW4One, 0, 0, 1};
    // the tiles find tokens' rows by offsets of 32 bits (in a copy, where x's own are too far apart)
    const bool held = !by_token || mq::w4_copy_size(T, K, mq::w4_planes(x_dtype)) <= kMaxOffset;
    const int64_t each = (T * k + E - 1) / E, cols = (N + 127) / 128;
    if (each <= (E * cols <= 256 ? 24 : 12) || !held)
        return {K > 2048 || x_dtype == MQ_F32 ? mq::kW4Rows16x32 : mq::kW4Rows16x64, 0, 0, 1};
    if (E * ((each + 63) / 64) * cols <= 1024) return tiles_way(each <= 32 ? 1 : 2, 1, 1, 1);
    return tiles_way(group == 32 ? 3 : 4, 2, 1, 1);
}

// Workspace of the tiles: the rows' sums, a copy of the rows (whether x needs one or not: the
// size is asked for without x), the W tiles' marks, row blocks, sums of parts of K
struct Parts {
    size_t copy, wild, tiles, partial, bytes;
    Parts(int64_t R, int64_t K, int x_dtype, int group, int64_t blocks, int parts, int64_t M, int64_t N, int64_t E) {
        const int planes = mq::w4_planes(x_dtype);
        copy = mq::w4_sums_size(R, K, planes, group);
        wild = copy + round16(mq::w4_copy_size(R, K, planes));
        tiles = wild + round16(E * mq::w4_row_tiles(N) * 4);
        partial = tiles + round16(blocks ? (4 + 4 * blocks) * 4 : 0);
        bytes = partial + (parts > 1 ? round16(parts * M * N * 4) : 0);
    }
};

// The rows' part, then the tiles. R: rows of x.
int wide(const mq::W4GemmArgs& a, Way way, int64_t R, const int32_t* offsets, void* workspace, size_t workspace_bytes, hipStream_t st) {
    const int64_t blocks = offsets ? mq::w4_blocks_cap(a.M, a.E, way.rt) : 0;
    const Parts parts(R, a.K, a.x_dtype, a.group, blocks, way.parts, a.M, a.N, offsets ? a.E : 1);
    if (workspace_bytes < parts.bytes || !workspace || off(workspace, 16)) return MQ_ERR_INVALID_ARG;
    uint8_t* const work = static_cast<uint8_t*>(workspace);
    const bool as_it_is = a.x_dtype != MQ_F32 && !off(a.x, 16) && a.stride_x % 8 == 0 && a.K % 128 == 0 &&
                          a.stride_x <= kMaxOffset / 2 / (a.by_token ? R + 1 : 129);
    mq::W4RowsArgs r = {};
    r.x = a.x;
    r.dtype = a.x_dtype;
    r.R = R;
    r.stride = a.stride_x;
    r.K = a.K;
    r.group = a.group;
    r.sums = work;
    r.copy = as_it_is ? nullptr : work + parts.copy;
    int32_t* const tiles = reinterpret_cast<int32_t*>(work + parts.tiles);
    r.rt = way.rt;
    r.scales = a.scales;
    r.tiles = a.scale_dtype == MQ_BF16 ? (offsets ? a.E : 1) * mq::w4_row_tiles(a.N) : 0;
    r.wild = reinterpret_cast<int*>(work + parts.wild);
    if (offsets) r.plan = {offsets, a.E, a.M / 16, tiles, static_cast<int>(blocks)};
    if (mq::launch_w4_rows(r, st) != hipSuccess) return MQ_ERR_HIP;
    mq::W4WideArgs w = {};
    const int64_t pitch = mq::w4_tiles(a.K) * mq::w4_planes(a.x_dtype) * 128;
    w.x = static_cast<const uint16_t*>(as_it_is ? a.x : r.copy);
    w.x_dtype = a.x_dtype;
    w.ldx = as_it_is ? a.stride_x : pitch;
    w.rows_x = R;
    w.planes = mq::w4_planes(a.x_dtype);
    w.sums = static_cast<const uint4*>(r.sums);
    w.wild = r.wild;
    w.codes = a.codes;
    w.scales = a.scales;
    w.zeros = a.zeros;
    w.scale_dtype = a.scale_dtype;
    w.group = a.group;
    w.M = a.M;
    w.N = a.N;
    w.K = a.K;
    w.bias = a.bias;
    w.y = a.y;
    w.y_dtype = a.y_dtype;
    w.row_token = a.row_token;
    w.tiles = offsets ? tiles : nullptr;
    w.by_token = a.by_token;
    w.E = a.E;
    w.T = a.T;
    w.parts = way.parts;
    w.partial = way.parts > 1 ? reinterpret_cast<float*>(work + parts.partial) : nullptr;
    return status_of(mq::launch_w4_wide(w, way.rt, way.ct, st));
}

}  // namespace

extern "C" {

size_t mq_w4_codes_bytes(int64_t R, int64_t K) {
    return check_matrix(1, R, K, 128) ? 0 : static_cast<size_t>(mq::w4_codes_size(R, K));
}

size_t mq_w4_scales_bytes(int64_t R, int64_t K, int group) {
    return check_matrix(1, R, K, group) ? 0 : static_cast<size_t>(mq::w4_scales_size(R, K, group));
}

int mq_w4_quantize(const void* x, int x_dtype, int64_t B, int64_t stride_b, int64_t R, int64_t stride_r, int64_t K, int group,
                   int scale_dtype, uint8_t* codes, void* scales, void* zeros, void* stream) {
    int rc = check_matrix(B, R, K, group);
    if (rc) return rc;
    if (bad_type(x_dtype) || bad_scales(scale_dtype) || stride_b < 0 || stride_r < 0) return MQ_ERR_INVALID_ARG;
    if (B == 0 || R == 0) return MQ_OK;
    if (!x || off(x, type_size(x_dtype))) return MQ_ERR_INVALID_ARG;
    if ((rc = check_weights(codes, scales, zeros, scale_dtype))) return rc;
    mq::W4QuantArgs a = matrix(B, R, K, group, codes, scales, zeros);
    a.x = x;
    a.dtype = x_dtype;
    a.stride_b = stride_b;
    a.stride_r = stride_r;
    a.scale_dtype = scale_dtype;
    return status_of(mq::launch_w4_quant(a, static_cast<hipStream_t>(stream)));
}

int mq_w4_pack(const uint8_t* c, int64_t B, int64_t stride_b, int64_t R, int64_t stride_r, int64_t K, int group, const void* s,
               const void* z, uint8_t* codes, void* scales, void* zeros, void* stream) {
    int rc = check_matrix(B, R, K, group);
    if (rc) return rc;
    if (stride_b < 0 || stride_r < 0) return MQ_ERR_INVALID_ARG;
    if (B == 0 || R == 0) return MQ_OK;
    if (!c || !s || off(s, 2) || off(z, 2) || (z == nullptr) != (zeros == nullptr)) return MQ_ERR_INVALID_ARG;
    if ((rc = check_weights(codes, scales, zeros, MQ_F16))) return rc;
    mq::W4QuantArgs a = matrix(B, R, K, group, codes, scales, zeros);
    a.x = c;
    a.stride_b = stride_b;
    a.stride_r = stride_r;
    a.s = static_cast<const uint16_t*>(s);
    a.z = static_cast<const uint16_t*>(z);
    return status_of(mq::launch_w4_pack(a, static_cast<hipStream_t>(stream)));
}

int mq_w4_dequantize(const uint8_t* codes, const void* scales, const void* zeros, int scale_dtype, int64_t B, int64_t R,
                     int64_t K, int group, void* y, int y_dtype, void* stream) {
    int rc = check_matrix(B, R, K, group);
    if (rc) return rc;
    if (bad_type(y_dtype) || bad_scales(scale_dtype)) return MQ_ERR_INVALID_ARG;
    if (B == 0 || R == 0) return MQ_OK;
    if ((rc = check_weights(codes, scales, zeros, scale_dtype))) return rc;
    if (!y || off(y, 16)) return MQ_ERR_INVALID_ARG;
    mq::W4QuantArgs a = matrix(B, R, K, group, codes, scales, zeros);
    a.scale_dtype = scale_dtype;
    return status_of(mq::launch_w4_dequant(a, y, y_dtype, static_cast<hipStream_t>(stream)));
}

size_t mq_w4_linear_workspace_bytes(int64_t M, int64_t N, int64_t K, int x_dtype, int group) {
    if (check_product(M, N, K, group) || bad_type(x_dtype)) return 0;
    const Way way = dense_way(M, N, K, x_dtype, group);
    return way.rt ? Parts(M, K, x_dtype, group, 0, way.parts, M, N, 1).bytes : 0;
}

int mq_w4_linear_way(int64_t M, int64_t N, int64_t K, int x_dtype, int group) {
    const int rc = check_product(M, N, K, group);
    if (rc) return rc;
    if (bad_type(x_dtype)) return MQ_ERR_INVALID_ARG;
    const Way way = dense_way(M, N, K, x_dtype, group);
    return way.rt ? 8 * way.parts + (way.ct == 1 ? way.rt - 1 : way.rt) : way.few;
}

int mq_w4_linear(const void* x, int x_dtype, int64_t stride_m, const uint8_t* codes, const void* scales, const void* zeros,
                 int scale_dtype, int group, int64_t M, int64_t N, int64_t K, const float* bias, void* y, int y_dtype,
                 void* workspace, size_t workspace_bytes, void* stream) {
    int rc = check_product(M, N, K, group);
    if (rc) return rc;
    if (bad_type(x_dtype) || bad_type(y_dtype) || bad_scales(scale_dtype) || stride_m < 0 || off(bias, 4))
        return MQ_ERR_INVALID_ARG;
    if (M == 0) return MQ_OK;
    if (!x || off(x, type_size(x_dtype)) || !y || off(y, 16)) return MQ_ERR_INVALID_ARG;
    if ((rc = check_weights(codes, scales, zeros, scale_dtype))) return rc;
    mq::W4GemmArgs a = product(x, x_dtype, stride_m, codes, scales, zeros, scale_dtype, group, M, N, K, y, y_dtype);
    a.bias = bias;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    const Way way = dense_way(M, N, K, x_dtype, group);
    return way.rt ? wide(a, way, M, nullptr, workspace, workspace_bytes, st) : status_of(mq::launch_w4_few(a, way.few, st));
}

size_t mq_w4_experts_workspace_bytes(int64_t T, int64_t k, int64_t E, int64_t N, int64_t K, int by_token, int x_dtype, int group) {
    if (check_experts(T, k, E, N, K, group) || bad_type(x_dtype)) return 0;
    const Way way = experts_way(T, k, E, N, K, by_token != 0, x_dtype, group);
    const int64_t P = mq::plan_rows(T, k, E);
    return way.rt ? Parts(by_token ? T : P, K, x_dtype, group, mq::w4_blocks_cap(P, E, way.rt), way.parts, P, N, E).bytes : 0;
}

int mq_w4_experts(const void* x, int x_dtype, int64_t stride_r, int by_token, int64_t T, int64_t k, int64_t E, int64_t N,
                  int64_t K, const int32_t* offsets, const int32_t* row_token, const uint8_t* codes, const void* scales,
                  const void* zeros, int scale_dtype, int group, void* y, int y_dtype, void* workspace, size_t workspace_bytes, void* stream) {
    int rc = check_experts(T, k, E, N, K, group);
    if (rc) return rc;
    if (bad_type(x_dtype) || bad_type(y_dtype) || bad_scales(scale_dtype) || stride_r < 0) return MQ_ERR_INVALID_ARG;
    if (T == 0) return MQ_OK;
    if (!x || off(x, type_size(x_dtype)) || !y || off(y, 16)) return MQ_ERR_INVALID_ARG;
    if (!offsets || off(offsets, 4) || !row_token || off(row_token, 4)) return MQ_ERR_INVALID_ARG;
    if ((rc = check_weights(codes, scales, zeros, scale_dtype))) return rc;
    mq::W4GemmArgs a = product(x, x_dtype, stride_r, codes, scales, zeros, scale_dtype, group, mq::plan_rows(T, k, E), N, K, y,
                               y_dtype);
    a.offsets = offsets;
    a.row_token = row_token;
    a.by_token = by_token != 0;
    a.E = static_cast<int>(E);
    a.T = static_cast<int>(T);
    const hipStream_t st = static_cast<hipStream_t>(stream);
    const Way way = experts_way(T, k, E, N, K, by_token != 0, x_dtype, group);
    return way.rt ? wide(a, way, by_token ? T : a.M, offsets, workspace, workspace_bytes, st) : status_of(mq::launch_w4_few(a, way.few, st));
}

int mq_experts_gather(const void* x, int x_dtype, int64_t stride_t, int64_t T, int64_t k, int64_t E, int64_t D,
                      const int32_t* row_token, const int32_t* row_of, const float* weights, void* rows, int rows_dtype,
                      const void* other, float* dots, void* stream) {
    const int rc = check_rows(T, k, E, D);
    if (rc) return rc;
    if (bad_type(x_dtype) || bad_type(rows_dtype) || stride_t < 0 || off(weights, 4)) return MQ_ERR_INVALID_ARG;
    if ((other == nullptr) != (dots == nullptr) || off(other, type_size(rows_dtype)) || off(dots, 4)) return MQ_ERR_INVALID_ARG;
    if (T == 0) return MQ_OK;
    if (!x || off(x, type_size(x_dtype)) || !rows || off(rows, 16)) return MQ_ERR_INVALID_ARG;
    if (!row_token || off(row_token, 4) || !row_of || off(row_of, 4)) return MQ_ERR_INVALID_ARG;
    mq::RowsArgs a = rows_of(T, k, E, D, x, x_dtype, stride_t, rows, rows_dtype, row_of, weights, other, dots);
    a.row_token = row_token;
    return status_of(mq::launch_rows_gather(a, static_cast<hipStream_t>(stream)));
}

int mq_experts_combine(const void* rows, int rows_dtype, int64_t T, int64_t k, int64_t E, int64_t D, const int32_t* row_of,
                       const float* weights, void* x, int x_dtype, const void* other,
                       int64_t stride_o, float* dots, void* stream) {
    const int rc = check_rows(T, k, E, D);
    if (rc) return rc;
    if (bad_type(x_dtype) || bad_type(rows_dtype) || off(weights, 4) || stride_o < 0) return MQ_ERR_INVALID_ARG;
    if ((other == nullptr) != (dots == nullptr) || off(other, type_size(x_dtype)) || off(dots, 4)) return MQ_ERR_INVALID_ARG;
    if (T == 0) return MQ_OK;
    if (!rows || off(rows, type_size(rows_dtype)) || !x || off(x, 16) || !row_of || off(row_of, 4)) return MQ_ERR_INVALID_ARG;
    mq::RowsArgs a = rows_of(T, k, E, D, x, x_dtype, D, rows, rows_dtype, row_of, weights, other, dots);
    a.stride_o = stride_o;
    return status_of(mq::launch_rows_combine(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
