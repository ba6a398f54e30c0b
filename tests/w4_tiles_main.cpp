// Sweeps the addresses of csrc/w4_tiles.h: every load of every lane lies within the wave's
// buffer, and every column that is stored was computed from its own tile. Prints the first
// mistake of each kind and ends with 1, or ends with 0.
#include <stdio.h>

#include <algorithm>

#include "../dense_sparse_bit_amd/csrc/w4_tiles.h"

static int bad = 0;
static void check(bool ok, const char* what, int N, int K, int GS, int blocks, int lane) {
    if (!ok && bad++ < 10) printf("%s: N %d K %d groups %d blocks %d lane %d\n", what, N, K, GS, blocks, lane);
}

// One wave whose columns begin at n0: `blocks` blocks of `per` tiles.
static void wave(int N, int K, int GS, int n0, int blocks, int per) {
    const int G = (K + 127) / 128, Q = (G + 3) / 4, tiles = (N + 15) / 16;
    const int tile0 = per == 1 ? n0 / 16 : std::min(n0 / 16, tiles - 1), have = std::min(tiles - tile0, per * blocks);
    check(have >= 1, "no tile", N, K, GS, blocks, 0);
    const long codes = static_cast<long>(have) * G * 1024, scales = static_cast<long>(have) * mq::w4_scale_bytes(Q, GS);
    for (int j = 0; j < blocks; ++j) {
        const int t = mq::w4_block_tile(j, per, have);
        for (int h : {0, G / 2, G - 1})
            for (int lane = 0; lane < 64; ++lane) {
                const int code = per == 1 ? mq::w4_lane_code(lane) : mq::w4_pair_code(lane, have, G);
                const int scale = per == 1 ? mq::w4_lane_scale(lane, GS) : mq::w4_pair_scale(lane, have, Q, GS);
                for (int part = 0; part < per; ++part) {
                    const long at = code + mq::w4_code_at(t, h, G) + 512 * part;
                    check(at >= 0 && at + 16 <= codes, "codes past the end", N, K, GS, blocks, lane);
                }
                const long at = scale + mq::w4_scale_at(t, h, Q, GS);
                check(at >= 0 && at + 2 * GS <= scales, "scales past the end", N, K, GS, blocks, lane);
            }
        // the block's results go to columns 16 t on; those that are stored have their own tile's
        for (int lane = 0; lane < 64; ++lane) {
            const int c = 16 * t + (lane & (16 * per - 1)), took = per == 1 ? t : t + mq::w4_pair_second(lane, have);
            if (n0 / 16 == tile0 && n0 + c < N) check(took == c / 16, "another column's tile", N, K, GS, blocks, lane);
        }
    }
    // and every column has a block
    for (int c = 0; c < 16 * std::min(have, per * blocks); ++c) {
        bool there = false;
        for (int j = 0; j < blocks; ++j) {
            const int t = mq::w4_block_tile(j, per, have);
            there = there || (c >= 16 * t && c < 16 * (t + per));
        }
        check(there, "a column without a block", N, K, GS, blocks, c);
    }
}

int main() {
    for (int N = 1; N <= 600; ++N)
        for (int K : {1, 128, 129, 513, 4096, 14336})
            for (int GS : {1, 2, 4}) {
                for (int NT : {1, 2, 4})                                    // workgroups of few rows
                    for (int n0 = 0; n0 < N; n0 += 16 * NT) wave(N, K, GS, n0, NT, 1);
                for (int CT : {1, 2})                                       // the four waves of a tile, past N too
                    for (int n0 = 0; n0 < (N + 128 * CT - 1) / (128 * CT) * 128 * CT; n0 += 32 * CT) wave(N, K, GS, n0, CT, 2);
            }
    if (bad) printf("%d mistakes\n", bad);
    return bad ? 1 : 0;
}
