// Where a workgroup's loads of 4-bit weights go: byte offsets into the column tiles that its
// waves take. Plain functions of whole numbers, which the kernels and a test on the host call.
//
// A wave's buffers begin at its first column tile and hold the `have` tiles from there to the
// matrix's end, or all that it takes where that is nearer. A load's address is a lane's offset
// and a scalar one; only the lane's part is certain to be checked against the buffer's size,
// so the sum of both stays within it for every lane.
#pragma once

namespace mq {

// The first of `per` (1 or 2) neighbouring column tiles that block j of a wave takes: where fewer
// are left the last ones once more, whose columns then have the same results twice.
constexpr int w4_block_tile(int j, int per, int have) { return j * per + per <= have ? j * per : (have > per ? have - per : 0); }

// Codes and scales of `per` tiles: the scalar part for tile t and 128 inputs h of G (Q quads of
// them), and the lane's. GS: groups in 128 inputs.
constexpr int w4_code_at(int t, int h, int G) { return (t * G + h) * 1024; }
constexpr int w4_scale_bytes(int Q, int GS) { return Q * 16 * 4 * GS * 2; }
constexpr int w4_scale_at(int t, int h, int Q, int GS) { return t * w4_scale_bytes(Q, GS) + ((h >> 2) * 64 + (h & 3)) * GS * 2; }

// One tile: a lane's 16 bytes; the scales of its column.
constexpr int w4_lane_code(int lane) { return lane * 16; }
constexpr int w4_lane_scale(int lane, int GS) { return (lane & 15) * 8 * GS; }
// Two tiles, the second for the lanes whose bit 4 is set (all take a lone one): a lane's 16
// bytes of each half of a tile.
constexpr int w4_pair_second(int lane, int have) { return have > 1 ? lane >> 4 & 1 : 0; }
constexpr int w4_pair_code(int lane, int have, int G) { return w4_pair_second(lane, have) * G * 1024 + ((lane >> 5) * 16 + (lane & 15)) * 16; }
constexpr int w4_pair_scale(int lane, int have, int Q, int GS) { return w4_pair_second(lane, have) * w4_scale_bytes(Q, GS) + (lane & 15) * 8 * GS; }

}  // namespace mq
