// Where the lanes of paged_attn.hip read in a key's or a value's row of D elements (es
// bytes each).  Plain arithmetic, so that a host program can go through every case.
#pragma once

namespace tcm {

// The instance that takes heads of D elements: D rounded up to 64, 128 or 256.
constexpr int head_instance(int D) { return D <= 64 ? 64 : D <= 128 ? 128 : 256; }

// A key: 16-byte pieces, one a lane.  Is piece c inside the row?
constexpr bool key_piece_in(int c, int D, int es) { return 16 * c < D * es; }

// A value: dp / 16 elements a lane, in loads of at most 16 bytes.
constexpr int value_bytes(int dp, int es) { return dp / 16 * es; }
constexpr int value_load(int dp, int es) { return value_bytes(dp, es) < 16 ? value_bytes(dp, es) : 16; }

// The offset of load i of lane c (0 .. 15).  A load that would begin past the row's end reads
// the row's beginning, for elements that nobody stores; each load is judged by itself, since a
// lane's elements may straddle the end (D = 136: lane 8 has 128 .. 143).  A load that begins
// inside ends inside: rows are whole 16-byte pieces.
constexpr int value_at(int c, int i, int D, int dp, int es) {
    const int at = c * value_bytes(dp, es) + i * value_load(dp, es);
    return at < D * es ? at : 0;
}

}  // namespace tcm
