// Where the tiled products' loads go: plain arithmetic, for the kernels and for a check of it on the host.
#pragma once

#include <cstdint>

namespace moe {

constexpr int kStepK = 64;                                   // of K a step
constexpr uint32_t kNowhere = 0x80000000u;                   // an offset past every reach: the load gives zeros

// LDS serves a 16 B read sixteen lanes at a time: lanes 0-3, 12-15, 20-23 and 24-27, then 4-11, 16-19 and 28-31, and the
// other half alike; the rows of two share the 256 B of its banks.
constexpr int swizzle(int r) { return r >> 1 & 7; }

// The slot of a 32 B piece of K step k, where K lies across the rows of an operand of W.
template <int W>
constexpr int turn(int k) {
    return ((k & 3) | (k >> 3 & 3) << 2) & (W / 16 - 1);
}

// One step of an operand's W rows, in 1 KB loads of 64 lanes and 16 bytes each.  TR: K lies across the rows of memory, so
// that a line is a K step and its chunks are rows of the operand; else a line is a row and its chunks are K.
template <int W, bool TR>
struct Lines {
    static constexpr int kChunks = TR ? W / 8 : kStepK / 8;  // 16 B chunks of a line
    static constexpr int kPer = 64 / kChunks;                // lines of a load

    // the line and the chunk of it that lane `lane` brings with load `block`
    static constexpr int line(int block, int lane) { return block * kPer + lane / kChunks; }
    static constexpr int chunk(int block, int lane) {
        if constexpr (TR) return (lane % kChunks) ^ (turn<W>(line(block, lane)) << 1);
        else return (lane % kChunks) ^ swizzle(line(block, lane));
    }
    // Bytes from the load's first element to the lane's, ld elements from line to line.  TR: none where the chunk lies past
    // the last `left` of the operand's rows (whole chunks of them), so that nothing behind a line's end is read.
    static constexpr uint32_t offset(int block, int lane, int ld, int left) {
        const uint32_t at = (uint32_t)(lane / kChunks) * (uint32_t)(ld * 2) + (uint32_t)chunk(block, lane) * 16;
        return TR && 8 * chunk(block, lane) >= left ? kNowhere : at;
    }
    // Elements that a load may reach from its first: TR, `left` rows of the operand from the tile's first, K bounded by
    // in_step; else `left` rows from the load's first (none or fewer: no row) and `kleft` of K from the part's first.
    static constexpr int reach(int ld, int left, int kleft) {
        const int rows = left < kPer ? left : kPer, cols = TR ? (left < W ? left : W) : kleft < kStepK ? kleft : kStepK;
        return ((TR ? kPer : rows) - 1) * ld + cols;
    }
    // whether the lane's chunk begins within the `kleft` of K that are left at this step
    static constexpr bool in_step(int block, int lane, int kleft) {
        if constexpr (TR) return lane / kChunks < kleft - block * kPer;
        else return 8 * chunk(block, lane) < kleft;
    }
};

// ---------------------------------------------------------------- who takes which tile
// Workgroup b runs on XCD b % 8; each XCD takes a run of a product's `total` tiles, its workgroups slots of that run.
constexpr int kXcds = 8, kCus = 256;                         // of an MI355X

constexpr int run_of(int total) { return (total + kXcds - 1) / kXcds; }

// The tile in slot `slot` of XCD `xcd`'s run, and whether there is one; if not, none is in the slots behind it.
constexpr int tile_of(int total, int xcd, int slot) { return xcd * run_of(total) + slot; }
constexpr bool has_tile(int total, int xcd, int slot) { return slot < run_of(total) && tile_of(total, xcd, slot) < total; }

// How many tiles XCD `xcd`'s run has.
constexpr int tiles_of(int total, int xcd) {
    const int run = run_of(total), rest = total - xcd * run, most = rest < run ? rest : run;
    return most > 0 ? most : 0;
}

// The slot of turn `turn` in a second product's run, for an XCD's workgroup `me` of `all`: those that the first product's last
// round left out (from `left` on) begin with `ahead` tiles each (none where its rounds are whole), the rest of the run goes
// round as ever.
constexpr int slot_behind(int me, int all, int left, int ahead, int turn) {
    const int free = all - left;
    if (me < left) return ahead * free + turn * all + me;
    return turn < ahead ? turn * free + me - left : ahead * free + (turn - ahead) * all + me;
}

}  // namespace moe
