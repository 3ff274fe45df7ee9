// Replays the tiled products' loads on the host: every lane of every load of every step of every tile of one operand.
#include "dense_index.h"

using namespace moe;

namespace {

// What is wrong with the loads of an operand of `rows` rows and `K` of K, `ld` elements from line to line in memory, in
// tiles of W rows and parts of kper of K, by `waves` wavefronts of L loads each: 0, or 1 for a piece that does not lie within
// one line's elements, 2 for one cut short, 3 for a wrong one, 4 for one that is missing, 5 for one past its part's end.
template <int W, int L, bool TR>
int check(int waves, int rows, int K, int ld, int kper) {
    typedef Lines<W, TR> At;
    for (int kbeg = 0; kbeg < K; kbeg += kper) {
        const int kend = kbeg + kper < K ? kbeg + kper : K;
        for (int row0 = 0; row0 < rows; row0 += W)
            for (int k0 = kbeg; k0 < kend + kStepK; k0 += kStepK)
                for (int wave = 0; wave < waves; ++wave)
                    for (int i = 0; i < L; ++i)
                        for (int lane = 0; lane < 64; ++lane) {
                            const int b = wave * L + i, left = TR ? rows - row0 : rows - row0 - b * At::kPer;
                            const int64_t reach = At::reach(ld, left, kend - kbeg), bytes = reach > 0 ? 2 * reach : 0;
                            const uint32_t off = At::in_step(b, lane, kend - k0) ? At::offset(b, lane, ld, left) : kNowhere;
                            const int64_t first = TR ? (int64_t)(k0 + b * At::kPer) * ld + row0
                                                     : (int64_t)(row0 + b * At::kPer) * ld + k0;
                            const int line = At::line(b, lane), chunk = 8 * At::chunk(b, lane);
                            const int row = row0 + (TR ? chunk : line), k = k0 + (TR ? line : chunk);
                            const bool there = row < rows && k < kend;
                            if (off >= bytes) {
                                if (there) return 4;
                                continue;
                            }
                            const int64_t e = first + off / 2;
                            if (e / ld >= (TR ? K : rows) || e % ld + 8 > (TR ? rows : K)) return 1;
                            if (bytes - off < 16) return 2;
                            if (e != (TR ? (int64_t)k * ld + row : (int64_t)row * ld + k)) return 3;
                            if (!there) return 5;
                        }
    }
    return 0;
}

// How often the workgroups of one launch take each tile of a product, the second of a pair's two where dw > 0.
void walk(int total, int dw, int grid, int ahead, int* taken) {
    for (int b = 0; b < grid; ++b) {
        const int xcd = b % kXcds, me = b / kXcds, all = grid / kXcds;
        const int left = tiles_of(dw, xcd) % all;
        for (int turn = 0;; ++turn) {
            const int slot = dw ? slot_behind(me, all, left, left ? ahead : 0, turn) : me + turn * all;
            if (!has_tile(total, xcd, slot)) break;
            ++taken[tile_of(total, xcd, slot)];
        }
    }
}

}  // namespace

extern "C" void count_tiles(int total, int dw, int grid, int ahead, int* taken) { walk(total, dw, grid, ahead, taken); }

extern "C" int check_loads(int width, int across, int rows, int K, int ld, int kper) {
    if (width == 256) return across ? check<256, 4, true>(8, rows, K, ld, kper) : check<256, 4, false>(8, rows, K, ld, kper);
    if (width == 128) return across ? check<128, 4, true>(4, rows, K, ld, kper) : check<128, 4, false>(4, rows, K, ld, kper);
    return across ? check<64, 2, true>(4, rows, K, ld, kper) : check<64, 2, false>(4, rows, K, ld, kper);
}
