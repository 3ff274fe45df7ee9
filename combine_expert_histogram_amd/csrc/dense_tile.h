// Tiled matrix products of 16-bit rows: C[m, n] = sum_k A(m, k) B(n, k) in fp32, each operand with K along its rows or
// across them.
//
// A persistent workgroup walks over tiles of BM x BN results.  Its wavefronts hold RW x CW of them each in registers
// (v_mfma_f32_16x16x32, operands swapped, so that a lane holds four consecutive columns of a row) and take 64 of K a step
// from a two-step ring in LDS, which loads go to directly.  All of it is one stream over the tiles: a step's last 32 of K
// are multiplied after the barrier that frees its place, while the step after the next is loaded there and the next
// step's first fragments are read; a tile's last steps load the next tile's first ones, which arrive while its sums are
// written.  Two sets of fragments alternate, and the order of products, LDS reads and loads is laid out by hand.
//
// What bounds it (16384 x 4096 x 7168 bf16, 256 x 256 tiles, counters): the matrix cores are busy 0.67 of the time at 1.95
// GHz, the clock that the card's power leaves them; with all operands in the caches they are busy 0.79 of it at 1.81 GHz.
// LDS is busy a quarter of the time.  It reads 1.4 GB, as often as tiles of this size have to from the XCDs' L2.  With 2048 of
// K they are busy 0.54: a tile's sums go out in a burst from all CUs at once, about 7 us of 53 at a large copy's rate, 13
// with a residual (held four and eight pieces ahead, and the next tile's first step not waiting for the stores: the same
// times).  Tried: 32 x 32 MFMAs (as fast), four wavefronts of 128 x 128 (0.55 busy: one
// wavefront a SIMD cannot multiply while its loads queue), four steps of 32 of K (as fast, slower along rows: half lines),
// wavefront priorities (none), 128 x 128 tiles (0.8 of the rate).
#pragma once

#include "dense.h"

namespace moe {
namespace {

constexpr int kBK = kStepK;

template <int BM_, int BN_, int WM_, int WN_>
struct TileCfg {
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_;
    static constexpr int kWaves = WM * WN, kThreads = kWaves * MOE_WAVE;
    static constexpr int kPerCu = 8 / kWaves;                // workgroups: two wavefronts to a SIMD
    static constexpr int RW = BM / WM, CW = BN / WN, MI = RW / 16, NJ = CW / 16;
    static constexpr int A_BYTES = BM * kBK * 2, B_BYTES = BN * kBK * 2, STAGE = A_BYTES + B_BYTES;
    static constexpr int A_LOADS = A_BYTES / 1024 / kWaves, B_LOADS = B_BYTES / 1024 / kWaves;
    static constexpr int LOADS = A_LOADS + B_LOADS;
    static constexpr int LDS = 2 * STAGE + kWaves * 4096;    // the ring, and a piece of the epilogue's for each wavefront
    static_assert(CW == 64 && RW % 16 == 0, "the epilogue's pieces are 16 x 64");
    static_assert(A_LOADS * 1024 * kWaves == A_BYTES && B_LOADS * 1024 * kWaves == B_BYTES, "whole loads");
    static_assert(LDS * kPerCu <= 160 * 1024, "LDS");
};

struct TileArgs {
    Product p;
    Epilogue e;
    float* part;
    int64_t part_step;       // floats of one part: m * n
    int kper, splits, tiles_m, tiles_n, total;
};

enum TileEnd { kPlain, kGated, kPart };
// the operands' rows: whole 16-byte pieces on 16-byte boundaries; anywhere, eight elements and more; anything
enum Rows { kAligned, kAnywhere, kTiny };

// One operand of a tile: W rows (of A or B), 64 of K a step, in LDS 1 KB pieces of which the workgroup's wavefronts load
// L each.
//   K along the rows (TR = false): row r holds 128 B, its 16 B chunk c in slot c ^ swizzle(r), so that what LDS serves
//   of an MFMA operand (sixteen rows, four chunks) at a time lies in different 16 B columns of the 256 B that its banks span;
//   K across (TR = true): K step k holds 2 W bytes, the 32 B piece p (sixteen rows) in slot p ^ turn(k); read by
//   ds_read_b64_tr_b16, in which sixteen lanes take four K steps of a piece and come out with one row's four each.
template <class T, int W, int L, bool TR, Rows ROWS, bool PAIRED>
struct Loader {
    static constexpr bool ALIGNED = ROWS == kAligned;
    typedef typename Vec<T>::x8 x8;
    typedef Lines<W, TR> At;
    static constexpr int kPer = At::kPer;                    // rows in LDS of a load: K steps (TR) or rows of the operand
    const T* base;           // element (row0, k = 0) where TR; else row 0 of the operand
    int64_t ld;
    int row0, rows;          // the tile's first row; rows of the operand (PAIRED: of one half)
    int k0, kend;            // K of the next step, and its end
    int kstep;               // of K from step to step
    int64_t by;              // elements from step to step
    int blk0, lane;
    const T* at[ALIGNED ? L : 1];                            // load i's next place,
    int bytes[ALIGNED ? L : 1];                              // what it may reach from there,
    uint32_t off[ALIGNED ? L : 1];                           // and this lane's offset
    x8 held[ALIGNED ? 1 : L];
    int held_k0, held_kend, held_row0;

    // PAIRED: every 64 rows of the tile are 32 of the gate's and the same 32 of the up projection's
    __device__ __forceinline__ int row_of(int r) const { return PAIRED ? row0 + (r >> 6) * 32 + (r & 31) : row0 + r; }
    __device__ __forceinline__ int64_t half_of(int r) const { return PAIRED && (r & 32) ? rows : 0; }

    __device__ __forceinline__ int line(int i) const { return At::line(blk0 + i, lane); }
    __device__ __forceinline__ int chunk(int i) const { return At::chunk(blk0 + i, lane); }

    __device__ __forceinline__ void start(const void* p, int64_t ld_, int rows_, bool again, int wave, int lane_) {
        base = static_cast<const T*>(p);
        ld = ld_, rows = rows_, blk0 = wave * L, lane = lane_;
        kstep = again ? 0 : kBK, by = again ? 0 : TR ? kBK * ld : kBK;
        if constexpr (ALIGNED && !TR) {
#pragma unroll
            for (int i = 0; i < L; ++i) off[i] = At::offset(blk0 + i, lane, (int)ld, 0);
        }
    }
    // the tile whose rows start at row0_, its K from kbeg to kend_; a tile without K gives zeros
    __device__ __forceinline__ void tile(int row0_, int kbeg, int kend_) {
        row0 = row0_, k0 = kbeg, kend = kend_;
        if constexpr (ALIGNED) {
#pragma unroll
            for (int i = 0; i < L; ++i) {
                const int b = blk0 + i;
                int left;
                if constexpr (TR) {
                    at[i] = base + (int64_t)(kbeg + b * kPer) * ld + row0;
                    left = rows - row0;
                    off[i] = At::offset(b, lane, (int)ld, left);
                } else {
                    const int r = row_of(b * kPer);
                    at[i] = base + (half_of(b * kPer) + r) * ld + kbeg;
                    left = rows - r;
                }
                bytes[i] = kend > kbeg ? max(At::reach((int)ld, left, kend - kbeg), 0) * 2 : 0;
            }
        }
    }

    // load I's next piece into its place in the stage at `lds`; past the end of K come zeros
    template <int I>
    __device__ __forceinline__ void direct(uint32_t lds) {
        load_to_lds<I * 1024>(at[I], bytes[I], At::in_step(blk0 + I, lane, kend - k0) ? off[I] : kNowhere, lds);
        at[I] += by;
        if constexpr (I == L - 1) k0 += kstep;
    }

    // the first element of line `line` (128 bytes) of the 256 or fewer that step [k, k + 64) of the tile holds
    __device__ __forceinline__ const T* line_at(int line, int k) const {
        if constexpr (TR) {
            return base + (int64_t)(k + line / (W / 64)) * ld + min(row0 + line % (W / 64) * 64, rows - 1);
        } else {
            const int r = min(row_of(line), rows - 1);
            return base + (half_of(line) + r) * ld + k;
        }
    }

    // The same through registers: fetch, and put a step later.  kAnywhere takes whole 16-byte pieces, which memory serves
    // from any address: a row past the end is the last one again, and a piece that runs over its row's end is fetched from
    // eight elements before the end and shifted to its place, zeros behind it, where it is put.
    template <int I>
    __device__ __forceinline__ void fetch() {
        const int l = line(I), c = chunk(I) * 8;
        if constexpr (TR) {
            const int k = k0 + l;
            if constexpr (ROWS == kTiny)
                held[I] = load8(base + (int64_t)k * ld + row0 + c, k < kend ? min(8, rows - row0 - c) : 0);
            else
                __builtin_memcpy(&held[I], base + (int64_t)max(min(k, kend - 1), 0) * ld + min(row0 + c, rows - 8), 16);
        } else {
            const int r = row_of(l);
            if constexpr (ROWS == kTiny)
                held[I] = load8(base + (half_of(l) + r) * ld + k0 + c, r < rows ? min(8, kend - k0 - c) : 0);
            else
                __builtin_memcpy(&held[I], base + (half_of(l) + min(r, rows - 1)) * ld + max(min(k0 + c, kend - 8), 0), 16);
        }
        if constexpr (I == 0) held_k0 = k0, held_kend = kend, held_row0 = row0;
        if constexpr (I == L - 1) k0 += kstep;
    }
    __device__ __forceinline__ void put(uint8_t* lds) const {
        const bool whole = held_k0 + kBK <= held_kend && (!TR || held_row0 + W <= rows);
        if (ROWS == kTiny || whole) {
#pragma unroll
            for (int i = 0; i < L; ++i) *reinterpret_cast<x8*>(lds + (blk0 + i) * 1024 + lane * 16) = held[i];
        } else {
#pragma unroll
            for (int i = 0; i < L; ++i) {
                const int c = chunk(i) * 8, over = TR ? held_row0 + c - (rows - 8) : held_k0 + c - (held_kend - 8);
                const bool in = !TR || held_k0 + line(i) < held_kend;
                const int by = 16 * max(over, 0);
                typedef uint64_t u64x2 __attribute__((ext_vector_type(2)));
                const u64x2 v = __builtin_bit_cast(u64x2, held[i]);
                u64x2 o = {by < 64 ? v.x >> by | (by ? v.y << (64 - by) : 0) : by < 128 ? v.y >> (by - 64) : 0,
                           by < 64 ? v.y >> by : 0};
                if (!in) o = u64x2{0, 0};
                *reinterpret_cast<u64x2*>(lds + (blk0 + i) * 1024 + lane * 16) = o;
            }
        }
    }
};

// A wavefront's operand of one MFMA: rows r0 .. r0 + 15 of the tile's operand, K 32 s .. + 31 of the step.  `place` is the
// lane's part of the address, which lies clear of r0's and s's bits.
template <int W, bool TR>
__device__ __forceinline__ uint32_t place_of(int lane) {
    if constexpr (TR) {
        const int k = 8 * (lane >> 4) + (lane >> 2 & 3);     // and k + 4, which turns alike
        return k * (2 * W) + (turn<W>(k) << 5) + (lane & 3) * 8;
    } else {
        const int l = lane & 15;
        return l * (2 * kBK) + (((lane >> 4) ^ swizzle(l)) << 4);
    }
}

template <class T, int W, bool TR>
__device__ __forceinline__ typename Vec<T>::x8 fragment(const uint8_t* lds, int r0, int s, uint32_t place) {
    typedef typename Vec<T>::x8 x8;
    if constexpr (TR) {
        typedef short s16x4 __attribute__((ext_vector_type(4)));
        typedef __attribute__((address_space(3))) s16x4 lds_x4;
        typedef short s16x8 __attribute__((ext_vector_type(8)));
        const uint8_t* p = lds + 32 * s * (2 * W) + (place ^ (r0 << 1));
        const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_x4*)(p));
        const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_x4*)(p + 4 * 2 * W));
        const s16x8 v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        return __builtin_bit_cast(x8, v);
    } else {
        return *reinterpret_cast<const x8*>(lds + r0 * (2 * kBK) + (place ^ (s << 6)));
    }
}

// A workgroup's tiles.  Workgroup b runs on XCD b % 8; each XCD takes a run of the order below, in which 8 row tiles go down
// a column before the next, so that the 32 tiles in flight on an XCD share 8 + 4 operand slabs in its L2 instead of 32 + 1.
struct Tile {
    int m0, n0, split, kbeg, kend, steps;
};

template <class C, bool PAIRED>
__device__ __forceinline__ bool tile_at(const TileArgs& t, int slot, Tile& w) {
    constexpr int kGroup = 8;
    const int xcd = (int)(blockIdx.x % kXcds), id = tile_of(t.total, xcd, slot);
    if (!has_tile(t.total, xcd, slot)) return false;
    const int tiles = t.tiles_m * t.tiles_n;
    w.split = id / tiles;
    const int in = id - w.split * tiles;
    const int group = in / (kGroup * t.tiles_n);
    const int first = group * kGroup, high = min(kGroup, t.tiles_m - first);
    const int at = in - group * kGroup * t.tiles_n;
    w.m0 = (first + at % high) * C::BM;
    w.n0 = at / high * (PAIRED ? C::BN / 2 : C::BN);
    w.kbeg = w.split * t.kper;
    w.kend = min(t.p.k, w.kbeg + t.kper);
    // the ring holds two
    w.steps = max((w.kend - w.kbeg + kBK - 1) / kBK, 2);
    return true;
}

// One product's tiles, `slot_of(turn)` the place in the XCD's run of this workgroup's turn-th one; its arguments lie ARGS
// bytes into the kernel's.
template <class T, class C, bool AT, bool BT, Rows ROWS, TileEnd END, bool PAIRED, int ARGS, class SlotOf>
__device__ __forceinline__ void walk(const TileArgs& t, uint8_t* lds, SlotOf&& slot_of) {
    typedef typename Vec<T>::x8 x8;
    constexpr int MI = C::MI, NJ = C::NJ;
    constexpr bool ALIGNED = ROWS == kAligned;
    const int lane = threadIdx.x % MOE_WAVE;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / MOE_WAVE);
    const int wm = wave / C::WN, wn = wave % C::WN;
    int turn = 0;
    Tile w;
    if (!tile_at<C, PAIRED>(t, slot_of(turn), w)) return;

    Loader<T, C::BM, C::A_LOADS, AT, ROWS, false> la;
    Loader<T, C::BN, C::B_LOADS, BT, ROWS, PAIRED> lb;
    la.start(t.p.a, t.p.lda, t.p.m, false, wave, lane);
    lb.start(t.p.b, t.p.ldb, PAIRED ? t.p.inter : t.p.n, BT && t.p.b_rows, wave, lane);
    auto begin = [&](const Tile& w) __attribute__((always_inline)) {
        la.tile(w.m0, w.kbeg, w.kend);
        const bool again = BT && t.p.b_rows && w.kend;
        lb.tile(w.n0, again ? 0 : w.kbeg, again ? t.p.b_rows : w.kend);
    };
    begin(w);

    const uint32_t ring = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)MOE_LDS(lds));
    const uint32_t ring_a = ring + wave * C::A_LOADS * 1024, ring_b = ring + C::A_BYTES + wave * C::B_LOADS * 1024;
    // load i of the next step, A's before B's, for place `at` of the ring
    auto issue = [&](auto i, int at) __attribute__((always_inline)) {
        constexpr int I = decltype(i)::value;
        if constexpr (!ALIGNED) {
            if constexpr (I < C::A_LOADS) la.template fetch<I>();
            else lb.template fetch<I - C::A_LOADS>();
        } else {
            if constexpr (I < C::A_LOADS) la.template direct<I>(ring_a + at * C::STAGE);
            else lb.template direct<I - C::A_LOADS>(ring_b + at * C::STAGE);
        }
    };
    auto put = [&](int at) __attribute__((always_inline)) {
        uint8_t* to = lds + at * C::STAGE;
        la.put(to);
        lb.put(to + C::A_BYTES);
    };
    auto barrier = []() __attribute__((always_inline)) {
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
    };

    f32x4 acc[MI][NJ];
    x8 fa[2][MI], fb[2][NJ];
    uint32_t place_a = place_of<C::BM, AT>(lane), place_b = place_of<C::BN, BT>(lane);
    // fragment r of part s of the step in place `at`, in the order of first use: A's first, all of B's, the rest of A's
    auto read = [&](auto r, auto set, int at, int s) __attribute__((always_inline)) {
        constexpr int R = decltype(r)::value, S = decltype(set)::value;
        const uint8_t* from = lds + at * C::STAGE;
        if constexpr (R >= 1 && R <= NJ) {
            fb[S][R - 1] = fragment<T, C::BN, BT>(from + C::A_BYTES, wn * C::CW + 16 * (R - 1), s, place_b);
        } else {
            constexpr int i = R == 0 ? 0 : R - NJ;
            fa[S][i] = fragment<T, C::BM, AT>(from, wm * C::RW + 16 * i, s, place_a);
        }
    };

    // Part s of the step in place `at` (32 of K, in fragment set s): its products, and between them the reads of the next
    // part's fragments (none after a tile's last).  Before the second part every wavefront holds its fragments and the next
    // step has landed: from the barrier on the place is filled again.  TOUCH: requests in flight behind the step's loads.
    constexpr int kProducts = MI * NJ, kReads = MI + NJ;
    constexpr int kReadSpan = kProducts * 3 / 4, kLoadSpan = kProducts / 2;      // products over which they are spread
    auto part = [&](auto s_, auto ends, auto touches, int at) __attribute__((always_inline)) {
        constexpr int s = decltype(s_)::value;
        constexpr bool kReadOn = !(s == 1 && decltype(ends)::value);
        // (opaque, or the compiler keeps every fragment's address in a register through all of the kernel)
        asm volatile("" : "+v"(place_a), "+v"(place_b));
        if constexpr (s == 1) {
            if constexpr (!ALIGNED) put(1 - at);
            __builtin_amdgcn_s_waitcnt(kWaitLds0);
            if constexpr (ALIGNED) __builtin_amdgcn_s_waitcnt(wait_vm(decltype(touches)::value));
            barrier();
        }
        unroll<kProducts>([&](auto t) __attribute__((always_inline)) {
            constexpr int i = decltype(t)::value / NJ, j = decltype(t)::value % NJ;
            acc[i][j] = mfma(fb[s][j], fa[s][i], acc[i][j]);
            constexpr auto due = [](int n, int all, int span) { return n * all / span < all ? n * all / span : all; };
            constexpr int n = decltype(t)::value;
            constexpr int r0 = kReadOn ? due(n, kReads, kReadSpan) : 0, r1 = kReadOn ? due(n + 1, kReads, kReadSpan) : 0;
            unroll<r1 - r0>([&](auto r) __attribute__((always_inline)) {
                read(std::integral_constant<int, r0 + decltype(r)::value>{}, std::integral_constant<int, 1 - s>{},
                     s == 1 ? 1 - at : at, 1 - s);
            });
            constexpr int u0 = s == 1 ? due(n, C::LOADS, kLoadSpan) : 0, u1 = s == 1 ? due(n + 1, C::LOADS, kLoadSpan) : 0;
            unroll<u1 - u0>([&](auto u) __attribute__((always_inline)) {
                issue(std::integral_constant<int, u0 + decltype(u)::value>{}, at);
            });
            if constexpr (r1 > r0 || u1 > u0) __builtin_amdgcn_sched_barrier(0);
        });
    };

    // The sums through LDS, so that a lane holds eight columns of a row: pieces of 16 rows x 64 columns, one at a time (4 KB
    // a wavefront, the 16 B chunks swizzled by row).
    constexpr bool kPairs = PAIRED && END == kGated;
    constexpr int kRows = kPairs ? 1 : 2;                    // of a piece to a lane
    auto write = [&](const Tile& w) __attribute__((always_inline)) {
        // The lane and the arguments anew: held through the loop over K they cost registers that spill, and a spilled one's
        // reload waits for every load in flight.
        int lane;
        asm volatile("v_mbcnt_lo_u32_b32 %0, -1, 0\n\tv_mbcnt_hi_u32_b32 %0, -1, %0" : "=v"(lane));
        uint64_t segment = (uint64_t)__builtin_amdgcn_kernarg_segment_ptr() + ARGS;
        asm volatile("" : "+s"(segment));
        const auto* from = (const __attribute__((address_space(4))) TileArgs*)segment;
        TileArgs t;
        t.e.bias = from->e.bias, t.e.res = from->e.res, t.e.z = from->e.z, t.e.y = from->e.y;
        t.e.res_ld = from->e.res_ld, t.e.z_ld = from->e.z_ld, t.e.y_ld = from->e.y_ld;
        t.e.n = from->e.n, t.e.act = from->e.act;
        if constexpr (BT && END == kPlain) t.e.unit = from->e.unit;      // the backward pass's
        const float unit = unit_of<T>(t.e);
        t.part = from->part, t.part_step = from->part_step;
        t.p.m = from->p.m, t.p.n = from->p.n, t.p.inter = from->p.inter;
        uint8_t* stage = lds + 2 * C::STAGE + wave * 4096;
        const int lrow = kPairs ? lane >> 2 : lane >> 3, lcol = (kPairs ? lane & 3 : lane & 7) * 8;
        // the wait that a read of the last MFMA's result needs; the reads below are tied behind it
        asm volatile("s_nop 15");
        __builtin_amdgcn_sched_barrier(0);
        const int most = PAIRED ? t.p.inter : t.p.n;
        auto staged = [&](int row, int c, float (&v)[8]) __attribute__((always_inline)) {
            const uint8_t* at = stage + row * 256;
            const f32x4 lo = *reinterpret_cast<const f32x4*>(at + ((c ^ row) << 4));
            const f32x4 hi = *reinterpret_cast<const f32x4*>(at + (((c + 1) ^ row) << 4));
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = lo[i], v[4 + i] = hi[i];
        };
        // the row and column that a lane finishes of a piece, and its half h
        auto row_at = [&](int piece, int h) __attribute__((always_inline)) {
            return w.m0 + wm * C::RW + 16 * piece + 8 * h + lrow;
        };
        const int col = PAIRED ? w.n0 + wn * 32 + (lcol & 31) : w.n0 + wn * 64 + lcol, n = min(8, most - col);
        auto residual = [&](int piece, int h) __attribute__((always_inline)) {
            const int row = row_at(piece, h);
            return residual_of<T>(t.e, row, col, row < t.p.m ? n : 0);
        };
        x8 res[2][kRows], bias;
        if constexpr (END == kPlain) {
            bias = bias_of<T>(t.e, col, n);
#pragma unroll
            for (int h = 0; h < kRows; ++h) res[0][h] = residual(0, h);
        }
#pragma unroll
        for (int piece = 0; piece < MI; ++piece) {
            if constexpr (END == kPlain) {
                if (piece + 1 < MI) {
#pragma unroll
                    for (int h = 0; h < kRows; ++h) res[(piece + 1) & 1][h] = residual(piece + 1, h);
                }
            }
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                asm volatile("" : "+v"(acc[piece][j]));
                const int row = lane & 15;
                *reinterpret_cast<f32x4*>(stage + row * 256 + (((4 * j + (lane >> 4)) ^ row) << 4)) = acc[piece][j];
            }
            if constexpr (kPairs) {
                float gate[8], up[8];
                staged(lrow, lcol / 4, gate);
                staged(lrow, 8 + lcol / 4, up);
                if (row_at(piece, 0) < t.p.m && n > 0) finish_gated<T>(t.e, row_at(piece, 0), col, gate, up, n);
            } else {
#pragma unroll
                for (int h = 0; h < kRows; ++h) {
                    const int row = row_at(piece, h);
                    float v[8];
                    staged(8 * h + lrow, lcol / 4, v);
                    if (row >= t.p.m || n <= 0) continue;
                    if constexpr (END == kPart) {
                        float* to = t.part + w.split * t.part_step + (int64_t)row * t.p.n + col;
                        if (PAIRED && (lcol & 32)) to += t.p.inter;      // gate columns, then the up projection's
                        if (n == 8) {
                            __builtin_memcpy(to, v, 32);
                        } else {
#pragma unroll
                            for (int x = 0; x < 8; ++x)
                                if (x < n) to[x] = v[x];
                        }
                    } else {
                        if constexpr (BT) in_units<T>(v, unit);
                        finish<T>(t.e, row, col, v, n, bias, res[piece & 1][h]);
                    }
                }
            }
        }
    };

    // What the steps ahead will load, brought into the XCD's L2: the 32 workgroups of an XCD work side by side on 8 x 4
    // tiles, and each asks for its share of its two operands' lines four steps early (one request a wavefront and step, 12
    // lanes; the values go to the epilogue's corner of LDS, unread).  Where K lies along the rows of both operands, so that a
    // step takes half a kilobyte of lines from every row: 16384 x 4096 x 7168 bf16 718 -> 676 us, gated 692 -> 662, 16384 x
    // 7168 x 2048 with a residual 425 -> 412.  Across (dx, dw) it takes time: 692 -> 735 and 750 -> 758.
    constexpr bool kTouch = ALIGNED && C::kPerCu == 1 && !AT && !BT;
    constexpr std::integral_constant<int, kTouch> touches{};
    constexpr int kAhead = 3 * kBK, kShareA = 4, kShareB = 8;
    const uint8_t* touch_at = nullptr;
    int64_t touch_by = 0;
    int touch_left = 0;
    auto touch_tile = [&]() __attribute__((always_inline)) {
        constexpr int kLinesA = C::BM / kShareA / C::kWaves, kLinesB = C::BN / kShareB / C::kWaves;
        const int tm = w.m0 / C::BM, tn = w.n0 / (PAIRED ? C::BN / 2 : C::BN);
        const int k = w.kbeg + kAhead < w.kend ? w.kbeg + kAhead : w.kbeg;
        const bool of_b = lane >= kLinesA && lane < kLinesA + kLinesB;
        const int line = of_b ? (tm % kShareB * C::kWaves + wave) * kLinesB + lane - kLinesA
                              : (tn % kShareA * C::kWaves + wave) * kLinesA + lane % kLinesA;
        const uint64_t a = (uint64_t)la.line_at(line, k), b = (uint64_t)lb.line_at(line, k);
        touch_at = reinterpret_cast<const uint8_t*>(of_b ? b : a);
        const int64_t by_a = 2 * kBK * (AT ? t.p.lda : 1), by_b = 2 * kBK * (BT ? t.p.ldb : 1);
        touch_by = of_b ? by_b : by_a;
        touch_left = (w.kend - k) / kBK - 1;                 // whole steps behind that one
    };
    auto touch_step = [&]() __attribute__((always_inline)) {
        asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dword %0, off" ::"v"((uint64_t)touch_at),
                     "s"(ring + 2 * C::STAGE + wave * 4096)
                     : "memory");
        touch_at += touch_left > 0 ? touch_by : 0;
        --touch_left;
    };

    constexpr std::integral_constant<int, 0> zero{};
    constexpr std::integral_constant<int, 1> one{};
    unroll<C::LOADS>([&](auto i) __attribute__((always_inline)) { issue(i, 0); });
    if constexpr (!ALIGNED) put(0);
    unroll<C::LOADS>([&](auto i) __attribute__((always_inline)) { issue(i, 1); });
    __builtin_amdgcn_s_waitcnt(ALIGNED ? wait_vm(C::LOADS) : kWaitLds0);
    barrier();

    // (With a workgroup to a tile, 16384 x 7168 x 2048 with a residual took 458 us instead of 430.)
    int at = 0;
    for (bool more = true; more;) {
        unroll<kReads>([&](auto r) __attribute__((always_inline)) { read(r, zero, at, 0); });
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int j = 0; j < NJ; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
        if constexpr (kTouch) {
            touch_tile();
            touch_step();                                    // counted on by the first step's wait, as by the others'
        }
        for (int g = 0; g < w.steps - 2; ++g, at ^= 1) {
            part(zero, zero, touches, at);
            part(one, zero, touches, at);
            if constexpr (kTouch) touch_step();
        }
        const Tile done = w;
        more = tile_at<C, PAIRED>(t, slot_of(++turn), w);
        if (!more) w.kbeg = w.kend = 0;
        begin(w);
        part(zero, zero, zero, at);
        part(one, zero, zero, at);
        at ^= 1;
        part(zero, one, zero, at);
        part(one, one, zero, at);
        at ^= 1;
        write(done);
    }
    if constexpr (ALIGNED) __builtin_amdgcn_s_waitcnt(wait_vm(0));       // the loads past the last tile
}

using Wide = TileCfg<256, 256, 2, 4>;
using Narrow = TileCfg<128, 128, 2, 2>;
using Small = TileCfg<64, 64, 4, 1>;

template <class T, class C, bool AT, bool BT, Rows ROWS, TileEnd END, bool PAIRED>
__global__ void __launch_bounds__(C::kThreads, 2) tile_kernel(TileArgs t) {
    __shared__ __align__(16) uint8_t lds[C::LDS];
    const int first = blockIdx.x / kXcds, step = gridDim.x / kXcds;
    walk<T, C, AT, BT, ROWS, END, PAIRED, 0>(t, lds, [=](int turn) { return first + turn * step; });
}

// A backward pass's two products in one launch, dw = d^T x and then dx = d w: neither leaves a last round with most of the
// workgroups idle.  Those that dw's last round left out (an XCD's from `left` on) begin with as many of dx's tiles as one of
// dw's takes time for; the rest of them goes round as ever.  8192 x 7168 -> 4096: 1.75 rounds of 128 steps and 3.5 of 64 are
// 7 of 64 and not 8.
struct PairArgs {
    TileArgs dw, dx;
    int ahead;               // dx's tiles to one of dw's
};

template <class T>
__global__ void __launch_bounds__(Wide::kThreads, 2) pair_kernel(PairArgs t) {
    __shared__ __align__(16) uint8_t lds[Wide::LDS];
    const int me = blockIdx.x / kXcds, all = gridDim.x / kXcds;
    walk<T, Wide, true, true, kAligned, kPlain, false, offsetof(PairArgs, dw)>(t.dw, lds,
                                                                              [=](int turn) { return me + turn * all; });
    __syncthreads();
    const int left = tiles_of(t.dw.total, (int)(blockIdx.x % kXcds)) % all, ahead = left ? t.ahead : 0;
    walk<T, Wide, false, true, kAligned, kPlain, false, offsetof(PairArgs, dx)>(
        t.dx, lds, [=](int turn) { return slot_behind(me, all, left, ahead, turn); });
}

template <class C, bool PAIRED>
bool tile_args(const Plan& plan, const Product& p, const Epilogue& e, float* part, TileArgs* t) {
    t->p = p, t->e = e, t->part = part, t->part_step = (int64_t)p.m * p.n;
    t->kper = plan.kper, t->splits = plan.splits;
    t->tiles_m = (p.m + C::BM - 1) / C::BM;
    const int columns = PAIRED ? p.inter : p.n, width = PAIRED ? C::BN / 2 : C::BN;
    t->tiles_n = (columns + width - 1) / width;
    const int64_t total = (int64_t)t->tiles_m * t->tiles_n * plan.splits;
    t->total = (int)total;
    return total < (1 << 30);
}

template <class T, class C, bool AT, bool BT, Rows ROWS, TileEnd END, bool PAIRED>
moe_status launch_tile(const Plan& plan, const Product& p, const Epilogue& e, float* part, hipStream_t stream) {
    TileArgs t;
    if (!tile_args<C, PAIRED>(plan, p, e, part, &t)) return MOE_ERR_UNSUPPORTED;
    hipLaunchKernelGGL((tile_kernel<T, C, AT, BT, ROWS, END, PAIRED>),
                       dim3(std::min((t.total + kXcds - 1) / kXcds * kXcds, kCus * C::kPerCu)), dim3(C::kThreads), 0, stream, t);
    return launch_status();
}

template <class T, bool AT, bool BT, TileEnd END, bool PAIRED>
moe_status launch_rows(bool aligned, const Plan& plan, const Product& p, const Epilogue& e, float* part, hipStream_t stream) {
    if (aligned) {
        if (plan.tile == 256) return launch_tile<T, Wide, AT, BT, kAligned, END, PAIRED>(plan, p, e, part, stream);
        if (plan.tile == 64) return launch_tile<T, Small, AT, BT, kAligned, END, PAIRED>(plan, p, e, part, stream);
        return launch_tile<T, Narrow, AT, BT, kAligned, END, PAIRED>(plan, p, e, part, stream);
    }
    if (std::min(AT ? p.m : p.k, BT ? p.n : p.k) < 8)
        return launch_tile<T, Small, AT, BT, kTiny, END, PAIRED>(plan, p, e, part, stream);
    if (plan.tile == 64) return launch_tile<T, Small, AT, BT, kAnywhere, END, PAIRED>(plan, p, e, part, stream);
    return launch_tile<T, Narrow, AT, BT, kAnywhere, END, PAIRED>(plan, p, e, part, stream);
}

template <bool AT, bool BT, TileEnd END, bool PAIRED>
moe_status launch_end(int dtype, bool aligned, const Plan& plan, const Product& p, const Epilogue& e, float* part,
                      hipStream_t stream) {
    if (dtype == MOE_BF16) return launch_rows<__bf16, AT, BT, END, PAIRED>(aligned, plan, p, e, part, stream);
    return launch_rows<_Float16, AT, BT, END, PAIRED>(aligned, plan, p, e, part, stream);
}

template <bool AT, bool BT>
moe_status launch_layout(int dtype, bool aligned, const Plan& plan, const Product& p, const Epilogue& e, float* part,
                         hipStream_t stream) {
    if constexpr (!AT && !BT) {
        if (p.inter) {
            if (plan.joined)
                return launch_end<AT, BT, kPart, true>(dtype, aligned, plan, p, e, part, stream);
            return launch_end<AT, BT, kGated, true>(dtype, aligned, plan, p, e, part, stream);
        }
    }
    if (plan.joined) return launch_end<AT, BT, kPart, false>(dtype, aligned, plan, p, e, part, stream);
    return launch_end<AT, BT, kPlain, false>(dtype, aligned, plan, p, e, part, stream);
}

}  // namespace
}  // namespace moe
