// Tiled matrix products of 16-bit rows: C[m, n] = sum_k A(m, k) B(n, k) in fp32, each operand with K along its rows or
// across them, a tile of BM x BN results to a workgroup.
#pragma once

#include "dense.h"

namespace moe {
namespace {

#define MOE_LDS(p) ((void __attribute__((address_space(3)))*)(p))

constexpr int kBK = kStepK;

constexpr int wait_vm(int n) { return (n & 0xF) | (0x7 << 4) | (0xF << 8) | ((n >> 4) << 14); }
constexpr int kWaitLds0 = 0xF | (0x7 << 4) | (0x3 << 14);

template <int BM_, int BN_, int WM_, int WN_, int STAGES_>
struct TileCfg {
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, STAGES = STAGES_;
    static constexpr int kWaves = WM * WN, kThreads = kWaves * MOE_WAVE;
    static constexpr int RW = BM / WM, CW = BN / WN, MI = RW / 16, NJ = CW / 16;
    static constexpr int A_BYTES = BM * kBK * 2, B_BYTES = BN * kBK * 2, STAGE = A_BYTES + B_BYTES;
    static constexpr int A_LOADS = A_BYTES / 1024 / kWaves, B_LOADS = B_BYTES / 1024 / kWaves;
    static constexpr int LOADS = A_LOADS + B_LOADS;
    static_assert(CW == 64 && RW % 16 == 0, "the epilogue's pieces are 16 x 64");
    static_assert(A_LOADS * 1024 * kWaves == A_BYTES && B_LOADS * 1024 * kWaves == B_BYTES, "whole loads");
    static_assert(STAGES * STAGE <= 160 * 1024 && kWaves * 4096 <= STAGES * STAGE && STAGES * LOADS < 64, "LDS");
};

struct TileArgs {
    Product p;
    Epilogue e;
    float* part;
    int64_t part_step;       // floats of one part: m * n
    int kper, splits, tiles_m, tiles_n, total;
};

enum TileEnd { kPlain, kGated, kPart };

// 16 bytes a lane from p + off (zeros where that is not below `bytes`) to lds + 16 * lane.  In asm, since the compiler
// takes every transposing LDS read for one that may depend on any such load in flight and waits for all of them; the
// caller counts them (vmcnt) and waits before a barrier.  s_nop 4: the descriptor's registers may come from a
// v_readlane, whose result a vector memory instruction may read five wait states later.
__device__ __forceinline__ void load_to_lds(const void* p, int bytes, uint32_t off, uint8_t* lds) {
    const uint64_t at = (uint64_t)p;
    const u32x4 rsrc = {(uint32_t)at, (uint32_t)(at >> 32) & 0xFFFFu, (uint32_t)bytes, 0x00020000u};
    const uint32_t to = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)MOE_LDS(lds));
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 4\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds" ::"v"(off), "s"(rsrc), "s"(to)
                 : "memory");                // m0 is the compiler's own: it sets it before each of its uses
}

// One operand of a tile: W rows (of A or B), kBK of K a step, in LDS 1 KB pieces of which the workgroup's wavefronts load
// L each.
//   K along the rows (TR = false): row r holds 128 B, its 16 B chunk c in slot c ^ (r & 7) ^ (r >> 3 & 1), so that the
//   sixteen rows that an MFMA operand reads at one chunk lie in sixteen different 16 B columns of the 256 B that LDS's
//   banks span;
//   K across (TR = true): K step k holds 2 W bytes, the 32 B piece p (sixteen rows) in slot p ^ turn(k); read by
//   ds_read_b64_tr_b16, in which sixteen lanes take four K steps of a piece and come out with one row's four each.
template <class T, int W, int L, bool TR, bool ALIGNED, bool PAIRED>
struct Loader {
    typedef typename Vec<T>::x8 x8;
    static constexpr int kChunks = W / 8;                    // TR: 16 B chunks of a K step
    const T* base;           // TR: element (row0, k = 0); else row 0 of the operand
    int64_t ld;
    int row0, rows;          // the tile's first row; rows of the operand (PAIRED: of one half)
    int kend;
    int blk0, lane;
    uint32_t off[L];
    x8 held[ALIGNED ? 1 : L];

    static __device__ __forceinline__ int turn(int k) { return ((k & 3) | (k >> 3 & 3) << 2) & (W / 16 - 1); }

    // PAIRED: every 64 rows of the tile are 32 of the gate's and the same 32 of the up projection's
    __device__ __forceinline__ int row_of(int r) const { return PAIRED ? row0 + (r >> 6) * 32 + (r & 31) : row0 + r; }
    __device__ __forceinline__ int64_t half_of(int r) const { return PAIRED && (r & 32) ? rows : 0; }

    __device__ __forceinline__ int chunk(int i) const {
        const int b = blk0 + i;
        if constexpr (TR) {
            const int k = (b * 64 + lane) / kChunks;
            return (lane % kChunks) ^ (turn(k) << 1);
        } else {
            return (lane & 7) ^ (lane >> 3) ^ (b & 1);
        }
    }

    __device__ __forceinline__ void setup(const void* p, int64_t ld_, int row0_, int rows_, int kend_, int wave, int lane_) {
        base = static_cast<const T*>(p);
        ld = ld_, row0 = row0_, rows = rows_, kend = kend_, blk0 = wave * L, lane = lane_;
#pragma unroll
        for (int i = 0; i < L; ++i) {
            if constexpr (TR) off[i] = (uint32_t)(lane / kChunks) * (uint32_t)(ld * 2) + chunk(i) * 16;
            else off[i] = (uint32_t)(lane >> 3) * (uint32_t)(ld * 2) + chunk(i) * 16;
        }
    }

    // load i of K step [k0, k0 + kBK) into its place in `lds`; what lies past the operand comes as zeros, by the range
    // that the buffer descriptor holds
    __device__ __forceinline__ void direct(int i, int k0, uint8_t* lds) const {
        const int b = blk0 + i, step = (int)ld;
        const T* p;
        int count;               // elements in range; 0 or fewer rows leave a negative one
        uint32_t o = off[i];
        if constexpr (TR) {
            constexpr int kPer = 64 / kChunks;               // K steps of a load
            const int k = k0 + b * kPer;
            p = base + (int64_t)k * ld + row0;
            count = (min(kPer, kend - k) - 1) * step + min(W, rows - row0);
        } else {
            const int r = row_of(b * 8);
            p = base + (half_of(b * 8) + r) * ld + k0;
            count = (min(8, rows - r) - 1) * step + (kend - k0);
            if (k0 + kBK > kend && k0 + chunk(i) * 8 >= kend) o = 0x80000000u;   // the last step of K, or one past it
        }
        load_to_lds(p, max(count, 0) * 2, o, lds + b * 1024);
    }

    // the same through registers, for rows that start anywhere: fetch, and put a step later
    __device__ __forceinline__ void fetch(int i, int k0) {
        const int b = blk0 + i;
        if constexpr (TR) {
            const int k = k0 + (b * 64 + lane) / kChunks, c = row0 + chunk(i) * 8;
            held[i] = load8(base + (int64_t)k * ld + c, k < kend ? min(8, rows - c) : 0);
        } else {
            const int r = row_of(b * 8 + (lane >> 3)), c = k0 + chunk(i) * 8;
            held[i] = load8(base + (half_of(b * 8) + r) * ld + c, r < rows ? min(8, kend - c) : 0);
        }
    }
    __device__ __forceinline__ void put(int i, uint8_t* lds) const {
        *reinterpret_cast<x8*>(lds + (blk0 + i) * 1024 + lane * 16) = held[i];
    }
};

// A wavefront's operand of one MFMA: rows r0 .. r0 + 15 of the tile's operand, K 32 s .. + 31 of the step.
template <class T, int W, bool TR>
__device__ __forceinline__ typename Vec<T>::x8 fragment(const uint8_t* lds, int r0, int s, int lane) {
    typedef typename Vec<T>::x8 x8;
    const int q = lane >> 4;
    if constexpr (TR) {
        typedef short s16x4 __attribute__((ext_vector_type(4)));
        typedef __attribute__((address_space(3))) s16x4 lds_x4;
        typedef short s16x8 __attribute__((ext_vector_type(8)));
        const int i = lane >> 2 & 3;
        const int turn = (i | q << 2) & (W / 16 - 1);        // of K step 32 s + 8 q + 4 h + i
        const uint8_t* p = lds + (32 * s + 8 * q + i) * (2 * W) + (((r0 >> 4) ^ turn) << 5) + (lane & 3) * 8;
        const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_x4*)(p));
        const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_x4*)(p + 4 * 2 * W));
        const s16x8 v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        return __builtin_bit_cast(x8, v);
    } else {
        const int l = lane & 15;
        const int sw = (l & 7) ^ (l >> 3);
        return *reinterpret_cast<const x8*>(lds + (r0 + l) * 128 + (((4 * s + q) ^ sw) << 4));
    }
}

// The tile that a workgroup takes.  Workgroup b runs on XCD b % 8; each XCD takes a run of the order below, in which 8
// row tiles go down a column before the next, so that the 32 tiles in flight on an XCD share 8 + 4 operand slabs in its
// L2 instead of 32 + 1.
__device__ __forceinline__ bool tile_of(const TileArgs& t, int& tm, int& tn, int& split) {
    constexpr int kXcds = 8, kGroup = 8;
    const int per = (t.total + kXcds - 1) / kXcds;
    const int id = (int)(blockIdx.x % kXcds) * per + (int)(blockIdx.x / kXcds);
    if (id >= t.total) return false;
    const int tiles = t.tiles_m * t.tiles_n;
    split = id / tiles;
    const int in = id - split * tiles;
    const int group = in / (kGroup * t.tiles_n);
    const int first = group * kGroup, high = min(kGroup, t.tiles_m - first);
    const int at = in - group * kGroup * t.tiles_n;
    tm = first + at % high;
    tn = at / high;
    return true;
}

template <class T, class C, bool AT, bool BT, bool ALIGNED, TileEnd END, bool PAIRED>
__global__ void __launch_bounds__(C::kThreads, 2)
tile_kernel(TileArgs t) {
    typedef typename Vec<T>::x8 x8;
    constexpr int MI = C::MI, NJ = C::NJ;
    __shared__ __align__(16) uint8_t lds[C::STAGES * C::STAGE];
    int tm, tn, split;
    if (!tile_of(t, tm, tn, split)) return;
    const int lane = threadIdx.x % MOE_WAVE;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / MOE_WAVE);
    const int wm = wave / C::WN, wn = wave % C::WN;
    const int m0 = tm * C::BM, n0 = tn * (PAIRED ? C::BN / 2 : C::BN);
    const int kbeg = split * t.kper, kend = min(t.p.k, kbeg + t.kper);
    const int steps = (kend - kbeg + kBK - 1) / kBK;

    Loader<T, C::BM, C::A_LOADS, AT, ALIGNED, false> la;
    Loader<T, C::BN, C::B_LOADS, BT, ALIGNED, PAIRED> lb;
    la.setup(t.p.a, t.p.lda, m0, t.p.m, kend, wave, lane);
    lb.setup(t.p.b, t.p.ldb, n0, PAIRED ? t.p.inter : t.p.n, kend, wave, lane);

    auto issue_a = [&](int i, int g) __attribute__((always_inline)) {
        if constexpr (ALIGNED) la.direct(i, kbeg + g * kBK, lds + (g % C::STAGES) * C::STAGE);
        else la.fetch(i, kbeg + g * kBK);
    };
    auto issue_b = [&](int i, int g) __attribute__((always_inline)) {
        if constexpr (ALIGNED) lb.direct(i, kbeg + g * kBK, lds + (g % C::STAGES) * C::STAGE + C::A_BYTES);
        else lb.fetch(i, kbeg + g * kBK);
    };
    auto put = [&](int g) __attribute__((always_inline)) {
        uint8_t* at = lds + (g % C::STAGES) * C::STAGE;
#pragma unroll
        for (int i = 0; i < C::A_LOADS; ++i) la.put(i, at);
#pragma unroll
        for (int i = 0; i < C::B_LOADS; ++i) lb.put(i, at + C::A_BYTES);
    };
    auto barrier = []() __attribute__((always_inline)) {
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
    };

    f32x4 acc[MI][NJ];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

    x8 fa[2][MI], fb[2][NJ];
    auto read_a = [&](int g, int s, int i) __attribute__((always_inline)) {
        return fragment<T, C::BM, AT>(lds + (g % C::STAGES) * C::STAGE, wm * C::RW + 16 * i, s, lane);
    };
    auto read_b = [&](int g, int s, int j) __attribute__((always_inline)) {
        return fragment<T, C::BN, BT>(lds + (g % C::STAGES) * C::STAGE + C::A_BYTES, wn * C::CW + 16 * j, s, lane);
    };

    // the ring: step g's loads go out as soon as every wavefront holds the last fragments of step g - STAGES, half a step
    // before that step's MFMAs end
    if constexpr (ALIGNED) {
#pragma unroll
        for (int g = 0; g < C::STAGES; ++g) {
#pragma unroll
            for (int i = 0; i < C::A_LOADS; ++i) issue_a(i, g);
#pragma unroll
            for (int i = 0; i < C::B_LOADS; ++i) issue_b(i, g);
        }
        __builtin_amdgcn_s_waitcnt(wait_vm((C::STAGES - 1) * C::LOADS));
    } else {
        static_assert(ALIGNED || C::STAGES == 2, "one step in registers, one in LDS, one free");
#pragma unroll
        for (int i = 0; i < C::A_LOADS; ++i) issue_a(i, 0);
#pragma unroll
        for (int i = 0; i < C::B_LOADS; ++i) issue_b(i, 0);
        put(0);
#pragma unroll
        for (int i = 0; i < C::A_LOADS; ++i) issue_a(i, 1);
#pragma unroll
        for (int i = 0; i < C::B_LOADS; ++i) issue_b(i, 1);
        __builtin_amdgcn_s_waitcnt(kWaitLds0);
    }
    barrier();
#pragma unroll
    for (int j = 0; j < NJ; ++j) fb[0][j] = read_b(0, 0, j);
#pragma unroll
    for (int i = 0; i < MI; ++i) fa[0][i] = read_a(0, 0, i);

    for (int g = 0; g < steps; ++g) {
        // first half: its MFMAs, between them the reads of the second half's fragments
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            if (i < NJ) fb[1][i] = read_b(g, 1, i);
            fa[1][i] = read_a(g, 1, i);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int j = 0; j < NJ; ++j) acc[i][j] = mfma(fb[0][j], fa[0][i], acc[i][j]);
            __builtin_amdgcn_sched_barrier(0);
        }
        if constexpr (!ALIGNED) put(g + 1);
        // every read of step g has returned; step g + 1 has landed
        __builtin_amdgcn_s_waitcnt(kWaitLds0);
        if constexpr (ALIGNED) __builtin_amdgcn_s_waitcnt(wait_vm((C::STAGES - 2) * C::LOADS));
        barrier();
        // second half: its MFMAs, between them step g + STAGES's loads and the first reads of step g + 1
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            if (i < NJ) fb[0][i] = read_b(g + 1, 0, i);
            fa[0][i] = read_a(g + 1, 0, i);
#pragma unroll
            for (int u = i * C::LOADS / MI; u < (i + 1) * C::LOADS / MI; ++u) {
                if (u < C::A_LOADS) issue_a(u, g + C::STAGES);
                else issue_b(u - C::A_LOADS, g + C::STAGES);
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int j = 0; j < NJ; ++j) acc[i][j] = mfma(fb[1][j], fa[1][i], acc[i][j]);
            __builtin_amdgcn_sched_barrier(0);
        }
    }

    // the sums through LDS, sixteen rows at a time, so that a lane holds eight columns of a row; each wavefront has 4 KB,
    // its 16 B chunks swizzled by row
    __builtin_amdgcn_s_waitcnt(kWaitLds0);
    __builtin_amdgcn_s_waitcnt(wait_vm(0));
    barrier();
    // the wait that a read of the last MFMA's result needs; the reads below are tied behind it
    asm volatile("s_nop 15");
    __builtin_amdgcn_sched_barrier(0);
    uint8_t* stage = lds + wave * 4096;
    const int srow = lane & 15, q = lane >> 4;
    auto staged = [&](int row, int c, float (&v)[8]) __attribute__((always_inline)) {
        const f32x4 lo = *reinterpret_cast<const f32x4*>(stage + row * 256 + ((c ^ row) << 4));
        const f32x4 hi = *reinterpret_cast<const f32x4*>(stage + row * 256 + (((c + 1) ^ row) << 4));
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = lo[i], v[4 + i] = hi[i];
    };
#pragma unroll
    for (int i = 0; i < MI; ++i) {
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            asm volatile("" : "+v"(acc[i][j]));
            *reinterpret_cast<f32x4*>(stage + srow * 256 + (((4 * j + q) ^ srow) << 4)) = acc[i][j];
        }
        const int mrow = m0 + wm * C::RW + 16 * i;
        if constexpr (PAIRED && END == kGated) {
            const int row = lane >> 2, c = (lane & 3) * 8, col = n0 + wn * 32 + c;
            float gate[8], up[8];
            staged(row, c / 4, gate);
            staged(row, 8 + c / 4, up);
            if (mrow + row < t.p.m && col < t.p.inter)
                finish_gated<T>(t.e, mrow + row, col, gate, up, min(8, t.p.inter - col));
        } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int row = 8 * h + (lane >> 3), c = (lane & 7) * 8;
                int col = n0 + wn * 64 + c, most = t.p.n;
                if constexpr (PAIRED) {                      // gate columns, then the up projection's
                    col = n0 + wn * 32 + (c & 31);
                    most = t.p.inter;
                }
                float v[8];
                staged(row, c / 4, v);
                if (mrow + row >= t.p.m || col >= most) continue;
                const int n = min(8, most - col);
                if constexpr (END == kPart) {
                    float* at = t.part + split * t.part_step + (int64_t)(mrow + row) * t.p.n + col;
                    if (PAIRED && (c & 32)) at += t.p.inter;
#pragma unroll
                    for (int x = 0; x < 8; ++x)
                        if (x < n) at[x] = v[x];
                } else {
                    finish<T>(t.e, mrow + row, col, v, n);
                }
            }
        }
    }
}

using Wide = TileCfg<256, 256, 2, 4, 2>;
using Narrow = TileCfg<128, 128, 2, 2, 2>;

template <class T, class C, bool AT, bool BT, bool ALIGNED, TileEnd END, bool PAIRED>
moe_status launch_tile(const Plan& plan, const Product& p, const Epilogue& e, float* part, hipStream_t stream) {
    TileArgs t;
    t.p = p, t.e = e, t.part = part, t.part_step = (int64_t)p.m * p.n;
    t.kper = plan.kper, t.splits = plan.splits;
    t.tiles_m = (p.m + C::BM - 1) / C::BM;
    const int columns = PAIRED ? p.inter : p.n, width = PAIRED ? C::BN / 2 : C::BN;
    t.tiles_n = (columns + width - 1) / width;
    const int64_t total = (int64_t)t.tiles_m * t.tiles_n * plan.splits;
    if (total > (1 << 24)) return MOE_ERR_UNSUPPORTED;
    t.total = (int)total;
    hipLaunchKernelGGL((tile_kernel<T, C, AT, BT, ALIGNED, END, PAIRED>), dim3((t.total + 7) / 8 * 8),
                       dim3(C::kThreads), 0, stream, t);
    return launch_status();
}

template <bool AT, bool BT, TileEnd END, bool PAIRED>
moe_status launch_end(int dtype, bool aligned, const Plan& plan, const Product& p, const Epilogue& e, float* part,
                      hipStream_t stream) {
    if (dtype == MOE_BF16) {
        if (!aligned) return launch_tile<__bf16, Narrow, AT, BT, false, END, PAIRED>(plan, p, e, part, stream);
        if (plan.tile == 256) return launch_tile<__bf16, Wide, AT, BT, true, END, PAIRED>(plan, p, e, part, stream);
        return launch_tile<__bf16, Narrow, AT, BT, true, END, PAIRED>(plan, p, e, part, stream);
    }
    if (!aligned) return launch_tile<_Float16, Narrow, AT, BT, false, END, PAIRED>(plan, p, e, part, stream);
    if (plan.tile == 256) return launch_tile<_Float16, Wide, AT, BT, true, END, PAIRED>(plan, p, e, part, stream);
    return launch_tile<_Float16, Narrow, AT, BT, true, END, PAIRED>(plan, p, e, part, stream);
}

template <bool AT, bool BT>
moe_status launch_layout(int dtype, bool aligned, const Plan& plan, const Product& p, const Epilogue& e, float* part,
                         hipStream_t stream) {
    if constexpr (!AT && !BT) {
        if (p.inter) {
            if (plan.splits > 1)
                return launch_end<AT, BT, kPart, true>(dtype, aligned, plan, p, e, part, stream);
            return launch_end<AT, BT, kGated, true>(dtype, aligned, plan, p, e, part, stream);
        }
    }
    if (plan.splits > 1) return launch_end<AT, BT, kPart, false>(dtype, aligned, plan, p, e, part, stream);
    return launch_end<AT, BT, kPlain, false>(dtype, aligned, plan, p, e, part, stream);
}

}  // namespace
}  // namespace moe
