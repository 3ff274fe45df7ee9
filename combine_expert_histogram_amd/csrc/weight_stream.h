// The inner loop shared by the few-token kernels: a wavefront multiplies tiles of 16 weight rows by up to 16 * CT
// token columns along a run of 128-element K blocks, the weights streamed from HBM once and never kept.
//
//   D[row, col] += sum_k W[row, k] * x[col, k]
//
// Matrix instruction: v_mfma_f32_16x16x32_bf16 with the weights as its A operand (lane l holds row l % 16) and the
// tokens as its B operand (column l % 16), so a lane's four results are four consecutive weight rows of one token.
// Every weight format widens to bf16 without rounding (an e4m3 or e2m1 code times a power of two; an integer
// 128 + q), so the products are those of the definition and the sums are fp32.  One token uses one column of the
// sixteen: with 4-bit weights the matrix cores take 16 cycles of a CU for a KiB and column tile, the weight stream 90
// (at 7 TB/s), so up to 64 tokens the stream is the floor.  What it comes to on one MI355X, us and TB/s of weights:
//   131072 x 7168 e2m1: 1 token 91 (5.5), 16 tokens 115 (4.4), 64 tokens 136 to 146 (3.7)
//   65536 x 7168 e4m3:  1 token 78 (6.0), 16 tokens 85 (5.6), 64 tokens 106 to 110 (4.4); e4m3_mx 81, 86, 109
//   131072 x 7168 int4, 1 token: groups of 128 98 (5.0), of 32 145 (3.9: vector instructions, 16 scales a row tile's
//   block and lane to convert and apply); 16 tokens 119 and 154
//
// An integer is widened as 128 + q, and a group's sum corrected by (128 + zero) times the sum of x.  The two sums are up
// to 143 scales of sum |x| where (q - zero) x itself stays below 15, so three to four of fp32's bits go to the
// difference: an error of about 1e-5 of an ordinary group's sum, unseen in a bf16 output unless the groups cancel.
// Exact signed values would take a conversion an element where this takes a mask and an or for two.
//
// Which k a lane holds is free as long as both operands agree.  A lane always loads 16 B of one weight row, four
// lanes cover 64 B of it, and the K order of the MFMAs follows from that:
//   8-bit codes: piece i (of two) of a block, MFMA s (of two): k = 64 i + 16 g + 8 s + j        (g = l / 16, j < 8)
//   e2m1:        MFMA s (of four):                              k = 32 g + 8 s + j: a lane's 16 B are one scale group
//   int4:        MFMA s (of four):                              k = 32 s + 8 g + j: an MFMA covers one group of 32
// The int4 storage order makes the last line contiguous in memory (word 4g + s of a block holds 32s + 8g .. + 7).
#pragma once

#include "common.h"

namespace moe {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int kKBlock = 128;

// One weight matrix (or one expert's) as the kernels see it.
struct WView {
    const uint8_t* data;     // [n, K] bytes or [n, K/2]
    const void* scale;
    const uint8_t* zero;     // int4 only, may be null
    int64_t n;
    int nb;                  // K blocks of 128
};

// FMT is a moe_weight_format; G the scale groups per block of an int4 format (1, 2 or 4), else 1.
template <int FMT, int G>
struct Fmt {
    static constexpr bool kInt4 = FMT == MOE_W_INT4;
    static constexpr bool kFour = FMT == MOE_W_INT4 || FMT == MOE_W_E2M1_MX;
    static constexpr bool kMx = FMT == MOE_W_E4M3_MX || FMT == MOE_W_E2M1_MX;
    static constexpr int kRowBytes = kFour ? 64 : 128;       // of a block
    static constexpr int kLoads = kFour ? 1 : 2;             // 16 B loads a lane, block and tile
};

// The scales of R tiles and one block, one load for all of them: the sixteen lanes that would repeat one tile's
// scales fetch other tiles' instead, and spread_rows or row_lane hands them round.
//   e4m3: the R tiles lie in one 128-row scale block, so every lane's own word serves all of them.
//   MX:   lane l fetches the word of row l % 16 of tile (l / 16) % R.
//   int4: lane l fetches the four rows 4 (l / 16) .. + 3 of tile (l % 16) % R.
template <int FMT, int G>
struct Scales {
    uint32_t w;                                              // MX codes, or the fp32 scale's bits
};
template <int G>
struct Scales<MOE_W_INT4, G> {
    uint32_t s[2 * G];                                       // 4 rows x G bf16
    uint32_t z[G];                                           // 4 rows x G bytes
};

// A memory instruction costs its CU one cycle for every run of adjacent lanes that reads within 64 B.  In the MFMA
// layout adjacent lanes hold different rows, which makes 64 such runs of 16 B; so the four lanes 4 r .. 4 r + 3 fetch
// 64 B of row r, and the wavefront turns the 1 KiB piece into the MFMA layout through its own corner of LDS (LDS
// instructions of one wavefront stay in order, so this takes no barrier).  Before: the cache accesses were busy 85 % of
// the time with 16 tokens (131072 x 7168 e2m1, 171 us; 115 since).  The swizzle makes the eight
// lanes that LDS serves at a time (four neighbours and four of the next sixteen lanes) fall on distinct banks, for the
// writes (two rows) and the reads (one 16 B column of four rows, the next column of the other four).
constexpr int kCorner = 4 * 64;                              // 16 B elements of a wavefront's corner

__device__ __forceinline__ int turn_slot(int row, int piece) { return row * 4 + (piece ^ (row >> 1 & 3) ^ (row >> 3)); }

__device__ __forceinline__ void turn_in(u32x4* lds, const u32x4& v) {
    const int l = lane_id();
    lds[turn_slot(l >> 2, l & 3)] = v;
}
__device__ __forceinline__ u32x4 turn_out(const u32x4* lds, int piece) { return lds[turn_slot(lane_id() & 15, piece)]; }

// R tiles of sixteen rows, as one lane addresses them.
template <int FMT, int G, int R>
struct Tiles {
    const uint8_t* w[R];     // row lane / 4 of each tile, at 16 B piece lane % 4
    const uint8_t* s;        // block 0's scales
    const uint8_t* z;
};

// a_row(t, i): the weight row in row i of tile t;  d_row(t, i): the first of the four rows of tile t that a lane of
// group i = lane / 16 holds results of.
template <int FMT, int G, int R, class ARow, class DRow>
__device__ __forceinline__ Tiles<FMT, G, R> tiles_of(const WView& v, ARow&& a_row, DRow&& d_row) {
    using F = Fmt<FMT, G>;
    const int l = lane_id(), g = l >> 4, c = l & 15;
    Tiles<FMT, G, R> t;
#pragma unroll
    for (int r = 0; r < R; ++r) t.w[r] = v.data + (int64_t)a_row(r, l >> 2) * v.nb * F::kRowBytes + 16 * (l & 3);
    t.z = nullptr;
    const uint8_t* s = static_cast<const uint8_t*>(v.scale);
    if constexpr (F::kInt4) {
        const int64_t row = d_row(c % R, g);
        t.s = s + row * 2 * G;
        if (v.zero) t.z = v.zero + row * G;
    } else if constexpr (F::kMx) {
        t.s = s + (int64_t)a_row(g % R, c) * 4;
    } else {
        t.s = s + (int64_t)(d_row(0, g) / 128) * v.nb * 4;
    }
    return t;
}

// A column tile of XT = 4, 8 or 16 tokens: with fewer than sixteen, token t owns the 16 / XT columns from t * 16 / XT,
// its lanes fetch different parts of the token's values and a quad permutation hands them round, so a block takes
// XT / 4 loads instead of four.
template <int FMT, int G, int R, int CT, int XT>
struct Step {                                                // one K block in flight
    u32x4 w[R][Fmt<FMT, G>::kLoads];
    Scales<FMT, G> s;
    u32x4 x[CT][XT / 4];
};

template <int FMT, int G, int R>
__device__ __forceinline__ void load_weights(const Tiles<FMT, G, R>& t, const WView& v, int kb,
                                             u32x4 (&w)[R][Fmt<FMT, G>::kLoads], Scales<FMT, G>& s) {
    using F = Fmt<FMT, G>;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const u32x4* p = reinterpret_cast<const u32x4*>(t.w[r] + (int64_t)kb * F::kRowBytes);
#pragma unroll
        for (int i = 0; i < F::kLoads; ++i) w[r][i] = p[4 * i];
    }
    if constexpr (F::kInt4) {
        const int64_t at = (int64_t)kb * v.n;
        const uint8_t* ps = t.s + at * 2 * G;
        if constexpr (G == 1) {
            const u32x2 a = *reinterpret_cast<const u32x2*>(ps);
            s.s[0] = a.x, s.s[1] = a.y;
        } else {
#pragma unroll
            for (int i = 0; i < G / 2; ++i) {
                const u32x4 a = *(reinterpret_cast<const u32x4*>(ps) + i);
                s.s[4 * i] = a.x, s.s[4 * i + 1] = a.y, s.s[4 * i + 2] = a.z, s.s[4 * i + 3] = a.w;
            }
        }
        if (v.zero) {
            const uint8_t* pz = t.z + at * G;
            if constexpr (G == 1) {
                s.z[0] = *reinterpret_cast<const uint32_t*>(pz);
            } else if constexpr (G == 2) {
                const u32x2 a = *reinterpret_cast<const u32x2*>(pz);
                s.z[0] = a.x, s.z[1] = a.y;
            } else {
                const u32x4 a = *reinterpret_cast<const u32x4*>(pz);
                s.z[0] = a.x, s.z[1] = a.y, s.z[2] = a.z, s.z[3] = a.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < G; ++i) s.z[i] = 0x08080808u;
        }
    } else if constexpr (F::kMx) {
        s.w = *reinterpret_cast<const uint32_t*>(t.s + (int64_t)kb * v.n * 4);
    } else {
        s.w = *reinterpret_cast<const uint32_t*>(t.s + (int64_t)kb * 4);
    }
}

// MX: tile t's word of this lane's row, from the lanes that fetched it.
template <int R>
__device__ __forceinline__ void spread_rows(uint32_t w, uint32_t (&o)[R]) {
    static_assert(R == 1 || R == 2 || R == 4, "tiles");
    if constexpr (R == 1) {
        o[0] = w;
    } else if constexpr (R == 2) {                           // rows of lanes [0 1 0 1] -> [0 0 0 0], [1 1 1 1]
        const auto p = __builtin_amdgcn_permlane16_swap(w, w, false, false);
        o[0] = p[0], o[1] = p[1];
    } else {                                                 // [0 1 2 3] -> [0 1 0 1], [2 3 2 3], then as above
        const auto h = __builtin_amdgcn_permlane32_swap(w, w, false, false);
        const auto p = __builtin_amdgcn_permlane16_swap(h[0], h[0], false, false);
        const auto q = __builtin_amdgcn_permlane16_swap(h[1], h[1], false, false);
        o[0] = p[0], o[1] = p[1], o[2] = q[0], o[3] = q[1];
    }
}

// int4: the word that lane t of each sixteen holds
template <int T>
__device__ __forceinline__ uint32_t row_lane(uint32_t w) {
    return (uint32_t)__builtin_amdgcn_mov_dpp((int)w, 0x150 + T, 0xF, 0xF, false);    // row_newbcast
}

// ... of tile r (a constant after unrolling)
template <int R>
__device__ __forceinline__ uint32_t tile_word(uint32_t w, int r) {
    if constexpr (R == 1) return w;
    return r == 0 ? row_lane<0>(w) : r == 1 ? row_lane<1>(w) : r == 2 ? row_lane<2>(w) : row_lane<3>(w);
}

template <int G, int R, int T = 0>
__device__ __forceinline__ void spread_lanes(const Scales<MOE_W_INT4, G>& s, Scales<MOE_W_INT4, G> (&o)[R]) {
    if constexpr (R == 1) {
        o[0] = s;
    } else if constexpr (T < R) {
#pragma unroll
        for (int i = 0; i < 2 * G; ++i) o[T].s[i] = row_lane<T>(s.s[i]);
#pragma unroll
        for (int i = 0; i < G; ++i) o[T].z[i] = row_lane<T>(s.z[i]);
        spread_lanes<G, R, T + 1>(s, o);
    }
}

// Element offset, inside a block, of the eight x values that MFMA q of the lane group g multiplies.
template <int FMT, int G>
__device__ __forceinline__ int x_offset(int q, int g) {
    using F = Fmt<FMT, G>;
    if constexpr (F::kInt4) return 32 * q + 8 * g;
    if constexpr (F::kFour) return 32 * g + 8 * q;
    return 64 * (q >> 1) + 16 * g + 8 * (q & 1);
}

template <int CTRL>
__device__ __forceinline__ u32x4 quad_perm(const u32x4& v) {
    u32x4 o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = (uint32_t)__builtin_amdgcn_mov_dpp((int)v[i], CTRL, 0xF, 0xF, true);
    return o;
}

// The eight token values of MFMA q of a block (q a constant after unrolling).
template <int XT>
__device__ __forceinline__ bf16x8 token_values(const u32x4 (&x)[XT / 4], int q) {
    u32x4 v;
    if constexpr (XT == 16) {
        v = x[q];
    } else if constexpr (XT == 8) {
        v = q & 1 ? quad_perm<0xF5>(x[q >> 1]) : quad_perm<0xA0>(x[q >> 1]);    // lanes 1 1 3 3 or 0 0 2 2
    } else {
        v = q == 0 ? quad_perm<0x00>(x[0]) : q == 1 ? quad_perm<0x55>(x[0])
                                         : q == 2 ? quad_perm<0xAA>(x[0]) : quad_perm<0xFF>(x[0]);
    }
    return __builtin_bit_cast(bf16x8, v);
}

// The eight bf16 values of MFMA q of a block (exact).  int4 gives 128 + code.
template <int FMT, int G>
__device__ __forceinline__ bf16x8 widen(const u32x4 (&w)[Fmt<FMT, G>::kLoads], float mx, int q) {
    using F = Fmt<FMT, G>;
    u32x4 o;
    if constexpr (F::kInt4) {
        const uint32_t v = w[0][q];
        // nibble p of the word is element 2p, nibble p + 4 element 2p + 1: 0x4300 | code is the bf16 128 + code
#pragma unroll
        for (int p = 0; p < 4; ++p) o[p] = ((v >> (4 * p)) & 0x000F000Fu) | 0x43004300u;
    } else if constexpr (F::kFour) {
        const uint32_t v = w[0][q];
        o[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, mx, 0));
        o[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, mx, 1));
        o[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, mx, 2));
        o[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, mx, 3));
    } else {
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            const uint32_t v = w[q >> 1][2 * (q & 1) + p];
            o[2 * p] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, mx, false));
            o[2 * p + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, mx, true));
        }
    }
    return __builtin_bit_cast(bf16x8, o);
}

__device__ __forceinline__ float e8m0_value(uint32_t word, int byte) {
    return __uint_as_float(((word >> (8 * byte)) & 0xFFu) << 23);
}

__device__ __forceinline__ f32x4 mfma(bf16x8 a, bf16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// Waits out the matrix pipeline before d is read.  The result of this MFMA (four passes) may be read by the VALU eight
// wait states after it, which is what the compiler leaves in straight code; where it moved the reading instructions
// behind a branch it left them out (seen in the listing: MFMA, s_cbranch, v_mov, v_fmac of the result, and a first
// component short of the last two MFMAs).  The asm ties the wait to the values, so no branch can come between.
template <int N>
__device__ __forceinline__ void settle(f32x4 (&d)[N]) {
    static_assert(N >= 1 && N <= 5, "tiles");
    if constexpr (N == 1) asm volatile("s_nop 15" : "+v"(d[0]));
    if constexpr (N == 2) asm volatile("s_nop 15" : "+v"(d[0]), "+v"(d[1]));
    if constexpr (N == 3) asm volatile("s_nop 15" : "+v"(d[0]), "+v"(d[1]), "+v"(d[2]));
    if constexpr (N == 4) asm volatile("s_nop 15" : "+v"(d[0]), "+v"(d[1]), "+v"(d[2]), "+v"(d[3]));
    if constexpr (N == 5)
        asm volatile("s_nop 15" : "+v"(d[0]), "+v"(d[1]), "+v"(d[2]), "+v"(d[3]), "+v"(d[4]));
}

// Fetched pieces of R tiles into the MFMA layout.
template <int FMT, int G, int R>
__device__ __forceinline__ void turn_weights(u32x4* corner, u32x4 (&w)[R][Fmt<FMT, G>::kLoads]) {
    constexpr int L = Fmt<FMT, G>::kLoads, kBuf = R * L < kCorner / 64 ? R * L : kCorner / 64;
#pragma unroll
    for (int r = 0; r < R; r += kBuf / L) {
#pragma unroll
        for (int p = 0; p < kBuf; ++p) turn_in(corner + 64 * p, w[r + p / L][p % L]);
#pragma unroll
        for (int p = 0; p < kBuf; ++p) w[r + p / L][p % L] = turn_out(corner + 64 * p, lane_id() >> 4);
    }
}

// acc += one K block.  cols: bit c set where column tile c has a token (uniform over the wavefront).
template <int FMT, int G, int R, int CT, int XT>
__device__ __forceinline__ void block_product(Step<FMT, G, R, CT, XT>& st, uint32_t cols, u32x4* corner,
                                              f32x4 (&acc)[R][CT]) {
    using F = Fmt<FMT, G>;
    if constexpr (XT == 16) {
#pragma unroll
        for (int c = 0; c < CT; ++c) {
            if (CT > 1 && !(cols >> c & 1)) continue;
#pragma unroll
            for (int q = 0; q < 4; ++q) turn_in(corner + 64 * q, st.x[c][q]);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int piece = x_offset<FMT, G>(q, lane_id() >> 4) / 8;       // of the block's sixteen 16 B pieces
                st.x[c][q] = turn_out(corner + (piece >> 2) * 64, piece & 3);
            }
        }
    }
    turn_weights<FMT, G, R>(corner, st.w);
    const int g = lane_id() >> 4;
    const f32x4 none = {0.f, 0.f, 0.f, 0.f};
    if constexpr (CT == 1 && G == 1) {
        // two tiles at a time, widened where they are used: what is live at once decides the wavefronts of a CU
        constexpr int TG = R < 2 ? R : 2;
        const u32x4 ones_bits = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
        uint32_t words[R];
        if constexpr (F::kMx) spread_rows<R>(st.s.w, words);
        f32x4 sum = none;                                    // int4: sum x, beside the first tiles
#pragma unroll
        for (int r0 = 0; r0 < R; r0 += TG) {
            const bool sums = F::kInt4 && r0 == 0;
            f32x4 d[F::kInt4 ? TG + 1 : TG];
#pragma unroll
            for (int r = 0; r < TG; ++r) d[r] = F::kMx ? acc[r0 + r][0] : none;
            if constexpr (F::kInt4) d[TG] = sum;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const bf16x8 b = token_values<XT>(st.x[0], q);
#pragma unroll
                for (int r = 0; r < TG; ++r) {
                    float mx = 1.0f;
                    if constexpr (F::kMx) mx = e8m0_value(words[r0 + r], F::kFour ? g : 2 * (q >> 1) + (g >> 1));
                    d[r] = mfma(widen<FMT, G>(st.w[r0 + r], mx, q), b, d[r]);
                }
                if constexpr (F::kInt4)
                    if (sums) d[TG] = mfma(__builtin_bit_cast(bf16x8, ones_bits), b, d[TG]);
            }
            settle(d);
            if constexpr (F::kInt4) sum = d[TG];
#pragma unroll
            for (int r = 0; r < TG; ++r) {
                if constexpr (F::kMx) {
                    acc[r0 + r][0] = d[r];
                } else if constexpr (F::kInt4) {
                    // sum (q - z) s x = s (sum (128 + q) x - (128 + z) sum x)
                    const uint32_t zw = tile_word<R>(st.s.z[0], r0 + r) | 0x80808080u;       // 128 + zero
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t sw = tile_word<R>(st.s.s[i >> 1], r0 + r);
                        const float s = i & 1 ? bf16_hi(sw) : bf16_lo(sw);
                        const float z = (float)((zw >> (8 * i)) & 0xFFu);
                        acc[r0 + r][0][i] = fmaf(s, fmaf(-z, sum[i], d[r][i]), acc[r0 + r][0][i]);
                    }
                } else {
                    const float s = __uint_as_float(st.s.w);
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[r0 + r][0][i] = fmaf(s, d[r][i], acc[r0 + r][0][i]);
                }
            }
        }
    } else if constexpr (F::kInt4) {
        // sum (q - z) s x = s (sum (128 + q) x - (128 + z) sum x) per scale group; sum x from an MFMA by ones
        const u32x4 ones_bits = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
        const bf16x8 ones = __builtin_bit_cast(bf16x8, ones_bits);
        constexpr int Q = 4 / G;                             // MFMAs per group
        Scales<FMT, G> sc[R];
        spread_lanes<G, R>(st.s, sc);
#pragma unroll
        for (int h = 0; h < G; ++h) {
            bf16x8 a[R][Q];
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int q = 0; q < Q; ++q) a[r][q] = widen<FMT, G>(st.w[r], 1.0f, h * Q + q);
#pragma unroll
            for (int c = 0; c < CT; ++c) {
                if (CT > 1 && !(cols >> c & 1)) continue;
                f32x4 d[R + 1];                              // the last one: sum x
#pragma unroll
                for (int r = 0; r <= R; ++r) d[r] = none;
#pragma unroll
                for (int q = 0; q < Q; ++q) {
                    const bf16x8 b = token_values<XT>(st.x[c], h * Q + q);
                    d[R] = mfma(ones, b, d[R]);
#pragma unroll
                    for (int r = 0; r < R; ++r) d[r] = mfma(a[r][q], b, d[r]);
                }
                settle(d);
#pragma unroll
                for (int r = 0; r < R; ++r)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int at = i * G + h;            // row i of the four, group h of the block
                        const uint32_t sw = sc[r].s[at >> 1];
                        const float s = at & 1 ? bf16_hi(sw) : bf16_lo(sw);
                        const uint32_t zw = sc[r].z[at >> 2] | 0x80808080u;      // 128 + zero
                        const float z = (float)((zw >> (8 * (at & 3))) & 0xFFu);
                        acc[r][c][i] = fmaf(s, fmaf(-z, d[R][i], d[r][i]), acc[r][c][i]);
                    }
            }
        }
    } else {
        bf16x8 a[R][4];
        uint32_t words[R];
        if constexpr (F::kMx) spread_rows<R>(st.s.w, words);
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float mx = 1.0f;
                if constexpr (F::kMx) mx = e8m0_value(words[r], F::kFour ? g : 2 * (q >> 1) + (g >> 1));
                a[r][q] = widen<FMT, G>(st.w[r], mx, q);
            }
#pragma unroll
        for (int c = 0; c < CT; ++c) {
            if (CT > 1 && !(cols >> c & 1)) continue;
            f32x4 d[R];
#pragma unroll
            for (int r = 0; r < R; ++r) d[r] = F::kMx ? acc[r][c] : none;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const bf16x8 b = token_values<XT>(st.x[c], q);
#pragma unroll
                for (int r = 0; r < R; ++r) d[r] = mfma(a[r][q], b, d[r]);
            }
            settle(d);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                if constexpr (F::kMx) {
                    acc[r][c] = d[r];
                } else {
                    const float s = __uint_as_float(st.s.w);
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[r][c][i] = fmaf(s, d[r][i], acc[r][c][i]);
                }
            }
        }
    }
}

// The same for more tiles than one asm can name: all of them are tied down before the wait and again after it, so that
// every read depends on an asm behind the wait (volatile ones keep their order; the empty ones emit nothing).
template <int R, int N>
__device__ __forceinline__ void settle_all(f32x4 (&d)[R][N]) {
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int c = 0; c < N; ++c) asm volatile("" : "+v"(d[r][c]));
    asm volatile("s_nop 15" : "+v"(d[0][0]));
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int c = 0; c < N; ++c) asm volatile("" : "+v"(d[r][c]));
}

// Tokens that a workgroup shares in LDS: piece p of token t in element 16 t + (p ^ shared_swizzle(t)).  LDS serves a
// 16 B read eight lanes at a time, four of one sixteen with four of the next (lanes 0 to 3 with 20 to 23, and so on),
// so the tokens t and t + 4 of neighbouring lane groups g, g + 1 have to differ in the low three bits: their pieces do
// for e2m1 (4 g + q), the swizzle has to for the others.
template <int FMT>
__device__ __forceinline__ int shared_swizzle(int t) { return FMT == MOE_W_E2M1_MX ? t & 11 : t & 15; }

// acc += one K block of weights in the MFMA layout times the tokens that the workgroup shares in LDS.
template <int FMT, int G, int R, int CT>
__device__ __forceinline__ void shared_product(const u32x4 (&w)[R][Fmt<FMT, G>::kLoads], const Scales<FMT, G>& s,
                                               const u32x4* xs, f32x4 (&acc)[R][CT]) {
    using F = Fmt<FMT, G>;
    const int l = lane_id(), c16 = l & 15, g = l >> 4;
    const f32x4 none = {0.f, 0.f, 0.f, 0.f};
    const auto tokens = [&](int c, int q) {
        const int piece = x_offset<FMT, G>(q, g) / 8;
        return __builtin_bit_cast(bf16x8, xs[(16 * c + c16) * 16 + (piece ^ shared_swizzle<FMT>(c16))]);
    };
    if constexpr (F::kInt4) {
        const u32x4 ones_bits = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
        const bf16x8 ones = __builtin_bit_cast(bf16x8, ones_bits);
        constexpr int Q = 4 / G;
        Scales<FMT, G> sc[R];
        spread_lanes<G, R>(s, sc);
#pragma unroll
        for (int h = 0; h < G; ++h) {
            f32x4 d[R + 1][CT];                              // the last row: sum x
#pragma unroll
            for (int r = 0; r <= R; ++r)
#pragma unroll
                for (int c = 0; c < CT; ++c) d[r][c] = none;
#pragma unroll
            for (int q = h * Q; q < (h + 1) * Q; ++q) {
                bf16x8 b[CT];
#pragma unroll
                for (int c = 0; c < CT; ++c) b[c] = tokens(c, q);
#pragma unroll
                for (int r = 0; r <= R; ++r) {
                    const bf16x8 a = r < R ? widen<FMT, G>(w[r < R ? r : 0], 1.0f, q) : ones;
#pragma unroll
                    for (int c = 0; c < CT; ++c) d[r][c] = mfma(a, b[c], d[r][c]);
                }
            }
            settle_all(d);
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int at = i * G + h;
                    const uint32_t sw = sc[r].s[at >> 1];
                    const float sv = at & 1 ? bf16_hi(sw) : bf16_lo(sw);
                    const uint32_t zw = sc[r].z[at >> 2] | 0x80808080u;          // 128 + zero
                    const float z = (float)((zw >> (8 * (at & 3))) & 0xFFu);
#pragma unroll
                    for (int c = 0; c < CT; ++c) acc[r][c][i] = fmaf(sv, fmaf(-z, d[R][c][i], d[r][c][i]), acc[r][c][i]);
                }
        }
    } else {
        uint32_t words[R];
        if constexpr (F::kMx) spread_rows<R>(s.w, words);
        f32x4 d[R][CT];
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int c = 0; c < CT; ++c) d[r][c] = F::kMx ? acc[r][c] : none;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            bf16x8 b[CT];
#pragma unroll
            for (int c = 0; c < CT; ++c) b[c] = tokens(c, q);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                float mx = 1.0f;
                if constexpr (F::kMx) mx = e8m0_value(words[r], F::kFour ? g : 2 * (q >> 1) + (g >> 1));
                const bf16x8 a = widen<FMT, G>(w[r], mx, q);
#pragma unroll
                for (int c = 0; c < CT; ++c) d[r][c] = mfma(a, b[c], d[r][c]);
            }
        }
        settle_all(d);
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int c = 0; c < CT; ++c) {
                if constexpr (F::kMx) {
                    acc[r][c] = d[r][c];
                } else {
                    const float sv = __uint_as_float(s.w);
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[r][c][i] = fmaf(sv, d[r][c][i], acc[r][c][i]);
                }
            }
    }
}

__device__ __forceinline__ void lds_barrier() {
    // orders LDS accesses only: loads stay in flight across it
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// Token rows are read through a buffer resource: a lane whose column has no token passes kNoRow, which lies past
// num_records, and reads zeros without a memory access.
constexpr uint32_t kNoRow = 0x80000000u;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t row_buffer(const void* base, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, (int)bytes, 0x00020000);
}

// row_bytes: where the row of the lane's token starts, or kNoRow.  A tile of sixteen is fetched like weights (token
// lane / 4) and turned in block_product.
template <int XT>
__device__ __forceinline__ int token_of_lane() {
    const int l = lane_id();
    return XT == 16 ? l >> 2 : (l & 15) / (16 / XT);
}

template <int FMT, int G, int XT>
__device__ __forceinline__ void load_rows(__amdgpu_buffer_rsrc_t rows, uint32_t row_bytes, int kb,
                                          u32x4 (&x)[XT / 4]) {
    constexpr int S = 16 / XT;
    const int l = lane_id(), g = l >> 4, sub = l % S;
#pragma unroll
    for (int i = 0; i < XT / 4; ++i) {
        const uint32_t at = XT == 16 ? 64 * i + 16 * (l & 3) : 2 * x_offset<FMT, G>(i * S + sub, g);
        x[i] = __builtin_amdgcn_raw_buffer_load_b128(rows, row_bytes + at, kb * (2 * kKBlock), 0);
    }
}

}  // namespace moe
