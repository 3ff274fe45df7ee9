// The inner loop shared by the few-token kernels: a wavefront multiplies tiles of 16 weight rows by up to 16 * CT
// token columns along a run of 128-element K blocks, the weights streamed from HBM once and never kept.
//
//   D[row, col] += sum_k W[row, k] * x[col, k]
//
// Matrix instruction: v_mfma_f32_16x16x32_bf16 with the weights as its A operand (lane l holds row l % 16) and the
// tokens as its B operand (column l % 16), so a lane's four results are four consecutive weight rows of one token.
// Every weight format widens to bf16 without rounding (an e4m3 or e2m1 code times a power of two; an integer
// 128 + q), so the products are those of the definition and the sums are fp32.  One token uses one column of the
// sixteen: the loop is bound by the weight stream up to 64 columns, not by the matrix cores.
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
typedef __bf16 bf16x2v __attribute__((ext_vector_type(2)));
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

template <int FMT, int G>
struct Scales {                                              // of one tile and block, as loaded
    uint32_t w;                                              // MX codes, or the fp32 scale's bits
};
template <int G>
struct Scales<MOE_W_INT4, G> {
    uint32_t s[2 * G];                                       // 4 rows x G bf16
    uint32_t z[G];                                           // 4 rows x G bytes
};

// The sixteen rows of a tile, as one lane addresses them.
template <int FMT, int G>
struct TileRows {
    const uint8_t* w;        // the lane's A row, at its 16 B
    const uint8_t* s;        // block 0's scales
    const uint8_t* z;
};

// arow: the lane's weight row (its A row); drow: the first of the four rows the lane's results belong to.
template <int FMT, int G>
__device__ __forceinline__ TileRows<FMT, G> tile_rows(const WView& v, int64_t arow, int64_t drow) {
    using F = Fmt<FMT, G>;
    const int g = lane_id() >> 4;
    TileRows<FMT, G> t;
    t.w = v.data + arow * (int64_t)v.nb * F::kRowBytes + 16 * g;
    t.z = nullptr;
    if constexpr (F::kInt4) {
        t.s = static_cast<const uint8_t*>(v.scale) + drow * 2 * G;
        if (v.zero) t.z = v.zero + drow * G;
    } else if constexpr (F::kMx) {
        t.s = static_cast<const uint8_t*>(v.scale) + arow * 4;
    } else {
        t.s = static_cast<const uint8_t*>(v.scale) + (drow / 128) * (int64_t)v.nb * 4;
    }
    return t;
}

template <int FMT, int G, int R, int CT>
struct Step {                                                // one K block in flight
    u32x4 w[R][Fmt<FMT, G>::kLoads];
    Scales<FMT, G> s[R];
    u32x4 x[CT][4];
};

template <int FMT, int G>
__device__ __forceinline__ void load_weights(const TileRows<FMT, G>& t, const WView& v, int kb,
                                             u32x4 (&w)[Fmt<FMT, G>::kLoads], Scales<FMT, G>& s) {
    using F = Fmt<FMT, G>;
    const u32x4* p = reinterpret_cast<const u32x4*>(t.w + (int64_t)kb * F::kRowBytes);
#pragma unroll
    for (int i = 0; i < F::kLoads; ++i) w[i] = __builtin_nontemporal_load(p + 4 * i);
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
        if (t.z) {
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

// Element offset, inside a block, of the eight x values that MFMA q of the lane group g multiplies.
template <int FMT, int G>
__device__ __forceinline__ int x_offset(int q, int g) {
    using F = Fmt<FMT, G>;
    if constexpr (F::kInt4) return 32 * q + 8 * g;
    if constexpr (F::kFour) return 32 * g + 8 * q;
    return 64 * (q >> 1) + 16 * g + 8 * (q & 1);
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

// Waits out the matrix pipeline before d is read.  An 8-pass MFMA's result may be read by the VALU 11 wait states
// after it; the compiler counts them within straight code, but where it moved the reading instructions behind a
// branch it left them out (seen in the listing: MFMA, s_cbranch, v_mov, v_fmac of the result, and a first component
// short of the last two MFMAs).  The asm ties the wait to the values, so no branch can come between.
template <int N>
__device__ __forceinline__ void settle(f32x4 (&d)[N]) {
    static_assert(N >= 1 && N <= 4, "tiles");
    if constexpr (N == 1) asm volatile("s_nop 15" : "+v"(d[0]));
    if constexpr (N == 2) asm volatile("s_nop 15" : "+v"(d[0]), "+v"(d[1]));
    if constexpr (N == 3) asm volatile("s_nop 15" : "+v"(d[0]), "+v"(d[1]), "+v"(d[2]));
    if constexpr (N == 4) asm volatile("s_nop 15" : "+v"(d[0]), "+v"(d[1]), "+v"(d[2]), "+v"(d[3]));
}

// acc += one K block.  cols: bit c set where column tile c has a token (uniform over the wavefront).
template <int FMT, int G, int R, int CT>
__device__ __forceinline__ void block_product(const Step<FMT, G, R, CT>& st, uint32_t cols, f32x4 (&acc)[R][CT]) {
    using F = Fmt<FMT, G>;
    const int g = lane_id() >> 4;
    const f32x4 none = {0.f, 0.f, 0.f, 0.f};
    if constexpr (F::kInt4) {
        // sum (q - z) s x = s (sum (128 + q) x - (128 + z) sum x) per scale group; sum x from an MFMA by ones
        const u32x4 ones_bits = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
        const bf16x8 ones = __builtin_bit_cast(bf16x8, ones_bits);
        constexpr int Q = 4 / G;                             // MFMAs per group
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
                    const bf16x8 b = __builtin_bit_cast(bf16x8, st.x[c][h * Q + q]);
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
                        const uint32_t sw = st.s[r].s[at >> 1];
                        const float s = at & 1 ? bf16_hi(sw) : bf16_lo(sw);
                        const float z = 128.0f + (float)((st.s[r].z[at >> 2] >> (8 * (at & 3))) & 0xFFu);
                        acc[r][c][i] = fmaf(s, fmaf(-z, d[R][i], d[r][i]), acc[r][c][i]);
                    }
            }
        }
    } else {
        bf16x8 a[R][4];
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float mx = 1.0f;
                if constexpr (F::kMx) mx = e8m0_value(st.s[r].w, F::kFour ? g : 2 * (q >> 1) + (g >> 1));
                a[r][q] = widen<FMT, G>(st.w[r], mx, q);
            }
#pragma unroll
        for (int c = 0; c < CT; ++c) {
            if (CT > 1 && !(cols >> c & 1)) continue;
            f32x4 d[R];
#pragma unroll
            for (int r = 0; r < R; ++r) d[r] = F::kMx ? acc[r][c] : none;
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int r = 0; r < R; ++r) d[r] = mfma(a[r][q], __builtin_bit_cast(bf16x8, st.x[c][q]), d[r]);
            settle(d);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                if constexpr (F::kMx) {
                    acc[r][c] = d[r];
                } else {
                    const float s = __uint_as_float(st.s[r].w);
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[r][c][i] = fmaf(s, d[r][i], acc[r][c][i]);
                }
            }
        }
    }
}

// Token rows are read through a buffer resource: a lane whose column has no token passes kNoRow, which lies past
// num_records, and reads zeros without a memory access.
constexpr uint32_t kNoRow = 0x80000000u;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t row_buffer(const void* base, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, (int)bytes, 0x00020000);
}

template <int FMT, int G>
__device__ __forceinline__ void load_rows(__amdgpu_buffer_rsrc_t rows, uint32_t row_bytes, int kb, u32x4 (&x)[4]) {
    const int g = lane_id() >> 4;
#pragma unroll
    for (int q = 0; q < 4; ++q)
        x[q] = __builtin_amdgcn_raw_buffer_load_b128(
            rows, row_bytes + 2u * (uint32_t)(x_offset<FMT, G>(q, g)), kb * (2 * kKBlock), 0);
}

}  // namespace moe
