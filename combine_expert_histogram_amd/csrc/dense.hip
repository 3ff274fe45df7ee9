// The dense layers' entry points: which kernels a product takes, the activations' gradients, and the sums over parts.
#include "dense.h"

namespace moe {

bool rows_aligned(const void* p, int64_t ld, int64_t contiguous) {
    return ((uintptr_t)p & 15) == 0 && ld % 8 == 0 && contiguous % 8 == 0;
}

// The tile and the number of parts of K, by an estimate of the time.  A round of workgroups takes the tile's own time for
// its first loads and its last stores, and a step of 64 of K so much with up to half of the places taken (one workgroup to a
// CU where there is room for two; half of the CUs, at a higher clock, with 256 x 256) and so much with more; parts of K cost a
// launch, a little a part, and a pass over their sums.  Fitted to some 2500 timings of 213 products (x w^T, dx and dw of 40
// shapes from 200 x 200 x 200 to 512 x 28672 x 4096, rows aligned and not, the weights from memory), which it meets to 13 %;
// what it takes of them is on average 0.6 % over the fastest.  Some (us; 64, 128 and 256 tiles, best parts): 1001 x 777 x 1111
// 12.7, 20.8, 20.9; 512 x 8192 x 8192 180, 95, 91; 1024 x 4096 x 7168 156, 91, 81; 1024 x 7168 x 2048 64, 34, 46; 2048 x 7168 x
// 2048 112, 61, 53; 512 x 8192 x 8192 of 256 tiles in one part and four 183, 91.
struct TileCost {
    int tile, slots;
    float once, half, full, half_anywhere, full_anywhere;    // us
};
constexpr TileCost kTileCosts[] = {
    {64, 512, 0.6f, 0.52f, 0.56f, 0.63f, 0.72f}, {128, 512, 3.5f, 0.68f, 1.0f, 0.97f, 1.4f}, {256, 256, 6.9f, 1.2f, 1.4f, 0, 0}};
constexpr float kJoin = 4.8f, kJoinPart = 0.38f, kJoinElement = 8 / 7.1e6f;    // 8 bytes, partly from the last cache

// Whether the weights are read in tiles of 16 rows, K cut among wavefronts, or as tiles of an ordinary product.  us at
// rows x n x K, 16-row tiles / square ones: aligned 17 x 8192 x 8192 31 / 38, 64 x 8192 x 8192 39 / 40, 64 x 32768 x 2048
// 37 / 38, 64 x 2048 x 8192 25 / 21; rows that start anywhere 8 x 8192 x 8192 43 / 42, 8 x 4096 x 7168 23 / 26, 1 of them
// 18 / 26, 17 x 8192 x 8192 44 / 42, 64 x 4096 x 7168 38 / 29, 8 x 32768 x 2048 58 / 38.
bool few_rows(int64_t m, int64_t n, int64_t k, bool aligned) {
    return aligned ? m <= 64 && n < (1 << 26) : m <= 16 && n < 16384 && k >= 8;}

Plan plan_product(Layout layout, int64_t m, int64_t n, int64_t k, bool aligned, int terms) {
    if (layout == kNT && few_rows(m, n, k, aligned)) return Plan{0, 1, (int)((k + kStepK - 1) / kStepK * kStepK), false};
    const uint32_t steps = (uint32_t)std::max<int64_t>((k + kStepK - 1) / kStepK, 1);     // no tokens: none for dw
    Plan best{64, 1, 0, false};
    float least = 0.0f;
    for (const TileCost& c : kTileCosts) {
        if (c.tile == 256 && !aligned) break;
        const int64_t tiles = (m + c.tile - 1) / c.tile * ((n + c.tile - 1) / c.tile);
        const float half = aligned ? c.half : c.half_anywhere, full = aligned ? c.full : c.full_anywhere;
        for (uint32_t splits = 1; splits <= std::min(16u, std::max(1u, steps / 2)); ++splits) {
            const uint32_t per = (steps + splits - 1) / splits, parts = (steps + per - 1) / per;
            const float join = parts > 1 ? kJoin + parts * (kJoinPart + kJoinElement * (float)(m * n)) : 0.0f;
            if (best.kper && join >= least) break;
            const int64_t all = tiles * parts, rounds = all / c.slots, rest = all & (c.slots - 1);
            const float us = join + (float)rounds * (c.once + per * full) +
                             (rest > c.slots / 2 ? c.once + per * full : rest ? c.once + per * half : 0.0f);
            if (best.kper && us >= least) continue;
            least = us;
            best = Plan{c.tile, (int)parts, (int)(per * kStepK), false};
        }
    }
    best.joined = best.splits > 1 || (terms == 2 && layout == kNN);
    return best;
}

int64_t plan_bytes(const Plan& p, int64_t m, int64_t n) {
    return p.joined ? (p.splits * m * n * 4 + 255) & ~int64_t(255) : 0;
}

moe_status launch_tiles(Layout layout, int dtype, bool aligned, const Plan& plan, const Product& p, const Epilogue& e,
                        float* part, hipStream_t stream) {
    if (layout == kNT) return launch_tiles_nt(dtype, aligned, plan, p, e, part, stream);
    if (layout == kNN) return launch_tiles_nn(dtype, aligned, plan, p, e, part, stream);
    return launch_tiles_tn(dtype, aligned, plan, p, e, part, stream);
}

namespace {

constexpr int kThreads = 256;

// ---------------------------------------------------------------- the parts of K summed, then the epilogue
// y = epilogue(sum over the parts), in the parts' order; eight columns of a row to a thread.  Bound by its launch, and by the
// parts' bytes where there are many (the fit's constants above).
struct JoinArgs {
    const float* part;
    int64_t step;            // floats of one part
    int64_t term;            // not 0: floats from a row of the first term to its row of the second
    int64_t items;
    int splits, n, chunks, inter;
    Epilogue e;
};

__device__ __forceinline__ void add_part(const float* p, float (&v)[8], int n) {
    if (n >= 8) {
        float f[8];
        __builtin_memcpy(f, p, 32);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += f[i];
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) v[i] += p[i];
    }
}

__device__ __forceinline__ void add_parts(const JoinArgs& t, int64_t at, float (&v)[8], int n) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.0f;
#pragma unroll 8
    for (int s = 0; s < t.splits; ++s) {
        add_part(t.part + s * t.step + at, v, n);
        if (t.term) add_part(t.part + s * t.step + t.term + at, v, n);
    }
}

template <class T>
__global__ void __launch_bounds__(kThreads) join_kernel(JoinArgs t) {
    const float unit = unit_of<T>(t.e);                      // gated ones, forward, have none
    for (int64_t item = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; item < t.items;
         item += (int64_t)gridDim.x * blockDim.x) {
        const int64_t row = t.items <= UINT32_MAX ? (uint32_t)item / (uint32_t)t.chunks : item / t.chunks;
        const int c = (int)(item - row * t.chunks) * 8;
        const int n = min(8, t.e.n - c);
        float v[8], u[8];
        add_parts(t, row * t.n + c, v, n);
        in_units<T>(v, unit);
        if (t.inter) {
            add_parts(t, row * t.n + t.inter + c, u, n);
            finish_gated<T>(t.e, row, c, v, u, n);
        } else {
            finish<T>(t.e, row, c, v, n, bias_of<T>(t.e, c, n), residual_of<T>(t.e, row, c, n));
        }
    }
}

int grid_of(int64_t items) { return (int)std::min<int64_t>((items + kThreads - 1) / kThreads, 16384); }

moe_status run_product(Layout layout, int dtype, bool aligned, const Product& p, const Epilogue& e, void* ws,
                       hipStream_t stream, int terms = 1) {
    const Plan plan = plan_product(layout, p.m, p.n, p.k, aligned, terms);
    if (plan.tile == 0) return launch_few(dtype, aligned, p, e, stream);
    float* part = static_cast<float*>(ws);
    moe_status st = launch_tiles(layout, dtype, aligned, plan, p, e, part, stream);
    if (st != MOE_OK || !plan.joined) return st;
    const bool two = terms == 2 && layout == kNN;            // the second term's rows follow the first's
    const int64_t rows = two ? p.m / 2 : p.m;
    JoinArgs t;
    t.part = part, t.step = (int64_t)p.m * p.n, t.term = two ? rows * p.n : 0;
    t.splits = plan.splits, t.n = p.n, t.inter = p.inter, t.e = e;
    t.chunks = (e.n + 7) / 8;
    t.items = (two ? e.rows : rows) * t.chunks;
    const int threads = t.items < 65536 ? MOE_WAVE : kThreads;           // few: on all of the CUs
    const dim3 grid((int)std::min<int64_t>((t.items + threads - 1) / threads, 16384));
    if (dtype == MOE_BF16) hipLaunchKernelGGL(join_kernel<__bf16>, grid, dim3(threads), 0, stream, t);
    else hipLaunchKernelGGL(join_kernel<_Float16>, grid, dim3(threads), 0, stream, t);
    return launch_status();
}

// ---------------------------------------------------------------- the activations' gradients
// What fp16 cannot hold.  The products take a computed gradient in 16 bits.  In fp16 one below 2^-14 loses bits, one below
// 2^-25 all of them, and a product of two fp16 values may be past its largest.  So fp16 gradients are scaled, all of a call's
// by one power of two that takes the largest finite one (dz: the largest dy, |act'| < 1.14) to 2^14 .. 2^15, and the
// products' sums back by its inverse: both exact.  What is left is off by its own rounding or by 2^-39 of the largest,
// whichever is more.  bf16 has fp32's range and needs none of it.
//
// The largest one: a pass of its own over what the gradients are made of, a maximum to a workgroup, which the next kernel's
// workgroups each join for themselves (maxima: the order does not matter); of [dg du]'s at most kScaledGroups, so that each
// has some work for it (16384 x 2 x 2048: 55 us, with 16384 of them 57.5).  Memory bound, kPeakAhead pieces of a thread on
// their way at a time: 16384 x 2 x 2048 50 us, 8192 x 4096 16 us; 24 x 4608 3.5 us, a launch.
constexpr int kPeakGroups = 1024, kPeakAhead = 4, kScaledGroups = 4096;
struct Peaks {
    float* most;             // [groups]; null: no scale
    float* unit;             // the inverse of the scale, for the products
    int groups;
};

__device__ __forceinline__ float group_max(float v) {
    __shared__ float lds[kThreads / MOE_WAVE];
#pragma unroll
    for (int s = MOE_WAVE / 2; s; s >>= 1) v = fmaxf(v, __shfl_xor(v, s));
    if (threadIdx.x % MOE_WAVE == 0) lds[threadIdx.x / MOE_WAVE] = v;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kThreads / MOE_WAVE; ++i) v = fmaxf(v, lds[i]);
    return v;
}

// The scale of this call's gradients, one workgroup leaving its inverse.
template <class T>
__device__ __forceinline__ float scale_of(const Peaks& p) {
    if constexpr (!std::is_same<T, _Float16>::value) return 1.0f;
    if (!p.most) return 1.0f;
    float most = 0.0f;
    for (int i = threadIdx.x; i < p.groups; i += kThreads) most = fmaxf(most, p.most[i]);
    most = group_max(most);
    const int up = most > 0.0f ? min(14 + 127 - (int)(__float_as_uint(most) >> 23), 126) : 0;
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *p.unit = __uint_as_float((uint32_t)(127 - up) << 23);
    return __uint_as_float((uint32_t)(127 + up) << 23);
}

// f(row, column, columns) of every piece of eight columns of [m, cols], each once over the grid
template <class F>
__device__ __forceinline__ void each_piece(int m, int cols, F&& f) {
    const int chunks = (cols + 7) / 8;
    const int64_t items = (int64_t)m * chunks, step = (int64_t)gridDim.x * kThreads;
    auto piece = [&](int64_t at) __attribute__((always_inline)) {
        const int64_t row = items <= UINT32_MAX ? (uint32_t)at / (uint32_t)chunks : at / chunks;
        const int c = (int)(at - row * chunks) * 8;
        f(row, c, min(8, cols - c));
    };
    int64_t item = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    for (; item + (kPeakAhead - 1) * step < items; item += kPeakAhead * step) {
#pragma unroll
        for (int a = 0; a < kPeakAhead; ++a) piece(item + a * step);
    }
    for (; item < items; item += step) piece(item);
}

__device__ __forceinline__ float peak_of(float most, const float (&d)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) most = fabsf(d[i]) < __builtin_inff() ? fmaxf(most, fabsf(d[i])) : most;
    return most;
}

// Up to kTermRows rows, what the products take of a gradient d is two terms: a 16-bit number a little nearer to zero than d,
// and what that leaves, rounded to 16 bits (rows 0 .. 63 and 64 .. 127 of the workspace, zeros behind the last token).
// Their sum is within 2^-16 of d in bf16, 2^-22 in fp16.  With one term the error of a few rows' products is off by chance
// from that of their own rounding to twice it and more (1 token, 64 x 64: 1 to 2.2 times; 64 tokens and more: 1.41).  It costs
// little: the second term are rows that the tile has anyway.  More tokens take one term, which is what their matrix
// instructions cost once.  Both terms have d's sign and neither is zero (but for d below the type's reach), so that an
// infinity in w or x comes out as one: rounded to nearest, the second term would be zero or point the other way, and the sum
// inf - inf.
__device__ __forceinline__ float nearer_to_zero(__bf16 v) {
    return (float)__builtin_bit_cast(__bf16, (uint16_t)(__builtin_bit_cast(uint16_t, v) - 1));
}
__device__ __forceinline__ float nearer_to_zero(_Float16 v) {
    return (float)__builtin_bit_cast(_Float16, (uint16_t)(__builtin_bit_cast(uint16_t, v) - 1));
}

template <class T>
__device__ __forceinline__ void store_terms(T* p, int64_t second, const float (&gradient)[8], int n, float scale) {
    float d[8], rest[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) d[i] = std::is_same<T, _Float16>::value ? gradient[i] * scale : gradient[i];
    if (second) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            rest[i] = d[i];                                  // of zeros, infinities and NaNs
            if (d[i] == 0.0f || !__builtin_isfinite(d[i])) continue;
            float first = (float)(T)d[i];
            if (fabsf(first) >= fabsf(d[i])) first = nearer_to_zero((T)first);
            if ((T)(d[i] - first) == (T)0.0f && first != 0.0f) first = nearer_to_zero((T)first);
            rest[i] = d[i] - first;
            d[i] = first;
        }
        store8(p + second, rest, n);
    }
    store8(p, d, n);
}

// d[row, :] = [dh u act'(g), dh act(g)]: read and written once, 8 columns of a row to a thread.  Memory bound: 16384 x 2 x
// 2048 bf16 51 us for 336 MB.
struct GateGradArgs {
    const void* dh;
    const void* gu;
    void* d;
    int64_t dh_ld, gu_ld, d_ld, items;
    int64_t second;          // elements to the second term, 0: one term
    int m, inter, chunks, act;
    Peaks peaks;
};

// dg and du of a piece of `n` columns from c
template <class T>
__device__ __forceinline__ void gate_grad(const GateGradArgs& t, int64_t row, int c, int n, float (&dg)[8], float (&du)[8]) {
    const T* gu = static_cast<const T*>(t.gu) + row * t.gu_ld + c;
    const auto dh = load8(static_cast<const T*>(t.dh) + row * t.dh_ld + c, n);
    const auto gv = load8(gu, n), uv = load8(gu + t.inter, n);
    float g[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) g[i] = (float)gv[i];
    activate_grad(g, du, dg, t.act);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        dg[i] *= (float)dh[i] * (float)uv[i];
        du[i] *= (float)dh[i];
    }
}

template <class T>
__global__ void __launch_bounds__(kThreads) gate_grad_kernel(GateGradArgs t) {
    const float scale = scale_of<T>(t.peaks);
    for (int64_t item = (int64_t)blockIdx.x * kThreads + threadIdx.x; item < t.items; item += (int64_t)gridDim.x * kThreads) {
        const int64_t row = item / t.chunks;
        const int c = (int)(item - row * t.chunks) * 8, n = min(8, t.inter - c);
        float dg[8], du[8];
        gate_grad<T>(t, row, c, row < t.m ? n : 0, dg, du);
        T* to = static_cast<T*>(t.d) + row * t.d_ld + c;
        store_terms(to, t.second, dg, n, scale);
        store_terms(to + t.inter, t.second, du, n, scale);
    }
}

template <class T>
__global__ void __launch_bounds__(kThreads) gate_peak_kernel(GateGradArgs t) {
    float most = 0.0f;
    each_piece(t.m, t.inter, [&](int64_t row, int c, int n) __attribute__((always_inline)) {
        float dg[8], du[8];
        gate_grad<T>(t, row, c, n, dg, du);
        most = peak_of(peak_of(most, dg), du);
    });
    most = group_max(most);
    if (threadIdx.x == 0) t.peaks.most[blockIdx.x] = most;
}

// dz = dy act'(z), kept for the products where `d` is not null, and its column sums over this workgroup's rows: a
// workgroup takes 256 columns (8 to a thread) and every eighth row of its share to one of its eight groups of threads.
// Memory bound: 8192 x 4096 bf16 43 us, 4.7 TB/s.  Few rows are bound by latency: 24 x 4608 5.5 us (64 rows to a workgroup 12).
constexpr int kColumns = 256, kRowGroups = kThreads * 8 / kColumns, kMaxRowParts = 128;

struct DzArgs {
    const void* dy;
    const void* z;           // null: no activation
    void* d;                 // null: not kept
    float* sums;             // [gridDim.y, n padded to 4], null: not wanted
    int64_t dy_ld, z_ld, d_ld, m, rows;
    int64_t second;          // elements to the second term, 0: one term
    int n, act;
    Peaks peaks;
};

template <class T>
__global__ void __launch_bounds__(kThreads) dz_peak_kernel(DzArgs t) {
    float most = 0.0f;
    each_piece((int)t.m, t.n, [&](int64_t row, int c, int n) __attribute__((always_inline)) {
        const auto dy = load8(static_cast<const T*>(t.dy) + row * t.dy_ld + c, n);
        float d[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) d[i] = (float)dy[i];
        most = peak_of(most, d);
    });
    most = group_max(most);
    if (threadIdx.x == 0) t.peaks.most[blockIdx.x] = most;
}

template <class T>
__global__ void __launch_bounds__(kThreads) dz_kernel(DzArgs t) {
    __shared__ float lds[kRowGroups][kColumns + 4];
    const float scale = scale_of<T>(t.peaks);
    const int c = blockIdx.x * kColumns + (threadIdx.x % (kColumns / 8)) * 8, group = threadIdx.x / (kColumns / 8);
    const int n = min(8, t.n - c);
    const int64_t first = blockIdx.y * t.rows, last = min(t.second ? (int64_t)kTermRows : t.m, first + t.rows);
    float sum[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) sum[i] = 0.0f;
    if (n > 0) {
        for (int64_t row = first + group; row < last; row += kRowGroups) {
            const int have = row < t.m ? n : 0;              // rows behind the last token: zeros
            const auto dy = load8(static_cast<const T*>(t.dy) + row * t.dy_ld + c, have);
            float d[8];
            if (t.z) {
                const auto zv = load8(static_cast<const T*>(t.z) + row * t.z_ld + c, have);
                float z[8], a[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) z[i] = (float)zv[i];
                activate_grad(z, a, d, t.act);
#pragma unroll
                for (int i = 0; i < 8; ++i) d[i] *= (float)dy[i];
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) d[i] = (float)dy[i];
            }
            if (t.d) store_terms(static_cast<T*>(t.d) + row * t.d_ld + c, t.second, d, n, scale);
#pragma unroll
            for (int i = 0; i < 8; ++i) sum[i] += d[i];
        }
    }
    if (!t.sums) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) lds[group][(threadIdx.x % (kColumns / 8)) * 8 + i] = sum[i];
    __syncthreads();
    const int col = blockIdx.x * kColumns + threadIdx.x;
    if (col >= t.n) return;
    float s = 0.0f;
#pragma unroll
    for (int g = 0; g < kRowGroups; ++g) s += lds[g][threadIdx.x];
    t.sums[(int64_t)blockIdx.y * pad4(t.n) + col] = s;
}

// rows of sixteen to a workgroup, two to a thread, as long as that is not too many rows of sums
int64_t row_parts(int64_t m) { return std::min<int64_t>((std::max<int64_t>(m, kTermRows) + 15) / 16, kMaxRowParts); }

int peak_groups(int64_t m, int64_t cols) {
    return (int)std::min<int64_t>((m * ((cols + 7) / 8) + kThreads - 1) / kThreads, kPeakGroups);
}

template <class T>
moe_status launch_dz(DzArgs t, void* dbias, hipStream_t stream) {
    const int64_t parts = row_parts(t.m);
    t.rows = (std::max<int64_t>(t.m, kTermRows) + parts - 1) / parts;
    if (t.peaks.most) {
        t.peaks.groups = peak_groups(t.m, t.n);
        hipLaunchKernelGGL(dz_peak_kernel<T>, dim3(t.peaks.groups), dim3(kThreads), 0, stream, t);
    }
    hipLaunchKernelGGL(dz_kernel<T>, dim3((t.n + kColumns - 1) / kColumns, (int)parts), dim3(kThreads), 0, stream, t);
    moe_status st = launch_status();
    if (st != MOE_OK || !dbias) return st;
    return join_columns<T>(t.sums, (int)parts, pad4(t.n), pad4(t.n), t.n, dbias, nullptr, stream);
}

template <class T>
__global__ void __launch_bounds__(kThreads) zero_rows_kernel(T* p, int64_t ld, int cols, int64_t items) {
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < items; i += (int64_t)gridDim.x * kThreads)
        p[i / cols * ld + i % cols] = (T)0.0f;
}

moe_status zero_rows(void* p, int64_t ld, int64_t rows, int cols, hipStream_t stream) {
    const int64_t items = rows * cols;
    hipLaunchKernelGGL(zero_rows_kernel<_Float16>, dim3(grid_of(items)), dim3(kThreads), 0, stream,
                       static_cast<_Float16*>(p), ld, cols, items);        // +0 in either type
    return launch_status();
}

// ---------------------------------------------------------------- checks and sizes
int64_t pad(int64_t bytes) { return (bytes + 255) & ~int64_t(255); }
int64_t pad8(int64_t n) { return (n + 7) & ~int64_t(7); }

bool bad_dtype(int dtype) { return dtype != MOE_BF16 && dtype != MOE_FP16; }
bool bad_act(int act) { return act < MOE_ACT_NONE || act > MOE_ACT_GELU_TANH; }
bool misplaced(const void* p, size_t to) { return ((uintptr_t)p & (to - 1)) != 0; }
// a matrix of rows of `cols` elements
bool bad_rows(const void* p, int64_t ld, int64_t cols) { return !p || misplaced(p, 2) || ld < cols; }
constexpr int64_t kMaxLd = 1 << 22, kMaxElements = (int64_t)1 << 40;

moe_status check_sizes(int64_t m, int64_t n, int64_t k) {
    if (m < 0 || n < 1 || k < 1) return MOE_ERR_INVALID_ARG;
    if (m * n >= kMaxElements || m * k >= kMaxElements || n * k >= kMaxElements ||
        std::max({m, n, k}) >= (1 << 30))
        return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

int64_t product_bytes(Layout layout, int64_t m, int64_t n, int64_t k, int terms = 1) {
    return std::max(plan_bytes(plan_product(layout, m, n, k, true, terms), m, n),
                    plan_bytes(plan_product(layout, m, n, k, false, terms), m, n));
}

// the backward passes' workspace: dz (or [dg du]) where it is computed, in one or two terms, the maxima for its scale, the
// bias's column sums, and the products' parts
struct Backward {
    int terms;
    int64_t peaks, sums, parts, bytes;
};
Backward backward_of(int64_t m, int64_t n, int64_t k, bool computed) {
    Backward b;
    b.terms = computed && m <= kTermRows ? 2 : 1;
    const int64_t rows = b.terms == 2 ? 2 * kTermRows : m;
    b.peaks = computed ? pad(rows * pad8(n) * 2) : 0;
    b.sums = b.peaks + (computed ? pad((kPeakGroups + 1) * 4) : 0);
    b.parts = b.sums + pad(row_parts(m) * pad4(n) * 4);
    b.bytes = b.parts + std::max(product_bytes(kNN, rows, k, n, b.terms), product_bytes(kTN, n, k, rows, b.terms));
    return b;
}

Peaks peaks_at(const Backward& b, int dtype, uint8_t* ws) {
    if (dtype != MOE_FP16) return Peaks{nullptr, nullptr, 0};
    float* most = reinterpret_cast<float*>(ws + b.peaks);
    return Peaks{most, most + kPeakGroups, 0};
}

// dx = d w and dw = d^T x, either of them left out where it is null.  Two terms: dx's are rows of one product, summed as
// its parts are; dw's are two steps of K, of which x's rows are read in each.
moe_status run_backward(const Backward& b, int64_t m, int64_t n, int64_t k, int dtype, const void* d, int64_t d_ld,
                        const void* x, int64_t x_ld, const void* w, int64_t w_ld, void* dx, int64_t dx_ld, void* dw,
                        int64_t dw_ld, const float* unit, void* ws, hipStream_t stream) {
    moe_status st = MOE_OK;
    const int rows = b.terms == 2 ? 2 * kTermRows : (int)m;
    const Product p_dx{d, w, d_ld, w_ld, rows, (int)k, (int)n, 0, 0};
    const Epilogue e_dx{nullptr, nullptr, nullptr, dx, 0, 0, dx_ld, (int)k, MOE_ACT_NONE, (int)m, unit};
    const bool fast_dx = dx && rows_aligned(d, d_ld, n) && rows_aligned(w, w_ld, k);
    const Product p_dw{d, x, d_ld, x_ld, (int)n, (int)k, rows, 0, b.terms == 2 ? (int)m : 0};
    const Epilogue e_dw{nullptr, nullptr, nullptr, dw, 0, 0, dw_ld, (int)k, MOE_ACT_NONE, (int)n, unit};
    const bool fast_dw = dw && rows_aligned(d, d_ld, n) && rows_aligned(x, x_ld, k);
    if (fast_dx && fast_dw) {
        const Plan plan_dx = plan_product(kNN, rows, k, n, true, b.terms), plan_dw = plan_product(kTN, n, k, rows, true, b.terms);
        if (plan_dx.tile == 256 && plan_dw.tile == 256 && !plan_dx.joined && !plan_dw.joined)
            return launch_pair(dtype, plan_dw, p_dw, e_dw, plan_dx, p_dx, e_dx, stream);
    }
    if (dx) st = run_product(kNN, dtype, fast_dx, p_dx, e_dx, ws, stream, b.terms);
    if (dw && st == MOE_OK) st = run_product(kTN, dtype, fast_dw, p_dw, e_dw, ws, stream, b.terms);
    return st;
}

bool wide(int64_t a, int64_t b, int64_t c, int64_t d, int64_t e) {
    return std::max({a, b, c, d, e}) >= kMaxLd;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status moe_linear_workspace(int32_t m, int32_t n, int32_t k, size_t* bytes) {
    const moe_status st = check_sizes(m, n, k);
    if (st != MOE_OK) return st;
    if (!bytes) return MOE_ERR_INVALID_ARG;
    *bytes = (size_t)product_bytes(kNT, m, n, k);
    return MOE_OK;
}

extern "C" moe_status moe_linear(int32_t m, int32_t n, int32_t k, int32_t dtype, const void* x, int64_t x_stride,
                                 const void* w, int64_t w_stride, const void* bias, int32_t act, const void* residual,
                                 int64_t residual_stride, void* z, int64_t z_stride, void* y, int64_t y_stride, void* ws,
                                 size_t ws_bytes, void* hip_stream) {
    const moe_status st = check_sizes(m, n, k);
    if (st != MOE_OK) return st;
    if (bad_dtype(dtype) || bad_act(act)) return MOE_ERR_INVALID_ARG;
    if (m == 0) return MOE_OK;
    if (bad_rows(x, x_stride, k) || bad_rows(w, w_stride, k) || bad_rows(y, y_stride, n) || misplaced(bias, 2) ||
        (residual && bad_rows(residual, residual_stride, n)) || (z && bad_rows(z, z_stride, n)))
        return MOE_ERR_INVALID_ARG;
    if (wide(x_stride, w_stride, y_stride, residual ? residual_stride : 0, z ? z_stride : 0)) return MOE_ERR_UNSUPPORTED;
    const int64_t need = product_bytes(kNT, m, n, k);
    if (need && (!ws || ws_bytes < (size_t)need)) return MOE_ERR_WORKSPACE;
    if (need && misplaced(ws, 16)) return MOE_ERR_INVALID_ARG;
    const Product p{x, w, x_stride, w_stride, m, n, k, 0, 0};
    const Epilogue e{bias, residual, z, y, residual_stride, z_stride, y_stride, n, act, m};
    return run_product(kNT, dtype, rows_aligned(x, x_stride, k) && rows_aligned(w, w_stride, k), p, e, ws,
                       reinterpret_cast<hipStream_t>(hip_stream));
}

extern "C" moe_status moe_linear_backward_workspace(int32_t m, int32_t n, int32_t k, int32_t act, size_t* bytes) {
    const moe_status st = check_sizes(m, n, k);
    if (st != MOE_OK) return st;
    if (!bytes || bad_act(act)) return MOE_ERR_INVALID_ARG;
    *bytes = (size_t)backward_of(m, n, k, act != MOE_ACT_NONE).bytes;
    return MOE_OK;
}

extern "C" moe_status moe_linear_backward(int32_t m, int32_t n, int32_t k, int32_t dtype, const void* dy, int64_t dy_stride,
                                          const void* x, int64_t x_stride, const void* w, int64_t w_stride, int32_t act,
                                          const void* z, int64_t z_stride, void* dx, int64_t dx_stride, void* dw,
                                          int64_t dw_stride, void* dbias, void* ws, size_t ws_bytes, void* hip_stream) {
    moe_status st = check_sizes(m, n, k);
    if (st != MOE_OK) return st;
    if (bad_dtype(dtype) || bad_act(act)) return MOE_ERR_INVALID_ARG;
    const bool keeps = act != MOE_ACT_NONE;
    const hipStream_t stream = reinterpret_cast<hipStream_t>(hip_stream);
    if ((dw && bad_rows(dw, dw_stride, k)) || misplaced(dbias, 2)) return MOE_ERR_INVALID_ARG;
    if (m == 0) {
        if (dw) st = zero_rows(dw, dw_stride, n, k, stream);
        if (dbias && st == MOE_OK) st = zero_rows(dbias, n, 1, n, stream);
        return st;
    }
    if (bad_rows(dy, dy_stride, n) || (keeps && bad_rows(z, z_stride, n)) || (dw && bad_rows(x, x_stride, k)) ||
        (dx && (bad_rows(w, w_stride, k) || bad_rows(dx, dx_stride, k))))
        return MOE_ERR_INVALID_ARG;
    if (wide(dy_stride, dw ? std::max(x_stride, dw_stride) : 0, dx ? std::max(w_stride, dx_stride) : 0,
             keeps ? std::max(z_stride, pad8(n)) : 0, 0))
        return MOE_ERR_UNSUPPORTED;
    if (!dx && !dw && !dbias) return MOE_OK;
    const Backward b = backward_of(m, n, k, keeps);
    if (!ws || ws_bytes < (size_t)b.bytes) return MOE_ERR_WORKSPACE;
    if (misplaced(ws, 16)) return MOE_ERR_INVALID_ARG;
    uint8_t* at = static_cast<uint8_t*>(ws);
    const void* d = dy;
    int64_t d_ld = dy_stride;
    const bool kept = keeps && (dx || dw);
    const Peaks peaks = kept ? peaks_at(b, dtype, at) : Peaks{nullptr, nullptr, 0};
    if (keeps || dbias) {
        const DzArgs t{dy, keeps ? z : nullptr, kept ? at : nullptr, dbias ? reinterpret_cast<float*>(at + b.sums) : nullptr,
                       dy_stride, z_stride, pad8(n), m, 0, kept && b.terms == 2 ? kTermRows * pad8(n) : 0, n, act, peaks};
        st = dtype == MOE_BF16 ? launch_dz<__bf16>(t, dbias, stream) : launch_dz<_Float16>(t, dbias, stream);
        if (st != MOE_OK) return st;
        if (kept) d = at, d_ld = pad8(n);
    }
    return run_backward(b, m, n, k, dtype, d, d_ld, x, x_stride, w, w_stride, dx, dx_stride, dw, dw_stride, peaks.unit,
                        at + b.parts, stream);
}

extern "C" moe_status moe_gated_linear_workspace(int32_t m, int32_t inter, int32_t hidden, size_t* bytes) {
    const moe_status st = check_sizes(m, inter < 1 ? inter : 2 * (int64_t)inter, hidden);
    if (st != MOE_OK) return st;
    if (!bytes) return MOE_ERR_INVALID_ARG;
    *bytes = (size_t)product_bytes(kNT, m, 2 * (int64_t)inter, hidden);
    return MOE_OK;
}

extern "C" moe_status moe_gated_linear(int32_t m, int32_t inter, int32_t hidden, int32_t dtype, const void* x,
                                       int64_t x_stride, const void* w, int64_t w_stride, int32_t act, void* gu,
                                       int64_t gu_stride, void* h, int64_t h_stride, void* ws, size_t ws_bytes,
                                       void* hip_stream) {
    const int64_t n = 2 * (int64_t)inter;
    const moe_status st = check_sizes(m, n, hidden);
    if (st != MOE_OK) return st;
    if (bad_dtype(dtype) || bad_act(act)) return MOE_ERR_INVALID_ARG;
    if (m == 0) return MOE_OK;
    if (bad_rows(x, x_stride, hidden) || bad_rows(w, w_stride, hidden) || bad_rows(h, h_stride, inter) ||
        (gu && bad_rows(gu, gu_stride, n)))
        return MOE_ERR_INVALID_ARG;
    if (wide(x_stride, w_stride, h_stride, gu ? gu_stride : 0, 0)) return MOE_ERR_UNSUPPORTED;
    const int64_t need = product_bytes(kNT, m, n, hidden);
    if (need && (!ws || ws_bytes < (size_t)need)) return MOE_ERR_WORKSPACE;
    if (need && misplaced(ws, 16)) return MOE_ERR_INVALID_ARG;
    const Product p{x, w, x_stride, w_stride, m, (int)n, hidden, inter, 0};
    const Epilogue e{nullptr, nullptr, gu, h, 0, gu_stride, h_stride, inter, act, m};
    return run_product(kNT, dtype, rows_aligned(x, x_stride, hidden) && rows_aligned(w, w_stride, hidden), p, e, ws,
                       reinterpret_cast<hipStream_t>(hip_stream));
}

extern "C" moe_status moe_gated_linear_backward_workspace(int32_t m, int32_t inter, int32_t hidden, size_t* bytes) {
    const moe_status st = check_sizes(m, inter < 1 ? inter : 2 * (int64_t)inter, hidden);
    if (st != MOE_OK) return st;
    if (!bytes) return MOE_ERR_INVALID_ARG;
    *bytes = (size_t)backward_of(m, 2 * (int64_t)inter, hidden, true).bytes;
    return MOE_OK;
}

extern "C" moe_status moe_gated_linear_backward(int32_t m, int32_t inter, int32_t hidden, int32_t dtype, const void* dh,
                                                int64_t dh_stride, const void* gu, int64_t gu_stride, const void* x,
                                                int64_t x_stride, const void* w, int64_t w_stride, int32_t act, void* dx,
                                                int64_t dx_stride, void* dw, int64_t dw_stride, void* ws, size_t ws_bytes,
                                                void* hip_stream) {
    const int64_t n = 2 * (int64_t)inter;
    moe_status st = check_sizes(m, n, hidden);
    if (st != MOE_OK) return st;
    if (bad_dtype(dtype) || bad_act(act)) return MOE_ERR_INVALID_ARG;
    const hipStream_t stream = reinterpret_cast<hipStream_t>(hip_stream);
    if (dw && bad_rows(dw, dw_stride, hidden)) return MOE_ERR_INVALID_ARG;
    if (m == 0) return dw ? zero_rows(dw, dw_stride, n, hidden, stream) : MOE_OK;
    if (bad_rows(dh, dh_stride, inter) || bad_rows(gu, gu_stride, n) || (dw && bad_rows(x, x_stride, hidden)) ||
        (dx && (bad_rows(w, w_stride, hidden) || bad_rows(dx, dx_stride, hidden))))
        return MOE_ERR_INVALID_ARG;
    if (wide(dh_stride, gu_stride, dw ? std::max(x_stride, dw_stride) : 0, dx ? std::max(w_stride, dx_stride) : 0, pad8(n)))
        return MOE_ERR_UNSUPPORTED;
    if (!dx && !dw) return MOE_OK;
    const Backward b = backward_of(m, n, hidden, true);
    if (!ws || ws_bytes < (size_t)b.bytes) return MOE_ERR_WORKSPACE;
    if (misplaced(ws, 16)) return MOE_ERR_INVALID_ARG;
    uint8_t* at = static_cast<uint8_t*>(ws);
    const bool two = b.terms == 2;
    GateGradArgs t{dh, gu, at, dh_stride, gu_stride, pad8(n), 0, two ? kTermRows * pad8(n) : 0, m, inter, (inter + 7) / 8, act,
                   peaks_at(b, dtype, at)};
    t.items = (int64_t)(two ? kTermRows : m) * t.chunks;
    if (dtype == MOE_BF16) {
        hipLaunchKernelGGL(gate_grad_kernel<__bf16>, dim3(grid_of(t.items)), dim3(kThreads), 0, stream, t);
    } else {
        t.peaks.groups = peak_groups(t.m, t.inter);
        hipLaunchKernelGGL(gate_peak_kernel<_Float16>, dim3(t.peaks.groups), dim3(kThreads), 0, stream, t);
        hipLaunchKernelGGL(gate_grad_kernel<_Float16>, dim3(std::min(grid_of(t.items), kScaledGroups)), dim3(kThreads), 0, stream, t);
    }
    if ((st = launch_status()) != MOE_OK) return st;
    return run_backward(b, m, n, hidden, dtype, at, pad8(n), x, x_stride, w, w_stride, dx, dx_stride, dw, dw_stride,
                        t.peaks.unit, at + b.parts, stream);
}
