// Layer norm, forward and backward.
//
//   forward   mean = sum x / H;  rstd = 1 / sqrt(sum (x - mean)^2 / H + eps);  y = (x - mean) rstd w + b
//   backward  n = (x - mean) rstd;  g = dy w;  dx = rstd (g - sum g / H - n sum(g n) / H);  dw = sum_rows dy n;
//             db = sum_rows dy
//
// Memory bound: a row is read once into registers, by one wavefront (short rows) or a workgroup, the variance is summed
// from the centred values there, and the backward pass's two row sums are taken together.  The columns' sums dw and db
// stay in the registers of the threads that hold those columns, over all rows of a workgroup; each workgroup leaves one
// row of partial sums, which a second launch adds up in a fixed order.  Rows longer than the registers hold are read
// again for each pass (from the caches, mostly).
//
// Measured: 16384 x 7168 bf16 forward 91 us, 5.2 TB/s (a large copy reaches 5.1); backward with weights in fp32 142 us, 5.0
// TB/s, and 6.4 us for the columns' join of 512 rows of partial sums; 777 x 1111 fp32 backward 7.4 and 4.1 us; a single row
// of 7168 4.2 us, a launch and one way to memory and back.
#include "dense.h"

namespace moe {
namespace {

// eight consecutive values as floats; those past n are zeros
template <class T>
__device__ __forceinline__ void loadf(const T* p, int n, float (&f)[8]) {
    if constexpr (sizeof(T) == 2) {
        const auto v = load8(p, n);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = (float)v[i];
    } else if (n >= 8) {
        __builtin_memcpy(f, p, 32);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = i < n ? p[i] : 0.0f;
    }
}

// the same, kept as they lie in memory
template <class T>
struct Raw {
    typename Vec<T>::x8 v;
    __device__ __forceinline__ void load(const T* p, int n) { v = load8(p, n); }
    __device__ __forceinline__ void floats(float (&f)[8]) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = (float)v[i];
    }
};
template <>
struct Raw<float> {
    float v[8];
    __device__ __forceinline__ void load(const float* p, int n) { loadf(p, n, v); }
    __device__ __forceinline__ void floats(float (&f)[8]) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = v[i];
    }
};

template <class T>
__device__ __forceinline__ void storef(T* p, const float (&f)[8], int n) {
    if constexpr (sizeof(T) == 2) {
        store8(p, f, n);
    } else if (n >= 8) {
        __builtin_memcpy(p, f, 32);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) p[i] = f[i];
    }
}

template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) {
    return v + __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v), CTRL, 0xF, 0xF, false));
}

// the sum over a wavefront, in every lane: pairs, quads, eights and sixteens by DPP, then the four sixteens
__device__ __forceinline__ float wave_sum(float v) {
    v = dpp_add<0xB1>(v);                                    // quad_perm [1,0,3,2]
    v = dpp_add<0x4E>(v);                                    // quad_perm [2,3,0,1]
    v = dpp_add<0x141>(v);                                   // row_half_mirror
    v = dpp_add<0x140>(v);                                   // row_mirror
    const int b = __float_as_int(v);
    return (__int_as_float(__builtin_amdgcn_readlane(b, 0)) + __int_as_float(__builtin_amdgcn_readlane(b, 16))) +
           (__int_as_float(__builtin_amdgcn_readlane(b, 32)) + __int_as_float(__builtin_amdgcn_readlane(b, 48)));
}

// the sum over the W wavefronts that hold a row; lds: W floats, another W for the next call
template <int W>
__device__ __forceinline__ float row_sum(float v, float* lds) {
    v = wave_sum(v);
    if constexpr (W > 1) {
        if (threadIdx.x % MOE_WAVE == 0) lds[threadIdx.x / MOE_WAVE] = v;
        __syncthreads();
        v = 0.0f;
#pragma unroll
        for (int i = 0; i < W; ++i) v += lds[i];
    }
    return v;
}

struct NormArgs {
    const void* x;
    const void* w;
    const void* b;
    void* y;
    float* mean;
    float* rstd;
    int64_t x_ld, y_ld;
    int rows, cols;
    float eps;
};

// W wavefronts to a row; V pieces of eight columns to a thread, piece v of thread i at column 8 (64 W v + i).  A row to a
// team: with rows in a loop, 16384 x 7168 took 98 us and not 91 (fewer loads in flight between rows).
template <class T, class P, int W, int V>
__global__ void __launch_bounds__(W == 1 ? 256 : W * MOE_WAVE) norm_kernel(NormArgs t) {
    constexpr int kTeam = W * MOE_WAVE, kTeams = W == 1 ? 4 : 1;
    __shared__ float lds[2][W];
    const int i = W == 1 ? threadIdx.x % MOE_WAVE : threadIdx.x;
    const int64_t row = (int64_t)blockIdx.x * kTeams + (W == 1 ? threadIdx.x / MOE_WAVE : 0);
    if (row >= t.rows) return;                               // whole wavefronts, where no barrier follows
    const T* x = static_cast<const T*>(t.x) + row * t.x_ld;
    float f[V][8];
    float sum = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = 8 * (kTeam * v + i);
        loadf(x + c, t.cols - c, f[v]);
    }
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
        for (int e = 0; e < 8; ++e) sum += f[v][e];
    const float mean = row_sum<W>(sum, lds[0]) / (float)t.cols;
    float sq = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int n = t.cols - 8 * (kTeam * v + i);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            f[v][e] = e < n ? f[v][e] - mean : 0.0f;
            sq = fmaf(f[v][e], f[v][e], sq);
        }
    }
    const float rstd = 1.0f / sqrtf(row_sum<W>(sq, lds[1]) / (float)t.cols + t.eps);
    T* y = static_cast<T*>(t.y) + row * t.y_ld;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = 8 * (kTeam * v + i), n = t.cols - c;
        if (n <= 0) continue;
        float w[8], b[8];
        if (t.w) loadf(static_cast<const P*>(t.w) + c, n, w);
        if (t.b) loadf(static_cast<const P*>(t.b) + c, n, b);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[v][e] = fmaf(f[v][e] * rstd, t.w ? w[e] : 1.0f, t.b ? b[e] : 0.0f);
        storef(y + c, f[v], n);
    }
    if (i == 0) {
        if (t.mean) t.mean[row] = mean;
        if (t.rstd) t.rstd[row] = rstd;
    }
}

// rows of any length, read three times
template <class T, class P>
__global__ void __launch_bounds__(1024) norm_long_kernel(NormArgs t) {
    __shared__ float lds[2][16];
    for (int64_t row = blockIdx.x; row < t.rows; row += gridDim.x) {
        const T* x = static_cast<const T*>(t.x) + row * t.x_ld;
        float sum = 0.0f, f[8];
        for (int c = 8 * threadIdx.x; c < t.cols; c += 8192) {
            loadf(x + c, t.cols - c, f);
#pragma unroll
            for (int e = 0; e < 8; ++e) sum += f[e];
        }
        const float mean = row_sum<16>(sum, lds[0]) / (float)t.cols;
        float sq = 0.0f;
        for (int c = 8 * threadIdx.x; c < t.cols; c += 8192) {
            const int n = t.cols - c;
            loadf(x + c, n, f);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float d = e < n ? f[e] - mean : 0.0f;
                sq = fmaf(d, d, sq);
            }
        }
        const float rstd = 1.0f / sqrtf(row_sum<16>(sq, lds[1]) / (float)t.cols + t.eps);
        T* y = static_cast<T*>(t.y) + row * t.y_ld;
        for (int c = 8 * threadIdx.x; c < t.cols; c += 8192) {
            const int n = t.cols - c;
            float w[8], b[8];
            loadf(x + c, n, f);
            if (t.w) loadf(static_cast<const P*>(t.w) + c, n, w);
            if (t.b) loadf(static_cast<const P*>(t.b) + c, n, b);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = fmaf((f[e] - mean) * rstd, t.w ? w[e] : 1.0f, t.b ? b[e] : 0.0f);
            storef(y + c, f, n);
        }
        if (threadIdx.x == 0) {
            if (t.mean) t.mean[row] = mean;
            if (t.rstd) t.rstd[row] = rstd;
        }
    }
}

struct NormGradArgs {
    const void* dy;
    const void* x;
    const void* w;
    const float* mean;
    const float* rstd;
    void* dx;                // null: not wanted
    float* sums;             // [gridDim.x, 2, cols padded to 4] of dw and db, null: not wanted
    int64_t dy_ld, x_ld, dx_ld;
    int rows, cols;
};

// A workgroup (W > 1) or a wavefront (W = 1, four to a workgroup) takes every gridDim-th row.  16-bit rows: the next row is
// on its way while a row is worked on, and the weights wait in LDS (asked for again with each row, they would queue behind
// the next row's loads: the row ahead without the weights in LDS was slower than neither).  Both, and the columns' sums joined
// by sixteen teams, took 16384 x 7168 bf16 from 197 us to 147.
template <class T, class P, int W, int V>
__global__ void __launch_bounds__(W == 1 ? 256 : W * MOE_WAVE) norm_grad_kernel(NormGradArgs t) {
    constexpr int kTeam = W * MOE_WAVE, kTeams = W == 1 ? 4 : 1;
    constexpr bool kAhead = sizeof(T) == 2;
    __shared__ float lds[2][2][W];
    __shared__ f32x4 weight[V * kTeam][2];
    const int i = W == 1 ? threadIdx.x % MOE_WAVE : threadIdx.x;
    const int team = W == 1 ? threadIdx.x / MOE_WAVE : 0;
    for (int k = threadIdx.x; k < V * kTeam; k += kTeam * kTeams) {
        float w[8];
        loadf(static_cast<const P*>(t.w) + 8 * k, t.w ? t.cols - 8 * k : 0, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) weight[k][e / 4][e % 4] = t.w ? w[e] : 1.0f;
    }
    __syncthreads();
    float dw[V][8], db[V][8];
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[v][e] = db[v][e] = 0.0f;
    Raw<T> xr[V], dyr[V];
    float next_mean = 0.0f, next_rstd = 0.0f;
    auto fetch = [&](int64_t row) __attribute__((always_inline)) {
        const T* x = static_cast<const T*>(t.x) + row * t.x_ld;
        const T* dy = static_cast<const T*>(t.dy) + row * t.dy_ld;
        next_mean = t.mean[row], next_rstd = t.rstd[row];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = 8 * (kTeam * v + i);
            xr[v].load(x + c, t.cols - c);
            dyr[v].load(dy + c, t.cols - c);
        }
    };
    int turn = 0;
    const int64_t step = gridDim.x * kTeams;
    int64_t row = blockIdx.x * kTeams + team;
    if (kAhead && row < t.rows) fetch(row);
    for (; row < t.rows; row += step, turn ^= 1) {
        if (!kAhead) fetch(row);
        const float mean = next_mean, rstd = next_rstd;
        float f[V][8], g[V][8];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            xr[v].floats(f[v]);
            dyr[v].floats(g[v]);
        }
        if (kAhead && row + step < t.rows) fetch(row + step);
        float sg = 0.0f, sgn = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int n = t.cols - 8 * (kTeam * v + i);
            const f32x4 w[2] = {weight[kTeam * v + i][0], weight[kTeam * v + i][1]};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                f[v][e] = e < n ? (f[v][e] - mean) * rstd : 0.0f;
                dw[v][e] = fmaf(g[v][e], f[v][e], dw[v][e]);
                db[v][e] += g[v][e];
                g[v][e] *= w[e / 4][e % 4];
                sg += g[v][e];
                sgn = fmaf(g[v][e], f[v][e], sgn);
            }
        }
        if (t.dx) {
            // two buffers: a row's sums are read while the next row's are written
            sg = wave_sum(sg), sgn = wave_sum(sgn);
            if constexpr (W > 1) {
                if (threadIdx.x % MOE_WAVE == 0) {
                    lds[turn][0][threadIdx.x / MOE_WAVE] = sg;
                    lds[turn][1][threadIdx.x / MOE_WAVE] = sgn;
                }
                __syncthreads();
                sg = sgn = 0.0f;
#pragma unroll
                for (int k = 0; k < W; ++k) sg += lds[turn][0][k], sgn += lds[turn][1][k];
            }
            sg /= (float)t.cols, sgn /= (float)t.cols;
            T* dx = static_cast<T*>(t.dx) + row * t.dx_ld;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int c = 8 * (kTeam * v + i);
#pragma unroll
                for (int e = 0; e < 8; ++e) g[v][e] = rstd * (g[v][e] - sg - f[v][e] * sgn);
                if (c < t.cols) storef(dx + c, g[v], t.cols - c);
            }
        }
    }
    if (!t.sums) return;
    if constexpr (W == 1) {
        // the four wavefronts' sums together, in order
        __shared__ float all[2][8 * kTeam * V];
        for (int k = 0; k < kTeams; ++k) {
            if (team == k) {
#pragma unroll
                for (int v = 0; v < V; ++v)
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int c = 8 * (kTeam * v + i) + e;
                        all[0][c] = k ? all[0][c] + dw[v][e] : dw[v][e];
                        all[1][c] = k ? all[1][c] + db[v][e] : db[v][e];
                    }
            }
            __syncthreads();
        }
        for (int c = threadIdx.x; c < t.cols; c += 256) {
            t.sums[blockIdx.x * 2 * pad4(t.cols) + c] = all[0][c];
            t.sums[(blockIdx.x * 2 + 1) * pad4(t.cols) + c] = all[1][c];
        }
    } else {
        float* to = t.sums + blockIdx.x * 2 * pad4(t.cols);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = 8 * (kTeam * v + i);
            if (c >= t.cols) continue;
            storef(to + c, dw[v], t.cols - c);
            storef(to + pad4(t.cols) + c, db[v], t.cols - c);
        }
    }
}

// dx of rows of any length, read twice; a workgroup of sixteen wavefronts to a row
template <class T, class P>
__global__ void __launch_bounds__(1024) norm_grad_long_kernel(NormGradArgs t) {
    __shared__ float lds[2][16];
    for (int64_t row = blockIdx.x; row < t.rows; row += gridDim.x) {
        const T* x = static_cast<const T*>(t.x) + row * t.x_ld;
        const T* dy = static_cast<const T*>(t.dy) + row * t.dy_ld;
        const float mean = t.mean[row], rstd = t.rstd[row];
        float f[8], g[8], w[8], sg = 0.0f, sgn = 0.0f;
        auto load = [&](int c) __attribute__((always_inline)) {
            const int n = t.cols - c;
            loadf(x + c, n, f);
            loadf(dy + c, n, g);
            if (t.w) loadf(static_cast<const P*>(t.w) + c, n, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                f[e] = e < n ? (f[e] - mean) * rstd : 0.0f;
                if (t.w) g[e] *= w[e];
            }
        };
        for (int c = 8 * threadIdx.x; c < t.cols; c += 8192) {
            load(c);
#pragma unroll
            for (int e = 0; e < 8; ++e) sg += g[e], sgn = fmaf(g[e], f[e], sgn);
        }
        sg = row_sum<16>(sg, lds[0]) / (float)t.cols;
        sgn = row_sum<16>(sgn, lds[1]) / (float)t.cols;
        T* dx = static_cast<T*>(t.dx) + row * t.dx_ld;
        for (int c = 8 * threadIdx.x; c < t.cols; c += 8192) {
            load(c);
#pragma unroll
            for (int e = 0; e < 8; ++e) g[e] = rstd * (g[e] - sg - f[e] * sgn);
            storef(dx + c, g, t.cols - c);
        }
    }
}

// The columns' sums of long rows: 2048 columns to a workgroup, every gridDim.y-th row.
template <class T>
__global__ void __launch_bounds__(256) norm_columns_kernel(NormGradArgs t) {
    const int c = 8 * (blockIdx.x * 256 + threadIdx.x), n = t.cols - c;
    if (n <= 0) return;
    float dw[8], db[8], f[8], g[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[e] = db[e] = 0.0f;
    for (int64_t row = blockIdx.y; row < t.rows; row += gridDim.y) {
        const float mean = t.mean[row], rstd = t.rstd[row];
        loadf(static_cast<const T*>(t.x) + row * t.x_ld + c, n, f);
        loadf(static_cast<const T*>(t.dy) + row * t.dy_ld + c, n, g);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            dw[e] = fmaf(g[e], (f[e] - mean) * rstd, dw[e]);
            db[e] += g[e];
        }
    }
    float* to = t.sums + blockIdx.y * 2 * pad4(t.cols);
    storef(to + c, dw, n);
    storef(to + pad4(t.cols) + c, db, n);
}

// how a row is held: wavefronts to a row and pieces of eight columns to a thread; 0 pieces: read again
struct Hold {
    int waves, pieces;
};

Hold hold_of(int cols) {
    if (cols <= 2048) return Hold{1, (cols + 511) / 512};
    if (cols <= 8192) return Hold{4, (cols + 2047) / 2048};
    if (cols <= 16384) return Hold{8, 4};
    return Hold{16, 0};
}

// In the backward pass eight wavefronts hold a row of 2049 .. 16384 columns: half the registers, twice the wavefronts on a CU
// (2048 x 7168 bf16 28.6 us, with four 33.2; 16384 x 7168 145 and 145; 16384 x 4096 85 and 82).
Hold grad_hold_of(int cols) {
    if (cols <= 2048) return Hold{1, (cols + 511) / 512};
    if (cols <= 16384) return Hold{8, cols <= 4096 ? 1 : cols <= 8192 ? 2 : 4};
    return Hold{16, 0};
}

// Workgroups of the backward pass.  Each leaves a row of partial sums, to be written and read again, so that few rows are
// better off with fewer: with 128, 256 and 512 of them 256 x 7168 takes 14.6, 19.0, - us, 2048 x 7168 35.9, 28.6, 32.5, 4096 x
// 7168 59.8, 40.9, 43.5, 16384 x 7168 248, 149, 145, 4096 x 2048 21.6, 18.2, 18.9.
int grad_grid(int rows, int cols) {
    const Hold h = grad_hold_of(cols);
    if (h.pieces == 0) return std::min(rows, 64);
    return std::min(h.waves == 1 ? (rows + 3) / 4 : rows, rows <= 512 ? 128 : rows < 8192 ? 256 : 512);
}

template <class T, class P, int W, int V>
moe_status launch_norm(NormArgs t, hipStream_t stream) {
    const int rows = W == 1 ? 4 : 1, threads = W == 1 ? 256 : W * MOE_WAVE;
    for (const int most = kMostGroups * rows; t.rows > most;) {
        NormArgs first = t;
        first.rows = most;
        const moe_status st = launch_norm<T, P, W, V>(first, stream);
        if (st != MOE_OK) return st;
        t.x = static_cast<const T*>(t.x) + most * t.x_ld;
        t.y = static_cast<T*>(t.y) + most * t.y_ld;
        if (t.mean) t.mean += most;
        if (t.rstd) t.rstd += most;
        t.rows -= most;
    }
    hipLaunchKernelGGL((norm_kernel<T, P, W, V>), dim3((t.rows + rows - 1) / rows), dim3(threads), 0, stream, t);
    return launch_status();
}

template <class T, class P, int W, int V>
moe_status launch_grad(const NormGradArgs& t, hipStream_t stream) {
    hipLaunchKernelGGL((norm_grad_kernel<T, P, W, V>), dim3(grad_grid(t.rows, t.cols)),
                       dim3(W == 1 ? 256 : W * MOE_WAVE), 0, stream, t);
    return launch_status();
}

template <class T, class P>
moe_status run_norm(const NormArgs& t, hipStream_t stream) {
    const Hold h = hold_of(t.cols);
    switch (h.waves * 8 + h.pieces) {
        case 9: return launch_norm<T, P, 1, 1>(t, stream);
        case 10: return launch_norm<T, P, 1, 2>(t, stream);
        case 11: return launch_norm<T, P, 1, 3>(t, stream);
        case 12: return launch_norm<T, P, 1, 4>(t, stream);
        case 34: return launch_norm<T, P, 4, 2>(t, stream);
        case 35: return launch_norm<T, P, 4, 3>(t, stream);
        case 36: return launch_norm<T, P, 4, 4>(t, stream);
        case 68: return launch_norm<T, P, 8, 4>(t, stream);
        default:
            hipLaunchKernelGGL((norm_long_kernel<T, P>), dim3(std::min(t.rows, kMostGroups)), dim3(1024), 0, stream, t);
            return launch_status();
    }
}

template <class T, class P>
moe_status run_grad(const NormGradArgs& t, void* dweight, void* dbias, hipStream_t stream) {
    const Hold h = grad_hold_of(t.cols);
    const int grid = grad_grid(t.rows, t.cols);
    moe_status st = MOE_OK;
    switch (h.waves * 8 + h.pieces) {
        case 9: st = launch_grad<T, P, 1, 1>(t, stream); break;
        case 10: st = launch_grad<T, P, 1, 2>(t, stream); break;
        case 11: st = launch_grad<T, P, 1, 3>(t, stream); break;
        case 12: st = launch_grad<T, P, 1, 4>(t, stream); break;
        case 65: st = launch_grad<T, P, 8, 1>(t, stream); break;
        case 66: st = launch_grad<T, P, 8, 2>(t, stream); break;
        case 68: st = launch_grad<T, P, 8, 4>(t, stream); break;
        default:
            // the columns first: dx may be dy or x itself
            if (t.sums) {
                hipLaunchKernelGGL(norm_columns_kernel<T>, dim3((t.cols + 2047) / 2048, grid), dim3(256), 0, stream, t);
                st = launch_status();
            }
            if (t.dx && st == MOE_OK) {
                hipLaunchKernelGGL((norm_grad_long_kernel<T, P>), dim3(std::min(t.rows, kMostGroups)), dim3(1024), 0, stream, t);
                st = launch_status();
            }
    }
    if (st != MOE_OK || !t.sums) return st;
    return join_columns<P>(t.sums, grid, 2 * pad4(t.cols), pad4(t.cols), t.cols, dweight, dbias, stream);
}

template <class P>
__global__ void __launch_bounds__(256) zero_kernel(P* a, P* b, int n) {
    const int i = blockIdx.x * 256 + threadIdx.x;
    if (i >= n) return;
    if (a) a[i] = (P)0.0f;
    if (b) b[i] = (P)0.0f;
}

bool misplaced(const void* p, size_t to) { return ((uintptr_t)p & (to - 1)) != 0; }
size_t size_of(int dtype) { return dtype == MOE_FP32 ? 4 : 2; }

moe_status check_norm(int64_t rows, int64_t cols) {
    if (rows < 0 || cols < 1) return MOE_ERR_INVALID_ARG;
    if (rows >= (1 << 30) || cols >= (1 << 30)) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}
bool bad_types(int dtype, int param_dtype) {
    return dtype < MOE_BF16 || dtype > MOE_FP32 || (param_dtype != dtype && param_dtype != MOE_FP32);
}

size_t grad_bytes(int rows, int cols) { return rows == 0 ? 0 : (size_t)grad_grid(rows, cols) * 2 * pad4(cols) * sizeof(float); }

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status moe_layer_norm(int32_t rows, int32_t cols, int32_t dtype, int32_t param_dtype, const void* x,
                                     int64_t x_stride, const void* weight, const void* bias, float eps, void* y,
                                     int64_t y_stride, float* mean, float* rstd, void* hip_stream) {
    const moe_status st = check_norm(rows, cols);
    if (st != MOE_OK) return st;
    if (bad_types(dtype, param_dtype) || !(eps >= 0.0f)) return MOE_ERR_INVALID_ARG;
    if (rows == 0) return MOE_OK;
    const size_t e = size_of(dtype), p = size_of(param_dtype);
    if (!x || !y || misplaced(x, e) || misplaced(y, e) || misplaced(weight, p) || misplaced(bias, p) ||
        misplaced(mean, 4) || misplaced(rstd, 4) || x_stride < cols || y_stride < cols)
        return MOE_ERR_INVALID_ARG;
    const NormArgs t{x, weight, bias, y, mean, rstd, x_stride, y_stride, rows, cols, eps};
    const hipStream_t stream = reinterpret_cast<hipStream_t>(hip_stream);
    if (dtype == MOE_FP32) return run_norm<float, float>(t, stream);
    if (dtype == MOE_BF16)
        return param_dtype == MOE_FP32 ? run_norm<__bf16, float>(t, stream) : run_norm<__bf16, __bf16>(t, stream);
    return param_dtype == MOE_FP32 ? run_norm<_Float16, float>(t, stream) : run_norm<_Float16, _Float16>(t, stream);
}

extern "C" moe_status moe_layer_norm_backward_workspace(int32_t rows, int32_t cols, size_t* bytes) {
    const moe_status st = check_norm(rows, cols);
    if (st != MOE_OK) return st;
    if (!bytes) return MOE_ERR_INVALID_ARG;
    *bytes = grad_bytes(rows, cols);
    return MOE_OK;
}

extern "C" moe_status moe_layer_norm_backward(int32_t rows, int32_t cols, int32_t dtype, int32_t param_dtype, const void* dy,
                                              int64_t dy_stride, const void* x, int64_t x_stride, const void* weight,
                                              const float* mean, const float* rstd, void* dx, int64_t dx_stride,
                                              void* dweight, void* dbias, void* ws, size_t ws_bytes, void* hip_stream) {
    moe_status st = check_norm(rows, cols);
    if (st != MOE_OK) return st;
    const size_t e = size_of(dtype), p = size_of(param_dtype);
    if (bad_types(dtype, param_dtype) || misplaced(dweight, p) || misplaced(dbias, p)) return MOE_ERR_INVALID_ARG;
    const hipStream_t stream = reinterpret_cast<hipStream_t>(hip_stream);
    if (rows == 0) {
        if (!dweight && !dbias) return MOE_OK;
        const dim3 grid((cols + 255) / 256);
        if (p == 4)
            hipLaunchKernelGGL(zero_kernel<float>, grid, dim3(256), 0, stream, static_cast<float*>(dweight),
                               static_cast<float*>(dbias), cols);
        else
            hipLaunchKernelGGL(zero_kernel<_Float16>, grid, dim3(256), 0, stream, static_cast<_Float16*>(dweight),
                               static_cast<_Float16*>(dbias), cols);      // +0 in either type
        return launch_status();
    }
    if (!dy || !x || !mean || !rstd || misplaced(dy, e) || misplaced(x, e) || misplaced(weight, p) || misplaced(mean, 4) ||
        misplaced(rstd, 4) || dy_stride < cols || x_stride < cols || (dx && (misplaced(dx, e) || dx_stride < cols)))
        return MOE_ERR_INVALID_ARG;
    if (!dx && !dweight && !dbias) return MOE_OK;
    float* sums = nullptr;
    if (dweight || dbias) {
        if (!ws || ws_bytes < grad_bytes(rows, cols)) return MOE_ERR_WORKSPACE;
        if (misplaced(ws, 16)) return MOE_ERR_INVALID_ARG;
        sums = static_cast<float*>(ws);
    }
    const NormGradArgs t{dy, x, weight, mean, rstd, dx, sums, dy_stride, x_stride, dx_stride, rows, cols};
    if (dtype == MOE_FP32) return run_grad<float, float>(t, dweight, dbias, stream);
    if (dtype == MOE_BF16)
        return param_dtype == MOE_FP32 ? run_grad<__bf16, float>(t, dweight, dbias, stream)
                                       : run_grad<__bf16, __bf16>(t, dweight, dbias, stream);
    return param_dtype == MOE_FP32 ? run_grad<_Float16, float>(t, dweight, dbias, stream)
                                   : run_grad<_Float16, _Float16>(t, dweight, dbias, stream);
}
