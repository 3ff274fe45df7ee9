// What the dense layers' kernels share: the 16-bit types, the activations, rows that start anywhere, the epilogue of a
// product, and the launches that the entry points choose from.
#pragma once

#include <type_traits>
#include <utility>

#include "common.h"
#include "dense_index.h"

namespace moe {

typedef float f32x4 __attribute__((ext_vector_type(4)));

template <class T>
struct Vec;
template <>
struct Vec<__bf16> {
    typedef __bf16 x8 __attribute__((ext_vector_type(8)));
    typedef __bf16 x4 __attribute__((ext_vector_type(4)));
};
template <>
struct Vec<_Float16> {
    typedef _Float16 x8 __attribute__((ext_vector_type(8)));
    typedef _Float16 x4 __attribute__((ext_vector_type(4)));
};

// D += A B over 32 of K, 16 x 16 results: lane l holds row l % 16 of A (column of B), K 8 (l / 16) .. + 7, and results
// [row 4 (l / 16) + v, column l % 16]
__device__ __forceinline__ f32x4 mfma(const Vec<__bf16>::x8& a, const Vec<__bf16>::x8& b, const f32x4& c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mfma(const Vec<_Float16>::x8& a, const Vec<_Float16>::x8& b, const f32x4& c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// Up to eight consecutive elements from anywhere a T may lie; those past n (n <= 8) are zeros.  Whole ones take one
// 16-byte access, which global memory serves from any address.
template <class T>
__device__ __forceinline__ typename Vec<T>::x8 load8(const T* p, int n) {
    typename Vec<T>::x8 v;
    if (n >= 8) {
        __builtin_memcpy(&v, p, 16);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < n ? p[i] : (T)0.0f;
    }
    return v;
}

template <class T>
__device__ __forceinline__ void store8(T* p, const float (&f)[8], int n) {
    typename Vec<T>::x8 v;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (T)f[i];
    if (n >= 8) {
        __builtin_memcpy(p, &v, 16);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) p[i] = v[i];
    }
}

// f(0), f(1), .. f(N - 1) with constants, in line
template <class F, int... I>
__device__ __forceinline__ void unroll_over(F&& f, std::integer_sequence<int, I...>) {
    (f(std::integral_constant<int, I>{}), ...);
}
template <int N, class F>
__device__ __forceinline__ void unroll(F&& f) {
    unroll_over(f, std::make_integer_sequence<int, N>{});
}

// ---------------------------------------------------------------- memory straight to LDS
#define MOE_LDS(p) ((void __attribute__((address_space(3)))*)(p))

// s_waitcnt immediates: at most n vector memory operations in flight; every LDS operation returned
constexpr int wait_vm(int n) { return (n & 0xF) | (0x7 << 4) | (0xF << 8) | ((n >> 4) << 14); }
constexpr int kWaitLds0 = 0xF | (0x7 << 4) | (0x3 << 14);

// 16 bytes a lane from p + off (zeros where that is not below `bytes`) to LDS at lds + AT + 16 * lane.  In asm, since the
// compiler takes every transposing LDS read for one that may depend on any such load in flight and waits for all of them;
// the caller counts them (vmcnt) and waits before a barrier.  s_nop 4: the descriptor's registers may come from a
// v_readlane, whose result a vector memory instruction may read five wait states later.  m0 is the compiler's own: it sets
// it before each of its uses.
template <int AT>
__device__ __forceinline__ void load_to_lds(const void* p, int bytes, uint32_t off, uint32_t lds) {
    const uint64_t at = (uint64_t)p;
    const u32x4 rsrc = {(uint32_t)at, (uint32_t)(at >> 32), (uint32_t)bytes, 0x00020000u};     // addresses have 48 bits
    asm volatile("s_add_u32 m0, %2, %3\n\ts_nop 4\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds" ::"v"(off), "s"(rsrc), "s"(lds),
                 "i"(AT)
                 : "memory", "scc");
}

// ---------------------------------------------------------------- activations
// In fp32; the exponential and the reciprocal are the hardware's (a few ulps), unseen behind a rounding to 16 bits.
//   silu      z s(z), s(z) = 1 / (1 + e^-z)
//   gelu      z P(z), P the normal distribution's; below 0, where 1 + erf would cancel, P(-u) = e^(-u^2 / 2) g(u) with
//             g(u) = e^(u^2 / 2) erfc(u / sqrt 2) / 2 = t Q(t), t = 1 / (1 + 3 u / 8), Q of degree 8 fitted to g (weighted
//             least squares, reweighted towards the largest error), whose fp32 constants give it to 2.6e-7 of it everywhere,
//             the most at 0; above 0, 1 - P(-u).  The library's erfc took 1001 x 777 outputs from 18 us to 36.
//   gelu_tanh z (1 + tanh u) / 2 = z s(2u), u = sqrt(2 / pi) (z + 0.044715 z^3)
__device__ __forceinline__ float sigmoid(float z) { return __builtin_amdgcn_rcpf(1.0f + __expf(-z)); }
// P(z); bell: e^(-z^2 / 2)
__device__ __forceinline__ float gelu_cdf(float z, float& bell) {
    const float t = __builtin_amdgcn_rcpf(fmaf(0.375f, fabsf(z), 1.0f));
    float q = -0.032911065965890884f;
    q = fmaf(q, t, 0.13687998056411743f);
    q = fmaf(q, t, -0.18652129173278809f);
    q = fmaf(q, t, 0.05063246563076973f);
    q = fmaf(q, t, 0.01562788337469101f);
    q = fmaf(q, t, 0.08863824605941772f);
    q = fmaf(q, t, 0.12844568490982056f);
    q = fmaf(q, t, 0.14960458874702454f);
    q = fmaf(q, t, 0.14960338175296783f);
    bell = __expf(-0.5f * z * z);
    const float below = bell * (q * t);
    return z > 0.0f ? 1.0f - below : below;
}
__device__ __forceinline__ float gelu_tanh_2u(float z) {
    return z * fmaf(z * z, 2.0f * 0.79788456080286536f * 0.044715f, 2.0f * 0.79788456080286536f);
}

template <int N>
__device__ __forceinline__ void activate(float (&z)[N], int act) {
    switch (act) {
        case MOE_ACT_RELU:
#pragma unroll
            for (int i = 0; i < N; ++i) z[i] = z[i] < 0.0f ? 0.0f : z[i];          // NaN stays
            break;
        case MOE_ACT_SILU:
#pragma unroll
            for (int i = 0; i < N; ++i) z[i] *= sigmoid(z[i]);
            break;
        case MOE_ACT_GELU:
#pragma unroll
            for (int i = 0; i < N; ++i) {
                float bell;
                z[i] *= gelu_cdf(z[i], bell);
            }
            break;
        case MOE_ACT_GELU_TANH:
#pragma unroll
            for (int i = 0; i < N; ++i) z[i] *= sigmoid(gelu_tanh_2u(z[i]));
            break;
        default: break;
    }
}

// a = act(z), d = act'(z)
template <int N>
__device__ __forceinline__ void activate_grad(const float (&z)[N], float (&a)[N], float (&d)[N], int act) {
    switch (act) {
        case MOE_ACT_RELU:
#pragma unroll
            for (int i = 0; i < N; ++i) {
                a[i] = z[i] < 0.0f ? 0.0f : z[i];
                d[i] = z[i] > 0.0f ? 1.0f : 0.0f;
            }
            break;
        case MOE_ACT_SILU:
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float s = sigmoid(z[i]);
                a[i] = z[i] * s;
                d[i] = s * fmaf(z[i], 1.0f - s, 1.0f);
            }
            break;
        case MOE_ACT_GELU:
#pragma unroll
            for (int i = 0; i < N; ++i) {
                float bell;
                const float p = gelu_cdf(z[i], bell);
                a[i] = z[i] * p;
                d[i] = fmaf(z[i], 0.39894228040143268f * bell, p);
            }
            break;
        case MOE_ACT_GELU_TANH:
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float s = sigmoid(gelu_tanh_2u(z[i]));
                a[i] = z[i] * s;
                const float slope = fmaf(z[i] * z[i], 6.0f * 0.79788456080286536f * 0.044715f,
                                         2.0f * 0.79788456080286536f);
                const float t = s * (1.0f - s);
                d[i] = t == 0.0f ? s : fmaf(z[i] * t, slope, s);       // where z^2 overflows, t is 0
            }
            break;
        default:
#pragma unroll
            for (int i = 0; i < N; ++i) {
                a[i] = z[i];
                d[i] = 1.0f;
            }
    }
}

// ---------------------------------------------------------------- columns' sums, as workgroups left them
// out_a[c] (out_b[c]) = the sum of column c (half + c) over `parts` rows of `sums`, `ld` floats (a multiple of 4) apart; each
// may be null.  64 columns to a workgroup, four to a thread, sixteen teams that take every sixteenth row: a fixed order.
// 512 rows of 2 x 7168: 42 us with four teams and a column to a thread.
constexpr int kMostGroups = 1 << 20;                         // of a launch, which holds less than 2^32 threads

__host__ __device__ inline int64_t pad4(int64_t n) { return (n + 3) & ~int64_t(3); }

template <class T>
__global__ void __launch_bounds__(256) join_columns_kernel(const float* sums, int parts, int64_t ld, int64_t from, int half, int n,
                                                           T* out_a, T* out_b) {
    constexpr int kTeams = 16;
    __shared__ f32x4 lds[kTeams][16];
    const int lane = threadIdx.x % 16, team = threadIdx.x / 16;
    const int64_t first = from + (int64_t)blockIdx.x * 64, c = first + lane * 4;
    f32x4 sum = {0.f, 0.f, 0.f, 0.f};
    if (c < ld) {
#pragma unroll 8
        for (int p = team; p < parts; p += kTeams) sum += *reinterpret_cast<const f32x4*>(sums + p * ld + c);
    }
    lds[team][lane] = sum;
    __syncthreads();
    if (threadIdx.x >= 64) return;
    const int64_t at = first + threadIdx.x;
    float s = 0.0f;
#pragma unroll
    for (int t = 0; t < kTeams; ++t) s += reinterpret_cast<const float*>(lds[t])[threadIdx.x];
    if (at < n) {
        if (out_a) out_a[at] = (T)s;
    } else if (at >= half && at < half + n) {
        if (out_b) out_b[at - half] = (T)s;
    }
}

template <class T>
inline moe_status join_columns(const float* sums, int parts, int64_t ld, int64_t half, int n, void* out_a, void* out_b,
                               hipStream_t stream) {
    moe_status st = MOE_OK;
    for (int64_t from = 0, groups = (ld + 63) / 64; groups > 0 && st == MOE_OK; groups -= kMostGroups, from += (int64_t)kMostGroups * 64) {
        hipLaunchKernelGGL(join_columns_kernel<T>, dim3((unsigned)std::min<int64_t>(groups, kMostGroups)), dim3(256), 0, stream, sums,
                           parts, ld, from, (int)half, n, static_cast<T*>(out_a), static_cast<T*>(out_b));
        st = launch_status();
    }
    return st;
}

// ---------------------------------------------------------------- the epilogue of a product
// What becomes of the fp32 sums z[row, c]: plain ones, y = act(z + bias) + res; gated ones, y = act(g) u with g and u the
// columns c and inter + c.  Stored once, rounded once; z (gu) as well where it is not null.
struct Epilogue {
    const void* bias;        // [n], null: none
    const void* res;         // rows of res_ld, null: none; may be y itself
    void* z;                 // rows of z_ld, null: not kept
    void* y;                 // rows of y_ld
    int64_t res_ld, z_ld, y_ld;
    int n;                   // columns of y
    int act;
    int rows;                // of y
    const float* unit = nullptr;     // not null: the sums are multiplied by it first (a power of two; see Peaks)
};

// n <= 8 columns from c of one row; bias and res: those of the bias and the residual, read beforehand
template <class T>
__device__ __forceinline__ typename Vec<T>::x8 residual_of(const Epilogue& e, int64_t row, int c, int n) {
    return e.res ? load8(static_cast<const T*>(e.res) + row * e.res_ld + c, n) : typename Vec<T>::x8{};
}

template <class T>
__device__ __forceinline__ typename Vec<T>::x8 bias_of(const Epilogue& e, int c, int n) {
    return e.bias ? load8(static_cast<const T*>(e.bias) + c, n) : typename Vec<T>::x8{};
}

// Only gradients of fp16 have a unit: it is one elsewhere, unread.
template <class T>
__device__ __forceinline__ float unit_of(const Epilogue& e) {
    if constexpr (std::is_same<T, _Float16>::value) return e.unit ? *e.unit : 1.0f;
    return 1.0f;
}

template <class T>
__device__ __forceinline__ void in_units(float (&v)[8], float unit) {
    if constexpr (std::is_same<T, _Float16>::value) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= unit;
    }
}

template <class T>
__device__ __forceinline__ void finish(const Epilogue& e, int64_t row, int c, float (&v)[8], int n,
                                       const typename Vec<T>::x8& bias, const typename Vec<T>::x8& res) {
    if (e.bias) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += (float)bias[i];
    }
    if (e.z) store8(static_cast<T*>(e.z) + row * e.z_ld + c, v, n);
    activate(v, e.act);
    if (e.res) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += (float)res[i];
    }
    store8(static_cast<T*>(e.y) + row * e.y_ld + c, v, n);
}

template <class T>
__device__ __forceinline__ void finish_gated(const Epilogue& e, int64_t row, int c, float (&g)[8], float (&u)[8], int n) {
    if (e.z) {
        T* gu = static_cast<T*>(e.z) + row * e.z_ld + c;
        store8(gu, g, n);
        store8(gu + e.n, u, n);
    }
    activate(g, e.act);
#pragma unroll
    for (int i = 0; i < 8; ++i) g[i] *= u[i];
    store8(static_cast<T*>(e.y) + row * e.y_ld + c, g, n);
}

// ---------------------------------------------------------------- products, as the entry points ask for them
// C[m, n] = sum_k A(m, k) B(n, k).  A(m, k) at a[m lda + k], or a[k lda + m] where it is transposed; B alike.
enum Layout { kNT, kNN, kTN };          // forward; dx = dy w (B transposed); dw = dy^T x (both)

struct Product {
    const void* a;
    const void* b;
    int64_t lda, ldb;
    int m, n, k;             // n: rows of B (gated: 2 inter)
    int inter;               // gated: columns of y, else 0
    int b_rows;              // not 0: B (K across its rows) has this many, at most a step, for every step of A's K
};

struct Plan {
    int tile;                // 0: few rows; 64, 128, 256: tiles of 64 x 64, 128 x 128, 256 x 256
    int splits;              // parts of K, summed by a second launch
    int kper;                // of K to a part, a multiple of kStepK
    bool joined;             // the sums go to a second launch
};

// terms = 2: A's rows (NN) or K (TN) are two terms of one operand, kTermRows apart (see run_backward)
Plan plan_product(Layout layout, int64_t m, int64_t n, int64_t k, bool aligned, int terms = 1);
int64_t plan_bytes(const Plan& p, int64_t m, int64_t n);          // of fp32 partial sums
constexpr int kTermRows = 64;

bool rows_aligned(const void* p, int64_t ld, int64_t contiguous); // 16-byte rows, whole 16-byte pieces

// one launch each; part: the partial sums where the plan is joined
moe_status launch_tiles(Layout layout, int dtype, bool aligned, const Plan& plan, const Product& p, const Epilogue& e,
                        float* part, hipStream_t stream);
moe_status launch_tiles_nt(int dtype, bool aligned, const Plan& plan, const Product& p, const Epilogue& e, float* part,
                           hipStream_t stream);
moe_status launch_tiles_nn(int dtype, bool aligned, const Plan& plan, const Product& p, const Epilogue& e, float* part,
                           hipStream_t stream);
moe_status launch_tiles_tn(int dtype, bool aligned, const Plan& plan, const Product& p, const Epilogue& e, float* part,
                           hipStream_t stream);
moe_status launch_pair(int dtype, const Plan& plan_dw, const Product& dw, const Epilogue& e_dw, const Plan& plan_dx,
                       const Product& dx, const Epilogue& e_dx, hipStream_t stream);
moe_status launch_few(int dtype, bool aligned, const Product& p, const Epilogue& e, hipStream_t stream);

}  // namespace moe
