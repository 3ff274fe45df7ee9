// y = x w^T for up to 64 rows of x: the weights are read once, by wavefronts that share a tile of 16 weight rows and cut
// K among themselves.
//
// The weights are the MFMA's A operand (lane l: weight row l % 16, K 8 (l / 16) .. + 7) and the tokens its B operand
// (column l % 16), so the tokens of one call are columns of one to four 16-wide tiles and a lane's results are four
// consecutive columns of y for one token.  The wavefronts' sums meet in LDS, where eight columns of a token at a time
// are summed in a fixed order and go through the epilogue.  Gated: a tile's rows are eight of the gate's and the same
// eight of the up projection's.
#include "dense.h"

namespace moe {
namespace {

constexpr int kFewWaves = 8, kChunk = 128;                   // K of a wavefront's turn

struct FewArgs {
    Product p;
    Epilogue e;
};

template <class T, int CT, bool PAIRED>
__global__ void __launch_bounds__(kFewWaves * MOE_WAVE)
few_kernel(FewArgs t) {
    typedef typename Vec<T>::x8 x8;
    __shared__ float sums[kFewWaves][16 * CT][16];           // [wavefront][token][weight row of the tile]
    const int lane = threadIdx.x % MOE_WAVE, wave = threadIdx.x / MOE_WAVE;
    const int l = lane & 15, q = lane >> 4;
    const int K = t.p.k, n0 = blockIdx.x * (PAIRED ? 8 : 16), most = PAIRED ? t.p.inter : t.p.n;
    // rows past the weight's or the tokens' end read the last one; what they give is not stored
    const int64_t row = PAIRED ? min(n0 + (l & 7), most - 1) + (int64_t)(l >> 3) * most : min(n0 + l, most - 1);
    const T* w = static_cast<const T*>(t.p.b) + row * t.p.ldb;
    const T* x[CT];
#pragma unroll
    for (int c = 0; c < CT; ++c) x[c] = static_cast<const T*>(t.p.a) + (int64_t)min(16 * c + l, t.p.m - 1) * t.p.lda;

    f32x4 acc[CT];
#pragma unroll
    for (int c = 0; c < CT; ++c) acc[c] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int k0 = wave * kChunk; k0 < K; k0 += kFewWaves * kChunk) {
        x8 wf[4], xf[CT][4];
        if (k0 + kChunk <= K) {
#pragma unroll
            for (int s = 0; s < 4; ++s) wf[s] = load8(w + k0 + 32 * s + 8 * q, 8);
#pragma unroll
            for (int c = 0; c < CT; ++c)
#pragma unroll
                for (int s = 0; s < 4; ++s) xf[c][s] = load8(x[c] + k0 + 32 * s + 8 * q, 8);
        } else {
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const int k = k0 + 32 * s + 8 * q, n = min(8, K - k);
                wf[s] = load8(w + k, n);
#pragma unroll
                for (int c = 0; c < CT; ++c) xf[c][s] = load8(x[c] + k, n);
            }
        }
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
            for (int c = 0; c < CT; ++c) acc[c] = mfma(wf[s], xf[c][s], acc[c]);
    }
    asm volatile("s_nop 15");                                // the wait before an MFMA's result is read
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int c = 0; c < CT; ++c) {
        asm volatile("" : "+v"(acc[c]));
        *reinterpret_cast<f32x4*>(&sums[wave][16 * c + l][4 * q]) = acc[c];
    }
    __syncthreads();
    for (int item = threadIdx.x; item < 16 * CT * (PAIRED ? 1 : 2); item += kFewWaves * MOE_WAVE) {
        const int token = PAIRED ? item : item >> 1, c = PAIRED ? 0 : 8 * (item & 1);
        if (token >= t.p.m || n0 + c >= most) continue;
        float v[8], u[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = u[i] = 0.0f;
#pragma unroll
        for (int wv = 0; wv < kFewWaves; ++wv) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                v[i] += sums[wv][token][c + i];
                if (PAIRED) u[i] += sums[wv][token][8 + i];
            }
        }
        const int n = min(8, most - n0 - c);
        if constexpr (PAIRED) finish_gated<T>(t.e, token, n0, v, u, n);
        else finish<T>(t.e, token, n0 + c, v, n);
    }
}

template <class T, bool PAIRED>
moe_status launch_tokens(const Product& p, const Epilogue& e, hipStream_t stream) {
    const int width = PAIRED ? 8 : 16, columns = PAIRED ? p.inter : p.n;
    const dim3 grid((columns + width - 1) / width), block(kFewWaves * MOE_WAVE);
    const FewArgs t{p, e};
    switch ((p.m + 15) / 16) {
        case 1: hipLaunchKernelGGL((few_kernel<T, 1, PAIRED>), grid, block, 0, stream, t); break;
        case 2: hipLaunchKernelGGL((few_kernel<T, 2, PAIRED>), grid, block, 0, stream, t); break;
        case 3: hipLaunchKernelGGL((few_kernel<T, 3, PAIRED>), grid, block, 0, stream, t); break;
        case 4: hipLaunchKernelGGL((few_kernel<T, 4, PAIRED>), grid, block, 0, stream, t); break;
        default: return MOE_ERR_UNSUPPORTED;
    }
    return launch_status();
}

}  // namespace

moe_status launch_few(int dtype, const Product& p, const Epilogue& e, hipStream_t stream) {
    if (dtype == MOE_BF16)
        return p.inter ? launch_tokens<__bf16, true>(p, e, stream) : launch_tokens<__bf16, false>(p, e, stream);
    return p.inter ? launch_tokens<_Float16, true>(p, e, stream) : launch_tokens<_Float16, false>(p, e, stream);
}

}  // namespace moe
