// y = x w^T for up to 64 rows of x: the weights are read once, by wavefronts that share a tile of 16 weight rows and cut
// K among themselves.
//
// The weights are the MFMA's A operand (lane l: weight row l % 16, K 8 (l / 16) .. + 7) and the tokens its B operand
// (column l % 16), so the tokens of one call are columns of one to four 16-wide tiles and a lane's results are four
// consecutive columns of y for one token.  The wavefronts' sums meet in LDS, where eight columns of a token at a time
// are summed in a fixed order and go through the epilogue.  Gated: a tile's rows are eight of the gate's and the same
// eight of the up projection's.
//
// Memory bound, so what counts is bytes in flight and whole lines: rows of whole 16-byte pieces go straight to LDS, 128
// bytes of eight rows to a load, through a ring that each wavefront keeps for itself (no barrier; its own loads it
// counts).  Loaded in the MFMA's layout instead (sixteen rows of 16 bytes side by side), a load takes the CU's address
// unit four times as long, and fewer are in flight: 1 x 7168 -> 2 x 2048 gated 11.5 us, 1 x 2048 -> 7168 7.9 us.
#include "dense.h"

namespace moe {
namespace {

constexpr int kFewWaves = 8, kChunk = 128;                   // K of a wavefront's turn

struct FewArgs {
    Product p;
    Epilogue e;
};

// The sums of the wavefronts, [wavefront][token][weight row of the tile] at `sums` + wavefront * step, through the epilogue.
template <class T, int CT, int W, bool PAIRED>
__device__ __forceinline__ void finish_tokens(const FewArgs& t, const float* sums, int step, int n0, int most) {
    for (int item = threadIdx.x; item < 16 * CT * (PAIRED ? 1 : 2); item += W * MOE_WAVE) {
        const int token = PAIRED ? item : item >> 1, c = PAIRED ? 0 : 8 * (item & 1);
        if (token >= t.p.m || n0 + c >= most) continue;
        float v[8], u[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = u[i] = 0.0f;
#pragma unroll
        for (int wv = 0; wv < W; ++wv) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                v[i] += sums[wv * step + token * 16 + c + i];
                if (PAIRED) u[i] += sums[wv * step + token * 16 + 8 + i];
            }
        }
        const int n = min(8, most - n0 - c);
        if constexpr (PAIRED) finish_gated<T>(t.e, token, n0, v, u, n);
        else finish<T>(t.e, token, n0 + c, v, n, bias_of<T>(t.e, n0 + c, n), residual_of<T>(t.e, token, n0 + c, n));
    }
}

// Rows that start anywhere.
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
    finish_tokens<T, CT, kFewWaves, PAIRED>(t, &sums[0][0][0], 16 * CT * 16, n0, most);
}

// Rows of whole 16-byte pieces.  W wavefronts; wavefront w takes every W-th 64 of K, D of them in flight.
template <class T, int CT, int W, int D, bool PAIRED>
__global__ void __launch_bounds__(W * MOE_WAVE) few_stream_kernel(FewArgs t) {
    typedef typename Vec<T>::x8 x8;
    constexpr int kStage = (1 + CT) * 2048, kLoads = 2 + 2 * CT;
    static_assert(W * D * kStage * (8 / W) <= 160 * 1024 && D * kStage >= CT * 1024 && D * kLoads < 64, "LDS");
    __shared__ __align__(16) uint8_t lds[W * D * kStage];
    const int lane = threadIdx.x % MOE_WAVE;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / MOE_WAVE);
    const int l = lane & 15, q = lane >> 4;
    const int K = t.p.k, n0 = blockIdx.x * (PAIRED ? 8 : 16), most = PAIRED ? t.p.inter : t.p.n;
    const int turns = max(0, ((K + 63) / 64 - wave + W - 1) / W);

    // eight rows to a load; lane l brings chunk l % 8 of row l / 8, by the swizzle of the sixteen rows' places
    const int chunk[2] = {(lane & 7) ^ swizzle(lane >> 3), (lane & 7) ^ swizzle(8 + (lane >> 3))};
    const T* at[kLoads];
    int bytes[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        const bool x = i >= 2;
        const int row = x ? 8 * (i - 2) : n0 + (PAIRED ? 0 : 8 * i), rows = min(8, (x ? t.p.m : most) - row);
        const int64_t ld = x ? t.p.lda : t.p.ldb;
        at[i] = static_cast<const T*>(x ? t.p.a : t.p.b) + (row + (PAIRED && i == 1 ? (int64_t)most : 0)) * ld + 64 * wave;
        bytes[i] = rows > 0 ? 2 * ((rows - 1) * (int)ld + min(64, K)) : 0;
    }
    uint32_t off_w[2], off_x[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        off_w[h] = (lane >> 3) * (uint32_t)(t.p.ldb * 2) + chunk[h] * 16;
        off_x[h] = (lane >> 3) * (uint32_t)(t.p.lda * 2) + chunk[h] * 16;
    }
    const uint32_t ring = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)MOE_LDS(lds)) + wave * D * kStage;
    int k0 = 64 * wave;
    auto issue = [&](int place) __attribute__((always_inline)) {
        const bool in[2] = {8 * chunk[0] < K - k0, 8 * chunk[1] < K - k0};
        unroll<kLoads>([&](auto i_) __attribute__((always_inline)) {
            constexpr int i = decltype(i_)::value;
            load_to_lds<i * 1024>(at[i], bytes[i], in[i & 1] ? (i < 2 ? off_w : off_x)[i & 1] : 0x80000000u,
                                  ring + place * kStage);
            at[i] += 64 * W;
        });
        k0 += 64 * W;
    };

    f32x4 acc[CT];
#pragma unroll
    for (int c = 0; c < CT; ++c) acc[c] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int d = 0; d < D; ++d) issue(d);                    // past the end of K: zeros
    int place = 0;
    for (int turn = 0; turn < turns; ++turn) {
        __builtin_amdgcn_s_waitcnt(wait_vm((D - 1) * kLoads));
        asm volatile("" ::: "memory");
        const uint8_t* from = lds + (wave * D + place) * kStage;
        auto fragment = [&](int tile, int s) __attribute__((always_inline)) {
            return *reinterpret_cast<const x8*>(from + tile * 2048 + l * 128 + (((4 * s + q) ^ swizzle(l)) << 4));
        };
        x8 wf[2], xf[2][CT];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            wf[s] = fragment(0, s);
#pragma unroll
            for (int c = 0; c < CT; ++c) xf[s][c] = fragment(1 + c, s);
        }
        __builtin_amdgcn_s_waitcnt(kWaitLds0);               // the place is read: fill it again
        __builtin_amdgcn_sched_barrier(0);
        issue(place);
        place = place + 1 == D ? 0 : place + 1;
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int c = 0; c < CT; ++c) acc[c] = mfma(wf[s], xf[s][c], acc[c]);
    }
    __builtin_amdgcn_s_waitcnt(wait_vm(0));
    asm volatile("s_nop 15" ::: "memory");                   // the wait before an MFMA's result is read
    __builtin_amdgcn_sched_barrier(0);
    float* sums = reinterpret_cast<float*>(lds);
    constexpr int kStep = D * kStage / 4;
#pragma unroll
    for (int c = 0; c < CT; ++c) {
        asm volatile("" : "+v"(acc[c]));
        *reinterpret_cast<f32x4*>(sums + wave * kStep + (16 * c + l) * 16 + 4 * q) = acc[c];
    }
    __syncthreads();
    finish_tokens<T, CT, W, PAIRED>(t, sums, kStep, n0, most);
}

template <class T, int CT, int D, bool PAIRED>
void launch_stream(int tiles, const FewArgs& t, hipStream_t stream) {
    // one workgroup of eight wavefronts to a CU, or two of four where there are more tiles than CUs
    if (tiles <= 256)
        hipLaunchKernelGGL((few_stream_kernel<T, CT, 8, D, PAIRED>), dim3(tiles), dim3(8 * MOE_WAVE), 0, stream, t);
    else
        hipLaunchKernelGGL((few_stream_kernel<T, CT, 4, D, PAIRED>), dim3(tiles), dim3(4 * MOE_WAVE), 0, stream, t);
}

template <class T, bool PAIRED>
moe_status launch_tokens(bool aligned, const Product& p, const Epilogue& e, hipStream_t stream) {
    const int width = PAIRED ? 8 : 16, columns = PAIRED ? p.inter : p.n, tiles = (columns + width - 1) / width;
    const dim3 grid(tiles), block(kFewWaves * MOE_WAVE);
    const FewArgs t{p, e};
    switch ((p.m + 15) / 16 + (aligned ? 0 : 4)) {
        case 1: launch_stream<T, 1, 4, PAIRED>(tiles, t, stream); break;
        case 2: launch_stream<T, 2, 3, PAIRED>(tiles, t, stream); break;
        case 3: launch_stream<T, 3, 2, PAIRED>(tiles, t, stream); break;
        case 4: launch_stream<T, 4, 2, PAIRED>(tiles, t, stream); break;
        case 5: hipLaunchKernelGGL((few_kernel<T, 1, PAIRED>), grid, block, 0, stream, t); break;
        case 6: hipLaunchKernelGGL((few_kernel<T, 2, PAIRED>), grid, block, 0, stream, t); break;
        case 7: hipLaunchKernelGGL((few_kernel<T, 3, PAIRED>), grid, block, 0, stream, t); break;
        case 8: hipLaunchKernelGGL((few_kernel<T, 4, PAIRED>), grid, block, 0, stream, t); break;
        default: return MOE_ERR_UNSUPPORTED;
    }
    return launch_status();
}

}  // namespace

moe_status launch_few(int dtype, bool aligned, const Product& p, const Epilogue& e, hipStream_t stream) {
    if (dtype == MOE_BF16)
        return p.inter ? launch_tokens<__bf16, true>(aligned, p, e, stream) : launch_tokens<__bf16, false>(aligned, p, e, stream);
    return p.inter ? launch_tokens<_Float16, true>(aligned, p, e, stream) : launch_tokens<_Float16, false>(aligned, p, e, stream);
}

}  // namespace moe
