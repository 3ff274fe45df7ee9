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
// unit four times as long, and fewer are in flight.  Gated 1 x 7168 -> 2 x 2048 11.0 us (5.3 TB/s of weights), 1 x 8192 ->
// 8192 28.6 us (4.7 TB/s, what a large copy reaches is 5.1); a call of a few microseconds is bound by its launch and by the
// first bytes' way from memory (1 x 2048 -> 7168 8.5 us, 3.5 TB/s).
#include "dense.h"

namespace moe {
namespace {

struct FewArgs {
    Product p;
    Epilogue e;
};

// The sums of the wavefronts, [wavefront][row tile][token][weight row] at `sums` + wavefront * step, through the epilogue.
template <class T, int CT, int R, int W, bool PAIRED>
__device__ __forceinline__ void finish_tokens(const FewArgs& t, const float* sums, int step, int n0, int most) {
    constexpr int kItems = 16 * CT * (PAIRED ? 1 : 2);       // of a row tile
    for (int i = threadIdx.x; i < R * kItems; i += W * MOE_WAVE) {
        const int tile = i / kItems, item = i % kItems;
        const int token = PAIRED ? item : item >> 1, c = PAIRED ? 0 : 8 * (item & 1), col = n0 + tile * (PAIRED ? 8 : 16) + c;
        if (token >= t.p.m || col >= most) continue;
        float v[8], u[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = u[e] = 0.0f;
#pragma unroll
        for (int wv = 0; wv < W; ++wv) {
            const float* from = sums + wv * step + (tile * 16 * CT + token) * 16 + c;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                v[e] += from[e];
                if (PAIRED) u[e] += from[8 + e];
            }
        }
        const int n = min(8, most - col);
        if constexpr (PAIRED) finish_gated<T>(t.e, token, col, v, u, n);
        else finish<T>(t.e, token, col, v, n, bias_of<T>(t.e, col, n), residual_of<T>(t.e, token, col, n));
    }
}

// Rows of whole 16-byte pieces.  W wavefronts, R row tiles each; wavefront w takes every W-th 64 of K, D of them in flight.
template <class T, int CT, int R, int W, int D, bool PAIRED>
__global__ void __launch_bounds__(W * MOE_WAVE) few_stream_kernel(FewArgs t) {
    typedef typename Vec<T>::x8 x8;
    constexpr int kStage = (R + CT) * 2048, kLoads = 2 * (R + CT);
    static_assert(W * D * kStage <= 160 * 1024 && D * kStage >= R * CT * 1024 && D * kLoads < 64, "LDS");
    __shared__ __align__(16) uint8_t lds[W * D * kStage];
    const int lane = threadIdx.x % MOE_WAVE;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / MOE_WAVE);
    const int l = lane & 15, q = lane >> 4;
    const int K = t.p.k, n0 = blockIdx.x * (PAIRED ? 8 : 16) * R, most = PAIRED ? t.p.inter : t.p.n;
    const int turns = max(0, ((K + 63) / 64 - wave + W - 1) / W);

    // eight rows to a load; lane l brings chunk l % 8 of row l / 8, by the swizzle of the sixteen rows' places
    const int chunk[2] = {(lane & 7) ^ swizzle(lane >> 3), (lane & 7) ^ swizzle(8 + (lane >> 3))};
    const T* at[kLoads];
    int bytes[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        const bool x = i >= 2 * R;
        const int row = x ? 8 * (i - 2 * R) : n0 + (PAIRED ? 8 * (i / 2) : 8 * i), rows = min(8, (x ? t.p.m : most) - row);
        const int64_t ld = x ? t.p.lda : t.p.ldb;
        at[i] = static_cast<const T*>(x ? t.p.a : t.p.b) + (row + (PAIRED && !x && i % 2 ? (int64_t)most : 0)) * ld + 64 * wave;
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
            load_to_lds<i * 1024>(at[i], bytes[i], in[i & 1] ? (i < 2 * R ? off_w : off_x)[i & 1] : kNowhere,
                                  ring + place * kStage);
            at[i] += 64 * W;
        });
        k0 += 64 * W;
    };

    f32x4 acc[R][CT];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int c = 0; c < CT; ++c) acc[r][c] = f32x4{0.f, 0.f, 0.f, 0.f};
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
        x8 wf[2][R], xf[2][CT];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
#pragma unroll
            for (int r = 0; r < R; ++r) wf[s][r] = fragment(r, s);
#pragma unroll
            for (int c = 0; c < CT; ++c) xf[s][c] = fragment(R + c, s);
        }
        __builtin_amdgcn_s_waitcnt(kWaitLds0);               // the place is read: fill it again
        __builtin_amdgcn_sched_barrier(0);
        issue(place);
        place = place + 1 == D ? 0 : place + 1;
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int c = 0; c < CT; ++c) acc[r][c] = mfma(wf[s][r], xf[s][c], acc[r][c]);
    }
    __builtin_amdgcn_s_waitcnt(wait_vm(0));
    asm volatile("s_nop 15" ::: "memory");                   // the wait before an MFMA's result is read
    __builtin_amdgcn_sched_barrier(0);
    float* sums = reinterpret_cast<float*>(lds);
    constexpr int kStep = D * kStage / 4;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int c = 0; c < CT; ++c) {
            asm volatile("" : "+v"(acc[r][c]));
            *reinterpret_cast<f32x4*>(sums + wave * kStep + (r * 16 * CT + 16 * c + l) * 16 + 4 * q) = acc[r][c];
        }
    __syncthreads();
    finish_tokens<T, CT, R, W, PAIRED>(t, sums, kStep, n0, most);
}

// Up to 16 rows that start anywhere, of eight elements and more: the same through registers, P turns ahead.  A piece that
// runs over its row's end is fetched from eight elements before the end and shifted to its place, zeros behind it, on its
// way to LDS.  1 x 8192 -> 8192 34 us (4.0 TB/s), 8 rows 43 us: an unaligned piece touches two lines.
template <class T, int W, int P, bool PAIRED>
__global__ void __launch_bounds__(W * MOE_WAVE) few_anywhere_kernel(FewArgs t) {
    typedef typename Vec<T>::x8 x8;
    typedef uint64_t u64x2 __attribute__((ext_vector_type(2)));
    constexpr int kStage = 4096, kLoads = 4;
    __shared__ __align__(16) uint8_t lds[W * kStage];
    const int lane = threadIdx.x % MOE_WAVE;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / MOE_WAVE);
    const int l = lane & 15, q = lane >> 4;
    const int K = t.p.k, n0 = blockIdx.x * (PAIRED ? 8 : 16), most = PAIRED ? t.p.inter : t.p.n;
    const int turns = max(0, ((K + 63) / 64 - wave + W - 1) / W);

    // rows past the end are the last one again: what they give is not stored
    const T* row[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        const bool x = i >= 2;
        const int r = (x ? 8 * (i - 2) : n0 + (PAIRED ? 0 : 8 * i)) + (lane >> 3);
        const int64_t at = min(r, (x ? t.p.m : most) - 1) + (PAIRED && i == 1 ? (int64_t)most : 0);
        row[i] = static_cast<const T*>(x ? t.p.a : t.p.b) + at * (x ? t.p.lda : t.p.ldb);
    }
    const int chunk[2] = {(lane & 7) ^ swizzle(lane >> 3), (lane & 7) ^ swizzle(8 + (lane >> 3))};
    u64x2 held[P][kLoads];
    auto fetch = [&](u64x2 (&to)[kLoads], int turn) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            __builtin_memcpy(&to[i], row[i] + min(64 * (wave + W * turn) + 8 * chunk[i & 1], K - 8), 16);
    };
    uint8_t* stage = lds + wave * kStage;
    auto put = [&](const u64x2 (&from)[kLoads], int turn) __attribute__((always_inline)) {
        const int k0 = 64 * (wave + W * turn);
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            u64x2 v = from[i];
            if (k0 + 64 > K) {
                const int by = 16 * max(k0 + 8 * chunk[i & 1] - (K - 8), 0);
                v = u64x2{by < 64 ? v.x >> by | (by ? v.y << (64 - by) : 0) : by < 128 ? v.y >> (by - 64) : 0,
                          by < 64 ? v.y >> by : 0};
            }
            *reinterpret_cast<u64x2*>(stage + i * 1024 + lane * 16) = v;
        }
    };
    f32x4 acc{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int p = 0; p < P; ++p) fetch(held[p], p);           // past the end of K: eight elements that are there
    for (int base = 0; base < turns; base += P) {
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const int turn = base + p;
            if (turn >= turns) break;
            put(held[p], turn);
            fetch(held[p], turn + P);
            auto fragment = [&](int tile, int s) __attribute__((always_inline)) {
                return *reinterpret_cast<const x8*>(stage + tile * 2048 + l * 128 + (((4 * s + q) ^ swizzle(l)) << 4));
            };
#pragma unroll
            for (int s = 0; s < 2; ++s) acc = mfma(fragment(0, s), fragment(1, s), acc);
        }
    }
    asm volatile("s_nop 15" ::: "memory");                   // the wait before an MFMA's result is read
    __builtin_amdgcn_sched_barrier(0);
    float* sums = reinterpret_cast<float*>(lds);
    constexpr int kStep = kStage / 4;
    asm volatile("" : "+v"(acc));
    *reinterpret_cast<f32x4*>(sums + wave * kStep + l * 16 + 4 * q) = acc;
    __syncthreads();
    finish_tokens<T, 1, 1, W, PAIRED>(t, sums, kStep, n0, most);
}

template <class T, int CT, int R, int W, int D, bool PAIRED>
void launch_stream_as(int tiles, const FewArgs& t, hipStream_t stream) {
    hipLaunchKernelGGL((few_stream_kernel<T, CT, R, W, D, PAIRED>), dim3((tiles + R - 1) / R), dim3(W * MOE_WAVE), 0, stream, t);
}
// One workgroup of eight wavefronts to a CU, or two of four where there are more tiles than CUs.  Where every CU gets four
// tiles and more and there are more than 16 tokens, a workgroup takes four: it reads the tokens once for all of them (64 x
// 2048 -> 32768 37 us, with a tile each 49; 17 tokens 32.7 and 33.0; one token 32 and 29).  Two, with two and more to a CU,
// pay off for more than 48 tokens (8192 -> 8192: 64 tokens 39.5 us and 44.5, 33 tokens 36.5 and 36.2).
template <class T, int CT, bool PAIRED>
void launch_stream(int tiles, const FewArgs& t, hipStream_t stream) {
    constexpr int kD = CT == 1 ? 4 : CT == 2 ? 3 : 2;
    if constexpr (CT >= 2)
        if (tiles >= 1024) return launch_stream_as<T, CT, 4, 4, CT == 2 ? 3 : 2, PAIRED>(tiles, t, stream);
    if constexpr (CT == 4)
        if (tiles >= 512) return launch_stream_as<T, CT, 2, 4, 3, PAIRED>(tiles, t, stream);
    if (tiles <= 256) launch_stream_as<T, CT, 1, 8, kD, PAIRED>(tiles, t, stream);
    else launch_stream_as<T, CT, 1, 4, kD, PAIRED>(tiles, t, stream);
}

template <class T, bool PAIRED>
moe_status launch_tokens(bool aligned, const Product& p, const Epilogue& e, hipStream_t stream) {
    const int width = PAIRED ? 8 : 16, columns = PAIRED ? p.inter : p.n, tiles = (columns + width - 1) / width;
    const FewArgs t{p, e};
    switch ((p.m + 15) / 16 + (aligned ? 0 : 4)) {
        case 1: launch_stream<T, 1, PAIRED>(tiles, t, stream); break;
        case 2: launch_stream<T, 2, PAIRED>(tiles, t, stream); break;
        case 3: launch_stream<T, 3, PAIRED>(tiles, t, stream); break;
        case 4: launch_stream<T, 4, PAIRED>(tiles, t, stream); break;
        case 5: hipLaunchKernelGGL((few_anywhere_kernel<T, 8, 4, PAIRED>), dim3(tiles), dim3(8 * MOE_WAVE), 0, stream, t); break;
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
