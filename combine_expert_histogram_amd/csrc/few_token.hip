// The serving forms for a few tokens: the matrix-vector products over block-scaled weights (moe_matvec) and the
// whole expert layer in two launches (moe_few_token_layer).  Both stream the weights once through the loop of
// weight_stream.h; everything else (tokens, ids, intermediate rows) stays in cache.
#include "weight_stream.h"

#include <cmath>
#include <type_traits>

namespace {

using namespace moe;

constexpr int kWaves = 8;                  // wavefronts of a workgroup; they split the K blocks
constexpr int kThreads = kWaves * MOE_WAVE;
// K blocks a wavefront keeps in flight, and the wavefronts of a SIMD that its registers allow: two workgroups to a CU
// hide each other's latencies (int4, groups of 128, 16 tokens: 99.7 -> 80.1 us for the gate and up products), which
// one column tile allows unless an int4 format carries two or four scale groups a block: under that limit their loops
// would keep up to 52 and 158 registers of a lane in scratch memory.  A few kernels keep some there within the limits
// taken: matvec e4m3 with four row and four column tiles 6 (16384 x 7168, 64 tokens: 39 us, against 46 with two row
// tiles and none), gate_up int4 in groups of 32 with four row tiles 2, and the down kernels named at down_waves.
constexpr int depth_of(int FMT, int R, int CT, int XT) {
    if (CT > 1) return 1;
    if (R == 4) return FMT == MOE_W_E2M1_MX && XT < 16 ? 2 : 1;
    return R == 2 || XT == 16 ? 2 : 4;
}
constexpr int waves_per_simd(int FMT, int G, int CT) { return CT == 1 && G == 1 ? 4 : 2; }
constexpr int kChunk = 64;                 // tokens a layer launch handles: one lane each, four column tiles
constexpr int kMaxTopK = 64;
constexpr int kMaxLocal = 1024;

__device__ __forceinline__ int wave_index() { return __builtin_amdgcn_readfirstlane(threadIdx.x / MOE_WAVE); }

// Sums the wavefronts' partial tiles (fixed order): element at (r * CT + c, lane).
template <int NW, int N>
__device__ __forceinline__ f32x4 sum_waves(const f32x4 (&red)[NW][N], int at) {
    f32x4 s = red[0][at];
#pragma unroll
    for (int w = 1; w < NW; ++w) s += red[w][at];
    return s;
}

__device__ __forceinline__ void store4(uint16_t* p, f32x4 v) {
    *reinterpret_cast<u32x2*>(p) = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
}

// acc += blocks [0, n) that load(step) brings, depth_of of them in flight; load returns block_product's cols, and done()
// follows each block.
template <int FMT, int G, int R, int CT, int XT, class Load, class Done>
__device__ __forceinline__ void stream_blocks(int n, Load&& load, u32x4* corner, f32x4 (&acc)[R][CT], Done&& done) {
    constexpr int kDepth = depth_of(FMT, R, CT, XT);
    Step<FMT, G, R, CT, XT> st[kDepth];
    uint32_t cols[kDepth];
#pragma unroll
    for (int u = 0; u < kDepth; ++u)
        if (u < n) cols[u] = load(st[u]);
    for (int i = 0; i < n; i += kDepth) {
#pragma unroll
        for (int u = 0; u < kDepth; ++u) {
            if (i + u < n) {
                block_product<FMT, G, R, CT, XT>(st[u], cols[u], corner, acc);
                done();
                if (i + u + kDepth < n) cols[u] = load(st[u]);
            }
        }
    }
}

// ---------------------------------------------------------------- y = x W^T
// A workgroup takes 16 R rows, its eight wavefronts an eighth of K each (so that one token against 4096 rows still
// fills the CUs), and adds their sums through LDS in a fixed order.  Bound by the weight stream where the matrix is
// large (the figures are in weight_stream.h), by a launch and one or two round trips to memory where it is small: one
// token, 7168 x 2048 e2m1 3.8 us, 4096 x 7168 e2m1 6.1 us (2.5 TB/s).
template <int FMT, int G, int R, int CT, int XT>
__global__ void __launch_bounds__(kThreads, waves_per_simd(FMT, G, CT))
matvec_kernel(WView w, const uint16_t* __restrict__ x, int64_t ldx, int M, uint16_t* __restrict__ y, int64_t ldy) {
    __shared__ f32x4 red[kWaves][R * CT * 64];
    __shared__ u32x4 corner[kWaves][kCorner];
    const int lane = lane_id(), wave = wave_index();
    const int64_t row0 = (int64_t)blockIdx.x * (16 * R);
    const int64_t col0 = (int64_t)blockIdx.y * (XT * CT);
    const int ncols = (int)min<int64_t>(M - col0, XT * CT);

    // rows past n repeat the last ones and are not stored
    const Tiles<FMT, G, R> tiles = tiles_of<FMT, G, R>(
        w, [&](int t, int i) { return min(row0 + 16 * t + i, w.n - 1); },
        [&](int t, int i) { return min(row0 + 16 * t + 4 * i, w.n - 4); });
    const __amdgpu_buffer_rsrc_t xb =
        row_buffer(x + col0 * ldx, (uint32_t)(((int64_t)(ncols - 1) * ldx + (int64_t)w.nb * kKBlock) * 2));
    uint32_t xrow[CT];
    uint32_t cols = 0;
#pragma unroll
    for (int c = 0; c < CT; ++c) {
        const int t = XT * c + token_of_lane<XT>();
        xrow[c] = t < ncols ? (uint32_t)(t * ldx * 2) : kNoRow;
        if (XT * c < ncols) cols |= 1u << c;
    }

    f32x4 acc[R][CT] = {};
    int kb = w.nb * wave / kWaves;
    const int n = w.nb * (wave + 1) / kWaves - kb;
    stream_blocks<FMT, G, R, CT, XT>(n, [&](Step<FMT, G, R, CT, XT>& st) {
        load_weights<FMT, G, R>(tiles, w, kb, st.w, st.s);
#pragma unroll
        for (int c = 0; c < CT; ++c)
            if (CT == 1 || (cols >> c & 1)) load_rows<FMT, G, XT>(xb, xrow[c], kb, st.x[c]);
        ++kb;
        return cols;
    }, corner[wave], acc, [] {});

#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int c = 0; c < CT; ++c) red[wave][(r * CT + c) * 64 + lane] = acc[r][c];
    __syncthreads();
    for (int at = threadIdx.x; at < R * CT * 64; at += kThreads) {
        const int r = at / (64 * CT), c = at / 64 % CT, l = at & 63;
        const int64_t row = row0 + 16 * r + 4 * (l >> 4);
        const int t = XT * c + (l & 15) / (16 / XT);
        if ((l & 15) % (16 / XT)) continue;              // a repeated column
        if (t < ncols && row < w.n) store4(y + (col0 + t) * ldy + row, sum_waves(red, at));
    }
}

// More than sixteen tokens against many rows: here the tokens' values are the larger stream (sixteen rows of 64 tokens
// read 16 KiB of them beside 1 or 2 KiB of weights), so the eight wavefronts share them.  Each takes 16 R rows over the
// whole of K; a block's token values go through LDS once (two buffers, one barrier a block), and the weights of two
// blocks are in flight in registers.  64 tokens, 131072 x 7168 e2m1: 136 to 146 us, 0.85 PFLOP/s (a large library
// product reaches 1.26), at 2.0 to 2.1 GHz.  No unit is the limit by itself (matrix cores 0.40 busy, LDS 0.35, loads
// 0.54): a block's turn, token reads and products follow each other, with a barrier for the workgroup.  65536 x 7168 e4m3
// 106 to 110 us, 4.4 TB/s; 131072 x 7168 int4 206 to 214 (groups of 128), 316 (of 32).
template <int FMT, int G, int R, int CT>
__global__ void __launch_bounds__(kThreads)
matvec_wide_kernel(WView w, const uint16_t* __restrict__ x, int64_t ldx, int M, uint16_t* __restrict__ y, int64_t ldy) {
    using F = Fmt<FMT, G>;
    constexpr int kPieces = CT * 16 * 16;                    // 16 B pieces of a block's token values
    constexpr int kMine = kPieces / kThreads;
    __shared__ u32x4 xs[2][kPieces];
    __shared__ u32x4 corner[kWaves][kCorner];
    const int lane = lane_id(), wave = wave_index();
    const int64_t row0 = ((int64_t)blockIdx.x * kWaves + wave) * (16 * R);
    const int64_t col0 = (int64_t)blockIdx.y * (16 * CT);
    const int ncols = (int)min<int64_t>(M - col0, 16 * CT);

    // rows past n repeat the last ones and are not stored
    const Tiles<FMT, G, R> tiles = tiles_of<FMT, G, R>(
        w, [&](int t, int i) { return min(row0 + 16 * t + i, w.n - 1); },
        [&](int t, int i) { return min(row0 + 16 * t + 4 * i, w.n - 4); });
    const __amdgpu_buffer_rsrc_t xb =
        row_buffer(x + col0 * ldx, (uint32_t)(((int64_t)(ncols - 1) * ldx + (int64_t)w.nb * kKBlock) * 2));
    uint32_t at[kMine];                                      // piece p of token t
    int to[kMine];
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
        const int id = threadIdx.x + kThreads * i, t = id >> 4, p = id & 15;
        at[i] = t < ncols ? (uint32_t)(t * ldx * 2 + 16 * p) : kNoRow;
        to[i] = t * 16 + (p ^ shared_swizzle<FMT>(t & 15));
    }
    u32x4 xr[kMine];
    const auto load_x = [&](int kb) {
#pragma unroll
        for (int i = 0; i < kMine; ++i)
            xr[i] = __builtin_amdgcn_raw_buffer_load_b128(xb, at[i], kb * (2 * kKBlock), 0);
    };
    const auto put_x = [&](int buf) {
#pragma unroll
        for (int i = 0; i < kMine; ++i) xs[buf][to[i]] = xr[i];
    };

    u32x4 wr[2][R][F::kLoads];
    Scales<FMT, G> sc[2];
    load_x(0);
    load_weights<FMT, G, R>(tiles, w, 0, wr[0], sc[0]);
    put_x(0);
    if (w.nb > 1) {
        load_weights<FMT, G, R>(tiles, w, 1, wr[1], sc[1]);
        load_x(1);
    }
    lds_barrier();
    f32x4 acc[R][CT] = {};
    for (int kb0 = 0; kb0 < w.nb; kb0 += 2) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int kb = kb0 + u;
            if (kb >= w.nb) break;
            turn_weights<FMT, G, R>(corner[wave], wr[u]);
            u32x4 wt[R][F::kLoads];
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int p = 0; p < F::kLoads; ++p) wt[r][p] = wr[u][r][p];
            const Scales<FMT, G> s = sc[u];
            if (kb + 2 < w.nb) load_weights<FMT, G, R>(tiles, w, kb + 2, wr[u], sc[u]);
            if (kb + 1 < w.nb) put_x(1 - u);
            if (kb + 2 < w.nb) load_x(kb + 2);
            shared_product<FMT, G, R, CT>(wt, s, xs[u], acc);
            // block kb's tokens are read and block kb + 1's are written, on both sides of it
            lds_barrier();
        }
    }
#pragma unroll
    for (int c = 0; c < CT; ++c) {
        const int t = 16 * c + (lane & 15);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t row = row0 + 16 * r + 4 * (lane >> 4);
            if (t < ncols && row < w.n) store4(y + (col0 + t) * ldy + row, acc[r][c]);
        }
    }
}

// ---------------------------------------------------------------- the layer
struct LayerArgs {
    const uint16_t* x;           // [T, H]
    const int32_t* ids;          // [T, k]
    const float* topk_w;         // [T, k]
    uint16_t* h;                 // [T * k, I], the workspace
    uint16_t* out;               // [T, H]
    int T, k, e0, L, H, I;       // T <= kChunk
};

// The set of local experts that the tokens name, as bits in LDS (cleared before; every thread calls; ends in a barrier).
__device__ __forceinline__ void expert_set(const LayerArgs& a, const int32_t* ids, uint32_t (&bits)[kMaxLocal / 32]) {
    for (int i = threadIdx.x; i < a.T * a.k; i += kThreads) {
        const int64_t e = (int64_t)ids[i] - a.e0;
        if (e >= 0 && e < a.L) atomicOr(&bits[e >> 5], 1u << (e & 31));
    }
    __syncthreads();
}

__device__ __forceinline__ int expert_count(const uint32_t (&bits)[kMaxLocal / 32]) {
    const int l = lane_id();
    return __builtin_amdgcn_readfirstlane(wave_sum(l < kMaxLocal / 32 ? __popc(bits[l]) : 0));
}

// The n-th expert of the set (n < expert_count), uniform.
__device__ __forceinline__ int nth_expert(const uint32_t (&bits)[kMaxLocal / 32], int n) {
    const int l = lane_id();
    const uint32_t mine = l < kMaxLocal / 32 ? bits[l] : 0;
    const int upto = wave_inclusive_scan(__popc(mine));
    const int word = __ffsll((unsigned long long)__ballot(upto > n)) - 1;
    uint32_t b = (uint32_t)__builtin_amdgcn_readlane((int)mine, word);
    int skip = n - (__builtin_amdgcn_readlane(upto, word) - __popc(b));
    for (; skip > 0; --skip) b &= b - 1;
    return word * 32 + __ffs(b) - 1;
}

template <int FMT, int G>
__device__ __forceinline__ WView expert_view(const WView& w, int e) {
    using F = Fmt<FMT, G>;
    WView v = w;
    v.data += (int64_t)e * w.n * w.nb * F::kRowBytes;
    const int64_t blocks = (int64_t)e * w.n * w.nb;
    if constexpr (F::kInt4) {
        v.scale = static_cast<const uint8_t*>(w.scale) + blocks * 2 * G;
        if (w.zero) v.zero = w.zero + blocks * G;
    } else if constexpr (F::kMx) {
        v.scale = static_cast<const uint8_t*>(w.scale) + blocks * 4;
    } else {
        v.scale = static_cast<const uint8_t*>(w.scale) + blocks / 128 * 4;
    }
    return v;
}

// The tokens that name local expert e, as bits (lane t looks at token t's ids in LDS); first: this lane's first slot.
__device__ __forceinline__ uint64_t tokens_of(const LayerArgs& a, const int32_t* ids, int e, int& first) {
    const int t = lane_id();
    first = -1;
    if (t < a.T)
        for (int j = a.k - 1; j >= 0; --j)
            if (ids[t * a.k + j] == a.e0 + e) first = j;
    return __ballot(first >= 0);
}

// First launch: h[t k + j] = w (silu(gate) up) in bf16, for the first slot j in which token t names the expert, w
// the sum of the token's weights for it.  A workgroup takes 8 R columns of h of one expert: a tile's sixteen weight
// rows are eight gate rows and the eight up rows that go with them.  The rounding of h to bf16 is the matrix
// instruction's input type; it is of the size of the output's own (a layer is off by 2.35e-3 of its size against 64
// bits, by 1.66e-3 with h in fp32).  The hardware exponential is off by a few 2^-24 and |gate| 2^-24, far below that.
// One token, 8 experts of 2 x 2048 x 7168 e2m1: 27.8 us, 4.5 TB/s, of which the start (launch, ids, lists, first round
// trip) is about 8; 64 tokens, 28 experts e4m3: 120 to 138 us, 6 TB/s.  An expert that every token names takes its passes
// one after the other in its own workgroups (that layer with one such expert: 209 -> 244 us; int4 of 128 152 -> 198).
template <int FMT, int G, int R, int CT, int XT>
__global__ void __launch_bounds__(kThreads, waves_per_simd(FMT, G, CT))
gate_up_kernel(WView w, LayerArgs a) {
    __shared__ f32x4 red[kWaves][R * CT * 64];
    __shared__ u32x4 corner[kWaves][kCorner];
    __shared__ uint32_t bits[kMaxLocal / 32];
    __shared__ int32_t tok[kWaves][kChunk], slot[kChunk];
    __shared__ float wt[kChunk];
    extern __shared__ int32_t ids[];         // [T * k], then the weights
    float* const tw = reinterpret_cast<float*>(ids + a.T * a.k);
    if (threadIdx.x < kMaxLocal / 32) bits[threadIdx.x] = 0;
    for (int i = threadIdx.x; i < a.T * a.k; i += kThreads) {
        ids[i] = a.ids[i];
        tw[i] = a.topk_w[i];
    }
    __syncthreads();
    expert_set(a, ids, bits);
    if ((int)blockIdx.y >= expert_count(bits)) return;
    const int e = nth_expert(bits, blockIdx.y);
    const int lane = lane_id(), wave = wave_index();

    int first;
    const uint64_t here = tokens_of(a, ids, e, first);
    const int ncols = __popcll(here);
    if (first >= 0) {                        // each wavefront its own list: no barrier before the stream
        const int at = __popcll(here & lanemask_lt());
        tok[wave][at] = lane;
        if (wave == 0) {
            float sum = 0.f;
            for (int j = first; j < a.k; ++j)
                if (ids[lane * a.k + j] == a.e0 + e) sum += tw[lane * a.k + j];
            slot[at] = lane * a.k + first, wt[at] = sum;
        }
    }
    __builtin_amdgcn_wave_barrier();         // one wavefront's LDS accesses stay in order

    const WView v = expert_view<FMT, G>(w, e);
    const int i0 = blockIdx.x * (8 * R);
    const auto row_of = [&](int t, int i) { return (i < 8 ? 0 : a.I - 8) + i0 + 8 * t + i; };
    const Tiles<FMT, G, R> tiles =
        tiles_of<FMT, G, R>(v, row_of, [&](int t, int i) { return row_of(t, 4 * i); });
    const __amdgpu_buffer_rsrc_t xb = row_buffer(a.x, (uint32_t)(a.T * a.H * 2));
    // an expert with more tokens than the column tiles hold takes further passes over the weights
    for (int col0 = 0; col0 < ncols; col0 += XT * CT) {
        uint32_t xrow[CT];
        uint32_t cols = 0;
#pragma unroll
        for (int c = 0; c < CT; ++c) {
            const int t = col0 + XT * c + token_of_lane<XT>();
            xrow[c] = t < ncols ? (uint32_t)(tok[wave][t] * a.H * 2) : kNoRow;
            if (col0 + XT * c < ncols) cols |= 1u << c;
        }

        f32x4 acc[R][CT] = {};
        int kb = v.nb * wave / kWaves;
        const int n = v.nb * (wave + 1) / kWaves - kb;
        stream_blocks<FMT, G, R, CT, XT>(n, [&](Step<FMT, G, R, CT, XT>& st) {
            load_weights<FMT, G, R>(tiles, v, kb, st.w, st.s);
#pragma unroll
            for (int c = 0; c < CT; ++c)
                if (CT == 1 || (cols >> c & 1)) load_rows<FMT, G, XT>(xb, xrow[c], kb, st.x[c]);
            ++kb;
            return cols;
        }, corner[wave], acc, [] {});

        if (col0 > 0) __syncthreads();       // the sums of the pass before are read
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int c = 0; c < CT; ++c) red[wave][(r * CT + c) * 64 + lane] = acc[r][c];
        __syncthreads();
        for (int at = threadIdx.x; at < R * CT * 32; at += kThreads) {
            const int r = at / (32 * CT), c = at / 32 % CT, l = at & 31;     // lanes 0..31: gate rows, 32..63: up rows
            const int t = col0 + XT * c + (l & 15) / (16 / XT);
            if ((l & 15) % (16 / XT) || t >= ncols) continue;                // a repeated or an empty column
            const f32x4 gate = sum_waves(red, (r * CT + c) * 64 + l);
            const f32x4 up = sum_waves(red, (r * CT + c) * 64 + l + 32);
            f32x4 h;
#pragma unroll
            for (int i = 0; i < 4; ++i) h[i] = gate[i] / (1.0f + __expf(-gate[i])) * up[i] * wt[t];
            store4(a.h + (int64_t)slot[t] * a.I + i0 + 8 * r + 4 * (l >> 4), h);
        }
    }
}

// The passes over the experts' weights that the tokens need, XT tokens each, in the experts' order: segs[i] holds expert
// and pass.  A token that names an expert twice counts twice and may leave a pass without tokens.  Every thread calls;
// ends in a barrier.  Returns their number.
constexpr uint32_t seg_expert(uint32_t s) { return s & 0xFFFFu; }
constexpr uint32_t seg_pass(uint32_t s) { return s >> 16; }

template <int XT, int NW>
__device__ __forceinline__ int list_passes(const LayerArgs& a, const int32_t* ids, uint32_t* segs) {
    __shared__ int32_t count[kMaxLocal];
    __shared__ int32_t before[NW];
    constexpr int kMine = kMaxLocal / (NW * MOE_WAVE);       // experts of a thread
    const int tid = threadIdx.x, wave = wave_index();
#pragma unroll
    for (int i = 0; i < kMine; ++i) count[kMine * tid + i] = 0;
    __syncthreads();
    for (int i = tid; i < a.T * a.k; i += NW * MOE_WAVE) {
        const int64_t e = (int64_t)ids[i] - a.e0;
        if (e >= 0 && e < a.L) atomicAdd(&count[e], 1);
    }
    __syncthreads();
    int passes[kMine], mine = 0;
#pragma unroll
    for (int i = 0; i < kMine; ++i) mine += passes[i] = (count[kMine * tid + i] + XT - 1) / XT;
    const int upto = wave_inclusive_scan(mine);
    if (lane_id() == MOE_WAVE - 1) before[wave] = upto;
    __syncthreads();
    int at = upto - mine, total = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
        if (w < wave) at += before[w];
        total += before[w];
    }
#pragma unroll
    for (int i = 0; i < kMine; ++i)
        for (int p = 0; p < passes[i]; ++p) segs[at++] = (uint32_t)(kMine * tid + i) | (uint32_t)p << 16;
    __syncthreads();
    return __builtin_amdgcn_readfirstlane(total);
}

// Wavefronts of a down workgroup.  One row tile is taken where the rows give every CU only one workgroup, which then
// needs sixteen to hide a block's latency (4096 rows, int4, 16 tokens: 52.4 us with eight, 42.4 with sixteen; with two
// row tiles both take the same); more scale groups would spill (up to 39 and 147 registers a lane) and four output tiles
// would not fit LDS.  Three of the kernels at 128 registers keep 2 to 7 in scratch memory.  Those with two row tiles and
// sixteen tokens' columns would be a little faster at two wavefronts a SIMD without (the layer, 16 tokens, 4 of 8
// experts, H = 7168: e4m3 71.2 against 69.5 us, int4 58.4 against 55.8); int4 with one row tile and eight takes the same
// either way (24 tokens, H = 4096: 65.3, with eight wavefronts 65.4).
constexpr int down_waves(int G, int R, int OT) { return R == 1 && OT <= 2 && G == 1 ? 16 : 8; }

// Second launch: out[t] = sum over the experts of W2[e] h[t, e], one long product whose K runs over the experts hit
// (each wavefront takes a run of it).  An expert's tokens sit in compact columns, so that the few tokens that an
// expert has take few loads; at the expert's end their sums move to the columns of the tokens (a lane permutation
// within the wavefront), which keeps the sum over experts in registers and its order fixed.  OT tiles of 16 tokens.
// One token, 8 experts of 7168 x 2048 e2m1: 17.4 us, 3.6 TB/s, about 7 of them the start; 64 tokens, 28 experts e4m3:
// 61 to 70 us, 6 TB/s (token columns instead of compact ones: 127).
template <int FMT, int G, int R, int XT, int OT, int NW>
__global__ void __launch_bounds__(NW * MOE_WAVE, waves_per_simd(FMT, G, OT > 2 || OT * XT > 16 ? OT : 1))
down_kernel(WView w, LayerArgs a) {
    __shared__ f32x4 red[NW][R * OT * 64];
    __shared__ u32x4 corner[NW][kCorner];
    __shared__ int32_t rows[NW][kChunk];
    extern __shared__ int32_t ids[];         // [T * k], then as many passes
    uint32_t* const segs = reinterpret_cast<uint32_t*>(ids + a.T * a.k);
    for (int i = threadIdx.x; i < a.T * a.k; i += NW * MOE_WAVE) ids[i] = a.ids[i];
    __syncthreads();
    const int64_t total = (int64_t)list_passes<XT, NW>(a, ids, segs) * w.nb;
    const int lane = lane_id(), wave = wave_index(), g = lane >> 4;
    const int row0 = blockIdx.x * (16 * R);
    const int64_t f0 = total * wave / NW;
    const int n = (int)(total * (wave + 1) / NW - f0);

    const __amdgpu_buffer_rsrc_t hb = row_buffer(a.h, (uint32_t)(a.T * a.k * a.I * 2));
    int seg = (int)(f0 / w.nb), kb = (int)(f0 % w.nb);       // of the next block to load
    int done_seg = seg, done_kb = kb;                        // of the next one to finish
    WView v = w;
    Tiles<FMT, G, R> tiles;
    uint32_t hrow[1];
    const auto enter = [&] {                 // this lane's rows and column of a pass
        const uint32_t s = __builtin_amdgcn_readfirstlane(segs[seg]);
        v = expert_view<FMT, G>(w, seg_expert(s));
        tiles = tiles_of<FMT, G, R>(
            v, [&](int t, int i) { return row0 + 16 * t + i; }, [&](int t, int i) { return row0 + 16 * t + 4 * i; });
        int first;
        const uint64_t here = tokens_of(a, ids, seg_expert(s), first);
        if (first >= 0) rows[wave][__popcll(here & lanemask_lt())] = lane * a.k + first;
        __builtin_amdgcn_wave_barrier();     // one wavefront's LDS accesses stay in order
        const int c = (int)seg_pass(s) * XT + token_of_lane<XT>();
        hrow[0] = c < __popcll(here) ? (uint32_t)(rows[wave][c] * a.I * 2) : kNoRow;
    };
    f32x4 acc[R][1] = {}, out[R][OT] = {};
    const auto leave = [&] {                 // the pass's columns to the tokens'
        const uint32_t s = __builtin_amdgcn_readfirstlane(segs[done_seg]);
        int first;
        const uint64_t here = tokens_of(a, ids, seg_expert(s), first);
#pragma unroll
        for (int o = 0; o < OT; ++o) {
            if (OT > 1 && (here >> (16 * o) & 0xFFFFu) == 0) continue;
            const int t = 16 * o + (lane & 15);
            const int c = __popcll(here & ((1ull << t) - 1)) - (int)seg_pass(s) * XT;
            const bool mine = (here >> t & 1) && c >= 0 && c < XT;
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float f = __shfl(acc[r][0][i], c * (16 / XT) + 16 * g, MOE_WAVE);
                    out[r][o][i] += mine ? f : 0.f;
                }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) acc[r][0] = f32x4{0.f, 0.f, 0.f, 0.f};
    };
    if (n > 0) enter();
    stream_blocks<FMT, G, R, 1, XT>(n, [&](Step<FMT, G, R, 1, XT>& st) {
        if (kb == w.nb) {
            kb = 0;
            ++seg;
            enter();
        }
        load_weights<FMT, G, R>(tiles, v, kb, st.w, st.s);
        load_rows<FMT, G, XT>(hb, hrow[0], kb, st.x[0]);
        ++kb;
        return 1u;
    }, corner[wave], acc, [&] {
        if (++done_kb < w.nb) return;
        leave();
        done_kb = 0;
        ++done_seg;
    });
    if (n > 0 && done_kb > 0) leave();

#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int o = 0; o < OT; ++o) red[wave][(r * OT + o) * 64 + lane] = out[r][o];
    __syncthreads();
    for (int at = threadIdx.x; at < R * OT * 64; at += NW * MOE_WAVE) {
        const int r = at / (64 * OT), o = at / 64 % OT, l = at & 63;
        const int t = 16 * o + (l & 15);
        if (t < a.T) store4(a.out + (int64_t)t * a.H + row0 + 16 * r + 4 * (l >> 4), sum_waves(red, at));
    }
}

// ---------------------------------------------------------------- host side
bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

// A weight descriptor for an [n, k] matrix (per expert), checked; groups = scale groups per K block for int4.
moe_status load_weight(const moe_weight* w, int64_t n, int64_t k, WView* v, int* groups) {
    if (!w || n < 4 || n % 4 != 0 || k < kKBlock || k % kKBlock != 0) return MOE_ERR_INVALID_ARG;
    *groups = 1;
    switch (w->format) {
        case MOE_W_E4M3:
            if (n % 128 != 0) return MOE_ERR_INVALID_ARG;
            break;
        case MOE_W_E4M3_MX:
        case MOE_W_E2M1_MX: break;
        case MOE_W_INT4:
            if (w->group != 32 && w->group != 64 && w->group != 128) return MOE_ERR_INVALID_ARG;
            *groups = kKBlock / w->group;
            break;
        default: return MOE_ERR_INVALID_ARG;
    }
    if (w->format != MOE_W_INT4 && w->zero) return MOE_ERR_INVALID_ARG;
    if (!w->data || !w->scale) return MOE_ERR_INVALID_ARG;
    if (!aligned(w->data, 16) || !aligned(w->scale, 16) || !aligned(w->zero, 16)) return MOE_ERR_INVALID_ARG;
    v->data = static_cast<const uint8_t*>(w->data);
    v->scale = w->scale;
    v->zero = w->zero;
    v->n = n;
    v->nb = (int)(k / kKBlock);
    return MOE_OK;
}

template <class F>
moe_status with_format(int format, int groups, F&& f) {
    switch (format) {
        case MOE_W_E4M3: return f(std::integral_constant<int, MOE_W_E4M3>{}, std::integral_constant<int, 1>{});
        case MOE_W_E4M3_MX: return f(std::integral_constant<int, MOE_W_E4M3_MX>{}, std::integral_constant<int, 1>{});
        case MOE_W_E2M1_MX: return f(std::integral_constant<int, MOE_W_E2M1_MX>{}, std::integral_constant<int, 1>{});
        default: break;
    }
    if (groups == 1) return f(std::integral_constant<int, MOE_W_INT4>{}, std::integral_constant<int, 1>{});
    if (groups == 2) return f(std::integral_constant<int, MOE_W_INT4>{}, std::integral_constant<int, 2>{});
    return f(std::integral_constant<int, MOE_W_INT4>{}, std::integral_constant<int, 4>{});
}

// Calls f(column tiles, tokens of a tile) for the tokens of a launch.
template <class F>
void with_cols(int64_t tokens, F&& f) {
    if (tokens <= 4) f(std::integral_constant<int, 1>{}, std::integral_constant<int, 4>{});
    else if (tokens <= 8) f(std::integral_constant<int, 1>{}, std::integral_constant<int, 8>{});
    else if (tokens <= 16) f(std::integral_constant<int, 1>{}, std::integral_constant<int, 16>{});
    else if (tokens <= 32) f(std::integral_constant<int, 2>{}, std::integral_constant<int, 16>{});
    else f(std::integral_constant<int, 4>{}, std::integral_constant<int, 16>{});
}

template <int... Rs, class F>
void with_rows(int r, F&& f) {
    ((r == Rs ? f(std::integral_constant<int, Rs>{}) : void()), ...);
}

constexpr int kCus = 256;

// Row tiles of a wavefront of the wide product, and whether it pays: its workgroups take 256 rows each and want every
// CU, while the plain form's token traffic grows with the column tiles.  us at K = 7168, plain form / wide form:
//                          16384 rows   32768 rows   65536 rows   131072 rows
//   e2m1, 24 tokens           21 / 58      39 / 60      73 / 66     142 / 108
//   e2m1, 64 tokens           29 / 67      53 / 69     101 / 79     196 / 142
//   e4m3, 24 tokens           26 / 74      49 / 77      94 / 95     187 / 164
//   e4m3, 64 tokens           39 / 90      73 / 92     143 / 110    282 / 216     (e4m3_mx: the same within 7 %)
//   int4 of 128, 24 tokens    23 / 76      42 / 76      80 / 80     156 / 135
//   int4 of 128, 64 tokens    43 / 100     82 / 100    158 / 107    311 / 214
//   int4 of 32, 24 tokens     33 / 116     63 / 117    122 / 119    239 / 235
//   int4 of 32, 64 tokens     63 / 155    122 / 157    240 / 159    475 / 316
// With four row tiles the wide form has half the LDS reads but one workgroup a CU, and takes the same (e2m1, 64 tokens,
// 131072 rows: 145 us).  Both forms step up where a workgroup more no longer fits the CUs at once (17 tokens, int4 of
// 32: 16384 rows 33 us, 16388 rows 55).
constexpr int kWideRows = 2;
constexpr int64_t kWideGroupRows = kWaves * 16 * kWideRows;
bool wide_pays(int64_t n, int64_t m) { return m > 16 && n >= kCus * kWideGroupRows; }

// Row tiles of a wavefront: the more, the fewer token loads a weight load takes beside it, as long as there is a
// workgroup for every CU.  us with 1 / 2 / 4 of them: 4096 x 7168 e2m1, 1 token: 6.2 / 7.5 / 11.6; 16384 x 4096 e2m1, 16
// tokens: - / 12.5 / 11.2; 131072 x 7168 e2m1, 16 tokens: - / 140 / 115; 16384 x 7168, 24 tokens: e2m1 33 / 24 / 21,
// e4m3 39 / 30 / 26, int4 in groups of 128 35 / 28 / 23, of 32 41 / 40 / 35; 64 tokens: e2m1 55 / 39 / 29, e4m3 66 / 46 /
// 39.  int4 takes two at most beside four column tiles: four would keep 59 to 95 registers of a lane in scratch memory
// (16384 x 7168, 64 tokens, groups of 128 / 64 / 32: one 65 / 73 / 92, two 42 / 48 / 63, four 79 / 75 / 110).
constexpr int most_rows(int FMT, int CT) { return FMT == MOE_W_INT4 && CT == 4 ? 2 : 4; }

int matvec_rows(int64_t n, int most) {
    int r = 1;
    while (r < most && n >= 16 * 2 * r * kCus) r *= 2;
    return r;
}

}  // namespace

extern "C" moe_status moe_matvec(int32_t m, int32_t n, int32_t k, const uint16_t* x_bf16, int64_t x_stride,
                                 const moe_weight* w, uint16_t* y_bf16, int64_t y_stride, void* hip_stream) {
    if (m < 0) return MOE_ERR_INVALID_ARG;
    WView v;
    int groups;
    moe_status st = load_weight(w, n, k, &v, &groups);
    if (st != MOE_OK) return st;
    if (m == 0) return MOE_OK;
    if (!x_bf16 || !y_bf16 || !aligned(x_bf16, 16) || !aligned(y_bf16, 8)) return MOE_ERR_INVALID_ARG;
    if (x_stride < k || x_stride % 8 != 0 || y_stride < n || y_stride % 4 != 0) return MOE_ERR_INVALID_ARG;
    // a workgroup's token rows are addressed with 31-bit byte offsets; the rest keeps the grid within its limits
    if (x_stride >= (1 << 24) || m > (1 << 20) || n > (1 << 27)) return MOE_ERR_UNSUPPORTED;
    hipStream_t stream = reinterpret_cast<hipStream_t>(hip_stream);
    return with_format(w->format, groups, [&](auto fmt, auto g) {
        if (wide_pays(n, m)) {
            const auto launch = [&](auto ct) {
                const dim3 grid((unsigned)((n + kWideGroupRows - 1) / kWideGroupRows),
                                (unsigned)((m + 16 * ct - 1) / (16 * ct)));
                matvec_wide_kernel<fmt, g, kWideRows, ct><<<grid, kThreads, 0, stream>>>(v, x_bf16, x_stride, m, y_bf16,
                                                                                        y_stride);
            };
            if (m <= 32) launch(std::integral_constant<int, 2>{});
            else launch(std::integral_constant<int, 4>{});
            return launch_status();
        }
        with_cols(m, [&](auto ct, auto xt) {
            const auto launch = [&](auto r) {
                const dim3 grid((unsigned)((n + 16 * r - 1) / (16 * r)), (unsigned)((m + xt * ct - 1) / (xt * ct)));
                matvec_kernel<fmt, g, r, ct, xt><<<grid, kThreads, 0, stream>>>(v, x_bf16, x_stride, m, y_bf16,
                                                                               y_stride);
            };
            constexpr int most = most_rows(fmt, ct);
            if constexpr (most == 4) with_rows<1, 2, 4>(matvec_rows(n, most), launch);
            else with_rows<1, 2>(matvec_rows(n, most), launch);
        });
        return launch_status();
    });
}

extern "C" moe_status moe_few_token_layer_workspace(const moe_dims* dims, int32_t inter, size_t* bytes) {
    Dims d;
    moe_status st = load_dims(dims, &d, true);
    if (st != MOE_OK) return st;
    if (!bytes || inter < 128 || inter % 128 != 0) return MOE_ERR_INVALID_ARG;
    // H and inter: the grids' limits
    if (d.L > kMaxLocal || d.k > kMaxTopK || inter >= (1 << 24) || d.H >= (1 << 24)) return MOE_ERR_UNSUPPORTED;
    *bytes = (size_t)(std::min<int64_t>(d.T, kChunk) * d.k * inter * 2 + 255) / 256 * 256;
    return MOE_OK;
}

extern "C" moe_status moe_few_token_layer(const moe_dims* dims, int32_t inter, const uint16_t* x_bf16,
                                          const int32_t* topk_ids, const float* topk_w, const moe_weight* w1,
                                          const moe_weight* w2, uint16_t* out_bf16, void* ws, size_t ws_bytes,
                                          void* hip_stream) {
    size_t need;
    moe_status st = moe_few_token_layer_workspace(dims, inter, &need);
    if (st != MOE_OK) return st;
    Dims d;
    st = load_dims(dims, &d, true);
    if (st != MOE_OK) return st;
    WView v1, v2;
    int g1, g2;
    st = load_weight(w1, 2 * (int64_t)inter, d.H, &v1, &g1);
    if (st != MOE_OK) return st;
    st = load_weight(w2, d.H, inter, &v2, &g2);
    if (st != MOE_OK) return st;
    if (d.T == 0) return MOE_OK;
    if (!x_bf16 || !topk_ids || !topk_w || !out_bf16) return MOE_ERR_INVALID_ARG;
    if (!aligned(x_bf16, 16) || !aligned(out_bf16, 8)) return MOE_ERR_INVALID_ARG;
    // token and intermediate rows are addressed with 31-bit byte offsets
    const int64_t chunk = std::min<int64_t>(d.T, kChunk);
    if (chunk * d.H * 2 > INT32_MAX || chunk * d.k * inter * 2 > INT32_MAX) return MOE_ERR_UNSUPPORTED;
    if (!ws || ws_bytes < need || !aligned(ws, 16)) return MOE_ERR_WORKSPACE;
    hipStream_t stream = reinterpret_cast<hipStream_t>(hip_stream);
    for (int64_t t0 = 0; t0 < d.T && st == MOE_OK; t0 += kChunk) {
        LayerArgs a;
        a.x = x_bf16 + t0 * d.H;
        a.ids = topk_ids + t0 * d.k;
        a.topk_w = topk_w + t0 * d.k;
        a.h = static_cast<uint16_t*>(ws);
        a.out = out_bf16 + t0 * d.H;
        a.T = (int)std::min<int64_t>(d.T - t0, kChunk);
        a.k = (int)d.k, a.e0 = (int)d.e0, a.L = (int)d.L, a.H = (int)d.H, a.I = inter;
        // columns for the tokens that an expert of uniform routing has, and two deviations more: an expert with more
        // takes a further pass
        const double mean = (double)a.T * d.k / d.E;
        const int64_t share = std::min<int64_t>(a.T, (int64_t)std::ceil(mean + 2.0 * std::sqrt(mean)));
        // workgroups of one row tile that uniform routing would keep busy: 1 / 2 / 4 tiles by the rule of moe_matvec
        // (one token, e2m1, 2048 workgroups: 43.0 / 29.2 / 28.2 us)
        const double hit = d.L * (1.0 - std::pow(1.0 - (double)d.k / d.E, (double)a.T));
        const int64_t busy = (int64_t)(hit * (inter / 8));
        const int r1 = busy >= 4 * kCus ? 4 : busy >= 2 * kCus ? 2 : 1;
        st = with_format(w1->format, g1, [&](auto fmt, auto g) {
            with_cols(std::min<int64_t>(share, 32), [&](auto ct, auto xt) {
                if constexpr (ct <= 2)
                    with_rows<1, 2, 4>(r1, [&](auto r) {
                        const dim3 grid((unsigned)(inter / (8 * r)), (unsigned)std::min<int64_t>(a.T * d.k, d.L));
                        gate_up_kernel<fmt, g, r, ct, xt><<<grid, kThreads, a.T * a.k * 8, stream>>>(v1, a);
                    });
            });
            return launch_status();
        });
        if (st != MOE_OK) return st;
        // two row tiles from three quarters of a workgroup a CU.  The layer's us with one / two (I = 2048; one token and
        // 8 experts e2m1, 16 tokens and 21 experts int4, 64 tokens and 28 experts e4m3): 4096 rows 29 / 31, 59 / 70,
        // 127 / 140; 5120 rows 41 / 37, 83 / 77, 176 / 162 (a second round of workgroups: two would pay here already);
        // 6144 rows 44 / 40, 92 / 85, 198 / 186; 7168 rows 49 / 45, 98 / 92, 216 / 210
        const int r2 = d.H >= 24 * kCus ? 2 : 1;
        st = with_format(w2->format, g2, [&](auto fmt, auto g) {
            with_cols(std::min<int64_t>(share, 16), [&](auto ct, auto xt) {
                if constexpr (ct == 1)
                    with_rows<1, 2>(r2, [&](auto r) {
                        with_rows<1, 2, 4>(a.T <= 16 ? 1 : a.T <= 32 ? 2 : 4, [&](auto ot) {
                            constexpr int NW = down_waves(g, r, ot);
                            down_kernel<fmt, g, r, xt, ot, NW>
                                <<<dim3((unsigned)(d.H / (16 * r))), NW * MOE_WAVE, a.T * a.k * 8, stream>>>(v2, a);
                        });
                    });
            });
            return launch_status();
        });
    }
    return st;
}
