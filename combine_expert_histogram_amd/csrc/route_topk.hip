// The router's choice: each token's k largest logits, their expert ids and their softmax weights.
//
// One wavefront per token.  The order is decided on the logits themselves (a monotone integer key), never on
// computed exponentials, so the ids are exact: larger first, ties to the lower id.  A logit of -inf or NaN gets the
// key 0 and is never chosen.
//
// Lane l holds the V experts l V .. l V + V - 1, sorted once (larger first, equal ones left in id order).  Each of the
// k rounds takes the largest head: the maximum by DPP within sixteen lanes and scalar beyond, the lowest lane that
// holds it by a ballot (the lowest id among equals, as lanes are in id order), and that lane drops its head.  The
// ballot and the scalar maximum take no LDS, where shuffles would wait for it twelve times a round (and did: 16384
// tokens of 256 experts, top-8, 19.8 us; 10.1 now, of which the 17 MB of logits are 3; one token 5.1 -> 2.3 us).
#include "common.h"

namespace {

using namespace moe;

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / MOE_WAVE;
constexpr int kMaxExperts = 1024;
constexpr int kMaxTopK = 64;

// Monotone key of a logit: 0 for -inf and NaN, else larger for larger values; -0 and +0 alike.
__device__ __forceinline__ uint32_t key_of(float v) {
    if (!(v > -INFINITY)) return 0;
    const uint32_t b = __float_as_uint(v + 0.0f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t key) {
    return __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);
}

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_mov(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xF, 0xF, true);
}

// Folds the sixteen lanes of each row: quad_perm [1 0 3 2], [2 3 0 1], row_half_mirror, row_mirror.
template <class Op>
__device__ __forceinline__ uint32_t row_fold(uint32_t v, Op&& op) {
    v = op(v, dpp_mov<0xB1>(v));
    v = op(v, dpp_mov<0x4E>(v));
    v = op(v, dpp_mov<0x141>(v));
    return op(v, dpp_mov<0x140>(v));
}

__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
    v = row_fold(v, [](uint32_t a, uint32_t b) { return max(a, b); });
    const uint32_t a = __builtin_amdgcn_readlane(v, 0), b = __builtin_amdgcn_readlane(v, 16);
    const uint32_t c = __builtin_amdgcn_readlane(v, 32), d = __builtin_amdgcn_readlane(v, 48);
    return max(max(a, b), max(c, d));
}

__device__ __forceinline__ float wave_fsum(float f) {
    const uint32_t v = row_fold(__float_as_uint(f), [](uint32_t a, uint32_t b) {
        return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
    });
    const auto row = [&](int l) { return __uint_as_float(__builtin_amdgcn_readlane(v, l)); };
    return (row(0) + row(16)) + (row(32) + row(48));
}

template <bool BF16, int V>
__global__ void __launch_bounds__(kThreads)
route_topk_kernel(const void* __restrict__ logits, int64_t stride, int64_t T, int E, int k, bool renormalise,
                  bool vector, float scale, int32_t* __restrict__ ids, float* __restrict__ w) {
    const int lane = lane_id();
    const int64_t t = (int64_t)blockIdx.x * kWaves + threadIdx.x / MOE_WAVE;
    if (t >= T) return;
    float v[V];
    if (vector && V >= 4) {                  // E a multiple of V and every row 16-byte aligned (bf16: 8-byte)
#pragma unroll
        for (int i = 0; i < V; i += 4) {
            const int e = lane * V + i;
            if constexpr (BF16) {
                uint2 p = {0xFF80FF80u, 0xFF80FF80u};
                if (e < E) p = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(logits) + t * stride + e);
                v[i] = bf16_lo(p.x), v[i + 1] = bf16_hi(p.x), v[i + 2] = bf16_lo(p.y), v[i + 3] = bf16_hi(p.y);
            } else {
                float4 p = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                if (e < E) p = *reinterpret_cast<const float4*>(static_cast<const float*>(logits) + t * stride + e);
                v[i] = p.x, v[i + 1] = p.y, v[i + 2] = p.z, v[i + 3] = p.w;
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = lane * V + i;
            v[i] = -INFINITY;
            if (e < E)
                v[i] = BF16 ? bf16_lo(static_cast<const uint16_t*>(logits)[t * stride + e])
                            : static_cast<const float*>(logits)[t * stride + e];
        }
    }
    uint32_t key[V];
    int id[V];
#pragma unroll
    for (int i = 0; i < V; ++i) key[i] = key_of(v[i]), id[i] = lane * V + i;
#pragma unroll
    for (int n = V - 1; n > 0; --n)          // adjacent exchanges keep equal keys in id order
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const bool swap = key[i] < key[i + 1];
            const uint32_t a = key[i], b = key[i + 1];
            const int c = id[i], d = id[i + 1];
            key[i] = swap ? b : a, key[i + 1] = swap ? a : b;
            id[i] = swap ? d : c, id[i + 1] = swap ? c : d;
        }

    const uint32_t top = wave_max(key[0]);
    // equal keys have difference 0, also where both are +inf
    const auto term = [&](uint32_t m) { return m == top ? 1.0f : expf(value_of(m) - value_of(top)); };
    float total = 0.f;
    if (!renormalise && top != 0) {
        float all = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (key[i]) all += term(key[i]);
        total = wave_fsum(all);
    }
    uint32_t my_key = 0;                     // lane j: the j-th choice
    int my_id = -1;
    uint32_t m = top;
    for (int j = 0; j < k && m != 0; ++j) {
        const int from = __ffsll((unsigned long long)__ballot(key[0] == m)) - 1;
        const int chosen = __builtin_amdgcn_readlane(id[0], from);
        if (lane == j) my_key = m, my_id = chosen;
        if (lane == from) {
#pragma unroll
            for (int i = 0; i + 1 < V; ++i) key[i] = key[i + 1], id[i] = id[i + 1];
            key[V - 1] = 0;
        }
        m = wave_max(key[0]);
    }
    const float p = my_key == 0 ? 0.f : term(my_key);
    if (renormalise) total = wave_fsum(p);
    if (lane < k) {
        ids[t * k + lane] = my_id;
        w[t * k + lane] = my_id >= 0 ? scale * (p / total) : 0.f;
    }
}

}  // namespace

extern "C" moe_status moe_route_topk(const moe_dims* dims, const void* logits, int32_t logits_bf16,
                                     int64_t logits_stride, int32_t renormalise, float scale, int32_t* topk_ids,
                                     float* topk_w, void* hip_stream) {
    Dims d;
    moe_status st = load_dims(dims, &d, false);
    if (st != MOE_OK) return st;
    if (logits_stride < d.E) return MOE_ERR_INVALID_ARG;
    if (d.E > kMaxExperts || d.k > kMaxTopK || d.T > (1 << 25)) return MOE_ERR_UNSUPPORTED;
    if (d.T == 0) return MOE_OK;
    if (!logits || !topk_ids || !topk_w) return MOE_ERR_INVALID_ARG;
    const unsigned grid = (unsigned)((d.T + kWaves - 1) / kWaves);
    hipStream_t stream = reinterpret_cast<hipStream_t>(hip_stream);
    auto launch = [&](auto bf16, auto v) {
        const bool vector = d.E % v == 0 && logits_stride % 4 == 0 &&
                            (reinterpret_cast<uintptr_t>(logits) & (bf16 ? 7 : 15)) == 0;
        route_topk_kernel<bf16, v><<<grid, kThreads, 0, stream>>>(logits, logits_stride, d.T, (int)d.E, (int)d.k,
                                                                 renormalise != 0, vector, scale, topk_ids,
                                                                 topk_w);
    };
    auto sized = [&](auto bf16) {
        if (d.E <= 64) launch(bf16, std::integral_constant<int, 1>{});
        else if (d.E <= 128) launch(bf16, std::integral_constant<int, 2>{});
        else if (d.E <= 256) launch(bf16, std::integral_constant<int, 4>{});
        else if (d.E <= 512) launch(bf16, std::integral_constant<int, 8>{});
        else launch(bf16, std::integral_constant<int, 16>{});
    };
    if (logits_bf16) sized(std::true_type{});
    else sized(std::false_type{});
    return launch_status();
}
