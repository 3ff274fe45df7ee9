// The router's choice: each token's k largest logits, their expert ids and their softmax weights.
//
// One wavefront per token.  The order is decided on the logits themselves (a monotone integer key), never on
// computed exponentials, so the ids are exact: larger first, ties to the lower id.  A logit of -inf or NaN gets the
// key 0 and is never chosen.  Lane l holds experts l, l + 64, ...; each of the k rounds takes the wavefront's
// largest (key, lowest id) pair and removes it.
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

template <bool BF16, int V>
__global__ void __launch_bounds__(kThreads)
route_topk_kernel(const void* __restrict__ logits, int64_t stride, int64_t T, int E, int k, bool renormalise,
                  float scale, int32_t* __restrict__ ids, float* __restrict__ w) {
    const int lane = lane_id();
    const int64_t t = (int64_t)blockIdx.x * kWaves + threadIdx.x / MOE_WAVE;
    if (t >= T) return;
    uint32_t key[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = lane + 64 * i;
        float v = -INFINITY;
        if (e < E)
            v = BF16 ? bf16_lo(static_cast<const uint16_t*>(logits)[t * stride + e])
                     : static_cast<const float*>(logits)[t * stride + e];
        key[i] = key_of(v);
    }
    uint32_t my_key = 0;                     // lane j: the j-th choice
    int my_id = -1;
    uint32_t top = 0;
    float all = 0.f;
    for (int j = 0; j < k; ++j) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) m = max(m, key[i]);
#pragma unroll
        for (int off = 32; off > 0; off >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, off, MOE_WAVE));
        if (m == 0) break;                   // nothing left to choose
        if (j == 0) {
            top = m;
            if (!renormalise) {
                const float vm = value_of(top);
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (key[i]) all += key[i] == top ? 1.0f : expf(value_of(key[i]) - vm);
#pragma unroll
                for (int off = 32; off > 0; off >>= 1) all += __shfl_xor(all, off, MOE_WAVE);
            }
        }
        int id = kMaxExperts;
#pragma unroll
        for (int i = V - 1; i >= 0; --i)
            if (key[i] == m) id = lane + 64 * i;
#pragma unroll
        for (int off = 32; off > 0; off >>= 1) id = min(id, __shfl_xor(id, off, MOE_WAVE));
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (lane + 64 * i == id) key[i] = 0;
        if (lane == j) my_key = m, my_id = id;
    }
    // equal keys have difference 0, also where both are +inf
    float p = my_key == 0 ? 0.f : my_key == top ? 1.0f : expf(value_of(my_key) - value_of(top));
    float total = all;
    if (renormalise) {
        total = p;
#pragma unroll
        for (int off = 32; off > 0; off >>= 1) total += __shfl_xor(total, off, MOE_WAVE);
    }
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
    if (d.E > kMaxExperts || d.k > kMaxTopK) return MOE_ERR_UNSUPPORTED;
    if (d.T == 0) return MOE_OK;
    if (!logits || !topk_ids || !topk_w) return MOE_ERR_INVALID_ARG;
    const unsigned grid = (unsigned)((d.T + kWaves - 1) / kWaves);
    hipStream_t stream = reinterpret_cast<hipStream_t>(hip_stream);
    auto launch = [&](auto bf16, auto v) {
        route_topk_kernel<bf16, v><<<grid, kThreads, 0, stream>>>(logits, logits_stride, d.T, (int)d.E, (int)d.k,
                                                                 renormalise != 0, scale, topk_ids, topk_w);
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
