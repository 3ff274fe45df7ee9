// Both products of a backward pass, dw = d^T x and dx = d w, in one launch.
#include "dense_tile.h"

namespace moe {

moe_status launch_pair(int dtype, const Plan& plan_dw, const Product& dw, const Epilogue& e_dw, const Plan& plan_dx,
                       const Product& dx, const Epilogue& e_dx, hipStream_t stream) {
    PairArgs t;
    if (!tile_args<Wide, false>(plan_dw, dw, e_dw, nullptr, &t.dw) || !tile_args<Wide, false>(plan_dx, dx, e_dx, nullptr, &t.dx))
        return MOE_ERR_UNSUPPORTED;
    t.ahead = std::max(1, (dw.k + dx.k / 2) / dx.k);
    if (dtype == MOE_BF16) hipLaunchKernelGGL(pair_kernel<__bf16>, dim3(kCus), dim3(Wide::kThreads), 0, stream, t);
    else hipLaunchKernelGGL(pair_kernel<_Float16>, dim3(kCus), dim3(Wide::kThreads), 0, stream, t);
    return launch_status();
}

}  // namespace moe
