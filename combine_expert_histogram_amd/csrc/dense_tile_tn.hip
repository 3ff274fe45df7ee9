// The tiled product dw = dy^T x.
#include "dense_tile.h"

namespace moe {

moe_status launch_tiles_tn(int dtype, bool aligned, const Plan& plan, const Product& p, const Epilogue& e, float* part,
                           hipStream_t stream) {
    return launch_layout<true, true>(dtype, aligned, plan, p, e, part, stream);
}

}  // namespace moe
