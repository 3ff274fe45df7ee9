// The tiled product forward: y = x w^T.
#include "dense_tile.h"

namespace moe {

moe_status launch_tiles_nt(int dtype, bool aligned, const Plan& plan, const Product& p, const Epilogue& e, float* part,
                           hipStream_t stream) {
    return launch_layout<false, false>(dtype, aligned, plan, p, e, part, stream);
}

}  // namespace moe
