// The tiled product dx = dy w.
#include "dense_tile.h"

namespace moe {

moe_status launch_tiles_nn(int dtype, bool aligned, const Plan& plan, const Product& p, const Epilogue& e, float* part,
                           hipStream_t stream) {
    return launch_layout<false, true>(dtype, aligned, plan, p, e, part, stream);
}

}  // namespace moe
