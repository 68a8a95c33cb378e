// res_f32_f32.hip -- the residual product's tiles for fp32 (the
// register-staged kernel).
#include "tile_kernel.h"

namespace ge {

template <int OPB>
ResFn pick_res_f32(int tile_id) {
    if (tile_id == 1) return ge_tile_kernel<GE_F32, GE_F32, OPB, 64, 64, 2, 2, ResArgs>;
    if (tile_id == 2) return ge_tile_kernel<GE_F32, GE_F32, OPB, 128, 128, 2, 2, ResArgs>;
    return nullptr;
}

ResFn pick_res_f32_f32(int op_b, int tile_id) {
    return op_b == GE_OP_T ? pick_res_f32<GE_OP_T>(tile_id) : pick_res_f32<GE_OP_N>(tile_id);
}

}  // namespace ge
