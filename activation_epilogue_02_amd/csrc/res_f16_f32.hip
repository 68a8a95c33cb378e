// res_f16_f32.hip -- the residual product's tiles for fp16 inputs and
// fp32 output.
#include "tile2_kernel.h"

namespace ge {

ResFn pick_res_f16_f32(int op_b, int tile_id) { return pick_res_op<GE_F16, GE_F32>(op_b, tile_id); }

}  // namespace ge
