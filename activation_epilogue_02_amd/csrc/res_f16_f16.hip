// res_f16_f16.hip -- the residual product's tiles for fp16 inputs and
// fp16 output.
#include "tile2_kernel.h"

namespace ge {

ResFn pick_res_f16_f16(int op_b, int tile_id) { return pick_res_op<GE_F16, GE_F16>(op_b, tile_id); }

}  // namespace ge
