// res_bf16_bf16.hip -- the residual product's tiles for bf16 inputs and
// bf16 output.
#include "tile2_kernel.h"

namespace ge {

ResFn pick_res_bf16_bf16(int op_b, int tile_id) { return pick_res_op<GE_BF16, GE_BF16>(op_b, tile_id); }

}  // namespace ge
