// res_f8_bf16.hip -- the residual product's tiles for fp8 (E4M3) inputs and
// bf16 output.
#include "tile2_kernel.h"

namespace ge {

ResFn pick_res_f8_bf16(int op_b, int tile_id) { return pick_res_op<GE_F8_E4M3, GE_BF16>(op_b, tile_id); }

}  // namespace ge
