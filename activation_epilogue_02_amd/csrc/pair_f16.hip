// pair_f16.hip -- two fp16 products in one launch (the backward pass's).
#include "tile2_kernel.h"

namespace ge {

PairFn pick_pair_f16(int op_b, int tile_id) { return pick_pair<GE_F16>(op_b, tile_id); }

}  // namespace ge
