// res_launch.hip -- launch tables of the residual product's tiles and of two
// products in one launch.
#include "bias_sum.h"
#include "tile_kernel.h"

namespace ge {

int launch_tile_res(int tile_id, int a_type, int d_type, int op_b, const KernelArgs& args, const ResArgs& res,
                    unsigned grid, void* stream) {
    const TileShape* t = nullptr;
    for (int i = 0; i < kNumResTiles; ++i)
        if (kResTiles[i].id == tile_id) t = &kResTiles[i];
    ResFn fn = nullptr;
    switch (a_type) {
    case GE_F32: fn = d_type == GE_F32 ? pick_res_f32_f32(op_b, tile_id) : nullptr; break;
    case GE_F16:
        fn = d_type == GE_F16 ? pick_res_f16_f16(op_b, tile_id)
             : d_type == GE_F32 ? pick_res_f16_f32(op_b, tile_id) : nullptr;
        break;
    case GE_BF16:
        fn = d_type == GE_BF16 ? pick_res_bf16_bf16(op_b, tile_id)
             : d_type == GE_F32 ? pick_res_bf16_f32(op_b, tile_id) : nullptr;
        break;
    case GE_F8_E4M3:
        fn = d_type == GE_BF16 ? pick_res_f8_bf16(op_b, tile_id)
             : d_type == GE_F16 ? pick_res_f8_f16(op_b, tile_id)
             : d_type == GE_F32 ? pick_res_f8_f32(op_b, tile_id) : nullptr;
        break;
    case GE_MXF8_E4M3:
        fn = d_type == GE_BF16 ? pick_res_mx_bf16(op_b, tile_id)
             : d_type == GE_F16 ? pick_res_mx_f16(op_b, tile_id)
             : d_type == GE_F32 ? pick_res_mx_f32(op_b, tile_id) : nullptr;
        break;
    }
    if (!t || !fn) return (int)hipErrorInvalidDeviceFunction;
    const unsigned slices = t->kernel == 5 ? (unsigned)args.split_k : 1u;   // K slices in z
    hipLaunchKernelGGL(fn, dim3(grid, 1, slices), dim3(t->wm * t->wn * 64), 0, (hipStream_t)stream, args, res);
    return (int)hipGetLastError();
}

int launch_tile_pair(int tile_id, int type, int op_b, const KernelArgs& first, const PairArgs& second, void* stream) {
    const TileShape* t = nullptr;
    for (int i = 0; i < kNumTiles; ++i)
        if (kTiles[i].id == tile_id) t = &kTiles[i];
    const PairFn fn = type == GE_F16 ? pick_pair_f16(op_b, tile_id) : type == GE_BF16 ? pick_pair_bf16(op_b, tile_id) : nullptr;
    if (!t || !fn) return (int)hipErrorInvalidDeviceFunction;
    const int64_t a = (int64_t)first.tiles_m * first.tiles_n, b = (int64_t)second.other.tiles_m * second.other.tiles_n;
    const int64_t c = second.len > 0 ? (second.len - 1) / kSumCols + 1 : 0;
    const int64_t x = a > b ? (a > c ? a : c) : (b > c ? b : c);
    hipLaunchKernelGGL(fn, dim3((unsigned)x, c > 0 ? 3 : 2), dim3(t->wm * t->wn * 64), 0, (hipStream_t)stream, first,
                       second);
    return (int)hipGetLastError();
}

}  // namespace ge
