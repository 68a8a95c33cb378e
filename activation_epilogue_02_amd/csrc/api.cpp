// api.cpp -- the C-ABI front end: handle life cycle, validation, the
// planner (tile / small-m / unfused choice and launch shape) and execute.
//
// Every check runs on the host before any HIP runtime call, so that a call
// that fails launches nothing (nvmath page, paragraph on dtype and shape
// rules: mismatched dtypes or a wrongly shaped bias make the fusion fail;
// epilog page, paragraph on epilog_inputs: tensors must be 16-byte aligned).
#include <hip/hip_runtime.h>

#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include <mutex>
#include <new>

#include "ge_host.h"
#include "grad_params.h"
#include "ge_params.h"

using namespace ge;

// ---- the workspace the library holds itself (gemm_epilog_execute_static) -----
// One fixed array per GPU in the library's code object, held until the
// process ends, for callers that cannot allocate.  Host code never uses the
// array's name as a device address (it is a host-side stand-in): the first
// call on a device asks the runtime for that device's copy
// (hipGetSymbolAddress with the device current) and every call passes that
// address to the kernels.
static __device__ __align__(256) uint8_t scratch[GE_STATIC_WORKSPACE_BYTES];

namespace {
constexpr int kMaxDevices = 64;
std::mutex g_scratch_mu;
void* g_scratch_ptr[kMaxDevices];

// The current device's copy of `scratch` (looked up once per device).
int scratch_of_current_device(void** p) {
    int dev = -1;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) return GE_ERR_HIP;
    std::lock_guard<std::mutex> lock(g_scratch_mu);
    if (!g_scratch_ptr[dev]) {
        void* q = nullptr;
        if (hipGetSymbolAddress(&q, HIP_SYMBOL(scratch)) != hipSuccess || !q) return GE_ERR_HIP;
        g_scratch_ptr[dev] = q;
    }
    *p = g_scratch_ptr[dev];
    return GE_OK;
}
}  // namespace

struct ge_plan_s {
    ge_desc d;
    bool planned = false;
    int32_t epilog = 0, axis = 0;
    int32_t path = 0, tile_id = 0, unfused = 0;
    int32_t split_k = 1, k_per_split = 0;
    int32_t tiles_m = 0, tiles_n = 0, group_m = 1;
    int32_t k_stagger = 0;
    unsigned grid = 0;
    size_t ws_c = 0;         // unfused intermediate bytes
    size_t ws_partial = 0;   // split-K partial bytes
    size_t ws_counters = 0;  // split-K counter bytes
    int64_t n_counters = 0;  // split-K arrival counters per product
    int64_t part_bytes = 0;  // split-K partial bytes per product
    size_t ws_bgrad = 0;     // bias-gradient partial bytes
    int32_t bgrad_parts = 0; // bias-gradient partials per entry
    ge_pref pref = {0, 0, 0, 0, 0};   // the preferences the plan was made with
    int64_t ldaux = 0;       // mask row stride, 32-bit words
    bool bstr_set = false;   // per-product strides given (else packed)
    ge_batch_strides bstr = {0, 0, 0, 0, 0};
    const float* scale_d = nullptr;   // fp8 output: D's scale (NULL = 1)
    float* amax_d = nullptr;          // fp8 output: largest |y| per product, or NULL
    // residual product (gemm_epilog_plan_residual): the plan is for
    // execute_residual only; skinny_mb = row groups of the streaming kernel (at the
    // planned rows: a call takes the shape of its own)
    bool residual = false;
    int32_t skinny_mb = 0;
    // its backward pass (gemm_epilog_plan_backward): dP (bytes, row stride),
    // the transposed operand of the weight's gradient, the bias partials, and
    // the two products' handles (owned by the handle)
    bool backward = false;
    size_t bw_dp = 0, bw_t = 0, bw_part = 0, bw_gemm = 0;
    int64_t ld_dp = 0, ld_t = 0;
    ge_plan_s* g_a = nullptr;
    ge_plan_s* g_b = nullptr;
    int32_t pair_tile = 0;   // both products in one launch of this tile, or 0
    size_t bw_t2 = 0;        // weight k x n: dP^T for that launch
};

namespace {

bool dtype_combo_ok(int a, int b, int d) {
    if (a != b) return false;
    switch (a) {
    case GE_F32: return d == GE_F32;
    case GE_F16: return d == GE_F16 || d == GE_F32 || d == GE_F8_E4M3;
    case GE_BF16: return d == GE_BF16 || d == GE_F32 || d == GE_F8_E4M3;
    case GE_F8_E4M3:
    case GE_MXF8_E4M3: return d == GE_BF16 || d == GE_F16 || d == GE_F32 || d == GE_F8_E4M3;
    }
    return false;
}

// Epilogues that add a bias (DRELU and DGELU read none).
bool has_bias(int e) {
    return e == GE_EPILOG_BIAS || e == GE_EPILOG_RELU_BIAS || e == GE_EPILOG_RELU_AUX_BIAS ||
           e == GE_EPILOG_GELU_BIAS || e == GE_EPILOG_GELU_AUX_BIAS || e == GE_EPILOG_TANH_BIAS;
}
// Epilogues with an aux buffer: a bit mask (written by RELU_AUX_BIAS, read by
// DRELU) or a pre-activation matrix in D's dtype (written by GELU_AUX_BIAS,
// read by DGELU).
bool is_bgrad(int e) { return e == GE_EPILOG_DRELU_BGRAD || e == GE_EPILOG_DGELU_BGRAD; }
bool has_aux(int e) {
    return e == GE_EPILOG_RELU_AUX_BIAS || e == GE_EPILOG_DRELU || e == GE_EPILOG_GELU_AUX_BIAS ||
           e == GE_EPILOG_DGELU || is_bgrad(e);
}
bool aux_is_matrix(int e) {
    return e == GE_EPILOG_GELU_AUX_BIAS || e == GE_EPILOG_DGELU || e == GE_EPILOG_DGELU_BGRAD;
}

const TileShape* find_tile(int id) {
    for (int i = 0; i < kNumTiles; ++i)
        if (kTiles[i].id == id) return &kTiles[i];
    return nullptr;
}

const TileShape* find_res_tile(int id) {
    for (int i = 0; i < kNumResTiles; ++i)
        if (kResTiles[i].id == id) return &kResTiles[i];
    return nullptr;
}

// The pipelined kernels' direct copies address a tile's rows of A, and of B
// (either layout), as 32-bit offsets from the tile's first row or column:
// the span must stay below 4 GiB.  (A K step is at most 128 elements.)
bool tile_span_ok(const TileShape* t, const ge_desc& d) {
    if (t->kernel == 1 || t->kernel == 3) return true;   // per-lane 64-bit addresses
    const int64_t es = elem_size(d.a_type), lim = (int64_t)1 << 32;
    if ((int64_t)t->bm * d.lda * es > lim) return false;
    if (d.op_b == GE_OP_T) return (int64_t)t->bn * d.ldb * es <= lim;
    return ((int64_t)128 * d.ldb + t->bn) * es <= lim;
}

// What a tile of the residual product costs: `fixed` us a round (prologue and
// epilogue) and us per 128 bytes of K, in a full round of `slots` workgroups
// and in one at most half full.
struct TileCost {
    int32_t id, bm, bn, slots;
    double fixed, full, half;
};

// The tile of the least estimated time among those whose rows lie close enough
// together (0: none): tiles come in rounds of as many as the
// chip holds, so 581 tiles of 64 x 64 take as long as 1024 would, and fewer,
// larger ones win.  The figures are fits to the measured (bias, residual, 16-bit
// output; us, estimate in brackets):
//   bf16 256 x 256: 4096 x 4096 x 4096 135 (138), x 1024 44 (42), 2048 x 4096 x 4096 89 (90);
//   128 x 128: 2048 x 4096 x 4096 89 (91), 4096 x 4096 x 1024 55 (55), 3000 x 2000 x 700 22 (21),
//     512 x 4096 x 4096 37 (41);
//   64 x 64: 512 x 4096 x 4096 33 (33), 5287 x 435 x 6081 91 (84), 1000 x 1000 x 1000 10 (10);
//   E4M3 256 x 128: 2048 x 4096 x 4096 41 (41), 1024 x 4096 x 4096 33 (33);
//   128 x 128: 2048 x 4096 x 4096 48 (48), 1024 x 4096 x 4096 24 (24), 5401 x 785 x 12557 131 (120);
//   64 x 128: 1024 x 4096 x 4096 30 (32), 500 x 2000 x 2000 13 (10), 1401 x 1801 x 428 15 (13).
int cheapest_tile(const TileCost* t, int n, const ge_desc& d) {
    const double steps = (double)ceil_div(d.k * elem_size(d.a_type), 128);
    int best = 0;
    double least = 0.0;
    for (int i = 0; i < n; ++i) {
        if (!tile_span_ok(find_res_tile(t[i].id), d)) continue;   // rows too far apart for it: the next one
        const int64_t tiles = ceil_div(d.m, t[i].bm) * ceil_div(d.n, t[i].bn), rest = tiles % t[i].slots;
        double us = (double)(tiles / t[i].slots) * (t[i].fixed + steps * t[i].full);
        if (rest > 0) us += t[i].fixed + steps * (2 * rest <= t[i].slots ? t[i].half : t[i].full);
        if (best == 0 || us < least) {
            best = t[i].id;
            least = us;
        }
    }
    return best;
}

// The residual product's tile.  E4M3: 256 x 256 where it gives every CU two tiles,
// else by cost.  Measured at K = 512 / 4096 / 16384, us, 256 x 256 against 256 x 128:
// 8192 x 4096 (512 tiles of 256 x 256) 46, 130, 428 / 54, 152, 449; 8192 x 5120 (640)
// 63, 186 / 63, 183; 8192 x 8192 (1024) 109, 286 / 116, 309; 16384 x 8192 (2048) 208,
// 544 / 220, 612; below, 6144 x 4096 (384) 45, 116, 372 / 43, 109, 337.  (One full round,
// 4096 x 4096, would win too: 25, 67, 214 / 32, 78, 228.)  Block-scaled 128 x 128:
// two workgroups per CU against one with four stages and split-K: 8192 x 8192 x
// 8192 758 / 875, 1300 x 4096 x 4096 (352 tiles) 53 / 60, 1024 x 4096 x 4096 (256) 38 / 34.
int choose_res_tile(const ge_desc& d) {
    static const TileCost k16[] = {{6, 256, 256, 256, 10.0, 2.0, 1.25},
                                   {8, 128, 128, 512, 6.5, 1.32, 0.54},
                                   {14, 64, 64, 512, 4.0, 0.45, 0.35}};
    static const TileCost k8[] = {{15, 256, 128, 256, 8.0, 1.02, 0.78},
                                  {8, 128, 128, 256, 5.0, 0.6, 0.5},
                                  {17, 64, 128, 256, 5.0, 0.34, 0.3}};
    const int64_t t128 = ceil_div(d.m, 128) * ceil_div(d.n, 128);
    switch (d.a_type) {
    case GE_F32: return t128 >= 256 ? 2 : 1;
    case GE_MXF8_E4M3: return t128 > 256 ? 19 : 18;
    case GE_F8_E4M3:
        return ceil_div(d.m, 256) * ceil_div(d.n, 256) >= 512 && tile_span_ok(find_res_tile(16), d)
                   ? 16 : cheapest_tile(k8, 3, d);
    }
    return cheapest_tile(k16, 3, d);
}

// K slices of a split-K tile: the power of two of the least estimated time, with
// the grid within one workgroup per CU.  A slice saves its share of the K steps
// (`us` each); meeting takes about 4 us, the last slice's reading of every
// partial, and the partials' share of the memory.  Measured, us at 1 / 2 / 4 / 8 slices: block-scaled 923 x 1265 x 7945 (80 tiles)
// 60 / 42, 713 x 185 x 3841 (12) 33 / 28 / 23 / 25, 512 x 2048 x 4096 (64) 28 / 25 / 24;
// E4M3 251 x 141 x 6795 (8) 26 / 22 / 17 / 17 (22 at 14), 255 x 86 x 2315 (4) 11 / 13 / 13 / 15,
// 1000 x 500 x 4096 (64) 13 / 15 / 15; bf16 400 x 700 x 3000 (77) 19 / 16, 111 x 1941 x
// 1129 (62) 9 / 11 / 11.
int res_split(const TileShape* t, int a_type, int64_t tiles, int64_t steps) {
    const double us = a_type == GE_MXF8_E4M3 ? 0.75 : a_type == GE_F8_E4M3 ? 0.34 : 0.4;
    int split = 1;
    double least = (double)steps * us;
    for (int s = 2; s <= 16 && tiles * s <= 256 && steps >= 2 * s; s *= 2) {
        const double part = 4.0 * t->bm * t->bn;   // bytes; read at 0.055 TB/s by one workgroup, 4 TB/s by all
        const double v = (double)steps * us / s + 4.0 + s * part / 55e3 + 2.0 * (double)(tiles * s) * part / 4e6;
        if (v < least) {
            least = v;
            split = s;
        }
    }
    return split;
}

// The register-staged tile kernel's tile for a problem (any dtype).
int choose_tile_plain(int64_t m, int64_t n) {
    const int64_t t256 = ceil_div(m, 256) * ceil_div(n, 256);
    const int64_t t128 = ceil_div(m, 128) * ceil_div(n, 128);
    if (t256 >= 512) return 3;
    if (t128 >= 512) return 2;
    if (t256 >= 256 && t128 < 256) return 3;
    if (t128 >= 256) return 2;
    return 1;
}

// Tile heuristic: the largest block tile that still gives every CU at least
// two tiles (256 CUs); below that, the shape with the most tiles.  Large
// tiles halve the L2 -> LDS traffic per flop; small problems need the
// parallelism more than the reuse.
int choose_tile(int64_t m, int64_t n, int a_type, int d_type) {
    const int64_t t256 = ceil_div(m, 256) * ceil_div(n, 256);
    const int64_t t128 = ceil_div(m, 128) * ceil_div(n, 128);
    // fp8 output: the tiles instantiated for it (the large one when it
    // gives every CU a tile, else 128 x 128)
    if (d_type == GE_F8_E4M3) {
        if (a_type == GE_MXF8_E4M3) return 8;
        if (a_type == GE_F8_E4M3) return t256 >= 512 ? 16 : ceil_div(m, 256) * ceil_div(n, 128) >= 512 ? 15 : 8;
        return t256 >= 256 ? 6 : 8;
    }
    // block-scaled fp8: the one tile the block-scaled MFMA compiles into
    // without register spills
    if (a_type == GE_MXF8_E4M3) return 8;
    if (a_type == GE_F8_E4M3) {
        // A CU takes about 0.2 128-byte lines per cycle into LDS, so tiles
        // with fewer bytes per flop keep the matrix cores busier: 256 x 256
        // with 8 waves and 64-byte K steps (four 32 KiB stages, spread
        // copies; tile 16) measures 8% faster than 256 x 128 (tile 15) on
        // 65536 x 8192 x 16384 (2379 against 2200 TFLOP/s).  With 128-byte
        // steps a 256 x 256 stage is 64 KiB and only two fit.  256 x 128 with
        // 8 waves (two per SIMD) beats 4 waves by 10% (1943 against 1765).
        const int64_t t2x1 = ceil_div(m, 256) * ceil_div(n, 128);
        if (t256 >= 512) return 16;
        if (t2x1 >= 512) return 15;
        if (t128 >= 256) return 8;
        return 1;
    }
    if (a_type == GE_F16 || a_type == GE_BF16) {
        // the pipelined direct-to-LDS kernel; at 256 x 256 the 8-wave
        // layout (two waves per SIMD fill each other's barrier gaps) with
        // four 64-byte K stages, whose copies are spread among the MFMAs,
        // measures fastest (65536 x 8192 x 16384: 1258 TFLOP/s against
        // 1164 for two 128-byte stages with the copies in one burst)
        if (t256 >= 512) return 6;
        if (t128 >= 512) return 8;
        if (t256 >= 256 && t128 < 256) return 6;
        if (t128 >= 256) return 8;
        return 13;   // small problems: 64 x 64 tiles, four deep stages
    }
    return choose_tile_plain(m, n);
}

// Tile rows per group of the launch order (see tile_coords).  The 32 tiles
// an XCD runs at once then cover g tile rows and 32 / g columns.  Fewer rows
// than the 8 that minimise the panels in flight measure faster: with eight,
// every B line is wanted by eight CUs at the same moment and A lines by
// four, and the requests queue behind the one that misses (65536 x 8192 x
// 16384 bf16, 256 x 256 tiles: 1207 / 1258 / 1236 TFLOP/s at 8 / 4 / 2 rows;
// the block-scaled 128 x 128 tile: 1150 / 1198 / 1278).
int32_t auto_group_m(const TileShape* t, int64_t tm, int a_type) {
    const int64_t g = a_type == GE_MXF8_E4M3 ? 2 : (t->kernel == 1 ? 8 : 4);
    return (int32_t)(tm < g ? (tm > 0 ? tm : 1) : g);
}

// Full K steps of rotation per tile row and column of a group (the
// pipelined kernel's K order).  The tiles that share a panel of A or B run in
// lock-step, so their requests for the same lines arrive together and queue
// behind the one that misses; rotating each tile's K order spreads them, at
// the cost of a longer stretch of each panel held in L2.  Measured on 65536 x
// 8192 x 16384 (TFLOP/s at 0 / 1 / 2 / 4 / 8 steps): the block-scaled 128 x
// 128 tile, 16 tiles on each A panel at once, 1290 / 1335 / 1356 / 1347 /
// 1290; the fp8 256 x 256 tile 2332-2367 unrotated against 2358-2392 at one
// step; the bf16 256 x 256 tile 1273-1276 / 1273 / 1262 / 1247 (none there).
// GE_K_STAGGER=<steps> in the environment overrides the choice.
int32_t auto_k_stagger(const TileShape* t, int a_type) {
    if (const char* e = getenv("GE_K_STAGGER")) {
        const int v = atoi(e);
        return v > 0 ? v : 0;
    }
    if (a_type == GE_MXF8_E4M3 && t->id == 8) return 2;
    if (a_type == GE_F8_E4M3 && t->id == 16) return 1;
    return 0;
}

// The pipelined kernel takes 16-bit and fp8 inputs (its 64 x 64 tile only
// 16-bit ones); block-scaled fp8 runs on its 128 x 128 tile only.
bool tile_supports(const TileShape* t, int a_type, int d_type) {
    if (d_type == GE_F8_E4M3) {   // fp8 output: the instantiated tiles only
        if (a_type == GE_MXF8_E4M3) return t->id == 8;
        if (a_type == GE_F8_E4M3) return t->id == 16 || t->id == 15 || t->id == 8;
        return t->id == 6 || t->id == 8;
    }
    if (a_type == GE_MXF8_E4M3) return t->id == 8;
    if (t->kernel == 1) return true;
    if (t->id == 13 || t->id == 14) return a_type == GE_F16 || a_type == GE_BF16;
    if (t->kernel == 6) return a_type == GE_F8_E4M3;
    return a_type == GE_F16 || a_type == GE_BF16 || a_type == GE_F8_E4M3;
}

bool smallm_supported(const ge_desc& d) {
    return d.m <= 16 && d.op_b == GE_OP_T && (d.a_type == GE_F16 || d.a_type == GE_BF16) &&
           (d.d_type == d.a_type || d.d_type == GE_F32);
}

// Automatic K split of the small-m path.  The kernel's register use leaves
// room for one workgroup per CU (256 CUs), so a grid beyond 256 runs in a
// second round that pays the whole load-latency chain again, and the
// split's serial device-scope round trips (partial store, arrival count,
// reload) only pay off when the column blocks alone leave CUs idle.  Hence:
// the largest power of two that keeps the grid within one round and each of
// the 8 waves at two or more 64-wide K spans.
int smallm_auto_split(int64_t tiles_n, int64_t spans) {
    constexpr int64_t kCUs = 256, kWaves = 8, kMinSpansPerWave = 2;
    int split = 1;
    while (tiles_n * split * 2 <= kCUs && spans >= split * 2 * kWaves * kMinSpansPerWave) split *= 2;
    return split;
}

}  // namespace

extern "C" {

int gemm_epilog_create(ge_handle* h, const ge_desc* desc) {
    if (!h || !desc) return GE_ERR_NULL;
    *h = nullptr;
    const ge_desc& d = *desc;
    if (d.m < 0 || d.n < 0 || d.k < 0) return GE_ERR_SHAPE;
    if (d.m > INT32_MAX || d.n > INT32_MAX || d.k > INT32_MAX) return GE_ERR_SHAPE;
    if (d.batch < 0 || d.batch > 65535 || (d.op_b != GE_OP_N && d.op_b != GE_OP_T)) return GE_ERR_SHAPE;
    if (!dtype_combo_ok(d.a_type, d.b_type, d.d_type)) return GE_ERR_DTYPE;
    // the bias follows D's dtype; for fp8 D it is bf16
    if (d.bias_type != (d.d_type == GE_F8_E4M3 ? GE_BF16 : d.d_type)) return GE_ERR_DTYPE;
    if (d.lda < d.k || d.ldd < d.n) return GE_ERR_SHAPE;
    if (d.ldb < (d.op_b == GE_OP_N ? d.n : d.k)) return GE_ERR_SHAPE;
    if ((d.lda * elem_size(d.a_type)) % 16 || (d.ldb * elem_size(d.b_type)) % 16 ||
        (d.ldd * elem_size(d.d_type)) % 16)
        return GE_ERR_ALIGN;
    ge_plan_s* p = new (std::nothrow) ge_plan_s();
    if (!p) return GE_ERR_ALLOC;
    p->d = d;
    *h = p;
    return GE_OK;
}

int gemm_epilog_plan(ge_handle h, int32_t epilog, int32_t bias_axis, const ge_pref* pref) {
    if (!h) return GE_ERR_NULL;
    if (epilog < GE_EPILOG_NONE || epilog > GE_EPILOG_TANH_BIAS) return GE_ERR_EPILOG;
    if (bias_axis != GE_BIAS_ROW && bias_axis != GE_BIAS_COL) return GE_ERR_EPILOG;
    ge_pref pr = {0, 0, 0, 0, 0};
    if (pref) pr = *pref;
    if (pr.path < 0 || pr.path > PATH_SMALLM || pr.unfused < 0 || pr.unfused > 1 || pr.split_k < 0 ||
        pr.group_m < 0)
        return GE_ERR_SHAPE;
    if (pr.tile != 0 && !find_tile(pr.tile)) return GE_ERR_SHAPE;
    const ge_desc& d = h->d;

    ge_plan_s q = *h;
    q.planned = false;
    q.residual = q.backward = false;
    q.k_stagger = 0;
    q.epilog = epilog;
    q.axis = bias_axis;
    q.unfused = (pr.unfused && epilog != GE_EPILOG_NONE) ? 1 : 0;
    // fp8 output serves the inference epilogues in the fused kernel (no aux
    // matrix in D's dtype, no backward epilogue, no fp8 intermediate)
    if (d.d_type == GE_F8_E4M3) {
        const bool inference = epilog <= GE_EPILOG_GELU_BIAS || epilog == GE_EPILOG_TANH_BIAS;
        if (!inference || q.unfused) return GE_ERR_DTYPE;
    }
    // aux row stride: round_up(n, 128) bits (mask, in 32-bit words) or
    // elements (pre-activation matrix)
    q.ldaux = !has_aux(epilog) ? 0
              : aux_is_matrix(epilog) ? (int64_t)round_up((size_t)d.n, 128)
                                      : (int64_t)round_up((size_t)d.n, 128) / 32;
    if (q.ldaux > INT32_MAX) return GE_ERR_SHAPE;

    // a batch takes product z's bias at z * len values: with a column bias
    // whose n values are not a whole number of 16-byte chunks, every other
    // product's bias would start misaligned for the kernels' 16-byte loads
    if (d.batch > 1 && bias_axis == GE_BIAS_COL && has_bias(epilog) && (d.n * elem_size(d.bias_type)) % 16 != 0)
        return GE_ERR_ALIGN;

    // the small-m kernel serves the inference epilogues only
    const bool smallm_epilog = epilog <= GE_EPILOG_GELU_BIAS || epilog == GE_EPILOG_TANH_BIAS;
    int path = pr.path;
    if (path == 0) path = (smallm_supported(d) && smallm_epilog) ? PATH_SMALLM : PATH_TILE;
    if (path == PATH_SMALLM && !smallm_supported(d)) return GE_ERR_SHAPE;
    if (path == PATH_SMALLM && !smallm_epilog) return GE_ERR_EPILOG;
    q.path = path;
    q.split_k = 1;
    q.ws_partial = q.ws_counters = 0;
    q.n_counters = q.part_bytes = 0;
    if (path == PATH_SMALLM) {
        q.tile_id = 0;
        q.tiles_m = 1;
        // column blocks of 16 * rg rows of W (rg row groups per wave, which
        // share each x fragment).  Every workgroup reads all of x, as many
        // load instructions per CU as its W slab needs, so two groups cut a
        // CU's loads by a quarter; they pay when the 32-column blocks alone
        // still fill the chip (measured at k = 4096: n = 8192 19.0 against
        // 21.0 us, 16384 33.2 against 39.8 us; four groups no better).  A K
        // split to make up the blocks does not: its partial exchange costs
        // about 6 us (n = 4096: 14.5 us with two groups in two slices,
        // 11.1 us with one group unsplit).
        if (pr.group_m != 0 && pr.group_m != 1 && pr.group_m != 2 && pr.group_m != 4) return GE_ERR_SHAPE;
        const int rg = pr.group_m > 0 ? pr.group_m : (ceil_div(d.n, 32) >= 256 ? 2 : 1);
        q.tiles_n = (int32_t)ceil_div(d.n, 16 * rg);
        // K slices of whole 64-element spans (the kernel's load unit)
        const int64_t spans = ceil_div(d.k, 64);
        int split = pr.split_k > 0 ? pr.split_k : smallm_auto_split(q.tiles_n, spans);
        if (split > spans) split = spans > 0 ? (int)spans : 1;
        q.k_per_split = (int32_t)(ceil_div(spans, split) * 64);
        split = q.k_per_split > 0 ? (int)ceil_div(d.k, q.k_per_split) : 1;
        q.split_k = split;
        q.group_m = rg;
        const int64_t grid = (int64_t)q.tiles_n * split;
        if (grid > INT32_MAX) return GE_ERR_SHAPE;
        q.grid = (unsigned)grid;
        if (split > 1) {
            const size_t nbs = d.batch > 1 ? (size_t)d.batch : 1;
            q.n_counters = q.tiles_n;
            q.part_bytes = (int64_t)split * q.tiles_n * 256 * rg * (int64_t)sizeof(float);
            q.ws_partial = round_up(nbs * (size_t)q.part_bytes, 256);
            q.ws_counters = round_up(nbs * (size_t)q.n_counters * sizeof(uint32_t), 256);
        }
    } else {
        q.tile_id = pr.tile ? pr.tile : choose_tile(d.m, d.n, d.a_type, d.d_type);
        // the automatic split-K 64 x 64 tile serves problems with so few tiles
        // and so long a K that the slices' parallelism outweighs their
        // partial exchange: at most 64 tiles with k >= 4096, or at most 128
        // with k >= 8192 (measured: 1024 x 512 x 8192 takes 29.2 us unsplit
        // and 22.6 us in 2 slices; 1024 x 512 x 2048 10.8 us unsplit and
        // 12.9 / 13.9 us in 2 / 4); the bias-gradient partials would share
        // its partial buffer
        const int64_t t64 = ceil_div(d.m, 64) * ceil_div(d.n, 64);
        if (!pr.tile && q.tile_id == 13 && !is_bgrad(epilog) &&
            ((t64 <= 64 && d.k >= 4096) || (t64 <= 128 && d.k >= 8192)))
            q.tile_id = 14;
        const TileShape* t = find_tile(q.tile_id);
        if (!tile_supports(t, d.a_type, d.d_type)) return GE_ERR_SHAPE;
        if (!tile_span_ok(t, d)) {
            if (pr.tile || d.a_type == GE_MXF8_E4M3 || d.d_type == GE_F8_E4M3) return GE_ERR_SHAPE;
            q.tile_id = choose_tile_plain(d.m, d.n);
            t = find_tile(q.tile_id);
        }
        if (pr.split_k > 1 && t->kernel != 5) return GE_ERR_SHAPE;   // only the split-K tile splits K
        if (t->kernel == 5 && is_bgrad(epilog)) return GE_ERR_EPILOG;
        const int64_t tm = ceil_div(d.m, t->bm), tn = ceil_div(d.n, t->bn);
        if (tm * tn > INT32_MAX) return GE_ERR_SHAPE;
        q.tiles_m = (int32_t)tm;
        q.tiles_n = (int32_t)tn;
        q.group_m = pr.group_m > 0 ? (int32_t)(pr.group_m < tm ? pr.group_m : (tm > 0 ? tm : 1))
                                   : auto_group_m(t, tm, d.a_type);
        q.grid = (unsigned)(tm * tn);
        q.k_per_split = (int32_t)d.k;
        q.k_stagger = auto_k_stagger(t, d.a_type);
        if (t->kernel == 5) {
            // K slices of whole 64-element steps: the largest power of two
            // that keeps the grid within 256 workgroups, every slice at 16 or
            // more steps (32 beyond 128 workgroups) and the split at most 8
            // (16 for at most 4 tiles), unless forced.  The last slice of a tile reads every partial, so
            // beyond that more slices cost more than they gain.  Measured
            // (bf16, the best split and its time): 128 x 128 x 65536 16,
            // 25.9 us (30.0 at 32); 256 x 256 x 4096 4, 12.4; 256 x 256 x
            // 8192 4-8, 14.6; 256 x 256 x 65536 8, 38.4 (41.4 at 16, 180 us
            // unsplit); 256 x 512 x 32768 8, 33.7; 512 x 512 x 8192 4, 17.5;
            // 512 x 512 x 16384 4, 23.5; 1024 x 512 x 16384 2, 37.8;
            // 1024 x 512 x 2048 1, 10.8 (12.9 in 2 slices of 16 steps)
            const int64_t steps = ceil_div(d.k, 64);
            int split = pr.split_k;
            if (split <= 0) {
                const int cap = tm * tn <= 4 ? 16 : 8;
                split = 1;
                while (split * 2 <= cap && tm * tn * split * 2 <= 256 &&
                       steps >= split * 2 * (tm * tn * split * 2 > 128 ? 32 : 16))
                    split *= 2;
            }
            if (split > steps) split = steps > 0 ? (int)steps : 1;
            if (split > 65535) return GE_ERR_SHAPE;
            q.k_per_split = (int32_t)(ceil_div(steps, split) * 64);
            split = q.k_per_split > 0 ? (int)ceil_div(d.k, q.k_per_split) : 1;
            q.split_k = split;
            if (split > 1) {
                const size_t nbs = d.batch > 1 ? (size_t)d.batch : 1;
                q.n_counters = tm * tn;
                q.part_bytes = tm * tn * split * (int64_t)t->bm * t->bn * (int64_t)sizeof(float);
                q.ws_partial = round_up(nbs * (size_t)q.part_bytes, 256);
                q.ws_counters = round_up(nbs * (size_t)q.n_counters * sizeof(uint32_t), 256);
            }
        }
    }
    const size_t nb = d.batch > 1 ? (size_t)d.batch : 1;   // products per launch
    q.ws_c = q.unfused ? round_up(nb * (size_t)d.m * (size_t)d.ldd * elem_size(d.d_type), 256) : 0;
    // bias gradient: one fp32 partial per tile row (COL) or column (ROW) and
    // gradient entry; the unfused pair sums its stored D in blocks of 256
    q.ws_bgrad = 0;
    q.bgrad_parts = 0;
    if (is_bgrad(epilog)) {
        const bool col = bias_axis == GE_BIAS_COL;
        const int64_t parts = q.unfused ? ceil_div(col ? d.m : d.n, 256) : (col ? q.tiles_m : q.tiles_n);
        if (parts > 65535) return GE_ERR_SHAPE;
        q.bgrad_parts = (int32_t)parts;
        q.ws_bgrad = round_up(nb * (size_t)parts * (size_t)(col ? d.n : d.m) * sizeof(float), 256);
    }
    q.planned = true;
    q.pref = pr;
    *h = q;
    if (plan_log()) {
        char line[512];
        gemm_epilog_describe(h, line, sizeof line);
        fprintf(stderr, "gemm_epilog: plan %s\n", line);
    }
    return GE_OK;
}

int gemm_epilog_workspace_size(ge_handle h, size_t* bytes) {
    if (!h || !bytes) return GE_ERR_NULL;
    if (!h->planned) return GE_ERR_STATE;
    *bytes = h->ws_c + h->ws_partial + h->ws_counters + h->ws_bgrad;
    return GE_OK;
}

int gemm_epilog_aux_ld(ge_handle h, int64_t* ld_bits) {
    if (!h || !ld_bits) return GE_ERR_NULL;
    const int64_t ld = (int64_t)round_up((size_t)h->d.n, 128);
    *ld_bits = (h->planned && aux_is_matrix(h->epilog)) ? ld * 8 * elem_size(h->d.d_type) : ld;
    return GE_OK;
}

// execute and execute_c: cin (NULL = no added term) is C in D's dtype with
// row stride ldc, scaled by the device scalar *beta.  static_ws: the
// workspace is the library's own array (execute_static), not the caller's.
// Per-product byte strides of a launch (the packed layout unless the caller
// set strides), validated: GE_OK or an error status.
struct ProductStrides {
    int64_t a, b, bias, d, aux, c, sa, sb;
};

static int product_strides(const ge_plan_s& h, int64_t ldc, ProductStrides* out) {
    const ge_desc& d = h.d;
    const int64_t ea = elem_size(d.a_type), ed = elem_size(d.d_type), eb = elem_size(d.bias_type);
    const bool aux_matrix = aux_is_matrix(h.epilog);
    const int64_t aux_es = aux_matrix ? ed : 4;
    const int64_t len = h.axis == GE_BIAS_ROW ? d.m : d.n;
    const int64_t mx_ld = GE_MX_SCALE_LD(d.k);
    ge_batch_strides s = {d.m * d.lda, (d.op_b == GE_OP_N ? d.k : d.n) * d.ldb, len, d.m * d.ldd,
                          d.m * h.ldaux};
    if (h.bstr_set && d.batch > 1) {
        s = h.bstr;
        // inputs: any stride (0 shares one operand); rows stay 16-byte aligned
        if ((s.a * ea) % 16 || (s.b * ea) % 16 || (s.d * ed) % 16 || (s.aux * aux_es) % 16) return GE_ERR_ALIGN;
        if (h.axis == GE_BIAS_COL && has_bias(h.epilog) && (s.bias * eb) % 16) return GE_ERR_ALIGN;
        // outputs: no two products may write the same element
        if (s.d < (d.m - 1) * d.ldd + d.n) return GE_ERR_SHAPE;
        const bool aux_out = h.epilog == GE_EPILOG_RELU_AUX_BIAS || h.epilog == GE_EPILOG_GELU_AUX_BIAS;
        if (aux_out && s.aux < d.m * h.ldaux) return GE_ERR_SHAPE;
        if (is_bgrad(h.epilog) && s.bias < len) return GE_ERR_SHAPE;
    }
    out->a = s.a * ea;
    out->b = s.b * ea;
    out->bias = s.bias * eb;
    out->d = s.d * ed;
    out->aux = s.aux * aux_es;
    out->c = d.m * ldc * ed;
    out->sa = d.m * mx_ld;
    out->sb = d.n * mx_ld;
    return GE_OK;
}

// m_run < 0: the planned m; else the rows of this call (0 .. planned m).
static int execute_impl(ge_handle h, const void* A, const void* B, const void* cin, int64_t ldc, const float* beta,
                        const void* bias, void* D, void* aux, const float* scale_a, const float* scale_b,
                        void* workspace, size_t workspace_bytes, void* stream, bool static_ws = false,
                        const void* mx_a = nullptr, const void* mx_b = nullptr, int64_t m_run = -1) {
    if (!h) return GE_ERR_NULL;
    if (!h->planned || h->residual) return GE_ERR_STATE;
    const ge_desc& d = h->d;
    if (m_run > d.m) return GE_ERR_SHAPE;
    const int64_t M = m_run >= 0 ? m_run : d.m;   // rows of this call
    // block-scaled fp8: the scales come with execute_mx, and only with it
    const bool mx = d.a_type == GE_MXF8_E4M3;
    if (!mx && (mx_a || mx_b)) return GE_ERR_DTYPE;
    if (mx && ((!mx_a && M * d.k > 0) || (!mx_b && d.n * d.k > 0))) return GE_ERR_NULL;
    if (!aligned(mx_a, 16) || !aligned(mx_b, 16)) return GE_ERR_ALIGN;
    // a pointer may be NULL only when its buffer holds no elements
    if ((!A && M * d.k > 0) || (!B && d.k * d.n > 0) || (!D && M * d.n > 0)) return GE_ERR_NULL;
    const int64_t bias_len = h->axis == GE_BIAS_ROW ? M : d.n;
    if ((has_bias(h->epilog) || is_bgrad(h->epilog)) && !bias && bias_len > 0) return GE_ERR_NULL;
    const bool want_aux = has_aux(h->epilog) && M > 0 && d.n > 0;   // else aux holds nothing
    if (aux && !has_aux(h->epilog)) return GE_ERR_EPILOG;
    if (want_aux && !aux) return GE_ERR_EPILOG;
    if (cin) {
        if (h->d.d_type == GE_F8_E4M3) return GE_ERR_DTYPE;
        if (ldc < h->d.n) return GE_ERR_SHAPE;
        if ((ldc * elem_size(h->d.d_type)) % 16 || !aligned(cin, 16) || !aligned(beta, 4)) return GE_ERR_ALIGN;
    }
    if (!aligned(A, 16) || !aligned(B, 16) || !aligned(D, 16) || !aligned(bias, 16) || !aligned(aux, 16) ||
        !aligned(workspace, 16) || !aligned(scale_a, 4) || !aligned(scale_b, 4))
        return GE_ERR_ALIGN;
    ProductStrides ps;
    {
        const int st = product_strides(*h, cin ? ldc : 0, &ps);
        if (st != GE_OK) return st;
    }
    const size_t need = h->ws_c + h->ws_partial + h->ws_counters + h->ws_bgrad;
    if (static_ws) {
        if (need > (size_t)GE_STATIC_WORKSPACE_BYTES) return GE_ERR_STATIC_LIMIT;
    } else if (need > 0 && (!workspace || workspace_bytes < need)) {
        return GE_ERR_WORKSPACE;
    }
    if (test_fail_launch()) return GE_ERR_HIP;
    if (static_ws && need > 0) {
        // validation is done: only now the first HIP call
        const int st = scratch_of_current_device(&workspace);
        if (st != GE_OK) return st;
        workspace_bytes = (size_t)GE_STATIC_WORKSPACE_BYTES;
    }
    // fp8 output: amax starts from 0 at every call (a kernel, so that the
    // call can be captured in a HIP graph)
    if (h->amax_d && launch_clear_counters((uint32_t*)h->amax_d, d.batch > 1 ? d.batch : 1, stream) != 0)
        return GE_ERR_HIP;
    if (M == 0 || d.n == 0) {
        // empty output; a bias gradient over no rows (or columns) is zero
        if (is_bgrad(h->epilog) && bias_len > 0) {
            KernelArgs z;
            memset(&z, 0, sizeof(z));
            z.bias = bias;
            z.m = (int32_t)M;
            z.n = (int32_t)d.n;
            z.axis = h->axis;
            z.batch = d.batch > 1 ? d.batch : 1;
            z.bs_bias = ps.bias;
            if (launch_bgrad_reduce(d.d_type, z, 0, stream) != 0) return GE_ERR_HIP;
        }
        return GE_OK;
    }

    KernelArgs a;
    memset(&a, 0, sizeof(a));
    a.A = A;
    a.B = B;
    a.bias = bias;
    a.D = D;
    a.aux = (uint32_t*)aux;
    a.scale_a = scale_a;
    a.scale_b = scale_b;
    a.m = (int32_t)M;
    a.n = (int32_t)d.n;
    a.k = (int32_t)d.k;
    a.epilog = h->epilog;
    a.axis = h->axis;
    a.ldaux = (int32_t)h->ldaux;
    a.lda = d.lda;
    a.ldb = d.ldb;
    a.ldd = d.ldd;
    a.tiles_m = h->tiles_m;
    a.tiles_n = h->tiles_n;
    a.group_m = h->group_m;
    a.split_k = h->split_k;
    a.k_per_split = h->k_per_split;
    a.k_stagger = h->k_stagger;
    unsigned grid = h->grid;
    int32_t bgrad_parts = h->bgrad_parts;
    if (h->path != PATH_SMALLM && M != d.m) {
        // fewer rows than planned: the same kernel over the tile rows there are
        const TileShape* t = find_tile(h->tile_id);
        a.tiles_m = (int32_t)ceil_div(M, t->bm);
        grid = (unsigned)(a.tiles_m * (int64_t)a.tiles_n);
        if (is_bgrad(h->epilog) && h->axis == GE_BIAS_COL)
            bgrad_parts = (int32_t)(h->unfused ? ceil_div(M, 256) : a.tiles_m);
    }
    // batched: per-product strides in bytes (counters: elements); the
    // workspace parts keep their planned (largest) size
    const int64_t len = h->axis == GE_BIAS_COL ? d.n : d.m;
    a.batch = d.batch > 1 ? d.batch : 1;
    a.bs_part = h->split_k > 1 ? h->part_bytes : (int64_t)h->bgrad_parts * len * (int64_t)sizeof(float);
    a.bs_cnt = h->n_counters;
    a.bs_a = ps.a;
    a.bs_b = ps.b;
    a.bs_bias = ps.bias;
    a.bs_d = ps.d;
    a.bs_aux = ps.aux;
    a.bs_c = ps.c;
    a.cin = cin;
    a.beta = beta;
    a.ldc = ldc;
    a.scale_d = h->scale_d;
    a.amax = h->amax_d;
    uint8_t* ws = (uint8_t*)workspace;
    if (h->split_k > 1) {
        a.partial = (float*)(ws + h->ws_c);
        a.counters = (uint32_t*)(ws + h->ws_c + h->ws_partial);
        if (launch_clear_counters(a.counters, (int)(h->n_counters * a.batch), stream) != 0) return GE_ERR_HIP;
    }

    if (is_bgrad(h->epilog)) a.partial = (float*)(ws + h->ws_c + h->ws_partial + h->ws_counters);

    KernelArgs k1 = a;
    if (h->unfused) {
        // kernel 1: the plain product, rounded to d_type, into the workspace
        k1.epilog = GE_EPILOG_NONE;
        k1.cin = nullptr;   // the second kernel adds beta * C
        k1.bias = nullptr;
        k1.aux = nullptr;
        k1.ldaux = 0;
        k1.D = ws;
        k1.bs_d = M * d.ldd * elem_size(d.d_type);   // packed, as the second kernel reads it
    }
    int err;
    if (h->path == PATH_SMALLM) {
        err = launch_smallm(d.a_type, d.d_type, d.op_b, h->group_m, k1, grid, stream);
    } else if (mx) {
        const MxArgs mxa = {(const uint8_t*)mx_a, (const uint8_t*)mx_b, (int32_t)GE_MX_SCALE_LD(d.k),
                            (int32_t)ceil_div(d.k, 32), ps.sa, ps.sb};
        err = launch_tile_mx(h->tile_id, d.d_type, d.op_b, k1, mxa, grid, stream);
    } else {
        err = launch_tile(h->tile_id, d.a_type, d.d_type, d.op_b, k1, grid, stream);
    }
    if (err != 0) return GE_ERR_HIP;
    if (h->unfused) {
        // kernel 2: D = act(C + bias) (+ mask)
        err = launch_elementwise(d.d_type, a, ws, stream);
        if (err != 0) return GE_ERR_HIP;
        // the bias gradient of the stored D
        if (is_bgrad(h->epilog) && launch_bgrad_sum(d.d_type, a, bgrad_parts, stream) != 0)
            return GE_ERR_HIP;
    }
    if (is_bgrad(h->epilog) && launch_bgrad_reduce(d.d_type, a, bgrad_parts, stream) != 0) return GE_ERR_HIP;
    return GE_OK;
}

int gemm_epilog_execute(ge_handle h, const void* A, const void* B, const void* bias, void* D, void* aux,
                        const float* scale_a, const float* scale_b, void* workspace, size_t workspace_bytes,
                        void* stream) {
    return execute_impl(h, A, B, nullptr, 0, nullptr, bias, D, aux, scale_a, scale_b, workspace, workspace_bytes,
                        stream);
}

int gemm_epilog_execute_c(ge_handle h, const void* A, const void* B, const void* C, int64_t ldc,
                          const float* beta, const void* bias, void* D, void* aux, const float* scale_a,
                          const float* scale_b, void* workspace, size_t workspace_bytes, void* stream) {
    if (!h) return GE_ERR_NULL;
    if (!beta || (!C && h->d.m * h->d.n > 0)) return GE_ERR_NULL;
    return execute_impl(h, A, B, C, ldc, beta, bias, D, aux, scale_a, scale_b, workspace, workspace_bytes, stream);
}

int gemm_epilog_execute_mx(ge_handle h, const void* A, const void* B, const void* a_scales, const void* b_scales,
                           const void* bias, void* D, void* aux, const float* scale_a, const float* scale_b,
                           void* workspace, size_t workspace_bytes, void* stream) {
    if (!h) return GE_ERR_NULL;
    if (h->d.a_type != GE_MXF8_E4M3) return GE_ERR_DTYPE;
    return execute_impl(h, A, B, nullptr, 0, nullptr, bias, D, aux, scale_a, scale_b, workspace, workspace_bytes,
                        stream, false, a_scales, b_scales);
}

int gemm_epilog_execute_m(ge_handle h, int64_t m, const void* A, const void* B, const void* bias, void* D,
                          void* aux, const float* scale_a, const float* scale_b, void* workspace,
                          size_t workspace_bytes, void* stream) {
    if (!h) return GE_ERR_NULL;
    if (m < 0 || m > h->d.m) return GE_ERR_SHAPE;
    if (h->d.a_type == GE_MXF8_E4M3) return GE_ERR_DTYPE;   // block scales come with execute_mx
    return execute_impl(h, A, B, nullptr, 0, nullptr, bias, D, aux, scale_a, scale_b, workspace, workspace_bytes,
                        stream, false, nullptr, nullptr, m);
}

int gemm_epilog_set_fp8_output(ge_handle h, const float* scale_d, float* amax_d) {
    if (!h) return GE_ERR_NULL;
    if (h->d.d_type != GE_F8_E4M3) return GE_ERR_DTYPE;
    if (!aligned(scale_d, 4) || !aligned(amax_d, 4)) return GE_ERR_ALIGN;
    h->scale_d = scale_d;
    h->amax_d = amax_d;
    return GE_OK;
}

int gemm_epilog_set_batch_strides(ge_handle h, const ge_batch_strides* s) {
    if (!h) return GE_ERR_NULL;
    if (!s) {
        h->bstr_set = false;
        return GE_OK;
    }
    if (s->a < 0 || s->b < 0 || s->bias < 0 || s->d < 0 || s->aux < 0) return GE_ERR_SHAPE;
    h->bstr = *s;
    h->bstr_set = true;
    return GE_OK;
}

int gemm_epilog_execute_static(ge_handle h, const void* A, const void* B, const void* bias, void* D, void* aux,
                               const float* scale_a, const float* scale_b, void* stream) {
    return execute_impl(h, A, B, nullptr, 0, nullptr, bias, D, aux, scale_a, scale_b, nullptr, 0, stream, true);
}

// ---- residual product ---------------------------------------------------------
// Few rows and a weight given n x k: W is streamed once.  Up to 64 rows, against
// the split-K tiles (us, streaming / tiles, at 1, 32 and 64 rows):
//   bf16 1024 x 1024 (n x k), 33 and 64 rows: 6.0 / 7.1, 6.4 / 7.3; 2048 x 2048: 8.0 / 10.6, 8.4 / 10.7
//     4096 x 4096 9.8 / 14.9, 12.4 / 14.9, 16.5 / 15.4; 1024 x 8192 8.9 / 13.2, 13.2 / 13.4, 17.6 / 13.6
//     4096 x 16384 31 / 37, 39 / 37, 50 / 38; 16384 x 4096 35 / 33, 37 / 33, 40 / 33
//   E4M3 4096 x 4096 6.4 / 11.9, 7.9 / 12.2, 9.2 / 12.9; 4096 x 16384 15.2 / 25.1, 19.8 / 25.6, 24.8 / 26.0
//   block-scaled 4096 x 4096 7.1 / 19.3, 8.8 / 19.8, 12.4 / 20.7; 4096 x 16384 15.7 / 35, 27 / 37, 41 / 38
// The limit is one for every type, though with 33 rows and more of large 16-bit
// weights the tiles win (x, read by every workgroup, is then more bytes than W).
static bool few_rows(const ge_desc& d, int64_t m) { return m <= 64 && d.op_b == GE_OP_T && d.a_type != GE_F32; }

// The streaming kernel for m rows: groups of 16 rows and of 16 columns per workgroup.
struct FewRowsShape {
    int32_t mb, rg, blocks;
};
static FewRowsShape few_rows_shape(const ge_desc& d, int64_t m) {
    const int32_t rg = ceil_div(d.n, 32) >= 256 ? 2 : 1;
    return {m <= 16 ? 1 : m <= 32 ? 2 : 4, rg, (int32_t)ceil_div(d.n, 16 * rg)};
}

int gemm_epilog_plan_residual(ge_handle h, int32_t epilog, int32_t bias_axis) {
    if (!h) return GE_ERR_NULL;
    const bool known = epilog == GE_EPILOG_NONE || has_bias(epilog);
    if (!known || (bias_axis != GE_BIAS_ROW && bias_axis != GE_BIAS_COL)) return GE_ERR_EPILOG;
    const ge_desc& d = h->d;
    if (d.batch > 1) return GE_ERR_SHAPE;
    if (d.d_type == GE_F8_E4M3) return GE_ERR_DTYPE;
    ge_plan_s q = *h;
    q.planned = true;
    q.residual = true;
    q.backward = false;
    q.epilog = epilog;
    q.axis = bias_axis;
    q.unfused = 0;
    q.pref = {0, 0, 0, 0, 0};
    q.k_stagger = 0;
    q.split_k = 1;
    q.k_per_split = (int32_t)d.k;
    q.ws_c = q.ws_partial = q.ws_counters = q.ws_bgrad = 0;
    q.n_counters = q.part_bytes = 0;
    q.bgrad_parts = 0;
    q.ldaux = !has_aux(epilog) ? 0
              : aux_is_matrix(epilog) ? (int64_t)round_up((size_t)d.n, 128)
                                      : (int64_t)round_up((size_t)d.n, 128) / 32;
    if (q.ldaux > INT32_MAX) return GE_ERR_SHAPE;
    if (few_rows(d, d.m)) {
        const FewRowsShape f = few_rows_shape(d, d.m);
        q.path = PATH_SKINNY;
        q.tile_id = 0;
        q.skinny_mb = f.mb;
        q.group_m = f.rg;
        q.tiles_m = 1;
        q.tiles_n = f.blocks;
        q.grid = (unsigned)f.blocks;
    } else {
        q.path = PATH_TILE;
        q.tile_id = choose_res_tile(d);
        const TileShape* t = find_res_tile(q.tile_id);
        if (!t || !tile_span_ok(t, d)) return GE_ERR_SHAPE;
        const int64_t tm = ceil_div(d.m, t->bm), tn = ceil_div(d.n, t->bn);
        if (tm * tn > INT32_MAX) return GE_ERR_SHAPE;
        q.tiles_m = (int32_t)tm;
        q.tiles_n = (int32_t)tn;
        q.group_m = auto_group_m(t, tm, d.a_type);
        q.k_stagger = auto_k_stagger(t, d.a_type);
        q.grid = (unsigned)(tm * tn);
        if (t->kernel == 5) {
            const int64_t step = elem_size(d.a_type) == 2 ? 64 : 128, steps = ceil_div(d.k, step);
            const int split = res_split(t, d.a_type, tm * tn, steps);
            q.k_per_split = (int32_t)(ceil_div(steps, split) * step);
            q.split_k = q.k_per_split > 0 ? (int32_t)ceil_div(d.k, q.k_per_split) : 1;
            if (q.split_k < 1) q.split_k = 1;
            if (q.split_k > 1) {
                q.n_counters = tm * tn;
                q.part_bytes = tm * tn * q.split_k * (int64_t)t->bm * t->bn * (int64_t)sizeof(float);
                q.ws_partial = round_up((size_t)q.part_bytes, 256);
                q.ws_counters = round_up((size_t)q.n_counters * sizeof(uint32_t), 256);
            }
        }
    }
    *h = q;
    if (plan_log()) {
        char line[512];
        gemm_epilog_describe(h, line, sizeof line);
        fprintf(stderr, "gemm_epilog: residual plan %s\n", line);
    }
    return GE_OK;
}

int gemm_epilog_execute_residual(ge_handle h, int64_t m, const void* A, const void* B, const void* a_scales,
                                 const void* b_scales, const void* bias, const void* residual, int64_t ldr,
                                 const float* row_scale, const float* col_scale, const float* scale_a,
                                 const float* scale_b, void* D, void* aux, void* workspace, size_t workspace_bytes,
                                 void* stream) {
    if (!h) return GE_ERR_NULL;
    if (!h->planned || !h->residual) return GE_ERR_STATE;
    const ge_desc& d = h->d;
    if (m < 0 || m > d.m) return GE_ERR_SHAPE;
    const bool mx = d.a_type == GE_MXF8_E4M3;
    if (!mx && (a_scales || b_scales)) return GE_ERR_DTYPE;
    if (mx && ((!a_scales && m * d.k > 0) || (!b_scales && d.n * d.k > 0))) return GE_ERR_NULL;
    if ((!A && m * d.k > 0) || (!B && d.k * d.n > 0) || (!D && m * d.n > 0)) return GE_ERR_NULL;
    if (has_bias(h->epilog) && !bias && (h->axis == GE_BIAS_ROW ? m : d.n) > 0) return GE_ERR_NULL;
    if (aux && !has_aux(h->epilog)) return GE_ERR_EPILOG;
    if (!aux && has_aux(h->epilog) && m * d.n > 0) return GE_ERR_EPILOG;
    if (residual && ldr < d.n) return GE_ERR_SHAPE;
    if (residual && (ldr * elem_size(d.d_type)) % 16) return GE_ERR_ALIGN;
    if (!aligned(A, 16) || !aligned(B, 16) || !aligned(D, 16) || !aligned(bias, 16) || !aligned(aux, 16) ||
        !aligned(a_scales, 16) || !aligned(b_scales, 16) || !aligned(residual, 16) || !aligned(col_scale, 16) ||
        !aligned(workspace, 16) || !aligned(row_scale, 4) || !aligned(scale_a, 4) || !aligned(scale_b, 4))
        return GE_ERR_ALIGN;
    // in place each value has to lie where it is written: with another stride a row of D
    // would overwrite rows of R that other workgroups still read
    if (residual && residual == D && ldr != d.ldd && m > 1) return GE_ERR_SHAPE;
    const size_t need = h->ws_partial + h->ws_counters;
    if (need > 0 && (!workspace || workspace_bytes < need)) return GE_ERR_WORKSPACE;
    if (test_fail_launch()) return GE_ERR_HIP;
    if (m == 0 || d.n == 0) return GE_OK;

    KernelArgs a;
    memset(&a, 0, sizeof(a));
    a.A = A;
    a.B = B;
    a.bias = has_bias(h->epilog) ? bias : nullptr;
    a.D = D;
    a.aux = (uint32_t*)aux;
    a.scale_a = scale_a;
    a.scale_b = scale_b;
    a.m = (int32_t)m;
    a.n = (int32_t)d.n;
    a.k = (int32_t)d.k;
    a.epilog = h->epilog;
    a.axis = h->axis;
    a.ldaux = (int32_t)h->ldaux;
    a.lda = d.lda;
    a.ldb = d.ldb;
    a.ldd = d.ldd;
    a.tiles_m = h->tiles_m;
    a.tiles_n = h->tiles_n;
    a.group_m = h->group_m;
    a.split_k = h->split_k;
    a.k_per_split = h->k_per_split;
    a.k_stagger = h->k_stagger;
    a.batch = 1;
    ResArgs r = {};
    r.sa = (const uint8_t*)a_scales;
    r.sb = (const uint8_t*)b_scales;
    r.ld = (int32_t)GE_MX_SCALE_LD(d.k);
    r.kb = (int32_t)ceil_div(d.k, 32);
    r.res = residual;
    r.row_scale = row_scale;
    r.col_scale = col_scale;
    r.ldr = ldr;
    // by this call's rows, not the plan's: a handle for prompts serves single tokens too, and its
    // tiles would walk all of K in a few workgroups (1 x 4096 x 16384 bf16 on a handle of 8192
    // rows 258 us, streamed 30; 64 rows on handles of 100 and 300 rows 51 and 80, streamed 49)
    if (few_rows(d, m)) {
        const FewRowsShape f = few_rows_shape(d, m);
        a.tiles_m = 1;
        a.tiles_n = f.blocks;
        return launch_skinny(d.a_type, d.d_type, f.mb, f.rg, a, r, (unsigned)f.blocks, stream) == 0 ? GE_OK
                                                                                                    : GE_ERR_HIP;
    }
    unsigned grid = h->grid;
    if (m != d.m) {
        a.tiles_m = (int32_t)ceil_div(m, find_res_tile(h->tile_id)->bm);
        grid = (unsigned)(a.tiles_m * (int64_t)a.tiles_n);
    }
    if (h->split_k > 1) {
        a.partial = (float*)workspace;
        a.counters = (uint32_t*)((uint8_t*)workspace + h->ws_partial);
        if (launch_clear_counters(a.counters, (int)h->n_counters, stream) != 0) return GE_ERR_HIP;
    }
    return launch_tile_res(h->tile_id, d.a_type, d.d_type, d.op_b, a, r, grid, stream) == 0 ? GE_OK : GE_ERR_HIP;
}

// ---- its backward pass ----------------------------------------------------------
// dA takes a weight k x n as its n x k operand, so the pair, which runs one
// layout, takes dB = A^T dP with both operands transposed then: dP^T beside A^T.
static ge_desc pair_desc_b(const ge_plan_s* h) {
    ge_desc b = h->g_b->d;
    if (h->d.op_b == GE_OP_N) {
        b.op_b = GE_OP_T;
        b.ldb = h->ld_t;
    }
    return b;
}

// The tile that runs both gradients' products in one launch, or 0: not for
// fp32, nor where a product is small enough for its plan to split its
// reduction, nor where each fills the chip many times over.  By both products'
// tiles together: 256 x 256 if they fill the chip, else 128 x 128 if those do, else
// 64 x 64.  Measured, bf16, weight n x k, us (m x n x k: tiles of 256 x 256 and 128 x 128;
// two launches, one of 256 x 256, 128 x 128, 64 x 64):
//   512 x 512 x 512 (8, 32)         19, 21, 13, 9
//   1000 x 520 x 1032 (35, 117)     27, 33, 20, 16
//   2133 x 952 x 1128 (65, 225)     52, 57, 41, 35
//   2048 x 2048 x 1024 (64, 256)    50, 49, 30, 38
//   2048 x 2048 x 2048 (128, 512)   82, 52, 50, 61
//   5687 x 1840 x 1232 (155, 600)   144, 129, 101, 135
//   2048 x 1024 x 4096 (192, 768)   78, 52, 54, 61
//   4096 x 4096 x 2048 (256, 1024)  184, 129, 153, 207
//   4096 x 4096 x 4096 (512, 2048)  327, 228, 290, 391
//   4096 x 16384 x 4096 (1280)      1230, 887, 1332, 1832
//   8192 x 8192 x 8192 (2048)       1667, 1666, 2590, 4159
//   8192 x 4096 x 16384 (3072)      1727, 1754, 2634, 3447
static int choose_pair_tile(const ge_plan_s* h) {
    for (const ge_plan_s* g : {h->g_a, h->g_b}) {
        if (elem_size(g->d.a_type) != 2 || g->path != PATH_TILE) return 0;
        if (g->tile_id != 6 && g->tile_id != 8 && g->tile_id != 13) return 0;
        if (g->d.m < 1 || g->d.n < 1 || g->d.k < 1) return 0;
    }
    const ge_desc &a = h->g_a->d, b = pair_desc_b(h);
    const int64_t t256 = ceil_div(a.m, 256) * ceil_div(a.n, 256) + ceil_div(b.m, 256) * ceil_div(b.n, 256);
    const int64_t t128 = ceil_div(a.m, 128) * ceil_div(a.n, 128) + ceil_div(b.m, 128) * ceil_div(b.n, 128);
    if (t256 >= 2048) return 0;
    const int id = t256 >= 256 ? 6 : t128 >= 256 ? 8 : 13;
    const TileShape* t = find_tile(id);
    return tile_span_ok(t, a) && tile_span_ok(t, b) ? id : 0;
}

// One of them: D = A B.
static KernelArgs pair_args(const ge_desc& d, int tile, const void* A, const void* B, void* D) {
    const TileShape* t = find_tile(tile);
    KernelArgs a;
    memset(&a, 0, sizeof(a));
    a.A = A;
    a.B = B;
    a.D = D;
    a.m = (int32_t)d.m;
    a.n = (int32_t)d.n;
    a.k = (int32_t)d.k;
    a.epilog = GE_EPILOG_NONE;
    a.axis = GE_BIAS_COL;
    a.lda = d.lda;
    a.ldb = d.ldb;
    a.ldd = d.ldd;
    a.tiles_m = (int32_t)ceil_div(d.m, t->bm);
    a.tiles_n = (int32_t)ceil_div(d.n, t->bn);
    a.group_m = auto_group_m(t, a.tiles_m, d.a_type);
    a.split_k = 1;
    a.k_per_split = a.k;
    a.k_stagger = auto_k_stagger(t, d.a_type);
    a.batch = 1;
    return a;
}

// dA (m x k) = dP B^T and dB = A^T dP (k x n) or dP^T A (n x k), both on the
// tile kernels.  Those take A untransposed, so the reduction over the rows of
// dP needs dP^T (weight n x k) or A^T (weight k x n) laid out once.
int gemm_epilog_plan_backward(ge_handle h) {
    if (!h) return GE_ERR_NULL;
    if (!h->planned || !h->residual) return GE_ERR_STATE;
    const ge_desc& d = h->d;
    if (d.a_type != d.d_type || elem_size(d.a_type) < 2) return GE_ERR_DTYPE;
    const int e = h->epilog;
    if (e != GE_EPILOG_NONE && e != GE_EPILOG_BIAS && e != GE_EPILOG_RELU_AUX_BIAS && e != GE_EPILOG_GELU_AUX_BIAS)
        return GE_ERR_EPILOG;
    const int64_t es = elem_size(d.a_type), per = 16 / es;
    if (ceil_div(d.m, kGradTile) > 65535) return GE_ERR_SHAPE;
    ge_plan_s q = *h;
    const bool act = has_aux(e);   // dP differs from dD
    q.ld_dp = act ? (int64_t)round_up((size_t)d.n, per) : d.ldd;
    q.bw_dp = act ? round_up((size_t)d.m * q.ld_dp * es, 256) : 0;
    q.ld_t = (int64_t)round_up((size_t)d.m, per);
    const bool kn = d.op_b == GE_OP_N;
    q.bw_t = round_up((size_t)(kn ? d.k : d.n) * q.ld_t * es, 256);
    q.bw_part = e == GE_EPILOG_NONE ? 0
                : round_up((h->axis == GE_BIAS_COL ? (size_t)ceil_div(d.m, kGradTile) * d.n
                                                   : (size_t)ceil_div(d.n, kGradTile) * d.m) * sizeof(float), 256);
    // dA: dP (m x n) times B^T; B given n x k is k-major for it (OP_N)
    const ge_desc da = {d.m, d.k, d.n, d.a_type, d.a_type, d.a_type, d.a_type, kn ? GE_OP_T : GE_OP_N, 0,
                        q.ld_dp, d.ldb, d.lda};
    // dB, k x n: A^T (k x m) times dP; n x k: dP^T (n x m) times A
    const ge_desc db = {kn ? d.k : d.n, kn ? d.n : d.k, d.m, d.a_type, d.a_type, d.a_type, d.a_type, GE_OP_N, 0,
                        q.ld_t, kn ? q.ld_dp : d.lda, d.ldb};
    ge_handle ga = nullptr, gb = nullptr;
    int st = gemm_epilog_create(&ga, &da);
    if (st == GE_OK) st = gemm_epilog_create(&gb, &db);
    if (st == GE_OK) st = gemm_epilog_plan(ga, GE_EPILOG_NONE, GE_BIAS_COL, nullptr);
    if (st == GE_OK) st = gemm_epilog_plan(gb, GE_EPILOG_NONE, GE_BIAS_COL, nullptr);
    if (st != GE_OK) {
        gemm_epilog_free(ga);
        gemm_epilog_free(gb);
        return st;
    }
    size_t wa = 0, wb = 0;
    gemm_epilog_workspace_size(ga, &wa);
    gemm_epilog_workspace_size(gb, &wb);
    q.bw_gemm = wa > wb ? wa : wb;   // the products run one after the other
    delete q.g_a;
    delete q.g_b;
    q.g_a = ga;
    q.g_b = gb;
    q.pair_tile = choose_pair_tile(&q);
    q.bw_t2 = q.pair_tile && kn ? round_up((size_t)d.n * q.ld_t * es, 256) : 0;
    q.backward = true;
    *h = q;
    return GE_OK;
}

int gemm_epilog_backward_workspace_size(ge_handle h, size_t* bytes) {
    if (!h || !bytes) return GE_ERR_NULL;
    if (!h->backward) return GE_ERR_STATE;
    *bytes = h->bw_dp + h->bw_t + h->bw_t2 + h->bw_part + h->bw_gemm;
    return GE_OK;
}

int gemm_epilog_backward(ge_handle h, const void* dD, const void* A, const void* B, const void* aux, void* dA, void* dB,
                         void* dbias, void* workspace, size_t workspace_bytes, void* stream) {
    if (!h) return GE_ERR_NULL;
    if (!h->planned || !h->residual || !h->backward) return GE_ERR_STATE;
    const ge_desc& d = h->d;
    const int e = h->epilog;
    const bool kn = d.op_b == GE_OP_N, act = has_aux(e);
    if ((!dD && d.m * d.n > 0) || (!A && d.m * d.k > 0 && dB) || (!B && d.k * d.n > 0 && dA)) return GE_ERR_NULL;
    if (aux && !act) return GE_ERR_EPILOG;
    if (!aux && act && d.m * d.n > 0) return GE_ERR_EPILOG;
    if (dbias && e == GE_EPILOG_NONE) return GE_ERR_EPILOG;
    if (!aligned(dD, 16) || !aligned(A, 16) || !aligned(B, 16) || !aligned(aux, 16) || !aligned(dA, 16) ||
        !aligned(dB, 16) || !aligned(dbias, 16) || !aligned(workspace, 16))
        return GE_ERR_ALIGN;
    const size_t need = h->bw_dp + h->bw_t + h->bw_t2 + h->bw_part + h->bw_gemm;
    if (need > 0 && (!workspace || workspace_bytes < need)) return GE_ERR_WORKSPACE;
    if (test_fail_launch()) return GE_ERR_HIP;
    uint8_t* ws = (uint8_t*)workspace;
    uint8_t *w_dp = ws, *w_t = ws + h->bw_dp, *w_t2 = w_t + h->bw_t, *w_part = w_t2 + h->bw_t2,
            *w_gemm = w_part + h->bw_part;
    const bool pair = (dA || dB) && h->pair_tile;
    // dP^T: the weight's gradient for a weight n x k, or for the pair
    uint8_t* dp_t = !dB ? nullptr : !kn ? w_t : pair ? w_t2 : nullptr;
    const void* dP = act ? w_dp : dD;
    const int64_t len = h->axis == GE_BIAS_COL ? d.n : d.m;
    // a sum over no rows (or columns) is zero; the products write zeros for an empty reduction
    if (d.m > 0 && d.n > 0 && (act || dbias || dp_t)) {
        GradArgs g = {};
        g.src = dD;
        g.aux = aux;
        g.dst = act ? w_dp : nullptr;
        g.dst_t = dp_t;
        g.partial = dbias ? (float*)w_part : nullptr;
        g.rows = (int32_t)d.m;
        g.cols = (int32_t)d.n;
        g.axis = h->axis;
        g.ldaux = (int32_t)h->ldaux;
        g.ld = d.ldd;
        g.ldd = h->ld_dp;
        g.ldt = h->ld_t;
        const int kind = e == GE_EPILOG_RELU_AUX_BIAS ? GRAD_MASK : e == GE_EPILOG_GELU_AUX_BIAS ? GRAD_GELU : GRAD_PLAIN;
        if (launch_grad_prepare(d.a_type, kind, g, stream) != 0) return GE_ERR_HIP;
    }
    const int parts = d.m > 0 && d.n > 0 ? (int)ceil_div(h->axis == GE_BIAS_COL ? d.m : d.n, kGradTile) : 0;
    if (dbias && len > 0 && !pair) {
        if (launch_grad_bias(d.a_type, (const float*)w_part, parts, (int)len, dbias, stream) != 0) return GE_ERR_HIP;
    }
    if (dB && kn && d.m > 0 && d.k > 0) {
        GradArgs g = {};
        g.src = A;
        g.dst_t = w_t;
        g.rows = (int32_t)d.m;
        g.cols = (int32_t)d.k;
        g.axis = GE_BIAS_COL;
        g.ld = d.lda;
        g.ldt = h->ld_t;
        if (launch_grad_prepare(d.a_type, GRAD_COPY, g, stream) != 0) return GE_ERR_HIP;
    }
    if (pair) {
        // one gradient alone runs the same kernel, the other without tiles: its
        // bits do not depend on what else is asked for
        KernelArgs pa = pair_args(h->g_a->d, h->pair_tile, dP, B, dA);
        KernelArgs pb = pair_args(pair_desc_b(h), h->pair_tile, w_t, kn ? (const void*)w_t2 : A, dB);
        if (!dA) pa.tiles_m = 0;
        if (!dB) pb.tiles_m = 0;
        // the longer reduction first: its tiles take longest
        const bool a_first = pa.k >= pb.k;
        PairArgs second = {a_first ? pb : pa, (const float*)w_part, dbias, parts, (int32_t)(dbias ? len : 0)};
        return launch_tile_pair(h->pair_tile, d.a_type, kn ? GE_OP_T : GE_OP_N, a_first ? pa : pb, second, stream) == 0
                   ? GE_OK : GE_ERR_HIP;
    }
    int st = GE_OK;
    if (dA)
        st = gemm_epilog_execute(h->g_a, dP, B, nullptr, dA, nullptr, nullptr, nullptr, h->bw_gemm ? w_gemm : nullptr,
                                 h->bw_gemm, stream);
    if (st == GE_OK && dB)
        st = gemm_epilog_execute(h->g_b, w_t, kn ? dP : A, nullptr, dB, nullptr, nullptr, nullptr,
                                 h->bw_gemm ? w_gemm : nullptr, h->bw_gemm, stream);
    return st;
}

int gemm_epilog_free(ge_handle h) {
    if (h) {
        delete h->g_a;
        delete h->g_b;
    }
    delete h;
    return GE_OK;
}

const char* gemm_epilog_status_string(int s) {
    switch (s) {
    case GE_OK: return "GE_OK: success";
    case GE_ERR_NULL: return "GE_ERR_NULL: a required pointer is NULL";
    case GE_ERR_SHAPE: return "GE_ERR_SHAPE: invalid dimension, leading dimension or plan option";
    case GE_ERR_DTYPE: return "GE_ERR_DTYPE: unsupported or mismatched dtypes";
    case GE_ERR_EPILOG: return "GE_ERR_EPILOG: invalid epilogue, bias axis or aux buffer";
    case GE_ERR_ALIGN: return "GE_ERR_ALIGN: pointer or row stride not 16-byte aligned";
    case GE_ERR_STATE: return "GE_ERR_STATE: handle not planned";
    case GE_ERR_WORKSPACE: return "GE_ERR_WORKSPACE: workspace missing or too small";
    case GE_ERR_HIP: return "GE_ERR_HIP: kernel launch failed";
    case GE_ERR_ALLOC: return "GE_ERR_ALLOC: host allocation failed";
    case GE_ERR_STATIC_LIMIT:
        return "GE_ERR_STATIC_LIMIT: the plan needs more workspace than the library's fixed array "
               "(GE_STATIC_WORKSPACE_BYTES)";
    }
    return "unknown status";
}

int gemm_epilog_autotune(ge_handle h, const void* A, const void* B, const void* bias, void* D, void* aux,
                         const float* scale_a, const float* scale_b, void* workspace, size_t workspace_bytes,
                         int32_t iters, void* stream, float* best_ms) {
    if (!h) return GE_ERR_NULL;
    if (!h->planned || h->residual) return GE_ERR_STATE;
    if (iters < 1) return GE_ERR_SHAPE;
    const ge_plan_s orig = *h;
    // candidates: tile ids (tile path) or row groups x K splits (small-m
    // path, encoded as 256 * row groups + split)
    int cand[kNumTiles + 24];
    int nc = 0;
    if (orig.path == PATH_SMALLM) {
        const int64_t spans = ceil_div(orig.d.k, 64);
        for (int rg = 1; rg <= 4; rg *= 2)
            for (int s = 1; s <= 64 && s <= (spans > 0 ? spans : 1); s *= 2) cand[nc++] = 256 * rg + s;
    } else {
        for (int i = 0; i < kNumTiles; ++i) cand[nc++] = kTiles[i].id;
    }
    hipEvent_t e0 = nullptr, e1 = nullptr;
    if (hipEventCreate(&e0) != hipSuccess) return GE_ERR_HIP;
    if (hipEventCreate(&e1) != hipSuccess) {
        (void)hipEventDestroy(e0);
        return GE_ERR_HIP;
    }
    ge_plan_s best = orig;
    float best_t = -1.0f;
    int status = GE_OK;
    for (int c = 0; c < nc && status == GE_OK; ++c) {
        ge_pref pr = orig.pref;
        if (orig.path == PATH_SMALLM) {
            pr.path = PATH_SMALLM;
            pr.group_m = cand[c] / 256;
            pr.split_k = cand[c] % 256;
        } else {
            pr.path = PATH_TILE;
            pr.tile = cand[c];
        }
        ge_plan_s trial = orig;
        if (gemm_epilog_plan(&trial, orig.epilog, orig.axis, &pr) != GE_OK) continue;   // not for this dtype
        size_t need = 0;
        gemm_epilog_workspace_size(&trial, &need);
        if (need > workspace_bytes) continue;
        // one untimed call (also validates the arguments), then the timed ones
        int r = gemm_epilog_execute(&trial, A, B, bias, D, aux, scale_a, scale_b, workspace, workspace_bytes,
                                    stream);
        if (r != GE_OK) {
            status = r;
            break;
        }
        if (hipEventRecord(e0, (hipStream_t)stream) != hipSuccess) { status = GE_ERR_HIP; break; }
        for (int i = 0; i < iters && r == GE_OK; ++i)
            r = gemm_epilog_execute(&trial, A, B, bias, D, aux, scale_a, scale_b, workspace, workspace_bytes,
                                    stream);
        if (r != GE_OK) { status = r; break; }
        float ms = 0.0f;
        if (hipEventRecord(e1, (hipStream_t)stream) != hipSuccess || hipEventSynchronize(e1) != hipSuccess ||
            hipEventElapsedTime(&ms, e0, e1) != hipSuccess) {
            status = GE_ERR_HIP;
            break;
        }
        ms /= (float)iters;
        if (best_t < 0.0f || ms < best_t) {
            best_t = ms;
            best = trial;
        }
    }
    (void)hipEventDestroy(e0);
    (void)hipEventDestroy(e1);
    if (status != GE_OK) return status;
    if (best_t < 0.0f) return GE_ERR_WORKSPACE;   // no candidate fits the workspace
    best.pref = orig.pref;
    *h = best;
    if (best_ms) *best_ms = best_t;
    return GE_OK;
}

int gemm_epilog_describe(ge_handle h, char* buf, size_t cap) {
    if (!h || !buf) return GE_ERR_NULL;
    if (cap == 0) return GE_OK;
    const ge_desc& d = h->d;
    if (!h->planned) {
        snprintf(buf, cap, "m=%lld n=%lld k=%lld unplanned", (long long)d.m, (long long)d.n, (long long)d.k);
        return GE_OK;
    }
    const TileShape* t = h->residual ? find_res_tile(h->tile_id) : find_tile(h->tile_id);
    if (h->path == PATH_SKINNY) {
        snprintf(buf, cap, "m=%lld n=%lld k=%lld a=%d d=%d op_b=%d epilog=%d axis=%d path=skinny rows=%d cols=%d grid=%u "
                 "workspace=0 residual=1", (long long)d.m, (long long)d.n, (long long)d.k, d.a_type, d.d_type, d.op_b,
                 h->epilog, h->axis, 16 * h->skinny_mb, 16 * h->group_m, h->grid);
        return GE_OK;
    }
    snprintf(buf, cap,
             "m=%lld n=%lld k=%lld a=%d d=%d op_b=%d epilog=%d axis=%d path=%s tile=%dx%d waves=%dx%d "
             "tile_id=%d kernel=%d stages=%d grid=%u group_m=%d split_k=%d unfused=%d workspace=%zu "
             "ldaux_words=%lld k_stagger=%d%s",
             (long long)d.m, (long long)d.n, (long long)d.k, d.a_type, d.d_type, d.op_b, h->epilog, h->axis,
             h->path == PATH_SMALLM ? "smallm" : "tile", t ? t->bm : 16, t ? t->bn : 16 * h->group_m, t ? t->wm : 1,
             t ? t->wn : 8, h->tile_id, t ? t->kernel : 0,
             t ? (t->kernel >= 2 && t->kernel != 3 ? tile2_stages(*t, elem_size(d.a_type)) : t->stages) : 0, h->grid, h->group_m,
             h->split_k,
             h->unfused,
             h->ws_c + h->ws_partial + h->ws_counters + h->ws_bgrad, (long long)h->ldaux,
             h->k_stagger, h->residual ? " residual=1" : "");
    return GE_OK;
}

}  // extern "C"
