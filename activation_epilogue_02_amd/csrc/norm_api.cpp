// norm_api.cpp -- the C-ABI front end of the RMS norm: validation, launch
// shapes, workspace.  Every check runs before any HIP runtime call.
#include <math.h>
#include <stdio.h>

#include <new>

#include "ge_host.h"
#include "norm_params.h"

using namespace ge;

struct ge_norm_s {
    ge_norm_desc d;
    NormShape fwd, bwd;
};

namespace {

// The smallest shape of a table whose threads hold a row in registers.
template <int N>
NormShape pick_shape(const NormShape (&table)[N], int64_t chunks) {
    for (int i = 0; i < N; ++i)
        if ((int64_t)table[i].threads * table[i].chunks >= chunks) return table[i];
    return kNormLong;
}

// Workgroups of a forward launch: one per row (per four of the one-wave
// shapes), up to a grid that the runtime takes; beyond it they walk the rows.
int64_t forward_blocks(const NormShape& s, int64_t rows) {
    const int64_t need = s.threads == 64 ? ceil_div(rows, 4) : rows;
    return need < 1 << 20 ? need : 1 << 20;
}

// Of a backward launch: one per CU, each walking rows blockIdx, blockIdx +
// blocks, ... (see norm_bwd).
int64_t backward_blocks(int64_t rows) { return rows < 256 ? rows : 256; }

size_t partial_bytes(const ge_norm_s& h, int64_t rows) {
    return round_up((size_t)backward_blocks(rows) * (size_t)h.d.cols * sizeof(float), 256);
}

}  // namespace

extern "C" {

int ge_rms_norm_create(ge_norm_handle* h, const ge_norm_desc* desc) {
    if (!h || !desc) return GE_ERR_NULL;
    *h = nullptr;
    const ge_norm_desc& d = *desc;
    if (d.rows < 0 || d.cols < 1 || d.rows > INT32_MAX || d.cols > INT32_MAX) return GE_ERR_SHAPE;
    if (d.out < GE_NORM_PLAIN || d.out > GE_NORM_MX) return GE_ERR_SHAPE;
    if (!(d.eps >= 0.0f) || !isfinite(d.eps)) return GE_ERR_SHAPE;
    if (d.type != GE_F32 && d.type != GE_F16 && d.type != GE_BF16) return GE_ERR_DTYPE;
    if (d.ld < d.cols || d.ldy < d.cols) return GE_ERR_SHAPE;
    const int es = elem_size(d.type);
    if ((d.ld * es) % 16 || (d.ldy * (d.out == GE_NORM_PLAIN ? es : 1)) % 16) return GE_ERR_ALIGN;
    ge_norm_s* p = new (std::nothrow) ge_norm_s();
    if (!p) return GE_ERR_ALLOC;
    p->d = d;
    const int64_t chunks = ceil_div(d.cols * es, 16);
    p->fwd = pick_shape(kNormFwd, chunks);
    p->bwd = pick_shape(kNormBwd, chunks);
    *h = p;
    if (plan_log()) {
        char line[256];
        ge_rms_norm_describe(p, line, sizeof line);
        fprintf(stderr, "ge_rms_norm: plan %s\n", line);
    }
    return GE_OK;
}

int ge_rms_norm_workspace_size(ge_norm_handle h, size_t* bytes) {
    if (!h || !bytes) return GE_ERR_NULL;
    *bytes = partial_bytes(*h, h->d.rows);
    return GE_OK;
}

int ge_rms_norm_forward(ge_norm_handle h, int64_t rows, const void* x, const void* residual, const void* gamma,
                        void* hsum, void* y, void* scales, float* rstd, void* stream) {
    if (!h) return GE_ERR_NULL;
    const ge_norm_desc& d = h->d;
    if (rows < 0 || rows > d.rows) return GE_ERR_SHAPE;
    if (!gamma || (rows > 0 && (!x || !y))) return GE_ERR_NULL;
    if (hsum && !residual) return GE_ERR_EPILOG;
    if (rows > 0 && (d.out == GE_NORM_PLAIN) != (scales == nullptr)) return GE_ERR_EPILOG;
    if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(gamma, 16) || !aligned(hsum, 16) || !aligned(y, 16) ||
        !aligned(scales, d.out == GE_NORM_MX ? 16 : 4) || !aligned(rstd, 4))
        return GE_ERR_ALIGN;
    // in place each value has to lie where it is written: with other rows (a stride of its own, or
    // 8-bit ones) y would overwrite rows that other workgroups still read
    if (rows > 0 && (y == x || y == residual || y == hsum) &&
        (d.out != GE_NORM_PLAIN || (d.ldy != d.ld && rows > 1)))
        return GE_ERR_SHAPE;
    if (test_fail_launch()) return GE_ERR_HIP;
    if (rows == 0) return GE_OK;
    NormArgs a = {};
    a.x = x;
    a.res = residual;
    a.gamma = gamma;
    a.h = hsum;
    a.y = y;
    a.scales = scales;
    a.rstd = rstd;
    a.rows = (int32_t)rows;
    a.cols = (int32_t)d.cols;
    a.blocks = (int32_t)forward_blocks(h->fwd, rows);
    a.lds = (int32_t)GE_MX_SCALE_LD(d.cols);
    a.ld = d.ld;
    a.ldy = d.ldy;
    a.eps = d.eps;
    a.inv_cols = (float)(1.0 / (double)d.cols);
    return launch_norm_forward(d.type, d.out, h->fwd, a, stream) == 0 ? GE_OK : GE_ERR_HIP;
}

int ge_rms_norm_backward(ge_norm_handle h, int64_t rows, const void* dy, const void* hsum, const void* gamma,
                         const float* rstd, const void* dh, void* dx, void* dgamma, void* workspace,
                         size_t workspace_bytes, void* stream) {
    if (!h) return GE_ERR_NULL;
    const ge_norm_desc& d = h->d;
    if (rows < 0 || rows > d.rows) return GE_ERR_SHAPE;
    if (!gamma || (rows > 0 && (!dy || !hsum || !rstd || !dx))) return GE_ERR_NULL;
    if (!aligned(dy, 16) || !aligned(hsum, 16) || !aligned(gamma, 16) || !aligned(dh, 16) || !aligned(dx, 16) ||
        !aligned(dgamma, 16) || !aligned(workspace, 16) || !aligned(rstd, 4))
        return GE_ERR_ALIGN;
    if (dgamma && rows > 0 && (!workspace || workspace_bytes < partial_bytes(*h, rows))) return GE_ERR_WORKSPACE;
    if (test_fail_launch()) return GE_ERR_HIP;
    NormArgs a = {};
    a.dy = dy;
    a.x = hsum;
    a.gamma = gamma;
    a.rstd = const_cast<float*>(rstd);
    a.dh = dh;
    a.dx = dx;
    a.dgamma = dgamma;
    a.partial = dgamma ? (float*)workspace : nullptr;
    a.rows = (int32_t)rows;
    a.cols = (int32_t)d.cols;
    a.blocks = (int32_t)backward_blocks(rows);
    a.ld = d.ld;
    a.eps = d.eps;
    a.inv_cols = (float)(1.0 / (double)d.cols);
    if (rows > 0 && launch_norm_backward(d.type, h->bwd, a, stream) != 0) return GE_ERR_HIP;
    if (dgamma && launch_norm_dgamma(d.type, a, stream) != 0) return GE_ERR_HIP;
    return GE_OK;
}

int ge_rms_norm_describe(ge_norm_handle h, char* buf, size_t cap) {
    if (!h || !buf) return GE_ERR_NULL;
    if (cap == 0) return GE_OK;
    snprintf(buf, cap, "rows=%lld cols=%lld type=%d out=%d forward=%dx%d backward=%dx%d blocks=%lld",
             (long long)h->d.rows, (long long)h->d.cols, h->d.type, h->d.out, h->fwd.threads, h->fwd.chunks,
             h->bwd.threads, h->bwd.chunks, (long long)backward_blocks(h->d.rows));
    return GE_OK;
}

int ge_rms_norm_free(ge_norm_handle h) {
    delete h;
    return GE_OK;
}

}  // extern "C"
