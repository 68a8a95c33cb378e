"""The residual product's C ABI without a GPU: what plan and execute refuse
before any HIP call, which kernel a plan takes, and the backward plan's
rules.  Addresses here are numbers that are never read."""
import ctypes

import pytest

from activation_epilogue_02_amd import GE_OP_N, GE_OP_T, GemmEpilog
from activation_epilogue_02_amd import binding as B

P = 0x10000
KINDS = ["none", "bias", "relu_bias", "relu_aux_bias", "gelu_bias", "gelu_aux_bias", "tanh_bias"]


def handle(m=100, n=64, k=128, a="bf16", d=None, op_b=GE_OP_T, **kw):
    return GemmEpilog(m, n, k, a, d or ("bf16" if a in ("e4m3", "mxf8") else a), op_b, **kw)


def status(f, *a, **kw):
    try:
        f(*a, **kw)
    except B.GemmEpilogError as e:
        return e.status
    return B.GE_OK


def ex(g, m=None, A=P, Bm=P, bias=P, R=None, ldr=64, D=P, **kw):
    kw.setdefault("workspace", P)
    kw.setdefault("workspace_bytes", 1 << 30)
    return status(B.gemm_epilog_execute_residual, g.h, g.desc.m if m is None else m, A, Bm, bias, R, ldr, D, **kw)


def test_plan_kinds():
    for kind in KINDS:
        with handle() as g:
            assert status(g.plan_residual, kind) == B.GE_OK
            assert "residual=1" in g.describe()
    for kind in ("drelu", "dgelu", "drelu_bgrad", "dgelu_bgrad", 11, -1):
        with handle() as g:
            assert status(g.plan_residual, kind) == B.GE_ERR_EPILOG
    with handle() as g:
        assert status(g.plan_residual, "bias", 2) == B.GE_ERR_EPILOG
        assert status(B.gemm_epilog_plan_residual, None, "bias") == B.GE_ERR_NULL
    with handle(batch=2) as g:
        assert status(g.plan_residual) == B.GE_ERR_SHAPE
    with handle(d="e4m3") as g:
        assert status(g.plan_residual) == B.GE_ERR_DTYPE


@pytest.mark.parametrize("a,m,n,k,op_b,want", [
    ("bf16", 1, 4096, 4096, GE_OP_T, "path=skinny rows=16 cols=16 "),
    ("f16", 17, 8192, 512, GE_OP_T, "path=skinny rows=32 cols=32 "),
    ("e4m3", 64, 104, 512, GE_OP_T, "path=skinny rows=64 cols=16 "),
    ("mxf8", 33, 104, 512, GE_OP_T, "path=skinny rows=64 cols=16 "),
    ("bf16", 1, 4096, 4096, GE_OP_N, "tile_id=14 "),
    ("e4m3", 1, 4096, 4096, GE_OP_N, "tile_id=17 "),
    ("mxf8", 1, 4096, 4096, GE_OP_N, "tile_id=18 "),
    ("f32", 1, 4096, 4096, GE_OP_T, "tile_id=1 "),
    ("f32", 4096, 4096, 64, GE_OP_T, "tile_id=2 "),
    ("f16", 8192, 4096, 64, GE_OP_T, "tile_id=6 "),
    ("f16", 2048, 4096, 64, GE_OP_T, "tile_id=8 "),
    ("f16", 65, 128, 8192, GE_OP_T, "tile_id=14 "),
    ("e4m3", 8192, 4096, 64, GE_OP_T, "tile_id=16 "),
    ("e4m3", 4096, 4096, 64, GE_OP_T, "tile_id=15 "),
    ("e4m3", 1024, 4096, 64, GE_OP_N, "tile_id=8 "),
    ("e4m3", 65, 128, 8192, GE_OP_T, "tile_id=17 "),
    ("mxf8", 2048, 4096, 4096, GE_OP_T, "tile_id=19 "),
])
def test_plan_choice(a, m, n, k, op_b, want):
    with handle(m, n, k, a, op_b=op_b) as g:
        g.plan_residual("bias")
        assert want in g.describe() + " ", g.describe()


def test_split_needs_its_workspace():
    with handle(100, 64, 16384) as g:
        g.plan_residual("bias")
        assert g.ws_bytes > 0
        assert ex(g, workspace=None, workspace_bytes=0) == B.GE_ERR_WORKSPACE
        assert ex(g, workspace_bytes=g.ws_bytes - 1) == B.GE_ERR_WORKSPACE


def test_states(monkeypatch):
    monkeypatch.setenv("GE_TEST_FAIL_LAUNCH", "1")
    with handle() as g:
        assert ex(g) == B.GE_ERR_STATE
        g.plan("bias", "col")
        assert ex(g) == B.GE_ERR_STATE
        assert status(g.plan_backward) == B.GE_ERR_STATE
        assert status(B.gemm_epilog_execute, g.h, P, P, P, P) == B.GE_ERR_HIP
        g.plan_residual("bias")
        assert ex(g) == B.GE_ERR_HIP    # past every check
        assert status(B.gemm_epilog_execute, g.h, P, P, P, P) == B.GE_ERR_STATE
        assert status(B.gemm_epilog_execute_m, g.h, 1, P, P, P, P) == B.GE_ERR_STATE
        assert status(B.gemm_epilog_autotune, g.h, P, P, P, P) == B.GE_ERR_STATE
        assert status(B.gemm_epilog_backward_workspace_size, g.h) == B.GE_ERR_STATE
        assert status(B.gemm_epilog_backward, g.h, P, P, P, None, P, P) == B.GE_ERR_STATE
        g.plan_backward()
        assert status(B.gemm_epilog_backward, g.h, P, P, P, None, P, P, workspace=P, workspace_bytes=1 << 30) == B.GE_ERR_HIP
        g.plan("bias", "col")           # a plan of the other kind ends both
        assert ex(g) == B.GE_ERR_STATE
        assert status(B.gemm_epilog_backward, g.h, P, P, P, None, P, P, workspace=P, workspace_bytes=1 << 30) == B.GE_ERR_STATE


@pytest.mark.parametrize("kw,want", [
    (dict(), B.GE_ERR_HIP),
    (dict(m=0), B.GE_ERR_HIP),
    (dict(m=-1), B.GE_ERR_SHAPE),
    (dict(m=101), B.GE_ERR_SHAPE),
    (dict(A=None), B.GE_ERR_NULL),
    (dict(Bm=None), B.GE_ERR_NULL),
    (dict(D=None), B.GE_ERR_NULL),
    (dict(bias=None), B.GE_ERR_NULL),
    (dict(aux=P), B.GE_ERR_EPILOG),
    (dict(R=P), B.GE_ERR_HIP),
    (dict(R=P, ldr=63), B.GE_ERR_SHAPE),
    (dict(R=P, ldr=68), B.GE_ERR_ALIGN),
    (dict(R=P + 8), B.GE_ERR_ALIGN),
    (dict(A=P + 8), B.GE_ERR_ALIGN),
    (dict(Bm=P + 8), B.GE_ERR_ALIGN),
    (dict(D=P + 8), B.GE_ERR_ALIGN),
    (dict(bias=P + 8), B.GE_ERR_ALIGN),
    (dict(row_scale=P + 2), B.GE_ERR_ALIGN),
    (dict(row_scale=P + 4), B.GE_ERR_HIP),
    (dict(col_scale=P + 4), B.GE_ERR_ALIGN),
    (dict(scale_a=P + 2), B.GE_ERR_ALIGN),
    (dict(a_scales=P), B.GE_ERR_DTYPE),
], ids=str)
def test_execute_refusals(kw, want, monkeypatch):
    monkeypatch.setenv("GE_TEST_FAIL_LAUNCH", "1")
    with handle() as g:
        g.plan_residual("bias")
        assert ex(g, **kw) == want


def test_execute_refusals_mx_and_aux(monkeypatch):
    monkeypatch.setenv("GE_TEST_FAIL_LAUNCH", "1")
    with handle(a="mxf8") as g:
        g.plan_residual("gelu_aux_bias")
        assert ex(g, aux=P) == B.GE_ERR_NULL
        assert ex(g, aux=P, a_scales=P, b_scales=P) == B.GE_ERR_HIP
        assert ex(g, aux=P, a_scales=P + 8, b_scales=P) == B.GE_ERR_ALIGN
        assert ex(g, a_scales=P, b_scales=P) == B.GE_ERR_EPILOG


def test_backward_plan():
    for a, d, kind, want in [("bf16", "bf16", "none", B.GE_OK), ("f16", "f16", "gelu_aux_bias", B.GE_OK),
                             ("f32", "f32", "relu_aux_bias", B.GE_OK), ("bf16", "f32", "bias", B.GE_ERR_DTYPE),
                             ("e4m3", "bf16", "bias", B.GE_ERR_DTYPE), ("mxf8", "f16", "bias", B.GE_ERR_DTYPE),
                             ("bf16", "bf16", "relu_bias", B.GE_ERR_EPILOG), ("bf16", "bf16", "gelu_bias", B.GE_ERR_EPILOG),
                             ("bf16", "bf16", "tanh_bias", B.GE_ERR_EPILOG)]:
        for op_b in (GE_OP_N, GE_OP_T):
            with handle(a=a, d=d, op_b=op_b) as g:
                g.plan_residual(kind)
                assert status(g.plan_backward) == want, (a, d, kind)


@pytest.mark.parametrize("kind,kw,want", [
    ("bias", dict(), B.GE_ERR_HIP),
    ("bias", dict(dD=None), B.GE_ERR_NULL),
    ("bias", dict(A=None), B.GE_ERR_NULL),
    ("bias", dict(A=None, dB=None), B.GE_ERR_HIP),
    ("bias", dict(Bm=None), B.GE_ERR_NULL),
    ("bias", dict(Bm=None, dA=None), B.GE_ERR_HIP),
    ("bias", dict(aux=P), B.GE_ERR_EPILOG),
    ("gelu_aux_bias", dict(), B.GE_ERR_EPILOG),
    ("gelu_aux_bias", dict(aux=P), B.GE_ERR_HIP),
    ("none", dict(), B.GE_ERR_EPILOG),
    ("none", dict(dbias=None), B.GE_ERR_HIP),
    ("bias", dict(dA=P + 8), B.GE_ERR_ALIGN),
    ("bias", dict(dB=P + 8), B.GE_ERR_ALIGN),
    ("bias", dict(dbias=P + 8), B.GE_ERR_ALIGN),
    ("bias", dict(workspace=None, workspace_bytes=0), B.GE_ERR_WORKSPACE),
], ids=str)
def test_backward_refusals(kind, kw, want, monkeypatch):
    monkeypatch.setenv("GE_TEST_FAIL_LAUNCH", "1")
    a = dict(dD=P, A=P, Bm=P, aux=None, dA=P, dB=P, dbias=P, workspace=P, workspace_bytes=1 << 30) | kw
    with handle() as g:
        g.plan_residual(kind)
        g.plan_backward()
        assert status(B.gemm_epilog_backward, g.h, a["dD"], a["A"], a["Bm"], a["aux"], a["dA"], a["dB"], a["dbias"],
                      a["workspace"], a["workspace_bytes"]) == want
        if want == B.GE_ERR_WORKSPACE:
            assert status(B.gemm_epilog_backward, g.h, P, P, P, None, P, P, P, P, g.backward_ws_bytes - 1) == want


def test_null_handles():
    L = B.lib()
    assert L.gemm_epilog_execute_residual(None, 0, *[None] * 6, 0, *[None] * 7, 0, None) == B.GE_ERR_NULL
    assert L.gemm_epilog_plan_backward(None) == B.GE_ERR_NULL
    assert L.gemm_epilog_backward_workspace_size(None, ctypes.byref(ctypes.c_size_t())) == B.GE_ERR_NULL
    assert L.gemm_epilog_backward(None, *[None] * 8, 0, None) == B.GE_ERR_NULL


def test_in_place_needs_the_same_rows(monkeypatch):
    """R = D with another row stride: rows of D would overwrite rows of R that are still to be read."""
    monkeypatch.setenv("GE_TEST_FAIL_LAUNCH", "1")
    for m in (100, 20):                 # tiles, few rows
        with handle(m, ldd=64) as g:
            g.plan_residual("bias")
            assert ex(g, R=P, ldr=64) == B.GE_ERR_HIP
            assert ex(g, R=P, ldr=72) == B.GE_ERR_SHAPE
            assert ex(g, R=P, ldr=72, m=1) == B.GE_ERR_HIP      # one row: nothing else to overwrite
            assert ex(g, R=P + (1 << 24), ldr=72) == B.GE_ERR_HIP


@pytest.mark.parametrize("a,m,n,lda,want", [
    # rows of 16, 32 and 64 MiB and more: 256, 128 and 64 of them are 4 GiB
    ("bf16", 8192, 4096, 1 << 23, "tile_id=6 "),
    ("bf16", 8192, 4096, 1 << 24, "tile_id=8 "),
    ("bf16", 8192, 4096, 1 << 25, "tile_id=14 "),
    ("bf16", 8192, 4096, 1 << 26, None),
    ("f16", 100, 64, 1 << 25, "tile_id=14 "),
    ("e4m3", 8192, 4096, 1 << 24, "tile_id=16 "),
    ("e4m3", 8192, 4096, 1 << 25, "tile_id=8 "),
    ("e4m3", 8192, 4096, 1 << 26, "tile_id=17 "),
    ("e4m3", 8192, 4096, 1 << 27, None),
    ("mxf8", 8192, 4096, 1 << 25, "tile_id=19 "),
    ("mxf8", 8192, 4096, 1 << 26, None),
    ("f32", 8192, 4096, 1 << 30, "tile_id=2 "),
])
def test_rows_far_apart(a, m, n, lda, want):
    """A tile that cannot address its rows leaves the choice to a smaller one."""
    with handle(m, n, 64, a, lda=lda) as g:
        assert status(g.plan_residual, "bias") == (B.GE_ERR_SHAPE if want is None else B.GE_OK)
        if want is not None:
            assert want in g.describe() + " ", g.describe()
