"""The residual product D = R + act(s * row_scale * col_scale * A*B + bias) and
its backward pass on the GPU against plain 64-bit forms.

Tolerances.  A result in type t is the fp32 value rounded once: eps(t)/2
relative.  An fp32 sum of k products is off by at most k 2^-24 times the sum of
their magnitudes S (each product of the input types is exact in fp32 or, for
fp32 inputs, off by 2^-24), the scales and the bias by 4 2^-24 more.  An
activation passes an error of its argument on at most 1.13 times (GELU's
largest slope), and GELU and its slope are evaluated with the hardware's
exponential and reciprocal, each good to 2^-22 relative, at arguments up to a
few tens: 2^-18 of the value.  Rounding dP to 16 bits adds eps/2 of each term.

The matrix instruction for 8-bit operands does not add its products in fp32: it
takes K in groups of eight, aligns each group's products to its largest and
drops what lies below 2^-13 of that one's power of two (measured: beside
2^16, 8 counts and 4 does not; two products in different groups do not
affect each other).  Seven products of a group can lose that much, so an 8-bit
sum is off by at most 7 2^-13 S more.  test_small_whole_numbers checks the
same kernels where nothing is dropped, bit for bit."""
import pytest
import torch

from activation_epilogue_02_amd import GE_OP_N, GE_OP_T, GemmEpilog, mx_scale_ld
from activation_epilogue_02_amd import binding as B

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn,
      "mxf8": torch.float8_e4m3fn}
U = 2.0 ** -24
KINDS = ["none", "bias", "relu_bias", "relu_aux_bias", "gelu_bias", "gelu_aux_bias", "tanh_bias"]
C0 = 0.7978845608028654


def gen(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return lambda *s: torch.randn(*s, generator=g, device="cuda")


def laid(v, dt, pad=1):
    """v in the type, rows padded to 16 bytes and `pad` chunks more, the padding NaN."""
    e = 16 // torch.empty(0, dtype=DT[dt]).element_size()
    ld = -(-v.shape[1] // e) * e + pad * e
    m = torch.full((v.shape[0], ld), float("nan"), device="cuda").to(DT[dt])
    m[:, :v.shape[1]] = v.to(DT[dt])
    return m[:, :v.shape[1]]


def untouched(m):
    rows, cols, ld = m.shape[0], m.shape[1], m.stride(0)
    return rows == 0 or m.as_strided((rows, ld - cols), (ld, 1), m.storage_offset() + cols).float().isnan().all()


def block_scales(rows, k, randn):
    s = torch.full((rows, mx_scale_ld(k)), 0xFF, dtype=torch.uint8, device="cuda")   # NaN past the last block
    nb = -(-k // 32)
    s[:, :nb] = (127 + 3 * randn(rows, nb)).round().clamp(110, 140).to(torch.uint8)
    return s, torch.exp2(s[:, :nb].double() - 127).repeat_interleave(32, 1)[:, :k]


def wrong(got, want, tol, t):
    """Where got (in type t) is not want within tol; beyond the type's range rounding gives an infinity."""
    top = torch.finfo(t).max
    over = (want.abs() + tol > top) & (got.double() == torch.copysign(torch.full_like(want, float("inf")), want))
    return ~(((got.double() - want).abs() <= tol) | over)


def gelu(x):
    return x / (1 + torch.exp(-2 * C0 * (x + 0.044715 * x ** 3)))


def gelu_slope(x):
    s = 1 / (1 + torch.exp(-2 * C0 * (x + 0.044715 * x ** 3)))
    return s + x * s * (1 - s) * 2 * C0 * (1 + 3 * 0.044715 * x * x)


ACT = {"relu_bias": lambda x: x.clamp(min=0), "relu_aux_bias": lambda x: x.clamp(min=0), "gelu_bias": gelu,
       "gelu_aux_bias": gelu, "tanh_bias": torch.tanh}


def bits(words, n):
    b = (words[:, :, None] >> torch.arange(32, device="cuda", dtype=torch.int32)) & 1
    return b.view(words.shape[0], -1)


def run(m, n, k, a, d, op_b, kind, axis="col", residual=True, scales=None, pad=1, seed=0, rows=None, inplace=False):
    print(f"case {m}x{n}x{k} {a}->{d} op_b={op_b} {kind} {axis} rows={rows}", flush=True)
    randn = gen(1000 * m + 10 * n + k + seed)
    scales = a == "e4m3" if scales is None else scales
    A = laid(randn(m, k), a, pad)
    W = randn(n, k) * max(k, 1) ** -0.5 * (8 if a in ("e4m3", "mxf8") else 1)
    Bm = laid(W if op_b == GE_OP_T else W.t(), a, pad)
    a64, b64 = A.double(), (Bm.t() if op_b == GE_OP_T else Bm).double()
    sa = sb = rs = cs = None
    if a == "mxf8":
        sa, fa = block_scales(m, k, randn)
        sb, fb = block_scales(n, k, randn)
        a64, b64 = a64 * fa, b64 * fb.t()
    P, S = a64 @ b64, a64.abs() @ b64.abs()
    if scales:
        rs, cs = torch.exp(0.5 * randn(m)), torch.exp(0.5 * randn(n)) / 8
        f = rs.double()[:, None] * cs.double()
        P, S = P * f, S * f
    group = 7 * 2.0 ** -13 * S if a in ("e4m3", "mxf8") else 0.0
    bias = None
    if kind != "none":
        bias = randn(n if axis == "col" else m).to(DT[d])
        bb = bias.double()[None, :] if axis == "col" else bias.double()[:, None]
        P, S = P + bb, S + bb.abs()
    R = laid(randn(m, n), d, pad + 1) if residual else None
    want = ACT.get(kind, lambda x: x)(P)
    tol = 1.13 * ((k + 8) * U * S + group) + (2.0 ** -18 if "gelu" in kind or "tanh" in kind else 0) * P.abs()
    ptol = (k + 8) * U * S + group
    if residual:
        want = want + R.double()
        tol = tol + U * R.double().abs()
    f = torch.finfo(DT[d])
    tol = tol + want.abs() * f.eps / 2 * (1 + 2.0 ** -6) + f.tiny * f.eps
    D = R if inplace else laid(torch.zeros(m, n, device="cuda"), d, pad)
    before = D.clone()
    with GemmEpilog(m, n, k, a, d, op_b, A.stride(0), Bm.stride(0), D.stride(0)) as g:
        g.plan_residual(kind, axis)
        aux = None
        if kind == "relu_aux_bias":
            aux = torch.full((m, g.aux_ld_bits // 32), -1, dtype=torch.int32, device="cuda")
        elif kind == "gelu_aux_bias":
            aux = torch.full((m, g.aux_ld_bits // f.bits), float("nan"), dtype=DT[d], device="cuda")
        ws = torch.full((g.ws_bytes,), 0xA5, dtype=torch.uint8, device="cuda") if g.ws_bytes else None
        mm = m if rows is None else rows
        g.execute_residual(A, Bm, bias, R, D, aux=aux, row_scale=rs, col_scale=cs, a_scales=sa, b_scales=sb,
                           workspace=ws, m=rows)
        torch.cuda.synchronize()
        assert untouched(D)
        bad = wrong(D[:mm], want[:mm], tol[:mm], D.dtype)
        assert not bad.any(), (g.describe(), int(bad.sum()), D[:mm][bad][:4], want[:mm][bad][:4], bad.nonzero()[:4])
        if rows is not None:
            assert torch.equal(D[rows:], before[rows:])
        if kind == "relu_aux_bias":
            b = bits(aux[:mm], n)
            sure = P[:mm].abs() > ptol[:mm]
            assert (b[:, :n][sure] == (P[:mm] > 0)[sure].int()).all() and (b[:, n:] == 0).all()
            assert (aux[mm:] == -1).all()
        if kind == "gelu_aux_bias":
            bad = wrong(aux[:mm, :n], P[:mm], ptol[:mm] + P[:mm].abs() * f.eps / 2 * (1 + 2.0 ** -6) + f.tiny * f.eps, D.dtype)
            assert not bad.any() and aux[:, n:].isnan().all() and aux[mm:].isnan().all()
        return g.describe(), D


COMBOS = [("f16", "f16"), ("f16", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("e4m3", "bf16"), ("e4m3", "f16"),
          ("e4m3", "f32"), ("mxf8", "bf16"), ("mxf8", "f16"), ("mxf8", "f32")]
IDS = [f"{a}-{d}" for a, d in COMBOS]


@pytest.mark.parametrize("a,d", COMBOS, ids=IDS)
@pytest.mark.parametrize("m", [1, 3, 16, 17, 32, 33, 64])
@pytest.mark.parametrize("n,k", [(1, 1), (16, 64), (100, 200), (33, 1032), (257, 128), (48, 4100), (130, 2047)])
def test_few_rows(a, d, m, n, k):
    i = m + n + k
    desc, _ = run(m, n, k, a, d, GE_OP_T, KINDS[i % 7], "row" if i % 5 == 0 else "col", residual=i % 3 != 0, scales=i % 2 == 0)
    assert "path=skinny" in desc


@pytest.mark.parametrize("a,d", COMBOS, ids=IDS)
@pytest.mark.parametrize("m", [5, 20, 64])
def test_few_rows_wide(a, d, m):
    """Two column groups per workgroup."""
    desc, _ = run(m, 8200, 264, a, d, GE_OP_T, "relu_aux_bias")
    assert "cols=32 " in desc


@pytest.mark.parametrize("a,d", COMBOS + [("f32", "f32")], ids=IDS + ["f32-f32"])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("op_b", [GE_OP_N, GE_OP_T], ids=["kn", "nk"])
def test_tiles_ragged(a, d, kind, op_b):
    run(150, 200, 136, a, d, op_b, kind, "col")
    run(70, 77, 333, a, d, op_b, kind, "row", scales=True, pad=0)


@pytest.mark.parametrize("a,d", COMBOS + [("f32", "f32")], ids=IDS + ["f32-f32"])
@pytest.mark.parametrize("m,n,k", [(1, 1, 1), (1, 64, 4096), (7, 130, 8200), (65, 129, 5000), (200, 300, 4229)])
def test_long_k(a, d, m, n, k):
    """Few tiles and a long K: the split-K tiles (and fp32's, which does not split)."""
    i = m + n + k
    desc, one = run(m, n, k, a, d, GE_OP_N, KINDS[i % 7])
    assert a == "f32" or k < 4096 or "split_k=1 " not in desc
    assert torch.equal(one, run(m, n, k, a, d, GE_OP_N, KINDS[i % 7])[1])   # equal bits


@pytest.mark.parametrize("a,d,m,n,k,tile", [
    ("bf16", "bf16", 4100, 8200, 200, 6), ("f16", "f16", 4100, 8200, 72, 6), ("f16", "f32", 2050, 2100, 264, 8),
    ("bf16", "bf16", 2050, 2100, 264, 8), ("e4m3", "bf16", 4100, 8200, 400, 16), ("e4m3", "f16", 4100, 4100, 1040, 15),
    ("e4m3", "f32", 1050, 2100, 272, 8), ("mxf8", "bf16", 2050, 2100, 400, 19), ("mxf8", "f16", 700, 2100, 1100, 18),
    ("f32", "f32", 2050, 2100, 136, 2)])
@pytest.mark.parametrize("op_b", [GE_OP_N, GE_OP_T], ids=["kn", "nk"])
def test_large_tiles(a, d, m, n, k, tile, op_b):
    for kind in ("bias", "relu_aux_bias", "gelu_aux_bias", "tanh_bias"):
        desc, _ = run(m, n, k, a, d, op_b, kind)
        assert f"tile_id={tile} " in desc


@pytest.mark.parametrize("a", ["e4m3", "mxf8", "bf16", "f16"])
@pytest.mark.parametrize("op_b", [GE_OP_N, GE_OP_T], ids=["kn", "nk"])
@pytest.mark.parametrize("m,n,k", [(1, 33, 128), (16, 40, 1000), (20, 64, 2047), (64, 8200, 333), (100, 200, 500),
                                   (70, 130, 9000), (2050, 2100, 272), (4100, 4100, 160), (4100, 8200, 400)])
def test_small_whole_numbers(a, op_b, m, n, k):
    """Whole operands from -4 to 4 and power-of-two scales: every product is
    a whole multiple of 2^-6 or more below 2^10, every sum below 2^24 of
    those, and nothing is rounded or dropped: D in fp32 is exact."""
    print(f"case {m}x{n}x{k} {a} op_b={op_b}", flush=True)
    g0 = torch.Generator(device="cuda").manual_seed(m + n + k)
    ints = lambda lo, hi, *s: torch.randint(lo, hi + 1, s, generator=g0, device="cuda").float()
    A, W = laid(ints(-4, 4, m, k), a), ints(-4, 4, n, k)
    Bm = laid(W if op_b == GE_OP_T else W.t(), a)
    a64, b64 = A.double(), (Bm.t() if op_b == GE_OP_T else Bm).double()
    sa = sb = None
    if a == "mxf8":
        nb = -(-k // 32)
        sa, sb = (torch.full((r, mx_scale_ld(k)), 0xFF, dtype=torch.uint8, device="cuda") for r in (m, n))
        sa[:, :nb], sb[:, :nb] = 127 + ints(-3, 3, m, nb), 127 + ints(-3, 3, n, nb)
        a64 = a64 * torch.exp2(sa[:, :nb].double() - 127).repeat_interleave(32, 1)[:, :k]
        b64 = b64 * torch.exp2(sb[:, :nb].double() - 127).repeat_interleave(32, 1)[:, :k].t()
    rs, cs = torch.exp2(ints(-2, 2, m)), torch.exp2(ints(-2, 2, n))
    bias, R = ints(-8, 8, n), laid(ints(-100, 100, m, n), "f32")
    want = (a64 @ b64) * rs.double()[:, None] * cs.double() + bias.double() + R.double()
    assert k * 16 * 64 < 2 ** 24 or a != "mxf8"
    D = laid(torch.zeros(m, n, device="cuda"), "f32")
    with GemmEpilog(m, n, k, a, "f32", op_b, A.stride(0), Bm.stride(0), D.stride(0)) as g:
        g.plan_residual("bias")
        ws = torch.empty(max(1, g.ws_bytes), dtype=torch.uint8, device="cuda")
        g.execute_residual(A, Bm, bias, R, D, row_scale=rs, col_scale=cs, a_scales=sa, b_scales=sb, workspace=ws)
        assert torch.equal(D.double(), want), g.describe()


@pytest.mark.parametrize("m", [9, 90])
@pytest.mark.parametrize("a,d", [("bf16", "bf16"), ("e4m3", "bf16"), ("mxf8", "f16")])
def test_in_place_and_fewer_rows(a, d, m):
    run(m, 200, 136, a, d, GE_OP_T, "gelu_bias", inplace=True, pad=0)
    for kind in ("relu_aux_bias", "gelu_aux_bias"):
        run(m, 200, 5000, a, d, GE_OP_T, kind, rows=m - 7)
    run(m, 200, 5000, a, d, GE_OP_T, "bias", rows=m - 7, inplace=True)
    run(m, 200, 64, a, d, GE_OP_T, "bias", rows=0)


@pytest.mark.parametrize("mnk", [(0, 70, 40), (50, 0, 40), (50, 70, 0), (5, 70, 0)])
@pytest.mark.parametrize("a,d", [("bf16", "bf16"), ("e4m3", "f16"), ("mxf8", "bf16"), ("f32", "f32")])
def test_empty(mnk, a, d):
    """No rows or columns: nothing happens.  k = 0: D = R + act(bias)."""
    run(*mnk, a, d, GE_OP_T, "gelu_bias")


@pytest.mark.parametrize("a", ["bf16", "e4m3", "mxf8"])
@pytest.mark.parametrize("m", [8, 100])
def test_bad_values_stay_in_their_rows(a, m):
    n, k = 96, 160
    randn = gen(4)
    A, W = laid(randn(m, k), a), laid(randn(n, k), a)
    clean = laid(A.float(), a)
    A[2, 5] = float("nan")
    sa = sb = None
    if a == "mxf8":
        sa, sb = (torch.full((r, mx_scale_ld(k)), 127, dtype=torch.uint8, device="cuda") for r in (m, n))
    out = []
    for X in (A, clean):
        D = laid(torch.zeros(m, n, device="cuda"), "bf16", 0)
        with GemmEpilog(m, n, k, a, "bf16", GE_OP_T, X.stride(0), W.stride(0), D.stride(0)) as g:
            g.plan_residual("none")
            g.execute_residual(X, W, None, None, D, a_scales=sa, b_scales=sb,
                               workspace=torch.empty(max(1, g.ws_bytes), dtype=torch.uint8, device="cuda"))
        out.append(D)
    assert out[0][2].isnan().all()
    keep = [i for i in range(m) if i != 2]
    assert torch.equal(out[0][keep], out[1][keep])


# ---- backward ---------------------------------------------------------------------
def backward_case(m, n, k, t, op_b, kind, axis="col", pad=1, seed=0):
    print(f"case {m}x{n}x{k} {t} op_b={op_b} {kind} {axis}", flush=True)
    randn = gen(100 * m + n + k + seed)
    A = laid(randn(m, k), t, pad)
    W = randn(n, k) * max(k, 1) ** -0.5
    Bm = laid(W if op_b == GE_OP_T else W.t(), t, pad + 1)
    dD = laid(randn(m, n), t, pad)
    f = torch.finfo(DT[t])
    aux, slope = None, None
    ldn = -(-n // 128) * 128
    if kind == "relu_aux_bias":
        on = torch.nn.functional.pad(randn(m, n) > 0, (0, ldn - n))
        w = (on.view(m, -1, 32).long() << torch.arange(32, device="cuda")).sum(2)
        aux = torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32)
        slope = on[:, :n].double()
        # a masked entry is zero whatever the gradient holds there
        if m > 1 and n > 1:
            i = int((slope[1] == 0).nonzero()[0]) if (slope[1] == 0).any() else None
            if i is not None:
                dD[1, i] = float("inf")
    elif kind == "gelu_aux_bias":
        aux = torch.full((m, ldn), float("nan"), dtype=DT[t], device="cuda")
        aux[:, :n] = randn(m, n)
        slope = gelu_slope(aux[:, :n].double())
    dP = dD.double() if slope is None else torch.where(slope == 0, torch.zeros_like(slope), dD.double() * slope)
    b64 = (Bm if op_b == GE_OP_T else Bm.t()).double()      # n x k
    dA, SA = dP @ b64, dP.abs() @ b64.abs()
    dB, SB = dP.t() @ A.double(), dP.abs().t() @ A.double().abs()
    if op_b == GE_OP_N:
        dB, SB = dB.t(), SB.t()
    db, Sb = (dP.sum(0), dP.abs().sum(0)) if axis == "col" else (dP.sum(1), dP.abs().sum(1))
    gel = 2.0 ** -18 if kind == "gelu_aux_bias" else 0.0
    step = f.eps / 2 * (1 + 2.0 ** -6) if kind == "gelu_aux_bias" else 0.0
    gA, gB = laid(torch.zeros(m, k, device="cuda"), t, pad), laid(torch.zeros(Bm.shape, device="cuda"), t, pad + 1)
    # (the slope passes through zero: its error there is against 1, not against itself)
    gelA = gel * ((dD.double().abs() @ b64.abs()) if gel else 0)
    gelB = gel * ((dD.double().abs().t() @ A.double().abs()) if gel else 0)
    if gel and op_b == GE_OP_N:
        gelB = gelB.t()
    gelb = gel * dD.double().abs().sum(0 if axis == "col" else 1) if gel else 0.0
    gb = torch.full((len(db) + 8,), 5.0, dtype=DT[t], device="cuda") if kind != "none" else None
    with GemmEpilog(m, n, k, t, t, op_b, A.stride(0), Bm.stride(0), dD.stride(0)) as g:
        g.plan_residual(kind, axis)
        g.plan_backward()
        ws = torch.full((max(1, g.backward_ws_bytes),), 0xA5, dtype=torch.uint8, device="cuda")
        g.backward(dD, A, Bm, gA, gB, dbias=gb, aux=aux, workspace=ws)
        torch.cuda.synchronize()

        def near(got, want, tol):
            tol = tol + want.abs() * f.eps / 2 * (1 + 2.0 ** -6) + f.tiny * f.eps
            bad = ~((got.double() - want).abs() <= tol)
            assert not bad.any(), (int(bad.sum()), got[bad][:4], want[bad][:4], bad.nonzero()[:4])

        near(gA, dA, SA * (step + (n + 8) * U) + gelA)
        near(gB, dB, SB * (step + (m + 8) * U) + gelB)
        assert untouched(gA) and untouched(gB)
        if gb is not None:
            near(gb[:len(db)], db, Sb * ((m if axis == "col" else n) + 8) * U + gelb)
            assert (gb[len(db):] == 5).all()
        # each output alone, and again: equal bits
        a2, b2 = gA.clone(), gB.clone()
        s2 = None if gb is None else gb.clone()
        gA.zero_(), gB.zero_()
        g.backward(dD, A, Bm, gA, None, aux=aux, workspace=ws)
        g.backward(dD, A, Bm, None, gB, aux=aux, workspace=ws)
        assert torch.equal(gA, a2) and torch.equal(gB, b2)
        if gb is not None:
            gb.fill_(5)
            g.backward(dD, A, Bm, None, None, dbias=gb, aux=aux, workspace=ws)
            assert torch.equal(gb, s2)


@pytest.mark.parametrize("t", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("kind", ["none", "bias", "relu_aux_bias", "gelu_aux_bias"])
@pytest.mark.parametrize("op_b", [GE_OP_N, GE_OP_T], ids=["kn", "nk"])
def test_backward(t, kind, op_b):
    backward_case(150, 200, 136, t, op_b, kind)
    backward_case(65, 77, 333, t, op_b, kind, "row", pad=0)
    backward_case(1, 1, 1, t, op_b, kind)
    backward_case(3, 130, 70, t, op_b, kind)
    backward_case(1000, 520, 72, t, op_b, kind)


@pytest.mark.parametrize("t", ["f16", "bf16"])
@pytest.mark.parametrize("m,n,k", [(9000, 72, 40), (17, 8200, 72), (70, 100, 8200), (2100, 2050, 2080), (4100, 300, 8210)])
@pytest.mark.parametrize("op_b", [GE_OP_N, GE_OP_T], ids=["kn", "nk"])
def test_backward_large(t, m, n, k, op_b):
    backward_case(m, n, k, t, op_b, "gelu_aux_bias" if m % 2 else "bias")


@pytest.mark.parametrize("mnk", [(0, 70, 40), (50, 0, 40), (50, 70, 0)])
@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("op_b", [GE_OP_N, GE_OP_T], ids=["kn", "nk"])
def test_backward_empty(mnk, t, op_b):
    """Sums over nothing are zero."""
    for axis in ("col", "row"):
        backward_case(*mnk, t, op_b, "gelu_aux_bias", axis)


@pytest.mark.parametrize("op_b", [GE_OP_N, GE_OP_T], ids=["kn", "nk"])
def test_backward_against_differences(op_b):
    """fp32 gradients of GELU(A B + bias) + R against central differences of the 64-bit form."""
    m, n, k, h = 4, 5, 6, 1e-5
    randn = gen(3)
    A, W, bias, dD = randn(m, k), randn(n, k), randn(n), randn(m, n)
    x = [A.double(), W.double(), bias.double()]
    pre = x[0] @ x[1].t() + x[2]

    def loss(v):
        return (dD.double() * gelu(v[0] @ v[1].t() + v[2])).sum()

    want = []
    for i in range(3):
        d = torch.empty_like(x[i])
        for j in range(x[i].numel()):
            e = torch.zeros_like(x[i])
            e.view(-1)[j] = h
            up, dn = ([*x[:i], x[i] + s * e, *x[i + 1:]] for s in (1, -1))
            d.view(-1)[j] = (loss(up) - loss(dn)) / (2 * h)
        want.append(d)
    A_, Bm, dD_ = laid(A, "f32", 0), laid(W if op_b == GE_OP_T else W.t(), "f32", 0), laid(dD, "f32", 0)
    aux = torch.zeros(m, 128, device="cuda")
    aux[:, :n] = pre
    gA, gB, gb = laid(torch.zeros(m, k, device="cuda"), "f32", 0), laid(torch.zeros(Bm.shape, device="cuda"), "f32", 0), torch.empty(n, device="cuda")
    with GemmEpilog(m, n, k, "f32", "f32", op_b, A_.stride(0), Bm.stride(0), dD_.stride(0)) as g:
        g.plan_residual("gelu_aux_bias")
        g.plan_backward()
        g.backward(dD_, A_, Bm, gA, gB, dbias=gb, aux=aux,
                   workspace=torch.empty(g.backward_ws_bytes, dtype=torch.uint8, device="cuda"))
    got = [gA.double(), (gB if op_b == GE_OP_T else gB.t()).double(), gb.double()]
    # the pre-activation is stored in fp32 (slope of the slope: at most 1), the slope good to 2^-18
    big = dD.double().abs()
    size = [big @ x[1].abs(), big.t() @ x[0].abs(), big.sum(0)]
    for a, b, s in zip(got, want, size):
        assert ((a - b).abs() <= s * (2.0 ** -17) + 1e-7).all()


def test_streams_and_graph():
    """Forward and backward on a side stream and captured; each replay gives the eager bits."""
    m, n, k = 70, 128, 8192
    randn = gen(9)
    A, W, R = laid(randn(m, k), "bf16", 0), laid(randn(n, k), "bf16", 0), laid(randn(m, n), "bf16", 0)
    mk = lambda r, c: laid(torch.zeros(r, c, device="cuda"), "bf16", 0)
    D, gA, gB = mk(m, n), mk(m, k), mk(n, k)
    bias, gb = (torch.ones(n, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    g = GemmEpilog(m, n, k, "bf16", "bf16", GE_OP_T, A.stride(0), W.stride(0), D.stride(0))
    g.plan_residual("gelu_aux_bias")
    g.plan_backward()
    assert "split_k=1 " not in g.describe()
    aux = torch.empty(m, g.aux_ld_bits // 16, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(max(g.ws_bytes, g.backward_ws_bytes), dtype=torch.uint8, device="cuda")

    def step():
        g.execute_residual(A, W, bias, R, D, aux=aux, workspace=ws)
        g.backward(D, A, W, gA, gB, dbias=gb, aux=aux, workspace=ws)

    step()
    outs = (D, gA, gB, gb)
    want = [t.clone() for t in outs]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=s):
            step()
    torch.cuda.current_stream().wait_stream(s)
    for i in range(3):
        for t in outs:
            t.fill_(i)
        ws.fill_(i)
        gr.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want)), i
        step()   # eager work between the replays
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want)), i
    g.free()


@pytest.mark.parametrize("a,d", COMBOS, ids=IDS)
@pytest.mark.parametrize("planned", [64, 70, 300])
def test_few_rows_of_a_larger_plan(a, d, planned):
    """A call's kernel follows its own rows: the bits are those of a handle planned for them."""
    n, k = 200, 4100
    randn = gen(21)
    A, W, R = laid(randn(planned, k), a), laid(randn(n, k), a), laid(randn(planned, n), d)
    sa, sb = (block_scales(r, k, randn)[0] if a == "mxf8" else None for r in (planned, n))
    rs, cs = torch.exp(0.5 * randn(planned)), torch.exp(0.5 * randn(n))
    bias = randn(n).to(DT[d])
    for kind in ("relu_aux_bias", "gelu_aux_bias"):
        for rows in (1, 16, 17, 33, 64):
            outs = []
            for size in (planned, rows):
                print(f"case {a}->{d} {kind} rows={rows} planned={size}", flush=True)
                D = laid(torch.zeros(planned, n, device="cuda"), d)
                before = D.clone()
                with GemmEpilog(size, n, k, a, d, GE_OP_T, A.stride(0), W.stride(0), D.stride(0)) as g:
                    g.plan_residual(kind)
                    aux = (torch.full((planned, g.aux_ld_bits // 32), -1, dtype=torch.int32, device="cuda")
                           if kind == "relu_aux_bias" else
                           torch.full((planned, g.aux_ld_bits // torch.finfo(DT[d]).bits), 3.0, dtype=DT[d], device="cuda"))
                    aux0 = aux.clone()
                    ws = torch.full((max(1, g.ws_bytes),), 0xA5, dtype=torch.uint8, device="cuda")
                    g.execute_residual(A, W, bias, R, D, aux=aux, row_scale=rs, col_scale=cs, a_scales=sa, b_scales=sb,
                                       workspace=ws, m=rows)
                assert untouched(D) and torch.equal(D[rows:], before[rows:]) and torch.equal(aux[rows:], aux0[rows:])
                outs.append((D[:rows].clone(), aux[:rows].clone()))
            assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1]), rows


@pytest.mark.parametrize("t", ["f16", "bf16", "f32"])
def test_gelu_gradient_of_stored_infinities(t):
    """The forward pass of P = -1e5 and below is finite, and fp16 stores that P as -inf: GELU' there is 0, at +inf 1,
    and at the type's largest values as well; NaN stays NaN and in its own row and column."""
    m, n, k = 40, 72, 48
    randn = gen(31)
    A, W, dD = laid(randn(m, k), t), laid(randn(n, k), t), laid(randn(m, n), t)
    top = torch.finfo(DT[t]).max
    aux = torch.zeros(m, 128, dtype=DT[t], device="cuda")
    aux[:, :n] = torch.tensor([-float("inf"), float("inf"), -top, top, 31.0, -31.0, -29.0], device="cuda")[
        torch.arange(m * n, device="cuda").view(m, n) % 7].to(DT[t])
    slope = (aux[:, :n].double() > 0).double()
    aux[3, 5] = float("nan")
    dP = dD.double() * slope
    gA, gB = laid(torch.zeros(m, k, device="cuda"), t), laid(torch.zeros(n, k, device="cuda"), t)
    gb = torch.empty(n, dtype=DT[t], device="cuda")
    with GemmEpilog(m, n, k, t, t, GE_OP_T, A.stride(0), W.stride(0), dD.stride(0)) as g:
        g.plan_residual("gelu_aux_bias").plan_backward()
        g.backward(dD, A, W, gA, gB, dbias=gb, aux=aux,
                   workspace=torch.empty(g.backward_ws_bytes, dtype=torch.uint8, device="cuda"))
    assert gA[3].isnan().all() and gB[5].isnan().all() and gb[5].isnan()
    rows, cols = (torch.arange(s, device="cuda") != i for s, i in ((m, 3), (n, 5)))
    f = torch.finfo(DT[t])
    for got, want, size, terms in ((gA[rows], (dP @ W.double())[rows], (dP.abs() @ W.double().abs())[rows], n),
                                   (gB[cols], (dP.t() @ A.double())[cols], (dP.abs().t() @ A.double().abs())[cols], m),
                                   (gb[cols], dP.sum(0)[cols], dP.abs().sum(0)[cols], m)):
        tol = size * (terms + 8) * U + want.abs() * f.eps / 2 * (1 + 2.0 ** -6) + f.tiny * f.eps
        assert ((got.double() - want).abs() <= tol).all()


@pytest.mark.parametrize("m", [1, 100])
@pytest.mark.parametrize("a", ["e4m3", "mxf8"])
def test_what_eight_bit_sums_keep(a, m):
    """As the header says of 8-bit operands: beside 2^16, 8 counts in the same group of eight K values, and in another
    group anything does; what is dropped is at most 7 2^-13 of the groups' largest products."""
    k, n, big = 128, 128, 65
    A, W = torch.zeros(m, k, device="cuda"), torch.zeros(n, k, device="cuda")
    A[:, big], W[:, big] = 256, 256
    A[:, :] += torch.where(torch.arange(k, device="cuda") == big, 0.0, 2.0)
    # row j of W: the product 2 w at K value j alone, w = 4 inside the group and 0.5 outside
    j = torch.arange(n, device="cuda")
    inside = j // 8 == big // 8
    W[j, j] += torch.where(j == big, 0.0, torch.where(inside, 4.0, 0.5))
    small = torch.where(inside, 8.0, 1.0).double()
    small[big] = 0
    sa, sb = (torch.full((r, mx_scale_ld(k)), 127, dtype=torch.uint8, device="cuda") if a == "mxf8" else None
              for r in (m, n))
    A, W = laid(A, a), laid(W, a)
    D = laid(torch.zeros(m, n, device="cuda"), "f32")
    with GemmEpilog(m, n, k, a, "f32", GE_OP_T, A.stride(0), W.stride(0), D.stride(0)) as g:
        g.plan_residual("none")
        ws = torch.empty(max(1, g.ws_bytes), dtype=torch.uint8, device="cuda")
        g.execute_residual(A, W, None, None, D, a_scales=sa, b_scales=sb, workspace=ws)
    assert torch.equal(D.double(), (65536.0 + small).expand(m, n))
    # seven products just below the border in the group of the largest
    W2 = torch.zeros(n, k, device="cuda")
    W2[:, big] = 256
    W2[:, 64:72] += torch.where(torch.arange(64, 72, device="cuda") == big, 0.0, 3.75)
    W2 = laid(W2, a)
    want = A.double() @ W2.double().t()
    with GemmEpilog(m, n, k, a, "f32", GE_OP_T, A.stride(0), W2.stride(0), D.stride(0)) as g:
        g.plan_residual("none")
        g.execute_residual(A, W2, None, None, D, a_scales=sa, b_scales=sb, workspace=ws)
    assert ((D.double() - want).abs() <= 7 * 2.0 ** -13 * 65536).all()


@pytest.mark.parametrize("d", ["bf16", "f32"])
def test_few_rows_of_a_split_k_plan(d):
    """A 16-bit weight of 16 MiB on a handle of 100 rows, which has split-K tiles: up to 64 rows stream (the bits of a
    handle of those rows), beyond the call keeps the tiles (the bits of those rows in a full call)."""
    planned, n, k = 100, 1024, 8192
    randn = gen(22)
    A, W, R = laid(randn(planned, k), "bf16"), laid(randn(n, k), "bf16"), laid(randn(planned, n), d)

    def call(size, rows):
        D = laid(torch.zeros(planned, n, device="cuda"), d)
        with GemmEpilog(size, n, k, "bf16", d, GE_OP_T, A.stride(0), W.stride(0), D.stride(0)) as g:
            g.plan_residual("none")
            if size == planned:
                assert "tile_id=14 " in g.describe() and "split_k=1 " not in g.describe()
            ws = torch.full((max(1, g.ws_bytes),), 0xA5, dtype=torch.uint8, device="cuda")
            g.execute_residual(A, W, None, R, D, workspace=ws, m=rows)
        assert untouched(D) and (D[rows:] == 0).all()
        return D[:rows]

    full = call(planned, planned)
    assert torch.equal(call(planned, 65), full[:65])
    for rows in (1, 32, 33, 64):
        got = call(planned, rows)
        assert torch.equal(got, call(rows, rows)), rows
        if d == "f32":   # (another order of adding)
            assert not torch.equal(got, full[:rows])
        want = A[:rows].double() @ W.double().t() + R[:rows].double()
        size = A[:rows].double().abs() @ W.double().abs().t() + R[:rows].double().abs()
        f = torch.finfo(DT[d])
        assert ((got.double() - want).abs() <= (k + 8) * U * size + want.abs() * f.eps / 2 * (1 + 2.0 ** -6)).all()
