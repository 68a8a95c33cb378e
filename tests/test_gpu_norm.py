"""RMS norm (residual addition, plain and 8-bit outputs) and its backward
pass on the GPU against plain 64-bit forms.

Tolerances.  An output in type t is the fp32 result rounded once: half a step,
eps(t)/2 relative.  The fp32 result itself: the row's sum of squares adds up
to `steps` terms one after another in a thread and then over at most 16 more
levels, so rstd is off by at most (steps + 24) 2^-24 relative, and the two
products by 2^-24 each; `K` below counts those steps for the row length."""
import pytest
import torch

from activation_epilogue_02_amd import RmsNorm, mx_scale_ld

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-6
U = 2.0 ** -24


def K(cols):
    return max(32, cols // 1024) + 32


def laid(v, dtype, pad):
    """v in dtype, rows padded to 16 bytes and `pad` chunks more; the padding holds NaN."""
    e = 128 // torch.finfo(dtype).bits
    ld = -(-v.shape[1] // e) * e + pad * e
    m = torch.full((v.shape[0], ld), float("nan"), dtype=dtype, device="cuda")
    m[:, :v.shape[1]] = v
    return m[:, :v.shape[1]]


def inputs(rows, cols, dtype, pad, seed, residual=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    level = torch.exp(torch.randn(rows, 1, generator=g, device="cuda"))
    x = laid(torch.randn(rows, cols, generator=g, device="cuda") * level, dtype, pad)
    r = laid(torch.randn(rows, cols, generator=g, device="cuda") * level, dtype, pad) if residual else None
    gamma = (1 + 0.3 * torch.randn(cols, generator=g, device="cuda")).to(dtype)
    return x, r, gamma


def exact(x, r, gamma):
    h = x if r is None else (x.float() + r.float()).to(x.dtype)
    hd = h.double()
    rstd = 1 / torch.sqrt((hd * hd).mean(1) + EPS)
    return h, rstd, hd * rstd[:, None] * gamma.double()


def near(got, want, dtype, k):
    """got (in dtype) is want rounded once, off by k fp32 steps before."""
    f = torch.finfo(dtype)
    tol = want.abs() * (f.eps / 2 * (1 + 2.0 ** -6) + k * U) + f.tiny * f.eps
    bad = (got.double() - want).abs() > tol
    assert not bad.any(), (int(bad.sum()), got[bad][:4], want[bad][:4])


SIZES = [(1, 1), (3, 7), (5, 64), (9, 520), (2, 1000), (7, 2048), (3, 2055), (2, 4104), (5, 8192), (3, 16383),
         (2, 16392), (2, 32768), (2, 40001)]


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("residual", [True, False], ids=["res", "nores"])
def test_plain(rows, cols, dtype, residual):
    t = DT[dtype]
    pad = cols % 3
    x, r, gamma = inputs(rows, cols, t, pad, cols, residual)
    h, rstd, y = exact(x, r, gamma)
    with RmsNorm(rows, cols, dtype, eps=EPS, ld=x.stride(0), ldy=x.stride(0)) as n:
        out = laid(torch.zeros(rows, cols, device="cuda"), t, pad)
        hs = laid(torch.zeros(rows, cols, device="cuda"), t, pad) if residual else None
        rs = torch.full((rows + 1,), -1.0, device="cuda")
        n.forward(x, gamma, out, residual=r, h=hs, rstd=rs)
        if residual:
            assert torch.equal(hs, h)
        near(out, y, t, K(cols))
        assert ((rs[:rows].double() - rstd).abs() <= rstd * K(cols) * U).all() and rs[rows] == -1
        # the padding is untouched
        for m in (out, hs):
            if m is not None:
                assert m.as_strided((rows, m.stride(0) - cols), (m.stride(0), 1), m.storage_offset() + cols).isnan().all()
        # without h, and with the output in place of x
        again = laid(x, t, pad)
        n.forward(again, gamma, again, residual=r)
        assert torch.equal(again, out)
        # h in place of the residual
        if residual:
            rr = laid(r, t, pad)
            n.forward(x, gamma, out, residual=rr, h=rr)
            assert torch.equal(rr, h) and torch.equal(again, out)


def check_codes(codes, v, k):
    """codes (E4M3) against v, whose fp32 counterpart is off by k steps: half
    a step is 2^-4 of the value, 2^-10 below 2^-6; beyond 448 saturates."""
    v = v.clamp(-448, 448)
    bad = (codes.double() - v).abs() > torch.maximum(v.abs() * 2.0 ** -4, torch.full_like(v, 2.0 ** -10)) + v.abs() * k * U
    assert not bad.any(), (int(bad.sum()), codes[bad][:4].float(), v[bad][:4])


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_row_scaled_codes(rows, cols, dtype):
    t = DT[dtype]
    x, r, gamma = inputs(rows, cols, t, 1, cols + 1)
    if rows > 1:
        x[1] = 0
        r[1] = 0
    h, _, y = exact(x, r, gamma)
    with RmsNorm(rows, cols, dtype, out="e4m3_row", eps=EPS, ld=x.stride(0)) as n:
        out, scales = n.alloc_outputs()
        out.as_strided((rows, n.ldy), (n.ldy, 1)).view(torch.uint8).fill_(0x55)
        hs = laid(torch.zeros(rows, cols, device="cuda"), t, 1)
        n.forward(x, gamma, out, residual=r, h=hs, scales=scales)
        assert torch.equal(hs, h)
        top = y.abs().amax(1)
        want = torch.where(top > 0, top / 448, torch.ones_like(top))
        assert ((scales.double() - want).abs() <= want * (K(cols) + 4) * U).all()
        check_codes(out, y / want[:, None], 2 * K(cols) + 8)
        # the largest value of a row has the largest code
        assert (out.float().abs().amax(1)[top > 0] == 448).all()
        if n.ldy > cols:
            rest = out.as_strided((rows, n.ldy - cols), (n.ldy, 1), cols)
            assert (rest.view(torch.uint8) == 0x55).all()


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_block_scaled_codes(rows, cols, dtype):
    t = DT[dtype]
    x, r, gamma = inputs(rows, cols, t, 0, cols + 2)
    # blocks of zeros, and of tiny and huge values beside ordinary ones
    if cols >= 96:
        x[:, 32:64] = 0
        r[:, 32:64] = 0
        gamma[64:96] *= 2.0 ** -12
    h, _, y = exact(x, r, gamma)
    with RmsNorm(rows, cols, dtype, out="mx", eps=EPS, ld=x.stride(0)) as n:
        out, scales = n.alloc_outputs()
        assert scales.shape == (rows, mx_scale_ld(cols))
        scales.fill_(0xEE)
        n.forward(x, gamma, out, residual=r, scales=scales)
        nb = -(-cols // 32)
        assert (scales[:, nb:] == 0xEE).all()
        top = torch.nn.functional.pad(y, (0, nb * 32 - cols)).view(rows, nb, 32).abs().amax(2)
        lo, hi = (torch.floor(torch.log2(torch.where(top > 0, top * (1 + s * K(cols) * U), torch.full_like(top, 256.0)))) - 8 + 127
                  for s in (-1, 1))
        b = scales[:, :nb].double()
        assert ((b == lo) | (b == hi)).all()
        check_codes(out, y * torch.exp2(127 - b).repeat_interleave(32, 1)[:, :cols], 2 * K(cols))


@pytest.mark.parametrize("out", ["plain", "e4m3_row", "mx"])
def test_bad_values(out):
    """A NaN or an infinity in a row makes that row NaN (an infinity: NaN and
    zeros) and leaves the others alone; codes hold NaN as NaN."""
    rows, cols = 6, 300
    x, _, gamma = inputs(rows, cols, torch.float32, 0, 3, False)
    clean = x.clone()
    x = laid(x, torch.float32, 0)
    x[1, 7] = float("nan")
    x[3, 299] = float("inf")
    x[4, 0] = -float("inf")
    with RmsNorm(rows, cols, "f32", out=out, ld=x.stride(0)) as n:
        y, scales = n.alloc_outputs()
        n.forward(x, gamma, y, scales=scales)
        y2, s2 = n.alloc_outputs()
        n.forward(laid(clean, torch.float32, 0), gamma, y2, scales=s2)
        y, y2 = y.float(), y2.float()
        for i in (0, 2, 5):
            assert torch.equal(y[i], y2[i]) and (scales is None or torch.equal(scales[i], s2[i]))
        assert y[1].isnan().all() and y[3, 299].isnan() and y[4, 0].isnan()
        assert (y[3, :299] == 0).all() and (y[4, 1:] == 0).all()
        if out == "e4m3_row":
            assert (scales[[1, 3, 4]] == 1).all()
        if out == "mx":
            assert (scales[[1, 3, 4], :10] == 127).all()


def grads(dy, h, gamma, rstd, dh):
    """The formula in 64 bits, and the size of what each result adds up."""
    dyd, hd, gd, r = dy.double(), h.double(), gamma.double(), rstd.double()[:, None]
    n, g = hd * r, dyd * gd
    mean = (g * n).mean(1, keepdim=True)
    dx = r * (g - n * mean)
    size = r * (g.abs() + n.abs() * (g * n).abs().mean(1, keepdim=True))
    if dh is not None:
        dx = dx + dh.double()
        size = size + dh.double().abs()
    return dx, size, (dyd * n).sum(0), (dyd * n).abs().sum(0)


@pytest.mark.parametrize("rows,cols", SIZES + [(1000, 33), (333, 2055), (2100, 96), (300, 40001)])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("with_dh", [True, False], ids=["dh", "nodh"])
def test_backward(rows, cols, dtype, with_dh):
    if cols == 40001 and rows > 2 and dtype != "f16":
        pytest.skip("many long rows: one type")
    t = DT[dtype]
    pad = cols % 3
    h, dy, gamma = inputs(rows, cols, t, pad, cols + 3)
    dh = inputs(rows, cols, t, pad, cols + 4)[0] if with_dh else None
    rstd = (1 / torch.sqrt((h.double() ** 2).mean(1) + EPS)).float()
    dx, size, dg, dgsize = grads(dy, h, gamma, rstd, dh)
    with RmsNorm(rows, cols, dtype, eps=EPS, ld=h.stride(0)) as n:
        got = laid(torch.zeros(rows, cols, device="cuda"), t, pad)
        gg = torch.full((cols + 8,), 7.0, dtype=t, device="cuda")
        ws = torch.full((n.workspace_bytes,), 0xA5, dtype=torch.uint8, device="cuda")
        n.backward(dy, h, gamma, rstd, got, gg[:cols], dh=dh, workspace=ws)
        f = torch.finfo(t)
        tol = dx.abs() * f.eps / 2 * (1 + 2.0 ** -6) + size * K(cols) * U + f.tiny * f.eps
        assert ((got.double() - dx).abs() <= tol).all()
        # dgamma: rows in turn, then at most 1024 partial sums
        tol = dg.abs() * f.eps / 2 * (1 + 2.0 ** -6) + dgsize * (rows // 4 + 48) * U + f.tiny * f.eps
        assert ((gg[:cols].double() - dg).abs() <= tol).all() and (gg[cols:] == 7).all()
        # dx alone, in place of dy, and again: equal bits
        ip = laid(dy, t, pad)
        n.backward(ip, h, gamma, rstd, ip, dh=dh)
        assert torch.equal(ip, got)
        g2 = torch.empty(cols, dtype=t, device="cuda")
        n.backward(dy, h, gamma, rstd, ip, g2, dh=dh, workspace=ws)
        assert torch.equal(g2, gg[:cols])


def test_backward_against_differences():
    """dx and dgamma against central differences of the 64-bit forward form."""
    rows, cols = 3, 37
    h, dy, gamma = inputs(rows, cols, torch.float32, 0, 11)
    hd, dyd, gd = h.double(), dy.double(), gamma.double()

    def loss(x, g):
        return (dyd * x / torch.sqrt((x * x).mean(1, keepdim=True) + EPS) * g).sum()

    step = 1e-5
    fx, fg = torch.empty_like(hd), torch.empty_like(gd)
    for i in range(rows):
        for j in range(cols):
            e = torch.zeros_like(hd)
            e[i, j] = step
            fx[i, j] = (loss(hd + e, gd) - loss(hd - e, gd)) / (2 * step)
    for j in range(cols):
        e = torch.zeros_like(gd)
        e[j] = step
        fg[j] = (loss(hd, gd + e) - loss(hd, gd - e)) / (2 * step)
    rstd = (1 / torch.sqrt((hd ** 2).mean(1) + EPS)).float()
    with RmsNorm(rows, cols, "f32", ld=h.stride(0)) as n:
        dx = laid(torch.zeros(rows, cols, device="cuda"), torch.float32, 0)
        dg = torch.empty(cols, device="cuda")
        n.backward(dy, h, gamma, rstd, dx, dg, workspace=torch.empty(n.workspace_bytes, dtype=torch.uint8, device="cuda"))
    _, size, _, dgsize = grads(dy, h, gamma, rstd, None)
    # differences: step^2 of the third derivative (a few times size / h^2) and 2^-53 |loss| / step, under 1e-8 here
    assert ((dx.double() - fx).abs() <= size * 70 * U + 1e-6 * size + 1e-8).all()
    assert ((dg.double() - fg).abs() <= dgsize * 70 * U + 1e-8).all()


def test_fewer_rows_and_none():
    with RmsNorm(64, 200, "bf16", ld=200) as n:
        x, r, gamma = inputs(64, 200, torch.bfloat16, 0, 5)
        full, part = (torch.full((64, 200), 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        n.forward(x, gamma, full, residual=r)
        n.forward(x, gamma, part, residual=r, rows=10)
        assert torch.equal(part[:10], full[:10]) and (part[10:] == 3).all()
        n.forward(x, gamma, part, rows=0)
        dg = torch.full((200,), 3.0, dtype=torch.bfloat16, device="cuda")
        n.backward(x, x, gamma, torch.ones(64, device="cuda"), part, dg, rows=0)
        assert (dg == 0).all() and (part[10:] == 3).all()


def test_offsets_past_32_bits():
    """Rows that start more than 2^32 bytes into their buffers."""
    rows, cols, ld = 5, 72, (1 << 29) + 64   # 2.1 GB a row of bf16: the last starts at 4.3 GB
    x = torch.empty((rows - 1) * ld + 80, dtype=torch.bfloat16, device="cuda").as_strided((rows, cols), (ld, 1))
    x.copy_(torch.randn(rows, cols, device="cuda"))
    gamma = torch.ones(cols, dtype=torch.bfloat16, device="cuda")
    small = x.contiguous()
    with RmsNorm(rows, cols, "bf16", ld=ld, ldy=72) as n, RmsNorm(rows, cols, "bf16", ld=72, ldy=72) as m:
        a, b = (torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        n.forward(x, gamma, a)
        m.forward(small, gamma, b)
        assert torch.equal(a, b)


def test_stream_and_graph():
    """On a side stream, and captured: every replay gives the eager result."""
    x, r, gamma = inputs(40, 1000, torch.bfloat16, 0, 8)
    dy = inputs(40, 1000, torch.bfloat16, 0, 9)[0]
    n = RmsNorm(40, 1000, "bf16", ld=x.stride(0), ldy=x.stride(0))
    mk = lambda: laid(torch.zeros(40, 1000, device="cuda"), torch.bfloat16, 0)
    y, h, dx = mk(), mk(), mk()
    rstd, dg = torch.empty(40, device="cuda"), torch.empty(1000, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(n.workspace_bytes, dtype=torch.uint8, device="cuda")

    def step():
        n.forward(x, gamma, y, residual=r, h=h, rstd=rstd)
        n.backward(dy, h, gamma, rstd, dx, dg, dh=y, workspace=ws)

    step()
    want = [t.clone() for t in (y, h, dx, dg)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            step()
    torch.cuda.current_stream().wait_stream(s)
    for k in range(3):
        for t in (y, h, dx, dg):
            t.fill_(k)
        ws.fill_(k)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((y, h, dx, dg), want)), k
    n.free()


def test_more_rows_than_workgroups():
    """4 M short rows: the launch is bounded and its waves walk the rows."""
    rows, cols = (1 << 22) + 3, 8
    g = torch.Generator(device="cuda").manual_seed(12)
    x = torch.randn(rows, cols, generator=g, device="cuda").bfloat16()
    gamma = torch.ones(cols, dtype=torch.bfloat16, device="cuda")
    y = torch.full_like(x, 9.0)
    with RmsNorm(rows, cols, "bf16", eps=EPS) as n:
        n.forward(x, gamma, y)
    near(y, exact(x, None, gamma)[2], torch.bfloat16, K(cols))


def test_tiny_rows_keep_a_normal_scale():
    """A row of values so small that max / 448 is no normal number: its scale is 2^-126, no code is NaN."""
    x = torch.full((2, 40), 1e-42, device="cuda")
    x[0, 3] = 0
    x[1] = 3e-37
    gamma = torch.ones(40, device="cuda")
    with RmsNorm(2, 40, "f32", out="e4m3_row", eps=1.0, ld=40) as n:
        y, s = n.alloc_outputs()
        n.forward(x, gamma, y, scales=s)
    assert (s == 2.0 ** -126).all() and (y[0].float() == 0).all()
    # 3e-37 * 2^126 = 25.5: the nearest code is 26
    assert (y[1].float() == 26).all()


@pytest.mark.parametrize("dtype,cols", [("f32", 1024), ("f32", 32768), ("f16", 512), ("f16", 65536), ("bf16", 256),
                                        ("bf16", 8192), ("bf16", 65536)])
def test_codes_are_those_of_the_quotient(dtype, cols):
    """Rows of +-1 with eps = 0 have rstd = 1 exactly, so y = +-gamma.  With gamma = c s for c half way between
    two codes and 448 s the largest, y / s = c exactly and the codes are c rounded to even."""
    t = DT[dtype]
    c = torch.tensor([(2 * j + 1) / 32 * 2.0 ** e for j in range(8, 16) for e in range(-5, 9)], dtype=torch.float64)
    c = torch.cat([c[c < 448], torch.tensor([448.0], dtype=torch.float64)])
    c = c.repeat(cols // len(c) + 1)[:cols]
    want = c.to(torch.float8_e4m3fn).float()
    sign = torch.where(torch.arange(cols) % 3 == 0, -1.0, 1.0)
    scales = {"bf16": [1.25, 1.5, 1.75, 0.75, 40.0], "f16": [1 + i / 16 for i in range(1, 16)],
              "f32": [1 + i / 512 for i in range(3, 512, 20)] + [1.7 * 2.0 ** -110, 1.3 * 2.0 ** 100]}[dtype]
    if dtype == "f32":
        scales = [float(torch.tensor(s, dtype=torch.float32).view(torch.int32).bitwise_and(-4096).view(torch.float32))
                  for s in scales]   # 12 bits: c s is exact
    with RmsNorm(2, cols, dtype, out="e4m3_row", eps=0.0) as n:
        x = (sign * torch.tensor([[1.0], [-1.0]])).to(t).cuda()
        y, row_scale = n.alloc_outputs()
        for s in scales:
            gamma = (c * s).to(t)
            assert torch.equal(gamma.double(), c * s)
            n.forward(x, gamma.cuda(), y, scales=row_scale)
            assert (row_scale.double().cpu() == s).all(), s
            got = y.float().cpu()
            assert torch.equal(got[0], sign * want) and torch.equal(got[1], -sign * want), s


def test_infinite_values_with_a_row_scale():
    """gamma so large that a value of y is infinite: the scale is infinite, that code NaN and the others zero."""
    gamma = torch.ones(64, device="cuda")
    gamma[5] = 3e38
    x = torch.zeros(1, 64, device="cuda")
    x[0, :8] = torch.arange(1, 9, device="cuda")
    with RmsNorm(1, 64, "f32", out="e4m3_row", eps=0.0) as n:
        y, s = n.alloc_outputs()
        n.forward(x, gamma, y, scales=s)
    y = y.float()
    assert s.isinf().all() and y[0, 5].isnan() and (y[0, :5] == 0).all() and (y[0, 6:] == 0).all()


@pytest.mark.parametrize("planned,rows,cols", [(3000, 2100, 96), (3000, 3000, 200), (700, 300, 2055), (700, 1, 4104),
                                               (400, 257, 8200), (600, 513, 1000), (40, 7, 40001)])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_backward_of_fewer_rows(planned, rows, cols, dtype):
    """0 < rows <= the handle's, with the workspace of the whole handle; dgamma under the bound of the launch: a group
    adds its rows in turn, the groups of a workgroup one after the other, then 32 lanes every 32nd workgroup's sum, and
    the 32 of them; each term is off by 3 roundings itself."""
    t = DT[dtype]
    h, dy, gamma = inputs(planned, cols, t, 1, cols + 5)
    dh = inputs(planned, cols, t, 1, cols + 6)[0]
    rstd = (1 / torch.sqrt((h.double() ** 2).mean(1) + EPS)).float()
    dx, size, dg, dgsize = grads(dy[:rows], h[:rows], gamma, rstd[:rows], dh[:rows])
    got = laid(torch.full((planned, cols), 3.0, device="cuda"), t, 1)
    gg = torch.full((cols + 8,), 7.0, dtype=t, device="cuda")
    with RmsNorm(planned, cols, dtype, eps=EPS, ld=h.stride(0)) as n:
        threads = int(n.describe().split("backward=")[1].split("x")[0])
        ws = torch.full((n.workspace_bytes,), 0xA5, dtype=torch.uint8, device="cuda")
        n.backward(dy, h, gamma, rstd, got, gg[:cols], dh=dh, workspace=ws, rows=rows)
    f = torch.finfo(t)
    assert (got[rows:] == 3).all() and (gg[cols:] == 7).all()
    tol = dx.abs() * f.eps / 2 * (1 + 2.0 ** -6) + size * K(cols) * U + f.tiny * f.eps
    assert ((got[:rows].double() - dx).abs() <= tol).all()
    blocks, groups = min(rows, 256), max(1, 512 // threads)
    steps = -(-rows // (blocks * groups)) + groups + -(-blocks // 32) + 32 + 3
    tol = dg.abs() * f.eps / 2 * (1 + 2.0 ** -6) + dgsize * steps * U + f.tiny * f.eps
    assert ((gg[:cols].double() - dg).abs() <= tol).all()
    # a handle of those rows gives the same bits
    with RmsNorm(rows, cols, dtype, eps=EPS, ld=h.stride(0)) as n:
        again = laid(torch.zeros(rows, cols, device="cuda"), t, 1)
        g2 = torch.empty(cols, dtype=t, device="cuda")
        n.backward(dy, h, gamma, rstd, again, g2, dh=dh, rows=rows,
                   workspace=torch.empty(n.workspace_bytes, dtype=torch.uint8, device="cuda"))
        assert torch.equal(again, got[:rows]) and torch.equal(g2, gg[:cols])
