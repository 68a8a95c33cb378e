"""The feed-forward example against the same block in 64 bits."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import feed_forward as ff  # noqa: E402

pytestmark = pytest.mark.gpu


def block64(x, r, gamma, w1, b1, w2, b2):
    h = x + r
    y = h / torch.sqrt((h * h).mean(1, keepdim=True) + ff.EPS) * gamma
    p = y @ w1.t() + b1
    u = p / (1 + torch.exp(-2 * 0.7978845608028654 * (p + 0.044715 * p ** 3)))
    return h + u @ w2.t() + b2


@pytest.mark.parametrize("tokens,d,f", [(1, 64, 96), (70, 200, 328), (300, 520, 1000)])
def test_training_step(tokens, d, f):
    """fp32 against automatic differentiation in 64 bits: each result is off by at
    most 2^-24 per addition of its longest chain (norm, two products, and back) relative
    to the result's size; GELU and its slope by 2^-18."""
    args = ff.inputs(tokens, d, f, "f32", 3)
    step = ff.Training(tokens, d, f, "f32")
    out = step.forward(*args)
    dout = ff._laid(torch.randn(tokens, d, device="cuda"), torch.float32)
    step.backward(dout, args[2], args[3], args[5])
    a64 = [a.double().requires_grad_() for a in args]
    want = block64(*a64)
    want.backward(dout.double())
    got = [out, step.dx, step.dx, step.dgamma, step.dw1, step.db1, step.dw2, step.db2]
    ref = [want.detach()] + [a.grad for a in a64]
    tol = 2.0 ** -16 + (2 * (d + f) + tokens) * 2.0 ** -24
    for g, w in zip(got, ref):
        assert (g.double() - w).norm() <= tol * w.norm()


@pytest.mark.parametrize("tokens", [1, 5, 64, 200])
def test_serving(tokens):
    """E4M3 on both sides of the first product: each code is off by at most 2^-4
    of its value, independently, so u by about 2^-4 sqrt(2) of its own size at
    the worst; the residual stream and the 16-bit rounding are far below that."""
    d, f = 256, 520
    args = ff.inputs(200, d, f, "bf16", 5)
    block = ff.Serving(200, *args[2:])
    x, r = args[0], args[1]
    out = block(x[:tokens], r[:tokens])
    h = (x.double() + r.double())[:tokens]
    want = block64(x[:tokens].double(), r[:tokens].double(), *[a.double() for a in args[2:]])
    assert (out.double() - want).norm() <= 2.0 ** -4 * 2 ** 0.5 * (want - h).norm() + 2.0 ** -7 * h.norm()
    # one row at a time gives what the batch gives, to the rounding of the output
    one = block(x[:1], r[:1]).clone()
    assert (one.double() - out[:1].double()).norm() <= 2.0 ** -4 * 2 ** 0.5 * (want[:1] - h[:1]).norm() + 2.0 ** -7 * h[:1].norm()


@pytest.mark.parametrize("planned", [64, 200])
@pytest.mark.parametrize("tokens", [1, 5, 17, 64, 65, 200])
def test_one_token_against_the_batch(planned, tokens):
    """A token alone against the same token in a batch.  Up to 64 rows both take the kernel for few rows, which adds
    in one order whatever the rows: equal bits.  Beyond, the first product is added in another order (off by far less
    than a rounding), so each u may round to a neighbour, a step of 2^-7 of it, and so may out."""
    if tokens > planned:
        pytest.skip("more tokens than planned")
    d, f = 256, 520
    args = ff.inputs(200, d, f, "bf16", 7)
    block = ff.Serving(planned, *args[2:])
    assert ("path=skinny" in block.up.describe()) == (planned <= 64)
    x, r = args[0], args[1]
    batch = block(x[:tokens], r[:tokens])[:1].clone()
    u_batch = block.u[:1].double()
    block.out.fill_(float("nan"))
    block.u.fill_(float("nan"))
    one = block(x[:1], r[:1]).clone()
    u = block.u[:1].double()
    assert one.shape == (1, d) and not one.isnan().any()
    if tokens <= 64:
        assert torch.equal(one, batch) and torch.equal(u, u_batch)
        return
    size = u.abs().maximum(u_batch.abs())
    assert ((u - u_batch).abs() <= size * 2.0 ** -7 + 2.0 ** -20).all()
    w2 = block.w2.double().abs()
    tol = (size * 2.0 ** -7 + 2.0 ** -20) @ w2.t() + (f + 8) * 2.0 ** -24 * (size @ w2.t()) + 2.0 ** -7 * one.double().abs()
    assert ((one.double() - batch.double()).abs() <= tol).all()
