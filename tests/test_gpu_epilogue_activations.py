"""The activations of the Linear with a fused epilogue at every BF16 value, in both
kernels: the products are 0 and the bias is the value.

Tolerance: half a step of BF16's output (2^-8 of the value, or 2^-134 in its
subnormals), the stated 2^-20 + |a| 2^-22 with a the exponential's argument, and
|x| 2^-126 where 1 + e^a exceeds 2^126 and the result is 0."""

import math

import pytest
import torch

import fp8_w8a8_static_b200 as fw

pytestmark = pytest.mark.gpu
DEV = "cuda"


def outputs(act, rows):
    x = torch.arange(-2 ** 15, 2 ** 15, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).to(DEV)
    one = torch.ones(1, device=DEV)
    xq, wq = (torch.zeros(n, 16, device=DEV).to(fw.FP8) for n in (rows, len(x)))
    y = fw.fp8_linear_epilogue(xq, wq, one, one, bias=x, act=act)
    assert torch.equal(y.view(torch.int16), y[:1].expand_as(y).contiguous().view(torch.int16))
    return x.double(), y[0].double()


@pytest.mark.parametrize("rows", [1, 200])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_every_value(act, rows):
    x, y = outputs(act, rows)
    a = -x if act == "silu" else -2 * math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3)
    want = x / (1 + torch.exp(a))
    fin = torch.isfinite(x)
    tol = want.abs() * (2.0 ** -8 + 2.0 ** -20 + a.abs() * 2.0 ** -22) + x.abs() * 2.0 ** -126 + 2.0 ** -134
    bad = fin & ~((y - want).abs() <= torch.where(torch.isfinite(tol), tol, torch.zeros_like(tol)))
    bad &= ~((want == 0) & (y == 0))
    assert not bad.any(), (x[bad][:8], y[bad][:8], want[bad][:8])
    assert torch.isnan(y[torch.isnan(x)]).all() and (y[x == math.inf] == math.inf).all()


@pytest.mark.parametrize("rows", [1, 200])
@pytest.mark.parametrize("act", ["none", "relu"])
def test_every_value_exactly(act, rows):
    x, y = outputs(act, rows)
    want = x if act == "none" else torch.where(x < 0, torch.zeros_like(x), x)
    fin = ~torch.isnan(x)
    assert torch.equal(y[fin], want[fin]) and torch.isnan(y[~fin]).all()
