"""fp8_linear_epilogue: bias, activation, residual and FP8 output against the
formula in 64 bits.

Tolerance, with v the exact value before the last rounding and a = s_in s_w
sum |x w| + |bias| + |residual|: the fp32 sum and the epilogue's few roundings
are within (K + 16) 2^-21 a (worst case, with slack for a tensor-core sum a few
bits short of fp32, as the other GEMM tests allow), times the activation's
slope, at most 1.13 (GELU); BF16 output rounds by 2^-8 |v|, FP8 by half a step of
E4M3 (2^-4 |v|, 2^-10 steps below the normal range) and, as it multiplies by the
reciprocal of s_out, 2^-23 |v|."""

import math

import pytest
import torch

import fp8_w8a8_static_b200 as fw

pytestmark = pytest.mark.gpu
DEV = "cuda"
F8 = torch.float8_e4m3fn


def one(x):
    return torch.tensor([x], dtype=torch.float32, device=DEV)


def make(M, N, K, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    xq = (rn(M, K) * 60).clamp(-448, 448).to(F8)
    wq = (rn(N, K) * 60).clamp(-448, 448).to(F8)
    return xq, wq, rn(N).bfloat16(), rn(M, N).bfloat16()


def formula(xq, wq, s, bias, act, residual):
    x, w = xq.double(), wq.double()
    v = x @ w.t() * s
    a = x.abs() @ w.abs().t() * s
    if bias is not None:
        v, a = v + bias.double(), a + bias.double().abs()
    if act == "relu":
        v = v.clamp(min=0)
    elif act == "silu":
        v = v * torch.sigmoid(v)
    elif act == "gelu":
        v = 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))
    if residual is not None:
        v, a = v + residual.double(), a + residual.double().abs()
    return v, a


def check(y, v, a, K, s_out=None):
    err = 1.13 * (K + 16) * 2.0 ** -21 * a
    if s_out is None:
        d, lim = (y.double() - v).abs(), err + 2.0 ** -8 * v.abs()
    else:
        t = v / s_out
        step = torch.maximum((2.0 ** -4 + 2.0 ** -23) * t.abs(), torch.full_like(t, 2.0 ** -10))
        d, lim = (y.float().double() - t.clamp(-448, 448)).abs(), err / s_out + step
    assert torch.isfinite(y.float()).all()
    assert (d <= lim).all(), (d - lim).max()


S_IN, S_W = 4.0 / 448, 0.05 / 448
SHAPES = [(1, 16, 16), (3, 32, 48), (17, 208, 256), (64, 704, 256), (128, 128, 128), (129, 272, 400),
          (255, 256, 2048), (300, 2048, 1040), (1000, 528, 2048), (513, 1040, 144)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("bias,act,residual,fp8", [
    (False, "none", False, False), (True, "none", True, False), (True, "gelu", False, True),
    (True, "silu", True, True), (False, "relu", True, False), (True, "silu", False, False),
    (False, "gelu", True, True)])
def test_against_the_formula(M, N, K, bias, act, residual, fp8):
    xq, wq, b, r = make(M, N, K, M + N + K)
    b, r = b if bias else None, r if residual else None
    s_out = 0.01 if fp8 else None
    y = fw.fp8_linear_epilogue(xq, wq, one(S_IN), one(S_W), b, act, r, one(s_out) if fp8 else None)
    assert y.dtype == (F8 if fp8 else torch.bfloat16)
    v, a = formula(xq, wq, float(one(S_IN).double() * one(S_W).double()), b, act, r)
    check(y, v, a, K, s_out)


@pytest.mark.parametrize("M", [31, 32, 33, 63, 64, 65, 100, 127, 128, 129, 255, 256, 257, 700])
@pytest.mark.parametrize("N,K", [(528, 2048), (96, 4112), (6000, 384), (264, 1424), (272, 1536)])
def test_row_counts_where_the_kernel_changes(M, N, K):
    """The kernels' borders in rows, each with K split over a cluster in
    several ways (its last range short), and the same bits again."""
    xq, wq, b, r = make(M, N, K, M)
    args = (xq, wq, one(S_IN), one(S_W), b, "gelu", r)
    y = fw.fp8_linear_epilogue(*args)
    v, a = formula(xq, wq, float(one(S_IN).double() * one(S_W).double()), b, "gelu", r)
    check(y, v, a, K)
    assert torch.equal(fw.fp8_linear_epilogue(*args), y)


@pytest.mark.parametrize("N", [8, 24, 1000])
def test_widths_of_eight(N):
    xq, wq, b, r = make(70, N, 64, N)
    y = fw.fp8_linear_epilogue(xq, wq, one(S_IN), one(S_W), b, "silu", r)
    v, a = formula(xq, wq, float(one(S_IN).double() * one(S_W).double()), b, "silu", r)
    check(y, v, a, 64)


@pytest.mark.parametrize("M", [1, 40, 700])
def test_plain_is_fp8_linear_static(M):
    """Without bias, activation and residual: the plain Linear, to the fp32
    sum's rounding order."""
    xq, wq, _, _ = make(M, 512, 1024, M)
    y = fw.fp8_linear_epilogue(xq, wq, one(S_IN), one(S_W))
    z = fw.fp8_linear_static(xq, wq, one(S_IN), one(S_W))
    _, a = formula(xq, wq, S_IN * S_W, None, "none", None)
    assert ((y.double() - z.double()).abs() <= 2.0 ** -7 * z.double().abs() + 2 * 1040 * 2.0 ** -21 * a).all()


@pytest.mark.parametrize("M", [5, 33, 64, 100, 600])
@pytest.mark.parametrize("K", [256, 1552])
def test_residual_in_place(M, K):
    xq, wq, b, r = make(M, 528, K, M)
    want = fw.fp8_linear_epilogue(xq, wq, one(S_IN), one(S_W), b, "none", r)
    got = r.clone()
    fw.fp8_linear_epilogue(xq, wq, one(S_IN), one(S_W), b, "none", got, out=got)
    assert torch.equal(got, want)


@pytest.mark.parametrize("M", [7, 300])
@pytest.mark.parametrize("fp8", [False, True])
def test_writes_its_output_and_nothing_else(M, fp8):
    N = 272
    xq, wq, b, r = make(M, N, 128, 4)
    flat = torch.full((M + 2, N), 99.0, device=DEV).to(F8 if fp8 else torch.bfloat16)
    y = flat[1:M + 1]
    fw.fp8_linear_epilogue(xq, wq, one(S_IN), one(S_W), b, "gelu", r, one(0.01) if fp8 else None, out=y)
    ref = fw.fp8_linear_epilogue(xq, wq, one(S_IN), one(S_W), b, "gelu", r, one(0.01) if fp8 else None)
    assert torch.equal(y.view(torch.uint8), ref.view(torch.uint8))
    edge = torch.full((N,), 99.0, device=DEV).to(flat.dtype)
    assert torch.equal(flat[0].float(), edge.float()) and torch.equal(flat[-1].float(), edge.float())


@pytest.mark.parametrize("M", [2, 140])
@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu"])
def test_nan_and_infinities(M, act):
    xq, wq, b, r = make(M, 64, 32, 9)
    b[3], b[5], b[7] = float("nan"), float("inf"), -1e30
    r[1, 9] = float("nan")
    y = fw.fp8_linear_epilogue(xq, wq, one(S_IN), one(S_W), b, act, r)
    assert torch.isnan(y[:, 3]).all() and torch.isnan(y[1, 9])
    assert (y[:, 5] == float("inf")).all()
    if act != "none":                      # the activations vanish far below zero
        assert torch.equal(y[:, 7], r[:, 7])
    others = torch.ones_like(y, dtype=torch.bool)
    others[:, [3, 5, 7]] = False
    others[1, 9] = False
    assert torch.isfinite(y[others]).all()


def test_captured_and_replayed():
    xq, wq, b, r = make(200, 528, 256, 6)
    s = [one(S_IN), one(S_W)]
    want = fw.fp8_linear_epilogue(xq, wq, *s, b, "gelu", r)
    out = torch.zeros_like(want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fw.fp8_linear_epilogue(xq, wq, *s, b, "gelu", r, out=out)
    for _ in range(3):
        out.fill_(float("nan"))
        g.replay()
        assert torch.equal(out, want)
