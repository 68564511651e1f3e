"""The edges of attention over the 4-bit cache with enough rows and heads for
the tensor-core kernel: contexts short enough for one block a row block, and
long ones whose tokens several blocks share.  Tolerances: test_gpu_fp4_kv.py's."""

import numpy as np
import pytest
import torch

import fp8_w8a8_static_b200 as fw
import _kv4
from test_gpu_fp4_kv import DEV, S_K, S_V, attend, check, filled, ints, one, rand

pytestmark = pytest.mark.gpu
HEADS = 6  # 256-row blocks in every call: more than a handful


@pytest.mark.parametrize("kv", [777, 3001])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("scale", [0.0, -0.1, 2.0])
def test_other_scales(kv, dim, scale):
    attend([70], [kv], HEADS, 2, dim, 64, True, scale=scale)


@pytest.mark.parametrize("kv", [[700, 80], [3000, 2000]])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("s_out", [0.004, 1e-3])
def test_fp8_output(kv, dim, s_out):
    attend([60, 50], kv, HEADS, 3, dim, 32, True, s_out=s_out)


@pytest.mark.parametrize("kv", [[0, 3, 0], [0, 2000, 59], [1, 0, 4000]])
def test_rows_without_tokens(kv):
    """Requests without tokens, and causal rows before the context's first."""
    out = attend([60, 60, 60], kv, HEADS, 3, 64, 16, True)
    for b, n in enumerate(kv):
        if n < 60:
            assert (out[60 * b:60 * (b + 1) - n] == 0).all()
    attend([60, 60, 60], kv, HEADS, 1, 128, 16, False)


@pytest.mark.parametrize("n", [600, 2500])
@pytest.mark.parametrize("dim", [64, 128])
def test_rising_scores(n, dim):
    cache, table = filled([n], HEADS, dim, 16, 3)
    k = torch.zeros(n, HEADS, dim)
    k[:, :, 0] = torch.arange(n)[:, None] * (60.0 / n)
    k[:, :, 1:] = torch.randn(n, HEADS, dim - 1, generator=torch.Generator().manual_seed(1)) * 0.1
    k[:, 1::2, 0] *= -1  # falling
    slots = table[0].repeat_interleave(16)[:n].long() * 16 + torch.arange(n, device=DEV) % 16
    fw.fp4_kv_append(k.bfloat16().to(DEV), rand(n, HEADS, dim, seed=8), slots, cache, one(S_K), one(S_V))
    q = rand(64, 2 * HEADS, dim, seed=9)
    q[:, :, 0] = 3.0
    q[:, 1::2] *= 1e-3
    q[1::2] *= 2.0 ** 20
    q[2::4] *= 2.0 ** -60
    args = (q, ints([0, 64]), ints([n]), table, cache, one(S_K), one(S_V), 64, 2.0 ** -20, True)
    out, lse = fw.fp4_kv_attention(*args, return_lse=True)
    check(out, lse, _kv4.attention(q, args[1], torch.tensor([n]), table, cache, S_K, S_V,
                                   2.0 ** -20, True), 6.0, n)


@pytest.mark.parametrize("kv", [[100, 100, 333], [1500, 1300, 2100]])
@pytest.mark.parametrize("causal", [True, False])
def test_pages_that_the_cache_lacks(kv, causal):
    cache, table = filled(kv, HEADS, 64, 16, 21)
    table[0, 2] = -1
    table[0, 0] = cache.shape[0]
    table[1, :] = -7
    table[2, 5:9] = 2 ** 31 - 1
    table[2, -20:] = -1                  # a whole chunk and more, at the end
    q = rand(180, 2 * HEADS, 64, seed=22)
    cu = ints([0, 60, 120, 180])
    out, lse = fw.fp4_kv_attention(q, cu, ints(kv), table, cache, one(S_K), one(S_V), 60, 0.125,
                                   causal, return_lse=True)
    ref = _kv4.attention(q, cu, torch.tensor(kv), table, cache, S_K, S_V, 0.125, causal)
    check(out, lse, ref, 4.0, max(kv))
    assert (out[60:120] == 0).all() and torch.isinf(lse[60:120]).all()


@pytest.mark.parametrize("cap", [64, 2048])
def test_lengths_beyond_the_table_and_offsets_beyond_the_rows(cap):
    cache, table = filled([cap, cap], HEADS, 64, 16, 31, extra_width=0)
    q = rand(120, 2 * HEADS, 64, seed=32)
    cu = ints([-5, 60, 1120])
    lens = [10 ** 9, cap]
    out, lse = fw.fp4_kv_attention(q, cu, ints(lens), table, cache, one(S_K), one(S_V), 60, 0.1,
                                   True, return_lse=True)
    check(out, lse, _kv4.attention(q, cu, torch.tensor(lens), table, cache, S_K, S_V, 0.1, True),
          4.0, cap)


@pytest.mark.parametrize("kv", [[50, 100, 7], [1050, 3100, 70]])
def test_rows_outside_every_request_stay(kv):
    q = [60, 70, 1]
    cache, table = filled(kv, HEADS, 128, 32, 41)
    x = rand(140, HEADS, 128, seed=42)
    out = torch.full_like(x, 77.0)
    lse = torch.full((140, HEADS), 55.0, device=DEV)
    cu = ints(list(2 + np.cumsum([0] + q)))
    fw.fp4_kv_attention(x, cu, ints(kv), table, cache, one(S_K), one(S_V), 70, 0.125, True,
                        out=out, lse=lse)
    assert (out[:2] == 77).all() and (out[133:] == 77).all()
    assert (lse[:2] == 55).all() and (lse[133:] == 55).all()
    ref = _kv4.attention(x, cu, torch.tensor(kv), table, cache, S_K, S_V, 0.125, True)
    check(out, lse, ref, 4.0, max(kv))


@pytest.mark.parametrize("where", ["k", "v"])
@pytest.mark.parametrize("n", [200, 3000])
def test_nan_reaches_the_rows_that_see_it_and_no_others(where, n):
    rows, at = 100, n - 50
    cache, table = filled([n], HEADS, 64, 16, 51)
    x = rand(1, HEADS, 64, seed=52)
    bad = x.clone()
    bad[0, 3, 17] = float("nan")         # of one head
    slot = table[0, at // 16].long().view(1) * 16 + at % 16
    k, v = (bad, x) if where == "k" else (x, bad)
    fw.fp4_kv_append(k, v, slot, cache, one(S_K), one(S_V))
    q = rand(rows, HEADS, 64, seed=53)
    out, lse = fw.fp4_kv_attention(q, ints([0, rows]), ints([n]), table, cache, one(S_K), one(S_V),
                                   rows, 0.125, True, return_lse=True)
    sees = torch.zeros(rows, HEADS, dtype=torch.bool, device=DEV)
    sees[rows - 50:, 3] = True           # row i sees at <= n - rows + i
    assert torch.isnan(out[sees]).all() and torch.isnan(lse[sees]).all()
    assert torch.isfinite(out[~sees]).all() and torch.isfinite(lse[~sees]).all()


@pytest.mark.parametrize("n", [90, 3000])
def test_every_seen_score_a_nan(n):
    """Sums that are NaN where no score was ever a number, joined over splits."""
    cache, table = filled([n], HEADS, 64, 16, 55)
    slots = table[0].repeat_interleave(16)[:n].long() * 16 + torch.arange(n, device=DEV) % 16
    x = rand(n, HEADS, 64, seed=56)
    bad = x.clone()
    bad[:, 2] = float("nan")
    fw.fp4_kv_append(bad, x, slots, cache, one(S_K), one(S_V))
    q = rand(60, HEADS, 64, seed=57)
    out = fw.fp4_kv_attention(q, ints([0, 60]), ints([n]), table, cache, one(S_K), one(S_V), 60)
    assert torch.isnan(out[:, 2]).all()
    assert torch.isfinite(out[:, [0, 1, 3, 4, 5]]).all()


@pytest.mark.parametrize("n", [90, 3000])
def test_nan_and_infinite_queries(n):
    cache, table = filled([n], HEADS, 64, 16, 61)
    q = rand(64, 2 * HEADS, 64, seed=62)
    q[0, 1, 3] = float("nan")
    q[0, 2, 3] = float("inf")
    out = fw.fp4_kv_attention(q, ints([0, 64]), ints([n]), table, cache, one(S_K), one(S_V), 64)
    assert torch.isnan(out[0, 1:3]).all()
    keep = torch.ones(64, 2 * HEADS, dtype=torch.bool)
    keep[0, 1:3] = False
    assert torch.isfinite(out[keep.to(DEV)]).all()


@pytest.mark.parametrize("dim", [64, 128])
def test_same_bits_again_whatever_the_workspace_held(dim):
    cache, table = filled([5000, 33, 900], HEADS, dim, 64, 81, extra_width=300)
    q = rand(133, HEADS, dim, seed=82)
    args = (q, ints([0, 60, 61, 133]), ints([5000, 33, 900]), table, cache, one(S_K), one(S_V), 72)
    ws = torch.full((fw.fp4_kv_attention_workspace(),), 0xFF, dtype=torch.uint8, device=DEV)
    a, la = fw.fp4_kv_attention(*args, return_lse=True, workspace=ws)
    b, lb = fw.fp4_kv_attention(*args, return_lse=True, workspace=ws)
    c = fw.fp4_kv_attention(*args)
    assert torch.equal(a, b) and torch.equal(la, lb) and torch.equal(a, c)
    check(a, la, _kv4.attention(q, args[1], torch.tensor([5000, 33, 900]), table, cache, S_K, S_V,
                                dim ** -0.5, True), 4.0, 5000)


def test_prompts_beside_many_single_tokens():
    kv = [(i * 61) % 500 + 1 for i in range(200)]
    q = [1 if i % 9 else 45 + i for i in range(200)]
    attend(q, [max(a, b) for a, b in zip(kv, q)], 2, 2, 64, 16, True)
