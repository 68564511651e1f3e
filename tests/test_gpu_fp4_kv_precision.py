"""How exact attention over the 4-bit cache is where many small weights make up
the output: one dominant token whose V is 0 before a long uniform tail, and long
contexts whose every 64 tokens show in some element of the output.

Tolerances.  The weights are FP16 values of 2^(s - m + 9) (log2 units, m a running
maximum no larger than the row's): half a step is 2^-11 of a weight from 2^-14 on,
2^-25 below, which is 2^-34 of the largest weight (m at the maximum; less of it while
m is behind).  With o the exact output, A = sum_j p_j |v_j| and Z = sum_j exp(s_j -
max s), the output is off by at most
  2^-8 |o|                  the output's rounding to BF16 (half a step)
  (2^-11 + 2^-13) A         half a step of each weight, and the fp32 errors of
                            scores (|s| <= 2^6 in log2 units here, each product
                            exact: 2^-17 of the weight), exponentials and sums
  n 2^-34 max|v| / Z        n weights below the normal range
lse is fp32: 2^-19 of reach + |lse| + 1, reach = max_j sum |q k|."""

import pytest
import torch

import fp8_w8a8_static_b200 as fw
import _kv4
from test_gpu_fp4_kv import DEV, S_K, S_V, ints, one, rand

pytestmark = pytest.mark.gpu
PAGE = 64
# rows of the request, query heads of the K/V head: the few-rows kernel with 8, 16
# and many rows, the many-rows kernel (whose blocks share the tokens)
FORMS = [(1, 3), (6, 2), (300, 1), (1200, 1)]


def stored(k, v):
    """Cache and table with these tokens, and their exact values."""
    n, heads, dim = k.shape
    pages = -(-n // PAGE)
    cache = fw.fp4_kv_cache(pages, heads, PAGE, dim, DEV)
    fw.fp4_kv_append(k, v, torch.arange(n, device=DEV), cache, one(S_K), one(S_V))
    kc, vc, ks, vs = _kv4.regions(cache)
    s_k, s_v = (float(one(s)) for s in (S_K, S_V))
    value = [_kv4.values(c, z, s).transpose(0, 1).reshape(heads, -1, dim)[:, :n]
             for c, z, s in ((kc, ks, s_k), (vc, vs, s_v))]
    return cache, ints([list(range(pages))]), value


def formula(q, k, v, scale):
    """(o, lse, A, Z, reach) in 64 bits of every row over every token."""
    g = q.shape[1] // k.shape[0]
    out = []
    for r in range(q.shape[1]):
        z = q[:, r].double() @ k[r // g].t() * scale
        top = z.amax(1, keepdim=True)
        w = torch.exp(z - top)
        total = w.sum(1, keepdim=True)
        p = w / total
        out.append((p @ v[r // g], (top + total.log())[:, 0], p @ v[r // g].abs(), total,
                    (q[:, r].double().abs() @ k[r // g].abs().t() * abs(scale)).amax(1)))
    return [torch.stack(x, 1) for x in zip(*out)]


def bound(o, a, z, v, n):
    return 2.0 ** -8 * o.abs() + (2.0 ** -11 + 2.0 ** -13) * a + n * 2.0 ** -34 * v.abs().max() / z


def check(q, cache, table, kv, n, scale):
    k, v = kv
    out, lse = fw.fp4_kv_attention(q, ints([0, len(q)]), ints([n]), table, cache, one(S_K), one(S_V),
                                   len(q), scale, False, return_lse=True)
    o, want_lse, a, z, reach = formula(q, k, v, scale)
    d = (out.double() - o).abs()
    lim = bound(o, a, z, v, n)
    assert (d <= lim).all(), (d / lim).max()
    d = (lse.double() - want_lse).abs()
    assert (d <= 2.0 ** -19 * (reach + want_lse.abs() + 1)).all()
    return o, a, z


@pytest.mark.parametrize("gap", [10.0, 15.0, 16.3, 17.4, 20.0])
@pytest.mark.parametrize("at", [0, -1])
@pytest.mark.parametrize("rows,group", FORMS)
@pytest.mark.parametrize("dim,n", [(64, 131072), (128, 20011)])
def test_a_dominant_token_without_value(rows, group, at, gap, dim, n):
    """The output is the tail alone, `gap` below the dominant token in the exponent;
    found first, or last, when the tail's sums have to be scaled down."""
    heads = 2
    k = torch.zeros(n, heads, dim, device=DEV)
    k[at, :, 5] = 1.0
    v = (1 + 0.2 * torch.randn(n, heads, dim, generator=torch.Generator().manual_seed(int(gap)))).to(DEV)
    v[at] = 0
    cache, table, kv = stored(k.bfloat16(), v.bfloat16())
    q = torch.zeros(rows, heads * group, dim, device=DEV)
    q[:, :, 5] = 1.0
    scale = gap / kv[0][0, at, 5].item()
    scale = torch.tensor(scale, dtype=torch.float32).item()
    o, _, _ = check(q.bfloat16(), cache, table, kv, n, scale)
    assert (o > 0).all()


@pytest.mark.parametrize("rows,group", FORMS)
@pytest.mark.parametrize("dim,n", [(128, 4096), (128, 20000), (128, 65537), (64, 65537)])
def test_every_chunk_of_a_long_context_counts(rows, group, dim, n):
    """Element d of V is nonzero for the d-th run of the tokens alone, so 64 tokens
    are a good part of some element: the bound tells every 64 tokens that are lost."""
    heads = 2
    t = torch.arange(n, device=DEV)
    v = rand(n, heads, dim, seed=n).abs() + 0.5
    v = v * (t[:, None, None] * dim // n == torch.arange(dim, device=DEV))
    k = rand(n, heads, dim, seed=n + 1)
    cache, table, kv = stored(k, v.to(torch.bfloat16))
    q = rand(rows, heads * group, dim, seed=n + 2, scale=0.5)
    scale = torch.tensor(dim ** -0.5, dtype=torch.float32).item()
    o, a, z = check(q, cache, table, kv, n, scale)
    lim = bound(o, a, z, kv[1], n)
    chunks = -(-n // 64)
    for r in range(heads * group):            # of the first row: what each chunk gives
        w = torch.softmax(q[0, r].double() @ kv[0][r // group].t() * scale, 0)
        part = w[:, None] * kv[1][r // group]
        part = torch.nn.functional.pad(part, (0, 0, 0, chunks * 64 - n)).view(chunks, 64, dim).sum(1)
        lost = (part > lim[0, r]).any(1)
        assert lost[:n // 64].all()


@pytest.mark.parametrize("rows,group", FORMS)
@pytest.mark.parametrize("dim", [64, 128])
def test_small_query_elements_are_exact_down_to_2_17_of_the_largest(dim, rows, group):
    """K is 0 where q's largest element is, so the scores are the small element's
    products alone: every significand of it at 2^-17 shows in lse."""
    n, heads = 700, 2
    k = torch.zeros(n, heads, dim, device=DEV)
    k[:, :, 5] = 1 + torch.arange(n, device=DEV)[:, None] % 7
    cache, table, kv = stored(k.bfloat16(), rand(n, heads, dim, seed=4))
    q = torch.zeros(rows, heads * group, dim, device=DEV)
    q[:, :, 40] = 1.0
    mantissa = torch.arange(rows * heads * group, device=DEV).view(rows, -1) * 37 % 128
    q[:, :, 5] = 2.0 ** -17 * (1 + mantissa / 128)
    check(q.bfloat16(), cache, table, kv, n, 2.0 ** 16)


def test_what_fp16_holds_of_a_small_query_element():
    """On its row's scale every BF16 significand is an FP16 value at 2^-17; at 2^-18
    half of them are not, by half a step of 2^-24."""
    x = 1 + torch.arange(128, dtype=torch.float64) / 128
    assert torch.equal((x * 2.0 ** -17).half().double(), x * 2.0 ** -17)
    off = ((x * 2.0 ** -18).half().double() - x * 2.0 ** -18).abs()
    assert (off > 0).sum() == 64 and off.max() == 2.0 ** -25


@pytest.mark.parametrize("n_free,used,wanted", [(4, 9, 3), (0, 5, 3), (4, 4, 3), (4, 2, 3)])
def test_pool_when_more_is_used_than_there_is(n_free, used, wanted):
    """pool = (used + taken, missing): where more is used than there are pages,
    nothing is taken and used stays."""
    free = torch.arange(100, 100 + n_free, dtype=torch.int32, device=DEV)
    table = torch.full((2, 4), -1, dtype=torch.int32, device=DEV)
    _, _, _, pool = fw.fp4_kv_tables(ints([0, 16]), ints([20, 1]), table, free, ints([used]), 16, 21)
    taken = min(wanted, max(n_free - used, 0))
    assert pool.tolist() == [used + taken, wanted - taken]
    got = table[table >= 0].tolist()
    assert got == list(range(100 + used, 100 + used + taken))
