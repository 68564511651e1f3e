"""The 4-bit K/V cache on the GPU: tables, append, gather and attention against
plain implementations in 64 bits, at the lengths, masks, pages and orders where
they can go wrong.

Tolerances.  With o the exact output and A = sum_j p_j |v_j|, the kernel's
output is off by at most
  2^-8 |o|                 the output's rounding to BF16 (half a step)
  (2^-11 + 2^-13) A        the weights' rounding to FP16, half a step each, and
                           the fp32 errors of scores, exponentials and sums
                           (scores: 2^-21 of sum |q k| <= 2^9 here)
  n 2^-24 max|v|           weights below FP16's normal range, n tokens
An FP8 output instead of the first term: half a step of E4M3, 2^-4 of the value
or 2^-10 for the subnormal codes.  lse is fp32: 2^-19 of reach + |lse| + 1, reach
= max_j sum |q k| (the products are exact; the sum of D of them and the
logarithm round)."""

import numpy as np
import pytest
import torch

import fp8_w8a8_static_b200 as fw
import _kv4

pytestmark = pytest.mark.gpu
DEV = "cuda"
S_K, S_V = 0.0071, 0.0019


def one(x, dtype=torch.float32):
    return torch.tensor([x], dtype=dtype, device=DEV)


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def rand(*shape, seed, scale=1.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return (torch.randn(*shape, generator=g, device=DEV) * scale).to(torch.bfloat16)


def check(out, lse, ref, v_max, tokens, s_out=None):
    o, want_lse, spread, reach = ref
    live = ~torch.isnan(o[..., 0])
    got = out.double() if s_out is None else out.float().double() * s_out
    err = (2.0 ** -11 + 2.0 ** -13) * spread + tokens * 2.0 ** -24 * v_max
    if s_out is None:
        err = err + 2.0 ** -8 * o.abs()
    else:
        err = err + torch.maximum(2.0 ** -4 * o.abs(), torch.full_like(o, 2.0 ** -10 * s_out))
        o = o.clamp(-448 * s_out, 448 * s_out)
    d = (got - o).abs()
    assert torch.isfinite(got[live]).all()
    assert (d[live] <= err[live]).all(), (d[live] - err[live]).max()
    if lse is not None:
        inf = torch.isinf(want_lse)
        assert torch.equal(torch.isinf(lse) & live, inf & live)
        assert (lse[inf & live] < 0).all()
        fin = live & ~inf
        d = (lse.double() - want_lse).abs()[fin]
        lim = (2.0 ** -19 * (reach + want_lse.abs() + 1))[fin]
        assert (d <= lim).all(), (d / lim).max()


def filled(kv_lens, heads, dim, page, seed, spare=2, extra_width=1):
    """A cache with the requests' tokens in shuffled pages, the rest of every
    page bytes of 0xFF (NaN scales); their table."""
    need = [-(-max(n, 0) // page) for n in kv_lens]
    total = sum(need)
    rng = np.random.default_rng(seed)
    order = rng.permutation(total + spare)
    table = np.full((len(kv_lens), max(need + [0]) + extra_width), -1, dtype=np.int32)
    at = 0
    slots = []
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
        t = np.arange(max(kv_lens[b], 0))
        slots.append(table[b, t // page].astype(np.int64) * page + t % page)
    cache = fw.fp4_kv_cache(total + spare, heads, page, dim, DEV)
    cache.fill_(0xFF)
    slots = torch.from_numpy(np.concatenate(slots) if slots else np.zeros(0, np.int64)).to(DEV)
    k, v = rand(len(slots), heads, dim, seed=seed + 1), rand(len(slots), heads, dim, seed=seed + 2)
    if len(slots):
        k[:, :, dim // 2] *= 5
        fw.fp4_kv_append(k, v, slots, cache, one(S_K), one(S_V))
    return cache, torch.from_numpy(table).to(DEV)


def attend(q_lens, kv_lens, heads, group, dim, page, causal, seed=0, s_out=None, scale=None,
           max_q=None):
    cache, table = filled(kv_lens, heads, dim, page, seed)
    q = rand(sum(q_lens), heads * group, dim, seed=seed + 3, scale=1.5)
    cu = ints([0] + list(np.cumsum(q_lens)))
    scale = dim ** -0.5 if scale is None else scale
    out, lse = fw.fp4_kv_attention(q, cu, ints(kv_lens), table, cache, one(S_K), one(S_V),
                                   max(q_lens) if max_q is None else max_q, scale, causal,
                                   s_out=None if s_out is None else one(s_out), return_lse=True)
    ref = _kv4.attention(q, cu, torch.tensor(kv_lens), table, cache, S_K, S_V, scale, causal)
    check(out, lse, ref, 4.0, max(kv_lens + [1]), s_out)
    return out


# ------------------------------------------------------------------ the store


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_append_bytes_are_the_definitions(dim, page):
    heads, T = 3, 77
    k, v = rand(T, heads, dim, seed=1), rand(T, heads, dim, seed=2, scale=0.2)
    k[3] = 0                                   # scale 0
    k[4, :, :16] *= 1e-4                       # a scale below E4M3's normal range
    k[5, :, 16:32] *= 3e38                     # the largest scale; an infinity saturates
    v[6, 0, 5] = float("inf")
    v[7, :, ::2] = -0.0
    k[8, :, 0], k[8, :, 1] = 6.0, 2.5          # ties of the code
    pages = -(-T // page) + 2
    cache = fw.fp4_kv_cache(pages, heads, page, dim, DEV)
    cache.fill_(0xEE)
    slots = torch.randperm(pages * page)[:T]
    fw.fp4_kv_append(k, v, slots.to(DEV), cache, one(S_K), one(S_V))
    kc, vc, ks, vs = (x.cpu().numpy() for x in _kv4.regions(cache.cpu()))
    seen = np.zeros((pages, page // 16, 16), bool)
    for x, s, code, scale in ((k, S_K, kc, ks), (v, S_V, vc, vs)):
        want_c, want_s = _kv4.quantize(x.float().cpu().numpy(), s)
        packed = want_c[..., 0::2] | want_c[..., 1::2] << 4
        for t, slot in enumerate(slots.tolist()):
            p, r, w = slot // page, slot % page // 16, slot % 16
            assert np.array_equal(code[p, :, r, w], packed[t]), t
            assert np.array_equal(scale[p, :, r, w], want_s[t]), t
            seen[p, r, w] = True
    for a in (kc, vc, ks, vs):                 # every other byte is as it was
        assert (np.moveaxis(a, 1, 3)[~seen] == 0xEE).all()


@pytest.mark.parametrize("s", [1.0, 2.0 ** -9, 3.3e-7, 1e-38, 1e30])
def test_append_at_other_scales(s):
    k, v = rand(64, 1, 128, seed=5, scale=min(s * 900, 1e30)), rand(64, 1, 128, seed=6)
    cache = fw.fp4_kv_cache(1, 1, 64, 128, DEV)
    fw.fp4_kv_append(k, v, torch.arange(64, device=DEV), cache, one(s), one(s))
    kc, vc, ks, vs = (x.cpu().numpy() for x in _kv4.regions(cache.cpu()))
    for x, code, scale in ((k, kc, ks), (v, vc, vs)):
        c, z = _kv4.quantize(x.float().cpu().numpy()[:, 0], np.float32(s))
        assert np.array_equal(code[0, 0].reshape(64, -1), c[..., 0::2] | c[..., 1::2] << 4)
        assert np.array_equal(scale[0, 0].reshape(64, -1), z)


def test_every_tie_and_neighbour_of_the_codes():
    """x = the midpoints of neighbouring codes times a power-of-two scale, and
    the BF16 values beside them."""
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.bfloat16)
    up = (mids.view(torch.int16) + 1).view(torch.bfloat16)
    down = (mids.view(torch.int16) - 1).view(torch.bfloat16)
    row = torch.cat([mids, up[:8], torch.tensor([6.0, -6.0]).bfloat16()])
    k = torch.zeros(2, 1, 64, dtype=torch.bfloat16)
    k[0, 0, :16], k[0, 0, 16:32] = row, -row
    k[1, 0, :9] = torch.cat([down, torch.tensor([6.0, 0.0]).bfloat16()])
    cache = fw.fp4_kv_cache(1, 1, 16, 64, DEV)
    fw.fp4_kv_append(k.to(DEV), k.to(DEV), torch.arange(2, device=DEV), cache, one(1.0), one(1.0))
    c, z = _kv4.quantize(k.float().numpy()[:, 0], 1.0)
    kc, _, ks, _ = (x.cpu().numpy() for x in _kv4.regions(cache.cpu()))
    assert np.array_equal(kc[0, 0, 0, :2], c[..., 0::2] | c[..., 1::2] << 4)
    assert np.array_equal(ks[0, 0, 0, :2], z)


@pytest.mark.parametrize("dim", [64, 128])
def test_gather_reads_back(dim):
    T, heads, page = 1003, 2, 32
    cache, table = filled([T], heads, dim, page, 11)
    t = torch.arange(T, device=DEV)
    slots = table[0, t // page].long() * page + t % page
    slots = torch.cat([slots.flip(0), slots[:5], torch.tensor([-1, cache.shape[0] * page, -2 ** 40], device=DEV)])
    k, v = fw.fp4_kv_gather(cache, slots, one(S_K), one(S_V))
    kc, vc, ks, vs = _kv4.regions(cache)
    ok = slots[:-3]
    p, r, w = ok // page, ok % page // 16, ok % 16
    for got, code, scale, s in ((k, kc, ks, S_K), (v, vc, vs, S_V)):
        want = _kv4.values(code[p, :, r, w], scale[p, :, r, w], np.float32(s))
        # two roundings: to fp32 (2^-24) and to BF16 (2^-8)
        assert ((got[:-3].double() - want).abs() <= want.abs() * (2.0 ** -8 + 2.0 ** -23)).all()
        assert (got[-3:] == 0).all()


def test_append_skips_slots_outside():
    cache = fw.fp4_kv_cache(2, 1, 16, 64, DEV)
    cache.fill_(0x55)
    x = rand(5, 1, 64, seed=1)
    slots = torch.tensor([-1, 32, 2 ** 40, -2 ** 62, 31], device=DEV)
    fw.fp4_kv_append(x, x, slots, cache, one(1.0), one(1.0))
    raw = cache.cpu().numpy()
    assert (raw[0] == 0x55).all() and (raw[1] != 0x55).sum() <= 64 + 8
    k, _ = fw.fp4_kv_gather(cache, slots[-1:], one(1.0), one(1.0))
    assert (k - x[-1]).abs().max() <= x[-1].abs().max() / 6 + 1e-3


# ----------------------------------------------------------------- attention


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("group", [1, 3, 8, 16])
@pytest.mark.parametrize("page", [16, 64, 256])
def test_single_tokens(dim, group, page):
    lens = [1, 2, 15, 16, 17, 31, 63, 64, 65, 127, 128, 129, 255, 257, 500, 1023]
    attend([1] * len(lens), lens, 2, group, dim, page, True)


@pytest.mark.parametrize("kv", [1, 64, 1001, 4096, 20000, 65537])
@pytest.mark.parametrize("group", [1, 3, 8])
def test_one_request(kv, group):
    """One request spread over the whole GPU, its parts merged."""
    attend([1], [kv], 2, group, 128, 64, True, seed=kv)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("group", [1, 3, 5])
def test_ragged_rows(dim, causal, group):
    q = [1, 2, 0, 7, 33, 1, 130]
    kv = [5, 2, 40, 64, 200, 1000, 131]
    attend(q, kv, 2, group, dim, 16, causal)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("q_len,kv", [(16, 16), (127, 127), (128, 128), (129, 300), (300, 129),
                                      (257, 1000), (512, 4000)])
@pytest.mark.parametrize("dim,group", [(128, 3), (64, 2), (128, 1), (64, 8)])
def test_prompts(q_len, kv, causal, dim, group):
    """Chunks of prompts; more rows than tokens leave causal rows empty."""
    attend([q_len], [kv], 2, group, dim, 64, causal, seed=q_len)


@pytest.mark.parametrize("q_len", [39, 40, 41, 128, 129, 256, 257])
@pytest.mark.parametrize("batch", [1, 3])
def test_rows_where_the_kernel_changes(q_len, batch):
    """The borders in rows between the two kernels and between row tiles; one
    request's row blocks share the GPU by splits of its tokens."""
    attend([q_len] * batch, [1500 - 700 * b for b in range(batch)], 1, 1, 128, 32, True, seed=q_len)


@pytest.mark.parametrize("kv", [63, 64, 65, 600, 20000])
@pytest.mark.parametrize("dim", [64, 128])
def test_splits_of_the_tokens(kv, dim):
    """Five row blocks in all: the splits' ranges end anywhere, some are empty."""
    attend([1270], [kv], 1, 1, dim, 64, False, seed=kv)


def test_more_rows_than_the_table_has_requests_for():
    """max_q above every request's rows (a captured graph's bound)."""
    attend([3, 1, 50], [90, 7, 50], 2, 2, 64, 16, True, max_q=4096)
    attend([3], [90], 2, 2, 64, 16, True, max_q=4096)


@pytest.mark.parametrize("q_len", [1, 40])
def test_rows_without_tokens(q_len):
    q = [q_len, q_len, q_len]
    out = attend(q, [0, 3, 0], 1, 3, 64, 16, True)
    assert (out[:q_len] == 0).all() and (out[2 * q_len:] == 0).all()


@pytest.mark.parametrize("s_out", [0.004, 1e-3])
@pytest.mark.parametrize("q", [[1, 1], [1, 50]])
def test_fp8_output(s_out, q):
    attend(q, [700, 80], 2, 3, 128, 32, True, s_out=s_out)


@pytest.mark.parametrize("q_len", [1, 70])
@pytest.mark.parametrize("scale", [0.0, -0.1, 2.0])
def test_other_scales(q_len, scale):
    """Uniform weights, a negative scale, and weights that one token dominates
    (the running maximum moves far, again and again)."""
    attend([q_len], [777], 1, 2, 128, 64, True, scale=scale)


@pytest.mark.parametrize("q_len", [1, 64])
def test_rising_scores(q_len):
    """Scores that rise along the context by far more than the slack of the
    running maximum, and rows of very different magnitudes."""
    n, dim = 600, 64
    cache, table = filled([n], 1, dim, 16, 3)
    k = torch.zeros(n, 1, dim)
    k[:, 0, 0] = torch.arange(n) * 0.1
    k[:, 0, 1:] = torch.randn(n, dim - 1) * 0.1
    slots = table[0].repeat_interleave(16)[:n].long() * 16 + torch.arange(n, device=DEV) % 16
    v = rand(n, 1, dim, seed=8)
    fw.fp4_kv_append(k.bfloat16().to(DEV), v, slots, cache, one(S_K), one(S_V))
    q = rand(q_len, 2, dim, seed=9)
    q[:, :, 0] = 3.0
    q[:, 1] *= 1e-3
    if q_len > 1:
        q[1::2] *= 2.0 ** 20
        q[2::4] *= 2.0 ** -60
    cu = ints([0, q_len])
    sc = 2.0 ** -20 if q_len > 1 else 1.0
    out, lse = fw.fp4_kv_attention(q, cu, ints([n]), table, cache, one(S_K), one(S_V), q_len, sc,
                                   True, return_lse=True)
    check(out, lse, _kv4.attention(q, cu, torch.tensor([n]), table, cache, S_K, S_V, sc, True),
          6.0, n)


@pytest.mark.parametrize("rows", [1, 20])
def test_pages_that_the_cache_lacks(rows):
    kv = [100, 100, 333]
    cache, table = filled(kv, 2, 64, 16, 21)
    table[0, 2] = -1
    table[0, 0] = cache.shape[0]
    table[1, :] = -7                     # nothing left: rows without tokens
    table[2, 5:9] = 2 ** 31 - 1
    q = rand(3 * rows, 6, 64, seed=22)
    cu = ints([0, rows, 2 * rows, 3 * rows])
    out, lse = fw.fp4_kv_attention(q, cu, ints(kv), table, cache, one(S_K), one(S_V), rows, 0.125,
                                   True, return_lse=True)
    ref = _kv4.attention(q, cu, torch.tensor(kv), table, cache, S_K, S_V, 0.125, True)
    check(out, lse, ref, 4.0, 333)
    assert (out[rows:2 * rows] == 0).all()


@pytest.mark.parametrize("rows", [1, 30])
def test_lengths_beyond_the_table_and_offsets_beyond_the_rows(rows):
    """Lengths past the table row's capacity count as the capacity, offsets
    past total_q as total_q, negative ones as 0."""
    cache, table = filled([64, 64], 1, 64, 16, 31, extra_width=0)
    q = rand(2 * rows, 2, 64, seed=32)
    cu = ints([-5, rows, 2 * rows + 1000])
    lens = [10 ** 9, 64]
    out = torch.zeros_like(q)
    got, lse = fw.fp4_kv_attention(q, cu, ints(lens), table, cache, one(S_K), one(S_V), rows, 0.1,
                                   True, out=out, return_lse=True)
    check(got, lse, _kv4.attention(q, cu, torch.tensor(lens), table, cache, S_K, S_V, 0.1, True),
          4.0, 64)


@pytest.mark.parametrize("q", [[1, 1, 1], [3, 40, 1]])
def test_rows_outside_every_request_stay(q):
    kv = [50, 100, 7]
    cache, table = filled(kv, 2, 64, 32, 41)
    n = sum(q)
    x = rand(n + 9, 4, 64, seed=42)
    out = torch.full_like(x, 77.0)
    lse = torch.full((n + 9, 4), 55.0, device=DEV)
    cu = ints(list(2 + np.cumsum([0] + q)))
    fw.fp4_kv_attention(x, cu, ints(kv), table, cache, one(S_K), one(S_V), max(q), 0.125, True,
                        out=out, lse=lse)
    assert (out[:2] == 77).all() and (out[n + 2:] == 77).all()
    assert (lse[:2] == 55).all() and (lse[n + 2:] == 55).all()
    ref = _kv4.attention(x, cu, torch.tensor(kv), table, cache, S_K, S_V, 0.125, True)
    check(out, lse, ref, 4.0, 100)


@pytest.mark.parametrize("where", ["k", "v"])
def test_nan_reaches_the_rows_that_see_it_and_no_others(where):
    n, rows = 200, 100
    cache, table = filled([n], 1, 64, 16, 51)
    x = rand(1, 1, 64, seed=52)
    bad = x.clone()
    bad[0, 0, 17] = float("nan")
    at = 150                       # seen by row i where at <= n - rows + i
    slot = table[0, at // 16].long().view(1) * 16 + at % 16
    k, v = (bad, x) if where == "k" else (x, bad)
    fw.fp4_kv_append(k, v, slot, cache, one(S_K), one(S_V))
    for lo, cnt in ((0, rows), (90, 10), (0, 1)):
        q = rand(cnt, 3, 64, seed=53)
        cu = ints([0, cnt])
        kv = n - rows + lo + cnt
        out, lse = fw.fp4_kv_attention(q, cu, ints([kv]), table, cache, one(S_K), one(S_V), cnt,
                                       0.125, True, return_lse=True)
        sees = torch.arange(cnt) + kv - cnt >= at
        assert torch.isnan(out[sees.to(DEV)]).all() and torch.isnan(lse[sees.to(DEV)]).all()
        assert torch.isfinite(out[~sees.to(DEV)]).all()
        assert torch.isfinite(lse[~sees.to(DEV)]).all()


@pytest.mark.parametrize("q_len", [1, 20])
def test_nan_and_infinite_queries(q_len):
    cache, table = filled([90], 1, 64, 16, 61)
    q = rand(q_len, 4, 64, seed=62)
    q[0, 1, 3] = float("nan")
    q[0, 2, 3] = float("inf")
    out = fw.fp4_kv_attention(q, ints([0, q_len]), ints([90]), table, cache, one(S_K), one(S_V), q_len)
    assert torch.isnan(out[0, 1:3]).all()
    keep = torch.ones(q_len, 4, dtype=torch.bool)
    keep[0, 1:3] = False
    assert torch.isfinite(out[keep.to(DEV)]).all()


def test_offsets_past_32_bits():
    """Pages of a cache of over 4 GiB, the first and the last."""
    heads, dim, page = 8, 128, 64
    per = heads * page // 16 * 18 * dim
    pages = (2 ** 32 + 2 ** 30) // per
    cache = torch.empty(pages, heads, page // 16, 18 * dim, dtype=torch.uint8, device=DEV)
    kv, rows = [130, 130], [1, 40]
    table = ints([[pages - 1, 0, pages - 2], [1, pages - 3, pages // 2]])
    t = torch.arange(130, device=DEV)
    slots = torch.cat([table[b, t // page].long() * page + t % page for b in (0, 1)])
    k, v = rand(260, heads, dim, seed=71), rand(260, heads, dim, seed=72)
    fw.fp4_kv_append(k, v, slots, cache, one(S_K), one(S_V))
    k2, _ = fw.fp4_kv_gather(cache, slots, one(S_K), one(S_V))
    assert (k2 - k).abs().max() <= k.abs().max() / 6 + 0.1
    q = rand(41, 8 * 3, dim, seed=73)
    cu = ints([0, 1, 41])
    for m in (1, 40):
        cuq = ints([0, 1, 2]) if m == 1 else cu
        out, lse = fw.fp4_kv_attention(q, cuq, ints(kv), table, cache, one(S_K), one(S_V), m, 0.1,
                                       True, return_lse=True)
        ref = _kv4.attention(q, cuq, torch.tensor(kv), table, cache, S_K, S_V, 0.1, True)
        check(out, lse, ref, 4.0, 130)


def test_many_requests():
    """More requests than a block's threads, most of them short."""
    kv = [(i * 37) % 90 for i in range(700)]
    q = [1 if i % 5 else i % 3 for i in range(700)]
    attend(q, kv, 1, 2, 64, 16, True, max_q=2)


def test_same_bits_again_whatever_the_workspace_held():
    cache, table = filled([5000, 33, 900], 2, 128, 64, 81)
    q = rand(3, 6, 128, seed=82)
    args = (q, ints([0, 1, 2, 3]), ints([5000, 33, 900]), table, cache, one(S_K), one(S_V), 1)
    ws = torch.full((fw.fp4_kv_attention_workspace(),), 0xFF, dtype=torch.uint8, device=DEV)
    a, la = fw.fp4_kv_attention(*args, return_lse=True, workspace=ws)
    b, lb = fw.fp4_kv_attention(*args, return_lse=True, workspace=ws)
    c = fw.fp4_kv_attention(*args)
    assert torch.equal(a, b) and torch.equal(la, lb) and torch.equal(a, c)


# -------------------------------------------------------------------- tables


def plain_tables(lens, new, table, free, used, page, n_slots):
    table = table.copy()
    W = table.shape[1]
    cu, kv, slots = [0], [], [-1] * n_slots
    taken = missing = 0
    for b, (o, a) in enumerate(zip(lens, new)):
        o, a = max(o, 0), max(a, 0)
        for j in range(min(-(-o // page), W), min(-(-(o + a) // page), W)):
            i = used + taken + missing
            table[b, j] = free[i] if i < len(free) else -1
            if i < len(free):
                taken += 1
            else:
                missing += 1
        for i in range(a):
            t, pos = cu[-1] + i, o + i
            if t < n_slots and pos // page < W and table[b, pos // page] >= 0:
                slots[t] = int(table[b, pos // page]) * page + pos % page
        cu.append(cu[-1] + a)
        kv.append(o + a)
    return cu, kv, slots, [used + taken, missing], table


@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("batch,max_len,max_new,pad", [
    (1, 0, 1, 0), (1, 1000, 1, 3), (7, 100, 1, 0), (33, 300, 40, 100), (512, 50, 2, 0),
    (513, 50, 3, 7), (1500, 20, 5, 1), (3, 0, 3000, 50)])
def test_tables(page, batch, max_len, max_new, pad):
    rng = np.random.default_rng(batch + page)
    lens = rng.integers(0, max_len + 1, batch)
    new = rng.integers(0, max_new + 1, batch)
    if batch > 2:
        lens[1], new[2] = -4, -9
    W = -(-(max_len + max_new) // page) + 1
    table = rng.integers(0, 9999, (batch, W)).astype(np.int32)
    free = rng.permutation(100000)[:batch * W + 5].astype(np.int32)
    n_slots = int(np.maximum(new, 0).sum()) + pad
    want = plain_tables(lens, new, table, free, 3, page, n_slots)
    t = ints(table.tolist())
    cu, kv, slots, pool = fw.fp4_kv_tables(ints(lens.tolist()), ints(new.tolist()), t,
                                           ints(free.tolist()), ints([3]), page, n_slots)
    assert cu.tolist() == want[0] and kv.tolist() == want[1]
    assert slots.tolist() == want[2] and pool.tolist() == want[3]
    assert np.array_equal(t.cpu().numpy(), want[4])


@pytest.mark.parametrize("n_free,used,width,n_slots", [(4, 0, 9, 60), (4, 2, 9, 60), (0, 0, 9, 60),
                                                       (4, 9, 9, 60), (50, 0, 2, 60), (50, 0, 9, 11),
                                                       (50, 0, 9, 0)])
def test_tables_short_of_pages_rows_or_slots(n_free, used, width, n_slots):
    lens, new, page = [16, 30, 0, 5], [17, 3, 20, 0], 16
    table = np.full((4, width), 77, np.int32)
    free = np.arange(100, 100 + n_free).astype(np.int32)
    want = plain_tables(lens, new, table, free, min(used, n_free) if used > n_free else used, page, n_slots)
    t = ints(table.tolist())
    out = fw.fp4_kv_tables(ints(lens), ints(new), t, torch.tensor(free, device=DEV), ints([used]), page, n_slots)
    assert out[0].tolist() == want[0] and out[1].tolist() == want[1] and out[2].tolist() == want[2]
    assert np.array_equal(t.cpu().numpy(), want[4])
    if used <= n_free:
        assert out[3].tolist() == want[3]


def test_tables_advance_in_place():
    """Lengths and pool in place over several steps, captured in a graph."""
    page, B = 16, 5
    lens, pool = ints([0, 15, 16, 33, 7]), ints([0, 0])
    table = ints([[i * 100 + j if j * page < [0, 15, 16, 33, 7][i] else -1 for j in range(20)] for i in range(B)])
    added, free = ints([1, 1, 2, 0, 30]), ints(list(range(1000, 1100)))
    cu, slots = torch.empty(B + 1, dtype=torch.int32, device=DEV), torch.empty(40, dtype=torch.int64, device=DEV)
    h_lens, h_table, used = lens.tolist(), table.cpu().numpy(), 0
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fw.fp4_kv_tables(lens, added, table, free, pool, page, 40, out=(cu, lens, slots, pool))
    for _ in range(6):
        g.replay()
        w = plain_tables(h_lens, added.tolist(), h_table, free.tolist(), used, page, 40)
        h_lens, h_table, used = w[1], w[4], w[3][0]
        assert lens.tolist() == h_lens and slots.tolist() == w[2] and pool.tolist() == w[3]
        assert np.array_equal(table.cpu().numpy(), h_table)


def test_tables_empty_batch():
    e = torch.empty(0, dtype=torch.int32, device=DEV)
    cu, kv, slots, pool = fw.fp4_kv_tables(e, e, e.view(0, 4), ints([1, 2]), ints([1]), 16, 5)
    assert cu.tolist() == [0] and slots.tolist() == [-1] * 5 and pool.tolist() == [1, 0]
