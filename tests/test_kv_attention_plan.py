"""Host logic of the attention over the 4-bit cache, on the CPU (no device is
touched): which kernel takes which rows, and how the tokens are split."""

import ctypes

import pytest

import fp8_w8a8_static_b200 as fw

ALL = 2 ** 31 - 1


def plan(rows, heads, tokens, batch=1, dim=128, group=8):
    """`batch` requests of `rows` rows of each of `heads` K/V heads."""
    q = rows // group
    return fw.kv_attention_plan(batch * q, heads * group, heads, dim, batch, q, tokens)


def test_single_tokens_are_the_few_rows_kernels():
    for batch in (1, 48, 300):
        for group in (1, 8, 40):
            p = fw.kv_attention_plan(batch, 8 * group, 8, 128, batch, 1, 100000)
            assert p == dict(few_rows=ALL, blocks=0, splits=1)


# us of the few-rows and of the many-rows kernel, one B200: rows of a request, K/V
# heads, tokens, requests, head_dim
TIMED = [
    (64, 1, 131072, 1, 128, 49, 86), (128, 1, 131072, 1, 128, 61, 88), (512, 1, 131072, 1, 128, 177, 79),
    (1016, 1, 131072, 1, 128, 337, 90), (128, 2, 131072, 1, 128, 98, 67), (128, 4, 131072, 1, 128, 177, 72),
    (256, 4, 131072, 1, 128, 338, 90), (128, 1, 32768, 1, 128, 30, 35), (512, 1, 32768, 1, 128, 55, 43),
    (1016, 1, 32768, 1, 128, 95, 46), (256, 1, 8192, 1, 128, 21, 25), (1016, 1, 8192, 1, 128, 35, 26),
    (1016, 1, 512, 1, 128, 14, 19), (256, 2, 2048, 1, 128, 16, 21), (512, 1, 131072, 2, 128, 337, 105),
    (64, 1, 131072, 2, 128, 61, 69), (256, 4, 512, 1, 128, 14, 19),
    (1016, 1, 131072, 1, 64, 214, 81), (256, 1, 131072, 1, 64, 63, 86), (512, 1, 8192, 1, 64, 18, 22),
    (128, 4, 131072, 1, 64, 113, 64),
]


@pytest.mark.parametrize("rows,heads,tokens,batch,dim,few,many", TIMED)
def test_the_faster_kernel_of_a_handful_of_row_blocks(rows, heads, tokens, batch, dim, few, many):
    assert (plan(rows, heads, tokens, batch, dim)["blocks"] == 0) == (few < many)


def test_more_row_blocks_are_the_many_rows_kernels():
    for tokens in (64, 1000, 100000):
        assert plan(2048, 8, tokens, batch=2)["blocks"] >= 2 * 8 * 8
        assert plan(128, 8, tokens)["blocks"] >= 8


@pytest.mark.parametrize("batch", [1, 2, 5])
@pytest.mark.parametrize("heads", [1, 3, 8])
@pytest.mark.parametrize("rows", [41, 128, 256, 257, 512, 1000, 5000])
@pytest.mark.parametrize("tokens", [1, 600, 20000, 131072])
def test_plans_hold_what_there_is(tokens, rows, heads, batch):
    """No request lacks a kernel or a block, and the partial sums fit 148 places."""
    p = fw.kv_attention_plan(batch * rows, heads, heads, 128, batch, rows, tokens)
    if p["blocks"] == 0:
        assert p["few_rows"] == ALL and p["splits"] == 1
    else:
        assert p["few_rows"] == (0 if batch == 1 else 40)
        assert p["blocks"] >= batch * heads * -(-rows // 256)
        assert p["splits"] == 1 or p["blocks"] * p["splits"] <= 148
        assert 1 <= p["splits"] <= max(1, tokens // 512)


@pytest.mark.parametrize("heads", [1, 3, 8])
@pytest.mark.parametrize("rows", [256, 255, 257, 512, 768, 5000, 5120])
def test_one_request_has_no_block_too_many(rows, heads):
    p = fw.kv_attention_plan(rows, heads, heads, 128, 1, rows, 131072)
    if p["blocks"]:
        assert p["blocks"] == heads * -(-rows // 256)
        assert p["splits"] == max(1, 148 // p["blocks"])


def test_blocks_of_several_requests_are_a_bound_for_any_lengths():
    """Requests of any rows up to max_q with the same sum."""
    for rows in ([256, 256], [300, 300, 40], [41, 41, 41, 41], [1, 1, 1, 700], [512] * 5, [257] * 3):
        p = fw.kv_attention_plan(sum(rows), 8, 8, 128, len(rows), max(rows), 4096)
        assert p["blocks"] >= 8 * sum(-(-r // 256) for r in rows if r > 40)
        assert p["blocks"] < 8 * (sum(rows) / 256 + len(rows))


@pytest.mark.parametrize("max_q", [5, 64, 4096, 2 ** 31, 2 ** 62, 2 ** 63 - 1])
@pytest.mark.parametrize("total_q,batch", [(5, 1), (5, 3), (64, 1), (64, 2)])
def test_a_bound_above_the_rows_that_there_are_counts_as_those(total_q, batch, max_q):
    p = fw.kv_attention_plan(total_q, 32, 8, 128, batch, max_q, 4096)
    assert p == fw.kv_attention_plan(total_q, 32, 8, 128, batch, min(max_q, total_q), 4096)
    if total_q == 5:  # 20 rows of a K/V head
        assert p == dict(few_rows=ALL, blocks=0, splits=1)


def test_refusals():
    ok = dict(total_q=4, q_heads=8, kv_heads=2, head_dim=64, batch=2, max_q=2, tokens=100)
    fw.kv_attention_plan(**ok)
    for bad in (dict(total_q=-1), dict(total_q=2 ** 30), dict(q_heads=7), dict(kv_heads=0), dict(head_dim=96),
                dict(batch=-1), dict(max_q=-1), dict(tokens=-1), dict(tokens=2 ** 31), dict(sms=0)):
        with pytest.raises(fw.FP8WSError) as e:
            fw.kv_attention_plan(**{**ok, **bad})
        assert e.value.status == fw.ERR_SHAPE
    x = ctypes.byref(ctypes.c_int())
    assert fw.load().fp8ws_kv_attention_plan(4, 8, 2, 64, 2, 2, 100, 148, x, None, x) == fw.ERR_NULL
