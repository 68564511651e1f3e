"""The attention block as a decoder runs it: tables, shared-quant Q/K/V, the
store into the 4-bit cache, attention with FP8 output at o_proj's input scale,
o_proj onto the residual stream -- prompts first, then single tokens, the steps
captured in a CUDA graph and replayed.  And the calls' streams and empty forms.

The chain is checked against the formulas in 64 bits on the library's own q, k,
v and cache bytes (the projections and the store have tests of their own), so
what remains is the attention's and o_proj's error.  An FP8 code is off by at
most half a step, 2^-4 of its value, 3.6% (2^-4 / sqrt 3) in the root of the
mean square; the codes' errors are independent, so the product over 256 of them
is off by 3.6% of its norm, and the attention's own 2^-10 and BF16's 2^-8 are
within the rest of 4%."""

import pytest
import torch

import fp8_w8a8_static_b200 as fw
import _kv4

pytestmark = pytest.mark.gpu
DEV = "cuda"
HEADS, GROUP, DIM, PAGE, D = 2, 2, 64, 16, 256


def one(x):
    return torch.tensor([x], dtype=torch.float32, device=DEV)


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


class Block:
    """One decoder layer's attention block with its cache."""

    def __init__(self, seed):
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        self.g = g
        rn = lambda *s: (torch.randn(*s, generator=g, device=DEV) * 0.06).bfloat16()  # noqa: E731
        self.w = {n: fw.fp8_rtn_quantize_weight(rn(o, D)) for n, o in
                  (("q", HEADS * GROUP * DIM), ("k", HEADS * DIM), ("v", HEADS * DIM), ("o", D))}
        self.s_in, self.s_o = one(4.0 / 448), one(2.0 / 448)
        self.s_k, self.s_v = one(0.004), one(0.004)
        self.cache = fw.fp4_kv_cache(40, HEADS, PAGE, DIM, DEV)
        self.cache.fill_(0xFF)
        self.free = torch.randperm(40, generator=torch.Generator().manual_seed(seed)).int().to(DEV)
        self.lens, self.pool = ints([0, 0, 0]), ints([0, 0])
        self.table = torch.full((3, 9), -1, dtype=torch.int32, device=DEV)

    def step(self, x, added, n_slots, max_q):
        """x [n_slots, D] -> the block's output, and what it was made from."""
        cu = torch.empty(4, dtype=torch.int32, device=DEV)
        slots = torch.empty(n_slots, dtype=torch.int64, device=DEV)
        fw.fp4_kv_tables(self.lens, added, self.table, self.free, self.pool, PAGE, n_slots,
                         out=(cu, self.lens, slots, self.pool))
        q, k, v = fw.qkv_shared_quant(x, self.s_in, *self.w["q"], *self.w["k"], *self.w["v"])
        fw.fp4_kv_append(k, v, slots, self.cache, self.s_k, self.s_v)
        q = q.view(n_slots, HEADS * GROUP, DIM)
        a = torch.zeros(q.shape, dtype=fw.FP8, device=DEV)
        fw.fp4_kv_attention(q, cu, self.lens, self.table, self.cache, self.s_k, self.s_v, max_q,
                            s_out=self.s_o, out=a)
        y = fw.fp8_linear_epilogue(a.view(n_slots, -1), self.w["o"][0], self.s_o, self.w["o"][1],
                                   residual=x)
        return y, q, cu

    def check(self, x, y, q, cu, rows):
        """The formulas on the library's q and cache bytes."""
        o, _, _, _ = _kv4.attention(q, cu, self.lens.cpu(), self.table, self.cache,
                                    float(self.s_k), float(self.s_v), DIM ** -0.5, True)
        w = self.w["o"][0].double() * self.w["o"][1].double()
        want = o[:rows].reshape(rows, -1) @ w.t()
        got = y[:rows].double() - x[:rows].double()
        # (the sum with the residual rounds to BF16: half a step of the sum)
        err = (got - want).norm() - (y[:rows].double() * 2.0 ** -8).norm()
        assert err <= 0.04 * want.norm(), (err / want.norm())


def test_prompts_then_tokens():
    b = Block(1)
    rows = [70, 5, 33]
    x = torch.randn(sum(rows) + 4, D, generator=b.g, device=DEV).bfloat16()  # a padded batch
    y, q, cu = b.step(x, ints(rows), len(x), 70)
    assert b.lens.tolist() == rows and b.pool.tolist() == [5 + 1 + 3, 0]
    b.check(x, y, q, cu, sum(rows))
    # a decode step, captured once and replayed, its lengths and pages advancing in place
    x1 = torch.randn(3, D, generator=b.g, device=DEV).bfloat16()
    ones = ints([1, 1, 1])
    state = [t.clone() for t in (b.lens, b.pool, b.table, b.cache)]
    b.step(x1, ones, 3, 1)  # first use of the shapes outside the capture
    for t, s in zip((b.lens, b.pool, b.table, b.cache), state):
        t.copy_(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y1, q1, cu1 = b.step(x1, ones, 3, 1)
    for n in range(1, 21):
        x1.copy_(torch.randn(3, D, generator=b.g, device=DEV))
        g.replay()
        assert b.lens.tolist() == [r + n for r in rows]
        b.check(x1, y1, q1, cu1, 3)
    assert b.pool[1] == 0
    used = b.pool[0].item()
    assert used == sum(-(-(r + 20) // PAGE) for r in rows)
    pages = b.table[b.table >= 0].tolist()
    assert len(pages) == len(set(pages)) == used


@pytest.mark.parametrize("q_len", [1, 50])
def test_on_other_streams_at_once(q_len):
    """Two calls on two streams, neither the current one, workspaces left to the
    binding, which allocates them on the current stream."""
    made = []
    for seed in (3, 4):
        b = Block(seed)
        x = torch.randn(3 * q_len, D, generator=b.g, device=DEV).bfloat16()
        _, q, cu = b.step(x, ints([q_len] * 3), 3 * q_len, q_len)
        args = (q, cu, b.lens, b.table, b.cache, b.s_k, b.s_v, q_len)
        made.append((args, fw.fp4_kv_attention(*args)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        outs = []
        for (args, _), s in zip(made, streams):
            for _ in range(8):
                out = torch.empty_like(args[0])
                s.wait_stream(torch.cuda.current_stream())
                fw.fp4_kv_attention(*args, out=out, stream=s)
                torch.empty(1 << 20, device=DEV).fill_(1.0)  # may take a workspace's memory
                outs.append(out)
        torch.cuda.synchronize()
        for i, out in enumerate(outs):
            assert torch.equal(out, made[i // 8][1])


def test_raw_stream_handle():
    b = Block(6)
    x = torch.randn(3, D, generator=b.g, device=DEV).bfloat16()
    y, q, cu = b.step(x, ints([1, 1, 1]), 3, 1)
    want = fw.fp4_kv_attention(q, cu, b.lens, b.table, b.cache, b.s_k, b.s_v, 1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = fw.fp4_kv_attention(q, cu, b.lens, b.table, b.cache, b.s_k, b.s_v, 1, stream=s.cuda_stream)
    s.synchronize()
    assert torch.equal(got, want)


def test_two_graphs_share_a_workspace():
    b = Block(7)
    x = torch.randn(120, D, generator=b.g, device=DEV).bfloat16()
    _, q, cu = b.step(x, ints([40, 40, 40]), 120, 40)
    ws = torch.empty(fw.fp4_kv_attention_workspace(), dtype=torch.uint8, device=DEV)
    few = (q[:3].contiguous(), ints([0, 1, 2, 3]), b.lens, b.table, b.cache, b.s_k, b.s_v, 1)
    many = (q, cu, b.lens, b.table, b.cache, b.s_k, b.s_v, 40)
    wants = [fw.fp4_kv_attention(*a) for a in (few, many)]
    graphs, outs = [], []
    for a in (few, many):
        out = torch.empty_like(a[0])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            fw.fp4_kv_attention(*a, out=out, workspace=ws)
        graphs.append(g)
        outs.append(out)
    for _ in range(3):
        for o in outs:
            o.fill_(float("nan"))
        graphs[0].replay()
        graphs[1].replay()
        graphs[0].replay()
        assert torch.equal(outs[0], wants[0]) and torch.equal(outs[1], wants[1])


def test_empty_calls():
    n0 = fw.launch_count()
    e16 = torch.empty(0, 2, 64, dtype=torch.bfloat16, device=DEV)
    none = torch.empty(0, dtype=torch.int64, device=DEV)
    cache = fw.fp4_kv_cache(0, 2, 16, 64, DEV)
    fw.fp4_kv_append(e16, e16, none, cache, one(1.0), one(1.0))
    k, v = fw.fp4_kv_gather(cache, none, one(1.0), one(1.0))
    assert k.shape == (0, 2, 64) and v.shape == (0, 2, 64)
    q = torch.empty(0, 4, 64, dtype=torch.bfloat16, device=DEV)
    out = fw.fp4_kv_attention(q, ints([0]), ints([]), ints([]).view(0, 3), cache, one(1.0), one(1.0), 0)
    assert out.shape == q.shape
    w = torch.zeros(32, 64, device=DEV).to(fw.FP8)
    y = fw.fp8_linear_epilogue(torch.empty(0, 64, device=DEV).to(fw.FP8), w, one(1.0), one(1.0))
    assert y.shape == (0, 32)
    assert fw.launch_count() == n0
    # a cache without pages: every slot is outside it, every token unseen
    x = torch.ones(2, 2, 64, dtype=torch.bfloat16, device=DEV)
    slots = torch.tensor([0, 5], device=DEV)
    fw.fp4_kv_append(x, x, slots, cache, one(1.0), one(1.0))
    k, v = fw.fp4_kv_gather(cache, slots, one(1.0), one(1.0))
    assert (k == 0).all() and (v == 0).all()
    for n in (1, 60):
        q = torch.ones(n, 4, 64, dtype=torch.bfloat16, device=DEV)
        out, lse = fw.fp4_kv_attention(q, ints([0, n]), ints([30]), ints([[0, 1]]), cache, one(1.0),
                                       one(1.0), n, return_lse=True)
        assert (out == 0).all() and torch.isinf(lse).all()


def test_device_status_is_clean():
    torch.cuda.synchronize()
    assert fw.device_status() == (0, 0)
