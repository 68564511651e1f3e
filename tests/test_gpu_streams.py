"""Calls on a stream that is not the current one, their workspaces and results
left to the binding, with no wait between the two streams but for the inputs."""

import pytest
import torch

import fp8_w8a8_static_b200 as fw
from test_gpu_fp4_kv import DEV, S_K, S_V, filled, ints, one, rand

pytestmark = pytest.mark.gpu
LONG = 4_000_000  # cycles, about 2 ms


def attention_args(q_len, kv, seed):
    cache, table = filled([kv], 2, 128, 64, seed)
    return (rand(q_len, 6, 128, seed=seed), ints([0, q_len]), ints([kv]), table, cache, one(S_K),
            one(S_V), q_len)


def linear_args(seed, m=300):
    x, w = (rand(*s, seed=seed + i).to(fw.FP8) for i, s in enumerate(((m, 256), (512, 256))))
    return x, w, one(0.01), one(0.02)


def mlp_args(seed):
    w = [(rand(*s, seed=seed + i, scale=0.1).to(fw.FP8), one(0.01))
         for i, s in enumerate(((256, 128), (256, 128), (128, 256)))]
    (g, sg), (u, su), (d, sd) = w
    return rand(64, 128, seed=seed + 9), one(0.01), g, sg, u, su, one(0.01), d, sd


CALLS = {
    "attention, one row": lambda: (fw.fp4_kv_attention, attention_args(1, 20000, 3)),
    "attention, rows": lambda: (fw.fp4_kv_attention, attention_args(300, 3000, 5)),
    "epilogue": lambda: (fw.fp8_linear_epilogue, linear_args(7)),
    "linear": lambda: (fw.fp8_linear_static, linear_args(8)),
    "mlp": lambda: (fw.gated_mlp_static_fp8, mlp_args(9)),
}


def made(name):
    """A call, its inputs, and its result alone."""
    fn, a = CALLS[name]()
    want = fn(*a)
    torch.cuda.synchronize()
    return fn, a, want


@pytest.mark.parametrize("name", sorted(CALLS))
def test_result_is_not_memory_that_the_current_stream_still_uses(name):
    fn, a, want = made(name)
    s = torch.cuda.Stream()
    for _ in range(3):
        held = torch.zeros_like(want)
        torch.cuda._sleep(LONG)
        held.fill_(7.0)                     # queued, not run yet
        at = held.data_ptr()
        del held
        out = fn(*a, stream=s)
        assert out.data_ptr() != at
        s.synchronize()
        assert torch.equal(out, want)
        torch.cuda.synchronize()
        assert torch.equal(out, want)


@pytest.mark.parametrize("name", sorted(CALLS))
def test_result_is_kept_for_the_current_streams_reader(name):
    fn, a, want = made(name)
    s = torch.cuda.Stream()
    fn(*a, stream=s)
    out = fn(*a, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda._sleep(LONG)
    copy = out.clone()
    at = out.data_ptr()
    del out
    again = [fn(*a, stream=s) for _ in range(3)]
    assert at not in [o.data_ptr() for o in again]
    torch.cuda.synchronize()
    assert torch.equal(copy, want) and all(torch.equal(o, want) for o in again)


@pytest.mark.parametrize("q_len,kv", [(1, 60000), (300, 6000)])
def test_calls_of_two_streams_have_a_workspace_each(q_len, kv):
    """One call on the current stream and one on another that waits for the
    inputs alone, over many rounds, both with partial sums in their workspaces."""
    jobs = []
    for seed in (11, 13):
        a = attention_args(q_len, kv, seed)
        jobs.append((a, fw.fp4_kv_attention(*a, return_lse=True)))
    s = torch.cuda.Stream()
    ready = torch.cuda.Event()
    ready.record()
    s.wait_event(ready)
    for _ in range(20):
        torch.cuda._sleep(LONG // 40)
        outs = []
        for _ in range(10):
            outs.append((fw.fp4_kv_attention(*jobs[0][0], return_lse=True), 0))
            outs.append((fw.fp4_kv_attention(*jobs[1][0], return_lse=True, stream=s), 1))
        torch.cuda.synchronize()
        for (o, lse), i in outs:
            assert torch.equal(o, jobs[i][1][0]) and torch.equal(lse, jobs[i][1][1])


@pytest.mark.parametrize("handle", [0, 1, None])
def test_raw_handles(handle):
    """The legacy default stream's two handles, and another stream's."""
    fn, a, want = made("attention, one row")
    s = torch.cuda.Stream()
    out = fn(*a, stream=s.cuda_stream if handle is None else handle)
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    fn, a, want = made("mlp")
    out = fn(*a, stream=s.cuda_stream if handle is None else handle)
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_captured_on_a_side_stream():
    """A capture that forks: the calls of the side stream allocate in the graph's pool."""
    fn, a, want = made("attention, one row")
    lin, b, want_lin = made("linear")
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.wait_stream(torch.cuda.current_stream())
        out = fn(*a, stream=s)
        y = lin(*b)
        torch.cuda.current_stream().wait_stream(s)
    for _ in range(3):
        out.zero_()
        y.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(y, want_lin)
