"""Refusals of the 4-bit cache's calls and of the Linear with a fused epilogue,
without a GPU: the C ABI reports a bad argument before any CUDA call (the
pointers here are fake), the binding before it calls the library."""

import pytest
import torch

import fp8_w8a8_static_b200 as fw
from fp8_w8a8_static_b200 import build as fw_build

A = 1 << 20  # an aligned address, never dereferenced


@pytest.fixture(scope="module")
def lib():
    fw_build.build()
    return fw.load()


def call(fn, defaults, **changes):
    bad = set(changes) - set(defaults)
    assert not bad, bad
    return fn(*{**defaults, **changes}.values())


LINEAR = dict(xq=A, wq=A, M=4, N=32, K=32, s_in=A, s_w=A, bias=A, act=3, residual=A, s_out=A, y=A,
              stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(xq=None), "NULL"), (dict(wq=None), "NULL"), (dict(s_in=None), "NULL"),
    (dict(s_w=None), "NULL"), (dict(y=None), "NULL"), (dict(M=-1), "SHAPE"), (dict(N=4), "SHAPE"),
    (dict(N=24), "SHAPE"),             # FP8 output: N % 16
    (dict(K=40), "SHAPE"), (dict(M=2 ** 31), "SHAPE"), (dict(act=-1), "SHAPE"),
    (dict(act=4), "SHAPE"), (dict(xq=A + 8), "ALIGN"), (dict(wq=A + 8), "ALIGN"),
    (dict(bias=A + 8), "ALIGN"), (dict(residual=A + 2), "ALIGN"), (dict(y=A + 4), "ALIGN")])
def test_linear_epilogue_refuses(lib, change, status):
    n = fw.launch_count()
    assert call(lib.fp8_linear_epilogue, LINEAR, **change) == getattr(fw, "ERR_" + status)
    assert fw.launch_count() == n


TABLES = dict(lens=A, added=A, batch=3, page_size=16, block_table=A, width=4, free=A, n_free=9,
              used=A, pool=A, cu_q=A, kv_lens=A, slots=A, n_slots=5, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(lens=None), "NULL"), (dict(added=None), "NULL"), (dict(block_table=None), "NULL"),
    (dict(free=None), "NULL"), (dict(used=None), "NULL"), (dict(pool=None), "NULL"),
    (dict(cu_q=None), "NULL"), (dict(kv_lens=None), "NULL"), (dict(slots=None), "NULL"),
    (dict(batch=-1), "SHAPE"), (dict(batch=2 ** 31), "SHAPE"), (dict(page_size=24), "SHAPE"),
    (dict(page_size=8), "SHAPE"), (dict(page_size=512), "SHAPE"), (dict(page_size=0), "SHAPE"),
    (dict(page_size=-16), "SHAPE"), (dict(width=-1), "SHAPE"), (dict(n_free=-1), "SHAPE"),
    (dict(n_slots=-1), "SHAPE"), (dict(n_slots=2 ** 31), "SHAPE")])
def test_tables_refuses(lib, change, status):
    assert call(lib.fp4_kv_tables, TABLES, **change) == getattr(fw, "ERR_" + status)


APPEND = dict(k=A, v=A, tokens=3, kv_heads=2, dim=64, slots=A, s_k=A, s_v=A, cache=A, pages=4,
              page_size=16, stream=None)
GATHER = dict(cache=A, pages=4, page_size=16, kv_heads=2, dim=64, slots=A, tokens=3, s_k=A, s_v=A,
              k=A, v=A, stream=None)


@pytest.mark.parametrize("which", ["append", "gather"])
@pytest.mark.parametrize("change,status", [
    (dict(k=None), "NULL"), (dict(v=None), "NULL"), (dict(slots=None), "NULL"),
    (dict(s_k=None), "NULL"), (dict(s_v=None), "NULL"), (dict(cache=None), "NULL"),
    (dict(tokens=-1), "SHAPE"), (dict(tokens=2 ** 31), "SHAPE"), (dict(kv_heads=0), "SHAPE"),
    (dict(kv_heads=65536), "SHAPE"), (dict(dim=96), "SHAPE"), (dict(dim=256), "SHAPE"),
    (dict(page_size=48), "SHAPE"), (dict(pages=-1), "SHAPE"), (dict(k=A + 8), "ALIGN"),
    (dict(v=A + 2), "ALIGN"), (dict(cache=A + 8), "ALIGN")])
def test_append_and_gather_refuse(lib, which, change, status):
    fn, defaults = ((lib.fp4_kv_append, APPEND) if which == "append" else (lib.fp4_kv_gather, GATHER))
    assert call(fn, defaults, **change) == getattr(fw, "ERR_" + status)


def attention_defaults(lib):
    return dict(q=A, total_q=3, q_heads=6, batch=2, cu_q=A, kv_lens=A, max_q=2, table=A, width=4,
                cache=A, pages=4, page_size=16, kv_heads=2, dim=64, s_k=A, s_v=A, scale=0.125,
                causal=1, s_out=None, out=A, lse=None, workspace=A,
                workspace_bytes=lib.fp4_kv_attention_workspace(), stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(q=None), "NULL"), (dict(cu_q=None), "NULL"), (dict(kv_lens=None), "NULL"),
    (dict(table=None), "NULL"), (dict(cache=None), "NULL"), (dict(s_k=None), "NULL"),
    (dict(s_v=None), "NULL"), (dict(out=None), "NULL"), (dict(total_q=-1), "SHAPE"),
    (dict(q_heads=0), "SHAPE"), (dict(q_heads=5), "SHAPE"), (dict(q_heads=65536), "SHAPE"),
    (dict(batch=-1), "SHAPE"), (dict(max_q=-1), "SHAPE"), (dict(width=-1), "SHAPE"),
    (dict(width=2 ** 27), "SHAPE"), (dict(total_q=2 ** 30), "SHAPE"), (dict(page_size=20), "SHAPE"),
    (dict(dim=80), "SHAPE"), (dict(kv_heads=4), "SHAPE"), (dict(scale=float("nan")), "BAD_SCALE"),
    (dict(scale=float("inf")), "BAD_SCALE"), (dict(q=A + 8), "ALIGN"), (dict(out=A + 2), "ALIGN"),
    (dict(cache=A + 8), "ALIGN"), (dict(workspace=None), "WORKSPACE"),
    (dict(workspace=A + 16), "WORKSPACE"), (dict(workspace_bytes=1024), "WORKSPACE")])
def test_attention_refuses(lib, change, status):
    assert call(lib.fp4_kv_attention, attention_defaults(lib), **change) == \
        getattr(fw, "ERR_" + status)


def test_workspace_is_aligned_to_its_regions(lib):
    assert lib.fp4_kv_attention_workspace() % 256 == 0


# the binding, on CPU tensors: it refuses them all, whatever else is right

def t(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


def test_binding_refuses_shapes():
    f8, f32, i32, i64 = torch.float8_e4m3fn, torch.float32, torch.int32, torch.int64
    s = t(1, dtype=f32)
    x, w = t(4, 32).to(f8), t(64, 32).to(f8)
    for bad in (dict(bias=t(32)), dict(residual=t(4, 32)), dict(act="tanh"), dict(out=t(4, 32))):
        with pytest.raises(ValueError):
            fw.fp8_linear_epilogue(x, w, s, s, **bad)
    with pytest.raises(ValueError):
        fw.fp8_linear_epilogue(x, t(64, 48).to(f8), s, s)
    with pytest.raises(ValueError):
        fw.fp4_kv_cache(4, 2, 24, 64, "cpu")
    with pytest.raises(ValueError):
        fw.fp4_kv_cache(4, 2, 16, 96, "cpu")
    cache = fw.fp4_kv_cache(4, 2, 16, 64, "cpu")
    assert tuple(cache.shape) == (4, 2, 1, 1152) and cache.dtype == torch.uint8
    with pytest.raises(ValueError):
        fw.fp4_kv_append(t(3, 2, 128), t(3, 2, 64), t(3, dtype=i64), cache, s, s)
    with pytest.raises(ValueError):
        fw.fp4_kv_append(t(3, 2, 64), t(3, 2, 64), t(2, dtype=i64), cache, s, s)
    with pytest.raises(ValueError):
        fw.fp4_kv_append(t(3, 2, 64), t(3, 2, 64), t(3, dtype=i64), cache[..., :-1], s, s)
    lens = t(3, dtype=i32)
    with pytest.raises(ValueError):
        fw.fp4_kv_tables(lens, t(2, dtype=i32), t(3, 4, dtype=i32), lens, lens, 16, 5)
    with pytest.raises(ValueError):
        fw.fp4_kv_tables(lens, lens, t(2, 4, dtype=i32), lens, lens, 16, 5)
    q = t(3, 4, 64)
    for bad in (dict(q=t(3, 3, 64)), dict(q=t(3, 4, 128)), dict(cu_q=lens), dict(table=t(2, 4, dtype=i32)),
                dict(out=t(3, 4, 32))):
        a = dict(q=q, cu_q=t(4, dtype=i32), table=t(3, 4, dtype=i32), out=None)
        a.update(bad)
        with pytest.raises(ValueError):
            fw.fp4_kv_attention(a["q"], a["cu_q"], lens, a["table"], cache, s, s, 1, out=a["out"])


@pytest.mark.parametrize("name", ["append", "gather", "tables", "attention", "linear"])
def test_binding_refuses_cpu_tensors(name):
    f8, f32, i32, i64 = torch.float8_e4m3fn, torch.float32, torch.int32, torch.int64
    s, lens = t(1, dtype=f32), t(3, dtype=i32)
    cache = fw.fp4_kv_cache(4, 2, 16, 64, "cpu")
    with pytest.raises(ValueError, match="CUDA"):
        if name == "append":
            fw.fp4_kv_append(t(3, 2, 64), t(3, 2, 64), t(3, dtype=i64), cache, s, s)
        elif name == "gather":
            fw.fp4_kv_gather(cache, t(3, dtype=i64), s, s)
        elif name == "tables":
            fw.fp4_kv_tables(lens, lens, t(3, 4, dtype=i32), lens, lens, 16, 5)
        elif name == "attention":
            fw.fp4_kv_attention(t(3, 4, 64), t(4, dtype=i32), lens, t(3, 4, dtype=i32), cache, s, s, 1)
        else:
            fw.fp8_linear_epilogue(t(4, 32).to(f8), t(64, 32).to(f8), s, s)
