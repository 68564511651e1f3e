"""What a call allocates belongs to the stream it runs on, read from the
binding's own source (no GPU): memory of the current stream may still be in use
by work that another stream is not ordered behind."""

import ast
import inspect

import pytest

import fp8_w8a8_static_b200 as fw

HELPERS = {"_empty", "_new", "_workspace"}
FACTORIES = {"empty", "zeros", "ones", "full", "empty_like", "zeros_like", "new_empty",
             "new_zeros", "new_full", "contiguous", "clone"}


def functions():
    tree = ast.parse(inspect.getsource(fw))
    return {f.name: f for f in tree.body if isinstance(f, ast.FunctionDef)
            and "stream" in [a.arg for a in f.args.args + f.args.kwonlyargs]}


def calls(f):
    return [c for c in ast.walk(f) if isinstance(c, ast.Call)]


CALLS = sorted(n for n in functions() if not n.startswith("_"))


def test_every_call_is_looked_at():
    assert len(CALLS) >= 25 and "fp4_kv_attention" in CALLS and "gated_mlp_static_fp8" in CALLS


@pytest.mark.parametrize("name", CALLS)
def test_call_allocates_on_its_stream(name):
    for c in calls(functions()[name]):
        if isinstance(c.func, ast.Attribute):
            assert c.func.attr not in FACTORIES, ast.unparse(c)
        elif isinstance(c.func, ast.Name) and c.func.id in HELPERS:
            assert ast.unparse(c.args[-1]) == "stream", ast.unparse(c)


@pytest.mark.parametrize("name", sorted(HELPERS))
def test_helpers_take_the_stream(name):
    assert functions()[name].args.args[-1].arg == "stream"
