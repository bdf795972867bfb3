"""Router and product configs as values: copied, pickled and sent to another
process, a config stands for its own memory.  No GPU."""

import copy
import ctypes
import dataclasses
import gc
import os
import pickle
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ep():
    from conftest import load_build_module

    load_build_module().build()
    import combine_get_layout_gb300 as ep

    return ep


def make(ep, kind):
    if kind == "router":
        return ep.RouterConfig(256, 8, "sigmoid", 8, 4, True, 2.5)
    return ep.W4Config(60, 256, 130, 64, True, True, True)


def fields_of(c):
    """The numbers of a config's ABI struct (of a router's second, for bf16)."""
    one = c.c(True) if hasattr(c, "num_topk") else c.c()
    return [getattr(one, name) for name, _ in one._fields_]


def holds_its_own(c):
    return c._at == ctypes.addressof(c._c)


@pytest.mark.parametrize("kind", ["router", "w4"])
@pytest.mark.parametrize("how", [copy.copy, copy.deepcopy, lambda c: copy.deepcopy([c, {1: c}])[0],
                                 lambda c: dataclasses.replace(c),
                                 *(lambda c, p=p: pickle.loads(pickle.dumps(c, p))
                                   for p in range(pickle.HIGHEST_PROTOCOL + 1))])
def test_a_copy_has_its_own_struct(ep, kind, how):
    c = make(ep, kind)
    d, want, text = how(c), fields_of(c), repr(c)
    assert d == c and type(d) is type(c) and hash(d) == hash(c)
    assert holds_its_own(c) and holds_its_own(d)
    del c
    gc.collect()
    assert fields_of(d) == want and repr(d) == text
    size = ctypes.sizeof(type(d.c()))
    at = d._at + (size if kind == "router" else 0)
    assert ctypes.string_at(at, size) == bytes(d.c(True) if kind == "router" else d.c())


@pytest.mark.parametrize("kind", ["router", "w4"])
def test_another_process_gets_a_struct_of_its_own(ep, kind):
    c = make(ep, kind)
    code = ("import ctypes, pickle, sys; c = pickle.loads(bytes.fromhex(sys.argv[1]));"
            "one = c.c(True) if hasattr(c, 'num_topk') else c.c();"
            "assert c._at == ctypes.addressof(c._c);"
            "print([getattr(one, n) for n, _ in one._fields_])")
    env = dict(os.environ, PYTHONPATH=ROOT + os.pathsep + os.environ.get("PYTHONPATH", ""))
    r = subprocess.run([sys.executable, "-c", code, pickle.dumps(c).hex()], capture_output=True,
                       text=True, env=env, cwd=ROOT, timeout=300)
    assert r.returncode == 0, r.stderr
    assert r.stdout.strip() == str(fields_of(c))


@pytest.mark.parametrize("make_one", [
    lambda ep: ep.RouterConfig(2**32 + 16, 2), lambda ep: ep.RouterConfig(16, 2**32 + 2),
    lambda ep: ep.RouterConfig(16, 2, num_groups=2**32 + 1),
    lambda ep: ep.RouterConfig(16, 2, topk_groups=1 - 2**32),
    lambda ep: ep.W4Config(2**32 + 1, 128, 64), lambda ep: ep.W4Config(1, 2**32 + 128, 64),
    lambda ep: ep.W4Config(1, 128, 2**40 + 64), lambda ep: ep.W4Config(1, 128, 64, 128 - 2**32),
])
def test_numbers_that_a_field_does_not_hold_are_refused(ep, make_one):
    """A field of 32 bits keeps the lower ones of a larger number."""
    with pytest.raises(ep.EpError) as e:
        make_one(ep)
    assert e.value.status == ep.EP_ERR_INVALID_ARG
