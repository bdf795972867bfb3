"""Which stream the router's scratch memory and the outputs are allocated
for, on a stand-in for torch's streams and allocator.  No GPU."""

import contextlib
import types

import pytest
import torch


@pytest.fixture(scope="module")
def ep():
    from conftest import load_build_module

    load_build_module().build()
    import combine_get_layout_gb300 as ep

    return ep


class Streams:
    """The current stream, those under capture, and every allocation (stream,
    bytes, tensor)."""

    def __init__(self, monkeypatch):
        self.current, self.capturing, self.made = self.stream(1), set(), []
        empty = torch.empty

        def make(shape, dtype=None, device=None):
            t = empty(shape, dtype=dtype, device="cpu")
            self.made.append((self.current.cuda_stream, t.nbytes, t))
            return t

        @contextlib.contextmanager
        def under(stream):
            was, self.current = self.current, stream
            yield
            self.current = was

        monkeypatch.setattr(torch, "empty", make)
        monkeypatch.setattr(torch.cuda, "stream", under)
        monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: self.current)
        monkeypatch.setattr(torch.cuda, "is_current_stream_capturing",
                            lambda: self.current.cuda_stream in self.capturing)
        monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream",
                            lambda dev: self.current.cuda_stream, raising=False)
        monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)

    @staticmethod
    def stream(handle):
        return types.SimpleNamespace(cuda_stream=handle)


@pytest.fixture
def streams(monkeypatch, ep):
    monkeypatch.setattr(ep, "_workspaces", {})
    return Streams(monkeypatch)


class Logits:
    is_cuda, shape, device = True, (8, 16), torch.device("cuda", 0)

    def get_device(self):
        return 0


def balance(ep, monkeypatch, stream, B=1, experts=16):
    """The scratch memory that one call hands to the library."""
    used = []
    monkeypatch.setattr(ep, "_calls", types.SimpleNamespace(
        route_balance=lambda *a: used.append((a[11], a[12], a[13])) or 0))
    seq = None if B == 1 else types.SimpleNamespace(shape=(B + 1,))
    ep.route_balance(ep.RouterConfig(experts, 2), Logits(), seq_start=seq, out=(None,) * 6,
                     stream=stream)
    (memory, size, handle), = used
    used.clear()
    assert memory.nbytes >= size and handle == (None if stream is None else stream.cuda_stream)
    return memory


def made_for(streams, memory):
    return next(s for s, _, t in streams.made if t is memory)


def test_scratch_memory_is_made_for_the_stream_that_uses_it(ep, streams, monkeypatch):
    s = streams.stream(2)
    assert made_for(streams, balance(ep, monkeypatch, None)) == 1
    mine = balance(ep, monkeypatch, s)
    assert made_for(streams, mine) == 2 and streams.current.cuda_stream == 1
    assert balance(ep, monkeypatch, s) is mine                  # kept
    streams.current = s
    assert balance(ep, monkeypatch, None) is mine               # the same stream
    assert balance(ep, monkeypatch, streams.stream(1)) is not mine


def test_a_capturing_stream_gets_memory_that_its_graph_owns(ep, streams, monkeypatch):
    s = streams.stream(2)
    kept = balance(ep, monkeypatch, s), balance(ep, monkeypatch, None)
    streams.capturing = {2}                     # the given stream alone
    a, b = balance(ep, monkeypatch, s), balance(ep, monkeypatch, s)
    assert a is not b and all(t is not k for t in (a, b) for k in kept)
    assert made_for(streams, a) == made_for(streams, b) == 2
    streams.capturing = {1, 2}                  # and the current one, which it joined
    c = balance(ep, monkeypatch, s)
    assert all(c is not k for k in (a, b, *kept)) and made_for(streams, c) == 2
    streams.capturing = {1}                     # the given one is not part of it
    assert balance(ep, monkeypatch, s) is kept[0]


def test_kept_memory_is_bounded_and_what_is_outgrown_is_released(ep, streams, monkeypatch):
    import gc
    import weakref

    small = balance(ep, monkeypatch, None)
    ref, size = weakref.ref(small), small.nbytes
    del small
    large = balance(ep, monkeypatch, None, B=4000, experts=512)
    assert large.nbytes > size
    streams.made.clear()
    gc.collect()
    assert ref() is None                        # the larger block took its place
    assert balance(ep, monkeypatch, None) is large
    refs = []
    for handle in range(100, 400):
        refs.append(weakref.ref(balance(ep, monkeypatch, streams.stream(handle))))
        streams.made.clear()
    gc.collect()
    alive = sum(r() is not None for r in refs)
    assert 16 <= alive <= 64 and refs[-1]() is not None


def test_the_table_turns_over_while_other_threads_use_it(ep, streams, monkeypatch):
    import itertools
    import threading

    number, said = itertools.count(), []
    monkeypatch.setattr(ep, "_get_ident", lambda: next(number))

    def work():
        try:
            for _ in range(2000):
                assert ep._workspace_of(Logits(), None, 100).nbytes >= 100
                streams.made.clear()
        except Exception as e:
            said.append(repr(e))

    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not said, said[0]
    assert len(ep._workspaces) <= 64


class Fake:
    """A CUDA tensor as far as the Python layer looks at one."""

    is_cuda, device = True, torch.device("cuda", 0)

    def __init__(self, shape, dtype):
        self.shape, self.dtype = torch.Size(shape), dtype

    def is_contiguous(self):
        return True

    def get_device(self):
        return 0

    def data_ptr(self):
        return 0x10000


def calls_that_allocate(ep):
    router, w4 = ep.RouterConfig(16, 2), ep.W4Config(2, 128, 64, has_zeros=True)
    x, rows = Fake((8, 16), torch.float32), Fake((4, 128), torch.bfloat16)
    codes, scales = Fake((2, 64, 64), torch.uint8), Fake((2, 64, 1), torch.bfloat16)
    zeros = Fake((2, 64, 1), torch.uint8)
    return {
        "route": (2, lambda s: ep.route(router, x, stream=s)),
        "route_balance": (6, lambda s: ep.route_balance(router, x, workspace=x, stream=s)),
        "route_backward": (1, lambda s: (ep.route_backward(router, x, stream=s),)),
        "expert_w4": (1, lambda s: (ep.expert_w4(w4, rows, *[None] * 4, 4, stream=s),)),
        "w4_pack": (3, lambda s: ep.w4_pack(w4, codes, scales, zeros, stream=s)),
    }


@pytest.mark.parametrize("name", ["route", "route_balance", "route_backward", "expert_w4",
                                  "w4_pack"])
def test_outputs_are_made_for_the_stream_that_writes_them(ep, streams, monkeypatch, name):
    """And recorded on the current one, on which the caller goes on."""
    recorded = []
    monkeypatch.setattr(torch.Tensor, "record_stream",
                        lambda t, s: recorded.append((t, s.cuda_stream)), raising=False)
    monkeypatch.setattr(ep, "_calls", types.SimpleNamespace(**{
        n: lambda *a: 0 for n in ("route", "route_balance", "route_backward", "expert_w4")}))
    monkeypatch.setattr(ep, "ep_w4_pack", lambda *a: 0)
    many, call = calls_that_allocate(ep)[name]
    for stream, made_on in ((streams.stream(2), 2), (streams.stream(1), 1), (None, 1)):
        streams.made.clear()
        recorded.clear()
        out = call(stream)
        assert len(out) == many and [s for s, _, _ in streams.made] == [made_on] * many
        assert all(any(t is o for _, _, t in streams.made) for o in out)
        marks = [(t, s) for t, s in recorded]
        assert len(marks) == (many if made_on == 2 else 0) and all(s == 1 for _, s in marks)
        assert streams.current.cuda_stream == 1
