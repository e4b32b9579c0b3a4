"""Where a call on another stream than the current one takes the memory of a result that it
allocates itself.  CPU only: the streams are stand-ins that note what is allocated on them."""
import contextlib

import pytest
import torch

import paged_varlen_flash_gb300 as ua
from tests.test_step_checks import BLOCKS, B, D, HK, HQ, N, T, WIDTH, i32, p  # noqa: F401
from tests.test_binding_checks import _built, reaches_the_library  # noqa: F401


class OnGpu(torch.Tensor):
    is_cuda = True
    notes = []

    def record_stream(self, stream):
        OnGpu.notes.append(("kept for", stream.cuda_stream))

    @classmethod
    def __torch_function__(cls, func, types, args=(), kwargs=None):
        if func is torch.empty_like:
            OnGpu.notes.append(("memory of", Stream.current))
        return super().__torch_function__(func, types, args, kwargs)


class Stream:
    current = 7

    def __init__(self, raw, device=None):
        self.cuda_stream = raw


@pytest.fixture(autouse=True)
def streams(monkeypatch):
    @contextlib.contextmanager
    def on(stream):
        before, Stream.current = Stream.current, stream.cuda_stream
        yield
        Stream.current = before

    monkeypatch.setattr(torch.cuda, "ExternalStream", Stream)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Stream(Stream.current))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: Stream(0))
    OnGpu.notes.clear()


def bf(*s):
    return torch.zeros(*s, dtype=torch.bfloat16)


def calls(p):
    q, cache = bf(T, HQ, D).as_subclass(OnGpu), bf(BLOCKS, B, HK, D)
    rest = cache, cache, i32(N, WIDTH), i32(N + 1), i32(N), N, T, 5, 50
    return dict(
        forward=lambda **kw: p.forward(q, *rest, ua.UA_FLAG_CAUSAL, **kw),
        topk=lambda **kw: p.forward_topk(q, *rest, i32(T, 8), i32(T), ua.UA_FLAG_CAUSAL, **kw),
        weights=lambda **kw: p.forward_weights(q, *rest, ua.UA_FLAG_CAUSAL, None, torch.zeros(N, HK, 50), **kw),
        tree=lambda **kw: p.forward_tree(q, *rest, ua.UA_FLAG_CAUSAL, i32(T, 1), **kw),
        rope=lambda **kw: p.rope_store(q, bf(T, HK, D), bf(T, HK, D), i32(T), torch.zeros(T, dtype=torch.int64), T, cache,
                                       cache, **kw))


@pytest.mark.parametrize("name", ["forward", "topk", "weights", "tree", "rope"])
def test_results_are_memory_of_the_stream_that_writes_them(p, name):  # noqa: F811
    call = calls(p)[name]
    for stream, raw in ((11, 11), (Stream(11), 11), (0, 0)):
        OnGpu.notes.clear()
        reaches_the_library(call, stream=stream)
        assert OnGpu.notes == [("memory of", raw), ("kept for", 7)], (stream, OnGpu.notes)
    for stream in (7, Stream(7)):
        OnGpu.notes.clear()
        reaches_the_library(call, stream=stream)
        assert OnGpu.notes == [("memory of", 7)]
