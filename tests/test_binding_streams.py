"""Calls that make their own outputs and scratch make them on the stream they launch on:
the zero fill of a workspace is then ordered before the kernels, and the allocator gives
the memory to nobody else while they run.  Checked on the host, with torch's stream
context and allocations watched and the launches replaced."""
import contextlib
from unittest import mock

import pytest
import torch


@pytest.fixture
def bind(host_lib):
    from paged_kv_decode_10_gb300 import binding
    return binding


@pytest.fixture
def watched(bind, monkeypatch):
    """A list of (what, the stream that was current)."""
    now, log = [None], []

    @contextlib.contextmanager
    def stream(s):
        before = now[0]
        now[0] = before if s is None else s
        yield
        now[0] = before

    monkeypatch.setattr(torch.cuda, "stream", stream)
    for name in ("empty", "empty_like", "zeros"):
        real = getattr(torch, name)

        def made(*a, _real=real, _name=name, **kw):
            log.append((_name, now[0]))
            kw.pop("device", None)
            return _real(*a, **kw)
        monkeypatch.setattr(torch, name, made)
    return now, log


def replace(bind, monkeypatch, log, now, *names):
    for name in names:
        def call(*a, _name=name, **kw):
            log.append((_name, now[0]))
        monkeypatch.setattr(bind, name, call)


def check(log, stream, *expected):
    assert {what for what, _ in log} >= set(expected)
    assert all(at is stream for _, at in log), log


@pytest.mark.parametrize("stream", ["side", None])
def test_shared_attention_allocates_on_its_stream(bind, watched, monkeypatch, stream):
    now, log = watched
    replace(bind, monkeypatch, log, now, "make_shared_args", "decode_attn_shared_args")
    q = torch.ones(2, 4, 64)
    log.clear()
    bind.decode_attention_shared(q, None, None, None, None, 1.0, stream=stream)
    check(log, stream, "empty_like", "make_shared_args", "decode_attn_shared_args")


@pytest.mark.parametrize("stream", ["side", None])
def test_eviction_allocates_on_its_stream(bind, watched, monkeypatch, stream):
    now, log = watched
    replace(bind, monkeypatch, log, now, "make_evict_args", "evict_args")
    cache, tables = torch.ones(4, 2, 16, 64), torch.ones(3, 2)
    log.clear()
    bind.evict(cache, cache, None, tables, None, None, 8, stream=stream)
    check(log, stream, "empty", "make_evict_args", "evict_args")


@pytest.mark.parametrize("stream", ["side", None])
def test_rotary_append_allocates_on_its_stream(bind, watched, monkeypatch, stream):
    now, log = watched
    replace(bind, monkeypatch, log, now, "make_rotary_args", "rotary_append_args")
    q = torch.ones(2, 4, 64)
    log.clear()
    bind.rotary_append(None, q, q, None, None, stream=stream)
    check(log, stream, "empty", "make_rotary_args", "rotary_append_args")


@pytest.mark.parametrize("stream", ["side", None])
@pytest.mark.parametrize("name", ["rope", "rope_append"])
def test_rope_allocates_on_its_stream(bind, watched, monkeypatch, stream, name):
    now, log = watched
    monkeypatch.setattr(bind, "load", lambda: mock.MagicMock())
    monkeypatch.setattr(bind, "_check", lambda rc: None)
    for f in ("_stream", "_ptr", "_meta_ptr"):
        monkeypatch.setattr(bind, f, lambda *a: None)
    q, cache = torch.ones(2, 4, 64), torch.ones(4, 4, 16, 64)
    log.clear()
    if name == "rope":
        bind.rope(q, q, None, stream=stream)
    else:
        bind.rope_append(q, q, q, None, None, cache, cache, stream=stream)
    check(log, stream, "empty_like")


@pytest.mark.parametrize("stream", ["side", None])
def test_attention_allocates_on_its_stream(bind, watched, monkeypatch, stream):
    now, log = watched
    replace(bind, monkeypatch, log, now, "alloc_workspace")
    monkeypatch.setattr(bind, "decode_attn_split", lambda *a: None)
    q, cache = torch.ones(2, 4, 64), torch.ones(4, 2, 16, 64)
    log.clear()
    bind.decode_attention(q, cache, cache, None, None, 1.0, num_parts=4, stream=stream)
    check(log, stream, "empty_like", "alloc_workspace")
