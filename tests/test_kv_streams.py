"""Where the binding takes a call's work buffer from when it is given none (on the CPU, with the
allocator and the streams replaced)."""
import contextlib

import pytest
import torch


@pytest.fixture(scope="module")
def e():
    from lossless_entropy_coded_gb300 import build
    build.build()
    from lossless_entropy_coded_gb300 import _ec
    return _ec


@pytest.fixture()
def taken(monkeypatch):
    """The streams that were current at each allocation of bytes."""
    current, seen, empty = ["current"], [], torch.empty

    class External:
        def __init__(self, ptr, device=None):
            self.cuda_stream = ptr

    @contextlib.contextmanager
    def on(s):
        current.append(s.cuda_stream)
        yield
        current.pop()

    def alloc(*a, **kw):
        if kw.get("dtype") == torch.uint8:
            seen.append(current[-1])
        return empty(*a, **kw)

    monkeypatch.setattr(torch.cuda, "ExternalStream", External)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch, "empty", alloc)
    return seen


class Seqs:
    n, packed, pages, device, lens = 2, bytes(32), 3, -1, torch.zeros(2)


class Handle:  # as other libraries pass streams
    cuda_stream = 4096


@pytest.mark.parametrize("stream,at", [(4096, 4096), (Handle(), 4096)])
def test_a_buffer_belongs_to_the_launch_stream(e, taken, monkeypatch, stream, at):
    cache = e.kv_cache(1, 4, 2, 64, 16, device=-1)
    x, refs = torch.zeros((2, 2, 64)), torch.zeros(4, dtype=torch.int32)
    monkeypatch.setattr(e, "gemm_work_bytes", lambda *a: 64)
    monkeypatch.setattr(e, "gemm_group_work_bytes", lambda *a: 64)
    W = e.Matrix(0, 4, 4, 0, -1)
    calls = [lambda s: e.kv_attend(cache, 0, Seqs, x, x.clone(), stream=s), lambda s: e.kv_fork(cache, Seqs, refs, Seqs, refs.clone(), stream=s),
             lambda s: e.kv_compact(cache, Seqs, refs, Seqs, refs.clone(), stream=s), lambda s: e.gemm(W, x, x, 1, stream=s)]
    for call in calls:
        taken.clear()
        with pytest.raises(e.EcError):  # no device: each call is refused after its buffer was taken
            call(stream)
        assert taken == [at]
    taken.clear()
    with pytest.raises(Exception):
        e.gemm_group([W], [x], [x], 1, stream=stream)
    assert taken == [at]
    taken.clear()
    with pytest.raises(e.EcError):
        e.kv_attend(cache, 0, Seqs, x, x.clone())
    assert taken == ["current"]
