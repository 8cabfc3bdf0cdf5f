"""Where the serving calls allocate what they return, and their scratch, when
the work is for another stream than the current one (no GPU: the library, the
streams and the allocator's side of them are recorded stand-ins)."""
import contextlib

import pytest
import torch

from sparse_mixture_experts_03_b200 import moe

BF, E4M3, F32 = torch.bfloat16, moe.E4M3, torch.float32


class FakeStream:
    def __init__(self, name):
        self.name, self.cuda_stream = name, 1


class Library:
    def __getattr__(self, name):
        return lambda *args: 4096 if name.endswith("bytes") else 0


@pytest.fixture
def world(monkeypatch):
    current, side = FakeStream("current"), FakeStream("side")
    now = [current]
    allocated, recorded = {}, {}
    real_empty = torch.empty

    @contextlib.contextmanager
    def stream(s):
        now.append(s)
        yield
        now.pop()

    def empty(*args, **kw):
        t = real_empty(*args, **kw)
        allocated[t.data_ptr()] = now[-1].name
        return t

    def record(t, s):
        recorded.setdefault(t.data_ptr(), set()).add(s.name)

    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: now[-1])
    monkeypatch.setattr(torch.Tensor, "record_stream", record)
    monkeypatch.setattr(moe, "lib", lambda: Library())
    monkeypatch.setattr(moe, "_on_current", lambda name, t, s: (t.data_ptr(), 0))
    return side, allocated, recorded


def few(**kw):
    z = lambda *s, dtype=BF: torch.zeros(*s, dtype=dtype)
    return moe.forward_few(z(2, 256), z(4, 256), z(4, 256, 256), z(4, 256, 128), None, 2, 1, 1,
                           128, 0, **kw)


CALLS = {
    "rows": lambda **kw: moe.quantize_rows(torch.zeros(3, 256, dtype=BF), **kw),
    "swiglu": lambda **kw: moe.swiglu_quantize_rows(torch.zeros(3, 512, dtype=BF), **kw),
    "weight": lambda **kw: moe.quantize_weight(torch.zeros(2, 64, 256, dtype=BF), **kw),
    "product": lambda **kw: moe.matmul_fp8(torch.zeros(3, 128, dtype=E4M3), torch.zeros(1, 3),
                                           torch.zeros(64, 128, dtype=E4M3), torch.zeros(1, 1), **kw),
    "few": few,
}


@pytest.mark.parametrize("name", CALLS)
def test_memory_for_another_stream_is_that_streams(world, name):
    """A block of the current stream's may still have work queued on it there,
    which the other stream does not wait for."""
    side, allocated, recorded = world
    got = CALLS[name](stream=side)
    got = got if isinstance(got, tuple) else (got,)
    assert set(allocated.values()) == {"side"}
    # the caller reads the results on the current stream, too
    assert all("current" in recorded[t.data_ptr()] for t in got)


@pytest.mark.parametrize("name", CALLS)
def test_memory_for_the_current_stream_is_the_current_streams(world, name):
    _, allocated, recorded = world
    CALLS[name]()
    assert set(allocated.values()) == {"current"} and not recorded


def test_the_callers_buffers_are_recorded_on_the_stream_that_uses_them(world):
    side, allocated, recorded = world
    q, s, y = torch.zeros(3, 256, dtype=E4M3), torch.zeros(2, 3), torch.zeros(2, 256)
    moe.quantize_rows(torch.zeros(3, 256, dtype=BF), q=q, scales=s, stream=side)
    ws = torch.zeros(4096, dtype=torch.uint8)
    few(y=y, workspace=ws, stream=side)
    assert not allocated
    assert all("side" in recorded[t.data_ptr()] for t in (q, s, y, ws))
