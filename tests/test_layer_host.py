"""What the layer binding does on the host around a launch, with stand-ins for the tensors and the library (CPU-only)."""
from __future__ import annotations

import contextlib
import itertools
import threading
import time

import pytest
import torch

from split_bf16_gemm_swap_gb300 import layer

_address = itertools.count(1 << 20, 1 << 20)


class FakeTensor:
    """As much of a contiguous CUDA tensor as the binding's checks look at."""

    is_cuda = True

    def __init__(self, *shape, dtype=torch.bfloat16, device=0):
        self.shape, self.dtype, self.index, self.address = torch.Size(shape), dtype, device, next(_address)

    @property
    def device(self):
        return torch.device("cuda", self.index)

    def get_device(self):
        return self.index

    def data_ptr(self):
        return self.address

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def is_contiguous(self):
        return True

    def stride(self):
        out, n = [], 1
        for s in reversed(self.shape):
            out.insert(0, n)
            n *= s
        return tuple(out)


def fake_empty(shape, *more, dtype=None, device=None):
    return FakeTensor(*([shape] if isinstance(shape, int) else shape), dtype=dtype, device=torch.device(device).index)


@pytest.fixture
def library(monkeypatch):
    """Replaces the library's launching functions by `library.call`, and every stream by each device's default one."""
    class Library:
        call = staticmethod(lambda name, args: 0)

    lib = Library()
    functions = {n: (lambda *args, n=n: lib.call(n, args)) for n in layer.ABI_FUNCTIONS if not n.endswith("_workspace")}
    monkeypatch.setattr(layer, "_functions", functions)
    monkeypatch.setattr(layer, "_attention_bytes", lambda *sizes: 4096)
    monkeypatch.setattr(layer, "_moe_bytes", lambda *sizes: 8192)
    monkeypatch.setattr(layer, "_current_stream", lambda device: 0)
    monkeypatch.setattr(layer, "_current_device", lambda: 0, raising=False)
    monkeypatch.setattr(layer, "_kept", {})
    monkeypatch.setattr(torch, "empty", fake_empty)
    return lib


def operators(device=0, **kw):
    """Calls of the four operators with tensors on `device`, by name."""
    def t(*shape, dtype=torch.bfloat16):
        return FakeTensor(*shape, dtype=dtype, device=device)

    i32, i64, f32 = torch.int32, torch.int64, torch.float32
    x, cache = t(4, 64), t(8, 16, 2, 64)
    q, kv = t(4, 8, 64), t(4, 2, 64)
    return {
        "residual_norm": lambda: layer.residual_norm(x, t(4, 64), **kw),
        "rope_append": lambda: layer.rope_append(q, kv, kv, t(99, 64, dtype=f32), t(4, dtype=i64), t(4, dtype=i64), cache,
                                                 t(8, 16, 2, 64), **kw),
        "paged_attention": lambda: layer.paged_attention(q, cache, t(8, 16, 2, 64), t(4, 2, dtype=i32), t(4, dtype=i32),
                                                         t(5, dtype=i32), **kw),
        "moe": lambda: layer.moe(x, t(8, 64), t(8, 64, 64), t(8, 64, 32), 2, **kw),
    }


def test_threads_do_not_share_a_workspace_while_a_call_is_enqueued(library):
    # An operator with a workspace is two launches: between them no other call may be given the same memory.
    busy, shared, lock = {}, [], threading.Lock()

    def call(name, args):
        work = args[-3]
        with lock:
            if busy.get(work, 0):
                shared.append(name)
            busy[work] = busy.get(work, 0) + 1
        time.sleep(0.002)                              # ctypes lets other threads run during a call
        with lock:
            busy[work] -= 1
        return 0

    library.call = call
    failed = []

    def run(name):
        try:
            for _ in range(10):
                operators()[name]()
        except Exception as e:                         # pragma: no cover
            failed.append(e)

    threads = [threading.Thread(target=run, args=(n,)) for n in ("moe", "paged_attention") * 2]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed and not shared


def test_a_call_made_while_another_is_enqueued_by_the_same_thread_goes_through(library):
    # (by a finaliser, which Python may run at any time)
    calls = []

    def call(name, args):
        calls.append(name)
        if len(calls) == 1:
            operators()["paged_attention"]()
        return 0

    library.call = call
    operators()["moe"]()
    assert calls == ["lowm_moe", "lowm_paged_attention"]


@pytest.mark.parametrize("name", sorted(operators()))
@pytest.mark.parametrize("current,device", [(0, 0), (0, 1), (1, 0)])
def test_the_tensors_device_is_current_during_a_call(library, monkeypatch, name, current, device):
    # the library launches on the current device, whatever device its pointers belong to
    now, seen, entered = [current], [], []

    @contextlib.contextmanager
    def guard(index):
        entered.append(index)
        before, now[0] = now[0], index
        try:
            yield
        finally:
            now[0] = before

    monkeypatch.setattr(layer, "_current_device", lambda: now[0])
    monkeypatch.setattr(torch.cuda, "device", guard)
    library.call = lambda n, args: seen.append((n, now[0])) or 0
    operators(device)[name]()
    assert seen == [("lowm_" + name, device)] and now == [current]
    assert entered == ([] if current == device else [device])


@pytest.mark.parametrize("name", sorted(operators()))
def test_a_stream_of_another_device_is_refused(library, monkeypatch, name):
    # its device would become current, and the call would take the current stream of the tensors' device instead
    class Stream:
        device, cuda_stream = torch.device("cuda", 1), 1234

    entered = []
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: entered.append(s) or contextlib.nullcontext())
    library.call = lambda n, args: pytest.fail("launched")
    with pytest.raises(ValueError, match="stream"):
        operators(0, stream=Stream())[name]()
    assert not entered
    library.call = lambda n, args: 0
    monkeypatch.setattr(layer, "_current_device", lambda: 1)
    stream = Stream()
    operators(1, stream=stream)[name]()
    assert entered == [stream]
