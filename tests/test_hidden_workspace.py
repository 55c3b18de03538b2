"""The binding's cached workspaces and host threads, on the CPU: the library's entry points are
replaced by functions that note when they begin and end, and the stream queries by one fixed
stream, so that the threads meet at will."""
import threading
import time
from types import SimpleNamespace

import pytest
import torch

from weight_only_int4_w4_b200 import build


@pytest.fixture
def w4(monkeypatch):
    build.build_library()
    from weight_only_int4_w4_b200 import w4 as mod
    monkeypatch.setattr(mod, "_raw_stream", lambda dev: 7)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    return mod


class Calls:
    """Stands for a library call of several launches: `most` is how many were under way at a time
    on one workspace."""

    def __init__(self):
        self.lock, self.inside, self.most, self.count = threading.Lock(), {}, 0, 0

    def __call__(self, *args):
        ws = getattr(args[-3], "value", args[-3])
        with self.lock:
            self.count += 1
            self.inside[ws] = self.inside.get(ws, 0) + 1
            self.most = max(self.most, self.inside[ws])
        time.sleep(0.01)
        with self.lock:
            self.inside[ws] -= 1
        return 0


def in_threads(n, f):
    errors = []

    def work():
        try:
            for _ in range(3):
                f()
        except Exception as e:  # seen by the test
            errors.append(e)

    ts = [threading.Thread(target=work) for _ in range(n)]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    assert not errors, errors


def test_calls_of_two_threads_on_one_stream_do_not_share_a_workspace_in_time(w4, monkeypatch):
    """A fused call hands data from launch to launch through its workspace, and other threads
    run during the call: on one stream, the next call begins when the first has ended."""
    bufs = {}
    monkeypatch.setattr(w4, "_fused_workspace",
                        lambda need, dev, raw, stream: bufs.setdefault((dev, raw), torch.empty(need, dtype=torch.uint8)))
    calls = Calls()
    in_threads(3, lambda: w4._fused_call("t", calls, lambda *s: 64, (1, 2, 3), 0, None, None, (0,)))
    assert calls.count == 9 and calls.most == 1


def test_calls_on_two_streams_run_at_the_same_time(w4, monkeypatch):
    raws = threading.local()
    monkeypatch.setattr(w4, "_raw_stream", lambda dev: raws.__dict__.setdefault("raw", threading.get_ident()))
    monkeypatch.setattr(w4, "_fused_workspace", lambda need, dev, raw, stream: torch.empty(need, dtype=torch.uint8))
    meet = threading.Barrier(2, timeout=20)

    def call(*args):  # both threads are inside, or the barrier breaks
        meet.wait()
        return 0

    in_threads(2, lambda: w4._fused_call("t", call, lambda *s: 64, (1, 2, 3), 0, None, None, (0,)))


def test_a_call_inside_the_allocation_does_not_wait_for_itself(w4, monkeypatch):
    """A finalizer that runs while the workspace is allocated may make a call of its own."""
    calls, depth = Calls(), []

    def alloc(need, dev, raw, stream):
        if not depth:
            depth.append(1)
            w4._fused_call("t", calls, lambda *s: 64, (1, 2, 3), 0, None, None, (0,))
        return torch.empty(need, dtype=torch.uint8)

    monkeypatch.setattr(w4, "_fused_workspace", alloc)
    t = threading.Thread(target=lambda: w4._fused_call("t", calls, lambda *s: 64, (1, 2, 3), 0, None, None, (0,)), daemon=True)
    t.start()
    t.join(20)
    assert not t.is_alive() and calls.count == 2


@pytest.mark.parametrize("name", ["w4a16_gemm", "w4a16_gemm_host", "w4a16_gemm_host_async", "w4a16_gemm_outliers"])
def test_the_plain_product_likewise(w4, monkeypatch, name):
    """w4a16_gemm and its relatives stage their operand in the cached workspace from 4 tokens on."""
    calls, ws, t = Calls(), torch.empty(64, dtype=torch.uint8), torch.empty(16, dtype=torch.float32)
    monkeypatch.setattr(w4._lib, name, calls)
    monkeypatch.setattr(w4, "workspace", lambda M, N, K, device, stream=None: ws)
    X = SimpleNamespace(is_cuda=True, dim=lambda: 2, is_contiguous=lambda: True, dtype=torch.bfloat16, shape=(16, 128),
                        device=torch.device("cuda", 0), data_ptr=lambda: 256)
    kw = dict(stream=SimpleNamespace(cuda_stream=7))
    in_threads(3, {"w4a16_gemm": lambda: w4.w4a16_gemm(X, t, t, t, out=t, **kw),
                   "w4a16_gemm_host": lambda: w4.w4a16_gemm_host(X, X, t, t, t, t, t, **kw),
                   "w4a16_gemm_host_async": lambda: w4.w4a16_gemm_host(X, X, t, t, t, t, t, wait=False, **kw),
                   "w4a16_gemm_outliers": lambda: w4.w4a16_gemm_outliers(X, t, t, t, (t, t, t), out=t, **kw)}[name])
    assert calls.count == 9 and calls.most == 1


def test_the_cached_workspace_is_zeroed_on_the_stream_that_uses_it(w4, monkeypatch):
    """Zero-filled on the current stream, its counters may not be zero yet when a call on another
    stream starts (and a buffer that is replaced would go back to the wrong stream)."""
    on = []

    class Use:
        def __init__(self, s):
            self.s = s

        def __enter__(self):
            on.append(self.s)

        def __exit__(self, *a):
            on.pop()

    monkeypatch.setattr(w4, "_ws_cache", {})
    monkeypatch.setattr(torch.cuda, "stream", Use)
    monkeypatch.setattr(w4, "w4a16_gemm_workspace_size", lambda M, N, K: 64)
    filled = []
    monkeypatch.setattr(w4.torch, "zeros", lambda n, **kw: filled.append(list(on)) or torch.empty(n, dtype=torch.uint8))
    side = SimpleNamespace(cuda_stream=9)
    a = w4.workspace(1, 2, 3, torch.device("cuda", 0), side)
    assert a is w4.workspace(1, 2, 3, torch.device("cuda", 0), side) and filled == [[side]] and not on
