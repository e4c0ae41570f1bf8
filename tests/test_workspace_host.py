"""The binding's workspaces on the host: a fake of the library's call and CPU buffers, no GPU."""
import contextlib
import gc
import threading
import time
import weakref

import pytest

torch = pytest.importorskip("torch")
from trellis_quantized_weight_gb300 import binding  # noqa: E402


class Stream:
    def __init__(self, handle):
        self.cuda_stream, self.capturing = handle, False


device = [0]                                               # of the thread


@contextlib.contextmanager
def on_device(index):
    device.append(index)
    try:
        yield
    finally:
        device.pop()


@pytest.fixture(autouse=True)
def host(monkeypatch):
    monkeypatch.setattr(binding, "_ws_cache", {})
    monkeypatch.setattr(binding, "_zeros", lambda nbytes, index, stream: torch.zeros(nbytes, dtype=torch.uint8))
    monkeypatch.setattr(binding, "_current_device", lambda: device[-1])
    monkeypatch.setattr(binding, "_on_device", on_device)
    monkeypatch.setattr(binding, "_is_capturing", lambda stream: stream.capturing)


def call(needs, body=None):
    """A fake entry point that refuses a workspace of fewer bytes than `needs` and notes the ones it takes."""
    def trellis_fake(ptr, size, handle):
        if ptr is None or size < needs:
            return -7
        trellis_fake.taken.append((ptr, size, handle))
        return body() if body is not None else 0
    trellis_fake.taken = []
    return trellis_fake


def launch(fn, needs, handle=1, ask=False, capturing=False):
    stream = Stream(handle)
    stream.capturing = capturing
    binding._launch(fn, (), 0, stream, lambda: needs, ask=ask)
    return fn.taken[-1]


def test_a_workspace_a_stream_and_growth():
    for ask in (False, True):
        first = launch(call(1000), 1000, 3 + ask, ask)
        assert launch(call(500), 500, 3 + ask, ask) == first
        assert launch(call(5000), 5000, 3 + ask, ask)[1] >= 5000
        other = launch(call(10), 10, 13 + ask, ask)
        assert other[0] not in (first[0], launch(call(1), 1, 3 + ask, ask)[0])


def test_a_refusal_is_raised():
    fn = call(0, lambda: -2)
    with pytest.raises(binding.TrellisError, match="trellis_fake"):
        launch(fn, 16)
    launch(call(16), 16)                                   # and the lock is free again


def test_calls_of_threads_on_one_stream_take_turns():
    inside, most = [0, 0], [0, 0]

    def body_of(k):
        def body():
            inside[k] += 1
            most[k] = max(most[k], inside[k])
            time.sleep(0.002)
            inside[k] -= 1
            return 0
        return body

    def work(k):
        for i in range(5):
            launch(call(100 + 400 * i, body_of(k)), 100 + 400 * i, handle=k)
    threads = [threading.Thread(target=work, args=(k % 2,)) for k in range(6)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert most == [1, 1]


def test_a_buffer_in_use_is_not_replaced():
    """While a call is under way another thread that needs more waits: the buffer that it was given stays."""
    started, checked, alive = threading.Event(), threading.Event(), []

    def body():
        ref = weakref.ref(binding._ws_cache[(0, 1)].buf)
        started.set()
        checked.wait(0.2)                                  # the other thread asks for more meanwhile
        gc.collect()
        alive.append(ref() is not None)
        return 0
    t = threading.Thread(target=lambda: (started.wait(5), launch(call(9000), 9000), checked.set()))
    t.start()
    launch(call(100, body), 100)
    t.join()
    assert alive == [True] and binding._ws_cache[(0, 1)].size >= 9000


@pytest.mark.parametrize("ask", [False, True])
def test_a_captured_buffer_outlives_its_growth(ask):
    """What a graph was captured with stays allocated when a later call needs more; what none was, does not."""
    launch(call(100), 100, ask=ask)
    plain = weakref.ref(binding._ws_cache[(0, 1)].buf)
    launch(call(1000), 1000, ask=ask)
    gc.collect()
    assert plain() is None
    ws = binding._ws_cache[(0, 1)]
    captured, taken = weakref.ref(ws.buf), ws.ptr
    assert launch(call(1000), 1000, ask=ask, capturing=True)[0] == taken
    for n in (5000, 20000):                                # the second one outgrows a buffer that no graph has
        assert launch(call(n), n, ask=ask)[0] != taken
    gc.collect()
    assert captured() is not None and captured().data_ptr() == taken and len(ws.kept) == 1


@pytest.mark.parametrize("ask", [False, True])
def test_a_buffer_made_during_a_capture_is_the_graphs_alone(ask):
    """Its zero-fill runs in replays only, so no call outside the graph may get it."""
    inside = launch(call(1000), 1000, ask=ask, capturing=True)
    ws = binding._ws_cache[(0, 1)]
    assert inside[1] >= 1000 and ws.buf is None and ws.size == 0 and not ws.in_graph
    launch(call(1000), 1000, ask=ask)
    before = ws.ptr
    launch(call(9000), 9000, ask=ask, capturing=True)
    assert ws.ptr == before and ws.size < 9000


def test_calls_run_on_the_tensors_device():
    """The library launches on the thread's current device: a call whose tensors are elsewhere changes it meanwhile."""
    seen = []

    def trellis_fake(ptr, size, handle):
        seen.append(device[-1])
        return 0 if size >= 1000 else -7

    def trellis_plain(a, handle):
        seen.append((device[-1], a, handle))
        return 0
    sizes = []
    for index in (1, 0, 3):
        for ask in (False, True):
            binding._launch(trellis_fake, (), index, Stream(5), lambda: sizes.append(device[-1]) or 1000, ask=ask)
        binding._enqueue(trellis_plain, (7,), index, Stream(5))
        assert [s if isinstance(s, int) else s[0] for s in seen] == [index] * len(seen) and (index, 7, 5) in seen
        assert sizes == [index] * len(sizes) and device == [0]
        seen.clear()
        sizes.clear()
    assert sorted(k[0] for k in binding._ws_cache) == [0, 1, 3]
    with pytest.raises(binding.TrellisError, match="trellis_plain"):
        def trellis_plain(handle):
            return -5
        binding._enqueue(trellis_plain, (), 1, Stream(5))
    assert device == [0]
