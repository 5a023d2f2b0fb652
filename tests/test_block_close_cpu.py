"""What a cache in 8 bits waits for before its memory goes back, without a GPU: the stream of its creation, for which the
library's call waits and to which the memory goes back, first waits for every stream that a call was made on."""
import contextlib
import ctypes
from types import SimpleNamespace

import pytest
import torch

from tiered_kv_cache_decode_gb300 import binding


HOME = 3


class Stream:
    def __init__(self, raw, log, capturing=False):
        self.cuda_stream, self.log, self.capturing = raw, log, capturing

    def wait_stream(self, other):
        self.log.append((self.cuda_stream, other.cuda_stream))


def cache(log, B=2, Hq=8, Hkv=2, capacity=128):
    c = binding.BlockCache.__new__(binding.BlockCache)
    c.B, c.Hq, c.Hkv, c.capacity, c.device, c.layers, c._dev = B, Hq, Hkv, capacity, 0, 1, torch.device("cpu")
    c._per_seq, c._per_token, c._home, c._streams = (B,), (B, Hkv, capacity), Stream(HOME, log), {}
    done = {n: lambda *a: 0 for n in ("append", "attention", "read", "evict", "clear_status")}
    done["destroy"] = lambda *a: log.append("destroy") or 0
    c.lib = SimpleNamespace(**{"qevict_block_" + n: f for n, f in done.items()})
    c.handle = ctypes.c_void_p(4096)
    return c


@pytest.fixture
def world(monkeypatch):
    w = SimpleNamespace(log=[], current=None)

    @contextlib.contextmanager
    def stream(s):
        before, w.current = w.current, s
        yield
        w.current = before

    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: w.current)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: w.current.capturing)
    w.stream = lambda raw, **kw: Stream(raw, w.log, **kw)
    w.current = w.stream(1)
    return w


def t(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


LEN, W = t(2, dtype=torch.int32), t(2, 2, 128, dtype=torch.float32)
CALLS = {
    "append": lambda c, s: c.append(0, t(2, 3, 2, 128), t(2, 3, 2, 128), stream=s),
    "attend": lambda c, s: c.attend(0, t(2, 1, 8, 128), LEN, stream=s),
    "read": lambda c, s: c.read(0, LEN, 5, stream=s),
    "evict": lambda c, s: c.evict(0, LEN, 64, 0, W, stream=s),
    "clear_status": lambda c, s: c.clear_status(stream=s),
}


@pytest.mark.parametrize("call", CALLS)
def test_close_waits_for_the_streams_of_all_calls(world, call):
    c = cache(world.log)
    CALLS[call](c, world.stream(7))
    CALLS[call](c, world.stream(8))
    CALLS[call](c, world.stream(7))
    CALLS[call](c, world.stream(HOME))
    CALLS[call](c, None)   # torch's current one
    c.close()
    assert sorted(world.log[:-1]) == [(HOME, 1), (HOME, 7), (HOME, 8)] and world.log[-1] == "destroy"
    c.close()
    assert len(world.log) == 4


def test_both_caches_of_an_eviction_wait(world):
    c, d = cache(world.log), cache(world.log)
    c.evict(0, LEN, 64, 0, W, into=d, weights_out=W.clone(), stream=world.stream(9))
    d.close()
    assert world.log == [(HOME, 9), "destroy"]
    c.close()
    assert world.log == [(HOME, 9), "destroy"] * 2


def test_a_stream_in_capture_is_not_waited_for(world):
    """Its work runs when the graph is replayed; a wait would join the capture."""
    c = cache(world.log)
    CALLS["append"](c, world.stream(5))
    CALLS["append"](c, world.stream(6, capturing=True))
    c.close()
    assert world.log == [(HOME, 5), "destroy"]
    c = cache(world.log)
    CALLS["append"](c, world.stream(5))
    c._home.capturing = True
    c.close()
    assert world.log == [(HOME, 5), "destroy", "destroy"]


def test_the_memory_goes_back_also_where_a_wait_fails(world):
    c = cache(world.log)
    c._home.wait_stream = lambda s: (_ for _ in ()).throw(RuntimeError("gone"))
    CALLS["append"](c, world.stream(5))
    with pytest.raises(RuntimeError):
        c.close()
    assert world.log == ["destroy"] and not c.handle
