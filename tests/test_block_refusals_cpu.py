"""Host-side refusals of the cache in 8 bits; no GPU is touched (a NULL handle, configurations that are out of range,
an allocator that fails, and the binding's checks on CPU tensors)."""
import ctypes

import pytest
import torch

from tiered_kv_cache_decode_gb300 import binding
from tiered_kv_cache_decode_gb300 import build as B


@pytest.fixture(scope="module")
def lib():
    B.build()
    return binding.load()


def cfg(**kw):
    base = dict(batch=2, num_layers=3, num_q_heads=8, num_kv_heads=2, head_dim=128, capacity=300, format=0, score_queries=1)
    base.update(kw)
    return binding.BlockConfig(**base)


def test_null_handle_is_refused(lib):
    P = ctypes.c_void_p(4096)
    assert lib.qevict_block_append(None, 0, P, 256, P, 256, 1, None, None, None, None) == 1
    assert lib.qevict_block_attention(None, 0, P, 1, P, P, None, None, 0, None) == 1
    assert lib.qevict_block_read(None, 0, P, None, 1, P, P, None) == 1
    assert lib.qevict_block_evict(None, 0, P, 64, 0, P, None, 0, None, P, P, None) == 1
    assert b"NULL" in lib.qevict_last_error()
    assert lib.qevict_block_view(None, 0, ctypes.byref(P), ctypes.byref(P)) == 1
    assert lib.qevict_block_get_status(None, None) == 1 and lib.qevict_block_clear_status(None, None) == 1
    assert lib.qevict_block_destroy(None) == 1 and lib.qevict_block_capacity(None) == -1


@pytest.mark.parametrize("bad", [dict(batch=0), dict(batch=65536), dict(num_layers=0), dict(num_q_heads=7), dict(num_q_heads=18),
                                 dict(num_kv_heads=0), dict(head_dim=64), dict(capacity=0), dict(capacity=2 ** 21 + 1),
                                 dict(format=2), dict(format=-1), dict(score_queries=-1), dict(score_queries=9),
                                 dict(batch=60000, num_kv_heads=1, num_q_heads=1, capacity=2 ** 21)])
def test_create_refuses_bad_configurations(lib, bad):
    h = ctypes.c_void_p()
    assert lib.qevict_block_create(ctypes.byref(cfg(**bad)), None, None, ctypes.byref(h)) == 1, bad
    assert not h.value and lib.qevict_last_error()


def test_create_refuses_missing_arguments(lib):
    h = ctypes.c_void_p()
    assert lib.qevict_block_create(None, None, None, ctypes.byref(h)) == 1
    assert lib.qevict_block_create(ctypes.byref(cfg()), None, None, None) == 1
    half = binding.Allocator(binding.ALLOC_FN(lambda *a: None), binding.FREE_FN(), None)
    assert lib.qevict_block_create(ctypes.byref(cfg()), ctypes.byref(half), None, ctypes.byref(h)) == 1


@pytest.mark.parametrize("fail_at", [0, 1, 2, 4])   # scratch, logits, the first and the last layer
def test_failing_allocator_leaves_nothing(lib, fail_at):
    live, calls = set(), [0]

    def _a(size, stream, ctx):
        i = calls[0]
        calls[0] += 1
        if i == fail_at:
            return None
        live.add(0x10000000 + 0x100000 * i)
        return 0x10000000 + 0x100000 * i

    al = binding.Allocator(binding.ALLOC_FN(_a), binding.FREE_FN(lambda p, s, c: live.remove(p)), None)
    h = ctypes.c_void_p()
    assert lib.qevict_block_create(ctypes.byref(cfg()), ctypes.byref(al), None, ctypes.byref(h)) == 2
    assert not h.value and calls[0] == fail_at + 1 and not live


class Reached:
    """A library none of whose calls may be reached."""

    def __getattr__(self, name):
        return lambda *a: pytest.fail(f"{name} was called")


class Shell(binding.BlockCache):
    """The binding's checks without a handle behind them."""

    def __init__(self, B, Hq, Hkv, capacity, device="cuda"):
        self.B, self.Hq, self.Hkv, self.capacity, self.device = B, Hq, Hkv, capacity, 0
        self._dev = torch.device(device) if device == "cpu" else torch.device("cuda", 0)
        self._per_seq, self._per_token = (B,), (B, Hkv, capacity)
        self.handle, self.lib = None, Reached()


def t(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


I = torch.int32


@pytest.mark.parametrize("call", [
    lambda c: c.append(0, t(2, 3, 2, 128, dtype=torch.float32), t(2, 3, 2, 128)),
    lambda c: c.append(0, t(2, 3, 2, 128), t(2, 4, 2, 128)),
    lambda c: c.append(0, t(2, 3, 3, 128), t(2, 3, 3, 128)),
    lambda c: c.append(0, t(2, 3, 2, 128), t(2, 3, 2, 128), start=t(2, dtype=torch.int64)),
    lambda c: c.append(0, t(2, 3, 2, 128), t(2, 3, 2, 128), n_new=t(3, dtype=I)),
    lambda c: c.append(0, t(2, 3, 2, 128), t(2, 3, 2, 128), weights=t(2, 2, 100, dtype=torch.float32)),
    lambda c: c.attend(0, t(2, 1, 9, 128), t(2, dtype=I)),
    lambda c: c.attend(0, t(2, 1, 8, 128), t(2, dtype=torch.int64)),
    lambda c: c.attend(0, t(2, 2, 8, 128)[:, ::2], t(2, dtype=I)),
    lambda c: c.attend(0, t(2, 1, 8, 128), t(2, dtype=I), out=t(2, 1, 8, 128, dtype=torch.float32)),
    lambda c: c.attend(0, t(2, 1, 8, 128), t(2, dtype=I), lse=t(2, 8, dtype=torch.float32)),
    lambda c: c.attend(0, t(2, 1, 8, 128), t(2, dtype=I), weights=t(2, 2, 128)),
    lambda c: c.read(0, t(2, dtype=torch.int64), 5),
    lambda c: c.read(0, None, 5),
    lambda c: c.read(0, t(2, dtype=I), 5, k_out=t(2, 4, 2, 128)),
    lambda c: c.evict(0, t(2, dtype=I), 64, 0, t(2, 2, 127, dtype=torch.float32)),
    lambda c: c.evict(0, t(2, dtype=I), 64, 0, None),
    lambda c: c.evict(0, t(2, dtype=I), 64, 0, t(2, 2, 128, dtype=torch.float32), kept=t(2, 2, 128, dtype=I)),
])
def test_binding_refuses_wrong_tensors(call):
    with pytest.raises(ValueError):
        call(Shell(2, 8, 2, 128, "cpu"))


def test_binding_refuses_tensors_of_another_device():
    c = Shell(2, 8, 2, 128)
    with pytest.raises(ValueError):
        c.attend(0, t(2, 1, 8, 128), t(2, dtype=I))
    with pytest.raises(ValueError):
        c.read(0, t(2, dtype=I), 5)


def test_unknown_format_is_refused(lib):
    with pytest.raises(ValueError):
        binding.BlockCache(1, 1, 1, 1, 64, "fp8")
