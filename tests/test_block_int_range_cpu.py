"""Numbers that do not fit the library's 32 bits: the calls on the cache in 8 bits refuse them instead of cutting them to
others (2^32 + 1 layers on is not layer 1). No GPU is touched."""
import pytest
import torch

from tiered_kv_cache_decode_gb300 import binding
from test_block_refusals_cpu import I, Shell, t

OVER = [2 ** 31, 2 ** 32, 2 ** 32 + 1, 2 ** 64, -2 ** 31 - 1, -2 ** 32]


def W():
    return t(2, 2, 128, dtype=torch.float32)


@pytest.mark.parametrize("x", OVER)
@pytest.mark.parametrize("call", [
    lambda c, x: c.append(x, t(2, 3, 2, 128), t(2, 3, 2, 128)),
    lambda c, x: c.attend(x, t(2, 1, 8, 128), t(2, dtype=I)),
    lambda c, x: c.read(x, t(2, dtype=I), 5),
    lambda c, x: c.read(0, t(2, dtype=I), x, k_out=t(2, 5, 2, 128), v_out=t(2, 5, 2, 128)),
    lambda c, x: c.evict(x, t(2, dtype=I), 64, 0, W()),
    lambda c, x: c.evict(0, t(2, dtype=I), x, 0, W(), kept=t(2, 2, 64, dtype=I)),
    lambda c, x: c.evict(0, t(2, dtype=I), 64, x, W()),
    lambda c, x: c.evict(0, t(2, dtype=I), 64, 0, W(), into=Shell(2, 8, 2, 128, "cpu"), into_layer=x),
    lambda c, x: c.blocks(x),
], ids=["append", "attend", "read", "read n", "evict", "evict keep", "evict recent", "evict into_layer", "blocks"])
def test_calls_refuse(call, x, monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: pytest.fail("the call went on"))
    with pytest.raises(ValueError, match="32 bits"):
        call(Shell(2, 8, 2, 128, "cpu"), x)


@pytest.mark.parametrize("x", OVER)
@pytest.mark.parametrize("name", ["batch", "num_layers", "num_q_heads", "num_kv_heads", "capacity", "score_queries", "head_dim"])
def test_configurations_refuse(name, x, monkeypatch):
    monkeypatch.setattr(binding, "load", lambda: None)
    args = dict(batch=1, num_layers=1, num_q_heads=1, num_kv_heads=1, capacity=64)
    with pytest.raises(ValueError, match="32 bits"):
        binding.BlockCache(**{**args, name: x})
