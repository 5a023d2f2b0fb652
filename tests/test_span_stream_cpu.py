"""The stream that the calls between projections and the cache run on, without a GPU: the one given, or torch's
current one on the cache's device, asked of torch's public interface."""
from types import SimpleNamespace

import torch

from tiered_kv_cache_decode_gb300 import binding


def test_default_stream_is_torchs_current_one(monkeypatch):
    cache = binding.TieredCache.__new__(binding.TieredCache)
    cache.device, cache.handle = 3, None
    asked = []

    def current_stream(device=None):
        asked.append(device)
        return SimpleNamespace(cuda_stream=4242)

    monkeypatch.setattr(torch.cuda, "current_stream", current_stream)
    assert cache._raw_stream(None) == 4242 and asked == [3]
    assert cache._raw_stream(SimpleNamespace(cuda_stream=77)) == 77 and asked == [3]
