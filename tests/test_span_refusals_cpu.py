"""Host-side refusals of the calls between projections and the cache; no GPU is
touched (a NULL cache, and the binding's checks on CPU tensors)."""
import ctypes

import pytest
import torch

from tiered_kv_cache_decode_gb300 import binding
from tiered_kv_cache_decode_gb300 import build as B


@pytest.fixture(scope="module")
def lib():
    B.build()
    return binding.load()


def test_null_cache_is_refused(lib):
    P = ctypes.c_void_p(4096)
    assert lib.qevict_qk_norm_rope(None, 0, P, 128, P, 128, None, 0, 1, None, None, None, 0.0, P, 0, P, P, None,
                                   None) == 1
    assert lib.qevict_span_attention(None, 0, P, 1, P, P, 1, None, None, 0, 0, P, None, None) == 1
    assert lib.qevict_span_scores(None, 0, P, 1, P, 1, None, None, 0, 0, P, P, None) == 1
    assert b"NULL" in lib.qevict_last_error()


class Shell(binding.TieredCache):
    """The binding's checks without a cache behind them."""

    def __init__(self, B, Hq, Hkv, w):
        self.B, self.Hq, self.Hkv, self.w, self.units, self.device = B, Hq, Hkv, w, B, 0
        self._dev = torch.device("cuda", 0)
        self.handle = None


def t(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


@pytest.mark.parametrize("q,k", [(t(2, 3, 8, 128, dtype=torch.float32), t(2, 3, 2, 128)), (t(2, 3, 7, 128), t(2, 3, 2, 128)),
                                 (t(1, 3, 8, 128), t(2, 3, 2, 128)), (t(2, 3, 8, 64), t(2, 3, 2, 64)),
                                 (t(2, 3, 8, 128), t(2, 3, 2, 128))])   # the last: on the CPU
def test_binding_refuses_wrong_tensors(q, k):
    c = Shell(2, 8, 2, 64)
    with pytest.raises(ValueError):
        c.qk_norm_rope(0, q, k, t(64, dtype=torch.float32))
    with pytest.raises(ValueError):
        c.span_attention(0, q, k, k)
    with pytest.raises(ValueError):
        c.span_scores(0, q, k, t(2, 8, 3, dtype=torch.float32))


def test_token_strides():
    c, one = Shell(2, 8, 2, 64), Shell(1, 8, 2, 64)
    c._dev = one._dev = torch.device("cpu")   # the layouts alone
    fused = t(2, 5, 12, 128)
    assert c._tokens(fused[:, :, :8], 8, "q") == (5, 12 * 128)
    assert c._tokens(fused[:, :, 8:10], 2, "k") == (5, 12 * 128)
    assert c._tokens(t(2, 1, 8, 128), 8, "q") == (1, 8 * 128)
    assert c._tokens(t(2, 8, 128), 8, "q") == (1, 8 * 128)
    assert c._tokens(fused[:, 2, :8], 8, "q") == (1, 5 * 12 * 128)     # one token of each sequence
    assert one._tokens(t(1, 1, 8, 128), 8, "q") == (1, 8 * 128)
    assert one._tokens(t(1, 7, 8, 128)[:, ::2], 8, "q") == (4, 2 * 8 * 128)
    for bad in (t(2, 9, 8, 128)[:, ::2], fused[:, 1:, :8], t(2, 5, 8, 256)[..., ::2],
                t(2, 8, 5, 128).transpose(1, 2)):
        with pytest.raises(ValueError):
            c._tokens(bad, 8, "q")
    with pytest.raises(ValueError):
        c._dense(fused[:, :, :8], 8, "q")
