"""The rotation's angle near zero, where one member of a channel pair is 0 and the other's turn into it is all
there is: sin(angle) has to be right to its own last bits, not to a fixed fraction of a turn."""
import numpy as np
import pytest
import torch

from tiered_kv_cache_decode_gb300 import binding

pytestmark = pytest.mark.gpu
D = 128


@pytest.fixture(autouse=True, scope="module")
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from tiered_kv_cache_decode_gb300 import build
    build.build()
    binding.load()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("first", ["theta", "small"])
def test_small_angles(interleaved, first):
    """y = (-b sin t, b cos t) of pairs (0, b) at positions -3 .. 3. The angle's fraction of a turn is a 64-bit
    number (2^-64 turns per position against angles of 2^-43 turns and more: 2^-21 relative, below 2^-31 for the
    frequencies of a model), rounded to fp32 (2^-24); where the cosine is smallest here, -0.051 at 1.62,
    that moves it by 1.62 * 2^-24 / 0.051 < 2^-18.9 relative (the sine less, 2^-19.6 at 3), and sine and product
    round by 2^-23 and 2^-24. Beside bf16's half step, 2^-8, all of that is below 2^-18."""
    Hq, Hkv = 4, 2
    i = torch.arange(64, dtype=torch.float64)
    inv = (500000.0 ** (-i / 64)).float() if first == "theta" else (2.0 ** (-i * 0.625)).float()
    pos = torch.tensor([[-3, -2, -1, 0, 1, 2, 3]])
    n = pos.shape[1]
    g = torch.Generator().manual_seed(7)
    x = torch.randn(1, n, Hq + Hkv, D, generator=g).bfloat16()
    low = slice(0, D, 2) if interleaved else slice(0, 64)
    high = slice(1, D, 2) if interleaved else slice(64, D)
    x[..., low] = 0.0
    cache = binding.TieredCache(1, 1, Hq, Hkv, 64, 64, fp_capacity=1, ledger_capacity=1)
    q, k = x.cuda().split([Hq, Hkv], 2)
    got = torch.cat(cache.qk_norm_rope(0, q, k, inv.cuda(), positions=pos.cuda(), interleaved=interleaved), 2)
    y, b = got.double().cpu().numpy(), x[..., high].double().numpy()
    t = pos.double().numpy()[:, :, None, None] * inv.double().numpy()
    bound = 2.0 ** -8 + 2.0 ** -18
    for part, ref in ((low, -b * np.sin(t)), (high, b * np.cos(t))):
        assert np.all(np.abs(y[..., part] - ref) <= bound * np.abs(ref))
    assert cache.status() == 0, cache.last_error()
