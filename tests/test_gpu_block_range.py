"""Attention over the cache in 8 bits with values of any magnitude that a cache holds, the largest and the smallest of
bf16 among them: an output is a mean of finite values, so it is finite, and as near to 64 bits as with values around 1
(tolerances: block_exact.py)."""
import numpy as np
import pytest
import torch

import block_exact as E
import block_util as U
from tiered_kv_cache_decode_gb300 import binding

pytestmark = pytest.mark.gpu
D, T = 128, 64
FORMATS = ["int8", "e4m3"]
LARGE = [2.0 ** 100, 2.0 ** 115, 2.4e38]
SMALL = [2.0 ** -100, 2.0 ** -112, 2.0 ** -126]


@pytest.fixture(autouse=True, scope="module")
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from tiered_kv_cache_decode_gb300 import build
    build.build()
    binding.load()


def ints(*x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def rand(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).bfloat16()


def attended(fmt, q, k, v, lens=None):
    """The call on a cache that holds k, v [B][n][Hkv][128], held to 64 bits."""
    B, n, Hkv, _ = k.shape
    n_q, Hq = q.shape[1:3]
    G, lens = Hq // Hkv, lens or [n] * B
    c = binding.BlockCache(B, 1, Hq, Hkv, n, fmt, score_queries=n_q)
    c.append(0, k.cuda(), v.cuda(), n_new=ints(*lens))
    w = torch.zeros(B, Hkv, c.capacity, device="cuda")
    out, lse = c.attend(0, q.cuda(), ints(*lens), weights=w)
    assert c.status() == 0, c.last_error()
    ref = U.Cache(B, Hkv, c.capacity, fmt)
    ref.append(k, v, [0] * B, lens)
    for b, L in enumerate(lens):
        ks, vs = (torch.from_numpy(ref.values(x, b, L)) for x in "kv")
        for h in range(Hkv):
            hs = slice(h * G, (h + 1) * G)
            E.check(q[b, :, hs], ks[h], vs[h], out[b, :, hs], lse[b, hs].T, w[b, h, :L])
    return out


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("scale", [2e34, *LARGE, 3.3e38, *SMALL])
def test_one_token_gives_its_value_back(fmt, scale):
    v = torch.where(rand(1, 1, 1, 2, D) > 0, scale, -scale).bfloat16()
    out = attended(fmt, rand(2, 1, 1, 8, D), rand(3, 1, 1, 2, D), v)
    assert torch.equal(out.cpu().view(1, 2, 4, D), v.view(1, 2, 1, D).expand(1, 2, 4, D))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("scale", LARGE + SMALL)
@pytest.mark.parametrize("n,n_q", [(20, 1), (63, 3), (64, 1), (193, 5), (1000, 2), (30011, 1), (9000, 8)])
def test_values_of_one_magnitude(fmt, scale, n, n_q):
    """An open block, full blocks, a pair in one run and in many, single tokens and drafts; values of both signs and, in
    the second KV head, of one (a sum of thousands of them passes what fp32 holds)."""
    v = (rand(1, 1, n, 2, D).float().clamp(-1.4, 1.4) * scale)
    v[:, :, 1] = v[:, :, 1].abs()
    attended(fmt, rand(2, 1, n_q, 8, D), rand(3, 1, n, 2, D), v.bfloat16())


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("first,then", [(1.0, 2.4e38), (2.4e38, 1.0), (2.0 ** 70, 2.4e38), (2.0 ** -126, 2.0 ** -100)])
@pytest.mark.parametrize("n_q", [1, 4])
def test_magnitudes_that_change_along_a_sequence(fmt, first, then, n_q):
    """Runs of several blocks (more than 3,000 in all) in which the magnitude changes: every third block has the other
    one, the open block too. Logits around 0, so that every token counts."""
    B, Hkv, n = 3, 8, 8 * 1024 + 40
    v = rand(1, B, n, Hkv, D).float().clamp(-1.4, 1.4)
    other = (torch.arange(n) // T % 3 == 2) | (torch.arange(n) >= n // T * T)
    v = (v * torch.where(other, then, first)[None, :, None, None]).bfloat16()
    attended(fmt, rand(2, B, n_q, 32, D) * 0.1, rand(3, B, n, Hkv, D), v, [n, n - 45, n - 64])


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("at", [300, 8000])
def test_masses_that_fall_on_values_around_one(fmt, at):
    """Values near the largest of bf16 in a block whose tokens get no mass beside those around 1: the outputs are those
    of the others, as near as ever. Tokens before, in and behind that block's run."""
    n = 8 * 1024 + 10
    q = torch.zeros(1, 1, 4, D)
    q[..., 0] = 8.0
    k = rand(1, 1, n, 1, D).float()
    k[..., 0] = 1.0
    v = rand(2, 1, n, 1, D).float().clamp(-1.4, 1.4)
    k[:, at:at + 8, :, 0] = -800.0   # e^-560 of the others
    k[:, at:at + 8, :, 1:] = 0.0
    v[:, at:at + 8] *= 2.4e38
    blk = slice(at // T * T, at // T * T + T)
    k[:, blk, :, 0] = -800.0   # the whole block: its other tokens share the scales
    attended(fmt, q.bfloat16(), k.bfloat16(), v.bfloat16())


@pytest.mark.parametrize("fmt", FORMATS)
def test_equal_values_come_back(fmt):
    """Tokens that all have one value: the output is that value, whatever it is. 127 s and 448 s are the value itself to
    a step of fp32."""
    for n in (7, 64, 640, 5000):
        for value in (2.4e38, -3.3e38, 2.0 ** 113, 2.0 ** -120):
            v = torch.full((1, n, 1, D), value).bfloat16()
            out = attended(fmt, rand(2, 1, 1, 4, D), rand(3, 1, n, 1, D), v)
            near = np.abs(out.cpu().double().numpy() / v[0, 0, 0, 0].double().item() - 1)
            assert near.max() <= 2.0 ** -7
