"""Attention over the cache in 8 bits with logits of any size that fp32 holds: the header's bound, max |q| max |k| below
2^120, and rows past it, which reach no other."""
import math

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


def ints(*x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def rand(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).bfloat16()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("eq,ek", [(0, 119), (119, 0), (60, 59), (-8, 127), (127, -8), (-120, 120), (-120, -120), (40, 20)])
@pytest.mark.parametrize("n,at", [(40, 17), (64, 63), (200, 130), (200, 198), (20000, 12345)])
def test_the_largest_logit_takes_all(fmt, eq, ek, n, at):
    """One token's key agrees with the query, all others' oppose it: logits x and -x, so that it has 1 / (1 + (n - 1)
    exp(-2 x)) of the mass: all of it, or where x is all but 0 no more than each other."""
    q, k = torch.full((1, 1, 4, D), 2.0 ** eq), torch.full((1, n, 1, D), -(2.0 ** ek))
    k[:, at] = 2.0 ** ek
    v = rand(1, 1, n, 1, D)
    c = binding.BlockCache(1, 1, 4, 1, n, fmt)
    c.append(0, k.bfloat16().cuda(), v.cuda())
    out, lse = c.attend(0, q.bfloat16().cuda(), ints(n))
    held = c.read(0, ints(n), n)[1][0, :, 0].double().cpu()
    x = 2.0 ** (eq + ek) * D ** 0.5
    rest = (n - 1) * math.exp(-2 * x)
    p = torch.full((n, 1), rest / (1 + rest) / (n - 1), dtype=torch.float64)
    p[at] = 1 / (1 + rest)
    want, mag = (p * held).sum(0), (p * held.abs()).sum(0)
    # bf16 of the output and of the values that were read back; probabilities off by 2^-11, sums of up to 20,000 by 2^-10
    allowed = 2.0 ** -7 * want.abs() + 2.0 ** -8 * mag
    assert torch.all((out[0, 0].double().cpu() - want).abs() <= allowed)
    top = x + math.log1p(rest)
    assert torch.all((lse.double() - top).abs() <= 2.0 ** -12 * top + 1e-5) and c.status() == 0


@pytest.mark.parametrize("n", [50, 3000])
def test_rows_past_fp32_reach_no_other(n):
    q, k, v = rand(1, 1, 1, 8, D).cuda(), rand(2, 1, n, 1, D).cuda(), rand(3, 1, n, 1, D).cuda()
    c = binding.BlockCache(1, 1, 8, 1, n)
    c.append(0, k, v)
    out, lse = c.attend(0, q, ints(n))
    big = q.clone()
    big[:, :, 1::2] = (q[:, :, 1::2].float() * 2.0 ** 124).bfloat16()
    o2, l2 = c.attend(0, big, ints(n))
    assert torch.equal(o2[:, :, ::2], out[:, :, ::2]) and torch.equal(l2[:, ::2], lse[:, ::2])
