"""Attention over the cache in 8 bits where a warp's or a ring's run has many units, so that every slot of shared memory is
filled again and again and the running maximum moves over what was added before: single tokens, and rings that 2 to 8
warps share. Outputs, log-sum-exps and weights against 64 bits (block_exact.py)."""
import pytest
import torch

import block_exact as E
import block_util as U
from tiered_kv_cache_decode_gb300 import binding

pytestmark = pytest.mark.gpu
D, T = 128, 64


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
@pytest.mark.parametrize("Hq,Hkv,n_q,lens", [
    # rows of a KV head: 1, 4, 7, 8 (a ring to a warp), then 10, 20, 28, 35 (five warps), 40, 48, 56, 64
    (2, 2, 1, [70001, 99968]), (32, 8, 1, [16000, 0, 13001]), (28, 4, 1, [40000, 25033]), (16, 2, 1, [98000, 63]),
    (8, 4, 5, [30000, 20001]), (32, 8, 5, [12345, 12352]), (28, 4, 4, [33000, 15001]), (28, 4, 5, [24000, 24010]),
    (16, 2, 5, [97001]), (32, 4, 6, [5, 49000]), (28, 4, 8, [30000, 20050]), (16, 2, 8, [64000, 36001])])
def test_runs_of_many_units(fmt, Hq, Hkv, n_q, lens):
    B, G = len(lens), Hq // Hkv
    units = sum(Hkv * -(-L // T) for L in lens)
    assert units > 2 * 1216   # what all rings hold at a time on 152 SMs (16 slots, two to a unit), twice
    c = binding.BlockCache(B, 1, Hq, Hkv, max(lens), fmt, score_queries=n_q)
    k, v, q = rand(1, B, max(lens), Hkv, D), rand(2, B, max(lens), Hkv, D), rand(3, B, n_q, Hq, D)
    # keys and values of unlike scales from block to block; logits that grow towards the end move the maximum all along
    block = torch.arange(max(lens)) // T
    k = (k * (0.5 + block / block.max())[None, :, None, None]).bfloat16()
    v = (v * 2.0 ** (block % 7 - 3)[None, :, None, None]).bfloat16()
    c.append(0, k.cuda(), v.cuda(), n_new=ints(*lens))
    w = torch.full((B, Hkv, c.capacity), 7.0, device="cuda")
    out, lse = c.attend(0, q.cuda(), ints(*lens), weights=w, accumulate=False)
    again = c.attend(0, q.cuda(), ints(*lens))
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1]) and c.status() == 0
    ref = U.Cache(B, Hkv, c.capacity, fmt)
    ref.append(k, v, [0] * B, lens)
    for b, L in enumerate(lens):
        assert torch.all(w[b, :, L:] == 7.0)
        if L == 0:
            assert not out[b].any() and torch.all(torch.isneginf(lse[b]))
            continue
        ks, vs = (torch.from_numpy(ref.values(x, b, L)) for x in "kv")
        for h in range(Hkv):
            hs = slice(h * G, (h + 1) * G)
            E.check(q[b, :, hs], ks[h], vs[h], out[b, :, hs], lse[b, hs].T, w[b, h, :L])
