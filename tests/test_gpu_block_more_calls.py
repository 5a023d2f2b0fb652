"""Calls on the cache in 8 bits that its documentation allows and that stood untested: weights at any 4-byte boundary,
several attention calls of one graph that share a handle's scratch, evictions of short sequences in a cache with room for
more keys than shared memory holds, caches whose memory others filled before. Bit by bit against the usual form."""
import pytest
import torch

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


@pytest.mark.parametrize("accumulate", [True, False])
@pytest.mark.parametrize("offset", [1, 2, 3])
def test_weights_at_any_word(offset, accumulate):
    B, Hq, Hkv, n = 2, 8, 2, 1000
    c = binding.BlockCache(B, 1, Hq, Hkv, n)
    k, q = rand(1, B, n, Hkv, D).cuda(), rand(2, B, 1, Hq, D).cuda()
    size = B * Hkv * c.capacity
    room = torch.full((size + 8,), 3.0, device="cuda")
    off, own = room[offset:offset + size].view(B, Hkv, c.capacity), torch.full((B, Hkv, c.capacity), 3.0, device="cuda")
    for w in (off, own):
        c.append(0, k, k, n_new=ints(n, 61), weights=w)
        c.attend(0, q, ints(n, 61), weights=w, accumulate=accumulate)
    assert torch.equal(off, own) and torch.all(own[1, :, 61:] == 3.0)
    assert torch.all(room[:offset] == 3.0) and torch.all(room[offset + size:] == 3.0)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_layers_of_a_graph_share_the_scratch(fmt):
    """Four layers of unlike lengths, drafts and single tokens, one behind the other in a graph that is replayed."""
    B, Hq, Hkv, n, layers = 2, 16, 4, 5000, 4
    c = binding.BlockCache(B, layers, Hq, Hkv, n, fmt, score_queries=5)
    qs, lens = [], [ints(n, 3), ints(70, n - 1), ints(0, 4097), ints(129, 128)]
    for i in range(layers):
        c.append(i, rand(3 * i, B, n, Hkv, D).cuda(), rand(3 * i + 1, B, n, Hkv, D).cuda(), n_new=lens[i])
        qs.append(rand(3 * i + 2, B, (1, 5, 2, 1)[i], Hq, D).cuda())
    shape = (B, Hkv, c.capacity)
    w = [torch.zeros(shape, device="cuda") for _ in range(layers)]
    outs = [(torch.zeros_like(q), torch.zeros(B, Hq, q.shape[1], device="cuda")) for q in qs]

    def step():
        for i in range(layers):
            c.attend(i, qs[i], lens[i], out=outs[i][0], lse=outs[i][1], weights=w[i] if i != 2 else None, accumulate=False)

    step()
    torch.cuda.synchronize()
    want = [x.clone() for x in w + [y for o in outs for y in o]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        for x in w + [y for o in outs for y in o]:
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, w + [y for o in outs for y in o]))
    assert c.status() == 0


@pytest.mark.parametrize("lens,keep,recent", [([700, 131], 128, 0), ([4000, 64], 512, 512), ([2047, 3000], 1024, 77),
                                              ([330000, 65], 64, 3)])
def test_eviction_in_a_cache_of_great_capacity(lens, keep, recent):
    """Room for more tokens than the selection keeps in shared memory; equal weights, NaN and infinities."""
    B, Hkv, cap = 2, 2, 400000
    c = binding.BlockCache(B, 1, Hkv, Hkv, cap, "e4m3")
    n = max(lens)
    k, v = rand(1, B, n, Hkv, D).cuda(), rand(2, B, n, Hkv, D).cuda()
    c.append(0, k, v, n_new=ints(*lens))
    w = torch.rand(B, Hkv, c.capacity, generator=torch.Generator().manual_seed(3))
    w = (w * 9).round() / 9
    w[..., ::7], w[..., 1::11], w[..., 2::13] = float("nan"), float("inf"), float("-inf")
    w[..., 3::17] = -0.0
    before = [x.cpu() for x in c.read(0, ints(*lens), n)]
    wc = w.cuda()
    new_len, kept = c.evict(0, ints(*lens), keep, recent, wc)
    m = int(new_len.max())
    after = [x.cpu() for x in c.read(0, new_len, m)]
    for b, L in enumerate(lens):
        full = L // T * T
        assert int(new_len[b]) == min(full, keep) + L - full
        for h in range(Hkv):
            at = torch.from_numpy(U.select(w[b, h].numpy(), full, keep, recent))
            got = kept[b, h].cpu().long()
            assert torch.equal(got[:len(at)], at) and torch.all(got[len(at):] == -1)
            src = torch.cat([at, torch.arange(full, L)])
            assert torch.equal(wc[b, h, :len(src)].cpu().nan_to_num(1e9), w[b, h][src].nan_to_num(1e9))
            for x, y in zip(before, after):   # requantised: within half a step of e4m3 and the bf16 that was read before
                p, a = x[b, src, h].double(), y[b, :len(src), h].double()
                step = torch.maximum(p.abs() * (2.0 ** -4 + 2.0 ** -7), p.abs().max() * 2.0 ** -17)
                assert torch.all((p - a).abs() <= step)
                assert torch.equal(p[len(at):], a[len(at):])
    assert c.status() == 0


def test_what_the_memory_held_before_changes_nothing():
    """A cache in memory that others have filled with NaN: rows behind a length take part in no result."""
    B, Hq, Hkv, n = 2, 8, 2, 300
    k, q = rand(1, B, n, Hkv, D).cuda(), rand(2, B, 3, Hq, D).cuda()
    results = []
    for fill in (0x00, 0xff):
        torch.cuda.empty_cache()
        x = torch.full((64 << 20,), fill, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        del x
        c = binding.BlockCache(B, 1, Hq, Hkv, 1000, score_queries=3)
        w = torch.zeros(B, Hkv, c.capacity, device="cuda")
        c.append(0, k, k, n_new=ints(n, 7))
        results.append([*c.attend(0, q, ints(n, 7), weights=w), w, *c.read(0, ints(n, 7), n)])
        c.close()
    assert all(torch.equal(a, b) for a, b in zip(*results)) and torch.isfinite(results[1][0]).all()
