"""Calls on the cache in 8 bits as programs make them: a prompt, its eviction and decode steps together; streams,
captured graphs, a process whose first calls are captured; handles side by side; refusals; many, empty and very long
sequences; rows that do not touch one another. Against plain forms in 64 bits with the tolerances of
test_gpu_block.py, or bit by bit against the same call in its usual form."""
import ctypes
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import block_util as U
import span_util
from tiered_kv_cache_decode_gb300 import binding

pytestmark = pytest.mark.gpu
D, T = 128, 64
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(autouse=True, scope="module")
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from tiered_kv_cache_decode_gb300 import build
    build.build()
    binding.load()


def ints(*x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def rand(seed, *shape, scale=1.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * scale).bfloat16()


def f64(t):
    return t.detach().cpu().double().numpy()


class Head:
    """One KV head of one sequence: the values of its full blocks, and the open block's bf16 rows."""

    def __init__(self, fmt):
        self.fmt, self.closed, self.open = fmt, np.zeros((0, D), np.float32), np.zeros((0, D), np.float32)

    def append(self, rows):
        x = np.concatenate([self.open, rows])
        full = len(x) // T * T
        self.closed = np.concatenate([self.closed, U.held(x[:full], self.fmt)])
        self.open = x[full:]

    def keep(self, at):
        self.closed = U.held(self.closed[at], self.fmt)

    def values(self):
        return np.concatenate([self.closed, self.open])


def check(q, k, v, out, lse):
    """One sequence: q [n_q][Hq][128], k, v [Hkv] lists of rows. Returns the weights and their relative tolerance."""
    want, wl, ww, mag, low, big = U.attention(f64(q), np.stack(k), np.stack(v))
    off = 2.0 ** -20 * big
    assert np.all(np.abs(f64(out) - want) <= 2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 2 * off) * mag + 2.0 ** -25 * low + 1e-5)
    seen = np.isfinite(wl)
    assert np.all(np.abs(f64(lse)[seen] - wl[seen]) <= 1e-5 + 2.0 ** -22 * np.abs(wl[seen]) + off)
    return ww, 2 * off + 2.0 ** -21 + 2.0 ** -22 * np.abs(wl[seen]).max(initial=0)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_prompt_eviction_and_decode_together(fmt):
    """Projections -> norms and rotation -> span attention over the prompt; its keys and values into the cache; weights
    from its last 8 queries; eviction; decode steps that append and accumulate; a second eviction in place."""
    B, Hq, Hkv, n, keep, recent = 2, 8, 2, 700, 192, 30
    lens = [700, 431]
    tiers = binding.TieredCache(B, 1, Hq, Hkv, 64, n, fp_capacity=1, ledger_capacity=1)
    cache = binding.BlockCache(B, 1, Hq, Hkv, n + 100, fmt, score_queries=8)
    inv = (10000.0 ** (-torch.arange(0, D, 2) / D)).cuda()
    x = rand(1, B, n, Hq + 2 * Hkv, D).cuda()
    q, k, v = tiers.qk_norm_rope(0, *x.split([Hq, Hkv, Hkv], 2)[:2], inv, v=x[:, :, Hq + Hkv:],
                                 positions=torch.arange(n, device="cuda").expand(B, n).contiguous())
    kv_len = ints(*lens)
    weights = torch.zeros(B, Hkv, cache.capacity, device="cuda")
    out, lse = tiers.span_attention(0, q, k, v, q_len=kv_len, kv_len=kv_len)
    cache.append(0, k, v, n_new=kv_len, weights=weights)
    model = [[(Head(fmt), Head(fmt)) for _ in range(Hkv)] for _ in range(B)]
    for b, L in enumerate(lens):
        for h in range(Hkv):
            for y, head in zip((k, v), model[b][h]):
                head.append(y[b, :L, h].float().cpu().numpy())

    def attend(qs, w, wref):
        o, s = cache.attend(0, qs, kv_len, weights=w)
        for b in range(B):
            ww, rel = check(qs[b], [model[b][h][0].values() for h in range(Hkv)],
                            [model[b][h][1].values() for h in range(Hkv)], o[b], s[b])
            L = ww.shape[1]
            wref[b][:, :L] += ww
            assert np.all(np.abs(f64(w[b, :, :L]) - wref[b][:, :L]) <= (rel + 2.0 ** -18) * wref[b][:, :L] + 1e-30)
        return o

    def evict(wref):
        nonlocal kv_len
        new_len, kept = cache.evict(0, kv_len, keep, recent, weights)
        wd = before.cpu().numpy()
        for b in range(B):
            L = int(kv_len[b])
            c = L // T * T
            for h in range(Hkv):
                at = U.select(wd[b, h], c, keep, recent)
                got = kept[b, h].cpu().numpy()
                assert np.array_equal(got[:len(at)], at) and np.all(got[len(at):] == -1)
                if c > keep:
                    for head in model[b][h]:
                        head.keep(at)
                moved = np.concatenate([wref[b][h, at], wref[b][h, c:L]])
                wref[b][h] = 0
                wref[b][h, :len(moved)] = moved
            assert int(new_len[b]) == len(model[b][0][0].values())
        kv_len = new_len

    last = torch.stack([q[b, L - 8:L] for b, L in enumerate(lens)])
    wref = [np.zeros((Hkv, cache.capacity)) for _ in range(B)]
    o8 = attend(last, weights, wref)
    # the cache's bf16 values through the attention over uncompressed keys: the same rows within the formats' step
    kb, vb = cache.read(0, kv_len, n)
    o2, _ = tiers.span_attention(0, last, kb, vb, q_len=ints(8, 8), kv_len=kv_len)
    for b, L in enumerate(lens):
        ref, _ = span_util.attention(f64(last[b:b + 1]), f64(kb[b:b + 1, :L]), f64(vb[b:b + 1, :L]), [8], [L], 0, 0)
        mag, _ = span_util.attention(f64(last[b:b + 1]), f64(kb[b:b + 1, :L]), np.abs(f64(vb[b:b + 1, :L])), [8], [L], 0, 0)
        assert np.all(np.abs(f64(o2[b]) - ref[0]) <= 2.0 ** -8 * (np.abs(ref[0]) + mag[0]) + 1e-5)
    assert o8.shape == o2.shape
    before = weights.clone()
    evict(wref)
    for step in range(70):
        qs, ks, vs = (rand(100 + 3 * step + i, B, h, D).cuda() for i, h in enumerate((Hq, Hkv, Hkv)))
        cache.append(0, ks, vs, start=kv_len, weights=weights)
        kv_len = kv_len + 1
        for b in range(B):
            for h in range(Hkv):
                for y, head in zip((ks, vs), model[b][h]):
                    head.append(y[b, h:h + 1].float().cpu().numpy())
                wref[b][h, int(kv_len[b]) - 1] = 0
        if step % 9 == 0 or step > 60:
            attend(qs[:, None], weights, wref)
    before = weights.clone()
    evict(wref)
    attend(rand(99, B, 1, Hq, D).cuda(), weights, wref)
    assert cache.status() == 0 and tiers.status() == 0


def decode(cache, qs, ks, vs, kv_len, weights, outs):
    cache.append(0, ks, vs, start=kv_len, weights=weights)
    kv_len += 1
    cache.attend(0, qs, kv_len, out=outs[0], lse=outs[1], weights=weights)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_captured_decode_follows_the_lengths(fmt):
    B, Hq, Hkv, n = 3, 8, 2, 200
    lens = [130, 0, 63]
    k, v = rand(1, B, n, Hkv, D).cuda(), rand(2, B, n, Hkv, D).cuda()
    qs, ks, vs = rand(3, B, 1, Hq, D).cuda(), rand(4, B, 1, Hkv, D).cuda(), rand(5, B, 1, Hkv, D).cuda()
    runs = []
    for captured in (False, True):
        cache = binding.BlockCache(B, 1, Hq, Hkv, 400, fmt)
        kv_len, weights = ints(*lens), torch.zeros(B, Hkv, cache.capacity, device="cuda")
        outs = torch.empty_like(qs), torch.empty(B, Hq, 1, device="cuda")
        q1, k1, v1 = qs.clone(), ks.clone(), vs.clone()
        cache.append(0, k, v, n_new=kv_len)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        if captured:
            with torch.cuda.graph(graph):
                decode(cache, q1, k1, v1, kv_len, weights, outs)
        got = []
        for step in range(5):
            for x, y in ((q1, qs), (k1, ks), (v1, vs)):
                x.copy_(y * (step + 1))
            if captured:
                graph.replay()
            else:
                decode(cache, q1, k1, v1, kv_len, weights, outs)
            got += [outs[0].clone(), outs[1].clone(), weights.clone()]
        new_len, kept = cache.evict(0, kv_len, 64, 5, weights)
        got += [new_len, kept, weights, *cache.read(0, new_len, 200)]
        assert cache.status() == 0
        runs.append(got)
    assert all(torch.equal(a, b) for a, b in zip(*runs))


def test_captured_eviction_repeats():
    B, Hkv, n = 2, 2, 1500
    src, dst = (binding.BlockCache(B, 1, Hkv, Hkv, c) for c in (n, 320))
    src.append(0, rand(1, B, n, Hkv, D).cuda(), rand(2, B, n, Hkv, D).cuda())
    kv_len, w = ints(n, 800), torch.rand(B, Hkv, src.capacity, device="cuda")
    w_out = torch.zeros(B, Hkv, dst.capacity, device="cuda")
    new_len, kept = ints(0, 0), torch.zeros(B, Hkv, 256, dtype=torch.int32, device="cuda")

    def run():
        src.evict(0, kv_len, 256, 20, w, into=dst, new_len=new_len, kept=kept, weights_out=w_out)

    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for seed in range(3):
        w.copy_(torch.rand(w.shape, generator=torch.Generator().manual_seed(seed)))
        graph.replay()
        got = [x.clone() for x in (new_len, kept, w_out, *dst.read(0, new_len, 320))]
        run()
        want = [new_len, kept, w_out, *dst.read(0, new_len, 320)]
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert src.status() == 0 and dst.status() == 0


def test_streams_layers_and_handles_side_by_side():
    """Two handles on two streams at once, other layers, outputs made on the call's stream."""
    B, Hq, Hkv, n = 2, 16, 4, 3000
    caches = [binding.BlockCache(B, 3, Hq, Hkv, n, f) for f in ("int8", "e4m3")]
    k, v, q = (rand(i, B, n, h, D).cuda() for i, h in ((1, Hkv), (2, Hkv), (3, Hq)))
    kv_len = ints(n, 1234)
    want = []
    for c in caches:
        c.append(2, k, v)
        w = torch.zeros(B, Hkv, c.capacity, device="cuda")
        want.append([*c.attend(2, q[:, :1].contiguous(), kv_len, weights=w), w, *c.read(2, kv_len, n)])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in caches]
    got = []
    for c, s in zip(caches, streams):
        w = torch.zeros(B, Hkv, c.capacity, device="cuda")
        qs = q[:, :1].contiguous()
        s.wait_stream(torch.cuda.current_stream())
        for layer in (0, 1):
            c.append(layer, k, v, stream=s)
        for _ in range(10):
            c.attend(0, qs, kv_len, stream=s)
        got.append([*c.attend(1, qs, kv_len, weights=w, stream=s), w, *c.read(1, kv_len, n, stream=s)])
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert all(c.status() == 0 for c in caches)


def test_one_token_forms_and_given_outputs():
    B, Hq, Hkv = 2, 8, 2
    c = binding.BlockCache(B, 1, Hq, Hkv, 100)
    k, v, q = rand(1, B, Hkv, D).cuda(), rand(2, B, Hkv, D).cuda(), rand(3, B, Hq, D).cuda()
    c.append(0, k, v)
    out, lse = c.attend(0, q, ints(1, 1))
    o2, l2 = c.attend(0, q[:, None], ints(1, 1))
    assert out.shape == q.shape and torch.equal(out, o2[:, 0]) and torch.equal(lse, l2)
    assert torch.equal(out.view(B, Hkv, 4, D), v[:, :, None].expand(B, Hkv, 4, D))   # one token: its value
    mine = torch.empty_like(q), torch.empty(B, Hq, 1, device="cuda")
    got = c.attend(0, q, ints(1, 1), out=mine[0], lse=mine[1])
    assert got[0] is mine[0] and got[1] is mine[1] and torch.equal(mine[0], out) and torch.equal(mine[1], lse)
    bare, none = c.attend(0, q, ints(1, 1), want_lse=False)
    assert none is None and torch.equal(bare, out)


@pytest.mark.parametrize("fmt,Hq,Hkv,n_q", [("int8", 4, 1, 1), ("e4m3", 6, 2, 3)])
def test_many_sequences_some_empty(fmt, Hq, Hkv, n_q):
    """More sequences than lanes, runs that begin and end anywhere, whole pairs inside a run, rows of empty ones."""
    B = 333
    g = torch.Generator().manual_seed(5)
    lens = torch.randint(0, 400, (B,), generator=g)
    lens[torch.rand(B, generator=g) < 0.3] = 0
    lens[40:110] = 0
    lens = lens.tolist()
    c = binding.BlockCache(B, 1, Hq, Hkv, 400, fmt, score_queries=n_q)
    k, v, q = rand(1, B, 400, Hkv, D), rand(2, B, 400, Hkv, D), rand(3, B, n_q, Hq, D)
    c.append(0, k.cuda(), v.cuda(), n_new=ints(*lens))
    w = torch.zeros(B, Hkv, c.capacity, device="cuda")
    out, lse = c.attend(0, q.cuda(), ints(*lens), weights=w)
    ref = U.Cache(B, Hkv, c.capacity, fmt)
    ref.append(k, v, [0] * B, lens)
    for b, L in enumerate(lens):
        if L == 0:
            assert not out[b].any() and torch.all(torch.isneginf(lse[b])) and not w[b].any()
            continue
        ww, rel = check(q[b], list(ref.values("k", b, L)), list(ref.values("v", b, L)), out[b], lse[b])
        assert np.all(np.abs(f64(w[b, :, :L]) - ww) <= rel * ww + 1e-30) and not w[b, :, L:].any()
    # no sequence at all
    c.attend(0, q.cuda(), torch.zeros(B, dtype=torch.int32, device="cuda"), out=out, lse=lse)
    assert not out.any() and torch.all(torch.isneginf(lse)) and c.status() == 0


@pytest.mark.parametrize("n_q", [1, 5])
def test_rows_do_not_touch_one_another(n_q):
    """Other queries, other heads' queries and a query of NaN and infinities change no bit of a row."""
    B, Hq, Hkv, n = 2, 16, 2, 1000
    c = binding.BlockCache(B, 1, Hq, Hkv, n, "e4m3", score_queries=n_q)
    c.append(0, rand(1, B, n, Hkv, D).cuda(), rand(2, B, n, Hkv, D).cuda())
    q = rand(3, B, n_q, Hq, D).cuda()
    kv_len = ints(n, n - 37)
    out, lse = c.attend(0, q, kv_len)
    other = (rand(4, B, n_q, Hq, D).float() * 20).bfloat16().cuda()
    other[:, :, 1::2, ::3] = float("nan")
    other[:, :, 2::3, 1::5] = float("inf")
    mine = torch.zeros(n_q, Hq, dtype=torch.bool)
    mine[n_q // 2, 5] = mine[-1, 9] = True
    mixed = torch.where(mine.cuda()[None, :, :, None], q, other)
    o2, l2 = c.attend(0, mixed, kv_len)
    for i, h in mine.nonzero().tolist():
        assert torch.equal(o2[:, i, h], out[:, i, h]) and torch.equal(l2[:, h, i], lse[:, h, i])
        assert torch.isfinite(o2[:, i, h]).all()
    bad = ~torch.isfinite(mixed.float()).all(-1)
    assert torch.isnan(o2[bad].float()).all()


def test_offsets_past_32_bits():
    """The last KV heads and tokens of a cache of 4.3 GB, with its weights, read back and evicted."""
    B, Hq, Hkv, n = 1, 8, 8, 2 ** 21
    c = binding.BlockCache(B, 1, Hq, Hkv, n, "int8")
    g = torch.Generator(device="cuda").manual_seed(1)
    for at in range(0, n, 2 ** 18):
        k = torch.randn(B, 2 ** 18, Hkv, D, generator=g, device="cuda").bfloat16()
        c.append(0, k, k, start=ints(at))
    tail = torch.randn(B, 200, Hkv, D, generator=g, device="cuda").bfloat16() * 4
    c.append(0, tail, tail, start=ints(n - 200 - 20))
    L = n - 20
    q = (tail[:, 150:151] * 0.5).contiguous()   # peaks on a token near the end
    w = torch.zeros(B, Hkv, c.capacity, device="cuda")
    out, lse = c.attend(0, q, ints(L), weights=w)
    kb, vb = c.read(0, ints(L), 300, first=ints(L - 300))
    assert torch.equal(kb, vb)
    for h in (0, 7):
        full, _ = c.read(0, ints(L), n)
        x = full[0, :L, h].double()
        logits = (x @ q[0, 0, h].double()) / np.sqrt(D)
        p = logits.softmax(0)
        # bf16 of the codes' values: 2^-9 of each term at most, in the logits too (the largest about 45 times 0.5 sqrt)
        slack = 2.0 ** -8 * (x.abs() @ q[0, 0, h].double().abs()).max().item() / np.sqrt(D)
        assert abs(lse[0, h, 0].item() - logits.logsumexp(0).item()) <= slack + 1e-4
        j = L - 200 + 150
        assert p[j] > 0.5 and abs(w[0, h, j].item() - p[j].item()) <= 2 * slack * p[j].item() + 1e-5
        assert abs(w[0, h].sum().item() - 1) <= 1e-4 and not w[0, h, L:].any()
        del x, full
    small = binding.BlockCache(B, 1, Hq, Hkv, 320, "int8")
    new_len, kept = c.evict(0, ints(L), 256, 64, w, into=small)
    c0 = L // T * T
    assert int(new_len) == 256 + L - c0 and torch.all(kept[0, :, -64:] == torch.arange(c0 - 64, c0, device="cuda"))
    assert torch.all((kept[0] == L - 50).any(1)) and torch.all(kept[0, :, 1:] > kept[0, :, :-1])
    top = torch.sort(w[0, :, :c0 - 64], dim=1, descending=True, stable=True).indices[:, :192].sort(1).values
    assert torch.equal(kept[0, :, :192].long(), top)
    assert c.status() == 0 and small.status() == 0


def test_refusals():
    B, Hq, Hkv = 2, 8, 2
    c = binding.BlockCache(B, 2, Hq, Hkv, 200, "int8", score_queries=2)
    other = binding.BlockCache(B, 1, Hq, Hkv, 128, "e4m3")
    wide = binding.BlockCache(B, 1, Hq, 4, 512, "int8")
    assert c.capacity == 256
    lib, H = c.lib, c.handle
    k = rand(1, B, 8, Hkv, D).cuda()
    q, n = rand(2, B, 1, Hq, D).cuda(), ints(8, 8)
    w = torch.zeros(B, Hkv, 256, device="cuda")
    out, lse = torch.empty_like(q), torch.empty(B, Hq, 1, device="cuda")
    kept, new = torch.zeros(B, Hkv, 128, dtype=torch.int32, device="cuda"), ints(0, 0)
    p = lambda t, off=0: None if t is None else ctypes.c_void_p(t.data_ptr() + off)   # noqa: E731
    bad = [
        lib.qevict_block_append(H, 2, p(k), 256, p(k), 256, 8, None, None, None, None),
        lib.qevict_block_append(H, -1, p(k), 256, p(k), 256, 8, None, None, None, None),
        lib.qevict_block_append(H, 0, None, 256, p(k), 256, 8, None, None, None, None),
        lib.qevict_block_append(H, 0, p(k, 2), 256, p(k), 256, 7, None, None, None, None),
        lib.qevict_block_append(H, 0, p(k), 255, p(k), 256, 7, None, None, None, None),
        lib.qevict_block_append(H, 0, p(k), 128, p(k), 256, 8, None, None, None, None),
        lib.qevict_block_append(H, 0, p(k), 256, p(k), 260, 7, None, None, None, None),
        lib.qevict_block_append(H, 0, p(k), 256, p(k), 256, 0, None, None, None, None),
        lib.qevict_block_append(H, 0, p(k), 256, p(k), 256, 2 ** 21 + 1, None, None, None, None),
        lib.qevict_block_append(H, 0, p(k), 256, p(k), 256, 8, None, None, p(k), None),
        lib.qevict_block_append(H, 0, p(k), 256, p(k), 256, 8, p(n, 1), None, None, None),
        lib.qevict_block_attention(H, 0, p(q), 0, p(n), p(out), None, None, 0, None),
        lib.qevict_block_attention(H, 0, p(q), 9, p(n), p(out), None, None, 0, None),
        lib.qevict_block_attention(H, 0, p(q), 3, p(n), p(out), None, p(w), 0, None),
        lib.qevict_block_attention(H, 0, p(q), 1, None, p(out), None, None, 0, None),
        lib.qevict_block_attention(H, 0, p(q), 1, p(n), p(q), None, None, 0, None),
        lib.qevict_block_attention(H, 0, p(q), 1, p(n), p(out), p(out), None, 0, None),
        lib.qevict_block_attention(H, 0, p(q), 1, p(n), p(out), p(lse), p(lse), 0, None),
        lib.qevict_block_attention(H, 0, p(q), 1, p(n), p(out, 8), None, None, 0, None),
        lib.qevict_block_read(H, 0, p(n), None, 0, p(k), p(q), None),
        lib.qevict_block_read(H, 0, p(n), None, 8, p(k), p(k), None),
        lib.qevict_block_read(H, 0, None, None, 8, p(k), p(q), None),
    ]
    assert bad == [1] * len(bad)

    def evict(keep=128, recent=0, weights=w, to=c, layer=0, w_out=None, new_len=new, kept_=kept):
        return lib.qevict_block_evict(H, 0, p(n), keep, recent, p(weights), to.handle, layer, p(w_out), p(new_len),
                                      p(kept_), None)

    bad = [evict(0), evict(100), evict(256), evict(recent=-1), evict(recent=129), evict(to=other), evict(to=wide),
           evict(layer=2), evict(weights=None), evict(new_len=None), evict(kept_=None), evict(w_out=kept),
           evict(new_len=n), evict(kept_=w), evict(w_out=w[:, :, :192])]
    assert bad[:-1] == [1] * (len(bad) - 1) and bad[-1] == 0   # the last names the weights' own address: in place
    torch.cuda.synchronize()
    for call in (lambda: c.evict(0, n, 192 + 64, 0, w), lambda: c.evict(0, n, 100, 0, w), lambda: c.attend(5, q, n),
                 lambda: c.attend(0, rand(3, B, 3, Hq, D).cuda(), n, weights=w)):
        with pytest.raises(binding.QevictError, match="INVALID_ARG"):
            call()
    assert c.status() == 0 and other.status() == 0 and wide.status() == 0


FIRST = """
import torch
from tiered_kv_cache_decode_gb300 import binding
B, Hq, Hkv, n, n_q, fmt = %s
g = torch.Generator().manual_seed(1)
x = torch.randn(B, n, Hq + 2 * Hkv, 128, generator=g).bfloat16().cuda()
q, k, v = x[:, -n_q:, :Hq].contiguous(), x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:]
c, d = (binding.BlockCache(B, 1, Hq, Hkv, n, fmt, score_queries=n_q) for _ in range(2))
lens = torch.full((B,), n, dtype=torch.int32).cuda()
w = torch.zeros(B, Hkv, c.capacity, device="cuda")

def layer():
    c.append(0, k, v)
    out, lse = c.attend(0, q, lens, weights=w, accumulate=False)
    new_len, kept = c.evict(0, lens, 64, 10, w, into=d)
    return (out, lse, new_len, kept, *d.read(0, new_len, 128))

torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = layer()
graph.replay()
torch.cuda.synchronize()
want = layer()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, want)) and c.status() == 0 and d.status() == 0
print("same bits")
"""


@pytest.mark.parametrize("sizes", ["(1, 8, 2, 300, 1, 'int8')", "(3, 28, 4, 777, 4, 'e4m3')"])
def test_first_calls_of_a_process_are_captured(sizes):
    r = subprocess.run([sys.executable, "-c", FIRST % sizes], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same bits" in r.stdout, r.stdout + r.stderr


@pytest.mark.parametrize("lens", [[130, 64], [500, 40]])
def test_in_place_eviction_with_weights_elsewhere(lens):
    """In place, the weights go to another tensor also where nothing leaves; into another layer they may not go to their
    own (the moves are in no order)."""
    B, Hkv, keep = 2, 2, 128
    c = binding.BlockCache(B, 2, Hkv, Hkv, 512)
    c.append(0, rand(1, B, 500, Hkv, D).cuda(), rand(2, B, 500, Hkv, D).cuda())
    w = torch.rand(B, Hkv, c.capacity, generator=torch.Generator().manual_seed(1)).cuda()
    out, kept_w = torch.full_like(w, 7.0), w.clone()
    new_len, kept = c.evict(0, ints(*lens), keep, 10, w, weights_out=out)
    assert torch.equal(w, kept_w)
    for b, L in enumerate(lens):
        full = L // T * T
        for h in range(Hkv):
            at = U.select(w[b, h].cpu().numpy(), full, keep, 10)
            want = torch.cat([w[b, h][torch.from_numpy(at).cuda()], w[b, h, full:L]])
            assert torch.equal(out[b, h, :len(want)], want) and torch.all(out[b, h, len(want):] == 7.0)
            assert int(new_len[b]) == len(want)
    with pytest.raises(binding.QevictError, match="INVALID_ARG"):
        c.evict(0, ints(*lens), keep, 10, w, into=c, into_layer=1, weights_out=w)
    assert c.status() == 0


def test_attention_and_eviction_clamp_lengths():
    B, Hq, Hkv, n = 3, 8, 2, 320
    c = binding.BlockCache(B, 1, Hq, Hkv, n)
    k = rand(1, B, n, Hkv, D).cuda()
    c.append(0, k, k)
    q = rand(2, B, 1, Hq, D).cuda()
    got, want = c.attend(0, q, ints(-7, 2 ** 31 - 1, n + 1)), c.attend(0, q, ints(0, n, n))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    d = binding.BlockCache(B, 2, Hkv, Hkv, 128)
    w = torch.rand(B, Hkv, n, device="cuda")
    got = c.evict(0, ints(-2 ** 31, 2 ** 31 - 1, n + 64), 64, 3, w, into=d)
    want = c.evict(0, ints(0, n, n), 64, 3, w, into=d, into_layer=1)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert all(torch.equal(a, b) for a, b in zip(d.read(0, got[0], 128), d.read(1, want[0], 128)))
