"""The operators between a layer's projections and its cache on the GPU, against
plain float64 forms: head norms with rotation, span attention, window scores,
and the three in a run with the prefill and the decode after them.

Tolerances. An output is rounded to bf16 once: at most 2^-9 of its magnitude's
power of two, 2^-8 relative, besides the fp32 arithmetic (relative 1e-5 here).
Attention also rounds each probability to bf16 (2^-8 relative at most, so at
most 2^-8 of sum p |v|), so |out - ref| <= 2^-8 (|ref| + sum p |v|) + 1e-5. The
log-sum-exp and the scores are fp32 sums of exact products: with 128 products
of magnitude a few and up to 2^15 terms, an error of 2^-24 per step and of
about 2^-22 in the exponential stays below 1e-5 of the sum; lse takes 1e-5
absolute for that and the rounding of logits up to some tens (2^-24 * 64).
"""
import numpy as np
import pytest
import torch

import oracle as O
import span_util as U
from tiered_kv_cache_decode_gb300 import binding

pytestmark = pytest.mark.gpu
D = 128


@pytest.fixture(autouse=True, scope="module")
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from tiered_kv_cache_decode_gb300 import build
    build.build()
    binding.load()


def cache_for(B, Hq, Hkv, w=64, max_context=4096, **kw):
    kw.setdefault("fp_capacity", 1)
    kw.setdefault("ledger_capacity", 1)
    return binding.TieredCache(B, 1, Hq, Hkv, w, max_context, **kw)


def rand(seed, *shape, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).bfloat16()


def f64(t):
    return t.detach().cpu().double().numpy()


# ---- head norms and rotation ---------------------------------------------------
def freqs(theta=10000.0):
    return (theta ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)).float()


@pytest.mark.parametrize("B,n,Hq,Hkv", [(1, 1, 1, 1), (2, 1, 28, 4), (3, 5, 8, 2), (1, 67, 32, 8), (2, 33, 7, 7),
                                        (1, 300, 24, 3)])
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_rope_matches_plain(B, n, Hq, Hkv, norm, interleaved):
    cache = cache_for(B, Hq, Hkv)
    qkv = rand(n, B, n, Hq + 2 * Hkv, D, scale=3.0)
    q, k, v = qkv.cuda().split([Hq, Hkv, Hkv], 2)
    wq, wk = ((1 + rand(s, D).float() * 0.2).bfloat16() if norm else None for s in (1, 2))
    pos = torch.randint(0, 200000, (B, n), generator=torch.Generator().manual_seed(n))
    inv = freqs(500000.0)
    gq, gk, gv = cache.qk_norm_rope(0, q, k, inv.cuda(), v=v, positions=pos.cuda(), eps=1e-5,
                                    q_weight=None if wq is None else wq.cuda(),
                                    k_weight=None if wk is None else wk.cuda(), interleaved=interleaved)
    x = f64(qkv)
    for got, rows, w in ((gq, x[:, :, :Hq], wq), (gk, x[:, :, Hq:Hq + Hkv], wk)):
        ref = U.norm_rope(rows, None if w is None else f64(w), 1e-5, pos.numpy(), inv.double().numpy(), interleaved)
        size = np.sqrt((rows ** 2).sum(-1, keepdims=True)) if w is None else 30.0   # of a row: bounds a, b
        assert np.all(np.abs(f64(got) - ref) <= 2.0 ** -8 * np.abs(ref) + 2e-6 * size)
    assert torch.equal(gv.cpu(), qkv[:, :, Hq + Hkv:])
    assert cache.status() == 0


def test_norm_rope_far_and_negative_positions():
    cache = cache_for(1, 2, 1)
    pos = torch.tensor([[0, 1, -1, -131072, 2 ** 31 - 1, 2 ** 31, 2 ** 36 + 12345, -(2 ** 36)]])
    n = pos.shape[1]
    q, k = rand(5, 1, n, 2, D), rand(6, 1, n, 1, D)
    inv = torch.cat([torch.tensor([1.0, 1.5, 3.0, -0.25, 0.0, 2.0 ** -30]), freqs()[6:]])
    gq, gk = cache.qk_norm_rope(0, q.cuda(), k.cuda(), inv.cuda(), positions=pos.cuda())
    # the angles modulo a turn, in integers: 2 pi to 200 bits, so that far positions are exact
    two_pi = 0x6487ED5110B4611A62633145C06E0E68948127044533E63A0105DF531D89CD9128A5043CC71A026EF7CA8CD9E69D218D
    bits = two_pi.bit_length() - 3
    ang = np.empty((n, 64))
    for i in range(n):
        for j in range(64):
            num, den = float(inv[j]).as_integer_ratio()
            t = (num * int(pos[0, i]) << bits) // den % two_pi
            ang[i, j] = float(t) / float(1 << bits)
    c, s = np.cos(ang)[None, :, None], np.sin(ang)[None, :, None]
    for x, got in ((f64(q), gq), (f64(k), gk)):
        a, b = x[..., :64], x[..., 64:]
        ref = np.concatenate([a * c - b * s, b * c + a * s], -1)
        assert np.all(np.abs(f64(got) - ref) <= 2.0 ** -8 * np.abs(ref) + 4e-6)


def test_norm_rope_layouts_in_place_and_default_positions():
    B, Hq, Hkv, n = 2, 8, 2, 3
    cache = cache_for(B, Hq, Hkv, w=16, max_context=64, fp_capacity=4, ledger_capacity=4)
    kv = rand(3, B, 10, Hkv, D).cuda()
    cache.prefill(0, kv, kv, tiers=torch.zeros(B, 1, dtype=torch.uint8, device="cuda"))
    inv = freqs().cuda()
    q, k = rand(1, B, n, Hq, D).cuda(), rand(2, B, n, Hkv, D).cuda()
    at = 10 + torch.arange(n, device="cuda").expand(B, n).contiguous()
    eq, ek = cache.qk_norm_rope(0, q, k, inv, positions=at)
    dq, dk = cache.qk_norm_rope(0, q, k, inv)            # the layer's length onwards
    assert torch.equal(dq, eq) and torch.equal(dk, ek)
    # a captured call follows the device length through replayed appends
    out = [torch.empty(B, 1, Hq, D, dtype=torch.bfloat16, device="cuda"),
           torch.empty(B, 1, Hkv, D, dtype=torch.bfloat16, device="cuda")]
    q1, k1 = q[:, :1].contiguous(), k[:, :1].contiguous()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        g.capture_begin()
        cache.qk_norm_rope(0, q1, k1, inv, q_out=out[0], k_out=out[1])
        cache.append(0, k1, k1)
        g.capture_end()
    for step in range(3):
        g.replay()
        torch.cuda.synchronize()
        cache.refresh_lengths()
        ref = cache.qk_norm_rope(0, q1, k1, inv, positions=torch.full((B, 1), 10 + step, device="cuda"))
        assert torch.equal(out[0], ref[0]) and torch.equal(out[1], ref[1]), step
    # in place, and one-token tensors without a token dimension
    q2, k2 = q.clone(), k.clone()
    cache.qk_norm_rope(0, q2, k2, inv, positions=at, q_out=q2, k_out=k2)
    assert torch.equal(q2, eq) and torch.equal(k2, ek)
    oq, ok = cache.qk_norm_rope(0, q[:, 0], k[:, 0], inv, positions=at[:, :1].contiguous())
    assert torch.equal(oq, eq[:, 0]) and torch.equal(ok, ek[:, 0])
    assert cache.status() == 0


# ---- attention -------------------------------------------------------------------
def check_attention(q, k, v, out, lse, q_len, kv_len, span, sinks):
    ref, rl = U.attention(f64(q), f64(k), f64(v), q_len, kv_len, span, sinks)
    mag, _ = U.attention(f64(q), f64(k), np.abs(f64(v)), q_len, kv_len, span, sinks)
    got, gl = f64(out), f64(lse)
    rows = ~np.isnan(rl)
    assert np.array_equal(np.isneginf(gl[rows]), np.isneginf(rl[rows]))
    fine = rows & np.isfinite(rl)
    assert np.all(np.abs(gl[fine] - rl[fine]) <= 1e-5 + 1e-6 * np.abs(rl[fine]))
    used = ~np.isnan(ref)
    err = np.abs(got - ref)[used]
    assert np.all(err <= 2.0 ** -8 * (np.abs(ref[used]) + mag[used]) + 1e-5), err.max()
    # the bound above is per element; over a whole tensor the two roundings average out
    assert np.linalg.norm(err) <= 4e-3 * np.linalg.norm(mag[used])


CASES = [  # B, Hq, Hkv, n_q, n_kv, span, sinks
    (1, 1, 1, 1, 1, 0, 0), (1, 8, 2, 128, 128, 0, 0), (1, 8, 2, 1, 700, 0, 0), (2, 28, 4, 130, 130, 0, 0),
    (1, 8, 1, 257, 257, 0, 0), (2, 6, 2, 300, 517, 0, 0), (1, 10, 2, 64, 1000, 200, 4), (2, 4, 4, 513, 513, 1, 0),
    (1, 4, 4, 513, 513, 1, 7), (1, 12, 2, 400, 1025, 128, 128), (1, 8, 2, 600, 600, 100, 300),
    (2, 14, 2, 1, 1500, 256, 16), (1, 32, 8, 1024, 1024, 511, 1), (3, 8, 8, 5, 2000, 0, 0), (1, 7, 1, 1, 4000, 1, 1),
    (1, 16, 2, 3, 4000, 1000, 130), (1, 2, 1, 1100, 1100, 5000, 9),
]


@pytest.mark.parametrize("B,Hq,Hkv,n_q,n_kv,span,sinks", CASES)
def test_span_attention_matches_plain(B, Hq, Hkv, n_q, n_kv, span, sinks):
    cache = cache_for(B, Hq, Hkv)
    q, k, v = rand(1, B, n_q, Hq, D), rand(2, B, n_kv, Hkv, D, scale=1.5), rand(3, B, n_kv, Hkv, D)
    out, lse = cache.span_attention(0, q.cuda(), k.cuda(), v.cuda(), span=span, sinks=sinks)
    assert cache.status() == 0, cache.last_error()
    check_attention(q, k, v, out, lse, [n_q] * B, [n_kv] * B, span, sinks)


@pytest.mark.parametrize("span,sinks", [(0, 0), (90, 3)])
def test_span_attention_padded_batch(span, sinks):
    """Ragged lengths (none, one, odd, all), more queries than keys, garbage past the ends, rows left alone."""
    B, Hq, Hkv, n_q, n_kv = 7, 14, 2, 300, 400
    q_len = [300, 0, 1, 77, 300, 200, 5]
    kv_len = [400, 50, 1, 400, 120, 200, 0]
    q, k, v = rand(1, B, n_q, Hq, D), rand(2, B, n_kv, Hkv, D), rand(3, B, n_kv, Hkv, D)
    for b in range(B):
        q[b, q_len[b]:] = float("nan")
        k[b, kv_len[b]:] = float("nan")
        v[b, kv_len[b]:] = float("inf")
    cache = cache_for(B, Hq, Hkv)
    out = torch.full((B, n_q, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((B, Hq, n_q), 7.0, device="cuda")
    lens = [torch.tensor(x, dtype=torch.int32, device="cuda") for x in (q_len, kv_len)]
    cache.span_attention(0, q.cuda(), k.cuda(), v.cuda(), span=span, sinks=sinks, q_len=lens[0], kv_len=lens[1],
                         out=out, lse=lse)
    assert cache.status() == 0, cache.last_error()
    qz, kz, vz = (torch.nan_to_num(x, nan=0.0, posinf=0.0) for x in (q, k, v))
    check_attention(qz, kz, vz, out, lse, q_len, kv_len, span, sinks)
    for b in range(B):
        assert torch.all(out[b, q_len[b]:] == 7.0) and torch.all(lse[b, :, q_len[b]:] == 7.0)
        blind = max(0, q_len[b] - kv_len[b])
        assert torch.all(out[b, :blind] == 0.0) and torch.all(torch.isneginf(lse[b, :, :blind]))


def test_span_attention_values_outside_the_span_may_be_anything():
    B, Hq, Hkv, n_q, n_kv, span, sinks = 1, 8, 2, 3, 1000, 70, 5
    q, k, v = rand(1, B, n_q, Hq, D), rand(2, B, n_kv, Hkv, D), rand(3, B, n_kv, Hkv, D)
    clean = [x.clone() for x in (k, v)]
    k[:, sinks:n_kv - n_q - span + 1] = float("nan")
    v[:, sinks:n_kv - n_q - span + 1] = float("nan")
    cache = cache_for(B, Hq, Hkv)
    out, lse = cache.span_attention(0, q.cuda(), k.cuda(), v.cuda(), span=span, sinks=sinks)
    check_attention(q, *clean, out, lse, [n_q], [n_kv], span, sinks)


@pytest.mark.parametrize("B,Hq,Hkv,n_q,n_kv,span,sinks,bad", [
    (1, 8, 2, 300, 300, 0, 0, (5, 130, 299)), (1, 4, 4, 700, 700, 0, 0, (0, 256, 511)), (2, 14, 2, 257, 257, 0, 0, (200,)),
    (1, 8, 2, 400, 400, 60, 5, (2, 100, 131, 260, 390)), (1, 4, 4, 600, 600, 130, 3, (1, 3, 255, 400)),
    (1, 16, 2, 20, 900, 0, 0, (890, 3)), (1, 8, 1, 17, 900, 50, 4, (840, 885, 2)), (1, 32, 8, 1100, 1100, 0, 0, (1000,))])
def test_span_attention_non_finite_values_reach_only_rows_that_see_them(B, Hq, Hkv, n_q, n_kv, span, sinks, bad):
    q, k, v = rand(1, B, n_q, Hq, D), rand(2, B, n_kv, Hkv, D), rand(3, B, n_kv, Hkv, D)
    clean = v.clone()
    for i, j in enumerate(bad):   # one channel of one KV head each, NaN and both infinities
        value = (float("nan"), float("inf"), float("-inf"))[i % 3]
        v[B - 1, j, i % Hkv, 7 * i + 3] = value
        clean[B - 1, j, i % Hkv, 7 * i + 3] = 0.0
    cache = cache_for(B, Hq, Hkv)
    out, lse = cache.span_attention(0, q.cuda(), k.cuda(), v.cuda(), span=span, sinks=sinks)
    assert cache.status() == 0, cache.last_error()
    seen = U.visible(n_q, n_kv, span, sinks)
    got, G = f64(out), Hq // Hkv
    where = np.zeros(got.shape, bool)
    for i, j in enumerate(bad):
        rows = np.zeros(got.shape, bool)
        for h in range(i % Hkv * G, (i % Hkv + 1) * G):
            rows[B - 1, seen[:, j], h, 7 * i + 3] = True
        if i % 3 == 0:
            assert np.all(np.isnan(got[rows]))
        else:
            assert np.all(np.isinf(got[rows]) & ((got[rows] > 0) == (i % 3 == 1)))
        where |= rows
    assert np.array_equal(~np.isfinite(got), where)
    ref, _ = U.attention(f64(q), f64(k), f64(clean), [n_q] * B, [n_kv] * B, span, sinks)
    mag, rl = U.attention(f64(q), f64(k), np.abs(f64(clean)), [n_q] * B, [n_kv] * B, span, sinks)
    err = np.abs(got - ref)[~where]
    assert np.all(err <= 2.0 ** -8 * (np.abs(ref) + mag)[~where] + 1e-5)
    assert np.all(np.abs(f64(lse) - rl) <= 1e-5 + 1e-6 * np.abs(rl))


def test_span_attention_all_values_nan():
    """Every value NaN, several units per SM: every row that sees a key is NaN, nothing else happens."""
    B, Hq, Hkv, n = 2, 16, 16, 1300
    q, k = rand(1, B, n, Hq, D), rand(2, B, n, Hkv, D)
    v = torch.full((B, n, Hkv, D), float("nan"), dtype=torch.bfloat16)
    cache = cache_for(B, Hq, Hkv)
    out, _ = cache.span_attention(0, q.cuda(), k.cuda(), v.cuda(), span=200, sinks=9)
    assert torch.all(torch.isnan(out)) and cache.status() == 0


def test_span_attention_large_logits_and_late_maxima():
    """Logits that grow along the keys by thousands: every tile moves the maximum."""
    B, Hq, Hkv, n = 1, 4, 2, 700
    q, k, v = rand(1, B, n, Hq, D), rand(2, B, n, Hkv, D), rand(3, B, n, Hkv, D)
    k = (k.float() * (0.05 * torch.arange(n)[None, :, None, None])).bfloat16()
    cache = cache_for(B, Hq, Hkv)
    out, lse = cache.span_attention(0, q.cuda(), k.cuda(), v.cuda())
    ref, rl = U.attention(f64(q), f64(k), f64(v), [n], [n], 0, 0)
    # logits of up to some hundreds: an error of 2^-24 of that in the exponent, and of the sums
    assert np.all(np.abs(f64(lse) - rl) <= 1e-6 * np.abs(rl) + 1e-4)
    mag, _ = U.attention(f64(q), f64(k), np.abs(f64(v)), [n], [n], 0, 0)
    assert np.all(np.abs(f64(out) - ref) <= (2.0 ** -8 + 3e-4) * (np.abs(ref) + mag) + 1e-5)


def test_span_attention_non_finite_query_stays_in_its_row():
    B, Hq, Hkv, n = 1, 4, 1, 150
    q, k, v = rand(1, B, n, Hq, D), rand(2, B, n, Hkv, D), rand(3, B, n, Hkv, D)
    bad = q.clone()
    bad[0, 40, 2] = float("nan")
    cache = cache_for(B, Hq, Hkv)
    a, la = cache.span_attention(0, q.cuda(), k.cuda(), v.cuda())
    b, lb = cache.span_attention(0, bad.cuda(), k.cuda(), v.cuda())
    assert torch.all(torch.isnan(b[0, 40, 2])) and torch.isnan(lb[0, 2, 40])
    keep = torch.ones(n, Hq, dtype=torch.bool)
    keep[40, 2] = False
    assert torch.equal(a[0][keep.cuda()], b[0][keep.cuda()])


@pytest.mark.parametrize("B,Hq,Hkv,n", [(1, 8, 2, 900), (3, 16, 8, 1500)])   # split, and several units per SM
def test_span_attention_streams_and_graph(B, Hq, Hkv, n):
    """Two calls at once on two streams, and a captured call on new inputs, give the same bits."""
    sets = [[rand(10 * s + i, B, n, h, D).cuda() for i, h in enumerate((Hq, Hkv, Hkv))] for s in range(2)]
    cache = cache_for(B, Hq, Hkv)
    ref = [cache.span_attention(0, *s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(5):
        got = []
        for s, st in zip(sets, streams):
            with torch.cuda.stream(st):
                got.append(cache.span_attention(0, *s))
        torch.cuda.synchronize()
        for (a, b), (x, y) in zip(ref, got):
            assert torch.equal(a, x) and torch.equal(b, y)
    bufs = [t.clone() for t in sets[0]]
    out, lse = torch.empty_like(ref[0][0]), torch.empty_like(ref[0][1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        g.capture_begin()
        cache.span_attention(0, *bufs, out=out, lse=lse)
        g.capture_end()
    for s, (a, b) in zip(sets, ref):
        for t, x in zip(bufs, s):
            t.copy_(x)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, a) and torch.equal(lse, b)


# ---- window scores ----------------------------------------------------------------
@pytest.mark.parametrize("w", [16, 48, 64, 128])
@pytest.mark.parametrize("B,Hq,Hkv,n_q,n_kv,span,sinks", [
    (1, 1, 1, 1, 1, 0, 0), (2, 8, 2, 64, 1000, 0, 0), (1, 28, 4, 333, 333, 0, 0), (2, 6, 3, 200, 700, 90, 5),
    (1, 10, 2, 300, 300, 1, 0), (1, 16, 16, 17, 517, 0, 0), (1, 8, 1, 130, 2000, 300, 200),
    (3, 14, 2, 20, 1700, 90, 5), (2, 8, 2, 1, 900, 0, 0), (1, 4, 1, 40, 3000, 50, 200), (2, 12, 4, 84, 84, 0, 0)])
@pytest.mark.parametrize("per_head", [False, True])
def test_span_scores_match_plain(B, Hq, Hkv, n_q, n_kv, span, sinks, w, per_head):
    cache = cache_for(B, Hq, Hkv, w=w, per_head=per_head)
    q, k = rand(1, B, n_q, Hq, D), rand(2, B, n_kv, Hkv, D, scale=1.5)
    _, lse = cache.span_attention(0, q.cuda(), k.cuda(), k.cuda(), span=span, sinks=sinks)
    got = cache.span_scores(0, q.cuda(), k.cuda(), lse, span=span, sinks=sinks)
    assert cache.status() == 0, cache.last_error()
    ref = U.scores(f64(q), f64(k), f64(lse), [n_q] * B, [n_kv] * B, span, sinks, w, per_head)
    assert np.all(np.abs(f64(got) - ref) <= 1e-5 * ref + 1e-9)
    # every query spreads one unit of mass
    assert np.allclose(f64(got).sum(-1), n_q, rtol=1e-5)
    again = cache.span_scores(0, q.cuda(), k.cuda(), lse, span=span, sinks=sinks)
    assert torch.equal(got, again)


@pytest.mark.parametrize("n_q", [100, 30])   # 30: two query tiles, the form for few queries
def test_span_scores_padded_batch(n_q):
    B, Hq, Hkv, n_kv, w, span, sinks = 6, 14, 2, 400, 32, 90, 3
    q_len, kv_len = [n_q, 0, 1, n_q - 23, n_q, 5], [400, 50, 1, 399, 20, 0]
    q, k = rand(1, B, n_q, Hq, D), rand(2, B, n_kv, Hkv, D)
    for b in range(B):
        q[b, q_len[b]:] = float("nan")
        k[b, kv_len[b]:] = float("nan")
    lens = [torch.tensor(x, dtype=torch.int32, device="cuda") for x in (q_len, kv_len)]
    cache = cache_for(B, Hq, Hkv, w=w)
    lse = torch.full((B, Hq, n_q), float("nan"), device="cuda")
    kw = dict(span=span, sinks=sinks, q_len=lens[0], kv_len=lens[1])
    cache.span_attention(0, q.cuda(), k.cuda(), torch.nan_to_num(k).cuda(), lse=lse, **kw)
    got = cache.span_scores(0, q.cuda(), k.cuda(), lse, **kw)
    ref = U.scores(f64(torch.nan_to_num(q)), f64(torch.nan_to_num(k)), f64(lse), q_len, kv_len, span, sinks, w)
    assert np.all(np.abs(f64(got) - ref) <= 1e-5 * ref + 1e-9)
    assert cache.status() == 0


@pytest.mark.parametrize("n_q", [1300, 64])
def test_span_scores_streams_layers_and_graph(n_q):
    """Calls on two layers at once, in parts that a second kernel sums, and a captured one."""
    B, Hq, Hkv, n, w = 1, 16, 4, 1300, 32
    cache = binding.TieredCache(B, 2, Hq, Hkv, w, n, fp_capacity=1, ledger_capacity=1)
    sets = [[rand(10 * s + i, B, m, h, D).cuda() for i, (m, h) in enumerate(((n_q, Hq), (n, Hkv)))] for s in range(2)]
    lse = [cache.span_attention(0, q, k, k)[1] for q, k in sets]
    ref = [cache.span_scores(0, q, k, x) for (q, k), x in zip(sets, lse)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(10):
        got = [cache.span_scores(i, *sets[i], lse[i], stream=st) for i, st in enumerate(streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(ref, got))
    bufs, x, out = [t.clone() for t in sets[0]], lse[0].clone(), torch.empty_like(ref[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        g.capture_begin()
        cache.span_scores(0, *bufs, x, out=out)
        g.capture_end()
    for s, l, r in zip(sets, lse, ref):
        for t, y in zip(bufs + [x], s + [l]):
            t.copy_(y)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, r)


def test_offsets_past_32_bits():
    """Keys, queries and outputs whose element offsets pass 2^31; only what is looked at is filled."""
    Hq, Hkv, n, span, sinks = 8, 8, 2 ** 21 + 300, 700, 3
    cache = cache_for(1, Hq, Hkv, w=128)
    k, v = (torch.empty(1, n, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    tail = n - 1100
    for t, s in ((k, 2), (v, 3)):
        t[:, :sinks] = rand(s, 1, sinks, Hkv, D).cuda()
        t[:, tail:] = rand(s + 2, 1, n - tail, Hkv, D).cuda()
    q = rand(1, 1, 5, Hq, D)
    out, lse = cache.span_attention(0, q.cuda(), k, v, span=span, sinks=sinks)
    keep = torch.cat([torch.arange(sinks), torch.arange(tail, n)]).cuda()
    j, p = keep.cpu().numpy()[None], n - 5 + np.arange(5)[:, None]
    seen = (j <= p) & ((j > p - span) | (j < sinks))
    kk, vv = f64(k[:, keep]), f64(v[:, keep])
    for h in range(Hq):
        o, s = U.attention_head(f64(q)[0, :, h], kk[0, :, h], vv[0, :, h], seen)
        mag, _ = U.attention_head(f64(q)[0, :, h], kk[0, :, h], np.abs(vv[0, :, h]), seen)
        assert np.all(np.abs(f64(out)[0, :, h] - o) <= 2.0 ** -8 * (np.abs(o) + mag) + 1e-5)
        assert np.all(np.abs(f64(lse)[0, h] - s) <= 1e-5 + 1e-6 * np.abs(s))
    sc = cache.span_scores(0, q.cuda(), k, lse, span=span, sinks=sinks)
    assert abs(float(sc.sum()) - 5) < 1e-4 and int((sc > 0).sum()) <= 8
    # the last 704 keys begin in window (n - 704) // 128 = W - 7
    assert float(sc[0, -7:].sum()) + float(sc[0, 0]) == pytest.approx(5, abs=1e-4)
    # the same tensor as queries: n rows of n keys with a narrow span, written past 2^31 elements
    out, lse = cache.span_attention(0, k, k, v, span=16)
    a, b = f64(k[:, -400:]), f64(v[:, -400:])
    ref, _ = U.attention(a, a, b, [400], [400], 16, 0)
    mag, _ = U.attention(a, a, np.abs(b), [400], [400], 16, 0)
    got = f64(out[:, -384:])
    assert np.all(np.abs(got - ref[:, -384:]) <= 2.0 ** -8 * (np.abs(ref) + mag)[:, -384:] + 1e-5)
    # and through norm and rotation
    pos = torch.arange(n, device="cuda")[None]
    gq, gk = cache.qk_norm_rope(0, k, v, freqs().cuda(), positions=pos)
    for t, g in ((k, gq), (v, gk)):
        r = U.norm_rope(f64(t[:, -4:]), None, 0, pos[:, -4:].cpu().numpy(), freqs().double().numpy())
        assert np.all(np.abs(f64(g[:, -4:]) - r) <= 2.0 ** -8 * np.abs(r) + 2e-5)
    assert cache.status() == 0


def test_refusals():
    """What the library refuses before it enqueues anything."""
    B, Hq, Hkv, n = 2, 8, 2, 40
    cache = cache_for(B, Hq, Hkv)
    q, k = rand(1, B, n, Hq, D).cuda(), rand(2, B, n, Hkv, D).cuda()
    v, inv = k.clone(), freqs().cuda()
    out, lse = cache.span_attention(0, q, k, v)
    kept = out.clone()
    big = torch.zeros(q.numel() + 8, dtype=torch.bfloat16, device="cuda")
    shifted = big[4:4 + q.numel()].view(q.shape)      # 8-byte aligned
    ahead = big[8:8 + q.numel()].view(q.shape)
    behind = big[:q.numel()].view(q.shape)
    for call, word in (
            (lambda: cache.span_attention(5, q, k, v), "layer"),
            (lambda: cache.span_attention(0, q, k, v, span=-1), "span"),
            (lambda: cache.span_attention(0, q, k, v, sinks=-1), "sinks"),
            (lambda: cache.span_attention(0, shifted, k, v), "aligned"),
            (lambda: cache.span_attention(0, q, k, v, out=q), "overlaps"),
            (lambda: cache.span_attention(0, ahead, k, v, out=behind), "overlaps"),
            (lambda: cache.span_scores(0, q, k, lse, span=-3), "span"),
            (lambda: cache.span_scores(0, q, k, lse, out=lse.view(-1)[:B].view(B, 1)), "overlaps"),
            (lambda: cache.qk_norm_rope(0, q, k, inv, eps=-1.0), "eps"),
            (lambda: cache.qk_norm_rope(0, q, k, inv, eps=float("nan")), "eps"),
            (lambda: cache.qk_norm_rope(0, ahead, k, inv, q_out=behind), "overlap"),
            (lambda: cache.qk_norm_rope(0, q, k, inv, k_out=q.view(-1)[:k.numel()].view(k.shape)), "overlap"),
            (lambda: cache.qk_norm_rope(0, q, k, inv, v=v, k_out=v), "overlap"),
            (lambda: cache.qk_norm_rope(0, shifted, k, inv), "aligned"),
            (lambda: cache.qk_norm_rope(7, q, k, inv), "layer")):
        with pytest.raises(binding.QevictError) as e:
            call()
        assert e.value.name == "INVALID_ARG" and word in str(e.value), str(e.value)
    for call in (lambda: cache.span_attention(0, q, k, v[:, :3]), lambda: cache.span_attention(0, q[:, ::2], k, v),
                 lambda: cache.span_attention(0, q[:, :0], k, v, out=out[:, :0], lse=lse[:, :, :0]),
                 lambda: cache.span_attention(0, q, k, v, q_len=torch.zeros(B, device="cuda")),
                 lambda: cache.span_scores(0, q, k, lse[:, :, :3]),
                 lambda: cache.qk_norm_rope(0, q, k, inv, positions=torch.zeros(B, n, device="cuda")),
                 lambda: cache.qk_norm_rope(0, q, k, inv[:3]), lambda: cache.qk_norm_rope(0, q, k[:, :3], inv),
                 lambda: cache.qk_norm_rope(0, q, k, inv, v_out=v)):
        with pytest.raises(ValueError):
            call()
    assert torch.equal(out, kept) and cache.status() == 0


def test_outputs_that_are_also_side_operands_are_refused():
    B, Hq, Hkv, n = 1, 8, 2, 4
    cache = cache_for(B, Hq, Hkv)
    q, k = rand(1, B, n, Hq, D).cuda(), rand(2, B, n, Hkv, D).cuda()
    mem = torch.zeros(n * Hq * D, dtype=torch.bfloat16, device="cuda")
    out = mem.view(B, n, Hq, D)
    inv, pos, w = mem[:128].view(torch.float32), mem[:16].view(torch.int64).view(B, n), mem[128:256]
    inv.copy_(freqs())
    good = freqs().cuda()
    for call in (lambda: cache.qk_norm_rope(0, q, k, inv, q_out=out),
                 lambda: cache.qk_norm_rope(0, q, k, good, positions=pos, q_out=out),
                 lambda: cache.qk_norm_rope(0, q, k, good, q_weight=w, q_out=out),
                 lambda: cache.qk_norm_rope(0, q, k, good, k_weight=w, q_out=out)):
        with pytest.raises(binding.QevictError) as e:
            call()
        assert e.value.name == "INVALID_ARG" and "overlaps" in str(e.value), str(e.value)
    assert torch.equal(inv, good) and cache.status() == 0


def test_spans_wider_than_32_bits_are_all_the_keys():
    B, Hq, Hkv, n = 1, 8, 2, 300
    cache = cache_for(B, Hq, Hkv)
    q, k, v = rand(1, B, n, Hq, D).cuda(), rand(2, B, n, Hkv, D).cuda(), rand(3, B, n, Hkv, D).cuda()
    out, lse = cache.span_attention(0, q, k, v)
    scores = cache.span_scores(0, q, k, lse)
    sunk = cache.span_attention(0, q, k, v, span=7, sinks=n)[0]
    sunk_scores = cache.span_scores(0, q, k, lse, span=7, sinks=n)
    for wide in (2 ** 31 - 1, 2 ** 32 + 5):
        a, b = cache.span_attention(0, q, k, v, span=wide)
        assert torch.equal(a, out) and torch.equal(b, lse)
        # (the tiles may be shared out otherwise under a short span, so it is the same call with n sinks that is equal)
        assert torch.equal(cache.span_attention(0, q, k, v, span=7, sinks=wide)[0], sunk)
        assert torch.equal(cache.span_scores(0, q, k, lse, span=wide), scores)
        assert torch.equal(cache.span_scores(0, q, k, lse, span=7, sinks=wide), sunk_scores)
    for kw in (dict(span=-2 ** 32), dict(sinks=-2 ** 32)):   # refused, not cut to 32 bits
        for call in (lambda: cache.span_attention(0, q, k, v, **kw), lambda: cache.span_scores(0, q, k, lse, **kw)):
            with pytest.raises(binding.QevictError):
                call()
    assert cache.status() == 0


# ---- the run of them -----------------------------------------------------------------
@pytest.mark.parametrize("budget", [0.5, 0.2])
@pytest.mark.parametrize("per_head", [False, True])
def test_prompt_to_tiered_decode(per_head, budget):
    """A prompt's projections through norm and rotation, attention, scores, the routed prefill and decode steps:
    the tiers follow the scores' ranking, and a decode over a cache that keeps everything equals span attention."""
    B, Hq, Hkv, n, w = 2, 8, 2, 700, 32
    W = -(-n // w)
    inv = freqs().cuda()
    wq, wk = (1 + rand(8, D).float() * 0.1).bfloat16().cuda(), (1 + rand(9, D).float() * 0.1).bfloat16().cuda()
    kw = dict(q_weight=wq, k_weight=wk, eps=1e-5)
    cache = binding.TieredCache(B, 1, Hq, Hkv, w, n + 64, budget_frac=budget, per_head=per_head)
    full = binding.TieredCache(B, 1, Hq, Hkv, w, n + 64, fp_capacity=W + 4, ledger_capacity=1)
    q, k, v = rand(4, B, n, Hq + 2 * Hkv, D).cuda().split([Hq, Hkv, Hkv], 2)
    q, k, v = cache.qk_norm_rope(0, q, k, inv, v=v, **kw)
    out, lse = cache.span_attention(0, q, k, v)
    sc = cache.span_scores(0, q, k, lse)
    cache.prefill(0, k, v, scores=sc)
    full.prefill(0, k, v, tiers=torch.zeros(B, W, dtype=torch.uint8, device="cuda"))
    assert cache.status() == 0, cache.last_error()
    tiers = cache.tables(0)[0].numpy()
    s = sc.cpu().numpy()
    for u in range(tiers.shape[0]):
        closed = np.arange(W - 1)
        for hi, lo in ((0, 1), (0, 2), (1, 2)):
            a, b = s[u][closed[tiers[u][:-1] == hi]], s[u][closed[tiers[u][:-1] == lo]]
            if len(a) and len(b):
                assert a.min() >= b.max()
        n_fp, n_q = O.route_counts(W, n, w, 1 if per_head else Hkv, D, budget, 0.5)
        assert tiers[u, -1] == 0 and [(tiers[u] == x).sum() for x in range(3)] == [n_fp, n_q, W - n_fp - n_q]
    keys, values = k, v
    for step in range(3):
        x = rand(20 + step, B, 1, Hq + 2 * Hkv, D).cuda().split([Hq, Hkv, Hkv], 2)
        q1, k1, v1 = full.qk_norm_rope(0, x[0], x[1], inv, v=x[2], **kw)      # at the layer's length
        c1 = cache.qk_norm_rope(0, x[0], x[1], inv, v=x[2], **kw)
        assert all(torch.equal(a, b) for a, b in zip((q1, k1, v1), c1))
        cache.decode_step(0, q1[:, 0], k1, v1)
        got, _ = full.decode_step(0, q1[:, 0].contiguous(), k1, v1)
        keys, values = torch.cat([keys, k1], 1), torch.cat([values, v1], 1)
        ref, _ = full.span_attention(0, q1, keys, values)
        mag, _ = full.span_attention(0, q1, keys, values.abs())
        assert torch.all((got - ref[:, 0].float()).abs() <= 2.0 ** -7 * mag[:, 0].float() + 2e-3)
    assert cache.status() == 0 and full.status() == 0
