"""What a row of the span attention and a window of the span scores depend on: the keys that it sees, and
nothing else. Results are compared bit by bit with those of other calls, or with the definition where
infinities and zeros decide.

The form that attention takes follows from its sizes (units of two query tiles, at least one per SM: wide;
fewer: split over clusters), so the sizes here name theirs.
"""
import numpy as np
import pytest
import torch

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


def cache_for(B, Hq, Hkv, w=64, **kw):
    return binding.TieredCache(B, 1, Hq, Hkv, w, 4096, fp_capacity=1, ledger_capacity=1, **kw)


def rand(seed, *shape, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).bfloat16()


def f64(t):
    return t.detach().cpu().double().numpy()


def bits(t):
    return t.view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32)


@pytest.mark.parametrize("B,H,n,key,span", [
    (2, 16, 1300, 394, 300),    # wide: the key's tile is masked for the second query tile of unit 512..767 alone
    (3, 16, 1100, 395, 333),
    (1, 4, 900, 394, 200)])     # split
def test_infinite_values_of_probability_zero(B, H, n, key, span):
    """A key whose probability rounds to 0 holds infinities and a NaN: the rows that see it take them, whichever
    of a tile's two query tiles masks some of its keys."""
    q, k, v = rand(1, B, n, H, D), rand(2, B, n, H, D), rand(3, B, n, H, D)
    q[..., 0] = 8.0
    k[:, key, :, 0] = -400.0     # a logit near -283: its probability is below every fp32 number
    clean = v.clone()
    for ch, value in ((5, float("inf")), (77, float("-inf")), (100, float("nan"))):
        v[:, key, :, ch] = value
        clean[:, key, :, ch] = 0.0
    cache = cache_for(B, H, H)
    dev = [x.cuda() for x in (q, k, v)]
    out, lse = cache.span_attention(0, *dev, span=span)
    assert cache.status() == 0, cache.last_error()
    got, seen = f64(out), U.visible(n, n, span, 0)[:, key]
    assert np.all(got[:, seen, :, 5] == np.inf) and np.all(got[:, seen, :, 77] == -np.inf)
    assert np.all(np.isnan(got[:, seen, :, 100]))
    rest = np.ones(got.shape, bool)
    rest[:, seen, :, 5] = rest[:, seen, :, 77] = rest[:, seen, :, 100] = False
    plain, lse_plain = cache.span_attention(0, dev[0], dev[1], clean.cuda(), span=span)
    assert np.array_equal(got[rest], f64(plain)[rest]) and torch.equal(lse, lse_plain)
    for _ in range(10):
        again, _ = cache.span_attention(0, *dev, span=span)
        assert torch.equal(bits(again), bits(out))


def repeats(n, H, Hkv, w, per_head, n_q=None, B=4, span=0):
    """Window scores of B copies of one sequence: every copy, and every call, adds in the same order."""
    q, k = rand(1, 1, n_q or n, H, D).expand(B, -1, -1, -1).contiguous().cuda(), \
        rand(2, 1, n, Hkv, D).expand(B, -1, -1, -1).contiguous().cuda()
    cache = cache_for(B, H, Hkv, w=w, per_head=per_head)
    lse = cache.span_attention(0, q, k, k, span=span)[1][:1].expand(B, -1, -1).contiguous()
    one, other = (cache.span_scores(0, q, k, lse, span=span).clone() for _ in range(2))
    by_copy = one.view(B, -1)
    assert torch.equal(by_copy, by_copy[:1].expand(B, -1))
    assert torch.equal(one, other)
    side = torch.cuda.Stream()
    busy = torch.randn(2048, 2048, device="cuda")
    torch.cuda.synchronize()
    for _ in range(20):     # beside other work, which moves the CTAs' starts
        with torch.cuda.stream(side):
            busy = torch.tanh(busy @ busy)
        assert torch.equal(cache.span_scores(0, q, k, lse, span=span), one)
    assert cache.status() == 0, cache.last_error()


@pytest.mark.parametrize("n,H,Hkv,w,per_head,n_q,span", [
    (2047, 28, 4, 64, False, None, 0), (2047, 28, 4, 64, True, None, 0), (4095, 24, 8, 32, False, None, 0),
    (2048, 8, 8, 64, True, None, 0), (3001, 14, 2, 16, True, 77, 0), (2500, 16, 4, 48, False, None, 300),
    (1300, 16, 4, 32, False, None, 0), (1000, 5, 1, 128, False, 333, 0)])
def test_window_scores_repeat(n, H, Hkv, w, per_head, n_q, span):
    repeats(n, H, Hkv, w, per_head, n_q, span=span)


@pytest.mark.parametrize("n,H,Hkv,per_head", [(2047, 28, 4, False), (2047, 28, 4, True), (8191, 28, 4, False)])
def test_window_scores_of_one_sequence_repeat(n, H, Hkv, per_head):
    repeats(n, H, Hkv, 64, per_head, B=1)


def same(a, b, rows=None):
    """Equal bits of two attention results (out [B][n][H][128], lse [B][H][n]), of some rows [n][H] of all."""
    for x, y, r in ((a[0], b[0], rows), (a[1], b[1], None if rows is None else rows.T)):
        x, y = bits(x), bits(y)
        if r is not None:
            x, y = x[:, r], y[:, r]
        if not torch.equal(x, y):
            return False
    return True


FORMS = [  # B, Hq, Hkv, n, span, sinks
    (3, 16, 8, 1500, 0, 0), (2, 28, 4, 700, 0, 0), (2, 28, 4, 700, 150, 5), (3, 16, 16, 1100, 300, 0),   # wide
    (1, 8, 2, 900, 0, 0), (1, 12, 2, 333, 70, 3), (1, 3, 1, 500, 0, 0)]                                    # split


@pytest.mark.parametrize("B,Hq,Hkv,n,span,sinks", FORMS)
def test_rows_do_not_depend_on_what_they_do_not_see(B, Hq, Hkv, n, span, sinks):
    """Large finite queries of other rows, later keys and keys before the span change no bit of a row."""
    cache = cache_for(B, Hq, Hkv)
    q, k, v = rand(1, B, n, Hq, D).cuda(), rand(2, B, n, Hkv, D).cuda(), rand(3, B, n, Hkv, D).cuda()

    def call(q=q, k=k, v=v):
        return cache.span_attention(0, q, k, v, span=span, sinks=sinks)

    base = call()
    every = torch.ones(n, Hq, dtype=torch.bool, device="cuda")
    for i in (n // 3, n - 2):
        louder = q.clone()
        louder[:, i, Hq // 2] *= 64
        rows = every.clone()
        rows[i, Hq // 2] = False
        assert same(base, call(q=louder), rows), f"query {i}"
    for p in (n // 2 + 3, n - 3):
        k2, v2 = k.clone(), v.clone()
        k2[:, p + 1:] *= 64
        v2[:, p + 1:] *= 64
        rows = every.clone()
        rows[p + 1:] = False
        assert same(base, call(k=k2, v=v2), rows), f"keys after {p}"
    if span:
        p = n // 2 + 3
        k2, v2 = k.clone(), v.clone()
        k2[:, sinks:p - span + 1] *= 64
        v2[:, sinks:p - span + 1] *= 64
        rows = every.clone()
        rows[:p] = False
        assert same(base, call(k=k2, v=v2), rows), f"keys before the span of {p}"
    assert cache.status() == 0, cache.last_error()


@pytest.mark.parametrize("B,Hq,Hkv,n,span,sinks", FORMS)
def test_padding_does_not_reach_the_rows(B, Hq, Hkv, n, span, sinks):
    """Queries and keys past a sequence's ends: zeros or large numbers, the same bits."""
    cache = cache_for(B, Hq, Hkv)
    q, k, v = rand(1, B, n, Hq, D), rand(2, B, n, Hkv, D), rand(3, B, n, Hkv, D)
    kv = [n - 5 - 37 * b for b in range(B)]
    nq = [x - 11 for x in kv]
    lens = dict(q_len=torch.tensor(nq, dtype=torch.int32).cuda(), kv_len=torch.tensor(kv, dtype=torch.int32).cuda())
    got, mass = [], []
    for scale in (0.0, 64.0):
        a, b, c = q.clone(), k.clone(), v.clone()
        for x, m in ((a, nq), (b, kv), (c, kv)):
            for s in range(B):
                x[s, m[s]:] *= scale
        a, b, c = a.cuda(), b.cuda(), c.cuda()
        out = torch.zeros(B, n, Hq, D, dtype=torch.bfloat16, device="cuda")
        lse = torch.zeros(B, Hq, n, device="cuda")
        got.append(cache.span_attention(0, a, b, c, span=span, sinks=sinks, out=out, lse=lse, **lens))
        lse = lse.clone()
        for s in range(B):
            lse[s, :, nq[s]:] = -scale
        mass.append(cache.span_scores(0, a, b, lse, span=span, sinks=sinks, **lens))
    assert same(*got) and torch.equal(bits(mass[0]), bits(mass[1]))
    assert cache.status() == 0, cache.last_error()


@pytest.mark.parametrize("G", [3, 5, 6, 7])
@pytest.mark.parametrize("B,Hkv,n", [(4, 8, 500), (2, 2, 150)])   # wide, split
def test_calls_leave_nothing_behind(G, B, Hkv, n):
    """Where a KV head's group does not divide a tile's 128 rows, rows that no query fills: copies of one
    sequence, and calls after calls on other data, give the same bits."""
    q, k, v = rand(1, 1, n, G * Hkv, D).expand(B, -1, -1, -1).contiguous().cuda(), \
        rand(2, 1, n, Hkv, D).expand(B, -1, -1, -1).contiguous().cuda(), \
        rand(3, 1, n, Hkv, D).expand(B, -1, -1, -1).contiguous().cuda()
    cache, loud = cache_for(B, G * Hkv, Hkv), cache_for(4, 16, 16)
    x = rand(4, 4, 700, 16, D, scale=40.0).cuda()
    out, lse = cache.span_attention(0, q, k, v)
    scores = cache.span_scores(0, q, k, lse)
    for b in range(1, B):
        assert torch.equal(bits(out[b]), bits(out[0])) and torch.equal(lse[b], lse[0])
        assert torch.equal(scores[b], scores[0])
    for i in range(6):
        y = x * (1 - 2 * (i & 1))
        _, l = loud.span_attention(0, y, x, x)
        loud.span_scores(0, y, x, l)
        assert same((out, lse), cache.span_attention(0, q, k, v)), i
        assert torch.equal(scores, cache.span_scores(0, q, k, lse)), i
    assert cache.status() == 0, cache.last_error()


@pytest.mark.parametrize("G", [3, 5, 6, 7, 4])
@pytest.mark.parametrize("per_head", [False, True])
def test_window_of_infinite_keys_scores_zero(G, per_head):
    """Keys whose every logit is -inf have no mass, also beside the rows of a query tile that no query fills."""
    B, Hkv, n, w = 1, 2, 400, 64
    q, k = rand(1, B, n, G * Hkv, D), rand(2, B, n, Hkv, D)
    q[..., 3] = q[..., 3].abs() + 0.5
    clean = k.clone()
    k[:, 64:128, :, 3] = float("-inf")
    clean[:, 64:128, :, 3] = -1e4     # a logit of -400 at the least: mass 0 in fp32 too
    cache = cache_for(B, G * Hkv, Hkv, w=w, per_head=per_head)
    _, lse = cache.span_attention(0, q.cuda(), k.cuda(), clean.cuda())
    # the first queries of the run see other keys besides: 64 on
    got = cache.span_scores(0, q.cuda(), k.cuda(), lse)
    assert torch.all(got[:, 1] == 0.0) and torch.all(torch.isfinite(got))
    assert torch.equal(got, cache.span_scores(0, q.cuda(), clean.cuda(), lse))
    ref = U.scores(f64(q), f64(clean), f64(lse), [n], [n], 0, 0, w, per_head)
    assert np.all(np.abs(f64(got) - ref) <= 1e-5 * ref + 1e-9)
    assert cache.status() == 0, cache.last_error()


@pytest.mark.parametrize("B,Hq,Hkv,n_q,n_kv", [
    (1, 4, 2, 1, 1), (1, 4, 2, 1, 200), (1, 4, 2, 1, 300), (2, 8, 8, 3, 4000), (1, 7, 1, 40, 900),    # split
    (4, 16, 16, 600, 600), (3, 28, 4, 1000, 1000), (8, 8, 8, 2048, 2048)])                            # wide
@pytest.mark.parametrize("lengths", ["all", "none", "no keys", "some"])
def test_calls_end_with_their_last_copies_and_products(B, Hq, Hkv, n_q, n_kv, lengths):
    """Before a CTA ends it waits for the copies and products that are under way, with a limit of about two
    seconds; one that waits for something that never comes would take those."""
    q, k = torch.randn(B, n_q, Hq, D).bfloat16().cuda(), torch.randn(B, n_kv, Hkv, D).bfloat16().cuda()
    some = [0 if b % 2 else 1 + b for b in range(B)]
    lens = {"all": {}, "none": dict(q_len=[0] * B), "no keys": dict(kv_len=[0] * B),
            "some": dict(q_len=[min(n_q, s * 37) for s in some], kv_len=[min(n_kv, s * 150) for s in some])}[lengths]
    lens = {x: torch.tensor(y, dtype=torch.int32).cuda() for x, y in lens.items()}
    cache = cache_for(B, Hq, Hkv)
    out, lse = torch.zeros_like(q), torch.zeros(B, Hq, n_q, device="cuda")
    scores = torch.zeros(B, -(-n_kv // 64), device="cuda")
    for _ in range(2):
        at = [torch.cuda.Event(enable_timing=True) for _ in range(3)]
        at[0].record()
        cache.span_attention(0, q, k, k, out=out, lse=lse, **lens)
        at[1].record()
        cache.span_scores(0, q, k, lse, out=scores, **lens)
        at[2].record()
        torch.cuda.synchronize()
    assert at[0].elapsed_time(at[1]) < 250 and at[1].elapsed_time(at[2]) < 250
    assert cache.status() == 0, cache.last_error()
