"""The cache in 8 bits on the GPU against its plain forms: codes, scales, values read back, kept positions and
lengths bit by bit; attention against 64 bits. Tolerances of attention: half a step of the output (bf16, 2^-8) and of
the probabilities (fp16, 2^-11 of sum p |v|; below 2^-14 of the largest, 2^-25 of the largest for each key), and 1e-5 for
fp32 sums. A logit is off by 2^-20 of sum |q k| / sqrt(128) at most (128 products added in fp32), a weight by twice that
and the exponential's 2^-21, relative."""
import numpy as np
import pytest
import torch

import block_util as U
from tiered_kv_cache_decode_gb300 import binding

pytestmark = pytest.mark.gpu
D, T = 128, 64
FORMATS = ["int8", "e4m3"]


@pytest.fixture(autouse=True, scope="module")
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from tiered_kv_cache_decode_gb300 import build
    build.build()
    binding.load()


def ints(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def rand(seed, *shape, scale=1.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * scale).bfloat16()


def f64(t):
    return t.detach().cpu().double().numpy()


def same(got, want):
    return np.array_equal(np.asarray(got), np.asarray(want))


def filled(B, Hq, Hkv, cap, fmt, lens, seed=0, scale=1.0, **kw):
    """A handle and its plain form, filled in one call each, blocks of unlike sizes."""
    c = binding.BlockCache(B, 1, Hq, Hkv, cap, fmt, **kw)
    n = max(max(lens), 1)
    k, v = rand(2 * seed, B, n, Hkv, D, scale=scale), rand(2 * seed + 1, B, n, Hkv, D)
    grow = 2.0 ** (torch.arange(n) // T % 5 - 2).float()
    k, v = (k * grow[None, :, None, None]).bfloat16(), (v * grow.flip(0)[None, :, None, None]).bfloat16()
    ref = U.Cache(B, Hkv, c.capacity, fmt)
    c.append(0, k.cuda(), v.cuda(), n_new=ints(lens))
    ref.append(k, v, [0] * B, lens)
    return c, ref


def check_values(c, ref, lens):
    n = max(max(lens), 1)
    k, v = c.read(0, ints(lens), n)
    for x, t in (("k", k), ("v", v)):
        for b, L in enumerate(lens):
            want = torch.from_numpy(ref.values(x, b, L)).bfloat16().transpose(0, 1)
            assert torch.equal(t[b, :L].cpu(), want), (x, b)
            assert not t[b, L:].any()


# ---- storage -------------------------------------------------------------------
@pytest.mark.parametrize("fmt", FORMATS)
def test_codes_and_scales(fmt):
    B, Hkv, n = 2, 3, 8 * T
    k, v = rand(0, B, n, Hkv, D), rand(1, B, n, Hkv, D)
    for j, s in enumerate([0.0, 2.0 ** -133, 3.0e-38, 2.0 ** -61, 1e-20, 2.4e38, 1.0]):   # blocks of extreme scales
        k[0, j * T:(j + 1) * T] = (k[0, j * T:(j + 1) * T].float().clamp(-1.4, 1.4) * s).bfloat16()
        v[1, j * T:(j + 1) * T] = (v[1, j * T:(j + 1) * T].float().clamp(-1.4, 1.4) * s).bfloat16()
    v[0, T + 5, 1, 7] = 1000.0
    c = binding.BlockCache(B, 1, Hkv, Hkv, n, fmt)
    c.append(0, k.cuda(), v.cuda())
    codes, scales = c.blocks(0)
    for x, t in enumerate((k, v)):
        blocks = t.float().numpy().transpose(0, 2, 1, 3).reshape(B, Hkv, -1, T, D)
        want, s = U.quantise(blocks, fmt)
        assert same(scales[:, :, :, x], s)
        assert same(codes[:, :, :, x].float(), want)
    assert c.status() == 0, c.last_error()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("B,Hkv,steps", [
    (1, 1, [1] * 70 + [63, 1, 64, 65, 2]), (3, 2, [100, 28, 1, 200, 63, 64, 1, 1]), (2, 8, [5, 300, 1]), (2, 1, [191, 130])])
def test_appends_add_up(fmt, B, Hkv, steps):
    """Chunks that start and end anywhere give the same cache as one call."""
    off = [7 * b for b in range(B)]
    n = sum(steps)
    k, v = rand(2, B, n + 50, Hkv, D).cuda(), rand(3, B, n + 50, Hkv, D).cuda()
    c = binding.BlockCache(B, 2, Hkv, Hkv, n + 50, fmt)
    c.append(1, k, v, n_new=ints(off))
    at = 0
    for m in steps:
        ks = torch.stack([k[b, off[b] + at:off[b] + at + m] for b in range(B)])
        vs = torch.stack([v[b, off[b] + at:off[b] + at + m] for b in range(B)])
        c.append(1, ks, vs, start=ints([o + at for o in off]))
        at += m
    lens = [o + n for o in off]
    whole = binding.BlockCache(B, 1, Hkv, Hkv, n + 50, fmt)
    whole.append(0, k, v, n_new=ints(lens))
    got, want = c.read(1, ints(lens), n + 50), whole.read(0, ints(lens), n + 50)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    ref = U.Cache(B, Hkv, whole.capacity, fmt)
    ref.append(k, v, [0] * B, lens)
    check_values(whole, ref, lens)
    assert c.status() == 0 and whole.status() == 0


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("back,again", [(3, 1), (40, 5), (64 + 11, 200)])
def test_set_back_within_the_last_full_block(fmt, back, again):
    """Drafted tokens that are rejected: a smaller start goes on exactly, also where a block had filled."""
    n = 3 * T + 12
    k, v = rand(4, 1, n + 200, 2, D).cuda(), rand(5, 1, n + 200, 2, D).cuda()
    c = binding.BlockCache(1, 1, 2, 2, n + 200, fmt)
    c.append(0, k[:, :n - 80].contiguous(), v[:, :n - 80].contiguous())
    c.append(0, rand(6, 1, 80, 2, D).cuda(), rand(7, 1, 80, 2, D).cuda(), start=ints([n - 80]))
    keep = n - back                                      # of which the drafted ones are replaced too
    first = min(keep, n - 80)
    c2 = binding.BlockCache(1, 1, 2, 2, n + 200, fmt)
    mixed_k, mixed_v = k.clone(), v.clone()
    mixed_k[:, n - 80:n] = rand(6, 1, 80, 2, D).cuda()
    mixed_v[:, n - 80:n] = rand(7, 1, 80, 2, D).cuda()
    mixed_k[:, keep:keep + again] = k[:, keep:keep + again]
    mixed_v[:, keep:keep + again] = v[:, keep:keep + again]
    assert first <= keep
    c.append(0, k[:, keep:keep + again].contiguous(), v[:, keep:keep + again].contiguous(), start=ints([keep]))
    c2.append(0, mixed_k[:, :keep + again].contiguous(), mixed_v[:, :keep + again].contiguous())
    got, want = c.read(0, ints([keep + again]), n + 200), c2.read(0, ints([keep + again]), n + 200)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("fmt", FORMATS)
def test_read_of_any_rows(fmt):
    lens = [0, 1, 64, 65, 300]
    c, ref = filled(5, 4, 2, 320, fmt, lens)
    check_values(c, ref, lens)
    whole = c.read(0, ints(lens), 400)
    first = [-3, 0, 10, 64, 250]
    k, v = torch.full((5, 90, 2, D), 7.0).bfloat16().cuda(), torch.full((5, 90, 2, D), 7.0).bfloat16().cuda()
    c.read(0, ints(lens), 90, first=ints(first), k_out=k, v_out=v)
    for got, full in ((k, whole[0]), (v, whole[1])):
        for b in range(5):
            for i in range(90):
                p = first[b] + i
                want = full[b, p] if 0 <= p < lens[b] else torch.full_like(got[b, i], 7.0)
                assert torch.equal(got[b, i], want), (b, i)
    for over, clamped in (([-5, 1, 64, 65, 2 ** 31 - 1], [0, 1, 64, 65, 320]), ([-2 ** 31] * 5, [0] * 5)):
        got, want = c.read(0, ints(over), 400), c.read(0, ints(clamped), 400)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_strided_tokens():
    x = rand(8, 2, 150, 12, D).cuda()
    k, v = x[:, :, 8:10], x[:, :, 10:]
    c, d = binding.BlockCache(2, 1, 8, 2, 150), binding.BlockCache(2, 1, 8, 2, 150)
    c.append(0, k, v)
    d.append(0, k.contiguous(), v.contiguous())
    assert all(torch.equal(a, b) for a, b in zip(c.read(0, ints([150] * 2), 150), d.read(0, ints([150] * 2), 150)))


def test_device_errors_of_append():
    B, cap = 4, 128
    c = binding.BlockCache(B, 1, 2, 2, cap)
    k, v = rand(0, B, 100, 2, D).cuda(), rand(1, B, 100, 2, D).cuda()
    w = torch.ones(B, 2, cap, device="cuda")
    c.append(0, k, v, start=ints([-1, 0, 0, 2 ** 31 - 5]), n_new=ints([100, -3, 1, 200]), weights=w)
    assert c.status() in (1, 8)   # the first of a negative start and a position past the capacity
    c.clear_status()
    assert c.status() == 0
    got = c.read(0, ints([63] * 4), cap)   # the rows of the open block
    assert not got[0][[0, 1, 3]].any() and torch.equal(got[0][2, 0], k[2, 0]) and not got[0][2, 1:].any()
    assert torch.equal(w.sum((1, 2)).cpu(), torch.tensor([256.0, 256.0, 254.0, 256.0]))
    c.append(0, k, v, start=ints([100, 0, 0, 28]))
    assert c.status() == 8
    c.clear_status()
    k2, v2 = k.clone(), v.clone()
    k2[1, 3, 0, 5], k2[2, 70, 1, 0], v2[1, 64, 1, 9] = float("nan"), float("-inf"), float("inf")
    c.append(0, k2, v2)
    assert c.status() == 7
    k2[1, 3, 0, 5], k2[2, 70, 1, 0], v2[1, 64, 1, 9] = 0, 0, 0
    d = binding.BlockCache(B, 1, 2, 2, cap)
    d.append(0, k2, v2)
    lens = ints([100] * 4)
    assert all(torch.equal(a, b) for a, b in zip(c.read(0, lens, cap), d.read(0, lens, cap))) and d.status() == 0


# ---- attention -----------------------------------------------------------------
def check_attention(c, ref, q, lens, got, weights=None, base=None):
    out, lse = got
    assert torch.isfinite(out).all()
    for b, L in enumerate(lens):
        want, wl, ww, mag, low, big = U.attention(f64(q[b]), ref.values("k", b, L), ref.values("v", b, L))
        off = 2.0 ** -20 * big
        err = np.abs(f64(out[b]) - want)
        assert np.all(err <= 2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 2 * off) * mag + 2.0 ** -25 * low + 1e-5), b
        seen = np.isfinite(wl)
        assert same(np.isfinite(f64(lse[b])), seen) and np.all(np.isneginf(f64(lse[b])[~seen]))
        assert np.all(np.abs(f64(lse[b])[seen] - wl[seen]) <= 1e-5 + 2.0 ** -22 * np.abs(wl[seen]) + off)
        assert np.all(f64(out[b])[np.abs(want).max(-1) == 0] == 0)
        if weights is not None:
            extra = f64(weights[b]) - f64(base[b])
            assert np.all(np.abs(extra[:, :L] - ww) <= (2 * off + 2.0 ** -21 + 2.0 ** -22 * np.abs(wl[seen]).max(initial=0)) * ww
                          + 2.0 ** -23 * f64(base[b])[:, :L] + 1e-30)
            assert not extra[:, L:].any()
    assert c.status() == 0, c.last_error()


SHAPES = [   # Hq, Hkv, n_q, lengths
    (1, 1, 1, [1]), (8, 2, 1, [2000]), (7, 1, 1, [0, 1, 5, 63, 64, 65, 96, 97, 127, 128, 129]),
    (28, 4, 1, [1000, 3, 640]), (32, 8, 1, [4097, 64, 0]), (16, 2, 2, [1, 2, 64, 66, 500]), (12, 4, 3, [130, 2, 67]),
    (5, 5, 5, [4, 5, 6, 70, 700]), (28, 4, 8, [1100, 7, 64]), (64, 8, 8, [300, 65, 2]), (6, 1, 4, [3000]),
    (32, 8, 5, [8191])]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("Hq,Hkv,n_q,lens", SHAPES)
def test_attention(fmt, Hq, Hkv, n_q, lens):
    B = len(lens)
    c, ref = filled(B, Hq, Hkv, max(lens) + 1, fmt, lens, score_queries=n_q)
    q = rand(9, B, n_q, Hq, D)
    w = torch.rand(B, Hkv, c.capacity, generator=torch.Generator().manual_seed(1)).cuda()
    base = w.clone()
    got = c.attend(0, q.cuda(), ints(lens), weights=w)
    check_attention(c, ref, q, lens, got, w, base)
    bare = c.attend(0, q.cuda(), ints(lens))   # the same bits without weights, and again
    assert all(torch.equal(a, b) for a, b in zip(got, bare))
    w2 = base.clone()
    c.attend(0, q.cuda(), ints(lens), weights=w2)
    assert torch.equal(w, w2)
    w3 = torch.full_like(w, 5.0)
    c.attend(0, q.cuda(), ints(lens), weights=w3, accumulate=False)
    for b, L in enumerate(lens):
        assert torch.all(w3[b, :, L:] == 5.0)
        assert torch.allclose(w3[b, :, :L] + base[b, :, :L], w[b, :, :L], rtol=2.0 ** -22, atol=0)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("scale", [2.0 ** -70, 30.0, 2.0 ** 40])
def test_attention_of_other_magnitudes(fmt, scale):
    """Keys of any magnitude (the query's is the reciprocal where logits would pass fp32), peaked rows."""
    lens = [333]
    c, ref = filled(1, 8, 2, 400, fmt, lens, scale=scale)
    q = rand(9, 1, 1, 8, D, scale=1.0 if scale == 30.0 else 3.0 / scale)
    check_attention(c, ref, q, lens, c.attend(0, q.cuda(), ints(lens)))


@pytest.mark.parametrize("fmt", FORMATS)
def test_attention_reads_values_of_unlike_scales(fmt):
    """A block of tiny values that holds nearly all of the mass, beside one of huge values that holds little."""
    n = 4 * T + 9
    c = binding.BlockCache(1, 1, 4, 1, n, fmt)
    k, v = rand(0, 1, n, 1, D, scale=0.02), rand(1, 1, n, 1, D)
    q = rand(2, 1, 1, 4, D)
    k[:, T:2 * T] = (q[:, :, :1].float() * 2).bfloat16()
    v[:, T:2 * T] *= 2.0 ** -12
    v[:, 3 * T:] = (v[:, 3 * T:].float() * 2.0 ** 10).bfloat16()
    ref = U.Cache(1, 1, c.capacity, fmt)
    c.append(0, k.cuda(), v.cuda())
    ref.append(k, v, [0], [n])
    check_attention(c, ref, q, [n], c.attend(0, q.cuda(), ints([n])))


def test_rows_behind_a_length_take_no_part():
    """What the cache held behind kv_len (longer before, now set back) changes no bit."""
    k, v = rand(0, 2, 400, 2, D).cuda(), rand(1, 2, 400, 2, D).cuda()
    c, d = (binding.BlockCache(2, 1, 8, 2, 400, score_queries=2) for _ in range(2))
    c.append(0, k, v)
    c.append(0, k[:, 64:150].contiguous(), v[:, 64:150].contiguous(), start=ints([64, 64]), n_new=ints([86, 37]))
    d.append(0, k, v, n_new=ints([150, 101]))
    q = rand(3, 2, 2, 8, D).cuda()
    w, x = torch.zeros(2, 2, 448, device="cuda"), torch.zeros(2, 2, 448, device="cuda")
    a, b = c.attend(0, q, ints([150, 101]), weights=w), d.attend(0, q, ints([150, 101]), weights=x)
    assert all(torch.equal(s, t) for s, t in zip(a, b)) and torch.equal(w, x)


# ---- eviction ------------------------------------------------------------------
EVICT = [   # Hkv, lengths, keep, recent
    (1, [130], 64, 0), (2, [64, 63, 0, 65, 128, 191, 1000], 64, 64), (4, [2047], 512, 64), (2, [5000, 700], 1024, 100),
    (1, [20000], 1088, 1), (3, [640, 641], 640, 3), (8, [900, 333], 256, 256)]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("Hkv,lens,keep,recent", EVICT)
@pytest.mark.parametrize("ties", [False, True])
@pytest.mark.parametrize("place", ["into", "in place"])
def test_eviction(fmt, Hkv, lens, keep, recent, ties, place):
    B = len(lens)
    c, ref = filled(B, Hkv, Hkv, max(max(lens), keep + 64), fmt, lens)
    g = torch.Generator().manual_seed(3)
    w = torch.rand(B, Hkv, c.capacity, generator=g).pow(8) * 4
    if ties:
        w = (w * 3).round() / 3
        w[..., ::7] = float("nan")
        w[..., 1::11] = -0.0
        w[..., 2::13] = -1.5
        w[..., 3::17] = float("inf")
        w[..., 4::19] = float("-inf")
    wc = w.cuda()
    if place == "into":
        to = binding.BlockCache(B, 2, Hkv, Hkv, keep + 64, fmt)
        w_out = torch.full((B, Hkv, to.capacity), 9.0, device="cuda")
        new_len, kept = c.evict(0, ints(lens), keep, recent, wc, into=to, into_layer=1, weights_out=w_out)
        layer = 1
    else:
        to, w_out, layer = c, wc, 0
        new_len, kept = c.evict(0, ints(lens), keep, recent, wc)
    n = [min(L // T * T, keep) + L % T for L in lens]
    assert new_len.tolist() == n
    k, v = to.read(layer, new_len, max(max(n), 1))
    for b, L in enumerate(lens):
        cl = L // T * T
        for h in range(Hkv):
            at = U.select(w[b, h].numpy(), cl, keep, recent)
            m = len(at)
            got = kept[b, h].cpu().numpy()
            assert same(got[:m], at) and np.all(got[m:] == -1), (b, h)
            moved = torch.cat([w[b, h][at], w[b, h, cl:L]])
            assert torch.equal(w_out[b, h, :n[b]].cpu().nan_to_num(1e9), moved.nan_to_num(1e9))
            rest = torch.full_like(w_out[b, h, n[b]:], 9.0) if place == "into" else wc.new_tensor(w[b, h, n[b]:].numpy())
            assert torch.equal(w_out[b, h, n[b]:].nan_to_num(1e9), rest.nan_to_num(1e9))
            for x, t in (("k", k), ("v", v)):
                vals = ref.values(x, b, L)[h]
                want = vals[at]
                if place == "into" or cl > keep:
                    want = U.held(want, fmt)
                want = torch.from_numpy(np.concatenate([want, vals[cl:]])).bfloat16()
                assert torch.equal(t[b, :n[b], h].cpu(), want), (b, h, x)
    assert c.status() == 0 and to.status() == 0
    # the cache goes on: the next tokens fill the open block, in its new place
    more_k, more_v = rand(20, B, 64, Hkv, D), rand(21, B, 64, Hkv, D)
    room = to.capacity - max(n)
    m = min(room, 64)
    if m:
        before = to.read(layer, new_len, max(n) + m)
        to.append(layer, more_k[:, :m].contiguous().cuda(), more_v[:, :m].contiguous().cuda(), start=new_len)
        after = to.read(layer, new_len + m, max(n) + m)
        for b in range(B):
            s, e = n[b] // T * T, (n[b] + m) // T * T
            for x, (p, a), new in (("k", (before[0], after[0]), more_k), ("v", (before[1], after[1]), more_v)):
                rows = torch.cat([p[b, s:n[b]].cpu(), new[b, :m]])
                if e > s:
                    full = torch.from_numpy(U.held(rows[:e - s].float().numpy().transpose(1, 0, 2), fmt)).bfloat16()
                    rows[:e - s] = full.transpose(0, 1)
                assert torch.equal(a[b, s:n[b] + m].cpu(), rows) and torch.equal(a[b, :s], p[b, :s])


@pytest.mark.parametrize("fmt", FORMATS)
def test_attention_keeps_what_a_sink_outweighs(fmt):
    """One token outweighs each of 60,000 others by e^16 or e^17 (2^-24.5); together they have 0.3 to 0.7 % of the mass, and
    values 512 times the one's, so that half of the output or more is theirs. Tolerance: half a step of the output, of
    each probability 2^-12 (2^-40 of the largest below 2^-29 of it)."""
    n = 60000
    c = binding.BlockCache(1, 1, 2, 1, n, fmt)
    k, v = torch.zeros(1, n, 1, D), torch.zeros(1, n, 1, D)
    k[:, :, :, 0] = 1.0
    k[:, 64 * 7, :, 0] = 2.0
    v[:, :, :, :64] = 512.0
    v[:, 64 * 7:64 * 8, :, :64] = 1.0
    k[:, 64 * 7 + 1:64 * 8, :, 0] = 1.0
    k, v = k.bfloat16(), v.bfloat16()
    q = torch.zeros(1, 1, 2, D)
    q[..., 0] = torch.tensor([17.0, 16.0]) * D ** 0.5
    q = q.bfloat16()
    ref = U.Cache(1, 1, c.capacity, fmt)
    c.append(0, k.cuda(), v.cuda())
    ref.append(k, v, [0], [n])
    out, _ = c.attend(0, q.cuda(), ints([n]))
    want, _, _, mag, low, big = U.attention(f64(q[0]), ref.values("k", 0, n), ref.values("v", 0, n))
    assert np.all(want[0, :, :64] > 1.5)   # the others' part is as large as the sink's at least
    off = 2.0 ** -20 * big
    err = np.abs(f64(out[0]) - want)
    assert np.all(err <= 2.0 ** -8 * np.abs(want) + (2.0 ** -12 + 2 * off) * mag + 2.0 ** -40 * low + 1e-6)
