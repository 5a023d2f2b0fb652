"""The operators of the cache in 8 bits, as a user's program calls them.

A layer's keys and values are held as 8-bit codes (int8 or e4m3) with an fp32
scale for each block of 64 tokens, KV head and tensor; the tokens of a block
that is not full yet stay bf16. Three paths:

* append: tokens go into the cache (a decode step, a chunk, a whole prompt);
  the rows of the blocks that they touch are read back;
* attend: attention of the last n_q positions over the cache, and (optional)
  the weight that each token receives, summed over the queries and averaged
  over the query heads of its KV head;
* evict: each (sequence, KV head) keeps its latest tokens and those with the
  largest accumulated weights, in order, in new blocks of another cache, which
  are read back.

`run` computes them in elementary torch operations (fp32, rounded once) where
`own` is false, and through the library where it is true.
"""
import math

import torch

own = False

D = 128          # head size
T = 64           # tokens of a block
TOP = {"int8": 127.0, "e4m3": 448.0}


def _case(name, op, fmt, B, Hq, Hkv, n, n_q=1, ragged=0, start=0, keep=0, recent=0, weights=False):
    c = dict(op=op, fmt=fmt, B=B, Hq=Hq, Hkv=Hkv, n=n, n_q=n_q, ragged=ragged, start=start, keep=keep, recent=recent,
             weights=weights)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one token of each of 16 conversations at unlike places of their blocks, one of which fills
        _case("append step b16", "append", "int8", 16, 28, 4, 1, start=16384 - 1, ragged=333),
        # two chunks of four prompts, the first of which ends inside a block, the second of odd length
        _case("append chunk 777", "append", "e4m3", 4, 32, 8, 777, start=5003, ragged=101),
        # a 32K prompt stored in one go
        _case("append prompt 32k", "append", "int8", 1, 32, 8, 32768),
        # a small model's decode step
        _case("attend step tiny", "attend", "int8", 1, 8, 2, 2000),
        # a decode step of 8 conversations of about 32K that accumulates the tokens' weights
        _case("attend step b8 32k weights", "attend", "int8", 8, 32, 8, 32768, ragged=501, weights=True),
        # a decode step of 16 conversations of unlike lengths, 7 query heads to a KV head
        _case("attend step b16 ragged", "attend", "e4m3", 16, 28, 4, 16384, ragged=777),
        # five drafted tokens of four conversations checked at once
        _case("attend draft 5", "attend", "e4m3", 4, 32, 8, 8191, n_q=5, ragged=13, weights=True),
        # a decode step at 128K: the largest
        _case("attend step b4 128k", "attend", "int8", 4, 32, 8, 131072, ragged=64),
        # a small model's cache cut to a quarter
        _case("evict tiny", "evict", "int8", 1, 8, 2, 2047, keep=512, recent=64),
        # 16 conversations of unlike lengths cut to 1K, some below it already
        _case("evict b16 ragged", "evict", "e4m3", 16, 28, 4, 4000, ragged=217, keep=1024, recent=100),
        # four prompts of 32K cut to a fifth, as after their prefill
        _case("evict b4 32k", "evict", "int8", 4, 32, 8, 32768, ragged=11, keep=6528, recent=512),
        # a context of 128K cut to a tenth
        _case("evict 128k", "evict", "e4m3", 1, 32, 8, 131000, keep=13056, recent=1000),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """A case of the ranges above, whose work does not pass the largest listed one's."""
    op, fmt = rng.choice(["append", "attend", "attend", "evict"]), rng.choice(["int8", "e4m3"])
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 4, 7, 8])
    if op == "append":
        B = _log(rng, 1, 16)
        n = rng.choice([1, _log(rng, 2, 700), _log(rng, 700, 32768 // B)])
        return _case("", op, fmt, B, Hq, Hkv, n, start=rng.choice([0, rng.randrange(20000)]), ragged=rng.randrange(999))
    n = _log(rng, 100, 131072)
    B = _log(rng, 1, max(1, min(32, 300000 // n)))
    ragged = rng.randrange(0, max(1, n // B))
    if op == "attend":
        return _case("", op, fmt, B, Hq, Hkv, n, n_q=rng.choice([1, 1, 2, 5, 8]), ragged=ragged,
                     weights=rng.random() < 0.5)
    keep = T * _log(rng, 1, max(1, min(n, 32768) // T))
    return _case("", op, fmt, B, Hq, Hkv, n, ragged=ragged, keep=keep, recent=rng.randrange(keep + 1))


def _lengths(case):
    return [max(1, case["n"] - b * case["ragged"]) for b in range(case["B"])]


def _starts(case):
    return [max(0, case["start"] - b * case["ragged"]) for b in range(case["B"])]


def _quantised(x, fmt):
    """fp32 [..., 64, 128] blocks as the codes (fp32 values) and the scales [..., 1, 1] that hold them."""
    s = x.abs().amax((-2, -1), keepdim=True)
    s = s / s.new_full((), TOP[fmt])   # a division: by a plain number it would be a product with the reciprocal
    y = torch.where(s > 0, x / s, 0.0)
    return (y.round() if fmt == "int8" else y.to(torch.float8_e4m3fn).float()), s


def _held(x, fmt):
    """fp32 values that a cache holds for the whole blocks x [..., n, 128] (n a multiple of 64)."""
    code, s = _quantised(x.unflatten(-2, (-1, T)), fmt)
    return (code * s).flatten(-3, -2)


def prepare(case, seed):
    B, Hq, Hkv, n, fmt = (case[k] for k in ("B", "Hq", "Hkv", "n", "fmt"))
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    def ints(x):
        return torch.tensor(x, dtype=torch.int32).cuda()

    outlier = torch.where(torch.rand(Hkv, D, generator=g, device="cuda") < 0.01, 4.0, 1.0)   # channels of the keys

    def tokens(m):
        return (normal(B, m, Hkv, D) * outlier).bfloat16(), normal(B, m, Hkv, D).bfloat16()

    s = dict(case)
    if case["op"] == "append":
        s["k"], s["v"] = tokens(n)
        s["k_open"], s["v_open"] = tokens(T)   # the rows that the open blocks hold already
        start = _starts(case)
        s["start"], s["first"] = ints(start), ints([a // T * T for a in start])
        s["off"] = s["start"] - s["first"]
        s["open_first"] = n > 1 and any(a % T for a in start)
        s["len"] = s["start"] + n
        s["rows"] = max(a % T for a in start) + n
        s["k_out"], s["v_out"] = (torch.zeros(B, s["rows"], Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in "kv")
        if own:
            from tiered_kv_cache_decode_gb300 import binding
            s["cache"] = binding.BlockCache(B, 1, Hq, Hkv, max(start) + n, fmt)
            s["cache"].append(0, s["k_open"], s["v_open"], start=s["first"], n_new=s["off"])
        return s
    lens = _lengths(case)
    s["kv_len"] = ints(lens)
    s["closed"] = s["kv_len"] // T * T
    pad = -(-n // T) * T
    k, v = tokens(pad)
    if own:
        from tiered_kv_cache_decode_gb300 import binding
        s["cache"] = binding.BlockCache(B, 1, Hq, Hkv, pad, fmt, score_queries=case["n_q"] if case["weights"] else 0)
        s["cache"].append(0, k, v, n_new=s["kv_len"])
    else:   # the same cache: codes and scales, and the rows of the open blocks
        for x, name in ((k, "k"), (v, "v")):
            x = x.transpose(1, 2)
            code, scale = _quantised(x.float().unflatten(2, (-1, T)), fmt)
            s[name + "_code"] = code.to(torch.int8 if fmt == "int8" else torch.float8_e4m3fn)
            s[name + "_scale"] = scale
            at = (s["closed"].clamp_max(pad - T)[:, None] + torch.arange(T, device="cuda")).long()
            s[name + "_open"] = x.gather(2, at[:, None, :, None].expand(B, Hkv, T, D))
    del k, v
    if case["op"] == "attend":
        s["q"] = normal(B, case["n_q"], Hq, D).bfloat16()
        # the caller's buffers; what lies past a sequence's tokens is left as it was
        s["weights_out"] = torch.zeros(B, Hkv, pad, device="cuda") if case["weights"] else None
        return s
    # accumulated weights: a few tokens hold most of the mass
    s["weight"] = torch.rand(B, Hkv, pad, generator=g, device="cuda").pow(8) * 4
    s["room"] = case["keep"] + T
    s["weights_out"] = torch.zeros(B, Hkv, s["room"], device="cuda")
    s["kept"] = torch.zeros(B, Hkv, case["keep"], dtype=torch.int32, device="cuda")
    s["k_out"], s["v_out"] = (torch.zeros(B, s["room"], Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    if own:
        s["into"] = binding.BlockCache(B, 1, Hq, Hkv, s["room"], fmt)
    return s


def _plain_append(s):
    B, rows, off = s["B"], s["rows"], s["off"][:, None]
    pad = -(-rows // T) * T
    r = torch.arange(pad, device="cuda")
    end = off + s["n"]
    new = (r - off).clamp(0, s["n"] - 1).long()
    for name in "kv":
        shape = (B, pad, s["Hkv"], D)
        x = s[name].gather(1, new[:, :, None, None].expand(shape))
        x[:, :T] = torch.where((r[:T] < off)[:, :, None, None], s[name + "_open"], x[:, :T])
        held = _held(x.transpose(1, 2).float(), s["fmt"]).transpose(1, 2).bfloat16()
        held = torch.where((r < end // T * T)[:, :, None, None], held, x)[:, :rows]
        s[name + "_out"] = torch.where((r < end)[:, :rows, None, None], held, s[name + "_out"])
    return s["k_out"], s["v_out"]


def _values(s, name):
    """fp32 [B][Hkv][pad][128]: what the cache holds, the open blocks' rows in their places."""
    x = (s[name + "_code"].float() * s[name + "_scale"]).flatten(2, 3)
    at = (s["closed"].clamp_max(x.shape[2] - T)[:, None] + torch.arange(T, device="cuda")).long()
    at = at[:, None, :, None].expand_as(s[name + "_open"])
    opened = (at >= s["closed"][:, None, None, None])
    return x.scatter_(2, at, torch.where(opened, s[name + "_open"].float(), x.gather(2, at)))


def _plain_attend(s):
    B, Hkv, n_q, G = s["B"], s["Hkv"], s["n_q"], s["Hq"] // s["Hkv"]
    k, v = _values(s, "k"), _values(s, "v")
    pad = k.shape[2]
    q = s["q"].float().view(B, n_q, Hkv, G, D).transpose(1, 2).reshape(B, Hkv, n_q * G, D)
    x = torch.matmul(q, k.transpose(2, 3)).mul_(D ** -0.5).view(B, Hkv, n_q, G, pad)
    j = torch.arange(pad, device="cuda")
    p = s["kv_len"][:, None] - n_q + torch.arange(n_q, device="cuda")
    x.masked_fill_((j > p[:, :, None])[:, None, :, None], -math.inf)
    top = x.amax(-1, keepdim=True).clamp_min(-3e38)
    x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    lse = (top + total.log())[..., 0].permute(0, 1, 3, 2).reshape(B, s["Hq"], n_q)
    x /= total.clamp_min(1e-38)
    out = torch.matmul(x.view(B, Hkv, n_q * G, pad), v).view(B, Hkv, n_q, G, D).transpose(1, 2)
    out = out.reshape(B, n_q, s["Hq"], D).bfloat16()
    if s["weights_out"] is None:
        return out, lse
    w = x.sum((2, 3)) / G
    s["weights_out"] = torch.where((j < s["kv_len"][:, None])[:, None], w, s["weights_out"])
    return out, lse, s["weights_out"]


def _plain_evict(s):
    B, Hkv, keep, room = s["B"], s["Hkv"], s["keep"], s["room"]
    c, pad = s["closed"][:, None, None], s["weight"].shape[2]
    j = torch.arange(pad, device="cuda")
    rank = torch.where(j >= c - min(s["recent"], keep), math.inf, s["weight"])
    rank = torch.where(j < c, rank, -math.inf)
    if pad < keep:
        rank = torch.nn.functional.pad(rank, (0, keep - pad), value=-math.inf)
    kept = rank.sort(dim=-1, descending=True, stable=True).indices[..., :keep].sort(-1).values
    stays = kept < c
    s["kept"] = torch.where(stays, kept, -1).int()
    closed = c.clamp_max(keep)
    new_len = (closed + s["kv_len"][:, None, None] - c)[:, 0, 0].int()
    # the kept tokens, then the open block's
    i = torch.arange(room, device="cuda")
    source = torch.nn.functional.pad(kept, (0, T))
    source = torch.where(i < closed, source, i - closed + c).clamp(0, pad - 1)
    used = i < new_len[:, None, None]
    s["weights_out"] = torch.where(used, s["weight"].gather(2, source), s["weights_out"])
    for name in "kv":
        x = _values(s, name).gather(2, source[..., None].expand(B, Hkv, room, D))
        held = torch.where((i < closed)[..., None], _held(x, s["fmt"]), x).transpose(1, 2).bfloat16()
        s[name + "_out"] = torch.where(used[:, 0, :, None, None], held, s[name + "_out"])
    return s["kept"], new_len, s["weights_out"], s["k_out"], s["v_out"]


def run(s):
    if not own:
        return {"append": _plain_append, "attend": _plain_attend, "evict": _plain_evict}[s["op"]](s)
    c = s["cache"]
    if s["op"] == "append":
        if s["open_first"]:   # the chunk before, which ends inside a block
            c.append(0, s["k_open"], s["v_open"], start=s["first"], n_new=s["off"])
        c.append(0, s["k"], s["v"], start=s["start"])
        return c.read(0, s["len"], s["rows"], first=s["first"], k_out=s["k_out"], v_out=s["v_out"])
    if s["op"] == "attend":
        out, lse = c.attend(0, s["q"], s["kv_len"], weights=s["weights_out"], accumulate=False)
        return (out, lse) if s["weights_out"] is None else (out, lse, s["weights_out"])
    new_len, kept = c.evict(0, s["kv_len"], s["keep"], s["recent"], s["weight"], into=s["into"], kept=s["kept"],
                            weights_out=s["weights_out"])
    k, v = s["into"].read(0, new_len, s["room"], k_out=s["k_out"], v_out=s["v_out"])
    return kept, new_len, s["weights_out"], k, v


def work(case):
    B, Hq, Hkv, n, n_q = (case[k] for k in ("B", "Hq", "Hkv", "n", "n_q"))
    row = 2 * D * Hkv   # codes of a token's keys and values
    if case["op"] == "append":
        back = sum(a % T + n for a in _starts(case))
        return {"bytes": B * n * row * 3 + back * row * 3, "flops": B * n * row * 2 + back * row}
    lens = _lengths(case)
    if case["op"] == "attend":
        tokens = sum(lens)
        rows = B * n_q * Hq
        return {"bytes": tokens * (row + (4 * Hkv if case["weights"] else 0)) + rows * (D * 4 + 4),
                "flops": 4 * D * Hq * n_q * tokens}
    kept = sum(min(a // T * T, case["keep"]) for a in lens)
    opened = sum(a % T for a in lens)
    return {"bytes": sum(lens) * Hkv * 4 + kept * (row * 5 + 8 * Hkv) + opened * row * 8, "flops": kept * row * 4}


def _exact_values(x, closed, fmt):
    """64-bit values that the cache holds for one head's tokens x [n][128]: the scale and the quotient are fp32 by
    definition (a quotient of two fp32 numbers rounded from 64 bits is the one rounded once)."""
    y = x.double().clone()
    for j in range(0, closed, 4096):
        z = y[j:min(j + 4096, closed)].view(-1, T * D)
        s = (z.abs().max(1, keepdim=True).values / TOP[fmt]).float().double()
        r = torch.where(s > 0, z / s, 0.0).float()
        code = torch.round(r).double() if fmt == "int8" else r.to(torch.float8_e4m3fn).double()
        y[j:min(j + 4096, closed)] = (code * s).view(-1, D)
    return y


def exact(case, seed):
    """The definitions in 64 bits, one (sequence, KV head) at a time."""
    B, Hq, Hkv, n, n_q, fmt = (case[k] for k in ("B", "Hq", "Hkv", "n", "n_q", "fmt"))
    G = Hq // Hkv
    s = prepare(case, seed)
    if case["op"] == "append":
        res = []
        for name in "kv":
            res.append(s[name + "_out"].double())
            for b, a in enumerate(_starts(case)):
                x = torch.cat([s[name + "_open"][b, :a % T], s[name][b]])
                for h in range(Hkv):
                    res[-1][b, :len(x), h] = _exact_values(x[:, h], len(x) // T * T, fmt)
        return tuple(res)

    def head(name, b, h, length):
        full = length // T * T
        code, scale = (s[name + x][b, h] for x in ("_code", "_scale"))
        x = (code.double() * scale.double()).flatten(0, 1)[:full]
        return torch.cat([x, s[name + "_open"][b, h, :length - full].double()])

    lens = _lengths(case)
    if case["op"] == "attend":
        out = torch.zeros(B, n_q, Hq, D, dtype=torch.float64, device="cuda")
        lse = torch.full((B, Hq, n_q), -math.inf, dtype=torch.float64, device="cuda")
        weights = None if s["weights_out"] is None else s["weights_out"].double()
        for b, L in enumerate(lens):
            for h in range(Hkv):
                k, v = head("k", b, h, L), head("v", b, h, L)
                for i in range(max(0, n_q - L), n_q):
                    e = L - n_q + i + 1
                    x = s["q"][b, i, h * G:h * G + G].double() @ k[:e].T / math.sqrt(D)
                    lse[b, h * G:h * G + G, i] = x.logsumexp(1)
                    p = x.softmax(1)
                    out[b, i, h * G:h * G + G] = p @ v[:e]
                    if weights is not None:
                        weights[b, h, :e] += p.mean(0)
        return (out, lse) if weights is None else (out, lse, weights)
    keep, recent = case["keep"], min(case["recent"], case["keep"])
    k_out, v_out, weights = s["k_out"].double(), s["v_out"].double(), s["weights_out"].double()
    kept = torch.full((B, Hkv, keep), -1, dtype=torch.int32, device="cuda")
    for b, L in enumerate(lens):
        c = L // T * T
        for h in range(Hkv):
            w = s["weight"][b, h]
            at = torch.arange(c, device="cuda")
            if c > keep:
                first = torch.argsort(-w[:c - recent].double(), stable=True)[:keep - recent]
                at = torch.cat([torch.sort(first).values, at[c - recent:]])
            m = len(at)
            kept[b, h, :m] = at.int()
            weights[b, h, :m + L - c] = torch.cat([w[:c][at], w[c:L]]).double()
            for name, res in (("k", k_out), ("v", v_out)):
                x = head(name, b, h, L)
                held = _exact_values(torch.cat([x[:c][at].float(), x[c:].float()]), m, fmt)
                res[b, :m + L - c, h] = held
    new_len = torch.tensor([min(a // T * T, keep) + a % T for a in lens], dtype=torch.int32, device="cuda")
    return kept, new_len, weights, k_out, v_out
